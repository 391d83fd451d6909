// What the prefill kernels share: parameters, work items, and the tiled copy of the keys that they read.
#pragma once
#include "common.cuh"
#include "kv4.cuh"
#include "ptx.cuh"

namespace cai {

constexpr int kRows = 128;                 // query rows per q-tile (MMA M)
constexpr int kKeys = 128;                 // keys per tile (MMA N of S, K of PV)
constexpr int kTileBytes = kKeys * kHeadDim * 2;  // 32 KB of 16-bit values
constexpr int kItemSlots = 4;              // items handed from one warp to the other roles

struct PrefillParams {
  const uint8_t* pages;
  int32_t num_pages, page_size, max_pages;
  const int32_t* table;
  const int32_t* prefix_len;
  const uint16_t* q;      // bf16 [rows of new tokens][Hq][128], sequence b's rows from q_row0(b)
  const int32_t* q_off;   // [B + 1] packed new-token offsets, or null: sequence b has n_new rows at b * n_new
  int32_t batch, n_new, total_new, num_heads, log2_heads, window, kt_rows, qtiles;  // n_new: the most per sequence; qtiles per sequence
  float scale_log2;
  // Work items: items [0, full_items) are whole q-tiles; the q-tiles after them (the
  // last, partial wave of a persistent grid) are cut into `pieces` key ranges each,
  // item full_items + t being piece t % pieces of q-tile full_items + t / pieces.  A
  // piece writes its normalised partial output and log2-sum-exp to piece_o / piece_lse
  // ([t][128 rows][128] and [t][128]); combine_pieces_kernel merges them.
  int32_t full_items, pieces, num_items;
  uint64_t wait_ns;  // limit of every bounded wait inside the kernel
  int32_t drop_stage;  // fault injection: K tile each CTA skips (-1: none)
  int32_t skip_single;  // see PrefillLaunch
  // Varlen calls: the items are only the q-tiles that hold rows, sequence by sequence,
  // through a list of their dense numbers that every CTA builds at its start (the dense
  // numbering, qtiles slots per sequence for the longest one, would make the grid walk
  // the empty slots of every short or one-token sequence); past kMaxCompactItems real
  // q-tiles, the dense numbering.  No pieces then.  (With the 4-bit cache one warp walks the sequences instead.)
  int32_t compact;
  float* piece_o;
  float* piece_lse;
  uint16_t* kb;  // scratch bf16 [B][KT][128]
  uint16_t* vh;  // scratch fp16 [B][KT][128]: V codes times the V scale
  float* ks;     // scratch [B][KT]: K scale * softmax scale * log2(e)
  float* out;
  float* lse_out;
  int32_t* err;
  // The 4-bit cache; elsewhere one K/V head and q_heads = num_heads.
  int32_t num_kv_heads, q_heads;
  const uint8_t* pages4[kMaxKvHeads];
  int32_t num_pages4[kMaxKvHeads];
  uint16_t* out16;
};

// New tokens of sequence b: rows [r0, r0 + n) of q / out, or n = -1 when its offsets
// are out of order or outside [0, total_new] (nothing of it is read or written).
struct SeqRows {
  int64_t r0;
  int n;
};

__device__ __forceinline__ SeqRows seq_rows(const PrefillParams& p, int b) {
  SeqRows s;
  if (!p.q_off) {
    s.r0 = (int64_t)b * p.n_new;
    s.n = p.n_new;
    return s;
  }
  const int32_t a = p.q_off[b], e = p.q_off[b + 1];
  s.r0 = a;
  s.n = (a >= 0 && a <= e && e <= p.total_new && e - a <= p.n_new) ? e - a : -1;
  if (p.skip_single && s.n == 1) s.n = 0;  // decoded by the decode kernel in the same call
  return s;
}

__device__ __forceinline__ bool seq_ok(const PrefillParams& p, int32_t p0, int n) {
  return n >= 0 && p0 >= 0 && (int64_t)p0 + n <= (int64_t)p.max_pages * p.page_size;
}

// One work item: a q-tile (128 consecutive (token, head) rows) of one
// sequence.  ok = false: no MMA work; the softmax groups then write zeros to the
// item's rows below `rows` (an invalid sequence) or nothing (rows beyond the chunk).
struct PItem {
  int b, row0, kt0, nkt;
  int kvh;        // K/V head (4-bit cache)
  int p0;         // the sequence's prefix length
  int64_t qrow0;  // first packed new-token row of the sequence
  int rows;       // (token, head) rows of the sequence, 0 if its offsets are invalid
  bool ok;
  int piece;      // -1: the whole key range; otherwise the piece's slot in piece_o / piece_lse
};

// q-tiles holding rows of sequence b (0 when it has no rows in this call), for each of its K/V heads.
__device__ __forceinline__ int seq_qtiles(const PrefillParams& p, int b) {
  const SeqRows sr = seq_rows(p, b);
  return sr.n > 0 ? (int)(((int64_t)sr.n * p.num_heads + kRows - 1) / kRows) : 0;
}

// The work split of a persistent grid over `total` q-tiles: items [0, full) are whole
// q-tiles; the q-tiles of a partial last wave are cut into `pieces` key ranges so that
// wave ends sooner (with r q-tiles left over, pieces = grid / r, at most 4), item
// full + t being piece t % pieces of q-tile full + t / pieces; num items in all.  The
// host applies it to a chunk call's q-tiles.
struct WorkSplit {
  int full, pieces, num;
};
__host__ __device__ inline WorkSplit work_split(int64_t total, int grid) {
  const int64_t rem = grid > 0 ? total % grid : 0;
  int pieces = rem > 0 ? (int)(grid / rem) : 1;
  if (pieces > 4) pieces = 4;
  if (pieces < 2) pieces = 1;
  WorkSplit w;
  w.pieces = pieces;
  w.full = (int)(pieces > 1 ? total - rem : total);
  w.num = (int)(w.full + (pieces > 1 ? rem * pieces : 0));
  return w;
}

// (token, head) row `row` of an item's sequence, as a row of q, out and lse_out.
template <bool kFour>
__device__ __forceinline__ int64_t q_row(const PrefillParams& p, const PItem& it, int64_t row) {
  return kFour ? (it.qrow0 + (row >> p.log2_heads)) * p.q_heads + it.kvh * p.num_heads + (row & (p.num_heads - 1))
               : it.qrow0 * p.num_heads + row;
}

// list: a varlen call's q-tile numbers, or null.
template <bool kFour>
__device__ __forceinline__ PItem prefill_item(const PrefillParams& p, int idx, const int32_t* list,
                                              const WorkSplit& ws) {
  PItem it;
  int qti = idx, piece = -1;
  if (idx >= ws.full) {
    const int t = idx - ws.full;
    qti = ws.full + t / ws.pieces;
    piece = t % ws.pieces;
    it.piece = t;
  } else {
    it.piece = -1;
  }
  const int qt = list ? list[qti] : qti;
  it.b = qt / p.qtiles;
  it.row0 = (qt - it.b * p.qtiles) * kRows;
  const int seq = kFour ? it.b / p.num_kv_heads : it.b;
  it.kvh = kFour ? it.b - seq * p.num_kv_heads : 0;
  const int32_t p0 = p.prefix_len[seq];
  it.p0 = p0;
  const SeqRows sr = seq_rows(p, seq);
  it.qrow0 = sr.r0;
  it.rows = sr.n > 0 ? sr.n * p.num_heads : 0;
  it.ok = seq_ok(p, p0, sr.n) && it.row0 < it.rows;
  if (!it.ok) {
    it.kt0 = it.nkt = 0;
    return it;
  }
  const int i0 = it.row0 >> p.log2_heads;
  const int i_last = min((it.row0 + kRows - 1) >> p.log2_heads, sr.n - 1);
  const int kv_hi = p0 + i_last + 1;
  const int kv_lo = p.window > 0 ? max(0, p0 + i0 + 1 - p.window) : 0;
  it.kt0 = kv_lo / kKeys;
  it.nkt = (kv_hi - 1) / kKeys - it.kt0 + 1;
  if (piece >= 0) {  // key tiles [per * piece, per * (piece + 1)) of the q-tile's range
    const int per = (it.nkt + ws.pieces - 1) / ws.pieces;
    const int a = min(it.nkt, per * piece), e = min(it.nkt, per * (piece + 1));
    it.kt0 += a;
    it.nkt = e - a;
  }
  return it;
}

// Attention over the copy of a 4-bit cache (prefill4.cu).
cudaError_t launch_attend4(const PrefillParams& p, int grid, cudaStream_t stream);

}  // namespace cai

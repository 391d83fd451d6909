// What the two decode kernels of the 4-bit cache share: the split of the work into pieces.
#pragma once
#include "common.cuh"
#include "kv4.cuh"
#include "ptx.cuh"

namespace cai {

// One piece of work: keys [start, end) of one sequence and K/V head (end = start: nothing to attend).
struct Piece4 {
  int32_t b, kvh, row;  // row: of q, out and lse_out
  int32_t start, end;
  int32_t slot;         // partial's slot, or -1: the piece is the whole attended range
};
constexpr int kPieces = 32;  // pieces listed at a time
// State of the list, in shared memory.
struct List4 {
  int32_t count, more;
  int32_t unit;           // next (sequence, K/V head) to list (or item, with fixed chunks)
  int64_t pos;            // its first position in the numbering of all tiles
  int64_t begin, end, total;  // this block's range of it, and its length
  int32_t ranges;         // blocks that share it: at most one per position
};

__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t x) {
  return pack_f16x2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}

// Sequence b's row in q / out / lse_out and its attended keys; false: not a row of this launch.
__device__ __forceinline__ bool seq_keys(const Decode4Params& p, int b, int32_t& row, SeqSplits& sp) {
  int32_t L = p.ctx_len[b];
  row = b;
  if (p.q_off) {
    const int32_t a = p.q_off[b], e = p.q_off[b + 1];
    if (!(a >= 0 && e == a + 1 && e <= p.total_rows)) return false;  // a chunk: the prefill kernel's
    row = a;
  }
  if (p.before_new) L = L < 0 || L >= p.max_pages * p.page_size ? -1 : L + 1;
  sp = seq_splits(L, p.window, p.max_pages * p.page_size, p.chunk > 0 ? p.chunk : 1);
  return true;
}

// Tiles of 128 keys that hold sequence b's attended keys (-1: not a row of this launch).  A tile is
// aligned to 128 positions of the sequence.
__device__ __forceinline__ int seq_tiles(const Decode4Params& p, int b) {
  int32_t row;
  SeqSplits sp;
  if (!seq_keys(p, b, row, sp)) return -1;
  return sp.hi > sp.lo ? (sp.hi - 1) / kDecodeTile - sp.lo / kDecodeTile + 1 : 0;
}

// Positions that a (sequence, K/V head) takes in the numbering that is cut into equal parts: its tiles,
// and as many as its start and merge cost.
__device__ __forceinline__ int unit_weight(const Decode4Params& p, int tiles) { return tiles < 0 ? 0 : tiles + p.piece_tiles; }

// x / y, x < 2^63 (32 bits where that is enough: a division of 64 bits takes several times as long).
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  return (x | y) >> 32 ? x / y : (int64_t)((uint32_t)x / (uint32_t)y);
}
// Block c's range is [c W / n, (c + 1) W / n), n <= W; the block whose range holds position x:
__device__ __forceinline__ int block_of(int64_t x, int64_t W, int n) { return (int)quotient((x + 1) * n - 1, W); }

// The whole block: W, this block's range and the unit it starts in.
template <int kThreads>
__device__ __forceinline__ void start_list(const Decode4Params& p, int c, List4& ls, int64_t* scan) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (p.chunk > 0) {
    if (tid == 0) {
      ls.unit = c;
      ls.more = 1;
    }
    __syncthreads();
    return;
  }
  // (Blocks of the same range but different head groups each store this, and later the same final value.)
  if (tid == 0) p.meta[c] = make_int2(-1, -1);
  const int per = (p.batch + kThreads - 1) / (kThreads);
  const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
  int64_t sum = 0;
  for (int b = b0; b < b1; b += 4) {
    int w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) w[u] = seq_tiles(p, min(b + u, b1 - 1));
#pragma unroll
    for (int u = 0; u < 4; ++u) sum += b + u < b1 ? unit_weight(p, w[u]) : 0;
  }
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int64_t before = 0, W = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scan[w];
    W += scan[w];
  }
  W *= p.num_kv_heads;
  const int n = (int)(W < p.ranges ? W : p.ranges);  // every block gets a position
  if (c >= n) {
    if (tid == 0) ls.more = 0;
    __syncthreads();
    return;
  }
  const int64_t begin = quotient(W * c, n), end = quotient(W * (c + 1), n);
  const int64_t mine = (before + incl - sum) * p.num_kv_heads;
  if (begin >= mine && begin < mine + sum * p.num_kv_heads) {  // one thread
    int64_t pos = mine;
    int b = b0;
    for (;; ++b) {
      const int64_t w = (int64_t)unit_weight(p, seq_tiles(p, b)) * p.num_kv_heads;
      if (begin < pos + w) break;
      pos += w;
    }
    const int w = unit_weight(p, seq_tiles(p, b));
    const int kvh = (int)((begin - pos) / w);
    ls.unit = b * p.num_kv_heads + kvh;
    ls.pos = pos + (int64_t)kvh * w;
    ls.begin = begin;
    ls.end = end;
    ls.total = W;
    ls.ranges = n;
    ls.more = 1;
  }
  __syncthreads();
}

// Warp 0: the next pieces of this block, one unit (or item) per lane.
__device__ __forceinline__ void next_pieces(const Decode4Params& p, int c, List4& ls, Piece4* list) {
  const int lane = threadIdx.x & 31;
  Piece4 x = {};
  bool have = false;
  const int units = p.batch * p.num_kv_heads;
  if (p.chunk > 0) {
    const int64_t item = ls.unit + (int64_t)lane * p.ranges;
    const int64_t items = (int64_t)units * p.splits;
    if (item < items) {
      const int split = (int)(item / units), unit = (int)(item - (int64_t)split * units);
      x.b = unit / p.num_kv_heads;
      x.kvh = unit - x.b * p.num_kv_heads;
      SeqSplits sp;
      if (seq_keys(p, x.b, x.row, sp) && (split < sp.nsplit || split == 0)) {
        have = true;
        x.start = sp.lo + split * p.chunk;
        x.end = min(sp.hi, x.start + p.chunk);
        x.slot = sp.nsplit > 1 ? unit * p.splits + split : -1;
        if (sp.nsplit == 0) x.end = x.start;
        if (!sp.valid && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
      }
    }
    __syncwarp();
    if (lane == 0) {
      const int64_t next = ls.unit + 32ll * p.ranges;
      ls.more = next < items;
      ls.unit = (int)next;
    }
  } else {
    const int unit = ls.unit + lane;
    int tiles = -1;
    SeqSplits sp = {};
    if (unit < units) {
      x.b = unit / p.num_kv_heads;
      x.kvh = unit - x.b * p.num_kv_heads;
      if (seq_keys(p, x.b, x.row, sp)) tiles = sp.hi > sp.lo ? (sp.hi - 1) / kDecodeTile - sp.lo / kDecodeTile + 1 : 0;
    }
    const int w = unit_weight(p, tiles);
    int incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int64_t base = ls.pos, begin = ls.begin, end = ls.end, total = ls.total;
    const int64_t pos = base + incl - w;  // the unit's first position
    if (tiles >= 0 && pos < end) {
      const int t0 = (int)(begin > pos ? begin - pos : 0);
      const int t1 = (int)(end - pos < tiles ? end - pos : tiles);
      if (tiles == 0) {
        have = begin <= pos;
        if (!sp.valid && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
      } else if (t0 < t1) {
        have = true;
        const int tile0 = sp.lo / kDecodeTile;
        x.start = max(sp.lo, (tile0 + t0) * kDecodeTile);
        x.end = min(sp.hi, (tile0 + t1) * kDecodeTile);
        x.slot = t0 == 0 && t1 == tiles ? -1 : 2 * c + (t0 == 0 ? 1 : 0);
      }
      if (have && t0 == 0 && pos + tiles > end) p.meta[c] = make_int2(unit, block_of(pos + tiles - 1, total, ls.ranges));
    }
    const int64_t after = base + __shfl_sync(0xffffffffu, incl, 31);
    __syncwarp();
    if (lane == 0) {
      ls.more = after < end && ls.unit + 32 < units;
      ls.unit += 32;
      ls.pos = after;
    }
  }
  const uint32_t m = __ballot_sync(0xffffffffu, have);
  if (have) list[__popc(m & ((1u << lane) - 1u))] = x;
  if (lane == 0) ls.count = __popc(m);
}

// The kernels' launches (decode4.cu: mma.m16n8k16, decode4_tc.cu: tcgen05).
int decode4_tc_heads(int group);   // query heads per block of the tcgen05 kernel (0: the group is not its)
cudaError_t launch_decode4_tc(const Decode4Params& p, cudaStream_t stream);

}  // namespace cai

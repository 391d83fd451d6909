// Shared definitions of the CUDA side of libcai: launch parameter blocks,
// constants and the split plan.
#pragma once
#include <cstdint>
#include <utility>
#include <cuda_runtime.h>

#include "cai.h"

namespace cai {

constexpr int kHeadDim = 128;
constexpr int kMaxSplits = 64;
constexpr int kDecodeTile = 128;       // tokens per decode tile (MMA M of the scores, K of PV)
constexpr int kRawTokens = 64;         // tokens per raw page stage (half a tile)
constexpr int kDecodeMaxHeads = 64;    // query heads per decode call at most (MMA N of the scores)
constexpr int kWorkspaceHeader = 256;  // decode workspace: work-queue counters, kept zero between calls
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Bytes of one page for head_dim 128: P * (2*128 + 8).
__host__ __device__ constexpr int page_bytes(int P) { return P * (2 * kHeadDim + 8); }

struct AppendParams {
  uint8_t* pages;
  int32_t num_pages, page_size, max_pages;
  const float* k_new;
  const float* v_new;
  int32_t batch, n_new;
  const int32_t* table;
  const int32_t* start_pos;
  int32_t* err;
};

// Work split of one decode launch.  The attended span [lo, hi) of every
// sequence is cut into consecutive chunks of `chunk` tokens starting at lo:
// split j covers [lo + j*chunk, min(hi, lo + (j+1)*chunk)).
struct DecodePlan {
  int32_t chunk;       // tokens per split, a multiple of kDecodeTile
  int32_t max_splits;  // upper bound of splits per sequence
};

constexpr int kMaxKvHeads = 8;         // KV heads (pools) one decode call can read

constexpr int kMaxDecodeJobs = 8;  // layers decoded by one launch

// One layer of a decode launch: its query, output and block table, its window and
// split plan, and the pool slots its KV heads read (slot0 + j for KV head j).
struct DecodeJob {
  int32_t slot0;
  int32_t window;
  const int32_t* table;  // [B][max_pages]
  int32_t max_pages;
  const uint16_t* q;     // bf16 bits [B][Hq][128]
  float* out;            // [B][Hq][128]
  float* lse_out;        // [B][Hq] natural log, nullable
  float* ws_o;           // [B][max_splits][Hq][128] partial outputs (normalised), null without splits
  float* ws_lse;         // [B][max_splits][Hq] partial lse, log2 units
  DecodePlan plan;
  int32_t item0;         // first work item of the layer; items are (b * KV heads + KV head) * max_splits + split
  // Continuous batching: when q_off is set, sequence b is decoded only if it brings exactly
  // one new token, q and out rows [q_off[b], q_off[b+1]) (< total_rows) of a packed batch,
  // and ctx_len holds its prefix length (the token sits at position ctx_len[b]); other
  // sequences are left to the prefill kernel.  Such a job is never split.
  const int32_t* q_off;
  int32_t total_rows;
};

// Row of sequence b in a job's q / out / lse_out.
__host__ __device__ inline int64_t job_row(const DecodeJob& jb, int b) { return jb.q_off ? jb.q_off[b] : b; }

struct DecodeParams {
  const uint8_t* pages[kMaxKvHeads];  // pool slots, one per (layer's) KV head, same page size
  int32_t slot_pages[kMaxKvHeads];    // pages in each slot
  int32_t num_slots;
  int32_t num_kv_heads;               // query heads [j*G, (j+1)*G) read KV head j, G = num_heads / num_kv_heads
  const int32_t* ctx_len;             // [B], shared by the layers
  int32_t batch, num_heads;
  float scale_log2;                   // softmax_scale * log2(e)
  int32_t num_jobs, num_items;
  DecodeJob job[kMaxDecodeJobs];
  uint32_t* queue;                    // [2]: next work item, CTAs finished (both zero between calls)
  int32_t* err;
  uint64_t wait_ns;                   // limit of every bounded wait inside the kernel
  int32_t drop_stage;                 // fault injection: K/V stage each CTA skips (-1: none)
  // 1: the kernel before this launch in the stream touches none of its memory and was
  // itself started only after everything before it had completed, so the launch does
  // not wait for it (it starts on SMs as that kernel's CTAs leave them).
  int32_t overlap_prev;
};

// Attended range and split bookkeeping shared by the decode and combine kernels.
struct SeqSplits {
  int32_t lo, hi;      // attended positions [lo, hi)
  int32_t nsplit;      // number of non-empty splits (0 if nothing to attend)
  bool valid;          // length within the block table
};

__host__ __device__ inline SeqSplits seq_splits(int32_t L, int32_t window, int32_t max_tokens, int32_t chunk) {
  SeqSplits s;
  s.valid = (L >= 0 && L <= max_tokens);
  if (!s.valid) L = 0;
  s.hi = L;
  s.lo = (window > 0 && L > window) ? L - window : 0;
  s.nsplit = s.hi > s.lo ? (s.hi - s.lo + chunk - 1) / chunk : 0;
  return s;
}

// Append of rows with a rotation, and reading rows back (one pool per K/V head; rows packed by q_off,
// or n_new per sequence when it is null).
struct AppendRowsParams {
  uint8_t* pages[kMaxKvHeads];
  int32_t num_pages[kMaxKvHeads];
  int32_t num_kv_heads, num_q_heads, page_size, max_pages;
  int32_t batch, n_new, total_new;
  const int32_t* q_off;
  const int32_t* table;
  const int32_t* start_pos;
  const void* k;                // fp32 or bf16 [rows][Hkv][128], rows k_stride elements apart
  const void* v;
  int64_t k_stride, v_stride, q_stride;
  const uint16_t* q;            // bf16 bits
  uint16_t* q_out;              // bf16 bits [rows][Hq][128]
  const float* cos;             // [num_positions][rot / 2]
  const float* sin;
  int32_t num_positions, rot, interleaved;  // rot 0: no rotation
  // Several axes: positions [rows][num_axes] (null: a row's position is that of its slot), the axis of pair i at bits
  // 2 (i % 16) of axis_bits[i / 16].
  const int32_t* positions;
  int32_t num_axes;
  uint32_t axis_bits[4];
  int32_t* err;
  // Filled by the launch: blocks that write K/V (by `groups` groups of 16 positions per sequence, or by rows
  // when 0), then blocks that rotate queries; whether the tables are 16-byte aligned.
  int32_t kv_blocks, groups, q_blocks, wide_tables;
};

struct ReadRowsParams {
  const uint8_t* pages[kMaxKvHeads];
  int32_t num_pages[kMaxKvHeads];
  int32_t num_kv_heads, page_size, max_pages;
  int32_t batch, n_new, total_new;
  const int32_t* q_off;
  const int32_t* table;
  const int32_t* start_pos;
  void* k_out;                  // fp32 or bf16 [rows][Hkv][128]; either may be null
  void* v_out;
  int32_t* err;
  int32_t groups;               // filled by the launch: groups of 16 positions that a sequence may have
};

// One decode launch over the 4-bit cache, or over lists of pages of either.  q_off / total_rows: as in DecodeJob.
struct Decode4Params {
  const uint8_t* pages[kMaxKvHeads];  // one pool per K/V head
  int32_t num_pages[kMaxKvHeads];
  int32_t num_heads, num_kv_heads, batch;
  int32_t page_size, max_pages, window;
  const int32_t* table;    // [B][max_pages]
  int32_t lists;           // the table has a row for every K/V head: [B][num_kv_heads][max_pages]
  const int32_t* ctx_len;  // [B]
  int32_t before_new;      // ctx_len does not count the new token (prefill calls)
  const int32_t* q_off;    // nullable
  int32_t total_rows;
  const uint16_t* q;       // bf16 bits
  uint16_t* out;           // bf16 bits
  float* lse_out;          // natural log, nullable
  // Work split (plan_decode4).  chunk 0: the keys of all sequences and K/V heads, in tiles of 128, are
  // cut into `ranges` equal parts, one per block; piece of block c: slot 2 c + 1 where it holds a
  // sequence's first tile, 2 c otherwise; meta[c] = {b * num_kv_heads + K/V head, last block} of what starts in
  // block c and goes on in the next, {-1, -1} if nothing does.  A sequence counts piece_tiles more than it has.
  // chunk > 0: every sequence is cut into `splits` ranges of chunk keys; slot (unit * splits + range).
  int32_t head_groups, ranges, chunk, splits, piece_tiles;
  int32_t eight;           // the int8 cache (lists only, attend.cu); set, as lists is, before plan_decode4
  int2* meta;
  float* ws_o;             // [slot][query heads of a K/V head][128] normalised partial outputs
  float* ws_lse;           // [slot][query heads of a K/V head] log2 units
  float scale_log2;
  int32_t* err;
  uint64_t wait_ns;
  int32_t drop_stage;
  int32_t overlap_prev;    // as in DecodeParams
};

// Page summaries of the pages that a call's new tokens lie in.
struct SummarizeParams {
  const uint8_t* pages[kMaxKvHeads];
  int32_t num_pages[kMaxKvHeads];
  uint8_t* data[kMaxKvHeads];   // [num_pages][256] codes, then [num_pages] scales
  int32_t num_kv_heads, page_size, max_pages;
  int32_t batch, n_new, total_new;
  const int32_t* q_off;
  const int32_t* table;
  const int32_t* start_pos;
  int32_t* err;
  int32_t groups;               // filled by the launch: pages that a sequence's new tokens may lie in
};

// Selection of pages for rows of queries.
struct SelectParams {
  const uint8_t* data[kMaxKvHeads];
  int32_t num_pages[kMaxKvHeads];
  int32_t num_kv_heads, num_q_heads, page_size, max_pages;
  int32_t batch, n_new, total_new;
  const int32_t* q_off;
  const int32_t* table;
  const int32_t* start_pos;
  const uint16_t* q;            // bf16 bits [rows][Hq][128]
  int32_t keep, first, last;    // pages of a row, of these at its start and its end
  float* scores;                // workspace: [rows][Hkv][stride]
  int64_t stride;
  int32_t* pages_out;           // [rows][Hkv][keep]
  int32_t* len_out;             // [rows]
  int32_t* err;
  uint64_t wait_ns;
  int32_t drop_stage;           // fault injection: the tile of pages whose products no block hears of (-1: none)
};

struct PrefillLaunch {
  const uint8_t* pages;
  int32_t num_pages, page_size, max_pages;
  const int32_t* table;
  const int32_t* prefix_len;
  const uint16_t* q;
  const int32_t* q_off;  // [batch + 1] packed new-token offsets (device), or null for n_new per sequence
  int32_t batch, n_new, total_new, num_heads, window;  // n_new: the most new tokens of any sequence
  float scale_log2;
  void* workspace;
  float* out;
  float* lse_out;
  int32_t* err;
  bool skip_single;      // with q_off: sequences with one new token are decoded elsewhere
  // The 4-bit cache (four): one pool per K/V head, num_heads then being the query heads of one K/V head
  // and q_heads all of them; the output is bf16.  Otherwise num_kv_heads = 1, q_heads = num_heads.
  bool four = false;
  const uint8_t* pages4[kMaxKvHeads];
  int32_t num_pages4[kMaxKvHeads];
  int32_t num_kv_heads = 1, q_heads = 0;
  uint16_t* out16 = nullptr;
};

// Limit of the kernels' bounded waits (cai_set_wait_limit_ns), read at every launch.
uint64_t wait_limit_ns();
// The stage every CTA skips (cai_set_fault_injection; -1: none), read at every launch.
int32_t fault_drop_stage();

size_t prefill_workspace_bytes(int32_t batch, int32_t max_pages_per_seq, int32_t page_size);
void prefill_piece_region(void* workspace, int32_t batch, int32_t max_pages_per_seq, int32_t page_size,
                          void** region, size_t* bytes);
cudaError_t launch_prefill(const PrefillLaunch& p, cudaStream_t stream);

// Launch with programmatic stream serialization: the grid may start while the
// previous kernel in the stream finishes; every kernel launched this way calls
// grid_dependency_wait() before it touches memory another kernel writes or reads.
template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Host side: the split plan for a launch (also used by the workspace query).
DecodePlan plan_decode(int32_t batch, int32_t max_pages_per_seq, int32_t page_size, int32_t window,
                       int32_t num_splits, int32_t num_sms, int32_t items_per_sm);
int num_sms();

// Entry-point helpers shared by the caches.
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool page_size_ok(int32_t P) { return P == 16 || P == 32 || P == 64; }

// CAI_OK for cudaSuccess; otherwise CAI_ERR_CUDA, with the error kept for
// cai_last_cuda_error() on this thread.
cai_status cuda_status(cudaError_t e);

// Kernel launchers (return cudaGetLastError()).
cudaError_t launch_append(const AppendParams* ps, int n, cudaStream_t stream);
cudaError_t launch_decode(const DecodeParams& p, int page_size, cudaStream_t stream);
cudaError_t launch_append_rows(AppendRowsParams p, bool four, bool bf16, cudaStream_t stream);
cudaError_t launch_read_rows(ReadRowsParams p, bool four, bool bf16, cudaStream_t stream);
cudaError_t launch_summarize(SummarizeParams p, bool four, cudaStream_t stream);
// Elements between the score rows of one query row and K/V head.
inline int64_t score_stride(int32_t max_pages) { return ((int64_t)max_pages + 3) / 4 * 4; }
cudaError_t launch_select(const SelectParams& p, cudaStream_t stream);
cudaError_t launch_decode4(const Decode4Params& p, cudaStream_t stream);
// Fills the split fields of p (batch, heads, page_size, max_pages and window given; num_splits 0: automatic) and
// returns the workspace bytes that they need; place_decode4 then sets the workspace's pointers.
size_t plan_decode4(Decode4Params& p, int32_t num_splits);
// Lists: enough for every plan of this many rows and pages or fewer, with the same heads, page size and num_splits.
size_t most_list_bytes(const Decode4Params& p, int32_t num_splits);
void place_decode4(Decode4Params& p, void* workspace);

}  // namespace cai

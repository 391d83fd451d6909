/*
 * cai.h - C ABI of the int8 MQA paged decode library (libcai.so).
 *
 * What the library computes comes from the pages it was written from:
 *  - "Character.AI: inference optimization", 03 Model architecture, technique
 *    table: Multi-Query Attention in every attention layer (all query heads
 *    read one K/V head); hybrid attention where most layers are local with a
 *    horizon of 1024 and one layer in six is global; KV shared by
 *    neighbouring layers.
 *  - same page, 05 Quantization and cost: the attention KV cache is int8.
 *  - same page, 04 Cache between turns, and the Red Hat page "Como funciona a
 *    inferencia de IA", section "3. Cache de prefixo": the KV of a cached
 *    prefix is reused and only new tokens are processed.
 *  - Red Hat page, section "1. PagedAttention": the cache is cut into
 *    fixed-size blocks placed anywhere in memory, with a per-request table of
 *    block ids.
 *  - Red Hat page, "Por que o cache KV existe": K and V are computed once for
 *    each new token and stored; the new token's query is compared with the
 *    keys of all tokens so far and the values are summed with those weights.
 *
 * Conventions for every call:
 *  - All pointers to tensors are DEVICE pointers unless marked "host".  The
 *    caller owns all memory; the library allocates nothing.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *    default stream).  Host-side validation failures return a status and
 *    launch nothing.  Problems only the device can see (a block-table entry
 *    outside the pool, a length beyond the table) set bits in `*err_flag`
 *    (atomic OR; nullable) and the affected work is skipped: outputs of
 *    affected rows are then unspecified, but no out-of-bounds access happens.
 *  - The library keeps no global state apart from a per-device attribute
 *    cache; calls on different streams are independent.
 *  - head_dim is 128.  Queries are bf16 and must be within the fp16 range
 *    (|q| <= 65504): the tensor-core path runs in fp16 with fp32 accumulation.
 *    K/V inputs must be finite.
 */
#ifndef CAI_H_
#define CAI_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum cai_status {
  CAI_OK = 0,
  CAI_ERR_INVALID_ARG = 1, /* null pointer, negative size, misaligned pointer, index out of range */
  CAI_ERR_UNSUPPORTED = 2, /* head_dim, page_size or head count outside what the kernels implement */
  CAI_ERR_WORKSPACE = 3,   /* workspace missing or smaller than cai_mqa_decode_workspace_size() */
  CAI_ERR_CUDA = 4         /* a CUDA runtime call or a launch failed */
} cai_status;

/* Bits OR-ed into *err_flag by the kernels. */
#define CAI_DEVERR_PAGE 1   /* a needed block-table entry is outside [0, num_pages) */
#define CAI_DEVERR_LENGTH 2 /* a length or position is negative or beyond max_pages_per_seq * page_size */
#define CAI_DEVERR_TIMEOUT 4 /* a bounded wait inside a kernel gave up; that launch's outputs are unspecified */

/* One KV buffer: a pool of fixed-size pages (PagedAttention blocks).
 * Page layout (bytes), for P = page_size and d = head_dim:
 *   [0,        P*d)        K codes, int8 [P][d] (token-major: slot s at s*d)
 *   [P*d,      2*P*d)      V codes, int8 [d][P] (channel-major: channel c at c*P)
 *   [2*P*d,    2*P*d+4*P)  K scales, fp32 [P]
 *   [2*P*d+4P, 2*P*d+8*P)  V scales, fp32 [P]
 * Token at position p of a sequence lives in page block_table[p / P], slot p % P.
 * `pages` must be 16-byte aligned; it holds num_pages * cai_page_bytes(P, d) bytes. */
typedef struct cai_kv_pool {
  void* pages;
  int32_t num_pages;
  int32_t page_size; /* 16, 32 or 64 tokens */
  int32_t head_dim;  /* 128 */
} cai_kv_pool;

/* Bytes of one page: page_size * (2*head_dim + 8).  0 for non-positive arguments. */
size_t cai_page_bytes(int32_t page_size, int32_t head_dim);

/* Quantize new tokens to int8 and write them into their pages.
 * Int8 KV cache ("Character.AI: inference optimization", 05), written once per
 * new token (Red Hat page, "Por que o cache KV existe").  For each token and
 * separately for K and V: s = max_i |x_i| / 127 (fp32, IEEE division),
 * code_i = clamp(round_half_even(x_i / s), -127, 127); codes 0 when s is 0 (an
 * all-zero vector, or max |x_i| / 127 below the smallest fp32 subnormal).
 * Results are bit-exact.
 *   pool        host pointer to the pool description
 *   k_new,v_new fp32 [batch][n_new][head_dim], 16-byte aligned
 *   block_table int32 [batch][max_pages_per_seq]; entries for the written positions must be valid pages
 *   start_pos   int32 [batch]: token i of sequence b goes to position start_pos[b] + i
 *   err_flag    int32, nullable
 * Positions outside [0, max_pages_per_seq * page_size) set CAI_DEVERR_LENGTH; bad
 * page ids set CAI_DEVERR_PAGE; such tokens are not written.  No other byte of the
 * pool changes (K and V of past tokens never change). */
cai_status cai_kv_append(const cai_kv_pool* pool, const float* k_new, const float* v_new, int32_t batch,
                         int32_t n_new, const int32_t* block_table, int32_t max_pages_per_seq,
                         const int32_t* start_pos, int32_t* err_flag, void* stream);

/* The append of one step into several KV buffers in one launch: for every i the
 * same as cai_kv_append(&pools[i], k_new[i], v_new[i], batch, n_new,
 * block_tables[i], max_pages_per_seq, start_pos[i], ...) (neighbouring layers
 * that share a buffer append once; "Character.AI: inference optimization"
 * page, 03 Model architecture).
 *   pools, num_pools       host array of 1..8 KV buffers
 *   k_new, v_new           host arrays [num_pools] of device fp32 [batch][n_new][head_dim], 16-byte aligned
 *   block_tables           host array [num_pools] of device int32 [batch][max_pages_per_seq]
 *   start_pos              host array [num_pools] of device int32 [batch]
 * Errors as for cai_kv_append; nothing is launched when an argument is rejected. */
cai_status cai_kv_append_pools(const cai_kv_pool* pools, int32_t num_pools, const float* const* k_new,
                               const float* const* v_new, int32_t batch, int32_t n_new,
                               const int32_t* const* block_tables, int32_t max_pages_per_seq,
                               const int32_t* const* start_pos, int32_t* err_flag, void* stream);

/* Bytes of workspace cai_mqa_decode needs for these arguments: a 256-byte
 * header (the counters of the kernel's work queue) plus, when sequences are
 * split, the partial outputs.  Arguments as for cai_mqa_decode.  The automatic
 * split plan (num_splits = 0) depends on the SM count of the current device:
 * query with the device that will run the call. */
size_t cai_mqa_decode_workspace_size(int32_t batch, int32_t num_q_heads, int32_t max_pages_per_seq,
                                     int32_t page_size, int32_t window, int32_t num_splits);

/* One decode step of one layer: MQA attention of one query token per sequence
 * over its int8 paged KV.
 *   pools, num_pools       host array of KV buffers
 *   layer_to_pool          host int32 [num_layers]: buffer read by each layer (layers may share one)
 *   layer                  the layer to run
 *   q                      bf16 bits [batch][num_q_heads][head_dim], 16-byte aligned
 *   num_q_heads            1..64 query heads, all sharing the single K/V head
 *   block_table            int32 [batch][max_pages_per_seq]
 *   ctx_len                int32 [batch]: cached tokens INCLUDING the current one (append first)
 *   window                 0 = global; W > 0 = local: only the last W positions
 *                          [max(0, L-W), L) are attended, pages wholly before them are never read
 *   softmax_scale          logit = softmax_scale * <q, k>
 *   num_splits             0 = automatic; otherwise the attended span of each sequence is cut
 *                          into at most this many consecutive chunks (1..64), processed as
 *                          separate work items and merged with their log-sum-exp
 *   workspace              device scratch of at least cai_mqa_decode_workspace_size() bytes,
 *                          256-byte aligned.  Its first 256 bytes must be zero before the first
 *                          call that uses it; every call leaves them zero again (after a call
 *                          that reported CAI_DEVERR_TIMEOUT, zero them before reuse).  Calls that
 *                          share a workspace must not overlap on the GPU.
 *   out                    fp32 [batch][num_q_heads][head_dim], 16-byte aligned
 *   lse_out                fp32 [batch][num_q_heads] natural-log log-sum-exp of the logits, nullable;
 *                          any 4-byte alignment (at 16 bytes it is written by bulk copies)
 * A sequence with nothing to attend (L = 0) gets out = 0 and lse = -inf. */
cai_status cai_mqa_decode(const cai_kv_pool* pools, int32_t num_pools, const int32_t* layer_to_pool,
                          int32_t num_layers, int32_t layer, const uint16_t* q, int32_t batch,
                          int32_t num_q_heads, const int32_t* block_table, int32_t max_pages_per_seq,
                          const int32_t* ctx_len, int32_t window, float softmax_scale, int32_t num_splits,
                          void* workspace, size_t workspace_bytes, float* out, float* lse_out,
                          int32_t* err_flag, void* stream);

/* Workspace bytes for cai_mqa_decode_layers (windows: host int32 [num_layers]); 0 if the
 * arguments are invalid. */
size_t cai_mqa_decode_layers_workspace_size(int32_t batch, int32_t num_q_heads, int32_t max_pages_per_seq,
                                            int32_t page_size, int32_t num_layers, const int32_t* windows,
                                            int32_t num_splits);

/* One decode step of several layers in one launch: for every layer l the same
 * computation as cai_mqa_decode, on the same work split, with the work items of
 * all the layers taken from one queue (global layers first) so that the SMs even
 * out over the whole step instead of layer by layer.  One call covers a decode
 * step of the hybrid stack ("Character.AI: inference optimization" page,
 * 03 Model architecture: local layers with a 1024 horizon, one global layer in
 * six, neighbouring layers sharing one KV buffer; 02 The bottleneck: reading the
 * attention KV dominates the I/O of a step).
 *   pools, num_pools       host array of KV buffers
 *   layer_to_pool          host int32 [num_layers]: buffer read by each layer (layers may share one)
 *   num_layers             1..8
 *   windows                host int32 [num_layers]: 0 = global, W > 0 = local (as in cai_mqa_decode)
 *   q                      host array [num_layers] of device bf16 bits [batch][num_q_heads][head_dim],
 *                          each 16-byte aligned
 *   block_tables           host array [num_layers] of device int32 [batch][max_pages_per_seq]
 *   ctx_len                int32 [batch], shared by the layers (append first)
 *   workspace              device scratch of cai_mqa_decode_layers_workspace_size() bytes, 256-byte
 *                          aligned, first 256 bytes zero (as for cai_mqa_decode)
 *   out                    host array [num_layers] of device fp32 [batch][num_q_heads][head_dim],
 *                          each 16-byte aligned
 *   lse_out                host array [num_layers] of nullable device fp32 [batch][num_q_heads], or null
 * All buffers must use one page size; at most 8 distinct buffers.  Errors as for
 * cai_mqa_decode; nothing is launched when an argument is rejected. */
cai_status cai_mqa_decode_layers(const cai_kv_pool* pools, int32_t num_pools, const int32_t* layer_to_pool,
                                 int32_t num_layers, const int32_t* windows, const uint16_t* const* q,
                                 int32_t batch, int32_t num_q_heads, const int32_t* const* block_tables,
                                 int32_t max_pages_per_seq, const int32_t* ctx_len, float softmax_scale,
                                 int32_t num_splits, void* workspace, size_t workspace_bytes, float* const* out,
                                 float* const* lse_out, int32_t* err_flag, void* stream);

/* Decode without any caller scratch.  The pages have no counterpart to this
 * entry point: it exists for callers that cannot allocate device memory at
 * the moment they decode -- a serving loop that forbids cudaMalloc after
 * warm-up (an allocation can synchronise the device and stall other
 * streams), a plug-in interface that passes only input and output buffers,
 * or a framework that owns all device memory and lends none to its plug-ins.
 * It computes exactly what cai_mqa_decode computes, with the same arguments
 * minus the workspace: the work-queue counters and the split partials live in
 * a scratch array built into the library, CAI_NO_ALLOC_SCRATCH_BYTES per GPU,
 * held by every GPU that loads the library until the process exits.  A call
 * whose plan needs more (cai_mqa_decode_workspace_size() above the limit)
 * returns CAI_ERR_WORKSPACE and launches nothing: lower num_splits (1 needs
 * only the 256-byte counter header).  The first call on a device looks up the
 * array's device address on that device (again after the device's primary
 * context was replaced, e.g. by cudaDeviceReset); make that first call before
 * any stream capture.  Each call clears the counter header with a
 * stream-ordered memset before its launch, so a call after one that reported
 * CAI_DEVERR_TIMEOUT starts clean.  All calls share the array and it keeps the
 * last call's contents: calls whose kernels overlap on the GPU (unordered
 * streams) race on it.  A device index of 64 or more returns
 * CAI_ERR_UNSUPPORTED; a failed address lookup returns CAI_ERR_CUDA with the
 * error in cai_last_cuda_error(). */
#define CAI_NO_ALLOC_SCRATCH_BYTES (32u << 20)
cai_status cai_mqa_decode_no_alloc(const cai_kv_pool* pools, int32_t num_pools, const int32_t* layer_to_pool,
                                   int32_t num_layers, int32_t layer, const uint16_t* q, int32_t batch,
                                   int32_t num_q_heads, const int32_t* block_table, int32_t max_pages_per_seq,
                                   const int32_t* ctx_len, int32_t window, float softmax_scale, int32_t num_splits,
                                   float* out, float* lse_out, int32_t* err_flag, void* stream);

/* Bytes of workspace cai_mqa_prefill_chunk needs: a contiguous 16-bit copy of
 * the K and V codes and the scales of up to max_pages_per_seq * page_size keys
 * per sequence (rounded up to 128).  Arguments as for cai_mqa_prefill_chunk. */
size_t cai_mqa_prefill_workspace_size(int32_t batch, int32_t max_pages_per_seq, int32_t page_size);

/* Attention for a chunk of new tokens appended on top of a reused prefix.
 * Prefix caching (Red Hat page, "3. Cache de prefixo") and the cross-turn
 * cache ("Character.AI: inference optimization", 04): the prefix K/V is read
 * from the int8 cache, not recomputed.  The chunk's own K/V must already be
 * appended (cai_kv_append with start_pos = prefix_len), so prefix and chunk
 * keys are read from the same int8 pages.  New token i of sequence b sits at
 * position p0 + i (p0 = prefix_len[b]) and attends keys [lo, p0 + i] with
 * lo = 0 (window 0) or max(0, p0 + i + 1 - window).
 *   q           bf16 bits [batch][n_new][num_q_heads][head_dim], 16-byte aligned
 *   num_q_heads a power of two from 1 to 128
 *   block_table int32 [batch][max_pages_per_seq]; prefix_len int32 [batch]
 *   workspace   device scratch of cai_mqa_prefill_workspace_size() bytes, 256-byte aligned
 *   out         fp32 [batch][n_new][num_q_heads][head_dim], 16-byte aligned
 *   lse_out     fp32 [batch][n_new][num_q_heads], natural log, nullable
 * A sequence whose prefix_len + n_new exceeds the table sets CAI_DEVERR_LENGTH and
 * gets out = 0, lse = -inf. */
cai_status cai_mqa_prefill_chunk(const cai_kv_pool* pool, const uint16_t* q, int32_t batch, int32_t n_new,
                                 int32_t num_q_heads, const int32_t* block_table, int32_t max_pages_per_seq,
                                 const int32_t* prefix_len, int32_t window, float softmax_scale, void* workspace,
                                 size_t workspace_bytes, float* out, float* lse_out, int32_t* err_flag,
                                 void* stream);

/* Grouped-query attention: num_kv_heads K/V heads, each shared by a group of
 * G = num_q_heads / num_kv_heads query heads (query heads [j*G, (j+1)*G) read KV head
 * j).  The pages compare Multi-Query Attention, one K/V head for all query heads,
 * against it: MQA keeps the KV cache 8X smaller than the grouped-query attention of
 * most open models ("Character.AI: inference optimization", section 03 and its
 * technique table).  Each KV head lives in its own pool (same page size and page
 * count, same block table and lengths) and is appended with cai_kv_append like an MQA
 * buffer; with num_kv_heads = 1 this is cai_mqa_decode.
 *   kv_pools    host array [num_kv_heads], 1 <= num_kv_heads <= 8
 *   num_q_heads a multiple of num_kv_heads with G <= 64
 *   q, out, lse_out, block_table, ctx_len, window, num_splits as cai_mqa_decode
 *   workspace   device scratch of cai_gqa_decode_workspace_size() bytes, 256-byte aligned,
 *               first 256 bytes zero before the first use (kept zero by every call) */
size_t cai_gqa_decode_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                     int32_t max_pages_per_seq, int32_t page_size, int32_t window,
                                     int32_t num_splits);
cai_status cai_gqa_decode(const cai_kv_pool* kv_pools, int32_t num_kv_heads, const uint16_t* q, int32_t batch,
                          int32_t num_q_heads, const int32_t* block_table, int32_t max_pages_per_seq,
                          const int32_t* ctx_len, int32_t window, float softmax_scale, int32_t num_splits,
                          void* workspace, size_t workspace_bytes, float* out, float* lse_out, int32_t* err_flag,
                          void* stream);

/* Continuous batching: the same attention for a batch whose sequences bring different
 * numbers of new tokens in one call -- decode steps (one token) next to prefill
 * chunks (Red Hat page, "2. Processamento contínuo em lotes" and its figure 7:
 * finished requests leave and new ones join as slots free up, instead of the whole
 * batch waiting for its slowest request).  Sequence b owns new-token rows [q_offsets[b], q_offsets[b+1])
 * of q, out and lse_out (packed), its token i sits at position prefix_len[b] + i and
 * attends as in cai_mqa_prefill_chunk.  Its K/V must already be appended.
 *   q           bf16 bits [total_new][num_q_heads][head_dim], 16-byte aligned
 *   q_offsets   int32 [batch + 1] (device), non-decreasing, q_offsets[batch] <= total_new
 *   max_new     host bound on q_offsets[b+1] - q_offsets[b] (sizes the launch)
 *   out         fp32 [total_new][num_q_heads][head_dim], 16-byte aligned;
 *               lse_out fp32 [total_new][num_q_heads], nullable
 * Other arguments, workspace and limits as cai_mqa_prefill_chunk.  A sequence whose
 * offsets are out of order, beyond total_new or longer than max_new, or whose
 * prefix_len + length exceeds the table, sets CAI_DEVERR_LENGTH; its rows (if its
 * offsets are valid) get out = 0, lse = -inf.  With num_q_heads <= 64 the sequences with
 * exactly one new token run through the decode kernel and the prefill kernel skips
 * them (the results are the same either way): on `stream`, the prefill's key copy and
 * attention launches, then the decode launch (and its split combine), which shares no
 * memory with the prefill and starts on the SMs that the prefill's CTAs leave; it ends
 * after the prefill, so work later in the stream finds both complete. */
cai_status cai_mqa_prefill_varlen(const cai_kv_pool* pool, const uint16_t* q, int32_t batch,
                                  const int32_t* q_offsets, int32_t total_new, int32_t max_new, int32_t num_q_heads,
                                  const int32_t* block_table, int32_t max_pages_per_seq, const int32_t* prefix_len,
                                  int32_t window, float softmax_scale, void* workspace, size_t workspace_bytes,
                                  float* out, float* lse_out, int32_t* err_flag, void* stream);

/* ---- Rotated appends, reading back, and the 4-bit cache --------------------
 * The calls of this section take one pool per K/V head (num_kv_heads of them, 1..8,
 * as cai_gqa_decode: the same page size, block table and lengths for all) and give
 * new tokens as rows.  Rows are either `n_new` per sequence (q_offsets null, sequence b
 * owning rows [b * n_new, (b + 1) * n_new); total_new is not read), or packed as in
 * cai_mqa_prefill_varlen: sequence b owns rows [q_offsets[b], q_offsets[b + 1]) of
 * total_new, at most n_new of them.  A sequence whose offsets are out of order, beyond
 * total_new or longer than n_new sets CAI_DEVERR_LENGTH and none of its rows is touched
 * (the appends may then leave out rows of other sequences, too).  With packed rows n_new
 * is a bound; appends and reads look through batch * num_kv_heads * n_new / 16 groups of
 * positions for those with rows, so a bound far above every count costs time.
 *
 * The 4-bit cache holds a token's K (and V) as 128 4-bit codes and four scales, one
 * per 32 channels: s = fp16(bf16(max |x| / 7)) (both roundings to nearest even, the
 * division IEEE fp32; at most 9344, so magnitudes above 65408 saturate), code =
 * clamp(round_half_even(x / s), -7, 7), codes 0 when s is 0.  A code stands for
 * code * s, exactly an fp16 number.  A token takes 144 bytes per K/V head, against 264
 * in the int8 cache. */

/* One buffer of the 4-bit cache.  A page is page_size / 16 blocks of 2304 bytes, 16
 * tokens each: K codes (1024 bytes), V codes (1024), K scales fp16 [16][4] (128), V
 * scales fp16 (128).  Codes are stored as code + 8 in a byte:
 *   K of token r: bits 4 i + 16 e (i = 0..3, e = 0, 1) of the 32-bit word at
 *     64 r + 16 t + 4 j hold channel 32 j + 8 t + 2 i + e;
 *   V: bits 4 i + 16 e of the word at 1024 + 4 ((32 h + 4 g + t) 4 + w) hold channel
 *     16 (4 h + w) + g + 8 (i mod 2) of token 8 (i div 2) + 2 t + e;
 *   V scales: token 8 b + 2 t + e, channels 32 j .. 32 j + 31 at 2176 + 2 (16 t + 8 b + 2 j + e).
 * `pages` must be 16-byte aligned; it holds num_pages * cai_kv4_page_bytes(P, d) bytes. */
typedef struct cai_kv4_pool {
  void* pages;
  int32_t num_pages;
  int32_t page_size; /* 16, 32 or 64 tokens */
  int32_t head_dim;  /* 128 */
} cai_kv4_pool;

/* Bytes of one page of the 4-bit cache: page_size * (head_dim + head_dim / 8).  0 unless
 * page_size is a positive multiple of 16 and head_dim one of 32. */
size_t cai_kv4_page_bytes(int32_t page_size, int32_t head_dim);

/* Position rotation.  Channels [0, rot_dim) pair up, i with i + rot_dim / 2, or 2 i with
 * 2 i + 1 if `interleaved` is not 0; at position p a pair (a, b) becomes
 * (a c - b s, b c + a s) with c = cos[p][i], s = sin[p][i], every product and sum
 * rounded to fp32 on its own.  The other channels pass.
 *   cos, sin       device fp32 [num_positions][rot_dim / 2], 4-byte aligned
 *   rot_dim        even, 2..128
 * A token at a position of num_positions or beyond sets CAI_DEVERR_LENGTH and is left out. */
typedef struct cai_rope {
  const float* cos;
  const float* sin;
  int32_t num_positions;
  int32_t rot_dim;
  int32_t interleaved;
} cai_rope;

/* Element type of K/V rows. */
typedef enum cai_dtype { CAI_FP32 = 0, CAI_BF16 = 1 } cai_dtype;

/* Rotate, quantize and append new tokens, and rotate their queries, in one launch.
 * Without a rotation cai_kv_append_rope writes the bytes that cai_kv_append writes for
 * every K/V head; cai_kv4_append is the same into the 4-bit cache.
 *   kv_pools      host array [num_kv_heads]
 *   rope          host pointer, null for no rotation (V is never rotated)
 *   k_new, v_new  kv_type [rows][num_kv_heads][128], rows k_stride / v_stride ELEMENTS
 *                 apart (so that they may be slices of one projection's output); 16-byte
 *                 aligned, strides a multiple of 16 bytes and at least num_kv_heads * 128
 *   q, q_out      bf16 bits: [rows][num_q_heads][128], rows q_stride elements apart, to
 *                 [rows][num_q_heads][128] contiguous; both null (num_q_heads 0) for none,
 *                 otherwise rope must be given.  16-byte aligned, q_stride a multiple of 8;
 *                 q_out may be q itself when q_stride is num_q_heads * 128, otherwise they
 *                 must not overlap
 *   start_pos     int32 [batch]: row i of sequence b goes to position start_pos[b] + i
 * Bad positions and page ids as in cai_kv_append (a token whose position is bad gets no
 * q_out row; one whose page is bad does). */
cai_status cai_kv_append_rope(const cai_kv_pool* kv_pools, int32_t num_kv_heads, const cai_rope* rope,
                              const void* k_new, const void* v_new, cai_dtype kv_type, int64_t k_stride,
                              int64_t v_stride, const uint16_t* q, int64_t q_stride, uint16_t* q_out,
                              int32_t num_q_heads, int32_t batch, int32_t n_new, const int32_t* q_offsets,
                              int32_t total_new, const int32_t* block_table, int32_t max_pages_per_seq,
                              const int32_t* start_pos, int32_t* err_flag, void* stream);
cai_status cai_kv4_append(const cai_kv4_pool* kv_pools, int32_t num_kv_heads, const cai_rope* rope,
                          const void* k_new, const void* v_new, cai_dtype kv_type, int64_t k_stride,
                          int64_t v_stride, const uint16_t* q, int64_t q_stride, uint16_t* q_out,
                          int32_t num_q_heads, int32_t batch, int32_t n_new, const int32_t* q_offsets,
                          int32_t total_new, const int32_t* block_table, int32_t max_pages_per_seq,
                          const int32_t* start_pos, int32_t* err_flag, void* stream);

/* cai_kv_append_rope and cai_kv4_append for tokens that have a position on several axes, as
 * those of images and video do (time, height, width): pair i of row r turns by row
 * positions[r][axis[i]] of the tables.  The slot that a row is written to is start_pos[b] + i
 * as ever.  With equal positions on all axes it is the rotation by that position.
 *   rope          must be given; num_positions is the tables' rows, for every axis
 *   axis          host uint8 [rot_dim / 2]: the axis of each pair, below num_axes (sections one
 *                 behind the other, in turn, or any other way)
 *   num_axes      1..4
 *   positions     int32 [rows][num_axes], 4-byte aligned, row by row as k_new (text: the same
 *                 number on all axes)
 * A row with a position outside [0, num_positions) on any axis, used by a pair or not, sets
 * CAI_DEVERR_LENGTH and is left out; other arguments and errors as cai_kv_append_rope. */
cai_status cai_kv_append_rope_axes(const cai_kv_pool* kv_pools, int32_t num_kv_heads, const cai_rope* rope,
                                   const uint8_t* axis, int32_t num_axes, const int32_t* positions,
                                   const void* k_new, const void* v_new, cai_dtype kv_type, int64_t k_stride,
                                   int64_t v_stride, const uint16_t* q, int64_t q_stride, uint16_t* q_out,
                                   int32_t num_q_heads, int32_t batch, int32_t n_new, const int32_t* q_offsets,
                                   int32_t total_new, const int32_t* block_table, int32_t max_pages_per_seq,
                                   const int32_t* start_pos, int32_t* err_flag, void* stream);
cai_status cai_kv4_append_axes(const cai_kv4_pool* kv_pools, int32_t num_kv_heads, const cai_rope* rope,
                               const uint8_t* axis, int32_t num_axes, const int32_t* positions, const void* k_new,
                               const void* v_new, cai_dtype kv_type, int64_t k_stride, int64_t v_stride,
                               const uint16_t* q, int64_t q_stride, uint16_t* q_out, int32_t num_q_heads,
                               int32_t batch, int32_t n_new, const int32_t* q_offsets, int32_t total_new,
                               const int32_t* block_table, int32_t max_pages_per_seq, const int32_t* start_pos,
                               int32_t* err_flag, void* stream);

/* Read cached tokens back as the values they stand for (code * scale in fp32; bf16 rounds
 * that once more): for an attention that the library does not have, or to move a dialogue
 * from one cache to the other.  Row i of sequence b comes from position start_pos[b] + i.
 *   k_out, v_out  out_type [rows][num_kv_heads][128], 16-byte aligned; one may be null
 * A bad position or page id sets its bit in *err_flag and its rows become 0. */
cai_status cai_kv_read(const cai_kv_pool* kv_pools, int32_t num_kv_heads, void* k_out, void* v_out,
                       cai_dtype out_type, int32_t batch, int32_t n_new, const int32_t* q_offsets,
                       int32_t total_new, const int32_t* block_table, int32_t max_pages_per_seq,
                       const int32_t* start_pos, int32_t* err_flag, void* stream);
cai_status cai_kv4_read(const cai_kv4_pool* kv_pools, int32_t num_kv_heads, void* k_out, void* v_out,
                        cai_dtype out_type, int32_t batch, int32_t n_new, const int32_t* q_offsets,
                        int32_t total_new, const int32_t* block_table, int32_t max_pages_per_seq,
                        const int32_t* start_pos, int32_t* err_flag, void* stream);

/* One decode step of one layer over the 4-bit cache: cai_gqa_decode's attention, reading
 * 144 bytes a token and K/V head.
 *   num_q_heads   a multiple of num_kv_heads; up to 128 query heads per K/V head
 *   q             multiplied as fp16: exact for magnitudes from 2^-17 to 65504, below that
 *                 off by 2^-25 at most
 *   softmax_scale finite; 0 and negative ones included
 *   out           bf16 bits [batch][num_q_heads][128], 16-byte aligned (fp32 sums, rounded
 *                 once; a weight enters its product with V as fp16, off by 2^-11 of itself or
 *                 2^-32 of the sum of the weights)
 *   workspace     cai_kv4_decode_workspace_size() bytes, 256-byte aligned; may be null when
 *                 that is 0.  It needs no preparation; calls that share it must not overlap
 *                 on the GPU.
 *   q, block_table, ctx_len, window, num_splits, lse_out otherwise as cai_gqa_decode
 * A sequence with nothing to attend, or of an invalid length (flagged), gets out = 0 and
 * lse = -inf.  Slots past a sequence's length are not looked at, whatever they hold. */
size_t cai_kv4_decode_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                     int32_t max_pages_per_seq, int32_t page_size, int32_t window,
                                     int32_t num_splits);
cai_status cai_kv4_decode(const cai_kv4_pool* kv_pools, int32_t num_kv_heads, const uint16_t* q, int32_t batch,
                          int32_t num_q_heads, const int32_t* block_table, int32_t max_pages_per_seq,
                          const int32_t* ctx_len, int32_t window, float softmax_scale, int32_t num_splits,
                          void* workspace, size_t workspace_bytes, uint16_t* out, float* lse_out,
                          int32_t* err_flag, void* stream);

/* Attention of new tokens on a reused prefix over the 4-bit cache: cai_mqa_prefill_chunk
 * (q_offsets null) and cai_mqa_prefill_varlen (packed rows, decode rows among them) for
 * num_kv_heads K/V heads.  The new tokens' K/V must already be appended.
 *   num_q_heads   num_kv_heads times a power of two from 1 to 128
 *   q             bf16 bits [rows][num_q_heads][128]; prefix_len int32 [batch]
 *   out           bf16 bits [rows][num_q_heads][128]; lse_out fp32 [rows][num_q_heads], nullable
 *   workspace     cai_kv4_prefill_workspace_size() bytes, 256-byte aligned (no preparation).
 *                 It holds an fp16 copy of the keys and values: 520 bytes for every token
 *                 that the tables have room for and K/V head, whatever the lengths and the window
 * Roundings as cai_kv4_decode's; other arguments and errors as for the int8 calls. */
size_t cai_kv4_prefill_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                      int32_t max_pages_per_seq, int32_t page_size);
cai_status cai_kv4_prefill(const cai_kv4_pool* kv_pools, int32_t num_kv_heads, const uint16_t* q, int32_t batch,
                           int32_t n_new, const int32_t* q_offsets, int32_t total_new, int32_t num_q_heads,
                           const int32_t* block_table, int32_t max_pages_per_seq, const int32_t* prefix_len,
                           int32_t window, float softmax_scale, void* workspace, size_t workspace_bytes,
                           uint16_t* out, float* lse_out, int32_t* err_flag, void* stream);

/* ---- Attention over a part of a long context --------------------------------
 * A query of a long context needs few of its pages.  Three operators, for both caches:
 * cai_kv_summarize keeps, for every page, the range of its keys; cai_kv_select reads these
 * summaries (260 bytes a page and K/V head) and lists the pages in which each query may have its
 * largest logits; cai_kv_attend_pages attends over the listed pages.  A decode step is
 * append, summarize, select, attend, each on the same block tables; a chunk of n_new tokens a
 * sequence is the same calls, every row with lists of its own.  Rows are given as in the
 * section on rotated appends (n_new a sequence, or packed by q_offsets); a call with batch or
 * n_new 0 does nothing.  Queries and cached keys are finite numbers: a query that is not selects any
 * pages and gives its head any output, and does nothing to other heads and rows. */

/* Summaries of one pool's pages: `data` holds int8 [num_pages][256], page by page the codes of
 * the 128 channels' largest keys and of their smallest, then fp32 [num_pages], the scales.  It
 * must be 16-byte aligned and holds cai_kv_summary_bytes(num_pages, head_dim) bytes.  A page's
 * summary belongs to the page: sequences that share the page share it. */
typedef struct cai_kv_summary {
  void* data;
  int32_t num_pages;
  int32_t page_size; /* 16, 32 or 64 tokens */
  int32_t head_dim;  /* 128 */
} cai_kv_summary;

/* num_pages * (2 * head_dim + 4); 0 for non-positive arguments. */
size_t cai_kv_summary_bytes(int32_t num_pages, int32_t head_dim);

/* Bring the summaries of the pages that new tokens lie in up to date: call it behind the append,
 * with the append's table, start_pos and counts (or with start_pos 0 and the lengths, for
 * dialogues whose summaries are not there).  Every page that holds a position of
 * [start_pos[b], start_pos[b] + n) is computed anew from the cached keys of its tokens, those
 * before start_pos included, none at or past start_pos[b] + n.
 * With x the fp32 values that the cached keys stand for, hi_c and lo_c their largest and smallest
 * of channel c: s = max_c max(|hi_c|, |lo_c|) / 127 (IEEE fp32 division), codes
 * min(127, ceil(hi_c / s)) and max(-127, floor(lo_c / s)); all 0 when s is 0.
 *   kv_pools, summaries   host arrays [num_kv_heads], of the same page counts
 *   n_new, q_offsets      as for the append; q_offsets[batch] is not limited here
 * Sequences of one call that share a page must have the same number of its tokens (shared
 * prefixes have whole pages).  Bad positions, page ids and offsets as in cai_kv_append_rope; other
 * summaries are not touched. */
cai_status cai_kv_summarize(const cai_kv_pool* kv_pools, const cai_kv_summary* summaries, int32_t num_kv_heads,
                            int32_t batch, int32_t n_new, const int32_t* q_offsets, const int32_t* block_table,
                            int32_t max_pages_per_seq, const int32_t* start_pos, int32_t* err_flag, void* stream);
cai_status cai_kv4_summarize(const cai_kv4_pool* kv_pools, const cai_kv_summary* summaries, int32_t num_kv_heads,
                             int32_t batch, int32_t n_new, const int32_t* q_offsets, const int32_t* block_table,
                             int32_t max_pages_per_seq, const int32_t* start_pos, int32_t* err_flag, void* stream);

/* For every row of queries and K/V head the pages to attend over.  Row i of sequence b sits at
 * position p = start_pos[b] + i (decode: start_pos = context length - 1) and sees the n = p / P + 1
 * pages of its table row.  It takes all of them where n <= num_selected; otherwise the `first`
 * first and `last` last ones, and those of the largest scores among the rest, ties by the lower
 * page.  A head's query becomes whole numbers q'_c = clamp(round_half_even(q_c / t), -127, 127),
 * t = max |q_c| / 127 (IEEE fp32 divisions; 0 when t is 0); with a page's codes hi, lo and
 * scale s, score = s * max over the group's heads of t * sum_c max(q'_c hi_c, q'_c lo_c), each of
 * the two products rounded to fp32 once: what the largest logit of the page may be, up to the
 * roundings and for positive softmax scales (negate q for a negative one).
 *   summaries     host array [num_kv_heads], one per K/V head, brought up to date
 *   q             bf16 bits [rows][num_q_heads][128] (rotated, as for the attention), 16-byte aligned
 *   num_q_heads   a multiple of num_kv_heads; up to 128 query heads per K/V head
 *   num_selected  pages of a row, first + last at least; first >= 0, last >= 1 (a row's own page
 *                 is always taken)
 *   workspace     cai_kv_select_workspace_size() bytes for the call's rows (batch * n_new, or
 *                 total_new), 256-byte aligned; no preparation.  Calls that share it must not
 *                 overlap on the GPU
 *   limits        (rows + batch) * num_kv_heads below 2^31
 *   pages_out     int32 [rows][num_kv_heads][num_selected]: page ids in the order of positions, -1
 *                 behind the last
 *   len_out       int32 [rows]: the tokens of these lists, the same for all K/V heads: all pages
 *                 are whole but the row's own, which comes last
 * A row that no sequence has (behind the last one, in a padded batch), of a sequence with invalid
 * offsets or at a position outside the table gets a list of -1 and length 0; the latter two
 * set CAI_DEVERR_LENGTH.  A page id outside the summaries sets CAI_DEVERR_PAGE; it has the least
 * score, and stands in the list if it is taken all the same. */
size_t cai_kv_select_workspace_size(int32_t batch, int32_t total_rows, int32_t num_q_heads, int32_t num_kv_heads,
                                    int32_t max_pages_per_seq);
cai_status cai_kv_select(const cai_kv_summary* summaries, int32_t num_kv_heads, const uint16_t* q, int32_t batch,
                         int32_t n_new, const int32_t* q_offsets, int32_t total_new, int32_t num_q_heads,
                         const int32_t* block_table, int32_t max_pages_per_seq, const int32_t* start_pos,
                         int32_t num_selected, int32_t first, int32_t last, void* workspace, size_t workspace_bytes,
                         int32_t* pages_out, int32_t* len_out, int32_t* err_flag, void* stream);

/* Attention of rows of queries over lists of pages, a list for each K/V head: over the tokens of
 * the listed pages in turn, the first len[r] of them.  The lists of cai_kv_select, or any other:
 * a page that stands in a list twice counts twice, and no token is masked but by len.
 *   q             bf16 bits [rows][num_q_heads][128], 16-byte aligned; rows <= 65535, as every call's
 *                 batch (no row depends on another: more of them, as cai_kv_select takes, are
 *                 given in several calls)
 *   num_q_heads   a multiple of num_kv_heads; up to 128 query heads per K/V head
 *   pages         int32 [rows][num_kv_heads][width]; entries behind ceil(len[r] / P) are not read
 *   len           int32 [rows]; 0: out = 0, lse = -inf.  Outside [0, width * P]: the same, and
 *                 CAI_DEVERR_LENGTH
 *   out           bf16 bits [rows][num_q_heads][128], 16-byte aligned, rounded once from fp32
 *   lse_out       fp32 [rows][num_q_heads], nullable
 *   workspace     cai_kv_attend_pages_workspace_size() bytes (cai_kv4_... for the 4-bit cache), 256-byte
 *                 aligned, no preparation; may be null when that is 0.  Enough for every call with the
 *                 same heads, page size and num_splits and as many rows and pages or fewer, on this
 *                 device.  Calls that share it must not overlap on the GPU
 *   num_splits, softmax_scale, roundings and errors otherwise as cai_kv4_decode, for the int8 cache, too
 *   (there a V scale below 2^-100, or below 2^-50 of the largest of the list's, may count as that: the output is off by
 *   2^-93, or by 2^-50 of the largest |V|, at most). */
size_t cai_kv_attend_pages_workspace_size(int32_t rows, int32_t num_q_heads, int32_t num_kv_heads, int32_t width,
                                          int32_t page_size, int32_t num_splits);
cai_status cai_kv_attend_pages(const cai_kv_pool* kv_pools, int32_t num_kv_heads, const uint16_t* q, int32_t rows,
                               int32_t num_q_heads, const int32_t* pages, int32_t width, const int32_t* len,
                               float softmax_scale, int32_t num_splits, void* workspace, size_t workspace_bytes,
                               uint16_t* out, float* lse_out, int32_t* err_flag, void* stream);
size_t cai_kv4_attend_pages_workspace_size(int32_t rows, int32_t num_q_heads, int32_t num_kv_heads, int32_t width,
                                           int32_t page_size, int32_t num_splits);
cai_status cai_kv4_attend_pages(const cai_kv4_pool* kv_pools, int32_t num_kv_heads, const uint16_t* q, int32_t rows,
                                int32_t num_q_heads, const int32_t* pages, int32_t width, const int32_t* len,
                                float softmax_scale, int32_t num_splits, void* workspace, size_t workspace_bytes,
                                uint16_t* out, float* lse_out, int32_t* err_flag, void* stream);

/* ---- Cross-turn KV cache in host memory ----------------------------------
 * "Character.AI: inference optimization", 04 Cache between turns: the KV of
 * every processed prefix and generated message is kept in host memory in an
 * LRU cache with a tree structure, indexed by a rolling hash of the prefix
 * tokens; a query retrieves the longest matching prefix.  Here the tree's
 * edges are whole pages (page_size tokens, all KV buffers of a layer stack);
 * matches are confirmed token by token, so hash collisions cannot return the
 * wrong KV; eviction removes the least recently used leaf.  Restored pages are
 * byte-identical to the stored ones.  The cache owns a host arena of
 * capacity_pages * num_buffers * cai_page_bytes() bytes (pinned when a GPU is
 * present).  Calls on one cache are serialised by a mutex. */
typedef struct cai_host_cache cai_host_cache;

/* NULL on bad arguments or when the arena cannot be allocated. */
cai_host_cache* cai_host_cache_create(int32_t page_size, int32_t head_dim, int32_t num_buffers,
                                      int64_t capacity_pages);
void cai_host_cache_destroy(cai_host_cache* cache);

/* Tokens of the longest cached prefix of tokens[0, n_tokens): a multiple of page_size
 * (0 on a miss).  Marks the matched path as recently used. */
int32_t cai_host_cache_match(cai_host_cache* cache, const int32_t* tokens, int32_t n_tokens);

/* Copy the cached pages of tokens[0, n_tokens) (n_tokens a multiple of page_size, all
 * cached) into pages block_table_row[0 .. n_tokens/page_size) of each of the num_buffers
 * pools.  block_table_row and pools are host arrays; pools[i].pages may be device or
 * host memory.  Device copies are asynchronous on `stream`: a copy kernel reads the
 * pinned host arena directly (the arena must stay alive until they are done). */
cai_status cai_host_cache_restore(cai_host_cache* cache, const int32_t* tokens, int32_t n_tokens,
                                  const cai_kv_pool* pools, const int32_t* block_table_row, void* stream);

/* cai_host_cache_restore for several sequences at once (a scheduler resuming a batch of
 * dialogues): sequence i copies its cached pages of tokens[i][0, n_tokens[i]) into pages
 * block_table_rows[i][...] of each pool.  tokens, n_tokens and block_table_rows are host
 * arrays [num_seqs]; every path is checked before anything is copied (CAI_ERR_INVALID_ARG
 * when one is not fully cached).  The device copies of all the sequences are queued on
 * `stream` together (one copy kernel per 1024 pages). */
cai_status cai_host_cache_restore_batch(cai_host_cache* cache, int32_t num_seqs, const int32_t* const* tokens,
                                        const int32_t* n_tokens, const cai_kv_pool* pools,
                                        const int32_t* const* block_table_rows, void* stream);

/* Keep the full pages of tokens[0, n_tokens) (a trailing partial page is ignored), read
 * from pages block_table_row[...] of each pool; pages already cached are not copied
 * again.  Evicts least recently used leaves when the arena is full; returns
 * CAI_ERR_WORKSPACE if the path alone does not fit.  Returns after the copies are done. */
cai_status cai_host_cache_store(cai_host_cache* cache, const int32_t* tokens, int32_t n_tokens,
                                const cai_kv_pool* pools, const int32_t* block_table_row, void* stream);

/* Counters: matches with at least one page, matches with none, pages held, evictions. */
void cai_host_cache_stats(cai_host_cache* cache, int64_t* hits, int64_t* misses, int64_t* pages_cached,
                          int64_t* evictions);

/* ---- Local-window page recycling.
 * A local layer attends only the last `window` positions ("Character.AI: inference
 * optimization", section 03, hybrid attention with a 1024-token horizon), so a buffer
 * read only by local layers needs to keep just the pages of that window.  It can hold
 * each sequence in a ring of pages: logical page k of the sequence lives in ring slot
 * k % ring.  The kernels read no page outside the call's own range: decode reads the
 * pages of [ctx_len - window, ctx_len), prefill those of
 * [max(0, prefix + 1 - window), prefix + n_new), append those it writes.  (The pages
 * describe the horizon but not how freed memory is reused; this ring is that reuse.) */

/* Ring length (pages per sequence) for a local buffer read with `window` and written at
 * most `max_new_tokens` positions per call (1 for decode, the chunk length for prefill):
 * ceil((window + max_new_tokens - 1) / page_size) + 1.  0 for invalid arguments
 * (window < 1, max_new_tokens < 1, page_size < 1). */
int32_t cai_ring_pages(int32_t window, int32_t page_size, int32_t max_new_tokens);

/* Fill one host block-table row for a sequence whose positions [0, hi) are written
 * (hi includes the tokens of the coming call): the last `ring` pages before
 * ceil(hi / page_size) map to ring_ids[k % ring]; every other entry is -1, so that a
 * kernel reading a freed or unwritten page sets CAI_DEVERR_PAGE instead of reading
 * another position's data.  row: host int32 [max_pages_per_seq]; ring_ids: host int32
 * [ring], distinct page ids of the buffer's pool.  Returns CAI_ERR_INVALID_ARG for null
 * pointers, ring < 1, page_size < 1, hi < 0 or ceil(hi / page_size) > max_pages_per_seq. */
cai_status cai_ring_table_row(int32_t* row, int32_t max_pages_per_seq, const int32_t* ring_ids, int32_t ring,
                              int32_t hi, int32_t page_size);

/* Limit, in nanoseconds, of every bounded wait inside the kernels: of decode, prefill,
 * attention over lists of pages and the selection's scores (process-wide, read at each launch; 0 restores the default of 2 s; a wait checks its
 * clock after each suspension of up to 1 ms, so shorter limits act as about 1 ms).  A
 * CTA whose wait runs out sets CAI_DEVERR_TIMEOUT, stops its work, waits for its own
 * copies and tensor-core operations in flight, frees its tensor memory and returns;
 * that launch's outputs are unspecified.  One wait has a limit of 2 s at least: that of
 * the warp that works out items ahead in packed prefill calls and in the 4-bit prefill,
 * which waits for whole items and ends as soon as another wait has given up.  A short
 * limit is for failure-detection tests; a serving process leaves the default. */
void cai_set_wait_limit_ns(uint64_t ns);

/* Fault injection for failure-detection tests (process-wide, read at each launch;
 * -1, the default, turns it off).  With stage = n >= 0, every CTA of the following
 * decode launches skips the load of its n-th K/V stage (64 tokens; over the 4-bit cache
 * its n-th tile of 128 keys, or, up to 8 heads per K/V head, each warp its n-th step of 32),
 * every CTA of the following launches of attention over lists that of the n-th tile of
 * 128 keys in each of its two halves (4-bit, up to 8 heads per K/V head: as the decode),
 * and every CTA of the following prefill launches that of its n-th K tile (128 keys); a
 * CTA of the selection's scores does not hear of its products with the n-th tile of 128
 * pages.  The waits for them run out after the wait limit and the launch reports
 * CAI_DEVERR_TIMEOUT.  Nothing faults: the load is simply never issued.  A CTA with
 * fewer stages than n + 1 is not affected. */
void cai_set_fault_injection(int32_t stage);

/* The CUDA runtime's description of the error behind the last CAI_ERR_CUDA returned on
 * this thread ("no error" if none). */
const char* cai_last_cuda_error(void);

/* Static description of a status code. */
const char* cai_status_string(cai_status status);

#ifdef __cplusplus
}
#endif

#endif /* CAI_H_ */

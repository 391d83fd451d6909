// Entry points of the row calls (rotated append, read) on both caches and of the attention over the
// 4-bit cache: argument validation, split planning and launches.
#include <cmath>
#include <cstdint>

#include "entry.cuh"
#include "kv4.cuh"

using namespace cai;

namespace {

constexpr int32_t kMaxAxes = 4;

// Positions on several axes (num 0: none).
struct Axes {
  const uint8_t* axis;
  int32_t num;
  const int32_t* positions;
};

template <class Pool>
cai_status append_rows(const Pool* pools, int32_t num_kv_heads, const cai_rope* rope, const Axes& axes, const void* k_new,
                       const void* v_new, cai_dtype kv_type, int64_t k_stride, int64_t v_stride, const uint16_t* q,
                       int64_t q_stride, uint16_t* q_out, int32_t num_q_heads, int32_t batch, int32_t n_new,
                       const int32_t* q_offsets, int32_t total_new, const int32_t* block_table,
                       int32_t max_pages_per_seq, const int32_t* start_pos, int32_t* err_flag, bool four,
                       void* stream) {
  cai_status st = check_pools(pools, num_kv_heads);
  if (st != CAI_OK) return st;
  if (!dtype_ok(kv_type) || num_q_heads < 0) return CAI_ERR_INVALID_ARG;
  if (num_q_heads > 1024) return CAI_ERR_UNSUPPORTED;
  int64_t rows;
  st = check_rows(batch, n_new, q_offsets, total_new, max_pages_per_seq, pools[0].page_size, &rows);
  if (st != CAI_OK) return st;
  AppendRowsParams p = {};
  if (rope) {
    if (rope->rot_dim < 2 || rope->rot_dim > kHeadDim || rope->rot_dim % 2 != 0) return CAI_ERR_UNSUPPORTED;
    if (!rope->cos || !rope->sin || rope->num_positions <= 0) return CAI_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(rope->cos) | reinterpret_cast<uintptr_t>(rope->sin)) & 3u) return CAI_ERR_INVALID_ARG;
    p.cos = rope->cos;
    p.sin = rope->sin;
    p.num_positions = rope->num_positions;
    p.rot = rope->rot_dim;
    p.interleaved = rope->interleaved != 0;
  }
  if (axes.num > 0) {
    for (int i = 0; i < p.rot / 2; ++i) {
      if (axes.axis[i] >= axes.num) return CAI_ERR_INVALID_ARG;
      p.axis_bits[i / 16] |= (uint32_t)axes.axis[i] << (2 * (i % 16));
    }
    p.num_axes = axes.num;
    p.positions = axes.positions;
  }
  const int64_t quantum = kv_type == CAI_FP32 ? 4 : 8;  // elements of 16 bytes
  const int64_t width = (int64_t)num_kv_heads * kHeadDim;
  if (k_stride < width || v_stride < width || k_stride % quantum || v_stride % quantum) return CAI_ERR_INVALID_ARG;
  if (num_q_heads > 0) {
    if (!rope || q_stride < (int64_t)num_q_heads * kHeadDim || q_stride % 8) return CAI_ERR_INVALID_ARG;
  } else if (q || q_out) {
    return CAI_ERR_INVALID_ARG;
  }
  if (rows == 0) return CAI_OK;
  if (!k_new || !v_new || !block_table || !start_pos) return CAI_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new)) return CAI_ERR_INVALID_ARG;
  if (axes.num > 0 && (!axes.positions || (reinterpret_cast<uintptr_t>(axes.positions) & 3u))) return CAI_ERR_INVALID_ARG;
  if (num_q_heads > 0) {
    if (!q || !q_out || !aligned16(q) || !aligned16(q_out)) return CAI_ERR_INVALID_ARG;
    if (q == q_out && q_stride != (int64_t)num_q_heads * kHeadDim) return CAI_ERR_INVALID_ARG;
  }
  fill_pools(pools, num_kv_heads, p);
  p.num_q_heads = num_q_heads;
  p.max_pages = max_pages_per_seq;
  p.batch = batch;
  p.n_new = n_new;
  p.total_new = total_new;
  p.q_off = q_offsets;
  p.table = block_table;
  p.start_pos = start_pos;
  p.k = k_new;
  p.v = v_new;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_stride = q_stride;
  p.q = q;
  p.q_out = q_out;
  p.err = err_flag;
  return cuda_status(launch_append_rows(p, four, kv_type == CAI_BF16, static_cast<cudaStream_t>(stream)));
}

template <class Pool>
cai_status read_rows(const Pool* pools, int32_t num_kv_heads, void* k_out, void* v_out, cai_dtype out_type,
                     int32_t batch, int32_t n_new, const int32_t* q_offsets, int32_t total_new,
                     const int32_t* block_table, int32_t max_pages_per_seq, const int32_t* start_pos,
                     int32_t* err_flag, bool four, void* stream) {
  cai_status st = check_pools(pools, num_kv_heads);
  if (st != CAI_OK) return st;
  if (!dtype_ok(out_type)) return CAI_ERR_INVALID_ARG;
  int64_t rows;
  st = check_rows(batch, n_new, q_offsets, total_new, max_pages_per_seq, pools[0].page_size, &rows);
  if (st != CAI_OK || rows == 0) return st;
  if ((!k_out && !v_out) || !block_table || !start_pos) return CAI_ERR_INVALID_ARG;
  if (!aligned16(k_out) || !aligned16(v_out)) return CAI_ERR_INVALID_ARG;
  ReadRowsParams p = {};
  fill_pools(pools, num_kv_heads, p);
  p.max_pages = max_pages_per_seq;
  p.batch = batch;
  p.n_new = n_new;
  p.total_new = total_new;
  p.q_off = q_offsets;
  p.table = block_table;
  p.start_pos = start_pos;
  p.k_out = k_out;
  p.v_out = v_out;
  p.err = err_flag;
  return cuda_status(launch_read_rows(p, four, out_type == CAI_BF16, static_cast<cudaStream_t>(stream)));
}

// A prefill workspace: the prefill kernel's part, then that of the decode launch of a packed call (whatever
// its window, which only shortens the ranges).
size_t prefill4_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads, int32_t max_pages_per_seq,
                      int32_t page_size) {
  Decode4Params d = {};
  d.num_heads = num_q_heads;
  d.num_kv_heads = num_kv_heads;
  d.batch = batch;
  d.page_size = page_size;
  d.max_pages = max_pages_per_seq;
  return prefill_workspace_bytes(batch * num_kv_heads, max_pages_per_seq, page_size) + plan_decode4(d, 0);
}

}  // namespace

extern "C" {

size_t cai_kv4_page_bytes(int32_t page_size, int32_t head_dim) {
  if (page_size <= 0 || head_dim <= 0 || page_size % kBlk != 0 || head_dim % 32 != 0) return 0;
  return (size_t)page_size * ((size_t)head_dim + head_dim / 8);
}

cai_status cai_kv_append_rope(const cai_kv_pool* kv_pools, int32_t num_kv_heads, const cai_rope* rope,
                              const void* k_new, const void* v_new, cai_dtype kv_type, int64_t k_stride,
                              int64_t v_stride, const uint16_t* q, int64_t q_stride, uint16_t* q_out,
                              int32_t num_q_heads, int32_t batch, int32_t n_new, const int32_t* q_offsets,
                              int32_t total_new, const int32_t* block_table, int32_t max_pages_per_seq,
                              const int32_t* start_pos, int32_t* err_flag, void* stream) {
  return append_rows(kv_pools, num_kv_heads, rope, Axes{}, k_new, v_new, kv_type, k_stride, v_stride, q, q_stride, q_out,
                     num_q_heads, batch, n_new, q_offsets, total_new, block_table, max_pages_per_seq, start_pos,
                     err_flag, false, stream);
}

cai_status cai_kv4_append(const cai_kv4_pool* kv_pools, int32_t num_kv_heads, const cai_rope* rope,
                          const void* k_new, const void* v_new, cai_dtype kv_type, int64_t k_stride,
                          int64_t v_stride, const uint16_t* q, int64_t q_stride, uint16_t* q_out,
                          int32_t num_q_heads, int32_t batch, int32_t n_new, const int32_t* q_offsets,
                          int32_t total_new, const int32_t* block_table, int32_t max_pages_per_seq,
                          const int32_t* start_pos, int32_t* err_flag, void* stream) {
  return append_rows(kv_pools, num_kv_heads, rope, Axes{}, k_new, v_new, kv_type, k_stride, v_stride, q, q_stride, q_out,
                     num_q_heads, batch, n_new, q_offsets, total_new, block_table, max_pages_per_seq, start_pos,
                     err_flag, true, stream);
}

cai_status cai_kv_append_rope_axes(const cai_kv_pool* kv_pools, int32_t num_kv_heads, const cai_rope* rope,
                     const uint8_t* axis, int32_t num_axes, const int32_t* positions, const void* k_new,
                     const void* v_new, cai_dtype kv_type, int64_t k_stride, int64_t v_stride, const uint16_t* q,
                     int64_t q_stride, uint16_t* q_out, int32_t num_q_heads, int32_t batch, int32_t n_new,
                     const int32_t* q_offsets, int32_t total_new, const int32_t* block_table,
                     int32_t max_pages_per_seq, const int32_t* start_pos, int32_t* err_flag, void* stream) {
  if (!rope || !axis) return CAI_ERR_INVALID_ARG;
  if (num_axes < 1 || num_axes > kMaxAxes) return CAI_ERR_UNSUPPORTED;
  return append_rows(kv_pools, num_kv_heads, rope, Axes{axis, num_axes, positions}, k_new, v_new, kv_type, k_stride,
                     v_stride, q, q_stride, q_out, num_q_heads, batch, n_new, q_offsets, total_new, block_table,
                     max_pages_per_seq, start_pos, err_flag, false, stream);
}

cai_status cai_kv4_append_axes(const cai_kv4_pool* kv_pools, int32_t num_kv_heads, const cai_rope* rope,
                     const uint8_t* axis, int32_t num_axes, const int32_t* positions, const void* k_new,
                     const void* v_new, cai_dtype kv_type, int64_t k_stride, int64_t v_stride, const uint16_t* q,
                     int64_t q_stride, uint16_t* q_out, int32_t num_q_heads, int32_t batch, int32_t n_new,
                     const int32_t* q_offsets, int32_t total_new, const int32_t* block_table,
                     int32_t max_pages_per_seq, const int32_t* start_pos, int32_t* err_flag, void* stream) {
  if (!rope || !axis) return CAI_ERR_INVALID_ARG;
  if (num_axes < 1 || num_axes > kMaxAxes) return CAI_ERR_UNSUPPORTED;
  return append_rows(kv_pools, num_kv_heads, rope, Axes{axis, num_axes, positions}, k_new, v_new, kv_type, k_stride,
                     v_stride, q, q_stride, q_out, num_q_heads, batch, n_new, q_offsets, total_new, block_table,
                     max_pages_per_seq, start_pos, err_flag, true, stream);
}

cai_status cai_kv_read(const cai_kv_pool* kv_pools, int32_t num_kv_heads, void* k_out, void* v_out,
                       cai_dtype out_type, int32_t batch, int32_t n_new, const int32_t* q_offsets,
                       int32_t total_new, const int32_t* block_table, int32_t max_pages_per_seq,
                       const int32_t* start_pos, int32_t* err_flag, void* stream) {
  return read_rows(kv_pools, num_kv_heads, k_out, v_out, out_type, batch, n_new, q_offsets, total_new, block_table,
                   max_pages_per_seq, start_pos, err_flag, false, stream);
}

cai_status cai_kv4_read(const cai_kv4_pool* kv_pools, int32_t num_kv_heads, void* k_out, void* v_out,
                        cai_dtype out_type, int32_t batch, int32_t n_new, const int32_t* q_offsets,
                        int32_t total_new, const int32_t* block_table, int32_t max_pages_per_seq,
                        const int32_t* start_pos, int32_t* err_flag, void* stream) {
  return read_rows(kv_pools, num_kv_heads, k_out, v_out, out_type, batch, n_new, q_offsets, total_new, block_table,
                   max_pages_per_seq, start_pos, err_flag, true, stream);
}

size_t cai_kv4_decode_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                     int32_t max_pages_per_seq, int32_t page_size, int32_t window,
                                     int32_t num_splits) {
  if (num_kv_heads < 1 || num_kv_heads > kMaxKvHeads || num_q_heads < 1 || num_q_heads % num_kv_heads != 0 ||
      num_q_heads / num_kv_heads > kMaxGroup || batch <= 0 || batch > 65535 || max_pages_per_seq <= 0 ||
      !page_size_ok(page_size) || (int64_t)max_pages_per_seq * page_size > (1ll << 30) || window < 0 ||
      num_splits < 0 || num_splits > kMaxSplits)
    return 0;
  Decode4Params p = {};
  p.num_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.batch = batch;
  p.page_size = page_size;
  p.max_pages = max_pages_per_seq;
  p.window = window;
  return plan_decode4(p, num_splits);
}

cai_status cai_kv4_decode(const cai_kv4_pool* kv_pools, int32_t num_kv_heads, const uint16_t* q, int32_t batch,
                          int32_t num_q_heads, const int32_t* block_table, int32_t max_pages_per_seq,
                          const int32_t* ctx_len, int32_t window, float softmax_scale, int32_t num_splits,
                          void* workspace, size_t workspace_bytes, uint16_t* out, float* lse_out,
                          int32_t* err_flag, void* stream) {
  const cai_status st = check_pools(kv_pools, num_kv_heads);
  if (st != CAI_OK) return st;
  if (batch < 0 || max_pages_per_seq <= 0 || window < 0 || num_splits < 0 || num_splits > kMaxSplits ||
      !std::isfinite(softmax_scale))
    return CAI_ERR_INVALID_ARG;
  if (num_q_heads < 1 || num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > kMaxGroup)
    return CAI_ERR_UNSUPPORTED;
  if ((int64_t)max_pages_per_seq * kv_pools[0].page_size > (1ll << 30) || batch > 65535) return CAI_ERR_UNSUPPORTED;
  if (batch == 0) return CAI_OK;
  if (!q || !block_table || !ctx_len || !out || !aligned16(q) || !aligned16(out)) return CAI_ERR_INVALID_ARG;
  Decode4Params p = {};
  fill_pools(kv_pools, num_kv_heads, p);
  p.num_heads = num_q_heads;
  p.batch = batch;
  p.max_pages = max_pages_per_seq;
  p.window = window;
  p.table = block_table;
  p.ctx_len = ctx_len;
  p.q = q;
  p.out = out;
  p.lse_out = lse_out;
  const size_t need = plan_decode4(p, num_splits);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned256(workspace))) return CAI_ERR_WORKSPACE;
  place_decode4(p, workspace);
  p.scale_log2 = softmax_scale * kLog2e;
  p.err = err_flag;
  p.wait_ns = wait_limit_ns();
  p.drop_stage = fault_drop_stage();
  return cuda_status(launch_decode4(p, static_cast<cudaStream_t>(stream)));
}

size_t cai_kv4_prefill_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                      int32_t max_pages_per_seq, int32_t page_size) {
  if (num_kv_heads < 1 || num_kv_heads > kMaxKvHeads || num_q_heads < 1 || num_q_heads % num_kv_heads != 0 ||
      batch <= 0 || batch > 65535 / num_kv_heads || max_pages_per_seq <= 0 || !page_size_ok(page_size) ||
      (int64_t)max_pages_per_seq * page_size > (1ll << 24))
    return 0;
  return prefill4_bytes(batch, num_q_heads, num_kv_heads, max_pages_per_seq, page_size);
}

cai_status cai_kv4_prefill(const cai_kv4_pool* kv_pools, int32_t num_kv_heads, const uint16_t* q, int32_t batch,
                           int32_t n_new, const int32_t* q_offsets, int32_t total_new, int32_t num_q_heads,
                           const int32_t* block_table, int32_t max_pages_per_seq, const int32_t* prefix_len,
                           int32_t window, float softmax_scale, void* workspace, size_t workspace_bytes,
                           uint16_t* out, float* lse_out, int32_t* err_flag, void* stream) {
  const cai_status st = check_pools(kv_pools, num_kv_heads);
  if (st != CAI_OK) return st;
  if (batch < 0 || n_new < 0 || (q_offsets && total_new < 0) || max_pages_per_seq <= 0 || window < 0 ||
      !std::isfinite(softmax_scale))
    return CAI_ERR_INVALID_ARG;
  const int32_t P = kv_pools[0].page_size;
  const int32_t group = num_q_heads > 0 && num_q_heads % num_kv_heads == 0 ? num_q_heads / num_kv_heads : 0;
  if (group < 1 || group > kMaxGroup || (group & (group - 1)) != 0) return CAI_ERR_UNSUPPORTED;
  if ((int64_t)max_pages_per_seq * P > (1ll << 24) || batch > 65535 / num_kv_heads) return CAI_ERR_UNSUPPORTED;
  const int64_t rows = batch == 0 || n_new == 0 ? 0 : q_offsets ? total_new : (int64_t)batch * n_new;
  if ((int64_t)n_new * group > (1ll << 24) || rows > (1ll << 31) / kHeadDim / num_q_heads) return CAI_ERR_UNSUPPORTED;
  // The kernel numbers its q-tiles in 32 bits, two per SM of slack for the pieces.
  if (ceil_div((int64_t)n_new * group, 128) * batch * num_kv_heads > (1ll << 30)) return CAI_ERR_UNSUPPORTED;
  if (rows == 0) return CAI_OK;
  if (!q || !block_table || !prefix_len || !out || !aligned16(q) || !aligned16(out)) return CAI_ERR_INVALID_ARG;
  const size_t need = prefill4_bytes(batch, num_q_heads, num_kv_heads, max_pages_per_seq, P);
  if (!workspace || workspace_bytes < need || !aligned256(workspace)) return CAI_ERR_WORKSPACE;
  PrefillLaunch L = {};
  L.four = true;
  for (int j = 0; j < num_kv_heads; ++j) {
    L.pages4[j] = static_cast<const uint8_t*>(kv_pools[j].pages);
    L.num_pages4[j] = kv_pools[j].num_pages;
  }
  L.num_kv_heads = num_kv_heads;
  L.q_heads = num_q_heads;
  L.num_heads = group;
  L.page_size = P;
  L.max_pages = max_pages_per_seq;
  L.table = block_table;
  L.prefix_len = prefix_len;
  L.q = q;
  L.q_off = q_offsets;
  L.batch = batch;
  L.n_new = n_new;
  L.total_new = (int32_t)rows;
  L.window = window;
  L.scale_log2 = softmax_scale * kLog2e;
  L.workspace = workspace;
  L.out16 = out;
  L.lse_out = lse_out;
  L.err = err_flag;
  // Packed rows: sequences with one new token are decode steps; the decode kernel takes them, launched
  // behind the prefill without waiting for it (disjoint output rows, and a part of the workspace of its own).
  L.skip_single = q_offsets != nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // One new token for every sequence: decode alone (64 sequences of 4000, 8 K/V heads: 71 us, through the copy
  // 380).
  const bool all_single = !q_offsets && n_new == 1;
  if (!all_single) {
    const cudaError_t e = launch_prefill(L, s);
    if (e != cudaSuccess || !L.skip_single) return cuda_status(e);
  }
  Decode4Params d = {};
  fill_pools(kv_pools, num_kv_heads, d);
  d.num_heads = num_q_heads;
  d.batch = batch;
  d.max_pages = max_pages_per_seq;
  d.window = window;
  d.table = block_table;
  d.ctx_len = prefix_len;
  d.before_new = 1;
  d.q_off = q_offsets;
  d.total_rows = (int32_t)rows;
  d.q = q;
  d.out = out;
  d.lse_out = lse_out;
  plan_decode4(d, 0);
  place_decode4(d, static_cast<uint8_t*>(workspace) + prefill_workspace_bytes(batch * num_kv_heads, max_pages_per_seq, P));
  d.scale_log2 = L.scale_log2;
  d.err = err_flag;
  d.wait_ns = wait_limit_ns();
  d.drop_stage = fault_drop_stage();
  d.overlap_prev = !all_single;
  return cuda_status(launch_decode4(d, s));
}

}  // extern "C"

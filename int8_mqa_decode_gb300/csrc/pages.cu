// Entry points of the long-context operators: page summaries, the selection of pages and attention over lists of
// pages.  Argument checks and launches.
#include <cmath>
#include <cstdint>

#include "entry.cuh"

using namespace cai;

namespace {

cai_status check_summaries(const cai_kv_summary* summaries, int32_t num_kv_heads) {
  if (!summaries) return CAI_ERR_INVALID_ARG;
  if (num_kv_heads < 1 || num_kv_heads > kMaxKvHeads) return CAI_ERR_UNSUPPORTED;
  for (int j = 0; j < num_kv_heads; ++j) {
    if (!summaries[j].data || summaries[j].num_pages <= 0 || !aligned16(summaries[j].data)) return CAI_ERR_INVALID_ARG;
    if (summaries[j].head_dim != kHeadDim || !page_size_ok(summaries[j].page_size)) return CAI_ERR_UNSUPPORTED;
    if (summaries[j].page_size != summaries[0].page_size) return CAI_ERR_INVALID_ARG;
  }
  return CAI_OK;
}

template <class Pool>
cai_status summarize(const Pool* pools, const cai_kv_summary* summaries, int32_t num_kv_heads, int32_t batch,
                     int32_t n_new, const int32_t* q_offsets, const int32_t* block_table, int32_t max_pages_per_seq,
                     const int32_t* start_pos, int32_t* err_flag, bool four, void* stream) {
  cai_status st = check_pools(pools, num_kv_heads);
  if (st == CAI_OK) st = check_summaries(summaries, num_kv_heads);
  if (st != CAI_OK) return st;
  for (int j = 0; j < num_kv_heads; ++j)
    if (summaries[j].num_pages != pools[j].num_pages || summaries[j].page_size != pools[j].page_size)
      return CAI_ERR_INVALID_ARG;
  int64_t rows;
  // (Packed, n_new may be a loose bound: the rows that a call may have, not batch * n_new, are limited.)
  st = check_rows(batch, n_new, q_offsets, 1 << 30, max_pages_per_seq, pools[0].page_size, &rows);
  if (st != CAI_OK || rows == 0) return st;
  if (!block_table || !start_pos) return CAI_ERR_INVALID_ARG;
  SummarizeParams p = {};
  for (int j = 0; j < num_kv_heads; ++j) {
    p.pages[j] = static_cast<const uint8_t*>(pools[j].pages);
    p.num_pages[j] = pools[j].num_pages;
    p.data[j] = static_cast<uint8_t*>(summaries[j].data);
  }
  p.num_kv_heads = num_kv_heads;
  p.page_size = pools[0].page_size;
  p.max_pages = max_pages_per_seq;
  p.batch = batch;
  p.n_new = n_new;
  p.total_new = 2147483647;  // no rows are read: the offsets count new tokens
  p.q_off = q_offsets;
  p.table = block_table;
  p.start_pos = start_pos;
  p.err = err_flag;
  return cuda_status(launch_summarize(p, four, static_cast<cudaStream_t>(stream)));
}

// Attention over lists of pages is a decode step whose tables have a row for every K/V head and hold the listed pages
// alone; its sequences are the call's rows.
size_t attend_bytes(int32_t rows, int32_t num_q_heads, int32_t num_kv_heads, int32_t width, int32_t page_size,
                    int32_t num_splits, bool eight) {
  if (num_kv_heads < 1 || num_kv_heads > kMaxKvHeads || num_q_heads < 1 || num_q_heads % num_kv_heads != 0 ||
      num_q_heads / num_kv_heads > kMaxGroup || rows <= 0 || rows > 65535 || width <= 0 || !page_size_ok(page_size) ||
      (int64_t)width * page_size > (1ll << 30) || num_splits < 0 || num_splits > kMaxSplits)
    return 0;
  Decode4Params p = {};
  p.num_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.batch = rows;
  p.page_size = page_size;
  p.max_pages = width;
  p.lists = 1;
  p.eight = eight;
  return most_list_bytes(p, num_splits);
}

template <class Pool>
cai_status attend_pages(const Pool* kv_pools, int32_t num_kv_heads, const uint16_t* q, int32_t rows,
                        int32_t num_q_heads, const int32_t* pages, int32_t width, const int32_t* len,
                        float softmax_scale, int32_t num_splits, void* workspace, size_t workspace_bytes,
                        uint16_t* out, float* lse_out, int32_t* err_flag, bool eight, void* stream) {
  const cai_status st = check_pools(kv_pools, num_kv_heads);
  if (st != CAI_OK) return st;
  if (rows < 0 || width <= 0 || num_splits < 0 || num_splits > kMaxSplits || !std::isfinite(softmax_scale))
    return CAI_ERR_INVALID_ARG;
  if (num_q_heads < 1 || num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > kMaxGroup)
    return CAI_ERR_UNSUPPORTED;
  if ((int64_t)width * kv_pools[0].page_size > (1ll << 30) || rows > 65535) return CAI_ERR_UNSUPPORTED;
  if (rows == 0) return CAI_OK;
  if (!q || !pages || !len || !out || !aligned16(q) || !aligned16(out)) return CAI_ERR_INVALID_ARG;
  Decode4Params p = {};
  fill_pools(kv_pools, num_kv_heads, p);
  p.num_heads = num_q_heads;
  p.batch = rows;
  p.max_pages = width;
  p.table = pages;
  p.lists = 1;
  p.eight = eight;
  p.ctx_len = len;
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

}  // namespace

extern "C" {

size_t cai_kv_summary_bytes(int32_t num_pages, int32_t head_dim) {
  if (num_pages <= 0 || head_dim <= 0) return 0;
  return (size_t)num_pages * (2 * (size_t)head_dim + 4);
}

cai_status cai_kv_summarize(const cai_kv_pool* kv_pools, const cai_kv_summary* summaries, int32_t num_kv_heads,
                            int32_t batch, int32_t n_new, const int32_t* q_offsets, const int32_t* block_table,
                            int32_t max_pages_per_seq, const int32_t* start_pos, int32_t* err_flag, void* stream) {
  return summarize(kv_pools, summaries, num_kv_heads, batch, n_new, q_offsets, block_table, max_pages_per_seq,
                   start_pos, err_flag, false, stream);
}

cai_status cai_kv4_summarize(const cai_kv4_pool* kv_pools, const cai_kv_summary* summaries, int32_t num_kv_heads,
                             int32_t batch, int32_t n_new, const int32_t* q_offsets, const int32_t* block_table,
                             int32_t max_pages_per_seq, const int32_t* start_pos, int32_t* err_flag, void* stream) {
  return summarize(kv_pools, summaries, num_kv_heads, batch, n_new, q_offsets, block_table, max_pages_per_seq,
                   start_pos, err_flag, true, stream);
}

size_t cai_kv_select_workspace_size(int32_t batch, int32_t total_rows, int32_t num_q_heads, int32_t num_kv_heads,
                                    int32_t max_pages_per_seq) {
  if (batch <= 0 || batch > 65535 || total_rows < 0 || num_kv_heads < 1 || num_kv_heads > kMaxKvHeads ||
      num_q_heads < 1 || num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > kMaxGroup ||
      max_pages_per_seq <= 0)
    return 0;
  return (size_t)total_rows * num_kv_heads * score_stride(max_pages_per_seq) * sizeof(float);
}

cai_status cai_kv_select(const cai_kv_summary* summaries, int32_t num_kv_heads, const uint16_t* q, int32_t batch,
                         int32_t n_new, const int32_t* q_offsets, int32_t total_new, int32_t num_q_heads,
                         const int32_t* block_table, int32_t max_pages_per_seq, const int32_t* start_pos,
                         int32_t num_selected, int32_t first, int32_t last, void* workspace, size_t workspace_bytes,
                         int32_t* pages_out, int32_t* len_out, int32_t* err_flag, void* stream) {
  cai_status st = check_summaries(summaries, num_kv_heads);
  if (st != CAI_OK) return st;
  if (first < 0 || last < 1 || num_selected < 1 || (int64_t)first + last > num_selected) return CAI_ERR_INVALID_ARG;
  if (num_q_heads < 1 || num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > kMaxGroup)
    return CAI_ERR_UNSUPPORTED;
  int64_t rows;
  st = check_rows(batch, n_new, q_offsets, total_new, max_pages_per_seq, summaries[0].page_size, &rows);
  if (st != CAI_OK) return st;
  if ((int64_t)num_selected * summaries[0].page_size > (1ll << 30)) return CAI_ERR_UNSUPPORTED;
  if ((rows + batch) * num_kv_heads > 2147483647ll) return CAI_ERR_UNSUPPORTED;  // blocks of a launch
  if (rows == 0) return CAI_OK;
  if (!q || !block_table || !start_pos || !pages_out || !len_out || !aligned16(q)) return CAI_ERR_INVALID_ARG;
  const size_t need = cai_kv_select_workspace_size(batch, (int32_t)rows, num_q_heads, num_kv_heads, max_pages_per_seq);
  if (!workspace || workspace_bytes < need || !aligned256(workspace)) return CAI_ERR_WORKSPACE;
  SelectParams p = {};
  for (int j = 0; j < num_kv_heads; ++j) {
    p.data[j] = static_cast<const uint8_t*>(summaries[j].data);
    p.num_pages[j] = summaries[j].num_pages;
  }
  p.num_kv_heads = num_kv_heads;
  p.num_q_heads = num_q_heads;
  p.page_size = summaries[0].page_size;
  p.max_pages = max_pages_per_seq;
  p.batch = batch;
  p.n_new = n_new;
  p.total_new = total_new;
  p.q_off = q_offsets;
  p.table = block_table;
  p.start_pos = start_pos;
  p.q = q;
  p.keep = num_selected;
  p.first = first;
  p.last = last;
  p.scores = static_cast<float*>(workspace);
  p.stride = score_stride(max_pages_per_seq);
  p.pages_out = pages_out;
  p.len_out = len_out;
  p.err = err_flag;
  p.wait_ns = wait_limit_ns();
  p.drop_stage = fault_drop_stage();
  return cuda_status(launch_select(p, static_cast<cudaStream_t>(stream)));
}

size_t cai_kv_attend_pages_workspace_size(int32_t rows, int32_t num_q_heads, int32_t num_kv_heads, int32_t width,
                                          int32_t page_size, int32_t num_splits) {
  return attend_bytes(rows, num_q_heads, num_kv_heads, width, page_size, num_splits, true);
}

cai_status cai_kv_attend_pages(const cai_kv_pool* kv_pools, int32_t num_kv_heads, const uint16_t* q, int32_t rows,
                               int32_t num_q_heads, const int32_t* pages, int32_t width, const int32_t* len,
                               float softmax_scale, int32_t num_splits, void* workspace, size_t workspace_bytes,
                               uint16_t* out, float* lse_out, int32_t* err_flag, void* stream) {
  return attend_pages(kv_pools, num_kv_heads, q, rows, num_q_heads, pages, width, len, softmax_scale, num_splits,
                      workspace, workspace_bytes, out, lse_out, err_flag, true, stream);
}

size_t cai_kv4_attend_pages_workspace_size(int32_t rows, int32_t num_q_heads, int32_t num_kv_heads, int32_t width,
                                          int32_t page_size, int32_t num_splits) {
  return attend_bytes(rows, num_q_heads, num_kv_heads, width, page_size, num_splits, false);
}

cai_status cai_kv4_attend_pages(const cai_kv4_pool* kv_pools, int32_t num_kv_heads, const uint16_t* q, int32_t rows,
                               int32_t num_q_heads, const int32_t* pages, int32_t width, const int32_t* len,
                               float softmax_scale, int32_t num_splits, void* workspace, size_t workspace_bytes,
                               uint16_t* out, float* lse_out, int32_t* err_flag, void* stream) {
  return attend_pages(kv_pools, num_kv_heads, q, rows, num_q_heads, pages, width, len, softmax_scale, num_splits,
                      workspace, workspace_bytes, out, lse_out, err_flag, false, stream);
}

}  // extern "C"

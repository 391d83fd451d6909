// Argument checks that the entry points over one pool per K/V head share.
#pragma once
#include "common.cuh"

namespace cai {

constexpr int32_t kMaxGroup = 128;  // query heads per K/V head

inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The pools of one call (cai_kv_pool and cai_kv4_pool have the same fields).
template <class Pool>
cai_status check_pools(const Pool* pools, int32_t num_kv_heads) {
  if (!pools) return CAI_ERR_INVALID_ARG;
  if (num_kv_heads < 1 || num_kv_heads > kMaxKvHeads) return CAI_ERR_UNSUPPORTED;
  for (int j = 0; j < num_kv_heads; ++j) {
    if (!pools[j].pages || pools[j].num_pages <= 0 || !aligned16(pools[j].pages)) return CAI_ERR_INVALID_ARG;
    if (pools[j].head_dim != kHeadDim || !page_size_ok(pools[j].page_size)) return CAI_ERR_UNSUPPORTED;
    if (pools[j].page_size != pools[0].page_size) return CAI_ERR_INVALID_ARG;
  }
  return CAI_OK;
}

// Rows, table and positions of one call; *rows = 0: nothing to do.
inline cai_status check_rows(int32_t batch, int32_t n_new, const int32_t* q_offsets, int32_t total_new,
                      int32_t max_pages_per_seq, int32_t page_size, int64_t* rows) {
  *rows = 0;
  if (batch < 0 || n_new < 0 || max_pages_per_seq <= 0 || (q_offsets && total_new < 0)) return CAI_ERR_INVALID_ARG;
  if ((int64_t)max_pages_per_seq * page_size > (1ll << 30) || batch > 65535) return CAI_ERR_UNSUPPORTED;
  const int64_t r = batch == 0 || n_new == 0 ? 0 : q_offsets ? total_new : (int64_t)batch * n_new;
  if (r > (1ll << 30) || n_new > (1 << 22)) return CAI_ERR_UNSUPPORTED;
  *rows = r;
  return CAI_OK;
}

template <class Pool, class Params>
void fill_pools(const Pool* pools, int32_t num_kv_heads, Params& p) {
  for (int j = 0; j < kMaxKvHeads; ++j) {
    p.pages[j] = j < num_kv_heads ? static_cast<uint8_t*>(pools[j].pages) : nullptr;
    p.num_pages[j] = j < num_kv_heads ? pools[j].num_pages : 0;
  }
  p.num_kv_heads = num_kv_heads;
  p.page_size = pools[0].page_size;
}

inline bool dtype_ok(cai_dtype t) { return t == CAI_FP32 || t == CAI_BF16; }

}  // namespace cai

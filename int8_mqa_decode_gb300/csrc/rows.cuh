// New-token rows of a call, whichever sequence they belong to: packed by offsets, or n_new per sequence.
#pragma once
#include "common.cuh"

namespace cai {

// New tokens of sequence b: rows [r0, r0 + n); n = -1 when its offsets are out of order, past the
// packed rows or more than n_new.
struct NewRows {
  int64_t r0;
  int n;
};
template <class Params>
__device__ __forceinline__ NewRows new_rows(const Params& p, int b) {
  if (!p.q_off) return NewRows{(int64_t)b * p.n_new, p.n_new};
  const int32_t a = p.q_off[b], e = p.q_off[b + 1];
  const bool ok = a >= 0 && a <= e && e <= p.total_new && e - a <= p.n_new;
  return NewRows{a, ok ? e - a : -1};
}

// x / y for x >= 0, y > 0, in 32 bits where that is enough; and the places of a position that is not negative.
// (A decode step of four sequences takes 5.2 us with its read, with 64-bit divisions 5.4.)
__device__ __forceinline__ int64_t over(int64_t x, int32_t y) {
  return x >> 32 ? x / y : (int64_t)((uint32_t)x / (uint32_t)y);
}
__device__ __forceinline__ int page_log2(int P) { return P == 16 ? 4 : P == 32 ? 5 : 6; }

// The sequence that packed row `row` belongs to (its rows [*a, *e)), by a search of 32 offsets at a
// time; -1 past the last.  Offsets that decrease are flagged elsewhere; here they may lose a row.
__device__ __forceinline__ int find_seq(const int32_t* off, int batch, int64_t row, int lane, int32_t* a, int32_t* e) {
  int lo = 0, n = batch + 1;  // the last offset <= row lies in [lo, lo + n)
  int32_t mine = 0;
  while (true) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    mine = lane * step < n ? off[at] : 2147483647;
    const uint32_t m = __ballot_sync(0xffffffffu, lane * step < n && mine <= row);
    if (m == 0) return -1;
    const int k = 31 - __clz(m);
    lo += k * step;
    if (step == 1) {
      if (lo >= batch) return -1;
      *a = __shfl_sync(0xffffffffu, mine, k);
      *e = off[lo + 1];
      return lo;
    }
    n = min(step, n - k * step);
  }
}

}  // namespace cai

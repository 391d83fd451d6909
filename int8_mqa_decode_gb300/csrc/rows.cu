// Rows in and out of the paged caches: rotate-quantise-append (int8 and 4-bit pages), and reading
// cached rows back as values.
//
// Append.  Token i of sequence b goes to position start_pos[b] + i.  With a rotation, channels pair up
// (i with i + rot/2, or 2 i with 2 i + 1) and (a, b) becomes (a c - b s, b c + a s), c and s being the
// position's row of the caller's tables; every product and sum is rounded to fp32 on its own, so the
// codes do not depend on how a compiler contracts them.  Then, for K and V of every K/V head,
//   int8:  s = max |x| / 127, code = clamp(rint(x / s)) (as cai_kv_append);
//   4-bit: for each 32 channels s = fp16(bf16(max |x| / 7)), code = clamp(rint(x / s)) in [-7, 7].
// The queries of the new tokens are rotated on the way (bf16 in and out), so that they need no pass
// of their own.
//
// Bound by HBM for chunks and by launch latency for one token a sequence.  One warp per (token, head)
// row; a lane holds four neighbouring channels.
#include "common.cuh"
#include "kv4.cuh"
#include "ptx.cuh"

namespace cai {
namespace {

constexpr int kRowWarps = 8;

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

__device__ __forceinline__ float4 load4(const float* x) { return *reinterpret_cast<const float4*>(x); }
__device__ __forceinline__ float4 load4(const uint16_t* x) {  // bf16
  const uint2 w = *reinterpret_cast<const uint2*>(x);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}
__device__ __forceinline__ float load1(const float* x) { return *x; }
__device__ __forceinline__ float load1(const uint16_t* x) { return __uint_as_float((uint32_t)*x << 16); }

__device__ __forceinline__ uint2 to_bf16x4(const float (&x)[4]) {
  return make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}

// Channels 4 lane .. 4 lane + 3 of row `src`, rotated for position `pos`.
template <class T>
__device__ __forceinline__ void load_rotated(const AppendRowsParams& p, const T* src, int64_t pos, int lane, float (&x)[4]) {
  const int c0 = 4 * lane;
  const float4 v = load4(src + c0);
  x[0] = v.x;
  x[1] = v.y;
  x[2] = v.z;
  x[3] = v.w;
  if (c0 >= p.rot) return;
  const int half = p.rot >> 1;
  const float* cos = p.cos + pos * half;
  const float* sin = p.sin + pos * half;
  if (p.interleaved) {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      if (c0 + e >= p.rot) break;
      const float c = __ldg(cos + c0 / 2 + e / 2), s = __ldg(sin + c0 / 2 + e / 2);
      const float a = x[e], b = x[e + 1];
      x[e] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
      x[e + 1] = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int ch = c0 + e;
      if (ch >= p.rot) break;
      const bool low = ch < half;
      const float y = load1(src + (low ? ch + half : ch - half));  // the partner channel (in L1)
      const float c = __ldg(cos + (low ? ch : ch - half)), s = __ldg(sin + (low ? ch : ch - half));
      x[e] = low ? __fsub_rn(__fmul_rn(x[e], c), __fmul_rn(y, s)) : __fadd_rn(__fmul_rn(x[e], c), __fmul_rn(y, s));
    }
  }
}

__device__ __forceinline__ float absmax4(const float (&x)[4]) {
  return fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
}

// One row into slot `slot` of an int8 page.
__device__ __forceinline__ void store_row8(uint8_t* pg, int P, int slot, bool is_v, int lane, const float (&x)[4]) {
  float amax = absmax4(x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float s = __fdiv_rn(amax, 127.0f);
  uint32_t packed = 0;
  if (s != 0.0f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      int c = __float2int_rn(__fdiv_rn(x[e], s));
      c = c > 127 ? 127 : (c < -127 ? -127 : c);
      packed |= (uint32_t)(c & 0xFF) << (8 * e);
    }
  }
  if (!is_v) {
    reinterpret_cast<uint32_t*>(pg + slot * kHeadDim)[lane] = packed;
  } else {
    uint8_t* v = pg + P * kHeadDim + slot;  // channel-major
#pragma unroll
    for (int e = 0; e < 4; ++e) v[(lane * 4 + e) * P] = (uint8_t)(packed >> (8 * e));
  }
  if (lane == 0) reinterpret_cast<float*>(pg + 2 * P * kHeadDim)[(is_v ? P : 0) + slot] = s;
}

// One row into token r of a 4-bit block (layout in kv4.cuh).
__device__ __forceinline__ void store_row4(uint8_t* blk, int r, bool is_v, int lane, const float (&x)[4]) {
  float amax = absmax4(x);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));  // 8 lanes: 32 channels
  const __half sh = scale4(amax);
  const float s = __half2float(sh);
  uint32_t u[4] = {8u, 8u, 8u, 8u};
  if (s > 0.0f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = code4(x[e], s);
  }
  const int j = lane >> 3;  // channel group
  if (!is_v) {
    // Lanes 2 k and 2 k + 1 share a word: channels 8 t + 0..3 and + 4..7 of the group.
    uint32_t w = (u[0] | (u[2] << 4) | (u[1] << 16) | (u[3] << 20)) << (lane & 1 ? 8 : 0);
    w |= __shfl_xor_sync(0xffffffffu, w, 1);
    if (!(lane & 1)) *reinterpret_cast<uint32_t*>(blk + r * 64 + ((lane & 7) >> 1) * 16 + j * 4) = w;
    if ((lane & 7) == 0) *reinterpret_cast<__half*>(blk + kBlkKs + r * 8 + j * 2) = sh;
  } else {
    // A byte holds this token's channels 16 m + g (low) and + 8 (high): lanes 4 m, 4 m + 1 and 4 m + 2, 4 m + 3.
    const uint32_t mine = u[0] | (u[1] << 8) | (u[2] << 16) | (u[3] << 24);
    const uint32_t up = __shfl_xor_sync(0xffffffffu, mine, 2);
    const int t = (r & 7) >> 1, e1 = r & 1, hb = r >> 3, m = lane >> 2;
    if (!(lane & 2)) {
      const uint32_t w = mine | (up << 4);
      uint8_t* v = blk + kBlkV + (((m >> 2) * 32 + 16 * (lane & 1) + t) * 4 + (m & 3)) * 4 + hb + 2 * e1;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e * 64] = (uint8_t)(w >> (8 * e));  // next g: four lanes of 16 bytes on
    }
    if ((lane & 7) == 0) *reinterpret_cast<__half*>(blk + kBlkVs + (t * 16 + hb * 8 + j * 2 + e1) * 2) = sh;
  }
}

template <bool kFour, class T>
__global__ void __launch_bounds__(kRowWarps * 32) append_rows_kernel(const __grid_constant__ AppendRowsParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int units = 2 * p.num_kv_heads + p.num_q_heads;
  const int64_t w = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const int64_t i = w / units;
  const int unit = (int)(w - i * units);
  const int b = blockIdx.y;
  const NewRows nr = new_rows(p, b);
  if (nr.n < 0 && w == 0 && lane == 0 && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
  if (i >= nr.n) return;
  const int64_t pos = (int64_t)p.start_pos[b] + i;
  const int P = p.page_size;
  if (pos < 0 || pos >= (int64_t)p.max_pages * P || (p.rot > 0 && pos >= p.num_positions)) {
    if (lane == 0 && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
    return;
  }
  const int64_t row = nr.r0 + i;
  float x[4];
  if (unit >= 2 * p.num_kv_heads) {
    const int h = unit - 2 * p.num_kv_heads;
    load_rotated(p, p.q + row * p.q_stride + h * kHeadDim, pos, lane, x);
    __syncwarp();  // the row is read before any of it is written (q_out may be q)
    reinterpret_cast<uint2*>(p.q_out + (row * p.num_q_heads + h) * kHeadDim)[lane] = to_bf16x4(x);
    return;
  }
  const int32_t page = p.table[(int64_t)b * p.max_pages + pos / P];
  const bool is_v = unit >= p.num_kv_heads;
  const int h = is_v ? unit - p.num_kv_heads : unit;
  if (page < 0 || page >= p.num_pages[h]) {
    if (lane == 0 && p.err) atomicOr(p.err, CAI_DEVERR_PAGE);
    return;
  }
  const int slot = (int)(pos % P);
  if (is_v) {
    const float4 v = load4(static_cast<const T*>(p.v) + row * p.v_stride + h * kHeadDim + 4 * lane);
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  } else {
    load_rotated(p, static_cast<const T*>(p.k) + row * p.k_stride + h * kHeadDim, pos, lane, x);
  }
  if constexpr (kFour)
    store_row4(p.pages[h] + (int64_t)page * page_bytes4(P) + (slot / kBlk) * kBlkBytes, slot % kBlk, is_v, lane, x);
  else
    store_row8(p.pages[h] + (int64_t)page * page_bytes(P), P, slot, is_v, lane, x);
}

__device__ __forceinline__ void store4(float* dst, const float (&x)[4]) {
  *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(uint16_t* dst, const float (&x)[4]) { *reinterpret_cast<uint2*>(dst) = to_bf16x4(x); }

// One warp per (token, K/V head): both rows.
template <bool kFour, class T>
__global__ void __launch_bounds__(kRowWarps * 32) read_rows_kernel(const __grid_constant__ ReadRowsParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const int64_t i = w / p.num_kv_heads;
  const int h = (int)(w - i * p.num_kv_heads);
  const int b = blockIdx.y;
  const NewRows nr = new_rows(p, b);
  if (nr.n < 0 && w == 0 && lane == 0 && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
  if (i >= nr.n) return;
  const int64_t pos = (int64_t)p.start_pos[b] + i;
  const int P = p.page_size;
  int bad = pos < 0 || pos >= (int64_t)p.max_pages * P ? CAI_DEVERR_LENGTH : 0;
  int32_t page = -1;
  if (!bad) {
    page = p.table[(int64_t)b * p.max_pages + pos / P];
    if (page < 0 || page >= p.num_pages[h]) bad = CAI_DEVERR_PAGE;
  }
  float k[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
  if (bad) {
    if (lane == 0 && p.err) atomicOr(p.err, bad);
  } else if constexpr (kFour) {
    const int slot = (int)(pos % P), r = slot % kBlk, j = lane >> 3;
    const uint8_t* blk = p.pages[h] + (int64_t)page * page_bytes4(P) + (slot / kBlk) * kBlkBytes;
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(blk + r * 64 + ((lane & 7) >> 1) * 16 + j * 4) >> (lane & 1 ? 8 : 0);
    const float ks = __half2float(*reinterpret_cast<const __half*>(blk + kBlkKs + r * 8 + j * 2));
    const int t = (r & 7) >> 1, e1 = r & 1, hb = r >> 3, m = lane >> 2;
    const uint8_t* vb = blk + kBlkV + (((m >> 2) * 32 + 16 * (lane & 1) + t) * 4 + (m & 3)) * 4 + hb + 2 * e1;
    const float vs = __half2float(*reinterpret_cast<const __half*>(blk + kBlkVs + (t * 16 + hb * 8 + j * 2 + e1) * 2));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      k[e] = (float)((int)((kw >> (4 * (e >> 1) + 16 * (e & 1))) & 15u) - 8) * ks;
      v[e] = (float)((int)((vb[e * 64] >> (lane & 2 ? 4 : 0)) & 15u) - 8) * vs;
    }
  } else {
    const int slot = (int)(pos % P);
    const uint8_t* pg = p.pages[h] + (int64_t)page * page_bytes(P);
    const float* sc = reinterpret_cast<const float*>(pg + 2 * P * kHeadDim);
    const uint32_t kw = reinterpret_cast<const uint32_t*>(pg + slot * kHeadDim)[lane];
    const float ks = sc[slot], vs = sc[P + slot];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      k[e] = (float)(int8_t)(kw >> (8 * e)) * ks;
      v[e] = (float)(int8_t)pg[P * kHeadDim + (4 * lane + e) * P + slot] * vs;
    }
  }
  const int64_t dst = ((nr.r0 + i) * p.num_kv_heads + h) * kHeadDim + 4 * lane;
  if (p.k_out) store4(static_cast<T*>(p.k_out) + dst, k);
  if (p.v_out) store4(static_cast<T*>(p.v_out) + dst, v);
}

}  // namespace

cudaError_t launch_append_rows(const AppendRowsParams& p, bool four, bool bf16, cudaStream_t stream) {
  const int64_t warps = (int64_t)p.n_new * (2 * p.num_kv_heads + p.num_q_heads);
  const dim3 grid((unsigned)((warps + kRowWarps - 1) / kRowWarps), (unsigned)p.batch), block(kRowWarps * 32);
  if (four)
    return bf16 ? launch_pdl(append_rows_kernel<true, uint16_t>, grid, block, 0, stream, p)
                : launch_pdl(append_rows_kernel<true, float>, grid, block, 0, stream, p);
  return bf16 ? launch_pdl(append_rows_kernel<false, uint16_t>, grid, block, 0, stream, p)
              : launch_pdl(append_rows_kernel<false, float>, grid, block, 0, stream, p);
}

cudaError_t launch_read_rows(const ReadRowsParams& p, bool four, bool bf16, cudaStream_t stream) {
  const int64_t warps = (int64_t)p.n_new * p.num_kv_heads;
  const dim3 grid((unsigned)((warps + kRowWarps - 1) / kRowWarps), (unsigned)p.batch), block(kRowWarps * 32);
  if (four)
    return bf16 ? launch_pdl(read_rows_kernel<true, uint16_t>, grid, block, 0, stream, p)
                : launch_pdl(read_rows_kernel<true, float>, grid, block, 0, stream, p);
  return bf16 ? launch_pdl(read_rows_kernel<false, uint16_t>, grid, block, 0, stream, p)
              : launch_pdl(read_rows_kernel<false, float>, grid, block, 0, stream, p);
}

}  // namespace cai

// Page summaries: for each of the 128 key channels of a page, the smallest and the largest cached value of
// its tokens, as 8-bit codes under one scale.
//
// x = code * scale of a cached key in fp32 (4-bit: an fp16 number exactly); hi_c = max x, lo_c = min x over the tokens
// that the page holds; s = max_c max(|hi_c|, |lo_c|) / 127; codes min(127, ceil(hi_c / s)) and
// max(-127, floor(lo_c / s)), 0 when s is 0.  Minima and maxima do not depend on an order, the divisions are IEEE: the
// result is the same bits however the work is split.
//
// A page is computed anew from the cache whenever a token is added to it, so a summary never holds what an earlier
// owner of the page wrote.  Bound by HBM where whole dialogues are summarized (the keys, half of the cache's bytes, are
// read once), by latency for the one page of a decode step.  A warp has a page of one K/V head: int8, a lane four
// channels and 16 tokens' words under way at a time; 4-bit, a lane eight channels of every other token, in fp16 pairs.
// A page that is not full reads its last token again in place of those that are not there.
#include <algorithm>

#include "kv4.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace cai {
namespace {

constexpr int kSumWarps = 8;
constexpr int kSumBlocks = 4;  // blocks of an SM

__device__ __forceinline__ float fmin3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint32_t hmin2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("min.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// Codes of a bound x under scale s > 0, away from the other bound.
__device__ __forceinline__ uint32_t code_up(float x, float s) { return (uint32_t)min(127, __float2int_ru(__fdiv_rn(x, s))) & 0xFFu; }
__device__ __forceinline__ uint32_t code_down(float x, float s) { return (uint32_t)max(-127, __float2int_rd(__fdiv_rn(x, s))) & 0xFFu; }

// Largest and smallest keys of the first `fill` (1 .. P) tokens of a page -> its record.
__device__ __forceinline__ void page8(const uint8_t* pg, int P, int fill, uint8_t* codes, float* scale, int lane) {
  const float* ks = reinterpret_cast<const float*>(pg + 2 * P * kHeadDim);
  float hi[4], lo[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) hi[e] = -INFINITY, lo[e] = INFINITY;
  for (int t0 = 0; t0 < fill; t0 += 16) {
    uint32_t w[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) w[r] = reinterpret_cast<const uint32_t*>(pg + min(t0 + r, fill - 1) * kHeadDim)[lane];
    const float s16 = ks[min(t0 + (lane & 15), fill - 1)];
    const uint64_t off = f2(-8388736.0f, -8388736.0f);  // 2^23 + 128
#pragma unroll
    for (int r = 0; r < 16; r += 2) {
      float x[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // code + 128 in the low mantissa byte of 2^23: exact.
        const uint32_t u = w[r + k] ^ 0x80808080u;
        const float s = __shfl_sync(0xffffffffu, s16, r + k);
        const uint64_t s2 = f2(s, s);
        const auto wide = [&](int i) { return __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + i)); };
        f2_split(f2_mul(f2_add(f2(wide(0), wide(1)), off), s2), x[k][0], x[k][1]);
        f2_split(f2_mul(f2_add(f2(wide(2), wide(3)), off), s2), x[k][2], x[k][3]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        hi[e] = fmax3(hi[e], x[0][e], x[1][e]);
        lo[e] = fmin3(lo[e], x[0][e], x[1][e]);
      }
    }
  }
  float amax = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) amax = fmax3(amax, fabsf(hi[e]), fabsf(lo[e]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float s = __fdiv_rn(amax, 127.0f);
  uint32_t up = 0, down = 0;
  if (s != 0.0f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      up |= code_up(hi[e], s) << (8 * e);
      down |= code_down(lo[e], s) << (8 * e);
    }
  }
  reinterpret_cast<uint32_t*>(codes)[lane] = up;
  reinterpret_cast<uint32_t*>(codes + kHeadDim)[lane] = down;
  if (lane == 0) *scale = s;
}

__device__ __forceinline__ void page4(const uint8_t* pg, int fill, uint8_t* codes, float* scale, int lane) {
  const int half = lane >> 4, word = lane & 15, j = word & 3;  // every other token; channels 32 j + 8 (word / 4) .. + 7
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) hi[i] = 0xFC00FC00u, lo[i] = 0x7C007C00u;
  for (int t0 = 0; t0 < fill; t0 += kBlk) {
    const uint8_t* blk = pg + t0 / kBlk * kBlkBytes;
    const int last = min(fill - t0, kBlk) - 1;
    uint32_t w[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = min(2 * i + half, last);
      w[i] = *reinterpret_cast<const uint32_t*>(blk + r * 64 + word * 4);
      s[i] = *reinterpret_cast<const uint16_t*>(blk + kBlkKs + r * 8 + j * 2);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t x[4];
      const uint32_t s2 = s[i] * 0x10001u;
      values_f16(w[i], s2, s2, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        hi[e] = hmax2(hi[e], x[e]);
        lo[e] = hmin2(lo[e], x[e]);
      }
    }
  }
  // One half of the warp goes on with the largest, the other with the smallest.
  float x[8], amax = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t mine = half ? lo[e] : hi[e], got = __shfl_xor_sync(0xffffffffu, half ? hi[e] : lo[e], 16);
    const uint32_t b = half ? hmin2(mine, got) : hmax2(mine, got);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&b));
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
    amax = fmax3(amax, fabsf(f.x), fabsf(f.y));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float s = __fdiv_rn(amax, 127.0f);
  uint32_t c[2] = {0u, 0u};
  if (s != 0.0f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e >> 2] |= (half ? code_down(x[e], s) : code_up(x[e], s)) << (8 * (e & 3));
  }
  *reinterpret_cast<uint2*>(codes + half * kHeadDim + 32 * j + 8 * (word >> 2)) = make_uint2(c[0], c[1]);
  if (lane == 0) *scale = s;
}

// Whether sequence b's new tokens reach its u-th page, counted from the first new token's.
__device__ __forceinline__ bool has_page(const SummarizeParams& p, int b, int64_t u) {
  const int n = new_rows(p, b).n;
  const int64_t start = n > 0 ? p.start_pos[b] : 0;
  const int lg = page_log2(p.page_size);
  return n > 0 && start + n > (((start >> lg) + u) << lg);
}

template <bool kFour>
__device__ __forceinline__ void summarize_page(const SummarizeParams& p, int b, int64_t u, int h, int lane) {
  const int P = p.page_size, lg = page_log2(P);
  const int64_t start = p.start_pos[b], end = start + new_rows(p, b).n;
  const int64_t at = (start >> lg) + u;  // (floor, also below 0)
  if (at < 0 || at >= p.max_pages) {
    if (lane == 0 && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
    return;
  }
  const int32_t page = p.table[(int64_t)b * p.max_pages + at];
  if (page < 0 || page >= p.num_pages[h]) {
    if (lane == 0 && p.err) atomicOr(p.err, CAI_DEVERR_PAGE);
    return;
  }
  const int64_t left = end - (at << lg);
  const int fill = (int)(left < P ? left : P);
  uint8_t* codes = p.data[h] + (int64_t)page * (2 * kHeadDim);
  float* scale = reinterpret_cast<float*>(p.data[h] + (int64_t)p.num_pages[h] * (2 * kHeadDim)) + page;
  if constexpr (kFour)
    page4(p.pages[h] + (int64_t)page * page_bytes4(P), fill, codes, scale, lane);
  else
    page8(p.pages[h] + (int64_t)page * page_bytes(P), P, fill, codes, scale, lane);
}

// A warp looks through its share of the (sequence, page, K/V head) triples, 32 at a time, for those with new tokens.
template <bool kFour>
__global__ void __launch_bounds__(kSumWarps * 32, kSumBlocks) summarize_kernel(const __grid_constant__ SummarizeParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t per_seq = (int64_t)p.groups * p.num_kv_heads, items = p.batch * per_seq;
  const int64_t step = (int64_t)gridDim.x * kSumWarps;
  for (int64_t w = (int64_t)blockIdx.x * kSumWarps + (threadIdx.x >> 5); w < items; w += 32 * step) {
    const int64_t mine = w + lane * step;
    int b = 0, h = 0;
    int64_t u = 0;
    bool there = false;
    if (mine < items) {
      const int64_t i = over(mine, p.num_kv_heads);
      h = (int)(mine - i * p.num_kv_heads);
      b = (int)over(i, p.groups);
      u = i - (int64_t)b * p.groups;
      there = has_page(p, b, u);
      if (u == 0 && h == 0 && new_rows(p, b).n < 0 && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
    }
    for (uint32_t m = __ballot_sync(0xffffffffu, there); m; m &= m - 1) {
      const int k = __ffs(m) - 1;
      summarize_page<kFour>(p, __shfl_sync(0xffffffffu, b, k), __shfl_sync(0xffffffffu, u, k), __shfl_sync(0xffffffffu, h, k), lane);
    }
  }
}

}  // namespace

cudaError_t launch_summarize(SummarizeParams p, bool four, cudaStream_t stream) {
  p.groups = (int32_t)(((int64_t)p.n_new + 2 * p.page_size - 2) / p.page_size);  // from any position in a page
  const int64_t items = (int64_t)p.batch * p.groups * p.num_kv_heads;
  // At most four waves of warps, each with a share of the triples: 64 dialogues of up to 8192 tokens, 4-bit, four K/V heads
  // 32 us (one wave 37, eight 36, a warp for each triple 39); int8 likewise (23; 25, 25, 30).
  const int64_t blocks = (items + kSumWarps - 1) / kSumWarps, wave = (int64_t)num_sms() * kSumBlocks;
  const dim3 grid((unsigned)std::min(blocks, 4 * wave));
  return four ? launch_pdl(summarize_kernel<true>, grid, dim3(kSumWarps * 32), 0, stream, p)
              : launch_pdl(summarize_kernel<false>, grid, dim3(kSumWarps * 32), 0, stream, p);
}

}  // namespace cai

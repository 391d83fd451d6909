// Page summaries: for each of the 128 key channels of a page, the smallest and the largest cached value of
// its tokens, as 8-bit codes under one scale.
//
// x = code * scale of a cached key in fp32 (4-bit: an fp16 number exactly); hi_c = max x, lo_c = min x over the tokens
// that the page holds; s = max_c max(|hi_c|, |lo_c|) / 127; codes min(127, ceil(hi_c / s)) and
// max(-127, floor(lo_c / s)), 0 when s is 0.  Minima and maxima do not depend on an order, the divisions are IEEE: the
// result is the same bits however the work is split.
//
// A page is computed anew from the cache whenever a token is added to it, so a summary never holds what an earlier
// owner of the page wrote.  Bound by instructions where whole dialogues are summarized (the keys, half of the cache's
// bytes, are read once: 64 dialogues of up to 8192 tokens, pages of 32, four K/V heads, 4-bit, 24 us, 49 MB at 2.1 TB/s, 720
// warp instructions a page of which the conversion and the minima take 400), by latency for the one page of a decode
// step (2.7 us).  A warp has a page of one K/V head: int8, a lane four channels and 16 tokens' words under way at a time;
// 4-bit, a lane eight channels of every other token, in fp16 pairs.  A page that is not full reads its last token
// again in place of those that are not there.
#include <algorithm>

#include "kv4.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace cai {
namespace {

constexpr int kSumWarps = 8;
constexpr int kSumBlocks = 5;  // blocks of an SM

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

__device__ __forceinline__ uint64_t f2_add_up(uint64_t a, uint64_t b) {  // rounded up
  uint64_t r;
  asm("add.rp.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The scale of a page whose largest magnitude is amax, and how its quotients are computed.
struct PageScale {
  float s, inv;  // inv 0: by divisions
};
__device__ __forceinline__ PageScale page_scale(float amax) {
  PageScale c;
  c.s = __fdiv_rn(amax, 127.0f);
  c.inv = c.s >= 0x1p-100f && c.s <= 1.0f ? __frcp_rn(c.s) : 0.0f;
  return c;
}

// Codes of four bounds: min(127, ceil(x / s)) with sign 1, max(-127, floor(x / s)) = -min(127, ceil(x / -s)) with -1.
// The quotients are rounded as the IEEE division does: twice corrected by their remainders, the second time from
// within an ulp, with the rounded inverse (Markstein, 1990).  Remainders and quotients of a page of scale 2^-100 to 1 are not
// subnormal where they count; other pages take divisions (an IEEE division for each of eight channels took a
// quarter of a page's instructions).
__device__ __forceinline__ uint32_t codes_of(const float* x, const PageScale& c, float sign) {
  uint32_t y[4];
  if (c.inv != 0.0f) {
    const uint64_t inv = f2(sign * c.inv, sign * c.inv), ns = f2(-sign * c.s, -sign * c.s);
    const uint64_t magic = f2(12582912.0f, 12582912.0f), sg = f2(sign, sign);  // 3 2^22: whole numbers in the low bits
    const uint64_t back = f2(12582912.0f * (1.0f - sign), 12582912.0f * (1.0f - sign));
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const uint64_t x2 = f2(x[e], x[e + 1]);
      uint64_t q = f2_mul(x2, inv);
      q = f2_fma(f2_fma(q, ns, x2), inv, q);
      q = f2_fma(f2_fma(q, ns, x2), inv, q);
      float a, b;
      f2_split(q, a, b);
      f2_split(f2_fma(f2_add_up(f2(fminf(a, 127.0f), fminf(b, 127.0f)), magic), sg, back), a, b);
      y[e] = __float_as_uint(a);
      y[e + 1] = __float_as_uint(b);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int up = c.s != 0.0f ? min(127, __float2int_ru(__fdiv_rn(sign * x[e], c.s))) : 0;
      y[e] = (uint32_t)(sign < 0.0f ? -up : up);
    }
  }
  return __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410);
}

// The largest of the warp's magnitudes (not NaN: not negative, they are ordered as whole numbers).
__device__ __forceinline__ float largest(float x) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x))); }

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
  const PageScale c = page_scale(largest(amax));
  reinterpret_cast<uint32_t*>(codes)[lane] = codes_of(hi, c, 1.0f);
  reinterpret_cast<uint32_t*>(codes + kHeadDim)[lane] = codes_of(lo, c, -1.0f);
  if (lane == 0) *scale = c.s;
}

__device__ __forceinline__ void page4(const uint8_t* pg, int fill, uint8_t* codes, float* scale, int lane) {
  const int half = lane >> 4, word = lane & 15, j = word & 3;  // every other token; channels 32 j + 8 (word / 4) .. + 7
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) hi[i] = 0xFC00FC00u, lo[i] = 0x7C007C00u;
  for (int t0 = 0; t0 < fill; t0 += kBlk) {
    const uint8_t* blk = pg + t0 / kBlk * kBlkBytes;
    const int last = fill - t0 - 1;
    uint32_t w[8], s[8];
    const uint8_t* pw = blk + half * 64 + word * 4;
    const uint8_t* ps = blk + kBlkKs + half * 8 + j * 2;
    if (last >= kBlk - 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[i] = *reinterpret_cast<const uint32_t*>(pw + i * 128);
        s[i] = *reinterpret_cast<const uint16_t*>(ps + i * 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = min(2 * i + half, last) - half;
        w[i] = *reinterpret_cast<const uint32_t*>(pw + r * 64);
        s[i] = *reinterpret_cast<const uint16_t*>(ps + r * 8);
      }
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
  const PageScale c = page_scale(largest(amax));
  const float sign = half ? -1.0f : 1.0f;
  *reinterpret_cast<uint2*>(codes + half * kHeadDim + 32 * j + 8 * (word >> 2)) = make_uint2(codes_of(x, c, sign), codes_of(x + 4, c, sign));
  if (lane == 0) *scale = c.s;
}

// A warp looks through its share of the (sequence, page, K/V head) triples, 32 at a time: a lane finds the place of one, and
// the warp goes through those that have new tokens.
template <bool kFour>
__global__ void __launch_bounds__(kSumWarps * 32, kSumBlocks) summarize_kernel(const __grid_constant__ SummarizeParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, P = p.page_size, lg = page_log2(P);
  const int64_t per_seq = (int64_t)p.groups * p.num_kv_heads, items = p.batch * per_seq;
  const int64_t step = (int64_t)gridDim.x * kSumWarps;
  for (int64_t w = blockIdx.x + (int64_t)gridDim.x * (threadIdx.x >> 5); w < items; w += 32 * step) {
    const int64_t mine = w + lane * step;
    int32_t page = -1;
    int h = 0, fill = 0;
    if (mine < items) {
      const int64_t i = over(mine, p.num_kv_heads);
      h = (int)(mine - i * p.num_kv_heads);
      const int b = (int)over(i, p.groups);
      const int64_t u = i - (int64_t)b * p.groups;  // counted from the first new token's page
      const int n = new_rows(p, b).n;
      if (n > 0) {
        const int64_t start = p.start_pos[b], at = (start >> lg) + u, left = start + n - (at << lg);  // (floor, also below 0)
        int bits = 0;
        if (left <= 0) {  // the tokens end before this page
        } else if (at < 0 || at >= p.max_pages) {
          bits = CAI_DEVERR_LENGTH;
        } else {
          page = p.table[(int64_t)b * p.max_pages + at];
          if (page < 0 || page >= p.num_pages[h]) bits = CAI_DEVERR_PAGE, page = -1;
        }
        fill = (int)(left < P ? left : P);
        if (bits && p.err) atomicOr(p.err, bits);
      } else if (n < 0 && u == 0 && h == 0 && p.err) {
        atomicOr(p.err, CAI_DEVERR_LENGTH);
      }
    }
    const int what = h << 8 | fill;
    for (uint32_t m = __ballot_sync(0xffffffffu, page >= 0); m; m &= m - 1) {
      const int k = __ffs(m) - 1, pg = __shfl_sync(0xffffffffu, page, k), hf = __shfl_sync(0xffffffffu, what, k);
      const int hk = hf >> 8, f = hf & 255;
      uint8_t* codes = p.data[hk] + (int64_t)pg * (2 * kHeadDim);
      float* scale = reinterpret_cast<float*>(p.data[hk] + (int64_t)p.num_pages[hk] * (2 * kHeadDim)) + pg;
      if constexpr (kFour)
        page4(p.pages[hk] + (int64_t)pg * page_bytes4(P), f, codes, scale, lane);
      else
        page8(p.pages[hk] + (int64_t)pg * page_bytes(P), P, f, codes, scale, lane);
    }
  }
}

}  // namespace

cudaError_t launch_summarize(SummarizeParams p, bool four, cudaStream_t stream) {
  p.groups = (int32_t)(((int64_t)p.n_new + 2 * p.page_size - 2) / p.page_size);  // from any position in a page
  const int64_t items = (int64_t)p.batch * p.groups * p.num_kv_heads;
  // One wave of warps, each with a share of the triples: the dialogues above take 23.7 us, with two waves 25.4, with four 27.5
  // (int8 18.3; 18.9, 21.1).  The warps of a block take triples far apart: those of one sequence are there, or are not,
  // together, and a block of neighbours has twice as many pages as another.
  const int64_t blocks = (items + kSumWarps - 1) / kSumWarps, wave = (int64_t)num_sms() * kSumBlocks;
  const dim3 grid((unsigned)std::min(blocks, wave));
  return four ? launch_pdl(summarize_kernel<true>, grid, dim3(kSumWarps * 32), 0, stream, p)
              : launch_pdl(summarize_kernel<false>, grid, dim3(kSumWarps * 32), 0, stream, p);
}

}  // namespace cai

// The 4-bit paged cache: its block layout, and the conversion of codes to fp16.
//
// A page of P tokens is P / 16 blocks of 2304 bytes, each block 16 consecutive tokens:
//   [0, 1024)     K codes, 64 bytes a token: word (t, j) (t = 0..3 the byte offset / 16, j = 0..3 the
//                 word within) holds channels 32 j + 8 t + 2 i + e at bits 4 i + 16 e (i = 0..3, e = 0, 1)
//   [1024, 2048)  V codes: word (h, g, t, w) at ((h * 32 + 4 g + t) * 4 + w) * 4, with m = 4 h + w, holds at
//                 bits 4 i + 16 e channel 16 m + g + 8 (i % 2) of token 8 (i / 2) + 2 t + e
//   [2048, 2176)  K scales fp16 [16 tokens][4 channel groups]
//   [2176, 2304)  V scales fp16 [t][token / 8][group][e]
// A code is stored as code + 8 (1 .. 15) and stands for code * scale; scales have at most 8
// significant bits, so every product is exact in fp16.
//
// The order is that of the A operands of mma.m16n8k16: lane (g, t) of a warp finds all it needs of a
// block's K in two 16-byte loads (token rows g and g + 8), of its V in two more, free of bank
// conflicts, and a page is contiguous, so a plain bulk copy brings it.
#pragma once
#include <cuda_fp16.h>

#include <cstdint>

namespace cai {

constexpr int kBlk = 16;               // tokens of a block
constexpr int kBlkBytes = 2304;
constexpr int kBlkV = 1024, kBlkKs = 2048, kBlkVs = 2176;
constexpr float kMaxScale4 = 9344.0f;  // 7 * 9344 = 65408 is finite in fp16

// Where a softmax reference is set or raised it lies this far (log2 units) below the largest logit: that has a weight of
// 2^7, and a logit may pass it by 2^8 before the next raise, so weights stay within 2^15 and finite in fp16.
// A weight below 2^-14 is a subnormal of fp16, off by up to 2^-25: 2^-32 of the sum at most, which is 2^7 and more.  (With the
// largest at 2^0 a flat rest of 131072 keys 2^25.5 below one key, 0.3% of the sum, was lost from the product.)
constexpr float kWeightLift = 7.0f;

__host__ __device__ constexpr int page_bytes4(int P) { return P / kBlk * kBlkBytes; }

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t y;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(a), "r"(b), "r"(c));
  return y;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// (w & mask) | base in one operation (written out: left to itself the compiler took two).
__device__ __forceinline__ uint32_t pick(uint32_t w, uint32_t mask, uint32_t base) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(w), "r"(mask), "r"(base));
  return y;
}

// u = code + 8 in four bits of both halves of a word -> the codes, in fp16.  Placed in the low mantissa
// bits of 1024 u reads as 1024 + u, one nibble higher as 1024 + 16 u; one exact operation of the
// half-precision pipe takes the offset off.  (Placing u at the top of the mantissa of 16 and taking
// (16 + u) s - 24 s would apply a scale in the same operation, but 24 s overflows where |x| passes 19000.)
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&r)[4]) {
  const uint32_t u = w >> 8;
  r[0] = hadd2(pick(w, 0x000F000Fu, 0x64006400u), 0xE408E408u);               // - 1032
  r[1] = hfma2(pick(w, 0x00F000F0u, 0x64006400u), 0x2C002C00u, 0xD480D480u);  // / 16 - 72
  r[2] = hadd2(pick(u, 0x000F000Fu, 0x64006400u), 0xE408E408u);
  r[3] = hfma2(pick(u, 0x00F000F0u, 0x64006400u), 0x2C002C00u, 0xD480D480u);
}
// ... and the values: pairs 0 and 1 under scales s0, pairs 2 and 3 under s1 (exact products).
__device__ __forceinline__ void values_f16(uint32_t w, uint32_t s0, uint32_t s1, uint32_t (&r)[4]) {
  codes_f16(w, r);
  r[0] = hmul2(r[0], s0);
  r[1] = hmul2(r[1], s0);
  r[2] = hmul2(r[2], s1);
  r[3] = hmul2(r[3], s1);
}

// Scale of a group whose largest magnitude is amax: amax / 7 rounded to bf16 (8 significant bits),
// then to fp16 (exact from 2^-14 up).
__device__ __forceinline__ __half scale4(float amax) {
  const float t = __fdiv_rn(amax, 7.0f);
  const float b = __uint_as_float((__float_as_uint(t) + 0x7FFFu + ((__float_as_uint(t) >> 16) & 1u)) & 0xFFFF0000u);
  return __float2half_rn(fminf(b, kMaxScale4));
}
// Code + 8 of x under scale s (s > 0).
__device__ __forceinline__ uint32_t code4(float x, float s) {
  const int c = __float2int_rn(__fdiv_rn(x, s));
  return (uint32_t)((c > 7 ? 7 : (c < -7 ? -7 : c)) + 8);
}

}  // namespace cai

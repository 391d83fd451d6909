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
// Bound by HBM for chunks and by launch latency for one token a sequence.  One launch, blocks of three
// kinds: K/V blocks, in chunk calls one per 16 aligned tokens of a head, so that V, which lies by
// channel, is written in words and not in bytes, otherwise a warp per token; query blocks, a warp per
// eight heads of a token (a lane eight channels of every other head, 16-byte loads and stores, all
// of them under way before the position and its part of the tables are known); and one block that
// checks packed offsets.  Reads go by 16 aligned tokens too.
#include <algorithm>

#include "common.cuh"
#include "kv4.cuh"
#include "ptx.cuh"

namespace cai {
namespace {

constexpr int kRowWarps = 8;
constexpr int kQHeads = 8;  // query heads of one warp (16: a decode step of 256 sequences 6.5 us, 8: 5.0; chunks within 5%)

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

__device__ __forceinline__ uint2 to_bf16x4(const float (&x)[4]) {
  return make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}

// A position's coefficients for channels c0 .. c0 + N - 1 (N is 4 or 8, c0 a multiple of N), where these lie below rot.
template <int N>
struct Turn {
  float c[N], s[N];  // per channel; half-split: s is negated for the first channel of a pair
  int mode;          // 0: none of these channels, 1: half-split in whole vectors, 2: half-split, odd sizes, 3: interleaved
};

template <int N>
__device__ __forceinline__ Turn<N> load_turn(const AppendRowsParams& p, int64_t pos, int c0) {
  Turn<N> t;
  const int half = p.rot >> 1;
  t.mode = 0;
  if (c0 >= p.rot) return t;
  const float* cos = p.cos + pos * half;
  const float* sin = p.sin + pos * half;
  if (p.interleaved) {
    t.mode = 3;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const bool on = c0 + e < p.rot;
      t.c[e] = on ? __ldg(cos + (c0 + e) / 2) : 1.0f;
      t.s[e] = on ? __ldg(sin + (c0 + e) / 2) : 0.0f;
    }
    return t;
  }
  const bool low = c0 < half;
  if (half % N == 0) {
    t.mode = 1;
    const int at = low ? c0 : c0 - half;
    if (p.wide_tables) {
#pragma unroll
      for (int e = 0; e < N; e += 4) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(cos + at + e));
        const float4 s = __ldg(reinterpret_cast<const float4*>(sin + at + e));
        t.c[e] = c.x, t.c[e + 1] = c.y, t.c[e + 2] = c.z, t.c[e + 3] = c.w;
        t.s[e] = s.x, t.s[e + 1] = s.y, t.s[e + 2] = s.z, t.s[e + 3] = s.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        t.c[e] = __ldg(cos + at + e);
        t.s[e] = __ldg(sin + at + e);
      }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) t.s[e] = low ? -t.s[e] : t.s[e];
    return t;
  }
  t.mode = 2;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int ch = c0 + e;
    const bool first = ch < half;
    const bool on = ch < p.rot;
    t.c[e] = on ? __ldg(cos + (first ? ch : ch - half)) : 1.0f;
    const float s = on ? __ldg(sin + (first ? ch : ch - half)) : 0.0f;
    t.s[e] = first ? -s : s;
  }
  return t;
}

__device__ __forceinline__ void load_n(const float* x, float (&v)[4]) {
  const float4 w = *reinterpret_cast<const float4*>(x);
  v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
}
__device__ __forceinline__ void load_n(const uint16_t* x, float (&v)[4]) {  // bf16
  const uint2 w = *reinterpret_cast<const uint2*>(x);
  v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xFFFF0000u);
  v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xFFFF0000u);
}
__device__ __forceinline__ void bf16x8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(u[e] << 16);
    v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ float load1(const float* x) { return *x; }
__device__ __forceinline__ float load1(const uint16_t* x) { return __uint_as_float((uint32_t)*x << 16); }

// x (channels c0 .. c0 + N - 1 of row src) turned in place; y: their partner channels where these are a whole vector
// (partner_of), otherwise they are read one by one.
// a c - b s and b c + a s: a product with -s and a sum round as the product with s and the difference do.
template <int N, class T>
__device__ __forceinline__ void turn_row(const AppendRowsParams& p, const Turn<N>& t, const T* src, int c0, float (&x)[N], const float (&y)[N]) {
  if (t.mode == 1) {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = __fadd_rn(__fmul_rn(x[e], t.c[e]), __fmul_rn(y[e], t.s[e]));
  } else if (t.mode == 3) {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float a = x[e], b = x[e + 1];
      if (c0 + e < p.rot) {
        x[e] = __fsub_rn(__fmul_rn(a, t.c[e]), __fmul_rn(b, t.s[e]));
        x[e + 1] = __fadd_rn(__fmul_rn(b, t.c[e]), __fmul_rn(a, t.s[e]));
      }
    }
  } else if (t.mode == 2) {
    const int half = p.rot >> 1;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int ch = c0 + e;
      if (ch < p.rot) {
        const float z = load1(src + (ch < half ? ch + half : ch - half));
        x[e] = __fadd_rn(__fmul_rn(x[e], t.c[e]), __fmul_rn(z, t.s[e]));
      }
    }
  }
}

// Offset of the partner channels of c0 .. c0 + N - 1 where they are a whole vector; 0 otherwise.
template <int N>
__device__ __forceinline__ int partner_of(const AppendRowsParams& p, int c0) {
  const int half = p.rot >> 1;
  if (p.interleaved || c0 >= p.rot || half % N != 0) return 0;
  return c0 < half ? half : -half;
}

__device__ __forceinline__ float absmax4(const float (&x)[4]) {
  return fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
}

// Codes of a lane's four channels, one a byte (int8: two's complement, 4-bit: code + 8), and the scale.
__device__ __forceinline__ uint32_t quantize8(const float (&x)[4], float& s) {
  float amax = absmax4(x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  s = __fdiv_rn(amax, 127.0f);
  uint32_t packed = 0;
  if (s != 0.0f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      int c = __float2int_rn(__fdiv_rn(x[e], s));
      c = c > 127 ? 127 : (c < -127 ? -127 : c);
      packed |= (uint32_t)(c & 0xFF) << (8 * e);
    }
  }
  return packed;
}
__device__ __forceinline__ uint32_t quantize4(const float (&x)[4], __half& sh) {
  float amax = absmax4(x);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));  // 8 lanes: 32 channels
  sh = scale4(amax);
  const float s = __half2float(sh);
  uint32_t packed = 0x08080808u;
  if (s > 0.0f) packed = code4(x[0], s) | (code4(x[1], s) << 8) | (code4(x[2], s) << 16) | (code4(x[3], s) << 24);
  return packed;
}

// One row into slot `slot` of an int8 page.
__device__ __forceinline__ void store_row8(uint8_t* pg, int P, int slot, bool is_v, int lane, const float (&x)[4]) {
  float s;
  const uint32_t packed = quantize8(x, s);
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
  __half sh;
  const uint32_t u = quantize4(x, sh);
  const int j = lane >> 3;  // channel group
  if (!is_v) {
    // Lanes 2 k and 2 k + 1 share a word: channels 8 t + 0..3 and + 4..7 of the group.
    uint32_t w = __byte_perm(u, 0u, 0x4140) | (__byte_perm(u, 0u, 0x4342) << 4);  // codes 0, 1 and 2, 3: bits 0, 16 and 4, 20
    w <<= lane & 1 ? 8 : 0;
    w |= __shfl_xor_sync(0xffffffffu, w, 1);
    if (!(lane & 1)) *reinterpret_cast<uint32_t*>(blk + r * 64 + ((lane & 7) >> 1) * 16 + j * 4) = w;
    if ((lane & 7) == 0) *reinterpret_cast<__half*>(blk + kBlkKs + r * 8 + j * 2) = sh;
  } else {
    // A byte holds this token's channels 16 m + g (low) and + 8 (high): lanes 4 m, 4 m + 1 and 4 m + 2, 4 m + 3.
    const uint32_t up = __shfl_xor_sync(0xffffffffu, u, 2);
    const int t = (r & 7) >> 1, e1 = r & 1, hb = r >> 3, m = lane >> 2;
    if (!(lane & 2)) {
      const uint32_t w = u | (up << 4);
      uint8_t* v = blk + kBlkV + (((m >> 2) * 32 + 16 * (lane & 1) + t) * 4 + (m & 3)) * 4 + hb + 2 * e1;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e * 64] = (uint8_t)(w >> (8 * e));  // next g: four lanes of 16 bytes on
    }
    if ((lane & 7) == 0) *reinterpret_cast<__half*>(blk + kBlkVs + (t * 16 + hb * 8 + j * 2 + e1) * 2) = sh;
  }
}

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

// Row `row` of the call: its sequence and position.  False: none, or its sequence's offsets are invalid.
__device__ __forceinline__ bool row_place(const AppendRowsParams& p, int64_t row, int lane, int& b, int64_t& pos) {
  int32_t a, e;
  if (p.q_off) {
    b = find_seq(p.q_off, p.batch, row, lane, &a, &e);
    if (b < 0 || a < 0 || row >= e || e > p.total_new || e - a > p.n_new) return false;
  } else {
    b = (int)over(row, p.n_new);
    a = b * p.n_new;
  }
  pos = (int64_t)p.start_pos[b] + (row - a);
  return true;
}
__device__ __forceinline__ bool pos_ok(const AppendRowsParams& p, int64_t pos) {
  return pos >= 0 && pos < (int64_t)p.max_pages * p.page_size && (p.rot == 0 || pos < p.num_positions);
}
__device__ __forceinline__ void flag(int32_t* err, int lane, int bits) {
  if (lane == 0 && err) atomicOr(err, bits);
}

// Heads h0 .. h0 + kQHeads - 1 of a token's queries.  A lane's partner channels are another lane's of its half warp.
__device__ __forceinline__ void rotate_queries(const AppendRowsParams& p, int64_t row, int h0, int lane) {
  constexpr int kN = kQHeads / 2;
  const int c0 = 8 * (lane & 15), h = h0 + (lane >> 4);
  const uint16_t* src = p.q + row * p.q_stride;
  uint16_t* dst = p.q_out + row * p.num_q_heads * kHeadDim + c0;
  uint4 x[kN];
#pragma unroll
  for (int u = 0; u < kN; ++u)
    x[u] = h + 2 * u < p.num_q_heads ? *reinterpret_cast<const uint4*>(src + (h + 2 * u) * kHeadDim + c0) : make_uint4(0u, 0u, 0u, 0u);
  int b;
  int64_t pos;
  if (!row_place(p, row, lane, b, pos)) return;
  if (!pos_ok(p, pos)) return flag(p.err, lane, CAI_DEVERR_LENGTH);
  const Turn<8> turn = load_turn<8>(p, pos, c0);
  const int other = lane + partner_of<8>(p, c0) / 8;
#pragma unroll
  for (int u = 0; u < kN; ++u) {
    if (h0 + 2 * u >= p.num_q_heads) break;  // (the same in the whole warp)
    const uint4 y = make_uint4(__shfl_sync(0xffffffffu, x[u].x, other), __shfl_sync(0xffffffffu, x[u].y, other),
                               __shfl_sync(0xffffffffu, x[u].z, other), __shfl_sync(0xffffffffu, x[u].w, other));
    float a[8], c[8];
    bf16x8(x[u], a);
    bf16x8(y, c);
    if (h + 2 * u < p.num_q_heads) turn_row(p, turn, src + (h + 2 * u) * kHeadDim, c0, a, c);
    x[u] = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7]));
  }
  __syncwarp();  // these heads are read before any of them is written (q_out may be q)
#pragma unroll
  for (int u = 0; u < kN; ++u)
    if (h + 2 * u < p.num_q_heads) *reinterpret_cast<uint4*>(dst + (h + 2 * u) * kHeadDim) = x[u];
}

// Row `row` of head h's K or V at position pos, four channels a lane.
template <class T>
__device__ __forceinline__ void load_row(const AppendRowsParams& p, int64_t row, int h, bool is_v, int64_t pos, int lane, float (&x)[4]) {
  if (is_v) {
    load_n(static_cast<const T*>(p.v) + row * p.v_stride + h * kHeadDim + 4 * lane, x);
  } else {
    const T* src = static_cast<const T*>(p.k) + row * p.k_stride + h * kHeadDim;
    float y[4];
    load_n(src + 4 * lane, x);
    load_n(src + 4 * lane + partner_of<4>(p, 4 * lane), y);
    const Turn<4> turn = load_turn<4>(p, pos, 4 * lane);
    turn_row(p, turn, src, 4 * lane, x, y);
  }
}

template <bool kFour, class T>
__device__ __forceinline__ void append_row(const AppendRowsParams& p, int64_t row, int h, bool is_v, int lane) {
  int b;
  int64_t pos;
  if (!row_place(p, row, lane, b, pos)) return;
  if (!pos_ok(p, pos)) return flag(p.err, lane, CAI_DEVERR_LENGTH);
  const int P = p.page_size;
  const int32_t page = p.table[(int64_t)b * p.max_pages + (pos >> page_log2(P))];
  if (page < 0 || page >= p.num_pages[h]) return flag(p.err, lane, CAI_DEVERR_PAGE);
  const int slot = (int)pos & (P - 1);
  float x[4];
  load_row<T>(p, row, h, is_v, pos, lane, x);
  if constexpr (kFour)
    store_row4(p.pages[h] + (int64_t)page * page_bytes4(P) + (slot / kBlk) * kBlkBytes, slot % kBlk, is_v, lane, x);
  else
    store_row8(p.pages[h] + (int64_t)page * page_bytes(P), P, slot, is_v, lane, x);
}

// Whether sequence b has rows in the u-th group of 16 aligned positions from its first one on.
template <class Params>
__device__ __forceinline__ bool has_group(const Params& p, int b, int64_t u) {
  const int n = new_rows(p, b).n;
  const int64_t start = n > 0 ? p.start_pos[b] : 0;
  return n > 0 && start + n > ((start >> 4) + u) * kBlk;
}

// The u-th group of 16 aligned positions that sequence b writes, head h's K and V, by a block: warp w takes
// tokens w and w + 8.  K rows and the rows of a group that is not written whole go out as they come;
// a whole group's V codes are gathered in shared memory ([token][channel] bytes).
template <bool kFour, class T>
__device__ __forceinline__ void append_group(const AppendRowsParams& p, int b, int64_t u, int h, uint32_t (*codes)[kHeadDim / 4]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const NewRows nr = new_rows(p, b);
  if (nr.n <= 0) return;
  const int64_t start = p.start_pos[b];
  const int64_t pos0 = ((start >> 4) + u) * kBlk;
  const int lo = (int)(start > pos0 ? start - pos0 : 0);
  const int64_t left = start + nr.n - pos0;
  if (left <= 0) return;
  int hi = (int)(left < kBlk ? left : kBlk);
  const int P = p.page_size;
  if (pos0 < 0 || pos0 >= (int64_t)p.max_pages * P) return flag(p.err, threadIdx.x, CAI_DEVERR_LENGTH);
  if (p.rot > 0 && pos0 + hi > p.num_positions) {
    flag(p.err, threadIdx.x, CAI_DEVERR_LENGTH);
    if (pos0 + lo >= p.num_positions) return;
    hi = (int)(p.num_positions - pos0);
  }
  const int32_t page = p.table[(int64_t)b * p.max_pages + (pos0 >> page_log2(P))];
  const int64_t row0 = nr.r0 + (pos0 - start);
  const bool whole = lo == 0 && hi == kBlk;
  float x[2][2][4];  // [token][K, V]
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = warp + 8 * k;
    if (r < lo || r >= hi) continue;
    load_row<T>(p, row0 + r, h, true, pos0 + r, lane, x[k][1]);
    load_row<T>(p, row0 + r, h, false, pos0 + r, lane, x[k][0]);
  }
  if (page < 0 || page >= p.num_pages[h]) return flag(p.err, threadIdx.x, CAI_DEVERR_PAGE);
  const int s0 = (int)pos0 & (P - 1);
  uint8_t* pg = p.pages[h] + (int64_t)page * (kFour ? page_bytes4(P) : page_bytes(P));
  uint8_t* blk = pg + s0 / kBlk * kBlkBytes;  // (4-bit)
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = warp + 8 * k;
    if (r < lo || r >= hi) continue;
    if constexpr (kFour) {
      store_row4(blk, r, false, lane, x[k][0]);
      if (whole) {
        __half sh;
        codes[r][lane] = quantize4(x[k][1], sh);
        if ((lane & 7) == 0)
          *reinterpret_cast<__half*>(blk + kBlkVs + (((r & 7) >> 1) * 16 + (r >> 3) * 8 + (lane >> 3) * 2 + (r & 1)) * 2) = sh;
      } else {
        store_row4(blk, r, true, lane, x[k][1]);
      }
    } else {
      store_row8(pg, P, s0 + r, false, lane, x[k][0]);
      if (whole) {
        float s;
        codes[r][lane] = quantize8(x[k][1], s);
        if (lane == 0) reinterpret_cast<float*>(pg + 2 * P * kHeadDim)[P + s0 + r] = s;
      } else {
        store_row8(pg, P, s0 + r, true, lane, x[k][1]);
      }
    }
  }
  if (!whole) return;
  __syncthreads();
  const uint8_t* cb = reinterpret_cast<const uint8_t*>(codes);
  const int i = threadIdx.x;
  if constexpr (kFour) {
    // Word i = ((h2 * 8 + g) * 4 + t) * 4 + w (m = 4 h2 + w): channels 16 m + g and + 8 of tokens
    // 2 t, 2 t + 8, 2 t + 1, 2 t + 9, a byte each.
    const int t = i >> 2 & 3, ch = 16 * (4 * (i >> 7) + (i & 3)) + (i >> 4 & 7);
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint8_t* c = cb + (2 * t + (e >> 1) + 8 * (e & 1)) * kHeadDim + ch;
      w |= (uint32_t)(c[0] | (c[8] << 4)) << (8 * e);
    }
    reinterpret_cast<uint32_t*>(blk + kBlkV)[i] = w;
  } else {
    // Channel i's (i < 128) 16 codes; two threads a channel, eight codes each.
    const int ch = i >> 1, r0 = 8 * (i & 1);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e >> 2] |= (uint32_t)cb[(r0 + e) * kHeadDim + ch] << (8 * (e & 3));
    *reinterpret_cast<uint2*>(pg + P * kHeadDim + ch * P + s0 + r0) = make_uint2(w[0], w[1]);
  }
}

// (Four blocks an SM at 64 registers, or three at 77: 6353 rows of 32 heads 30.2 or 34.5 us, a decode step of
// 256 sequences 5.0 or 5.6.)
// kMany: there are fewer blocks than groups that every sequence might have; a block looks through its share of these, 32
// at a time, for those with rows.  (A prompt of 4096 tokens beside 135 single ones, 8 K/V heads: 44 us, a block for each
// possible group 350.)
template <bool kFour, class T, bool kMany>
__global__ void __launch_bounds__(kRowWarps * 32, 4) append_rows_kernel(const __grid_constant__ AppendRowsParams p) {
  __shared__ uint32_t codes[kBlk][kHeadDim / 4];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t rows = p.q_off ? p.total_new : (int64_t)p.batch * p.n_new;
  int64_t blk = blockIdx.x;
  if (blk < p.kv_blocks) {
    if (p.groups > 0) {
      auto place = [&](int64_t item, int& b, int64_t& u, int& h) {
        const int64_t i = over(item, p.num_kv_heads);
        h = (int)(item - i * p.num_kv_heads);
        b = (int)over(i, p.groups);
        u = i - (int64_t)b * p.groups;
      };
      int b, h;
      int64_t u;
      if constexpr (kMany) {
        const int64_t items = (int64_t)p.batch * p.groups * p.num_kv_heads;
        for (; blk < items; blk += 32ll * p.kv_blocks) {
          const int64_t mine = blk + (int64_t)lane * p.kv_blocks;
          bool rows_there = false;
          if (mine < items) {
            place(mine, b, u, h);
            rows_there = has_group(p, b, u);
          }
          for (uint32_t m = __ballot_sync(0xffffffffu, rows_there); m; m &= m - 1) {  // (the same in all warps)
            place(blk + (int64_t)(__ffs(m) - 1) * p.kv_blocks, b, u, h);
            append_group<kFour, T>(p, b, u, h, codes);
            __syncthreads();  // the codes are read
          }
        }
      } else {
        place(blk, b, u, h);
        append_group<kFour, T>(p, b, u, h, codes);
      }
      return;
    }
    const int64_t w = blk * kRowWarps + warp, row = over(w, 2 * p.num_kv_heads);
    const int unit = (int)(w - row * (2 * p.num_kv_heads));
    const bool is_v = unit >= p.num_kv_heads;
    if (row < rows) append_row<kFour, T>(p, row, is_v ? unit - p.num_kv_heads : unit, is_v, lane);
    return;
  }
  blk -= p.kv_blocks;
  if (blk < p.q_blocks) {
    const int per = (p.num_q_heads + kQHeads - 1) / kQHeads;  // warps of a token
    const int64_t w = blk * kRowWarps + warp, row = over(w, per);
    if (row < rows) rotate_queries(p, row, (int)(w - row * per) * kQHeads, lane);
    return;
  }
  // Packed offsets.
  for (int b = threadIdx.x; b < p.batch; b += kRowWarps * 32)
    if (new_rows(p, b).n < 0 && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
}

// Rows out.
__device__ __forceinline__ void store_n(float* dst, const float (&x)[4]) {
  *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store_n(uint16_t* dst, const float (&x)[4]) { *reinterpret_cast<uint2*>(dst) = to_bf16x4(x); }
__device__ __forceinline__ void store_n(float* dst, const float (&x)[8]) {
  if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {  // a whole sector (outputs are 16-byte aligned at least)
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(x[0]), "f"(x[1]), "f"(x[2]),
                 "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
  } else {
    reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}
__device__ __forceinline__ void store_n(uint16_t* dst, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(dst) =
      make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store_two(float* dst, float a, float b) { *reinterpret_cast<float2*>(dst) = make_float2(a, b); }
__device__ __forceinline__ void store_two(uint16_t* dst, float a, float b) { *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(a, b); }

// Eight fp16 values -> fp32.
__device__ __forceinline__ void widen(const uint4& v, float (&x)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[e]));
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
}

// One warp per (16 aligned tokens, K/V head, K or V).
constexpr int kVRow = kHeadDim + 8;  // fp16 of a token's row in shared memory (bank spread)
template <bool kFour, class T>
__device__ __forceinline__ void read_group(const ReadRowsParams& p, int64_t w, int b, int lane, uint16_t* st) {
  const int units = 2 * p.num_kv_heads;
  const int64_t u = over(w, units);  // group of 16 positions, counted from start_pos's
  const int unit = (int)(w - u * units), h = unit >> 1;
  const NewRows nr = new_rows(p, b);
  if (nr.n < 0 && w == 0 && lane == 0 && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
  if (nr.n <= 0) return;
  const int64_t start = p.start_pos[b];
  const int64_t group = (start >> 4) + u;  // (floor, also below 0)
  const int64_t pos0 = group * kBlk;
  const int lo = (int)(start > pos0 ? start - pos0 : 0);  // tokens [lo, hi) of the group are asked for
  const int64_t left = start + nr.n - pos0;
  if (left <= 0) return;
  const int hi = (int)(left < kBlk ? left : kBlk);
  const int P = p.page_size;
  int bad = pos0 < 0 || pos0 >= (int64_t)p.max_pages * P ? CAI_DEVERR_LENGTH : 0;
  int32_t page = 0;
  if (!bad) {
    page = p.table[(int64_t)b * p.max_pages + (pos0 >> page_log2(P))];
    if (page < 0 || page >= p.num_pages[h]) bad = CAI_DEVERR_PAGE;
  }
  const int64_t step = (int64_t)p.num_kv_heads * kHeadDim;  // elements from one row to the next
  const int64_t out0 = (nr.r0 + (pos0 - start)) * step + (int64_t)h * kHeadDim;  // of the group's token 0
  T* ko = unit & 1 ? nullptr : static_cast<T*>(p.k_out);
  T* vo = unit & 1 ? static_cast<T*>(p.v_out) : nullptr;
  if (bad) {
    if (lane == 0 && p.err) atomicOr(p.err, bad);
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    for (int r = lo; r < hi; ++r) {
      if (ko) store_n(ko + out0 + r * step + 4 * lane, zero);
      if (vo) store_n(vo + out0 + r * step + 4 * lane, zero);
    }
    return;
  }
  if constexpr (kFour) {
    const uint8_t* blk = p.pages[h] + (int64_t)page * page_bytes4(P) + ((int)pos0 & (P - 1)) / kBlk * kBlkBytes;
    const int g = lane >> 2, t = lane & 3;
    if (ko) {
      // Lane (g, t) holds channels 32 j + 8 t .. + 7 of tokens g and g + 8.
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * e + g;
        const uint4 kw = *reinterpret_cast<const uint4*>(blk + e * 512 + lane * 16);
        const uint2 sc = *reinterpret_cast<const uint2*>(blk + kBlkKs + r * 8);
        const uint32_t ws[4] = {kw.x, kw.y, kw.z, kw.w};
        if (r >= lo && r < hi) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t s = __byte_perm(j < 2 ? sc.x : sc.y, 0u, j & 1 ? 0x3232u : 0x1010u);
            uint32_t v[4];
            float x[8];
            values_f16(ws[j], s, s, v);
            widen(make_uint4(v[0], v[1], v[2], v[3]), x);
            store_n(ko + out0 + r * step + 32 * j + 8 * t, x);
          }
        }
      }
    }
    if (vo) {
      // V comes a channel per lane: transposed 8 x 8 in registers, gathered to rows in shared memory.
      const uint4 s0 = *reinterpret_cast<const uint4*>(blk + kBlkVs + t * 32);
      const uint4 s1 = *reinterpret_cast<const uint4*>(blk + kBlkVs + t * 32 + 16);
      const uint32_t sa[4] = {s0.x, s0.y, s0.z, s0.w}, sb[4] = {s1.x, s1.y, s1.z, s1.w};
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const uint4 vw = *reinterpret_cast<const uint4*>(blk + kBlkV + hh * 512 + lane * 16);
        const uint32_t ws[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int m = hh * 4 + k, j = m >> 1;
          uint32_t x[4];
          values_f16(ws[k], sa[j], sb[j], x);
#pragma unroll
          for (int i = 0; i < 4; ++i)  // channels 16 m + 8 (i % 2) + 2 t, + 1 of token 8 (i / 2) + g
            *reinterpret_cast<uint32_t*>(st + (8 * (i >> 1) + g) * kVRow + 16 * m + 8 * (i & 1) + 2 * t) = transpose8x8(x[i]);
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // two tokens at a time, eight channels a lane
        const int r = 2 * i + (lane >> 4), c = 8 * (lane & 15);
        if (r >= lo && r < hi) {
          float x[8];
          widen(*reinterpret_cast<const uint4*>(st + r * kVRow + c), x);
          store_n(vo + out0 + r * step + c, x);
        }
      }
    }
  } else {
    const uint8_t* pg = p.pages[h] + (int64_t)page * page_bytes(P);
    const float* sc = reinterpret_cast<const float*>(pg + 2 * P * kHeadDim);
    const int s0 = (int)pos0 & (P - 1);
    if (ko) {
      const float ks = sc[s0 + (lane & 15)];
      uint32_t kw[kBlk];
#pragma unroll
      for (int r = 0; r < kBlk; ++r)
        kw[r] = r >= lo && r < hi ? reinterpret_cast<const uint32_t*>(pg + (s0 + r) * kHeadDim)[lane] : 0u;
#pragma unroll
      for (int r = 0; r < kBlk; ++r) {
        const float s = __shfl_sync(0xffffffffu, ks, r);
        const float x[4] = {(float)(int8_t)kw[r] * s, (float)(int8_t)(kw[r] >> 8) * s, (float)(int8_t)(kw[r] >> 16) * s,
                            (float)(int8_t)(kw[r] >> 24) * s};
        if (r >= lo && r < hi) store_n(ko + out0 + r * step + 4 * lane, x);
      }
    }
    if (vo) {
      // Channels 64 i + 2 lane, + 1: 16 tokens of a channel are one 16-byte load.
      const float vs = sc[P + s0 + (lane & 15)];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* v = pg + P * kHeadDim + (64 * i + 2 * lane) * P + s0;
        const uint4 a = *reinterpret_cast<const uint4*>(v), c = *reinterpret_cast<const uint4*>(v + P);
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int r = 0; r < kBlk; ++r) {
          const float s = __shfl_sync(0xffffffffu, vs, r);
          if (r >= lo && r < hi)
            store_two(vo + out0 + r * step + 64 * i + 2 * lane, (float)(int8_t)(aw[r >> 2] >> (8 * (r & 3))) * s,
                      (float)(int8_t)(cw[r >> 2] >> (8 * (r & 3))) * s);
        }
      }
    }
  }
}

// kMany: as in append_rows_kernel, a warp looking through the (sequence, group, unit) triples.
template <bool kFour, class T, bool kMany>
__global__ void __launch_bounds__(kRowWarps * 32) read_rows_kernel(const __grid_constant__ ReadRowsParams p) {
  __shared__ __align__(16) uint16_t stage[kFour ? kRowWarps : 1][kFour ? kBlk * kVRow : 8];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint16_t* st = stage[kFour ? warp : 0];
  int64_t w = (int64_t)blockIdx.x * kRowWarps + warp;
  if constexpr (kMany) {
    const int units = 2 * p.num_kv_heads, groups = p.groups;
    const int64_t items = (int64_t)p.batch * groups * units, step = (int64_t)gridDim.x * kRowWarps;
    for (; w < items; w += 32 * step) {
      const int64_t mine = w + lane * step;
      bool rows_there = false;
      if (mine < items) {
        const int64_t i = over(mine, units);
        const int b = (int)over(i, groups);
        rows_there = has_group(p, b, i - (int64_t)b * groups);
        if (mine == (int64_t)b * groups * units && new_rows(p, b).n < 0 && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
      }
      for (uint32_t m = __ballot_sync(0xffffffffu, rows_there); m; m &= m - 1) {
        const int64_t item = w + (__ffs(m) - 1) * step;
        const int b = (int)over(over(item, units), groups);
        read_group<kFour, T>(p, item - (int64_t)b * groups * units, b, lane, st);
        __syncwarp();  // the staged rows are read
      }
    }
  } else {
    read_group<kFour, T>(p, w, blockIdx.y, lane, st);
  }
}

}  // namespace

namespace {

// Groups of 16 positions that a sequence's new tokens touch at most, from any position.
template <class Params>
int32_t most_groups(const Params& p) {
  return (int32_t)(((int64_t)(p.q_off ? std::min(p.n_new, p.total_new) : p.n_new) + 2 * kBlk - 2) / kBlk);
}

template <bool kFour, class T>
cudaError_t launch_append_many(const AppendRowsParams& p, unsigned grid, bool many, cudaStream_t stream) {
  return many ? launch_pdl(append_rows_kernel<kFour, T, true>, dim3(grid), dim3(kRowWarps * 32), 0, stream, p)
              : launch_pdl(append_rows_kernel<kFour, T, false>, dim3(grid), dim3(kRowWarps * 32), 0, stream, p);
}
template <bool kFour, class T>
cudaError_t launch_read_many(const ReadRowsParams& p, dim3 grid, bool many, cudaStream_t stream) {
  return many ? launch_pdl(read_rows_kernel<kFour, T, true>, grid, dim3(kRowWarps * 32), 0, stream, p)
              : launch_pdl(read_rows_kernel<kFour, T, false>, grid, dim3(kRowWarps * 32), 0, stream, p);
}

}  // namespace

cudaError_t launch_append_rows(AppendRowsParams p, bool four, bool bf16, cudaStream_t stream) {
  const int64_t rows = p.q_off ? p.total_new : (int64_t)p.batch * p.n_new;
  const auto blocks = [](int64_t warps) { return (warps + kRowWarps - 1) / kRowWarps; };
  const int64_t q_blocks = blocks(rows * ((p.num_q_heads + kQHeads - 1) / kQHeads));
  // Chunks by groups of 16 positions, fewer new tokens by rows (64 sequences, 8 K/V heads, int8: 8 tokens 9.2 us by groups
  // and 8.3 by rows, 16 tokens 13.7 and 13.4, 64 tokens 22.5 and 43.4; 4-bit 5.8 and 5.2, 8.3 and 8.8, 19.4 and 28.5).
  p.groups = p.n_new >= kBlk ? most_groups(p) : 0;
  const int64_t seqs = (int64_t)p.batch * p.num_kv_heads;
  // (Ragged batches: one wave of blocks that look for their groups.  6353 rows of 48 sequences 28.8 us, with a block
  // for each possible group 30.1.)
  const int64_t wave = (int64_t)num_sms() * 4;
  const bool many = p.q_off && p.groups * seqs > wave;
  const int64_t kv_blocks = many ? wave : p.groups ? seqs * p.groups : blocks(rows * 2 * p.num_kv_heads);
  const int64_t grid = q_blocks + kv_blocks + (p.q_off ? 1 : 0);
  if (grid > 2147483647ll) return cudaErrorInvalidValue;
  p.q_blocks = (int32_t)q_blocks;
  p.kv_blocks = (int32_t)kv_blocks;
  p.wide_tables = ((reinterpret_cast<uintptr_t>(p.cos) | reinterpret_cast<uintptr_t>(p.sin)) & 15) == 0;
  const unsigned g = (unsigned)grid;
  if (four) return bf16 ? launch_append_many<true, uint16_t>(p, g, many, stream) : launch_append_many<true, float>(p, g, many, stream);
  return bf16 ? launch_append_many<false, uint16_t>(p, g, many, stream) : launch_append_many<false, float>(p, g, many, stream);
}

cudaError_t launch_read_rows(ReadRowsParams p, bool four, bool bf16, cudaStream_t stream) {
  p.groups = most_groups(p);
  const int64_t warps = (int64_t)p.groups * 2 * p.num_kv_heads;
  const int64_t per = (warps + kRowWarps - 1) / kRowWarps;
  // (Here looking for the groups pays only where most have no rows: 64 sequences of up to 1024 tokens, of four K/V
  // heads, take 14 us with a warp for each possible group and 22 so; the prompt beside 135 tokens 75 and 12.)
  const int64_t wave = (int64_t)num_sms() * 8;
  const bool many = p.q_off && per * p.batch > 4 * wave;
  const dim3 grid((unsigned)(many ? wave : per), (unsigned)(many ? 1 : p.batch));
  if (four) return bf16 ? launch_read_many<true, uint16_t>(p, grid, many, stream) : launch_read_many<true, float>(p, grid, many, stream);
  return bf16 ? launch_read_many<false, uint16_t>(p, grid, many, stream) : launch_read_many<false, float>(p, grid, many, stream);
}

}  // namespace cai

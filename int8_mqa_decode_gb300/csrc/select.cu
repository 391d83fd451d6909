// Selection of pages: for every row of queries and K/V head the pages in which it may have its largest logits.
//
// A query head's channels become whole numbers, q_c -> rint(q_c / t) with t = max |q_c| / 127; with a page's codes
// (summary.cu) D = sum_c max(q_c lo_c, q_c hi_c) bounds q . k / (t s) over the page's keys up to the roundings; the
// page's score is s max_h (t_h D_h) over the heads of the group.  D is a whole number below 128 * 127^2 < 2^21, exact in
// fp32 however it is summed; the two products are rounded once each: a score is the same number on any path, and so is
// the selection.  The first and last pages of a row's context are always taken, the others by score, ties by the lower page.
//
// As a product: with q+ = max(q, 0), q- = min(q, 0), D = q+ . hi + q- . lo, so pages are the rows (256 codes) and heads
// the columns of one matrix product: tcgen05.mma kind::f16 (codes are exact in fp16), 128 pages by up to 128 columns (query
// rows x heads of a sequence), K = 256.  A block keeps its columns in shared memory and goes through tiles of pages:
// its eight warps turn the codes, 16 bytes of a row a lane, into the A operand in tensor memory as they come (the order of
// the columns' channels follows), one lane issues the products, and while they run the next tile's codes are on their
// way; then a thread has a page and all columns, and takes the largest of each query row.  Two blocks share an SM, one
// converting while the other's products run.
//
// Measured: 4096 rows of 32 heads over 528 pages 67 us, of them 55 the scores: a block takes 7 thousand cycles until its first
// products (positions, page ids, codes and queries come one behind the other; what needs no position is loaded first, 71 us
// without that) and 3600 a tile of 128 columns, two blocks side by side: conversion 1300, products 1000 to 1400, of which
// the tensor pipe needs 1024, reading D 1000.  64 rows of 64 heads over 256 to 2048 pages 20 us, mostly latencies.
// Products in halves of the channels and columns, so that conversion and reading run beside them, changed nothing (70 us, 37 to
// 39 at middle lengths): 4800 warp instructions a tile are what the four schedulers issue.  A persistent block with a kind of warp
// for each step took 58 us and 21, and contexts of middle length 51 us instead of 37: its readers of D, with 80 registers a
// thread, became the longest step.
#include <algorithm>

#include "ptx.cuh"
#include "rows.cuh"

namespace cai {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kCols = 128;                        // columns (query rows x heads) of a block at most
constexpr int kTilePages = 128;
constexpr int kColBytes = 2 * 2 * kHeadDim;       // q+ and q- of a column in fp16
constexpr uint32_t kTmem = 256, kColD = 128;      // tensor memory: A (128 columns), D

// Columns that a row's group of G heads takes: a power of two up to 8, then a multiple of 8.
__host__ __device__ inline int padded_heads(int G) { return G <= 1 ? 1 : G <= 2 ? 2 : G <= 4 ? 4 : (G + 7) / 8 * 8; }

// Tile `tile` of the call: rows [row0, row0 + n) of sequence b, at positions pos0 .. (n = 0: none).
struct RowTile {
  int b, n;
  int64_t row0, pos0;
};
__device__ __forceinline__ RowTile find_tile(const SelectParams& p, int64_t tile, int per, int* shared) {
  RowTile t = {};
  if (!p.q_off) {
    const int tiles = (p.n_new + per - 1) / per;
    t.b = (int)over(tile, tiles);
    const int i0 = (int)(tile - (int64_t)t.b * tiles) * per;
    t.n = min(per, p.n_new - i0);
    t.row0 = (int64_t)t.b * p.n_new + i0;
    t.pos0 = (int64_t)p.start_pos[t.b] + i0;
    return t;
  }
  // Tiles of the sequences before: every thread sums a run of them.
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (p.batch + kThreads - 1) / (kThreads);
  const int b0 = min(p.batch, tid * run), b1 = min(p.batch, b0 + run);
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) sum += (max(new_rows(p, b).n, 0) + per - 1) / per;
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  int64_t* sums = reinterpret_cast<int64_t*>(shared);  // [kWarps], then the answer
  RowTile* found = reinterpret_cast<RowTile*>(sums + kWarps);
  if (lane == 31) sums[warp] = incl;
  if (tid == 0) found->n = 0;
  __syncthreads();
  int64_t at = incl - sum;
  for (int w = 0; w < warp; ++w) at += sums[w];
  if (tile >= at && tile < at + sum) {  // one thread
    for (int b = b0;; ++b) {
      const NewRows nr = new_rows(p, b);
      const int tiles = (max(nr.n, 0) + per - 1) / per;
      if (tile < at + tiles) {
        const int i0 = (int)(tile - at) * per;
        t.b = b;
        t.n = min(per, nr.n - i0);
        t.row0 = nr.r0 + i0;
        t.pos0 = (int64_t)p.start_pos[b] + i0;
        break;
      }
      at += tiles;
    }
    *found = t;
  }
  __syncthreads();
  return *found;
}

__device__ __forceinline__ uint32_t half2_max0(uint32_t x) {
  uint32_t y;
  asm("max.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0u));
  return y;
}
__device__ __forceinline__ uint32_t half2_min0(uint32_t x) {
  uint32_t y;
  asm("min.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0u));
  return y;
}

// The largest of m and t_c D_c, over N columns.
template <int N>
__device__ __forceinline__ float largest(float m, const uint32_t (&r)[N], const float* scale_of) {
#pragma unroll
  for (int e = 0; e < N; e += 4) {
    const float4 t = *reinterpret_cast<const float4*>(scale_of + e);
    float z[4];
    f2_split(f2_mul(f2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), f2(t.x, t.y)), z[0], z[1]);
    f2_split(f2_mul(f2(__uint_as_float(r[e + 2]), __uint_as_float(r[e + 3])), f2(t.z, t.w)), z[2], z[3]);
    m = fmax3(fmax3(m, z[0], z[1]), z[2], z[3]);
  }
  return m;
}

// rint(x / t) clamped, the division IEEE.
__device__ __forceinline__ float whole(float x, float t) { return fminf(fmaxf(rintf(__fdiv_rn(x, t)), -127.0f), 127.0f); }

// Scores of a tile of rows over `span` tiles of their pages.  Block: (row tile, K/V head, span), the span fastest.
__global__ void __launch_bounds__(kThreads, 2) score_kernel(const __grid_constant__ SelectParams p, int per, int spans, int span) {
  extern __shared__ __align__(128) uint8_t cols[];  // column n, channels of unit u (8 of K's 256): (n / 8) 4096 + 128 u + 16 (n % 8)
  __shared__ __align__(16) float scale_of[kCols];
  __shared__ __align__(16) int shared[2 * kWarps + (sizeof(RowTile) + 3) / 4];
  __shared__ uint64_t done, drain;  // a tile's products; all products of a block that gives up
  __shared__ WaitState wait;
  __shared__ uint32_t slot;
  volatile WaitState* wctl = &wait;
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int64_t item = over(blockIdx.x, spans);
  const int64_t tile = over(item, p.num_kv_heads);
  const int h = (int)(item - tile * p.num_kv_heads);
  const RowTile rt = find_tile(p, tile, per, shared);
  if (rt.n == 0) return;
  // What does not depend on the position is loaded first: the columns' queries and the first pages' ids (of table entries that may
  // be past the context; these are not used).
  const int G = p.num_q_heads / p.num_kv_heads, gp = padded_heads(G);
  const int used = (rt.n * gp + 15) / 16 * 16;
  const int g = lane >> 2, t4 = lane & 3, quarter = warp & 3, half = warp >> 2;
  uint4 w[2][2];
  const auto load_q = [&](int n0) {
    const int n = n0 + g, i = n / gp, head = min(n - i * gp, G - 1);
    const uint4* q = reinterpret_cast<const uint4*>(p.q + ((rt.row0 + i) * p.num_q_heads + h * G + head) * kHeadDim + 16 * t4);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k) w[c][k] = n0 < used && i < rt.n ? __ldg(q + 8 * c + k) : make_uint4(0u, 0u, 0u, 0u);
  };
  const int c0 = (int)(blockIdx.x - item * spans) * span * kTilePages;
  const int32_t* table = p.table + (int64_t)rt.b * p.max_pages;
  const int first = 32 * quarter + 16 * half;
  int c1 = p.max_pages;
  const auto page_of = [&](int blk) -> int32_t { return blk < c1 ? __ldg(table + blk) : 0; };
  int32_t id[2];
  const auto load_ids = [&](int base) {
#pragma unroll
    for (int r = 0; r < 2; ++r) id[r] = page_of(base + first + g + 8 * r);
  };
  load_ids(c0);
  int32_t page_next = page_of(c0 + 32 * quarter + lane);  // of this thread's page of D
  load_q(8 * warp);

  const int lg = page_log2(p.page_size);
  const int64_t room = (int64_t)p.max_pages << lg, last_pos = min(rt.pos0 + rt.n, room);  // (rows outside are refused by the selection)
  if (last_pos <= 0 || rt.pos0 >= room) return;
  const int blocks = (int)((last_pos - 1) >> lg) + 1;  // of the last row
  c1 = min(c0 + span * kTilePages, blocks - p.last);
  if (blocks <= p.keep || c0 >= c1) return;

  if (warp == 0) tmem_alloc(&slot, kTmem);
  if (tid == 0) {
    mbar_init(&done, 1);
    mbar_init(&drain, 1);
    wait.abort = 0;
    wait.limit_ns = p.wait_ns;
    fence_barrier_init();
  }
  const uint8_t* data = p.data[h];
  const float* scales = reinterpret_cast<const float*>(data + (int64_t)p.num_pages[h] * (2 * kHeadDim));
  const auto in_pool = [&](int32_t page) { return (uint32_t)page < (uint32_t)p.num_pages[h]; };
  // This lane's 64 codes, 16 of every 64, of pages (quarter, half) 16 + g and + 8 of a tile; their ids are loaded a tile ahead
  // of the codes, these a tile ahead of their use.
  uint4 a[2][4];
  const auto there = [&](int base) { return base + first < c1; };  // (this warp has pages of the tile)
  const auto load = [&](int base) {
    if (!there(base)) return;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint4* row = reinterpret_cast<const uint4*>(data + (int64_t)(in_pool(id[r]) ? id[r] : 0) * (2 * kHeadDim)) + t4;
#pragma unroll
      for (int c = 0; c < 4; ++c) a[r][c] = __ldg(row + 4 * c);
    }
  };
  load(c0);
  load_ids(c0 + kTilePages);

  // Columns: whole numbers of the rows' heads, eight columns a warp, lane (g, t) channels 64 c + 16 t .. + 15 of column g: they
  // stand at words t of units 8 c + e (q+) and 16 + 8 c + e (q-).  A group that does not fill its columns repeats its
  // last head, columns past the rows are 0.
  for (int n0 = 8 * warp; n0 < used; n0 += 8 * kWarps) {
    const int n = n0 + g, i = n / gp, head = min(n - i * gp, G - 1);
    float y[32], amax = 0.0f;
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const uint4& v = w[x >> 3][x >> 2 & 1];
      const uint32_t u = (x & 3) == 0 ? v.x : (x & 3) == 1 ? v.y : (x & 3) == 2 ? v.z : v.w;
      y[2 * x] = __uint_as_float(u << 16);
      y[2 * x + 1] = __uint_as_float(u & 0xFFFF0000u);
      amax = fmax3(amax, fabsf(y[2 * x]), fabsf(y[2 * x + 1]));
    }
    load_q(n0 + 8 * kWarps);  // (under way while these are turned)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // x / t as the IEEE division rounds it, by one correction of the product with the rounded inverse (Markstein, 1990);
    // for bf16 numerators and t = amax / 127 every pair of significands was tried.  (A product alone is wrong for 24 pairs
    // of 188480, near halves: x = amax / 2 is one.)  Below 2^-100, where the correction may be subnormal, the division itself.
    const float t = __fdiv_rn(amax, 127.0f), inv = t >= 0x1p-100f ? __frcp_rn(t) : 0.0f;
    const uint64_t inv2 = f2(inv, inv), t2 = f2(-t, -t), magic = f2(12582912.0f, 12582912.0f), unmagic = f2(-12582912.0f, -12582912.0f);  // 3 2^22
    uint32_t* dst = reinterpret_cast<uint32_t*>(cols + (n0 >> 3) * (8 * kColBytes) + g * 16 + t4 * 4);
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const uint64_t y2 = f2(y[2 * x], y[2 * x + 1]), z = f2_mul(y2, inv2);
      float q0, q1;
      f2_split(f2_add(f2_add(f2_fma(f2_fma(z, t2, y2), inv2, z), magic), unmagic), q0, q1);
      const uint32_t q2 = pack_f16x2(q0, q1);
      dst[x * 32] = half2_max0(q2);
      dst[(16 + x) * 32] = half2_min0(q2);
    }
    if (t > 0.0f && inv == 0.0f) {
      const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + ((rt.row0 + i) * p.num_q_heads + h * G + head) * kHeadDim + 16 * t4);
#pragma unroll 1
      for (int x = 0; x < 16; ++x) {
        const uint32_t u = __ldg(src + (x >> 3) * 32 + (x & 7));
        const uint32_t q2 = pack_f16x2(whole(__uint_as_float(u << 16), t), whole(__uint_as_float(u & 0xFFFF0000u), t));
        dst[x * 32] = half2_max0(q2);
        dst[(16 + x) * 32] = half2_min0(q2);
      }
    }
    if (t4 == 0) scale_of[n] = t;
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, slot, 0);
  const uint32_t mine = tmem + ((uint32_t)(32 * quarter) << 16);
  const uint64_t dq = smem_desc(smem_addr(cols), 128, 8 * kColBytes);
  const uint32_t idesc = idesc_f16_f32(kTilePages, used, 0, 0);

  bool ok = true;
  int phase = 0;
  for (int base = c0; base < c1; base += kTilePages, phase ^= 1) {
    const int blk = base + 32 * quarter + lane;  // this thread's page of D
    const int32_t page = page_next;
    const bool good = in_pool(page);
    const float s = good ? __ldg(scales + page) : 0.0f;
    if (!good && blk < c1 && half == 0 && p.err) atomicOr(p.err, CAI_DEVERR_PAGE);
    page_next = page_of(blk + kTilePages);
    // ---- A: column 32 c + 4 e + t holds channels 64 c + 16 t + 2 e, + 1 of the 256 codes.  (Rows of pages that are not
    // there keep what they held: D's rows are independent.)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (!there(base)) break;
      uint32_t r[16];
      const uint32_t x[4] = {a[0][c].x, a[0][c].y, a[0][c].z, a[0][c].w}, y[4] = {a[1][c].x, a[1][c].y, a[1][c].z, a[1][c].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        i8x4_to_f16x4(x[e], r[4 * e], r[4 * e + 2]);
        i8x4_to_f16x4(y[e], r[4 * e + 1], r[4 * e + 3]);
      }
      tmem_st_16x128b_x8(mine + ((uint32_t)(16 * half) << 16) + 32 * c, r);
    }
    tmem_wait_st();
    tc_fence_before();
    __syncthreads();  // A is there, and D was read
    if (warp == 0) {
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 16; ++k) mma_f16_ts(tmem + kColD, tmem + 8 * k, dq + (uint64_t)(k * 16), idesc, k > 0 ? 1u : 0u);
        if ((base - c0) / kTilePages != p.drop_stage) mma_commit(&done);  // (fault injection: never said)
      }
      __syncwarp();
    }
    load(base + kTilePages);
    load_ids(base + 2 * kTilePages);
    ok = mbar_wait_lean(&done, phase, wctl) && ok;
    __syncwarp();
    tc_fence_after();
    // ---- D: the two warps of a quarter take rows (below 8 columns a row: groups of 8 columns) in turn.
    const auto put = [&](int i, float best) {
      if (i < rt.n && blk < c1)
        p.scores[((rt.row0 + i) * p.num_kv_heads + h) * p.stride + blk] =
            good ? __fadd_rn(__fmul_rn(best, s), 0.0f) : -INFINITY;  // (-0 becomes 0)
    };
    if (base + 32 * quarter >= c1) {
    } else if ((gp & 31) == 0) {
      for (int i = half; i < rt.n; i += 2) {
        float m = -INFINITY;
        for (int c = 0; c < gp; c += 32) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(mine + kColD + i * gp + c, r);
          tmem_wait_ld();
          m = largest(m, r, scale_of + i * gp + c);
        }
        put(i, m);
      }
    } else if (gp >= 8) {
      for (int i = half; i < rt.n; i += 2) {
        float m = -INFINITY;
        for (int c = 0; c < gp; c += 8) {
          uint32_t r[8];
          tmem_ld_32x32b_x8(mine + kColD + i * gp + c, r);
          tmem_wait_ld();
          m = largest(m, r, scale_of + i * gp + c);
        }
        put(i, m);
      }
    } else {
      for (int n0 = 8 * half; n0 < rt.n * gp; n0 += 16) {
        uint32_t r[8];
        tmem_ld_32x32b_x8(mine + kColD + n0, r);
        tmem_wait_ld();
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = __fmul_rn(__uint_as_float(r[e]), scale_of[n0 + e]);
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const int i = (n0 + e) / gp;
          if (gp == 1) {
            put(i, z[e]);
            put(i + 1, z[e + 1]);
            put(i + 2, z[e + 2]);
            put(i + 3, z[e + 3]);
          } else if (gp == 2) {
            put(i, fmaxf(z[e], z[e + 1]));
            put(i + 1, fmaxf(z[e + 2], z[e + 3]));
          } else {
            put(i, fmaxf(fmaxf(z[e], z[e + 1]), fmaxf(z[e + 2], z[e + 3])));
          }
        }
      }
    }
    tc_fence_before();
    if (__syncthreads_or(!ok)) break;  // (D is read; a wait that gave up stops the block)
  }
  if (tid == 0 && wctl->abort && p.err) atomicOr(p.err, CAI_DEVERR_TIMEOUT);
  tc_fence_after();
  if (warp == 0) {
    if (__any_sync(0xffffffffu, !ok)) {  // the products have ended before tensor memory goes
      if (elect_one()) mma_commit(&drain);
      __syncwarp();
      mbar_wait_drain(&drain, 0);
    }
    __syncwarp();
    tmem_dealloc(tmem, kTmem);
  }
}

// fp32 -> whole numbers of the same order.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}

// A score among values of which 0 means none and 0xFFFFFFFF one that is taken anyhow (both are orders of NaNs).
__device__ __forceinline__ uint32_t looked_at(uint32_t x) { return min(max(x, 1u), 0xFFFFFFFEu); }

// What a row takes.  b < 0: no sequence has it; n = 0: nothing (flagged by the caller where b >= 0).
struct Row {
  int b, n;
  int64_t pos;
};
__device__ __forceinline__ Row find_row(const SelectParams& p, int64_t row, int lane) {
  Row r = {-1, 0, -1};
  if (p.q_off) {
    int32_t a, e;
    r.b = find_seq(p.q_off, p.batch, row, lane, &a, &e);
    if (r.b >= 0 && !(a >= 0 && row < e && e <= p.total_new && e - a <= p.n_new)) r.b = -1;
    if (r.b >= 0) r.pos = (int64_t)p.start_pos[r.b] + (row - a);
  } else {
    r.b = (int)over(row, p.n_new);
    r.pos = (int64_t)p.start_pos[r.b] + (row - (int64_t)r.b * p.n_new);
  }
  const int lg = page_log2(p.page_size);
  if (r.b >= 0 && r.pos >= 0 && r.pos < (int64_t)p.max_pages << lg) r.n = (int)(r.pos >> lg) + 1;
  return r;
}
__device__ __forceinline__ int row_length(const SelectParams& p, const Row& r) {
  const int lg = page_log2(p.page_size);
  return r.n <= p.keep ? (int)r.pos + 1 : ((p.keep - 1) << lg) + (int)(r.pos & (p.page_size - 1)) + 1;
}
// The list of a row that takes all of its pages (or none), by `threads` threads.
__device__ __forceinline__ void take_all(const SelectParams& p, const Row& r, int h, int32_t* out, int tid, int threads) {
  const int32_t* table = p.table + (int64_t)max(r.b, 0) * p.max_pages;
  bool bad = false;
  for (int i = tid; i < p.keep; i += threads) {
    const int32_t page = i < r.n ? __ldg(table + i) : -1;
    bad |= i < r.n && (uint32_t)page >= (uint32_t)p.num_pages[h];
    out[i] = page;
  }
  if (bad && p.err) atomicOr(p.err, CAI_DEVERR_PAGE);
}

// The m-th largest of a group of threads' values, kItems each (0: none, 0xFFFFFFFF: not looked at): the values above
// `least` and the first `ties` of it are the m largest.  The eight bits from the first in which the values differ are
// counted in shared memory; the bin of the m-th largest holds few values, which are gathered and ranked, a thread each
// (more than the group has threads: the next eight bits).  Ranks are by value, then by place, so the order of
// gathering does not matter.
struct Found {
  uint32_t bin, need, total;  // of the values in the bin `need` are among the m largest
};
template <int kItems, class Group>
__device__ __forceinline__ void find_least(const Group& group, const uint32_t (&x)[kItems], int items, uint32_t m, uint32_t& least, uint32_t& ties) {
  uint32_t low = 0xFFFFFFFFu, high = 0u;
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    if (k % 4 == 0 && k >= items) break;
    low = min(low, x[k] - 1u);           // (none: the largest)
    high = max(high, x[k] + 1u);         // (not looked at: 0)
  }
  group.range(low, high);
  low += 1u;
  high -= 1u;
  uint32_t prefix = high, mask = 0xFFFFFFFFu;  // bits that are known
  if (low != high) {
    const int top = 31 - __clz(low ^ high);
    mask = ~((2u << top) - 1u);
    prefix = high & mask;
    for (int shift = max(top - 7, 0);; shift = max(shift - 8, 0)) {
      const uint32_t digit = ~mask >> shift;  // (as many ones as bits are unknown from `shift` up: 255 at most)
      group.clear();
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        if (k % 4 == 0 && k >= items) break;
        if ((x[k] & mask) == prefix && x[k] + 1u > 1u) atomicAdd(group.hist + ((x[k] >> shift) & digit), 1u);
      }
      const Found f = group.scan(m);
      prefix |= f.bin << shift;
      mask = ~((1u << shift) - 1u);
      m = f.need;
      if (shift == 0) break;
      if (f.total <= (uint32_t)Group::kThreadsIn) {
        // Gathered: the value, its place in the order of pages.
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
          if (k % 4 == 0 && k >= items) break;
          group.gather((x[k] & mask) == prefix && x[k] + 1u > 1u, make_uint2(x[k], k * Group::kThreadsIn + group.thread()));
        }
        group.rank(f.total, m, least, ties);
        return;
      }
    }
  }
  least = prefix;  // all bits are known
  ties = m;
}
// Bins of 256, from the largest on: that of the m-th value.  One warp; `hist` is read, not changed.
__device__ __forceinline__ Found scan_bins(const uint32_t* hist, uint32_t m, int lane) {
  uint32_t c[8], sum = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) sum += c[e] = hist[255 - 8 * lane - e];
  uint32_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  uint32_t before = incl - sum;
  Found f = {0, 0, 0};
  bool found = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (!found && before < m && before + c[e] >= m) {
      f = {(uint32_t)(255 - 8 * lane - e), m - before, c[e]};
      found = true;
    }
    before += c[e];
  }
  const int who = 31 - __clz(__ballot_sync(0xffffffffu, found) | 1u);  // (one lane)
  f.bin = __shfl_sync(0xffffffffu, f.bin, who);
  f.need = __shfl_sync(0xffffffffu, f.need, who);
  f.total = __shfl_sync(0xffffffffu, f.total, who);
  return f;
}
struct WarpGroup {
  static constexpr int kThreadsIn = 32;
  uint32_t* hist;   // [256]
  uint2* list;      // [kThreadsIn]
  mutable uint32_t gathered;
  __device__ __forceinline__ void gather(bool have, uint2 v) const {
    const uint32_t m = __ballot_sync(0xffffffffu, have);
    if (have) list[gathered + __popc(m & ((1u << thread()) - 1u))] = v;
    gathered += __popc(m);
  }
  __device__ __forceinline__ int thread() const { return threadIdx.x & 31; }
  __device__ __forceinline__ void range(uint32_t& low, uint32_t& high) const {
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
  }
  __device__ __forceinline__ void clear() const {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) reinterpret_cast<uint4*>(hist)[32 * i + thread()] = make_uint4(0u, 0u, 0u, 0u);
    __syncwarp();
  }
  __device__ __forceinline__ Found scan(uint32_t m) const {
    __syncwarp();
    return scan_bins(hist, m, thread());
  }
  __device__ __forceinline__ void rank(uint32_t total, uint32_t need, uint32_t& least, uint32_t& ties) const {
    __syncwarp();
    const bool have = (uint32_t)thread() < total;
    const uint2 mine = have ? list[thread()] : make_uint2(0u, 0u);
    uint32_t before = 0;  // values ahead of this one
#pragma unroll 4
    for (uint32_t i = 0; i < total; ++i) {
      const uint2 v = list[i];
      before += v.x > mine.x || (v.x == mine.x && v.y < mine.y) ? 1u : 0u;
    }
    const uint32_t who = __ballot_sync(0xffffffffu, have && before == need - 1);
    least = __shfl_sync(0xffffffffu, mine.x, 31 - __clz(who | 1u));
    const uint32_t above = __popc(__ballot_sync(0xffffffffu, have && mine.x > least)), equal = __popc(__ballot_sync(0xffffffffu, have && mine.x == least));
    ties = need - above;
    if (ties == equal) least -= 1, ties = 0;  // all of them are taken
  }
};
struct BlockGroup {
  static constexpr int kThreadsIn = kThreads;
  uint32_t* hist;   // [256], then [2 kWarps] of the range, [3] of the scan, [3] of the rank
  uint32_t* count;
  uint2* list;
  __device__ __forceinline__ void gather(bool have, uint2 v) const {
    if (have) list[atomicAdd(count, 1u)] = v;
  }
  __device__ __forceinline__ int thread() const { return threadIdx.x; }
  __device__ __forceinline__ void range(uint32_t& low, uint32_t& high) const {
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    uint32_t* part = hist + 256;
    if ((threadIdx.x & 31) == 0) {
      part[threadIdx.x >> 5] = low;
      part[kWarps + (threadIdx.x >> 5)] = high;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      low = min(low, part[w]);
      high = max(high, part[kWarps + w]);
    }
  }
  __device__ __forceinline__ void clear() const {
    hist[threadIdx.x] = 0u;  // (read before the scan's barrier, if at all)
    if (threadIdx.x == 0) *count = 0u;
    if (threadIdx.x < 3) hist[256 + 2 * kWarps + 3 + threadIdx.x] = 0u;
    __syncthreads();
  }
  __device__ __forceinline__ Found scan(uint32_t m) const {
    __syncthreads();
    uint32_t* got = hist + 256 + 2 * kWarps;
    if (threadIdx.x < 32) {
      const Found f = scan_bins(hist, m, threadIdx.x);
      if (threadIdx.x == 0) got[0] = f.bin, got[1] = f.need, got[2] = f.total;
    }
    __syncthreads();
    return Found{got[0], got[1], got[2]};
  }
  __device__ __forceinline__ void rank(uint32_t total, uint32_t need, uint32_t& least, uint32_t& ties) const {
    uint32_t* got = hist + 256 + 2 * kWarps + 3;  // the least value; of the gathered ones, those above it and equal
    __syncthreads();
    const bool have = threadIdx.x < total;
    const uint2 mine = have ? list[threadIdx.x] : make_uint2(0u, 0u);
    if (have) {
      uint32_t before = 0;
#pragma unroll 4
      for (uint32_t i = 0; i < total; ++i) {
        const uint2 v = list[i];
        before += v.x > mine.x || (v.x == mine.x && v.y < mine.y) ? 1u : 0u;
      }
      if (before == need - 1) got[0] = mine.x;
    }
    __syncthreads();
    least = got[0];
    const uint32_t above = __popc(__ballot_sync(0xffffffffu, have && mine.x > least)), equal = __popc(__ballot_sync(0xffffffffu, have && mine.x == least));
    if ((threadIdx.x & 31) == 0 && (above | equal)) {
      atomicAdd(got + 1, above);
      atomicAdd(got + 2, equal);
    }
    __syncthreads();
    ties = need - got[1];
    if (ties == got[2]) least -= 1, ties = 0;
  }
};

// A warp per (row, K/V head), for contexts of up to 32 kItems pages: the scores stay in registers, page 32 k + l in lane l.
// (Four blocks an SM leave 64 registers: with 1024 pages a thread spills 56 bytes.)
template <int kItems>
__global__ void __launch_bounds__(kThreads, 4) select_warp_kernel(const __grid_constant__ SelectParams p, int64_t units) {
  __shared__ __align__(16) uint32_t hist[kWarps][256];
  __shared__ uint2 list[kWarps][32];
  __shared__ uint16_t taken[kWarps][32 * kItems];  // the pages' numbers, in order
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (p.q_off && blockIdx.x == 0)
    for (int i = tid; i < p.batch; i += kThreads)
      if (new_rows(p, i).n < 0 && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
  const int64_t unit = (int64_t)blockIdx.x * kWarps + warp;
  if (unit >= units) return;
  const int64_t row = over(unit, p.num_kv_heads);
  const int h = (int)(unit - row * p.num_kv_heads);
  int32_t* out = p.pages_out + unit * p.keep;
  const float* scores = p.scores + unit * p.stride;
  uint32_t x[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {  // (under way while the row is found; those past its pages are not looked at)
    const int i = 32 * k + lane;
    x[k] = i < p.max_pages ? __float_as_uint(__ldcs(scores + i)) : 0u;
  }
  const Row r = find_row(p, row, lane);
  if (lane == 0) {
    if (r.n == 0 && r.b >= 0 && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
    if (h == 0) p.len_out[row] = r.n ? row_length(p, r) : 0;
  }
  if (r.n <= p.keep) return take_all(p, r, h, out, lane, 32);
  const int lo = p.first, hi = r.n - p.last, items = (r.n + 31) / 32;
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int i = 32 * k + lane;
    x[k] = i >= lo && i < hi ? looked_at(order_of(__uint_as_float(x[k]))) : i < r.n ? 0xFFFFFFFFu : 0u;
  }
  uint32_t least = 0xFFFFFFFEu, ties = 0;
  if (p.keep > p.first + p.last) find_least(WarpGroup{hist[warp], list[warp], 0u}, x, items, p.keep - p.first - p.last, least, ties);
  const int32_t* table = p.table + (int64_t)r.b * p.max_pages;
  const uint32_t below = (1u << lane) - 1u;
  int at = 0;
  uint32_t tied = 0;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    if (k % 4 == 0 && k >= items) break;
    const int i = 32 * k + lane;
    bool take = x[k] > least;
    if (ties > tied) {  // (the same in the whole warp)
      const bool tie = x[k] == least;
      const uint32_t m = __ballot_sync(0xffffffffu, tie);
      take |= tie && tied + __popc(m & below) < ties;
      tied += __popc(m);
    }
    const uint32_t m = __ballot_sync(0xffffffffu, take);
    const int to = at + __popc(m & below);
    if (take) taken[warp][to] = (uint16_t)i;
    at += __popc(m);
  }
  // (Their ids are loaded together: one by one in the loop above they took half of its time.)
  __syncwarp();
#pragma unroll 4
  for (int t = lane; t < min(at, p.keep); t += 32) {
    const int32_t page = __ldg(table + taken[warp][t]);
    bad |= (uint32_t)page >= (uint32_t)p.num_pages[h];
    out[t] = page;
  }
  if (bad && p.err) atomicOr(p.err, CAI_DEVERR_PAGE);
}

// A block per (row, K/V head), for contexts of up to 256 kItems pages: page 256 k + t in thread t.
template <int kItems>
__global__ void __launch_bounds__(kThreads) select_block_kernel(const __grid_constant__ SelectParams p) {
  __shared__ uint32_t hist[256 + 2 * kWarps + 6];
  __shared__ uint32_t gathered;
  __shared__ uint2 list[kThreads];
  __shared__ uint16_t taken[kItems * kThreads];
  __shared__ uint32_t counts[kItems * kWarps];  // pages taken, and of the least score, of item k in warp w: low and high half
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = over(blockIdx.x, p.num_kv_heads);
  const int h = (int)(blockIdx.x - row * p.num_kv_heads);
  int32_t* out = p.pages_out + (int64_t)blockIdx.x * p.keep;
  if (p.q_off && blockIdx.x == 0)
    for (int i = tid; i < p.batch; i += kThreads)
      if (new_rows(p, i).n < 0 && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
  const float* scores = p.scores + (int64_t)blockIdx.x * p.stride;
  uint32_t x[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {  // (as above)
    const int i = kThreads * k + tid;
    x[k] = i < p.max_pages ? __float_as_uint(__ldcs(scores + i)) : 0u;
  }
  const Row r = find_row(p, row, lane);
  if (tid == 0) {
    if (r.n == 0 && r.b >= 0 && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
    if (h == 0) p.len_out[row] = r.n ? row_length(p, r) : 0;
  }
  if (r.n <= p.keep) return take_all(p, r, h, out, tid, kThreads);
  const int lo = p.first, hi = r.n - p.last, items = (r.n + kThreads - 1) / kThreads;
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int i = kThreads * k + tid;
    x[k] = i >= lo && i < hi ? looked_at(order_of(__uint_as_float(x[k]))) : i < r.n ? 0xFFFFFFFFu : 0u;
  }
  uint32_t least = 0xFFFFFFFEu, ties = 0;
  if (p.keep > p.first + p.last) find_least(BlockGroup{hist, &gathered, list}, x, items, p.keep - p.first - p.last, least, ties);
  // Every (item, warp)'s counts, then what comes before it.
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    if (k % 4 == 0 && k >= items) break;
    const bool sure = x[k] > least, tie = ties > 0 && x[k] == least;
    const uint32_t ms = __ballot_sync(0xffffffffu, sure), mt = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) counts[k * kWarps + warp] = (uint32_t)__popc(ms) | (uint32_t)__popc(mt) << 16;
  }
  __syncthreads();
  if (warp == 0) {
    const int total = items * kWarps, run = (total + 31) / 32, i0 = min(total, lane * run), i1 = min(total, i0 + run);
    uint32_t sum = 0;
    for (int i = i0; i < i1; ++i) sum += counts[i];
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    uint32_t at = incl - sum;
    for (int i = i0; i < i1; ++i) {
      const uint32_t c = counts[i];
      counts[i] = at;
      at += c;
    }
  }
  __syncthreads();
  const int32_t* table = p.table + (int64_t)r.b * p.max_pages;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    if (k % 4 == 0 && k >= items) break;
    const bool sure = x[k] > least, tie = ties > 0 && x[k] == least;
    const uint32_t ms = __ballot_sync(0xffffffffu, sure), mt = __ballot_sync(0xffffffffu, tie);
    if (!(ms | mt)) continue;
    const uint32_t before = counts[k * kWarps + warp];
    const uint32_t rank = (before >> 16) + __popc(mt & below);           // ties before this page
    const uint32_t to = (before & 0xFFFFu) + __popc(ms & below) + min(rank, ties);
    if ((sure || (tie && rank < ties)) && to < (uint32_t)p.keep) taken[to] = (uint16_t)(kThreads * k + tid);
  }
  __syncthreads();
#pragma unroll 4
  for (int t = tid; t < p.keep; t += kThreads) {
    const int32_t page = __ldg(table + min((int)taken[t], r.n - 1));
    bad |= (uint32_t)page >= (uint32_t)p.num_pages[h];
    out[t] = page;
  }
  if (bad && p.err) atomicOr(p.err, CAI_DEVERR_PAGE);
}

// A block per (row, K/V head), for contexts of any length.  The keep - first - last largest of the scores between: their
// least by a radix search of eight bits at a time, then the pages in order, ties from the front.
__global__ void __launch_bounds__(kThreads) select_kernel(const __grid_constant__ SelectParams p) {
  __shared__ int hist[256];
  __shared__ uint32_t found[2];  // digits so far, how many of the least score are taken
  __shared__ int sums[2][kWarps];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = over(blockIdx.x, p.num_kv_heads);
  const int h = (int)(blockIdx.x - row * p.num_kv_heads);
  int32_t* out = p.pages_out + (int64_t)blockIdx.x * p.keep;
  if (p.q_off && blockIdx.x == 0)
    for (int i = tid; i < p.batch; i += kThreads)
      if (new_rows(p, i).n < 0 && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
  const Row r = find_row(p, row, lane);
  const int n = r.n;
  if (tid == 0) {
    if (n == 0 && r.b >= 0 && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
    if (h == 0) p.len_out[row] = n ? row_length(p, r) : 0;
  }
  if (n <= p.keep) return take_all(p, r, h, out, tid, kThreads);
  const int32_t* table = p.table + (int64_t)r.b * p.max_pages;
  const auto bad = [&](int32_t page) { return (uint32_t)page >= (uint32_t)p.num_pages[h]; };
  const float* scores = p.scores + (int64_t)blockIdx.x * p.stride;
  const int lo = p.first, hi = n - p.last;
  uint32_t least = 0xFFFFFFFFu, ties = 0;  // taken: scores above `least`, and the first `ties` of it
  if (p.keep > p.first + p.last) {
    uint32_t prefix = 0, mask = 0;
    int need = p.keep - p.first - p.last;
    for (int shift = 24; shift >= 0; shift -= 8) {
      hist[tid] = 0;
      __syncthreads();
      for (int i = lo + tid; i < hi; i += kThreads) {
        const uint32_t x = order_of(scores[i]);
        if ((x & mask) == prefix) atomicAdd(&hist[(x >> shift) & 255u], 1);
      }
      __syncthreads();
      if (warp == 0) {
        // Lane l: digits 255 - 8 l down to 248 - 8 l.
        int c[8], sum = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += c[e] = hist[255 - 8 * lane - e];
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        int before = incl - sum;
        if (before < need && incl >= need) {
          int e = 0;
          for (; before + c[e] < need; ++e) before += c[e];
          found[0] = prefix | (uint32_t)(255 - 8 * lane - e) << shift;
          found[1] = need - before;
        }
      }
      __syncthreads();
      prefix = found[0];
      need = (int)found[1];
      mask |= 255u << shift;
    }
    least = prefix;
    ties = need;
  }
  int at = 0;        // pages written by the block so far
  uint32_t tied = 0; // of the least score seen so far
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + tid;
    const bool forced = i < lo || i >= hi;
    const uint32_t x = i < n && !forced ? order_of(scores[i]) : 0u;
    const bool over_it = i < n && !forced && x > least, tie = i < n && !forced && ties > 0 && x == least;
    const uint32_t tm = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) sums[0][warp] = __popc(tm);
    __syncthreads();
    uint32_t rank = tied + __popc(tm & ((1u << lane) - 1u));
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) rank += sums[0][w];
      tied += sums[0][w];
    }
    const bool take = i < n && (forced || over_it || (tie && rank < ties));
    const uint32_t m = __ballot_sync(0xffffffffu, take);
    if (lane == 0) sums[1][warp] = __popc(m);
    __syncthreads();
    int to = at + __popc(m & ((1u << lane) - 1u));
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) to += sums[1][w];
      at += sums[1][w];
    }
    if (take && to < p.keep) {
      const int32_t page = table[i];
      if (bad(page) && p.err) atomicOr(p.err, CAI_DEVERR_PAGE);
      out[to] = page;
    }
  }
}

}  // namespace

cudaError_t launch_select(const SelectParams& p, cudaStream_t stream) {
  const int64_t rows = p.q_off ? p.total_new : (int64_t)p.batch * p.n_new;
  if (p.max_pages > p.keep) {  // some row may have more pages than it takes
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !attr_set[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCols * kColBytes);
      if (e != cudaSuccess) return e;
      if (dev < 64) attr_set[dev] = true;
    }
    const int gp = padded_heads(p.num_q_heads / p.num_kv_heads);
    const int most = p.q_off ? std::min(p.n_new, p.total_new) : p.n_new;
    const int per = std::max(1, std::min(most, kCols / gp));
    const int64_t tiles = p.q_off ? rows / per + p.batch : (int64_t)p.batch * ((p.n_new + per - 1) / per);
    // Page tiles of a block: as many as leave four blocks an SM.
    const int64_t units = tiles * p.num_kv_heads, page_tiles = ((int64_t)p.max_pages + kTilePages - 1) / kTilePages;
    const int64_t want = std::max<int64_t>(1, 4 * num_sms() / units);
    const int span = (int)((page_tiles + want - 1) / want), spans = (int)((page_tiles + span - 1) / span);
    const int64_t grid = units * spans;
    if (grid > 2147483647ll) return cudaErrorInvalidValue;
    const size_t smem = (size_t)((per * gp + 15) / 16 * 16) * kColBytes;
    const cudaError_t e = launch_pdl(score_kernel, dim3((unsigned)grid), dim3(kThreads), smem, stream, p, per, spans, span);
    if (e != cudaSuccess) return e;
  }
  const int64_t units = rows * p.num_kv_heads, warps = (units + kWarps - 1) / kWarps;
  if (units > 2147483647ll) return cudaErrorInvalidValue;
  const auto by_warps = [&](auto kernel) { return launch_pdl(kernel, dim3((unsigned)warps), dim3(kThreads), 0, stream, p, units); };
  if (p.max_pages <= 256) return by_warps(select_warp_kernel<8>);
  if (p.max_pages <= 1024) return by_warps(select_warp_kernel<32>);
  if (p.max_pages <= 32 * kThreads) return launch_pdl(select_block_kernel<32>, dim3((unsigned)units), dim3(kThreads), 0, stream, p);
  return launch_pdl(select_kernel, dim3((unsigned)units), dim3(kThreads), 0, stream, p);
}

}  // namespace cai

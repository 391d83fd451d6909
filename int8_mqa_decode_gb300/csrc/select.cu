// Selection of pages: for every row of queries and K/V head the pages in which it may have its largest logits.
//
// A query head's channels become whole numbers, q_c -> rint(q_c / t) with t = max |q_c| / 127; with a page's codes
// (summary.cu) D = sum_c max(q_c lo_c, q_c hi_c) bounds q . k / (t s) over the page's keys up to the roundings; the
// page's score is s max_h (t_h D_h) over the heads of the group.  D is a whole number below 128 * 127^2 < 2^21, exact in
// fp32 however it is summed; the two products are rounded once each: a score is the same number on any path, and so is
// the selection.  The first and last pages of a row's context are always taken, the others by score, ties by the lower page.
//
// As a product: with q+ = max(q, 0), q- = min(q, 0), D = q+ . hi + q- . lo, so pages are the rows (256 codes) and heads
// the columns of one matrix product.  mma.m16n8k16 in fp16: codes are exact in it, and become its A operand in
// registers (16 bytes of a row a lane, in the order of memory, with the same order of channels in B).
#include <algorithm>

#include "ptx.cuh"
#include "rows.cuh"

namespace cai {
namespace {

constexpr int kWarps = 8;
constexpr int kCols = 128;                       // columns (query rows x heads) of a block at most
constexpr int kColBytes = 2 * 2 * kHeadDim + 16; // q+ and q- of a column in fp16, and a shift of banks
constexpr int kChunk = 256;                      // pages of a block

// Columns that a row's group of G heads takes: a power of two up to 8, then a multiple of 8.
__host__ __device__ inline int padded_heads(int G) { return G <= 1 ? 1 : G <= 2 ? 2 : G <= 4 ? 4 : (G + 7) / 8 * 8; }

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

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
  const int run = (p.batch + kWarps * 32 - 1) / (kWarps * 32);
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

// Scores of a tile's rows over a chunk of their pages.  Block: (tile, K/V head, chunk), the chunk fastest.
__global__ void __launch_bounds__(kWarps * 32) score_kernel(const __grid_constant__ SelectParams p, int per, int chunks) {
  extern __shared__ __align__(16) uint8_t cols[];  // [columns][kColBytes]
  __shared__ float scale_of[kCols];
  __shared__ __align__(16) int shared[2 * kWarps + (sizeof(RowTile) + 3) / 4];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t item = over(blockIdx.x, chunks);
  const int chunk = (int)(blockIdx.x - item * chunks);
  const int64_t tile = over(item, p.num_kv_heads);
  const int h = (int)(item - tile * p.num_kv_heads);
  const RowTile rt = find_tile(p, tile, per, shared);
  if (rt.n == 0) return;
  const int lg = page_log2(p.page_size);
  const int64_t end = min(rt.pos0 + rt.n, (int64_t)p.max_pages << lg);  // positions past the table are refused by the selection
  if (end <= 0) return;
  const int blocks = (int)((end - 1) >> lg) + 1;  // of the last row
  const int c0 = chunk * kChunk, c1 = min(c0 + kChunk, blocks - p.last);
  if (blocks <= p.keep || c0 >= c1) return;

  // Columns: whole numbers of the rows' heads, fp16.  A group that does not fill its columns repeats its last head.
  const int G = p.num_q_heads / p.num_kv_heads, gp = padded_heads(G);
  const int used = (rt.n * gp + 7) / 8 * 8;
  for (int c = warp; c < used; c += kWarps) {
    const int i = c / gp, head = min(c - i * gp, G - 1);
    uint2 w = make_uint2(0u, 0u);
    if (i < rt.n)
      w = __ldg(reinterpret_cast<const uint2*>(p.q + ((rt.row0 + i) * p.num_q_heads + h * G + head) * kHeadDim) + lane);
    const float x[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                        __uint_as_float(w.y & 0xFFFF0000u)};
    float amax = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float t = __fdiv_rn(amax, 127.0f);
    float code[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) code[e] = t > 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(x[e], t)), -127.0f), 127.0f) : 0.0f;
    uint2* dst = reinterpret_cast<uint2*>(cols + c * kColBytes) + lane;
    dst[0] = make_uint2(pack_f16x2(fmaxf(code[0], 0.0f), fmaxf(code[1], 0.0f)), pack_f16x2(fmaxf(code[2], 0.0f), fmaxf(code[3], 0.0f)));
    dst[32] = make_uint2(pack_f16x2(fminf(code[0], 0.0f), fminf(code[1], 0.0f)), pack_f16x2(fminf(code[2], 0.0f), fminf(code[3], 0.0f)));
    if (lane == 0) scale_of[c] = t;
  }
  __syncthreads();

  const int g = lane >> 2, t = lane & 3;
  const int32_t* table = p.table + (int64_t)rt.b * p.max_pages;
  const uint8_t* data = p.data[h];
  const float* scales = reinterpret_cast<const float*>(data + (int64_t)p.num_pages[h] * (2 * kHeadDim));
  for (int base = c0 + 16 * warp; base < c1; base += 16 * kWarps) {
    // Rows of A: pages base + g and base + g + 8.
    uint32_t a[2][4][8];  // [row][64 codes][fp16 pairs]
    float s[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int blk = base + g + 8 * r;
      const int32_t page = blk < c1 ? __ldg(table + blk) : -1;
      const bool ok = (uint32_t)page < (uint32_t)p.num_pages[h];
      if (blk < c1 && !ok && t == 0 && p.err) atomicOr(p.err, CAI_DEVERR_PAGE);
      const uint4* row = reinterpret_cast<const uint4*>(data + (int64_t)(ok ? page : 0) * (2 * kHeadDim)) + t;
      s[r] = __ldg(scales + (ok ? page : 0));
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 w = __ldg(row + 4 * c);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) i8x4_to_f16x4(ws[e], a[r][c][2 * e], a[r][c][2 * e + 1]);
      }
      if (!ok) s[r] = -INFINITY;
    }
    float m[2] = {-INFINITY, -INFINITY};
    const int tiles = used / 8, per_row = gp / 8;  // (per_row 0: several rows a tile)
    int in_row = 0, row = 0;
    for (int n = 0; n < tiles; ++n) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      const uint8_t* col = cols + (8 * n + g) * kColBytes + 32 * t;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 b0 = *reinterpret_cast<const uint4*>(col + 128 * c), b1 = *reinterpret_cast<const uint4*>(col + 128 * c + 16);
        const uint32_t b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mma_16816(acc, a[0][c][2 * e], a[1][c][2 * e], a[0][c][2 * e + 1], a[1][c][2 * e + 1], b[2 * e], b[2 * e + 1]);
      }
      const float t0 = scale_of[8 * n + 2 * t], t1 = scale_of[8 * n + 2 * t + 1];
      const float z[4] = {__fmul_rn(acc[0], t0), __fmul_rn(acc[1], t1), __fmul_rn(acc[2], t0), __fmul_rn(acc[3], t1)};
      // The score of page `blk` for row i of the tile.
      const auto put = [&](int i, int r, float best) {
        const int blk = base + g + 8 * r;
        if (i < rt.n && blk < c1)
          p.scores[((rt.row0 + i) * p.num_kv_heads + h) * p.stride + blk] =
              s[r] == -INFINITY ? -INFINITY : __fadd_rn(__fmul_rn(best, s[r]), 0.0f);  // (-0 becomes 0)
      };
      if (per_row > 0) {
        m[0] = fmaxf(m[0], fmaxf(z[0], z[1]));
        m[1] = fmaxf(m[1], fmaxf(z[2], z[3]));
        if (++in_row == per_row) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            m[r] = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], 1));
            m[r] = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], 2));
          }
          if (t < 2) put(row, t, t ? m[1] : m[0]);
          ++row;
          in_row = 0;
          m[0] = m[1] = -INFINITY;
        }
      } else if (gp == 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) put(8 * n + 2 * t + (e & 1), e >> 1, z[e]);
      } else {
        float x[2] = {fmaxf(z[0], z[1]), fmaxf(z[2], z[3])};
        if (gp == 4) {
#pragma unroll
          for (int r = 0; r < 2; ++r) x[r] = fmaxf(x[r], __shfl_xor_sync(0xffffffffu, x[r], 1));
          if (!(t & 1)) put(2 * n + (t >> 1), 0, x[0]);
          else put(2 * n + (t >> 1), 1, x[1]);
        } else {
          put(4 * n + t, 0, x[0]);
          put(4 * n + t, 1, x[1]);
        }
      }
    }
  }
}

// fp32 -> whole numbers of the same order.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}

// A block per (row, K/V head).  The keep - first - last largest of the scores between: their least by a radix search of
// eight bits at a time, then the pages in order, ties from the front.
__global__ void __launch_bounds__(kWarps * 32) select_kernel(const __grid_constant__ SelectParams p) {
  __shared__ int hist[256];
  __shared__ uint32_t found[2];  // digits so far, how many of the least score are taken
  __shared__ int sums[2][kWarps];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = over(blockIdx.x, p.num_kv_heads);
  const int h = (int)(blockIdx.x - row * p.num_kv_heads);
  int32_t* out = p.pages_out + (int64_t)blockIdx.x * p.keep;
  int b = -1;
  int64_t pos = -1;
  if (p.q_off) {
    int32_t a, e;
    b = find_seq(p.q_off, p.batch, row, lane, &a, &e);
    if (b >= 0 && !(a >= 0 && row < e && e <= p.total_new && e - a <= p.n_new)) b = -1;
    if (b >= 0) pos = (int64_t)p.start_pos[b] + (row - a);
  } else {
    b = (int)over(row, p.n_new);
    pos = (int64_t)p.start_pos[b] + (row - (int64_t)b * p.n_new);
  }
  if (p.q_off && blockIdx.x == 0)
    for (int i = tid; i < p.batch; i += kWarps * 32)
      if (new_rows(p, i).n < 0 && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
  const int lg = page_log2(p.page_size);
  const bool ok = b >= 0 && pos >= 0 && pos < (int64_t)p.max_pages << lg;
  if (!ok) {
    if (b >= 0 && tid == 0 && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
    for (int i = tid; i < p.keep; i += kWarps * 32) out[i] = -1;
    if (h == 0 && tid == 0) p.len_out[row] = 0;
    return;
  }
  const int n = (int)(pos >> lg) + 1;
  const int32_t* table = p.table + (int64_t)b * p.max_pages;
  const auto bad = [&](int32_t page) { return (uint32_t)page >= (uint32_t)p.num_pages[h]; };
  if (h == 0 && tid == 0) p.len_out[row] = n <= p.keep ? (int)pos + 1 : ((p.keep - 1) << lg) + (int)(pos & (p.page_size - 1)) + 1;
  if (n <= p.keep) {
    for (int i = tid; i < p.keep; i += kWarps * 32) {
      const int32_t page = i < n ? table[i] : -1;
      if (i < n && bad(page) && p.err) atomicOr(p.err, CAI_DEVERR_PAGE);
      out[i] = page;
    }
    return;
  }
  const float* scores = p.scores + (int64_t)blockIdx.x * p.stride;
  const int lo = p.first, hi = n - p.last;
  uint32_t least = 0xFFFFFFFFu, ties = 0;  // taken: scores above `least`, and the first `ties` of it
  if (p.keep > p.first + p.last) {
    uint32_t prefix = 0, mask = 0;
    int need = p.keep - p.first - p.last;
    for (int shift = 24; shift >= 0; shift -= 8) {
      hist[tid] = 0;
      __syncthreads();
      for (int i = lo + tid; i < hi; i += kWarps * 32) {
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
  for (int i0 = 0; i0 < n; i0 += kWarps * 32) {
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
    const int64_t chunks = ((int64_t)p.max_pages + kChunk - 1) / kChunk;
    const int64_t grid = tiles * p.num_kv_heads * chunks;
    if (grid > 2147483647ll) return cudaErrorInvalidValue;
    const size_t smem = (size_t)((per * gp + 7) / 8 * 8) * kColBytes;
    const cudaError_t e = launch_pdl(score_kernel, dim3((unsigned)grid), dim3(kWarps * 32), smem, stream, p, per, (int)chunks);
    if (e != cudaSuccess) return e;
  }
  const int64_t grid = rows * p.num_kv_heads;
  if (grid > 2147483647ll) return cudaErrorInvalidValue;
  return launch_pdl(select_kernel, dim3((unsigned)grid), dim3(kWarps * 32), 0, stream, p);
}

}  // namespace cai

// Decode attention over the 4-bit paged cache (layout in kv4.cuh), grouped query heads, and the
// log-sum-exp merge of its splits.
//
// What it computes: for one query token per sequence and every query head, softmax over the attended
// positions of softmax_scale * <q, k> and the weighted sum of v, k and v being the values that the
// 4-bit codes stand for; query heads [j G, (j + 1) G) read K/V head j.
//
// This file has the split of the work, the kernel for groups of up to 8 heads and the merge; groups of 9
// and more are decode4_tc.cu's.
//
// How.  Every block walks its share of the keys (split plan below) in pieces of one sequence and K/V
// head.  Its four warps take steps of 32 keys in turn, each with a ring of its own that one lane fills by
// bulk copies, so no warp waits for another before a piece ends.  Scores are computed transposed,
// S^T = K Q^T with mma.m16n8k16 (16 keys x 8 heads): the codes become the A operand in registers, query
// heads fill the N side.  A column of S^T is one head: the running maximum is a reference per head,
// raised only when a logit passes it by 2^15, so the common step has no reduction across lanes.  P^T goes
// to the B operand by an 8 x 8 transpose in registers, and O^T += V^T P^T accumulates channels x heads
// in registers.  At the end of a piece the warps' parts are merged through the ring's shared memory.
//
// Roundings, here and in decode4_tc.cu: the query to fp16 (exact for magnitudes from 2^-17 to 65504, below that off by
// 2^-25 at most), a weight to fp16 for its product with V (2^-11 of it, or 2^-32 of the sum of all where that is more, see
// kWeightLift; the sums take it unrounded, in fp32), the output to bf16 once; partial outputs stay fp32.
//
// Why this tensor path: at up to 8 heads a 16-key group's 32 m16n8k16 and the conversion of its codes take
// a sub-partition about as long as its bytes take the SM at the copy bandwidth (long contexts of 8 heads:
// 142 us for 4.97 M keys, of 106 at the copy bandwidth).  The tensor memory kernel's products are padded
// to 16 heads and its hand-offs cost more than they save there (172 us); at 16 heads this kernel, with
// twice the mma, took 188.
#include <cmath>

#include "decode4.cuh"

namespace cai {
namespace {

constexpr int kWarps = 4;
constexpr int kStepBlks = 2;                          // groups of 16 keys of one step of a warp
constexpr int kStep = kStepBlks * kBlk;               // its keys
constexpr int kStepBytes = kStepBlks * kBlkBytes;     // 4608
constexpr int kIdSteps = 32 / kStepBlks;              // steps whose page ids a warp holds, one per lane
constexpr int kORow = kHeadDim + 4;                   // floats of a head's row in the merge buffer (bank spread)
constexpr float kRaise4 = kWeightLift + 8.0f;         // log2 units a logit may exceed its reference by

constexpr int kHeads4 = 8;
constexpr int kBlocks4 = 4, kStages4 = 3;             // blocks per SM, stages of a warp's ring: 221 KB in flight on an SM
constexpr int kRing4 = kWarps * kStages4 * kStepBytes;
static_assert(kRing4 >= kWarps * kHeads4 * kORow * 4, "the merge's buffer is in the ring, drained by then");
constexpr int kOffBars4 = kRing4;
constexpr int kOffOk4 = kOffBars4 + kWarps * kStages4 * 8;
constexpr int kOffMl4 = (kOffOk4 + kWarps * kStages4 * 4 + 15) & ~15;  // references [warp][head], sums [warp][head]
constexpr int kOffWait4 = kOffMl4 + 2 * kWarps * kHeads4 * 4;
constexpr int kOffPieces4 = kOffWait4 + 16;
constexpr int kSmem4 = kOffPieces4 + kPieces * (int)sizeof(Piece4) + 64;  // and the list's state
static_assert(kBlocks4 * (kSmem4 + 1024) <= 228 * 1024, "shared memory of an SM");

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

__device__ __forceinline__ float half_of(uint32_t x, int hi) {
  return __half2float(__ushort_as_half((unsigned short)(hi ? x >> 16 : x)));
}

__device__ __forceinline__ uint2 pack_bf16x4(float a, float b, float c, float d) {
  return make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

__global__ void __launch_bounds__(kWarps * 32, kBlocks4) decode4_kernel(const __grid_constant__ Decode4Params p) {
  constexpr int NS = kStages4;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBars4);
  volatile uint32_t* ok_bits = reinterpret_cast<volatile uint32_t*>(smem + kOffOk4);
  float* ml = reinterpret_cast<float*>(smem + kOffMl4);
  volatile WaitState* wctl = reinterpret_cast<volatile WaitState*>(smem + kOffWait4);
  Piece4* pieces = reinterpret_cast<Piece4*>(smem + kOffPieces4);
  List4& ls = *reinterpret_cast<List4*>(smem + kOffPieces4 + kPieces * sizeof(Piece4));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int c = blockIdx.x;
  const int G = p.num_heads / p.num_kv_heads;

  if (lane == 0) {
    for (int s = 0; s < NS; ++s) mbar_init(&bars[warp * NS + s], 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    wctl->abort = 0;
    wctl->limit_ns = p.wait_ns;
  }
  // A launch beside the kernel before it (overlap_prev) shares no memory with it, but ends only after
  // it: every block waits for it on leaving.
  if (!p.overlap_prev) grid_dependency_wait();
  grid_launch_dependents();
  start_list<kWarps * 32>(p, c, ls, reinterpret_cast<int64_t*>(ml));

  const int P = p.page_size;
  const int per_log2 = P == 16 ? 0 : P == 32 ? 1 : 2;  // groups of 16 tokens in a page
  uint8_t* ring = smem + warp * NS * kStepBytes;
  uint64_t* full = bars + warp * NS;
  // The warp's next step lies in stage st, the step after the last one issued in stage st_in; phase bit s is
  // the parity of the next wait on stage s.  r counts the warp's steps (for the fault injection alone).
  int st = 0, st_in = 0, r = 0;
  uint32_t phase = 0;
  bool ok = true;  // no wait of this warp gave up

  while (ls.more) {  // (the same for all: written before the barriers of start_list and of the loop's end)
    __syncthreads();
    if (warp == 0) next_pieces(p, c, ls, pieces);
    __syncthreads();
    for (int pi = 0; pi < ls.count; ++pi) {
      const Piece4 pc = pieces[pi];
      const int64_t row0 = (int64_t)pc.row * p.num_heads + (int64_t)pc.kvh * G;  // the first head row
      const int start = pc.start, end = pc.end;
      if (start >= end) {  // nothing to attend, or an invalid length (flagged): out = 0, lse = -inf
        for (int i = threadIdx.x; i < G * kHeadDim / 4; i += kWarps * 32)
          reinterpret_cast<uint2*>(p.out + row0 * kHeadDim)[i] = make_uint2(0u, 0u);
        if (p.lse_out && threadIdx.x < G) p.lse_out[row0 + threadIdx.x] = -INFINITY;
        continue;
      }
      const int blk0 = start / kBlk, nblk = (end - 1) / kBlk - blk0 + 1;
      const int steps = (nblk + kStepBlks - 1) / kStepBlks;
      const int mine = (steps - warp + kWarps - 1) / kWarps;  // this warp's steps: warp, warp + kWarps, ...
      const uint8_t* pages = p.pages[pc.kvh];
      const int num_pages = p.num_pages[pc.kvh];
      const int32_t* table = p.table + (int64_t)pc.b * p.max_pages;
      const uint16_t* q = p.q + row0 * kHeadDim;
      __syncthreads();  // the last piece's merge has left the ring

      // Page ids of the warp's next steps: lane kStepBlks i + h holds group h of step i of the batch.
      auto load_ids = [&](int i0) -> int32_t {
        const int i = i0 + lane / kStepBlks;
        const int blk = kStepBlks * (warp + i * kWarps) + lane % kStepBlks;
        return i < mine && blk < nblk ? __ldg(table + ((blk0 + blk) >> per_log2)) : -1;
      };
      int32_t ids = load_ids(0);
      int32_t ids_next = mine > kIdSteps ? load_ids(kIdSteps) : -1;
      int issued = 0;
      // Starts the copies of the warp's next step into stage st_in.
      auto issue = [&]() {
        const int i = issued++, s = st_in;
        st_in = s + 1 == NS ? 0 : s + 1;
        if (i % kIdSteps == 0 && i > 0) {
          ids = ids_next;
          ids_next = i + kIdSteps < mine ? load_ids(i + kIdSteps) : -1;
        }
        const int blk = kStepBlks * (warp + i * kWarps) + lane % kStepBlks;
        const int32_t pid = __shfl_sync(0xffffffffu, ids, kStepBlks * (i % kIdSteps) + lane % kStepBlks);
        const bool live = lane < kStepBlks && blk < nblk;
        const bool in_range = (uint32_t)pid < (uint32_t)num_pages;
        const uint32_t okm = __ballot_sync(0xffffffffu, live && in_range);
        if (live && !in_range && p.err) atomicOr(p.err, CAI_DEVERR_PAGE);
        if (r + i == p.drop_stage) return;  // fault injection: never issued
        if (lane == 0) {
          ok_bits[warp * NS + s] = okm;
          mbar_arrive_expect_tx(&full[s], (uint32_t)__popc(okm) * kBlkBytes);
        }
        __syncwarp();
        if ((okm >> lane) & 1u)
          bulk_g2s(ring + s * kStepBytes + lane * kBlkBytes,
                   pages + (((int64_t)pid << per_log2) + ((blk0 + blk) & ((1 << per_log2) - 1))) * kBlkBytes, kBlkBytes,
                   &full[s]);
      };
      if (ok)
        while (issued < min(mine, NS)) issue();

      // B operand of S^T: lane (g, t) holds, for head g and channel group j, channels 32 j + 8 t ..
      // + 7 (one 16-byte load), two k steps of 16 whose channel order is that of the K words.
      uint4 qf[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 x = g < G ? __ldg(reinterpret_cast<const uint4*>(q + g * kHeadDim + 32 * j + 8 * t)) : make_uint4(0u, 0u, 0u, 0u);
        qf[j] = make_uint4(bf16x2_to_f16x2(x.x), bf16x2_to_f16x2(x.y), bf16x2_to_f16x2(x.z), bf16x2_to_f16x2(x.w));
      }

      float o[8][4];  // O^T: channels 16 m + g, + 8 x heads 2 t, + 1
#pragma unroll
      for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[m][e] = 0.0f;
      uint64_t mref = 0ull, l = 0ull;  // negated references (log2 units) and this lane's parts of the sums of its two heads
      bool have_ref = false;  // some key was attended (the same in the whole warp)

      int i = 0;
      for (; ok && i < mine; ++i) {
        if (!mbar_wait_warp(&full[st], (phase >> st) & 1u, wctl)) {
          ok = false;
          break;
        }
        const uint8_t* stage = ring + st * kStepBytes;
        const uint32_t okm = ok_bits[warp * NS + st];
        const int first = (blk0 + kStepBlks * (warp + i * kWarps)) * kBlk;  // position of the step's first key
        const bool edge = first < start || first + kStep > end || okm != (1u << kStepBlks) - 1;

        // ---- S^T = K Q^T.  A channel group's products are summed as codes (exact in fp16) and its scale applied to
        // the sum.
        float sc[kStepBlks][4];
        uint4 kw[kStepBlks][2];
        uint2 ks[kStepBlks][2];
#pragma unroll
        for (int h = 0; h < kStepBlks; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint8_t* blk = stage + h * kBlkBytes;
            kw[h][e] = *reinterpret_cast<const uint4*>(blk + e * 512 + lane * 16);
            ks[h][e] = *reinterpret_cast<const uint2*>(blk + kBlkKs + e * 64 + g * 8);
          }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int h = 0; h < kStepBlks; ++h) {
            uint32_t x[4], y[4];
            const uint32_t sa = j < 2 ? ks[h][0].x : ks[h][0].y, sb = j < 2 ? ks[h][1].x : ks[h][1].y;
            codes_f16(word(kw[h][0], j), x);
            codes_f16(word(kw[h][1], j), y);
            const float a = half_of(sa, j & 1), b = half_of(sb, j & 1);
            const uint64_t a2 = f2(a, a), b2 = f2(b, b);
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            mma_16816(acc, x[0], y[0], x[1], y[1], qf[j].x, qf[j].y);
            mma_16816(acc, x[2], y[2], x[3], y[3], qf[j].z, qf[j].w);
            if (j == 0) {
              f2_split(f2_mul(f2(acc[0], acc[1]), a2), sc[h][0], sc[h][1]);
              f2_split(f2_mul(f2(acc[2], acc[3]), b2), sc[h][2], sc[h][3]);
            } else {
              f2_split(f2_fma(f2(acc[0], acc[1]), a2, f2(sc[h][0], sc[h][1])), sc[h][0], sc[h][1]);
              f2_split(f2_fma(f2(acc[2], acc[3]), b2, f2(sc[h][2], sc[h][3])), sc[h][2], sc[h][3]);
            }
          }

        // ---- logits minus reference, in log2 units; masked after the scale, which may be 0 or negative
        const uint64_t sl2 = f2(p.scale_log2, p.scale_log2);
#pragma unroll
        for (int h = 0; h < kStepBlks; ++h)
#pragma unroll
          for (int e = 0; e < 4; e += 2) f2_split(f2_fma(f2(sc[h][e], sc[h][e + 1]), sl2, mref), sc[h][e], sc[h][e + 1]);
        if (edge) {
#pragma unroll
          for (int h = 0; h < kStepBlks; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = first + h * kBlk + e * 8 + g;
              if (!(key >= start && key < end && ((okm >> h) & 1u))) sc[h][2 * e] = sc[h][2 * e + 1] = -INFINITY;
            }
        }
        float mx = -INFINITY;
#pragma unroll
        for (int h = 0; h < kStepBlks; ++h)
#pragma unroll
          for (int e = 0; e < 4; e += 2) mx = fmax3(mx, sc[h][e], sc[h][e + 1]);
        if (__any_sync(0xffffffffu, have_ref ? mx > kRaise4 : mx > -INFINITY)) {
          // Raise the references that a logit passes by 2^15 (all of them at the first key).
          float up[2], f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = fmaxf(fmaxf(sc[0][e], sc[0][2 + e]), fmaxf(sc[1][e], sc[1][2 + e]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, x));
            up[e] = !have_ref || v > kRaise4 ? v - kWeightLift : 0.0f;
            f[e] = have_ref ? ex2_approx(-up[e]) : 0.0f;
#pragma unroll
            for (int m = 0; m < 8; ++m) {
              o[m][e] *= f[e];
              o[m][2 + e] *= f[e];
            }
#pragma unroll
            for (int h = 0; h < kStepBlks; ++h) {
              sc[h][e] -= up[e];
              sc[h][2 + e] -= up[e];
            }
          }
          mref = f2_add(mref, f2(-up[0], -up[1]));
          l = f2_mul(l, f2(f[0], f[1]));
          have_ref = true;
        }
        // ---- P^T = 2^z, transposed into the B operand
        uint32_t pf[kStepBlks][2];
        uint64_t ps = 0ull;  // this lane's sums of the step
#pragma unroll
        for (int h = 0; h < kStepBlks; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float a = ex2_approx(sc[h][2 * e]), b = ex2_approx(sc[h][2 * e + 1]);
            ps = f2_add(ps, f2(a, b));
            pf[h][e] = transpose8x8(pack_f16x2(a, b));
          }
        l = f2_add(l, ps);
        // ---- O^T += V^T P^T
#pragma unroll
        for (int h = 0; h < kStepBlks; ++h) {
          const uint8_t* blk = stage + h * kBlkBytes;
          // Scales of the four channel groups: keys 2 t, 2 t + 1, and 2 t + 8, 2 t + 9.
          const uint4 a = *reinterpret_cast<const uint4*>(blk + kBlkVs + t * 32), b = *reinterpret_cast<const uint4*>(blk + kBlkVs + t * 32 + 16);
          uint32_t s0[4] = {a.x, a.y, a.z, a.w}, s1[4] = {b.x, b.y, b.z, b.w};
          if (edge) {
            // Masked keys' scales become 0 (their slots may hold anything, NaN included).
            const int key = first + h * kBlk + 2 * t;
            const bool good = (okm >> h) & 1u;
            auto keep = [&](int k) { return good && k >= start && k < end; };
            const uint32_t ma = (keep(key) ? 0xFFFFu : 0u) | (keep(key + 1) ? 0xFFFF0000u : 0u);
            const uint32_t mb = (keep(key + 8) ? 0xFFFFu : 0u) | (keep(key + 9) ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int k = 0; k < 4; ++k) s0[k] &= ma, s1[k] &= mb;
          }
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const uint4 vw = *reinterpret_cast<const uint4*>(blk + kBlkV + hh * 512 + lane * 16);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int m = hh * 4 + u;
              uint32_t x[4];
              values_f16(word(vw, u), s0[m >> 1], s1[m >> 1], x);
              mma_16816(o[m], x[0], x[1], x[2], x[3], pf[h][0], pf[h][1]);
            }
          }
        }
        phase ^= 1u << st;
        st = st + 1 == NS ? 0 : st + 1;
        __syncwarp();  // every lane has read the stage
        if (issued < mine) issue();
      }
      if (!ok && i < mine) {
        // A wait gave up (now, or in an earlier piece: then nothing was issued).  Report it, and let the warp's
        // own copies land; it issues no more.
        if (lane == 0 && p.err) atomicOr(p.err, CAI_DEVERR_TIMEOUT);
        for (; i < issued; ++i) {
          if (r + i != p.drop_stage) mbar_wait_drain(&full[st], (phase >> st) & 1u);
          st = st + 1 == NS ? 0 : st + 1;
        }
      }
      r += mine;

      // ---- merge of the warps: out = sum 2^(m - M) O / sum 2^(m - M) l
      __syncthreads();  // every ring is read
      float m2[2], l2[2];
      f2_split(mref, m2[0], m2[1]);
      f2_split(l, l2[0], l2[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l2[e] += __shfl_xor_sync(0xffffffffu, l2[e], x);
        if (g == 0) {
          ml[warp * kHeads4 + 2 * t + e] = have_ref ? -m2[e] : -INFINITY;
          ml[(kWarps + warp) * kHeads4 + 2 * t + e] = l2[e];
        }
      }
      float* mo = reinterpret_cast<float*>(smem);
      if (mine > 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* dst = mo + (warp * kHeads4 + 2 * t + e) * kORow + g;
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            dst[16 * m] = o[m][e];
            dst[16 * m + 8] = o[m][2 + e];
          }
        }
      }
      __syncthreads();
      const int live = min(kWarps, steps);
      for (int h = warp; h < G; h += kWarps) {
        float M = -INFINITY;
        for (int w = 0; w < live; ++w) M = fmaxf(M, ml[w * kHeads4 + h]);
        float sum = 0.0f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < live; ++w) {
          const float f = M == -INFINITY ? 0.0f : ex2_approx(ml[w * kHeads4 + h] - M);
          sum = fmaf(f, ml[(kWarps + w) * kHeads4 + h], sum);
          const float4 x = *reinterpret_cast<const float4*>(mo + (w * kHeads4 + h) * kORow + 4 * lane);
          acc.x = fmaf(f, x.x, acc.x);
          acc.y = fmaf(f, x.y, acc.y);
          acc.z = fmaf(f, x.z, acc.z);
          acc.w = fmaf(f, x.w, acc.w);
        }
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        const float lse2 = sum > 0.0f ? M + log2f(sum) : -INFINITY;
        if (pc.slot < 0) {
          reinterpret_cast<uint2*>(p.out + (row0 + h) * kHeadDim)[lane] =
              pack_bf16x4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
          if (p.lse_out && lane == 0) p.lse_out[row0 + h] = lse2 * kLn2;
        } else {
          const int64_t at = (int64_t)pc.slot * G + h;
          reinterpret_cast<float4*>(p.ws_o + at * kHeadDim)[lane] =
              make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
          if (lane == 0) p.ws_lse[at] = lse2;
        }
      }
      fence_proxy_async_smem();  // the next piece's copies write where the merge was
    }
    __syncthreads();
  }
  if (p.overlap_prev) grid_dependency_wait();
}

// The pieces' normalised outputs merged by their log2-sum-exp.  At most one sequence and K/V head starts in
// a block's range and goes on into the next, so there is an item per range, not per sequence; four warps
// have one of its heads.
constexpr int kCombineWarps = 4, kCombineHeads = 2;
__global__ void __launch_bounds__(kCombineWarps * kCombineHeads * 32) combine4_kernel(const __grid_constant__ Decode4Params p) {
  __shared__ float parts[kCombineHeads][kCombineWarps][kHeadDim];
  __shared__ float pms[kCombineHeads][kCombineWarps], pls[kCombineHeads][kCombineWarps];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % kCombineWarps, which = threadIdx.x / (32 * kCombineWarps);
  const int G = p.num_heads / p.num_kv_heads, groups = (G + kCombineHeads - 1) / kCombineHeads;
  const int item = blockIdx.x / groups, hg = (blockIdx.x - item * groups) * kCombineHeads + which;  // head of the K/V head's group
  float (&part)[kCombineWarps][kHeadDim] = parts[which];
  float (&pm)[kCombineWarps] = pms[which], (&pl)[kCombineWarps] = pls[which];
  grid_dependency_wait();
  grid_launch_dependents();
  int unit = item, n = 0, first = 0;
  if (p.chunk == 0) {
    const int2 m = p.meta[item];  // the unit, and the last block with a piece of it
    if (m.x < 0) return;
    unit = m.x;
    first = item;
    n = m.y - item + 1;
  }
  const int b = unit / p.num_kv_heads, kvh = unit - b * p.num_kv_heads, h = kvh * G + hg;
  int32_t row;
  SeqSplits sp;
  if (!seq_keys(p, b, row, sp)) return;
  if (p.chunk > 0) n = sp.nsplit;
  if (n <= 1) return;  // written by the decode kernel
  auto slot = [&](int j) -> int64_t {
    return (p.chunk > 0 ? (int64_t)unit * p.splits + j : 2ll * (first + j) + (j == 0 ? 1 : 0)) * G + hg;
  };
  // Warp w takes pieces w, w + 4, ..., four at a time so that their loads overlap.
  float M = -INFINITY, sum = 0.0f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = warp; j0 < n && hg < G; j0 += 4 * kCombineWarps) {
    float4 x[4];
    float l[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + u * kCombineWarps;
      l[u] = j < n ? p.ws_lse[slot(j)] : -INFINITY;
      x[u] = j < n ? reinterpret_cast<const float4*>(p.ws_o + slot(j) * kHeadDim)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float m = fmaxf(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])), M);
    if (m == -INFINITY) continue;
    const float f = ex2_approx(M - m);
    M = m;
    sum *= f;
    acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float w = ex2_approx(l[u] - m);
      sum += w;
      acc.x = fmaf(w, x[u].x, acc.x);
      acc.y = fmaf(w, x[u].y, acc.y);
      acc.z = fmaf(w, x[u].z, acc.z);
      acc.w = fmaf(w, x[u].w, acc.w);
    }
  }
  reinterpret_cast<float4*>(part[warp])[lane] = acc;
  if (lane == 0) {
    pm[warp] = M;
    pl[warp] = sum;
  }
  __syncthreads();
  if (warp > 0 || hg >= G) return;
  M = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kCombineWarps; ++w) {
    const float f = M == -INFINITY ? 0.0f : ex2_approx(pm[w] - M);
    const float4 x = reinterpret_cast<const float4*>(part[w])[lane];
    sum = fmaf(f, pl[w], sum);
    acc.x = fmaf(f, x.x, acc.x);
    acc.y = fmaf(f, x.y, acc.y);
    acc.z = fmaf(f, x.z, acc.z);
    acc.w = fmaf(f, x.w, acc.w);
  }
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  const int64_t at = (int64_t)row * p.num_heads + h;
  reinterpret_cast<uint2*>(p.out + at * kHeadDim)[lane] = pack_bf16x4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  if (p.lse_out && lane == 0) p.lse_out[at] = sum > 0.0f ? (M + log2f(sum)) * kLn2 : -INFINITY;
}

cudaError_t launch_heads8(const Decode4Params& p, cudaStream_t stream) {
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(decode4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem4);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set[dev] = true;
  }
  return launch_pdl(decode4_kernel, dim3((unsigned)p.ranges), dim3(kWarps * 32), kSmem4, stream, p);
}

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t plan_decode4(Decode4Params& p, int32_t num_splits) {
  const int G = p.num_heads / p.num_kv_heads, tc = decode4_tc_heads(G);
  const int blocks = num_sms() * (tc ? 1 : kBlocks4);
  p.head_groups = tc ? (G + tc - 1) / tc : 1;
  // What the start and merge of a piece cost, in tiles, fitted from the times of blocks with different numbers of
  // tiles and pieces.  (Lognormal contexts of 32 heads: 77.5 us with one tile, 73.6 with five; 96 sequences of 8 heads:
  // 195 us with two, 198 with one, 197 with four; 1024 short ones 119, 120, 135.)
  p.piece_tiles = tc == 0 ? 2 : tc == 16 ? 4 : tc == 32 ? 5 : 8;
  const int64_t units = (int64_t)p.batch * p.num_kv_heads;
  const int64_t cap = (int64_t)p.max_pages * p.page_size;
  const int64_t span = p.window > 0 && p.window < cap ? p.window : cap;
  int64_t ranges = blocks / p.head_groups, most, slots;
  p.chunk = 0;
  p.splits = 0;
  // Sequences of at most 512 keys are not cut: the merge's launch costs more than four tiles one after the other
  // (a step of four sequences of 64 to 512 keys: 8.3 us cut, 7.6 whole).
  if (num_splits == 0 && span <= 4 * kDecodeTile) num_splits = 1;
  if (num_splits > 0) {
    p.chunk = (int32_t)(((span + num_splits - 1) / num_splits + kDecodeTile - 1) / kDecodeTile * kDecodeTile);
    p.splits = (int32_t)((span + p.chunk - 1) / p.chunk);
    most = units * p.splits;
    slots = p.splits > 1 ? most : 0;
  } else {
    most = units * ((span + kDecodeTile - 1) / kDecodeTile + 1 + p.piece_tiles);  // a window may start inside a tile
    slots = 0;
  }
  p.ranges = (int32_t)(ranges < most ? ranges : most);
  if (p.chunk == 0) slots = 2 * p.ranges;
  const int64_t rows = slots * G;
  return (size_t)((p.chunk == 0 ? up256(p.ranges * 8) : 0) + up256(rows * kHeadDim * 4) + up256(rows * 4));
}

void place_decode4(Decode4Params& p, void* workspace) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int64_t units = (int64_t)p.batch * p.num_kv_heads, G = p.num_heads / p.num_kv_heads;
  const int64_t slots = p.chunk == 0 ? 2ll * p.ranges : p.splits > 1 ? units * p.splits : 0;
  p.meta = reinterpret_cast<int2*>(ws);
  if (p.chunk == 0) ws += up256(p.ranges * 8);
  p.ws_o = reinterpret_cast<float*>(ws);
  p.ws_lse = reinterpret_cast<float*>(ws + up256(slots * G * kHeadDim * 4));
}

cudaError_t launch_decode4(const Decode4Params& p, cudaStream_t stream) {
  const cudaError_t e = decode4_tc_heads(p.num_heads / p.num_kv_heads) ? launch_decode4_tc(p, stream) : launch_heads8(p, stream);
  if (e != cudaSuccess || (p.chunk > 0 && p.splits <= 1)) return e;
  const int64_t G = p.num_heads / p.num_kv_heads, items = p.chunk == 0 ? p.ranges : (int64_t)p.batch * p.num_kv_heads;
  return launch_pdl(combine4_kernel, dim3((unsigned)(items * ((G + kCombineHeads - 1) / kCombineHeads))),
                    dim3(kCombineWarps * kCombineHeads * 32), 0, stream, p);
}

}  // namespace cai

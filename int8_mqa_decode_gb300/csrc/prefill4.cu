// Prefill attention over the tiled copy of a 4-bit cache (dequant_tile4 in prefill.cu writes it).
//
// What it computes: prefill.cu.  A row is a (new token, query head of the K/V head) pair of one sequence and K/V
// head; keys and values are fp16 (K exact), queries bf16 converted to fp16, outputs bf16.
//
// How.  A persistent block per SM takes q-tiles of 128 rows; bulk copies bring the key tiles into a K and a V ring.
// One warp issues S = Q K^T into two S buffers in tensor memory in turn, another O_h += P_h V_h for the two key
// halves h.  Eight softmax warps (thread = row and key half, 64 keys a tile) have a reference, sum and accumulator
// per half, merged at the end of an item; P overwrites the S that it came from.  So S is a tile ahead, a softmax
// warp waits for no product but the S it reads, and the halves may drift apart: while one does its exponentials
// the other has the other pipes.  (With one S buffer and P beside it both halves waited for the same S and came to
// their exponentials together: 1500 cycles a tile, now 1430.  Two q-tiles a block with all 128 keys a thread,
// S after PV in the same columns: 1740 a q-tile and tile, half of it the way from P to the next S.)
// The softmax is that of prefill.cu, a reference per row, with larger weights (kWeightLift): raised when a logit passes it
// by 2^15.
//
// Roundings: the query to fp16 (exact for magnitudes from 2^-17 to 65504, below that off by 2^-25 at most), a weight to
// fp16 for its product with V (2^-11 of it, or 2^-32 of the sum of all where that is more; the sums take it unrounded, in
// fp32), the output to bf16 once; a piece's partial output stays fp32.
//
// Bound: 16 products of 64 cycles a tile, and the exponentials, 512 cycles a sub-partition.
#include "prefill.cuh"

namespace cai {
namespace {

constexpr int kStagesK4 = 2, kStagesV4 = 3;
constexpr int kOffQ4 = 0;                                        // Q
constexpr int kOffK4 = kOffQ4 + kTileBytes;
constexpr int kOffV4 = kOffK4 + kStagesK4 * kTileBytes;
constexpr int kOffXch4 = kOffV4 + kStagesV4 * kTileBytes;        // row references, row sums [2 halves][128] each
constexpr int kOffBars4 = kOffXch4 + 4 * kRows * 4;
constexpr int kNumBars4 = 2 * kStagesK4 + 2 * kStagesV4 + 1 + 2 + 4 + 2 + 1 + 1 + 2 * kItemSlots;
constexpr int kOffMisc4 = kOffBars4 + 8 * kNumBars4;             // tensor memory slot, wait state
constexpr int kOffItems4 = (kOffMisc4 + 32 + 15) & ~15;          // items, 64 bytes each
constexpr int kSmem4 = kOffItems4 + kItemSlots * 64;
static_assert(sizeof(PItem) <= 64 && kSmem4 <= 227 * 1024, "shared memory");
// Warpgroup 0: producer, the issuers of S and of PV, items; warpgroups 1 and 2: softmax of key half 0 and 1.
constexpr int kThreads4 = 384;
constexpr int kRegsLaunch4 = 168, kRegsCtl4 = 72, kRegsSoft4 = 216;
static_assert(kRegsCtl4 * 128 + kRegsSoft4 * 256 <= kRegsLaunch4 * kThreads4, "register split");
constexpr uint32_t kColO4 = 256;  // S buffer b at b * 128 (P of half h over its first 32 columns of half h); O_h at kColO4 + h * 128
constexpr uint32_t kBarSoft4 = 1;
constexpr float kRaisePrefill4 = kWeightLift + 8.0f;  // log2 units a logit may exceed its reference by
constexpr int kItemUsers = 1 + 2 + 8;  // warps that read an item

template <bool kCompact>
__global__ void __launch_bounds__(kThreads4, 1) attend4_kernel(const __grid_constant__ PrefillParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBars4);
  uint64_t* k_full = bars;                      // [kStagesK4] producer -> issuers (tx bytes)
  uint64_t* k_empty = k_full + kStagesK4;       // [kStagesK4] S issuer's commit after S of the tile
  uint64_t* v_full = k_empty + kStagesK4;       // [kStagesV4] producer -> PV issuer
  uint64_t* v_empty = v_full + kStagesV4;       // [kStagesV4] PV issuer's commit after PV of the tile
  uint64_t* q_full = v_empty + kStagesV4;       // softmax (8 warps) -> S issuer
  uint64_t* s_full = q_full + 1;                // [buffer] S issuer's commit after S
  uint64_t* p_full = s_full + 2;                // [half][buffer] softmax of half h (4 warps) -> PV issuer
  uint64_t* pv_done = p_full + 4;               // [buffer] PV issuer's commit -> S issuer, softmax
  uint64_t* o_empty = pv_done + 2;              // softmax (8 warps) -> PV issuer: O is read
  uint64_t* drain = o_empty + 1;                // the issuers' last commits, at exit
  uint64_t* item_full = drain + 1;              // [kItemSlots] warp 3 -> the other roles
  uint64_t* item_empty = item_full + kItemSlots;  // [kItemSlots] the other roles -> warp 3
  PItem* items = reinterpret_cast<PItem*>(smem + kOffItems4);
  float* xref = reinterpret_cast<float*>(smem + kOffXch4);  // [2 halves][128 rows] references
  float* xsum = xref + 2 * kRows;                           // ... sums
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc4);
  volatile WaitState* const wctl = reinterpret_cast<volatile WaitState*>(smem + kOffMisc4 + 8);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (warp == 0) tmem_alloc(tmem_slot, 512);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStagesK4; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < kStagesV4; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(q_full, 8);
    mbar_init(o_empty, 8);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], 4);
      mbar_init(&p_full[2 + b], 4);
      mbar_init(&pv_done[b], 1);
    }
    mbar_init(drain, 2);
    for (int k = 0; k < kItemSlots; ++k) {
      mbar_init(&item_full[k], 1);
      mbar_init(&item_empty[k], kItemUsers);
    }
    wctl->abort = 0;
    wctl->limit_ns = p.wait_ns;
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  if (kCompact) grid_launch_dependents();  // (as in prefill.cu)
  bool ok = true;  // no wait of this warp gave up
  // The block's i-th item, nkt < 0 past its last; the slot is free again on return.
  auto get_item = [&](int i) -> PItem {
    const int s = i % kItemSlots;
    PItem it = {};
    it.nkt = -1;
    ok = mbar_wait_lean_warp(&item_full[s], (i / kItemSlots) & 1, wctl);
    if (!ok) return it;
    it = items[s];
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[s]);
    return it;
  };

  if (warp < 4) {
    setmaxnreg_dec<kRegsCtl4>();
    if (warp == 0) {
      // ------------------------------------------------------------ K/V producer
      int g = 0, gk = 0, gv = 0;  // tiles; tiles whose K and V loads were issued (or dropped)
      for (int i = 0;; ++i) {
        const PItem it = get_item(i);
        if (!ok || it.nkt < 0) break;
        const uint16_t* kb = p.kb + ((int64_t)it.b * p.kt_rows + (int64_t)it.kt0 * kKeys) * kHeadDim;
        const uint16_t* vh = p.vh + ((int64_t)it.b * p.kt_rows + (int64_t)it.kt0 * kKeys) * kHeadDim;
        for (int j = 0; j < it.nkt && ok; ++j, ++g) {
          const int sk = g % kStagesK4, sv = g % kStagesV4;
          ok = g < kStagesK4 || mbar_wait_lean_warp(&k_empty[sk], (g / kStagesK4 - 1) & 1, wctl);
          if (!ok) break;
          if (lane == 0 && g != p.drop_stage) {  // (fault injection: that K tile is never loaded)
            mbar_arrive_expect_tx(&k_full[sk], kTileBytes);
            bulk_g2s(smem + kOffK4 + sk * kTileBytes, kb + (int64_t)j * kKeys * kHeadDim, kTileBytes, &k_full[sk]);
          }
          gk = g + 1;
          ok = g < kStagesV4 || mbar_wait_lean_warp(&v_empty[sv], (g / kStagesV4 - 1) & 1, wctl);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&v_full[sv], kTileBytes);
            bulk_g2s(smem + kOffV4 + sv * kTileBytes, vh + (int64_t)j * kKeys * kHeadDim, kTileBytes, &v_full[sv]);
          }
          gv = g + 1;
          __syncwarp();
        }
      }
      // Every slot that was armed has landed before the block goes away.
      for (int i = max(0, gk - kStagesK4); i < gk; ++i)
        if (i != p.drop_stage) mbar_wait_drain(&k_full[i % kStagesK4], (i / kStagesK4) & 1);
      for (int i = max(0, gv - kStagesV4); i < gv; ++i) mbar_wait_drain(&v_full[i % kStagesV4], (i / kStagesV4) & 1);
    } else if (warp < 3) {
      // ------------------------------------------------------------ issuers: S (warp 1), PV (warp 2)
      constexpr uint32_t idesc_s = idesc_f16_f32(kRows, kKeys, 0, 0), idesc_o = idesc_f16_f32(kRows, kHeadDim, 0, 1);
      const uint64_t dq = smem_desc(smem_addr(smem + kOffQ4), 2048, 128);
      const uint64_t dk0 = smem_desc(smem_addr(smem + kOffK4), 2048, 128);
      const uint64_t dv0 = smem_desc(smem_addr(smem + kOffV4), 128, 2048);
      int g = 0, n = 0;  // tiles, items
      for (int i = 0; ok; ++i) {
        const PItem it = get_item(i);
        if (it.nkt < 0) break;
        if (!it.ok || it.nkt == 0) continue;  // no products; the softmax writes its zeros
        if (warp == 1) {
          ok = mbar_wait_lean_warp(q_full, n & 1, wctl);
          for (int j = 0; j < it.nkt && ok; ++j, ++g) {
            const int sk = g % kStagesK4, b = g & 1;
            // (the buffer's P was read by PV of tile g - 2)
            ok = mbar_wait_lean_warp(&k_full[sk], (g / kStagesK4) & 1, wctl) && (g < 2 || mbar_wait_lean_warp(&pv_done[b], (g / 2 - 1) & 1, wctl));
            if (!ok) break;
            tc_fence_after();
            const uint64_t dk = dk0 + (uint64_t)(sk * (kTileBytes / 16));
            if (elect_one()) {
#pragma unroll
              for (int ks = 0; ks < kHeadDim / 16; ++ks)
                mma_f16_ss(tmem + b * kKeys, dq + (uint64_t)(ks * 256), dk + (uint64_t)(ks * 256), idesc_s, ks > 0);
              mma_commit(&s_full[b]);
              mma_commit(&k_empty[sk]);
            }
            __syncwarp();
          }
        } else {
          for (int j = 0; j < it.nkt && ok; ++j, ++g) {
            const int sv = g % kStagesV4, b = g & 1;
            ok = (j > 0 || n == 0 || mbar_wait_lean_warp(o_empty, (n - 1) & 1, wctl)) &&
                 mbar_wait_lean_warp(&v_full[sv], (g / kStagesV4) & 1, wctl);
            const uint64_t dv = dv0 + (uint64_t)(sv * (kTileBytes / 16));
            for (int hh = 0; hh < 2 && ok; ++hh) {
              ok = mbar_wait_lean_warp(&p_full[2 * hh + b], (g / 2) & 1, wctl);
              if (!ok) break;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                  mma_f16_ts(tmem + kColO4 + hh * kHeadDim, tmem + b * kKeys + hh * 64 + ks * 8, dv + (uint64_t)((hh * 4 + ks) * 16), idesc_o,
                             (j > 0 || ks > 0) ? 1u : 0u);
                if (hh == 1) {
                  mma_commit(&pv_done[b]);
                  mma_commit(&v_empty[sv]);
                }
              }
              __syncwarp();
            }
          }
        }
        ++n;
      }
      // This issuer's products have ended before tensor memory is freed.
      if (elect_one()) mma_commit(drain);
      __syncwarp();
      mbar_wait_drain(drain, 0);
    } else {
      // ------------------------------------------------------------ items
      // Works out the items ahead of the other roles and brings their queries into L2.  A varlen call's are numbered
      // without the empty q-tiles that the longest sequence gives the others: lane l has the q-tiles of one sequence of
      // a window of 32, and the window moves on.
      WorkSplit ws;
      ws.full = p.full_items;
      ws.pieces = p.pieces;
      ws.num = p.num_items;
      int w0 = -32, n = 0, incl = 0, window = 0;  // first sequence; this lane's q-tiles, items up to it; the window's items
      int64_t before = 0;                         // items before the window
      for (int i = 0; !abort_seen_warp(wctl); ++i) {
        const int64_t at = blockIdx.x + (int64_t)i * gridDim.x;
        PItem it = {};
        it.nkt = -1;
        if constexpr (kCompact) {
          while (w0 < p.batch && at >= before + window) {
            before += window;
            w0 += 32;
            n = w0 + lane < p.batch ? seq_qtiles(p, w0 + lane) : 0;
            incl = n * p.num_kv_heads;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int v = __shfl_up_sync(0xffffffffu, incl, o);
              if (lane >= o) incl += v;
            }
            window = __shfl_sync(0xffffffffu, incl, 31);
          }
          if (w0 < p.batch) {
            const int rel = (int)(at - before), l = __ffs(__ballot_sync(0xffffffffu, incl > rel)) - 1;
            const int nl = __shfl_sync(0xffffffffu, n, l);
            const int e = rel - (__shfl_sync(0xffffffffu, incl, l) - nl * p.num_kv_heads), h = e / nl;
            it = prefill_item<true>(p, ((w0 + l) * p.num_kv_heads + h) * p.qtiles + (e - h * nl), nullptr, ws);
          }
        } else if (at < ws.num) {
          it = prefill_item<true>(p, (int)at, nullptr, ws);
        }
        const int s = i % kItemSlots;
        if (i >= kItemSlots && !mbar_wait_asleep_warp(&item_empty[s], (i / kItemSlots - 1) & 1, wctl)) break;
        if (lane == 0) {
          items[s] = it;
          mbar_arrive(&item_full[s]);
        }
        __syncwarp();
        if (it.nkt < 0) break;
        if (it.ok && it.nkt > 0) {
          for (int k = 0; k < kRows / 16; ++k) {
            const int64_t row = it.row0 + k * 16 + (lane >> 1);
            if (row < it.rows) prefetch_l2(p.q + q_row<true>(p, it, row) * kHeadDim + (lane & 1) * 64);
          }
        }
      }
    }
  } else {
    setmaxnreg_inc<kRegsSoft4>();
    // ------------------------------------------------------------ softmax
    const int h = (warp - 4) >> 2;  // key half of every tile, channel half of the output
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the q-tile
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
    auto has_products = [&](const PItem& it) { return it.ok && it.nkt > 0; };
    // This row's query of an item (zero beyond the chunk) as an operand: each half takes 8 of its 16 chunks.
    auto load_q = [&](const PItem& it, uint4 (&x)[8]) {
      const int64_t row = it.row0 + r;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + q_row<true>(p, it, row) * kHeadDim) + h * 8;
#pragma unroll
      for (int c = 0; c < 8; ++c) x[c] = row < it.rows ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto stage_q = [&](const uint4 (&x)[8]) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint32_t u[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = pack_f16x2(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xFFFF0000u));
        *reinterpret_cast<uint4*>(smem + kOffQ4 + (h * 8 + c) * 2048 + r * 16) = make_uint4(y[0], y[1], y[2], y[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    };
    int g = 0;  // tiles
    PItem next = get_item(0);
    if (ok && has_products(next)) {
      uint4 x[8];
      load_q(next, x);
      stage_q(x);
    }
    const uint64_t sl2 = f2(p.scale_log2, p.scale_log2);
    for (int i = 0;; ++i) {
      // The eight warps meet at an item's start (the exchange is read) and merge; there they stop together.
      if (bar_red_or(kBarSoft4, 256, !ok) || next.nkt < 0) break;
      const PItem it = next;
      const int64_t row = it.row0 + r;  // (token, head) row within the sequence
      const bool my_row = row < it.rows;
      float* part = it.piece >= 0 ? p.piece_o + ((int64_t)it.piece * kRows + r) * kHeadDim + h * 64 : nullptr;
      float* part_lse = it.piece >= 0 ? p.piece_lse + (int64_t)it.piece * kRows + r : nullptr;
      if (!has_products(it)) {
        // An invalid sequence (flagged by the dequant pass): 0, -inf; a piece without key tiles: weight 0 in the
        // merge; rows beyond the chunk: nothing.
        if (my_row && !it.ok) {
          const int64_t at = q_row<true>(p, it, row);
          for (int d = 0; d < 64; d += 8) *reinterpret_cast<uint4*>(p.out16 + at * kHeadDim + h * 64 + d) = make_uint4(0u, 0u, 0u, 0u);
          if (h == 0 && p.lse_out) p.lse_out[at] = -INFINITY;
        } else if (my_row && part) {
          for (int d = 0; d < 64; d += 4) *reinterpret_cast<float4*>(part + d) = make_float4(0.f, 0.f, 0.f, 0.f);
          if (h == 0) *part_lse = -INFINITY;
        }
        next = get_item(i + 1);
        if (ok && has_products(next)) {
          uint4 x[8];
          load_q(next, x);
          stage_q(x);
        }
        continue;
      }
      const int q_pos = it.p0 + (int)(row >> p.log2_heads);
      const int k_lo = p.window > 0 ? max(0, q_pos + 1 - p.window) : 0;
      float m_ref = -INFINITY, l_sum = 0.0f;
#pragma unroll 1
      for (int j = 0; j < it.nkt; ++j, ++g) {
        const int b = g & 1;
        ok = mbar_wait_lean_warp(&s_full[b], (g >> 1) & 1, wctl);
        if (!ok) break;
        tc_fence_after();
        const int key0 = (it.kt0 + j) * kKeys + h * 64;
        const uint32_t t_s = t_lane + b * kKeys + h * 64;
        // z: logit (log2 units) minus this half row's reference.
        const float m_use = m_ref == -INFINITY ? 0.0f : m_ref;
        const uint64_t nm2 = f2(-m_use, -m_use);
        float z[64];
        {
          uint32_t a[32], c[32];
          tmem_ld_32x32b_x32(t_s, a);
          tmem_ld_32x32b_x32(t_s + 32, c);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            f2_split(f2_fma(f2(__uint_as_float(a[e]), __uint_as_float(a[e + 1])), sl2, nm2), z[e], z[e + 1]);
            f2_split(f2_fma(f2(__uint_as_float(c[e]), __uint_as_float(c[e + 1])), sl2, nm2), z[32 + e], z[32 + e + 1]);
          }
        }
        if (!(key0 >= k_lo && key0 + 63 <= q_pos)) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (key0 + c < k_lo || key0 + c > q_pos) z[c] = -INFINITY;
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 64; c += 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e) mx4[e] = fmax3(mx4[e], z[c + 2 * e], z[c + 2 * e + 1]);
        }
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        // Raise the reference when the half row has none yet, or a logit exceeds it by 2^15.
        const bool raise = m_ref == -INFINITY ? mx > -INFINITY : mx > kRaisePrefill4;
        if (__any_sync(0xffffffffu, raise)) {
          const float up = mx - kWeightLift;
          const float alpha = raise ? ex2_approx(m_ref - (m_use + up)) : 1.0f;  // 0 when there was no reference
          if (j > 0) {  // O_h holds earlier tiles: wait for their PVs, then rescale this row of it
            ok = mbar_wait_lean_warp(&pv_done[b ^ 1], ((g - 1) >> 1) & 1, wctl);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < kHeadDim; c += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(t_lane + kColO4 + h * kHeadDim + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st_32x32b_x32(t_lane + kColO4 + h * kHeadDim + c, o);
            }
          }
          if (raise) {
            l_sum *= alpha;
            m_ref = m_use + up;
#pragma unroll
            for (int c = 0; c < 64; ++c) z[c] -= up;
          }
        }
        // P = 2^z as fp16, over the S that it came from: the A operand of this half's PV.
        uint64_t l01 = 0ull, l23 = 0ull;
        uint32_t pw[32];
#pragma unroll
        for (int e = 0; e < 64; e += 4) {
          const float e0 = ex2_approx(z[e]), e1 = ex2_approx(z[e + 1]), e2 = ex2_approx(z[e + 2]), e3 = ex2_approx(z[e + 3]);
          l01 = f2_add(l01, f2(e0, e1));
          l23 = f2_add(l23, f2(e2, e3));
          pw[e / 2] = pack_f16x2(e0, e1);
          pw[e / 2 + 1] = pack_f16x2(e2, e3);
        }
        tmem_st_32x32b_x32(t_s, pw);
        float l4[4];
        f2_split(l01, l4[0], l4[1]);
        f2_split(l23, l4[2], l4[3]);
        l_sum += (l4[0] + l4[1]) + (l4[2] + l4[3]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * h + b]);
      }
      // ---- end of item: the next one's query goes out while the last products end (every S of this one is done);
      // then the halves are merged, O = (w0 O_0 + w1 O_1) / (w0 l_0 + w1 l_1), w_h = 2^(m_h - M), M the larger
      // reference; this thread writes its channel half.
      xref[h * kRows + r] = m_ref;
      xsum[h * kRows + r] = l_sum;
      bool staged = false;
      uint4 qx[8];
      if (ok) {
        next = get_item(i + 1);
        staged = ok && has_products(next);
        if (staged) load_q(next, qx);
      }
      if (bar_red_or(kBarSoft4, 256, !ok)) break;
      const float m0 = xref[r], m1 = xref[kRows + r];
      const float M = fmaxf(m0, m1);
      const float w0 = m0 == -INFINITY ? 0.0f : ex2_approx(m0 - M);
      const float w1 = m1 == -INFINITY ? 0.0f : ex2_approx(m1 - M);
      const float Ls = w0 * xsum[r] + w1 * xsum[kRows + r];
      if (staged) stage_q(qx);
      ok = mbar_wait_lean_warp(&pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, wctl);
      if (!ok) continue;  // (the next barrier stops all)
      tc_fence_after();
      const float inv = Ls > 0.0f ? 1.0f / Ls : 0.0f;
      const float c0 = w0 * inv, c1 = w1 * inv;
      float o[64];
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        uint32_t o0[32], o1[32];
        tmem_ld_32x32b_x32(t_lane + kColO4 + h * 64 + c, o0);
        tmem_ld_32x32b_x32(t_lane + kColO4 + kHeadDim + h * 64 + c, o1);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[c + e] = fmaf(c0, __uint_as_float(o0[e]), c1 * __uint_as_float(o1[e]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_empty);
      const float lse2 = Ls > 0.0f ? M + __log2f(Ls) : -INFINITY;
      if (my_row && part) {
#pragma unroll
        for (int e = 0; e < 64; e += 4) *reinterpret_cast<float4*>(part + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        if (h == 0) *part_lse = lse2;
      } else if (my_row) {
        const int64_t at = q_row<true>(p, it, row);
        uint16_t* dst = p.out16 + at * kHeadDim + h * 64;
        uint32_t x[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
        if ((reinterpret_cast<uintptr_t>(p.out16) & 31) == 0) {  // (a tensor's rows; else 16-byte aligned)
#pragma unroll
          for (int e = 0; e < 32; e += 8) st_global_v8(dst + 2 * e, &x[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4) *reinterpret_cast<uint4*>(dst + 2 * e) = make_uint4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        }
        if (h == 0 && p.lse_out) p.lse_out[at] = lse2 * kLn2;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && wctl->abort && p.err) atomicOr(p.err, CAI_DEVERR_TIMEOUT);
  if (warp == 0) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_attend4(const PrefillParams& p, int grid, cudaStream_t stream) {
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_set[dev]) {
    cudaFuncAttributes fa;  // the register split assumes the launch's count
    for (const void* fn : {(const void*)attend4_kernel<false>, (const void*)attend4_kernel<true>}) {
      cudaError_t e = cudaFuncGetAttributes(&fa, fn);
      if (e != cudaSuccess) return e;
      if (fa.numRegs != kRegsLaunch4) return cudaErrorInvalidDeviceFunction;
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem4);
      if (e != cudaSuccess) return e;
    }
    if (dev < 64) attr_set[dev] = true;
  }
  if (p.compact) attend4_kernel<true><<<grid, kThreads4, kSmem4, stream>>>(p);
  else attend4_kernel<false><<<grid, kThreads4, kSmem4, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace cai

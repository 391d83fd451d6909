// Decode attention over the 4-bit paged cache for groups of 9 and more query heads per K/V head, on the
// 5th-generation tensor cores.  What is computed and how the work is split: decode4.cu, decode4.cuh.
//
// How.  A persistent block per SM walks its pieces in tiles of 128 keys.  Scores and outputs are
// transposed, S^T = K Q^T and O^T += V^T P^T, with tcgen05.mma kind::f16 (M = 128 keys or channels,
// N = heads padded to 16, 32 or 64, K = 128): A operands and accumulators in tensor memory, Q^T and
// P^T in shared memory.  The cache's order is that of tcgen05.st.16x128b (a lane holds column t of
// rows g and g + 8): a warp turns its 16-byte loads of codes into fp16 values (exact) and stores
// them as they come, with no exchange between lanes.
//
// Two sets take every other tile.  A set is four converting warps and four softmax warps (one of each per
// lane quarter of tensor memory), a producer and an issuer warp, with operands, accumulators and references of its
// own, so that a role runs ahead of the next as far as the buffers let it, and one set's latencies (a wait
// on an mbarrier costs 150 cycles and more even when its phase is over) pass under the other's work; a
// piece ends with the merge of the two.  A converter turns 32 keys of K, then 32 channels of V, into operands;
// a softmax thread has one key and all heads and writes its weights as 16-byte rows of P^T.
// A head's running maximum is a reference that the set's softmax warps share, raised only when a logit
// passes it by 2^15: the weights are written on the guess that none does, and one barrier of those four
// warps says whether the guess held; if not, O^T is rescaled in tensor memory.
//
// Why: mma.sync takes a sub-partition's issue slots (measured: 32 m16n8k16 alone 262 cycles, with the
// conversion that feeds them 353 whatever the number of warps), which at 32 heads leaves the
// register kernel at 2100 cycles a tile per SM; here the products cost no issue slots (16 instructions
// of 16 cycles at 32 heads, 32 at 64: elect.sync issues one every 16 cycles, a lane-0 branch one every
// 46).  Measured, 64 sequences of 16 to 131 thousand keys on one K/V head: 16 heads 172 us, 32 heads 187, 64 heads
// 243 (the cache's bytes take 106 at the copy bandwidth); with mma.sync 188, 281 and 536.  A tile takes 1200
// cycles up to 32 heads, of which the converters' instructions are 500 issue slots a sub-partition and the
// softmax's and issuers' 300 more: the rest is waits and instruction cache misses.  At 64 heads, 1550 cycles, the
// softmax is the longest role (64 heads a thread, 160 registers).
#include <cmath>

#include "decode4.cuh"

namespace cai {
namespace {

constexpr int kSets = 2;
// Warpgroups: control (a producer and an issuer per set), two of converters, two of softmax.
constexpr int kConv0 = 4, kSoft0 = kConv0 + 4 * kSets;
constexpr int kTcThreads = 32 * (kSoft0 + 4 * kSets);
constexpr int kSoftThreads = 128 * kSets;
constexpr int kT = kDecodeTile;                      // 128 keys
constexpr int kTileBlks = kT / kBlk;                 // 8
constexpr int kTileBytes = kTileBlks * kBlkBytes;    // 18432
constexpr int kInfo = 16;                            // ring of tiles' key ranges, longer than any lag
constexpr float kRaiseTc = kWeightLift + 8.0f;       // log2 units a logit may exceed its reference by
constexpr uint32_t kBarPiece = 1 + kSets;            // named barriers: 1 + set (its softmax), all softmax warps

template <int HN>
struct ShapeTc {
  static constexpr int kStages = HN == 64 ? 6 : 8;   // raw tiles
  static constexpr int kPBytes = HN * kT * 2;
  static constexpr int kOffP = kStages * kTileBytes;                 // P^T [set][2 tiles]
  static constexpr int kOffQ = kOffP + 2 * kSets * kPBytes;          // Q^T [2 pieces]
  static constexpr int kQBytes = HN * kHeadDim * 2;
  static constexpr int kOffX = kOffQ + 2 * kQBytes;                  // [set] exchange:
  // [4 quarters][HN] maxima; [2 pieces][4 quarters][HN] sums; the same of references (a copy per quarter)
  static constexpr int kXSum = 4 * HN, kXRef = 12 * HN, kXFloats = 20 * HN;
  static constexpr int kOffBars = kOffX + kSets * kXFloats * 4;
  static constexpr int kNumBars = 2 * kStages + kSets * 9 + 2 + 2 + 1;
  static constexpr int kOffInfo = (kOffBars + kNumBars * 8 + 15) & ~15;  // int4 per tile
  static constexpr int kOffScan = kOffInfo + kInfo * 16;             // start_list's
  static constexpr int kOffWait = kOffScan + kTcThreads / 32 * 8;
  static constexpr int kOffSlot = kOffWait + 16;
  static constexpr int kOffPieces = kOffSlot + 16;
  static constexpr int kSmem = kOffPieces + kPieces * (int)sizeof(Piece4) + 64;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // Columns of a set: K 64, V^T 64 (two of them where they fit: V is then converted a tile ahead of its PV), S^T HN,
  // O^T HN.
  static constexpr int kVBufs = HN == 64 ? 1 : 2;
  static constexpr uint32_t kColV = 64, kColS = kColV + 64 * kVBufs, kColO = kColS + HN, kSetCols = kColO + HN;
  static_assert(kSets * kSetCols <= 512, "tensor memory columns");
  // Registers a thread: launched with 96 (five warps on a sub-partition: 15360 of 16384), then the control and
  // converting warpgroups give up what the softmax takes.  The host checks the launch count.
  static constexpr int kRegsLaunch = 96, kRegsCtl = HN == 64 ? 48 : 56, kRegsConv = HN == 64 ? 56 : 72, kRegsSoft = HN == 64 ? 160 : 136;
  static_assert(128 * kRegsCtl + 256 * kRegsConv + 256 * kRegsSoft <= kRegsLaunch * kTcThreads, "register split");
};

// This thread's lane, N columns.
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : CAI_R8(r, 0) : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld_32x32b_x16(taddr, r); }
__device__ __forceinline__ void tmem_st_n(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), CAI_W8(r, 0) : "memory");
}

__device__ __forceinline__ int piece_tiles(const Piece4& pc) {
  return pc.start < pc.end ? (pc.end - 1) / kT - pc.start / kT + 1 : 0;
}

template <int HN>
__global__ void __launch_bounds__(kTcThreads, 1) decode4_tc_kernel(const __grid_constant__ Decode4Params p) {
  using S = ShapeTc<HN>;
  constexpr int NS = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];  // (aligned by hand, it would be addressed as generic memory)
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBars);
  uint64_t* raw_full = bars;                 // [NS] producer -> converters (tx bytes)
  uint64_t* raw_empty = raw_full + NS;       // [NS] converters (4) -> producer
  uint64_t* k_full = raw_empty + NS;         // [set] converters (4) -> issuer
  uint64_t* v_full = k_full + kSets;         // [set][2] converters (4) -> issuer
  uint64_t* s_full = v_full + 2 * kSets;     // [set] commit of S^T -> softmax, converters (K free)
  uint64_t* s_read = s_full + kSets;         // [set] softmax (4) -> issuer: S^T free
  uint64_t* p_full = s_read + kSets;         // [set][2] softmax (4) -> issuer
  uint64_t* pv_done = p_full + 2 * kSets;    // [set][2] commit of PV -> softmax (P^T free), converters (V^T free)
  uint64_t* q_full = pv_done + 2 * kSets;    // [2] producers -> issuers: a piece's Q^T
  uint64_t* o_free = q_full + 2;             // [2] softmax (8) -> issuers, producers: a piece's O^T is read
  uint64_t* drain = o_free + 2;              // the issuers' last commits
  volatile int4* info = reinterpret_cast<volatile int4*>(smem + S::kOffInfo);  // tile: first and last + 1 key, groups landed
  volatile WaitState* wctl = reinterpret_cast<volatile WaitState*>(smem + S::kOffWait);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffSlot);
  float* xch = reinterpret_cast<float*>(smem + S::kOffX);
  Piece4* pieces = reinterpret_cast<Piece4*>(smem + S::kOffPieces);
  List4& ls = *reinterpret_cast<List4*>(smem + S::kOffPieces + kPieces * sizeof(Piece4));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  // Blocks of one range but different head groups are neighbours: they read the same keys at the same time.
  const int G = p.num_heads / p.num_kv_heads;
  const int hgrp = blockIdx.x % p.head_groups, c = blockIdx.x / p.head_groups;
  const int h0 = hgrp * HN, nh = min(G - h0, HN);  // this block's heads of the K/V head's group

  if (warp == 0) tmem_alloc(tmem_slot, 512);
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);
    }
    for (int k = 0; k < kSets; ++k) {
      mbar_init(&k_full[k], 4);
      mbar_init(&s_full[k], 1);
      mbar_init(&s_read[k], 4);
    }
    for (int k = 0; k < 2 * kSets; ++k) {
      mbar_init(&p_full[k], 4);
      mbar_init(&v_full[k], 4);
      mbar_init(&pv_done[k], 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&q_full[k], kSets);
      mbar_init(&o_free[k], 4 * kSets);
    }
    mbar_init(drain, kSets);
    wctl->abort = 0;
    wctl->limit_ns = p.wait_ns;
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // (overlap_prev: see DecodeParams.)
  if (!p.overlap_prev) grid_dependency_wait();
  grid_launch_dependents();
  start_list<kTcThreads>(p, c, ls, reinterpret_cast<int64_t*>(smem + S::kOffScan));

  // Tiles (gt) and pieces with tiles (gp) since the start; every role keeps its own count.  Set s takes the
  // tiles with gt % 2 == s; the n-th of them is n = gt / 2.
  int gt = 0, gp = 0;
  bool ok = true;  // no wait of this thread gave up
  int issued = 0;  // producers: tiles up to this one were started

  // Every role goes through the lists of pieces; `work` is its part of one.  (The roles are the outermost branch:
  // the compiler gives each the registers that its setmaxnreg names.)
  auto lists = [&](auto&& work) {
    while (ls.more) {  // (written before the barriers of start_list and of the loop's end)
      __syncthreads();
      if (warp == 0) next_pieces(p, c, ls, pieces);
      __syncthreads();
      work(ls.count);
      __syncthreads();
      if (wctl->abort) break;  // (set by a wait that gave up; nobody waits now)
    }
  };

  if (warp < kConv0) {
    setmaxnreg_dec<S::kRegsCtl>();
    lists([&](int count) {
    if (warp < kSets) {
      // ------------------------------------------------------------------ producer of a set
      // One bulk copy a page (starting eight of them took one warp a thousand cycles: hence two producers, and
      // whole pages where they are longer than 16 tokens).  Lane l: page l of the tile.
      const int set = warp;
      const int P = p.page_size, per = P / kBlk, in_tile = kT / P;
      // Half of a piece's query as Q^T, its channels in the order of K's columns: word t of 16-byte unit 4 j + i of
      // a head holds channels 32 j + 8 t + 2 i, + 1.  The buffer is free once the piece before the last is through.
      auto write_q = [&](const Piece4& pc) {
        if (gp > 1 && !mbar_wait_lean_warp(&o_free[gp & 1], ((gp >> 1) - 1) & 1, wctl)) {
          ok = false;
          return;
        }
        const uint16_t* q = p.q + ((int64_t)pc.row * p.num_heads + (int64_t)pc.kvh * G + h0) * kHeadDim;
        uint8_t* dst = smem + S::kOffQ + (gp & 1) * S::kQBytes;
#pragma unroll 2
        for (int u = lane; u < HN * 8; u += 32) {
          const int t = u & 3, j = u >> 5 & 3, h = (u >> 2 & 7) | (u >> 7 << 4) | set << 3;
          uint4 x = make_uint4(0u, 0u, 0u, 0u);
          if (h < nh) x = __ldg(reinterpret_cast<const uint4*>(q + h * kHeadDim + 32 * j + 8 * t));
          uint32_t* y = reinterpret_cast<uint32_t*>(dst + (h >> 3) * 2048 + j * 512 + (h & 7) * 16 + t * 4);
          y[0] = bf16x2_to_f16x2(x.x);
          y[32] = bf16x2_to_f16x2(x.y);
          y[64] = bf16x2_to_f16x2(x.z);
          y[96] = bf16x2_to_f16x2(x.w);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[gp & 1]);
      };
      for (int pi = 0; pi < count && ok; ++pi) {
        const Piece4 pc = pieces[pi];
        const int nt = piece_tiles(pc);
        const int32_t* table = p.table + (int64_t)pc.b * p.max_pages;
        const uint8_t* pages = p.pages[pc.kvh];
        const int num_pages = p.num_pages[pc.kvh];
        const int first = pc.start / kBlk, last = (pc.end - 1) / kBlk;  // groups of 16 keys that the piece needs
        // This lane's groups of tile t: [lo, hi) of the tile's eight, none when lo >= hi.
        auto groups = [&](int t, int& lo, int& hi) {
          const int base = (pc.start / kT + t) * kTileBlks;
          lo = max(first - base, lane * per);
          hi = lane < in_tile ? min(last + 1 - base, (lane + 1) * per) : lo;
        };
        auto load_id = [&](int t) -> int32_t {
          int lo, hi;
          groups(t, lo, hi);
          return t < nt && lo < hi ? __ldg(table + ((pc.start / kT + t) * kT / P + lane)) : -1;
        };
        int t = (set - gt) & 1;
        int32_t id_next = load_id(t);
        bool q_written = nt == 0;
        for (; t < nt; t += 2) {
          const int x = gt + t, s = x % NS;
          const int32_t id = id_next;
          id_next = load_id(t + 2);
          if (x >= NS && !mbar_wait_lean_warp(&raw_empty[s], (x / NS - 1) & 1, wctl)) {
            ok = false;
            break;
          }
          int lo, hi;
          groups(t, lo, hi);
          const bool live = lo < hi, in_range = (uint32_t)id < (uint32_t)num_pages;
          if (live && !in_range && p.err) atomicOr(p.err, CAI_DEVERR_PAGE);
          const uint32_t okm = __reduce_or_sync(0xffffffffu, live && in_range ? ((1u << hi) - 1) & ~((1u << lo) - 1) : 0u);
          issued = x + 1;
          if (x == p.drop_stage) continue;  // fault injection: never issued
          if (lane == 0) {
            volatile int4* y = info + x % kInfo;
            const int base = (pc.start / kT + t) * kT;
            y->x = pc.start - base;
            y->y = pc.end - base;
            y->z = (int)okm;
            mbar_arrive_expect_tx(&raw_full[s], (uint32_t)__popc(okm) * kBlkBytes);
          }
          __syncwarp();
          if (live && in_range)
            bulk_g2s(smem + s * kTileBytes + lo * kBlkBytes, pages + ((int64_t)id * per + (lo - lane * per)) * kBlkBytes,
                     (uint32_t)(hi - lo) * kBlkBytes, &raw_full[s]);
          if (!q_written) {  // (after the piece's first copies)
            q_written = true;
            write_q(pc);
            if (!ok) break;
          }
        }
        if (!q_written && ok) write_q(pc);
        gt += nt;
        gp += nt > 0;
      }
    } else {
      // ------------------------------------------------------------------ issuer of a set
      // S^T of the set's next tile goes out before PV of this one, so that its softmax need not wait.
      const int set = warp - kSets;
      const uint32_t tm = tmem + set * S::kSetCols;
      const uint64_t dq = smem_desc(smem_addr(smem + S::kOffQ), 128, 2048);
      const uint64_t dp = smem_desc(smem_addr(smem + S::kOffP + 2 * set * S::kPBytes), 128, kT * 16);
      constexpr uint32_t idesc_s = idesc_f16_f32(kT, HN, 0, 0), idesc_o = idesc_f16_f32(kHeadDim, HN, 0, 1);
      auto issue_s = [&](int n, int piece, bool first) {
        ok = (!first || mbar_wait_lean_warp(&q_full[piece & 1], (piece >> 1) & 1, wctl)) && mbar_wait_lean_warp(&k_full[set], n & 1, wctl) &&
             (n == 0 || mbar_wait_lean_warp(&s_read[set], (n - 1) & 1, wctl));
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kHeadDim / 16; ++k)
            mma_f16_ts(tm + S::kColS, tm + k * 8, dq + (uint64_t)((piece & 1) * (S::kQBytes >> 4) + k * 16), idesc_s, k > 0 ? 1u : 0u);
          mma_commit(&s_full[set]);
        }
        __syncwarp();
      };
      auto issue_pv = [&](int n, int piece, bool first) {
        const int k2 = n & 1;
        // (the piece's first PV of the set starts the accumulator, once the last piece's has been read)
        ok = mbar_wait_lean_warp(&v_full[2 * set + k2], (n >> 1) & 1, wctl) && mbar_wait_lean_warp(&p_full[2 * set + k2], (n >> 1) & 1, wctl) &&
             (!first || piece == 0 || mbar_wait_lean_warp(&o_free[(piece - 1) & 1], ((piece - 1) >> 1) & 1, wctl));
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kT / 16; ++k)
            mma_f16_ts(tm + S::kColO, tm + S::kColV + (S::kVBufs == 2 ? k2 * 64 : 0) + k * 8, dp + (uint64_t)(k2 * (S::kPBytes >> 4) + k * 16), idesc_o,
                       (!first || k > 0) ? 1u : 0u);
          mma_commit(&pv_done[2 * set + k2]);
        }
        __syncwarp();
      };
      for (int pi = 0; pi < count && ok; ++pi) {
        const int nt = piece_tiles(pieces[pi]);
        if (nt == 0) continue;
        // (the set's last PV of a piece does not wait for a tile of the next, whose first PV waits for this piece's end)
        int last_n = -1;  // the tile whose PV is still to come
        bool last_first = false;
        for (int t = (set - gt) & 1; ok; t += 2) {
          const bool more = t < nt;
          const int n = (gt + t) >> 1;
          if (more) issue_s(n, gp, last_n < 0);
          if (ok && last_n >= 0) issue_pv(last_n, gp, last_first);
          if (!more) break;
          last_first = last_n < 0;
          last_n = n;
        }
        gt += nt;
        ++gp;
      }
    }
    });
  } else if (warp < kSoft0) {
    setmaxnreg_dec<S::kRegsConv>();
    lists([&](int count) {
      // ------------------------------------------------------------------ converters of a set
      // K of the set's next tile goes before V of this one: V may have to wait for the products that its softmax
      // comes before.  The waits are tried a step ahead (a wait costs 150 cycles and more even when its phase is
      // over), and a step's stores are waited for after the next one's loads.
      // A lane whose wait gave up carries on (on garbage) and releases nothing that it did not see land; the
      // lanes agree on stopping after each tile.
      const int set = (warp - kConv0) >> 2, quarter = warp & 3;
      const int g = lane >> 2, t4 = lane & 3;
      const uint32_t tm = tmem + set * S::kSetCols + ((uint32_t)(quarter * 32) << 16);
      int total = 0;
      for (int pi = 0; pi < count; ++pi) total += piece_tiles(pieces[pi]);
      const int end = gt + total;
      bool landed = false, raw_there = false;
      constexpr int kB = S::kVBufs;  // V^T's buffer was read by PV of the set's tile n - kB
      // (x: the tile whose V is converted, x + 2: K.  Loops are kept rolled: the roles' instructions together
      // pass the cache's size soon, unrolled twice as far this cost 20%.)
      constexpr int kAhead = kB == 1 ? 2 : 0;
      for (int x = gt + ((set - gt) & 1) - kAhead; x < end; x += 2) {
        const int n = x >> 1;
        const int xk = x + kAhead, nk = xk >> 1; const bool has_k = xk < end, has_v = x >= gt;
        bool landed_next = false;
        if (has_k) {
          // ---- K of two 16-key groups, column 16 j + 4 i + t: channels 32 j + 8 t + 2 i, + 1; free once S^T of the
          // set's last tile is done.
          const int s = xk % NS;
          const bool k_there = nk < 1 || mbar_test_wait(&s_full[set], (nk - 1) & 1);
          landed_next = raw_there || mbar_wait_lean(&raw_full[s], (xk / NS) & 1, wctl);
          ok = ok && landed_next;
          if (!k_there) ok = mbar_wait_lean(&s_full[set], (nk - 1) & 1, wctl) && ok;
          __syncwarp();
          tc_fence_after();
          const uint8_t* blk = smem + s * kTileBytes + 2 * quarter * kBlkBytes;
#pragma unroll 1
          for (int a = 0; a < 2; ++a, blk += kBlkBytes) {
            uint4 kw[2];
            uint2 ks[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              kw[e] = *reinterpret_cast<const uint4*>(blk + e * 512 + lane * 16);
              ks[e] = *reinterpret_cast<const uint2*>(blk + kBlkKs + e * 64 + g * 8);
            }
#pragma unroll
            for (int j2 = 0; j2 < 2; ++j2) {
              uint32_t r[16];
#pragma unroll
              for (int jj = 0; jj < 2; ++jj) {
                const uint32_t sel = jj ? 0x3232u : 0x1010u;
                const uint32_t sa = __byte_perm(j2 ? ks[0].y : ks[0].x, 0u, sel), sb = __byte_perm(j2 ? ks[1].y : ks[1].x, 0u, sel);
                uint32_t u[4], v[4];
                values_f16(j2 ? (jj ? kw[0].w : kw[0].z) : (jj ? kw[0].y : kw[0].x), sa, sa, u);
                values_f16(j2 ? (jj ? kw[1].w : kw[1].z) : (jj ? kw[1].y : kw[1].x), sb, sb, v);
#pragma unroll
                for (int e = 0; e < 4; ++e) r[8 * jj + 2 * e] = u[e], r[8 * jj + 2 * e + 1] = v[e];
              }
              tmem_st_16x128b_x8(tm + ((uint32_t)(16 * a) << 16) + j2 * 32, r);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&k_full[set]);
        }
        if (has_v) {
          // ---- V of this quarter's 32 channels, column k: keys 2 k, 2 k + 1
          const int s = x % NS;
          const bool v_there = n < kB || mbar_test_wait(&pv_done[2 * set + ((n - kB) & 1)], ((n - kB) >> 1) & 1);
          const int lo = info[x % kInfo].x, hi = info[x % kInfo].y, okm = info[x % kInfo].z;
          const bool edge = lo > 0 || hi < kT || okm != 255;
          if (!v_there) ok = mbar_wait_lean(&pv_done[2 * set + ((n - kB) & 1)], ((n - kB) >> 1) & 1, wctl) && ok;
          __syncwarp();
          tc_fence_after();
          const uint8_t* blk = smem + s * kTileBytes;
#pragma unroll 1
          for (int kh = 0; kh < 2; ++kh, blk += 4 * kBlkBytes) {
            uint2 vw[4];
            uint32_t s0[4], s1[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              vw[e] = *reinterpret_cast<const uint2*>(blk + e * kBlkBytes + kBlkV + (quarter >> 1) * 512 + lane * 16 + (quarter & 1) * 8);
              s0[e] = *reinterpret_cast<const uint32_t*>(blk + e * kBlkBytes + kBlkVs + t4 * 32 + quarter * 4);
              s1[e] = *reinterpret_cast<const uint32_t*>(blk + e * kBlkBytes + kBlkVs + t4 * 32 + 16 + quarter * 4);
            }
            if (edge) {
              // Masked keys' scales become 0 (their slots may hold anything, NaN included).
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int at = (4 * kh + e) * kBlk + 2 * t4;
                const bool good = (okm >> (4 * kh + e)) & 1;
                auto keep = [&](int y) { return good && y >= lo && y < hi; };
                s0[e] &= (keep(at) ? 0xFFFFu : 0u) | (keep(at + 1) ? 0xFFFF0000u : 0u);
                s1[e] &= (keep(at + 8) ? 0xFFFFu : 0u) | (keep(at + 9) ? 0xFFFF0000u : 0u);
              }
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              uint32_t r[16];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t u[4];
                values_f16(m == 0 ? vw[e].x : vw[e].y, s0[e], s1[e], u);
#pragma unroll
                for (int y = 0; y < 4; ++y) r[4 * e + y] = u[y];
              }
              tmem_st_16x128b_x8(tm + ((uint32_t)(16 * m) << 16) + S::kColV + (kB == 2 ? (n & 1) * 64 : 0) + kh * 32, r);
            }
          }
          raw_there = xk + 2 < end && mbar_test_wait(&raw_full[(xk + 2) % NS], ((xk + 2) / NS) & 1);
          tmem_wait_st();
          tc_fence_before();
          ok = __all_sync(0xffffffffu, ok);
          if (lane == 0) {
            if (kAhead ? landed : landed_next) mbar_arrive(&raw_empty[s]);
            mbar_arrive(&v_full[2 * set + (n & 1)]);
          }
          if (!ok) break;
        }
        landed = landed_next;
      }
      gt = end;
    });
  } else {
    setmaxnreg_inc<S::kRegsSoft>();
    lists([&](int count) {
      // ------------------------------------------------------------------ softmax of a set, merge, epilogue
      // A thread whose wait gave up carries on with the same steps (on garbage) until the set's next
      // barrier-reduction, which stops its four warps; at the piece's end both sets stop.
      const int set = (warp - kSoft0) >> 2, quarter = warp & 3;
      const uint32_t tm = tmem + set * S::kSetCols + ((uint32_t)(quarter * 32) << 16);
      const uint32_t bar = 1 + set;
      const int key = quarter * 32 + lane;       // this thread's key of a tile (and channel of O^T)
      float* wmax = xch + set * S::kXFloats;     // [quarter][HN] maxima of a raise
      const uint64_t sl2 = f2(p.scale_log2, p.scale_log2);

      for (int pi = 0; pi < count; ++pi) {
        const Piece4 pc = pieces[pi];
        const int nt = piece_tiles(pc);
        const int64_t row0 = (int64_t)pc.row * p.num_heads + (int64_t)pc.kvh * G + h0;  // the block's first head row
        if (nt == 0) {  // nothing to attend, or an invalid length (flagged): out = 0, lse = -inf
          const int tid = threadIdx.x - 32 * kSoft0;
          for (int i = tid; i < nh * kHeadDim / 4; i += kSoftThreads)
            reinterpret_cast<uint2*>(p.out + row0 * kHeadDim)[i] = make_uint2(0u, 0u);
          if (p.lse_out && tid < nh) p.lse_out[row0 + tid] = -INFINITY;
          continue;
        }
        float* nref = wmax + S::kXRef + ((gp & 1) * 4 + quarter) * HN;  // negated references (log2 units)
        float* part = wmax + S::kXSum + ((gp & 1) * 4 + quarter) * HN;  // sums of a piece
        if (lane < HN / 4) reinterpret_cast<float4*>(nref)[lane] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        __syncwarp();
        uint64_t l[HN / 2];     // this key's sums, per head pair
#pragma unroll
        for (int h = 0; h < HN / 2; ++h) l[h] = 0ull;
        bool have_ref = false;  // some key was attended (the same in the whole set)
        for (int t = (set - gt) & 1; t < nt; t += 2) {
          const int x = gt + t, n = x >> 1;
          ok = mbar_wait_lean(&s_full[set], n & 1, wctl) && ok;
          // P^T's buffer is free once PV of the set's tile n - 2 is done.
          if (n > 1) ok = mbar_wait_lean(&pv_done[2 * set + (n & 1)], ((n >> 1) - 1) & 1, wctl) && ok;
          __syncwarp();
          tc_fence_after();
          const int lo = info[x % kInfo].x, hi = info[x % kInfo].y, okm = info[x % kInfo].z;
          const bool edge = lo > 0 || hi < kT || okm != 255;
          const bool valid = key >= lo && key < hi && ((okm >> (key / kBlk)) & 1);
          float sv[HN];
          // Logits minus references, from S^T (which stays in tensor memory until the set says it is read); their largest.
          auto logits = [&]() -> float {
            float mx = -INFINITY;
#pragma unroll
            for (int h1 = 0; h1 < HN; h1 += 16) {
              uint32_t r[16];
              tmem_ld_n(tm + S::kColS + h1, r);
              tmem_wait_ld();
#pragma unroll
              for (int h = 0; h < 16; h += 4) {
                const float4 x4 = *reinterpret_cast<const float4*>(nref + h1 + h);
                f2_split(f2_fma(f2(__uint_as_float(r[h]), __uint_as_float(r[h + 1])), sl2, f2(x4.x, x4.y)), sv[h1 + h], sv[h1 + h + 1]);
                f2_split(f2_fma(f2(__uint_as_float(r[h + 2]), __uint_as_float(r[h + 3])), sl2, f2(x4.z, x4.w)), sv[h1 + h + 2], sv[h1 + h + 3]);
              }
            }
            if (edge) {
#pragma unroll
              for (int h = 0; h < HN; ++h) sv[h] = valid ? sv[h] : -INFINITY;
            }
#pragma unroll
            for (int h = 0; h < HN; h += 2) mx = fmax3(mx, sv[h], sv[h + 1]);
            return mx;
          };
          // The weights, in place of the logits, and P^T's row of this key: heads 8 i .. 8 i + 7 at i * 2048 + key * 16.
          uint8_t* dst = smem + S::kOffP + (2 * set + (n & 1)) * S::kPBytes + key * 16;
          auto weights = [&]() {
#pragma unroll
            for (int i = 0; i < HN / 8; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float& a = sv[8 * i + 2 * e];
                float& b = sv[8 * i + 2 * e + 1];
                a = ex2_approx(a);
                b = ex2_approx(b);
                w[e] = pack_f16x2(a, b);
              }
              *reinterpret_cast<uint4*>(dst + i * 2048) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          };
          bool raise = !have_ref, stop = false;
          while (true) {  // (one copy of the code: instruction cache)
            const float mx = logits();
            const bool raised = raise;
            if (raise) {
            // Raise the references that a logit passes by 2^15 (all of them at the first tile with a key).
#pragma unroll
            for (int h1 = 0; h1 < HN; h1 += 16) {  // 16 heads at a time
              float mine = -INFINITY;
#pragma unroll
              for (int h = 0; h < 16; ++h) {
                float m;
                asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(sv[h1 + h]));
                mine = lane == h ? m : mine;
              }
              if (lane < 16) wmax[quarter * HN + h1 + lane] = mine;
            }
            if (bar_red_or(bar, 128, !ok)) {
              stop = true;  // (all four warps are here)
              break;
            }
            if (have_ref) {
              // O^T holds earlier tiles of the piece: the set's last PV must be done before it is rescaled.
              if (n > 0) ok = mbar_wait_lean(&pv_done[2 * set + ((n - 1) & 1)], ((n - 1) >> 1) & 1, wctl) && ok;
              __syncwarp();
              tc_fence_after();
            }
            const bool any = okm != 0;  // some key of the tile is attended
#pragma unroll
            for (int h1 = 0; h1 < HN; h1 += 8) {
              float up = 0.0f, f = 0.0f;  // of head h1 + lane: what its reference rises by, and 2^-up
              if (lane < 8) {
                const float* w = wmax + h1 + lane;
                const float v = fmaxf(fmaxf(w[0], w[HN]), fmaxf(w[2 * HN], w[3 * HN]));
                up = any && (!have_ref || v > kRaiseTc) ? v - kWeightLift : 0.0f;
                f = ex2_approx(-up);
                nref[h1 + lane] -= up;
              }
#pragma unroll
              for (int h = 0; h < 8; ++h) sv[h1 + h] -= __shfl_sync(0xffffffffu, up, h);
              if (have_ref) {
                float fs[8];
#pragma unroll
                for (int h = 0; h < 8; ++h) fs[h] = __shfl_sync(0xffffffffu, f, h);
#pragma unroll
                for (int h = 0; h < 8; h += 2) l[(h1 + h) / 2] = f2_mul(l[(h1 + h) / 2], f2(fs[h], fs[h + 1]));
                uint32_t r[8];
                tmem_ld_n(tm + S::kColO + h1, r);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * fs[e]);
                tmem_st_n(tm + S::kColO + h1, r);
              }
            }
            if (have_ref) tmem_wait_st();
            have_ref = have_ref || any;
            }
            weights();
            if (raised) break;
            raise = bar_red_or(bar, 128, !ok || mx > kRaiseTc);
            if (!raise) break;
          }
          if (stop) {
            ok = false;
            break;
          }
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&s_read[set]);
            mbar_arrive(&p_full[2 * set + (n & 1)]);
          }
#pragma unroll
          for (int h = 0; h < HN; h += 2) l[h / 2] = f2_add(l[h / 2], f2(sv[h], sv[h + 1]));
        }
        const int g_end = gt + nt;

        // ---- end of piece: the set's sums over its keys, 16 heads at a time
#pragma unroll
        for (int h1 = 0; h1 < HN; h1 += 16) {
          float v[16];
#pragma unroll
          for (int h = 0; h < 16; h += 2) f2_split(l[(h1 + h) / 2], v[h], v[h + 1]);
          // Reduce-scatter: lane i ends with the warp's sum of head h1 + i % 16.
#pragma unroll
          for (int o = 8; o >= 1; o >>= 1) {
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int i = 0; i < o; ++i) {
              const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
              v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
          }
          v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
          if (lane < 16) {
            part[h1 + lane] = v[0];
            if (!have_ref) nref[h1 + lane] = INFINITY;  // nothing attended: weight 0
          }
        }
        if (bar_red_or(kBarPiece, kSoftThreads, !ok)) {
          ok = false;
          break;
        }
        // The sets' last PVs of the piece.
#pragma unroll
        for (int k = 0; k < kSets; ++k) {
          const int last = g_end - 1 - ((g_end - 1 - k) & 1);  // the last tile of set k
          const int n = last >> 1;
          if (last >= gt) ok = mbar_wait_lean(&pv_done[2 * k + (n & 1)], (n >> 1) & 1, wctl) && ok;
        }
        __syncwarp();
        tc_fence_after();
        // ---- merge of the sets: a warp has its quarter's channels of half of the heads, lane h the factors of the
        // h-th of these (0 for a set that attended nothing).
        const int64_t slot0 = (int64_t)pc.slot * G + h0;
        const int hh = set * (HN / 2);
        float f[kSets];
        {
          const float* x = xch + hh + (lane < HN / 2 ? lane : 0);
          const int at = (gp & 1) * 4 * HN;
          float m[kSets], M = -INFINITY, sum = 0.0f;
#pragma unroll
          for (int k = 0; k < kSets; ++k) {
            m[k] = -x[k * S::kXFloats + S::kXRef + at];
            M = fmaxf(M, m[k]);
          }
#pragma unroll
          for (int k = 0; k < kSets; ++k) {
            const float* y = x + k * S::kXFloats + S::kXSum + at;
            f[k] = m[k] == -INFINITY ? 0.0f : ex2_approx(m[k] - M);
            if (f[k] != 0.0f) sum = fmaf(f[k], (y[0] + y[HN]) + (y[2 * HN] + y[3 * HN]), sum);
          }
          const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
          for (int k = 0; k < kSets; ++k) f[k] *= inv;
          if (quarter == 0 && lane < HN / 2 && hh + lane < nh) {
            const float lse2 = sum > 0.0f ? M + log2f(sum) : -INFINITY;
            if (pc.slot >= 0) p.ws_lse[slot0 + hh + lane] = lse2;
            else if (p.lse_out) p.lse_out[row0 + hh + lane] = lse2 * kLn2;
          }
        }
#pragma unroll 1
        for (int h1 = 0; h1 < HN / 2; h1 += 8) {
          uint32_t r[kSets][8];
#pragma unroll
          for (int k = 0; k < kSets; ++k)
            tmem_ld_n(tmem + ((uint32_t)(quarter * 32) << 16) + k * S::kSetCols + S::kColO + hh + h1, r[k]);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            float x = 0.0f;
#pragma unroll
            for (int k = 0; k < kSets; ++k) {
              // (a set without a tile has no accumulator: whatever is there does not count)
              const float a = __shfl_sync(0xffffffffu, f[k], h1 + h);
              x = a != 0.0f ? fmaf(a, __uint_as_float(r[k][h]), x) : x;
            }
            if (hh + h1 + h < nh) {
              if (pc.slot < 0) p.out[(row0 + hh + h1 + h) * kHeadDim + key] = (uint16_t)pack_bf16x2(x, 0.0f);
              else p.ws_o[(slot0 + hh + h1 + h) * kHeadDim + key] = x;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[gp & 1]);
        // (sums and references of the next piece have the other buffer; both sets' readers of that one have come
        // to this piece's barrier)
        ++gp;
        gt = g_end;
      }
    });
  }

  // What this block started has ended before it goes away: the producer's copies, the issuers' products.
  if (warp < kSets) {
    for (int x = max(0, issued - NS); x < issued; ++x)
      if ((x & 1) == warp && x != p.drop_stage) mbar_wait_drain(&raw_full[x % NS], (x / NS) & 1);
  } else if (warp < 2 * kSets) {
    if (elect_one()) mma_commit(drain);
    __syncwarp();
    mbar_wait_drain(drain, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && wctl->abort && p.err) atomicOr(p.err, CAI_DEVERR_TIMEOUT);
  if (warp == 0) tmem_dealloc(tmem, 512);
  if (p.overlap_prev) grid_dependency_wait();
}

template <int HN>
cudaError_t launch_hn(const Decode4Params& p, cudaStream_t stream) {
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_set[dev]) {
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, decode4_tc_kernel<HN>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != ShapeTc<HN>::kRegsLaunch) return cudaErrorInvalidDeviceFunction;
    e = cudaFuncSetAttribute(decode4_tc_kernel<HN>, cudaFuncAttributeMaxDynamicSharedMemorySize, ShapeTc<HN>::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set[dev] = true;
  }
  return launch_pdl(decode4_tc_kernel<HN>, dim3((unsigned)(p.head_groups * p.ranges)), dim3(kTcThreads), ShapeTc<HN>::kSmem,
                    stream, p);
}

}  // namespace

int decode4_tc_heads(int group) { return group <= 8 ? 0 : group <= 16 ? 16 : group <= 32 ? 32 : 64; }

cudaError_t launch_decode4_tc(const Decode4Params& p, cudaStream_t stream) {
  switch (decode4_tc_heads(p.num_heads / p.num_kv_heads)) {
    case 16: return launch_hn<16>(p, stream);
    case 32: return launch_hn<32>(p, stream);
    default: return launch_hn<64>(p, stream);
  }
}

}  // namespace cai

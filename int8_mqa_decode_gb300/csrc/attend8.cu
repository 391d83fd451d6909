// Attention over lists of pages of the int8 cache, on the 5th-generation tensor cores: for every row of queries and
// K/V head the pages that its list names, in turn.  The split of the work, its pieces and the merge are the 4-bit
// decode's (decode4.cuh, decode4.cu), and so is the plan of the kernel (decode4_tc.cu): two sets of warps that take every
// other tile of 128 keys, S^T = K Q^T and O^T += V^T P^T with tcgen05.mma kind::f16, A operands and accumulators in tensor
// memory.  What differs follows from the cache's format.
//
// A page is rows of 128 bytes, K's codes token by token and V's channel by channel.  A tensor copy brings a page's code
// rows swizzled, so that a converting thread reads the row of its token (K) or channel (V) free of bank conflicts,
// and stores fp16 (exact) as its lane of the operand; the scales, one of K and one of V a token, follow in a bulk copy.
// A softmax thread has one token: it applies K's scale to the logits, and V's to the weights.
//
// V's scale goes into the exponent: with v the token's scale, the weight that multiplies V's codes is 2^(z + log2 v - r),
// r the reference, chosen so that the largest such weight is 2^7 to 2^15; the sum of the softmax takes it over v, in fp32.  So
// the weights keep fp16's eleven bits whatever the size of V: scaled after the exponential, a cache of small values
// (v about 2^-17) would leave them among the subnormals.  Scales below 2^-100 count as 2^-100, and so does that of a
// token whose V is 0: its codes are 0, and it moves no reference.
//
// Roundings: the query to fp16 (exact for magnitudes from 2^-17 to 65504, below that off by 2^-25 at most), a weight to
// fp16 for its product with V (2^-11 of it, or 2^-32 of the largest), the output to bf16 once; the rest is fp32.
#include <cmath>

#include "decode4.cuh"
#include "tma.cuh"

namespace cai {
namespace {

constexpr int kSets = 2;
// Warpgroups: control (a producer and an issuer per set), two of converters, two of softmax.
constexpr int kConv0 = 4, kSoft0 = kConv0 + 4 * kSets;
constexpr int kTcThreads = 32 * (kSoft0 + 4 * kSets);
constexpr int kSoftThreads = 128 * kSets;
constexpr int kT = kDecodeTile;                      // 128 keys
constexpr int kTileBlks = kT / kBlk;                 // groups of 16 tokens, the smallest page
constexpr int kCodeBytes = kT * 2 * kHeadDim;        // code rows of a tile's pages, then their scales
constexpr int kTileBytes = kCodeBytes + kT * 8;      // 33792, a multiple of the swizzle's 1024
constexpr int kInfo = 16;                            // ring of tiles' key ranges, longer than any lag
constexpr float kRaiseTc = kWeightLift + 8.0f;       // log2 units a logit may exceed its reference by
constexpr uint32_t kBarPiece = 1 + kSets;            // named barriers: 1 + set (its softmax), all softmax warps

template <int HN>
struct Shape8 {
  // Raw tiles, two a set: a stage belongs to a set, whose waits for it are then at most one phase behind.  (Five of them in
  // turn for both sets would fit: a set then takes the end of the phase before last for its tile's arrival.)
  static constexpr int kStages = 2 * kSets;
  static constexpr int kPBufs = HN == 64 ? 1 : 2;                    // P^T of a set: what fits beside the raw tiles
  static constexpr int kPBytes = HN * kT * 2;
  static constexpr int kOffP = kStages * kTileBytes;                 // P^T [set][kPBufs]
  static constexpr int kOffQ = kOffP + kPBufs * kSets * kPBytes;     // Q^T [2 pieces]
  static constexpr int kQBytes = HN * kHeadDim * 2;
  static constexpr int kOffX = kOffQ + 2 * kQBytes;                  // [set] exchange:
  // [4 quarters][HN] maxima; [2 pieces][4 quarters][HN] sums; the same of references (a copy per quarter)
  static constexpr int kXSum = 4 * HN, kXRef = 12 * HN, kXFloats = 20 * HN;
  static constexpr int kOffTok = kOffX + kSets * kXFloats * 4;       // [set][2 tiles][key]: K's scale (log2 units), V's
  static constexpr int kOffBars = kOffTok + kSets * 2 * kT * 8;
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

// Sixteen int8 codes -> eight pairs of fp16, exact.
__device__ __forceinline__ void codes8(const uint4& w, uint32_t* r) {
  i8x4_to_f16x4(w.x, r[0], r[1]);
  i8x4_to_f16x4(w.y, r[2], r[3]);
  i8x4_to_f16x4(w.z, r[4], r[5]);
  i8x4_to_f16x4(w.w, r[6], r[7]);
}

__device__ __forceinline__ int piece_tiles(const Piece4& pc) {
  return pc.start < pc.end ? (pc.end - 1) / kT - pc.start / kT + 1 : 0;
}

struct Attend8Args {
  Decode4Params p;
  CUtensorMap map[kMaxKvHeads];  // each pool as rows of 128 bytes; a box is the code rows of a page
};

template <int HN>
__global__ void __launch_bounds__(kTcThreads, 1) attend8_kernel(const __grid_constant__ Attend8Args args) {
  const Decode4Params& p = args.p;
  using S = Shape8<HN>;
  constexpr int NS = S::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];  // (aligned by hand, it would be addressed as generic memory)
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
      // Two copies a page, its code rows and its scales.  Lane l: page l of the tile.
      const int set = warp;
      const int P = p.page_size, per = P / kBlk, in_tile = kT / P;
      // Half of a piece's query as Q^T (8 channels a 16-byte unit).  The buffer is free once the piece before the last
      // is through.
      auto write_q = [&](const Piece4& pc) {
        if (gp > 1 && !mbar_wait_lean_warp(&o_free[gp & 1], ((gp >> 1) - 1) & 1, wctl)) {
          ok = false;
          return;
        }
        const uint16_t* q = p.q + ((int64_t)pc.row * p.num_heads + (int64_t)pc.kvh * G + h0) * kHeadDim;
        uint8_t* dst = smem + S::kOffQ + (gp & 1) * S::kQBytes;
#pragma unroll 2
        for (int u = lane; u < HN * 8; u += 32) {
          const int h = (u & 7) | (u >> 7 << 4) | set << 3, c8 = u >> 3 & 15;
          uint4 x = make_uint4(0u, 0u, 0u, 0u);
          if (h < nh) x = __ldg(reinterpret_cast<const uint4*>(q + h * kHeadDim + 8 * c8));
          *reinterpret_cast<uint4*>(dst + (h >> 3) * 2048 + c8 * 128 + (h & 7) * 16) =
              make_uint4(bf16x2_to_f16x2(x.x), bf16x2_to_f16x2(x.y), bf16x2_to_f16x2(x.z), bf16x2_to_f16x2(x.w));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[gp & 1]);
      };
      for (int pi = 0; pi < count && ok; ++pi) {
        const Piece4 pc = pieces[pi];
        const int nt = piece_tiles(pc);
        const int32_t* table = piece_table(p, pc);
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
          // (bits: groups of 16 tokens of the pages that are there; a page is copied whole)
          const uint32_t okm = __reduce_or_sync(0xffffffffu, live && in_range ? ((1u << per) - 1) << (lane * per) : 0u);
          issued = x + 1;
          if (x == p.drop_stage) continue;  // fault injection: never issued
          if (lane == 0) {
            volatile int4* y = info + x % kInfo;
            const int base = (pc.start / kT + t) * kT;
            y->x = pc.start - base;
            y->y = pc.end - base;
            y->z = (int)okm;
            mbar_arrive_expect_tx(&raw_full[s], (uint32_t)(__popc(okm) / per) * page_bytes(P));
          }
          __syncwarp();
          if (live && in_range) {
            uint8_t* stage = smem + s * kTileBytes;
            tma_load_2d(stage + lane * (2 * P * kHeadDim), &args.map[pc.kvh], 0, id * (page_bytes(P) / 128), &raw_full[s]);
            bulk_g2s(stage + kCodeBytes + lane * (8 * P), pages + (int64_t)id * page_bytes(P) + 2 * P * kHeadDim, 8 * P, &raw_full[s]);
          }
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
      const uint64_t dp = smem_desc(smem_addr(smem + S::kOffP + S::kPBufs * set * S::kPBytes), 128, kT * 16);
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
            mma_f16_ts(tm + S::kColO, tm + S::kColV + (S::kVBufs == 2 ? k2 * 64 : 0) + k * 8, dp + (uint64_t)((S::kPBufs == 2 ? k2 : 0) * (S::kPBytes >> 4) + k * 16), idesc_o,
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
      const int P = p.page_size, lg = P == 16 ? 4 : P == 32 ? 5 : 6;
      const int row = quarter * 32 + lane;  // this thread's key (K) and channel (V)
      // Its 128-byte row of K in a stage; the row and first chunk of its channel in a page's V.
      const uint32_t k_at = (uint32_t)((row >> lg) * 2 * P + (row & (P - 1))) * 128, k_x = row & 7;
      const uint32_t v_at = (uint32_t)(P + (row << lg >> 7)) * 128, v_c = (row << lg & 127) >> 4, v_x = (row << lg >> 7) & 7;
      const uint32_t s_at = kCodeBytes + ((row >> lg) * 2 * P + (row & (P - 1))) * 4;
      const uint32_t tm = tmem + set * S::kSetCols + ((uint32_t)(quarter * 32) << 16);
      float2* tok = reinterpret_cast<float2*>(smem + S::kOffTok) + set * 2 * kT;  // (a tile's is read before the S^T after the next goes out)
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
          // ---- K of this thread's key, column k: channels 2 k, 2 k + 1; free once S^T of the set's last tile is done.
          const int s = xk % NS;
          const bool k_there = nk < 1 || mbar_test_wait(&s_full[set], (nk - 1) & 1);
          landed_next = raw_there || mbar_wait_lean(&raw_full[s], (xk / NS) & 1, wctl);
          ok = ok && landed_next;
          if (!k_there) ok = mbar_wait_lean(&s_full[set], (nk - 1) & 1, wctl) && ok;
          __syncwarp();
          tc_fence_after();
          const uint8_t* stage = smem + s * kTileBytes;
          const float* sc = reinterpret_cast<const float*>(stage + s_at);
          tok[(nk & 1) * kT + row] = make_float2(sc[0] * p.scale_log2, sc[P]);
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            uint32_t r[16];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint4 w = *reinterpret_cast<const uint4*>(stage + k_at + (((2 * i + e) ^ k_x) << 4));
              codes8(w, r + 8 * e);
            }
            tmem_st_32x32b_x16(tm + i * 16, r);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&k_full[set]);
        }
        if (has_v) {
          // ---- V of this thread's channel, column k: keys 2 k, 2 k + 1
          const int s = x % NS;
          const bool v_there = n < kB || mbar_test_wait(&pv_done[2 * set + ((n - kB) & 1)], ((n - kB) >> 1) & 1);
          if (!v_there) ok = mbar_wait_lean(&pv_done[2 * set + ((n - kB) & 1)], ((n - kB) >> 1) & 1, wctl) && ok;
          __syncwarp();
          tc_fence_after();
          const uint8_t* stage = smem + s * kTileBytes + v_at;
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            uint32_t r[16];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int t0 = 16 * (2 * i + e);  // 16 keys of one page
              const uint4 w = *reinterpret_cast<const uint4*>(stage + (t0 >> lg) * (2 * P * kHeadDim) + (((v_c + ((t0 & (P - 1)) >> 4)) ^ v_x) << 4));
              codes8(w, r + 8 * e);
            }
            tmem_st_32x32b_x16(tm + S::kColV + (kB == 2 ? (n & 1) * 64 : 0) + i * 16, r);
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
      const float2* tok = reinterpret_cast<const float2*>(smem + S::kOffTok) + set * 2 * kT + key;

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
          __syncwarp();
          tc_fence_after();
          const int lo = info[x % kInfo].x, hi = info[x % kInfo].y, okm = info[x % kInfo].z;
          const bool edge = lo > 0 || hi < kT || okm != 255;
          const bool valid = key >= lo && key < hi && ((okm >> (key / kBlk)) & 1);
          // K's scale; V's as a power of two, and its inverse for the sums (values that are not there may be anything).
          const float2 sc = tok[(n & 1) * kT];
          const float v = fmaxf(sc.y, 0x1p-100f);
          const float ks = valid ? sc.x : 0.0f, lv = valid ? log2f(v) : 0.0f, iv = valid ? __fdividef(1.0f, v) : 0.0f;
          const uint64_t ks2 = f2(ks, ks), lv2 = f2(lv, lv), iv2 = f2(iv, iv);
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
                f2_split(f2_add(f2_fma(f2(__uint_as_float(r[h]), __uint_as_float(r[h + 1])), ks2, f2(x4.x, x4.y)), lv2), sv[h1 + h], sv[h1 + h + 1]);
                f2_split(f2_add(f2_fma(f2(__uint_as_float(r[h + 2]), __uint_as_float(r[h + 3])), ks2, f2(x4.z, x4.w)), lv2), sv[h1 + h + 2], sv[h1 + h + 3]);
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
          uint8_t* dst = smem + S::kOffP + (S::kPBufs == 2 ? 2 * set + (n & 1) : set) * S::kPBytes + key * 16;
          auto weights = [&]() {
            // P^T's buffer is free once PV of the set's tile n - kPBufs is done.
            constexpr int kB = S::kPBufs;
            if (n >= kB) ok = mbar_wait_lean(&pv_done[2 * set + ((n - kB) & 1)], ((n - kB) >> 1) & 1, wctl) && ok;
            __syncwarp();
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
          for (int h = 0; h < HN; h += 2) l[h / 2] = f2_fma(f2(sv[h], sv[h + 1]), iv2, l[h / 2]);
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
    cudaError_t e = cudaFuncGetAttributes(&fa, attend8_kernel<HN>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != Shape8<HN>::kRegsLaunch) return cudaErrorInvalidDeviceFunction;
    e = cudaFuncSetAttribute(attend8_kernel<HN>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape8<HN>::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set[dev] = true;
  }
  Attend8Args a;
  a.p = p;
  for (int j = 0; j < p.num_kv_heads; ++j)
    if (!encode_pool_map(&a.map[j], p.pages[j], p.num_pages[j], p.page_size)) return cudaErrorInvalidValue;
  return launch_pdl(attend8_kernel<HN>, dim3((unsigned)(p.head_groups * p.ranges)), dim3(kTcThreads), Shape8<HN>::kSmem,
                    stream, a);
}

}  // namespace

cudaError_t launch_attend8(const Decode4Params& p, cudaStream_t stream) {
  const int G = p.num_heads / p.num_kv_heads;
  return G <= 16 ? launch_hn<16>(p, stream) : G <= 32 ? launch_hn<32>(p, stream) : launch_hn<64>(p, stream);
}

}  // namespace cai

// Attention over lists of pages, on the 5th-generation tensor cores: for every row of queries and K/V head the pages that
// its list names, in turn, of the int8 cache (any group of heads) or the 4-bit cache (groups of 9 and more; smaller ones
// are decode4.cu's).  How the work is cut into pieces, and the merge of the pieces: decode4.cuh, decode4.cu.
//
// S^T = K Q^T and O^T += V^T P^T with tcgen05.mma kind::f16 (M = 128 keys or channels, N = heads padded to 16, 32 or 64,
// K = 128), A operands and accumulators in tensor memory, Q^T and P^T in shared memory, as in the 4-bit decode
// (decode4_tc.cu).  Lists are short, 16 tiles of 128 keys where the decode has hundreds, so the starts and ends of
// pieces count: a block's two sets of warps (a producer, an issuer, four converting and four softmax warps each) have
// pieces of their own and nothing in common but the block's entry and exit; while one set starts a row or
// merges it (5 k cycles), the other one's products run.  (Both sets on one piece, every other tile each, as in the decode:
// 4096 rows of 2048 tokens, 32 heads, 374 us 4-bit and 454 us int8; so 337 and 353.)  What bounds these is the issue
// slots (74% at 1200 cycles a tile): the conversion of codes, 500 instructions a warp and tile, and the softmax, 250.
// 64 rows of 4096 tokens, 64 heads, take 33 us int8 and 30 4-bit (71 MB at 2.2 TB/s): 5 k cycles until a set knows its
// piece, 8 k until its query and first tile are there (all sets ask at once), 4 k a tile, of which the converters of a set
// need 3, and 8 k for the sums and the partial output, which all sets write at once.
//
// int8.  A page is rows of 128 bytes, K's codes token by token and V's channel by channel.  A tensor copy brings a page's
// code rows swizzled, so that a converting thread reads the row of its token (K) or channel (V) free of bank conflicts,
// and stores fp16 (exact) as its lane of the operand; the scales, one of K and one of V a token, follow in a bulk copy.
// A softmax thread has one token: it applies K's scale to the logits, and V's to the weights.
//
// V's scale goes into the exponent: with v the token's scale, the weight that multiplies V's codes is 2^(z + log2 v - r),
// r the reference, chosen so that the largest such weight is 2^7 to 2^15; the sum of the softmax takes it over v, in fp32.  So
// the weights keep fp16's eleven bits whatever the size of V: scaled after the exponential, a cache of small values
// (v about 2^-17) would leave them among the subnormals.
//
// A weight below 2^-126 is 0, and its share of the sum with it; so scales count as 2^-60 U at least, those of zero vectors among
// them, with U a bound of the piece's scales so far: 2^-40, and when one passes it 2^10 times the largest of its tile.  A key of
// scale U or less set the reference at a weight of 2^7, so that it has z >= r + 7 - log2 U; a key whose weight is lost has
// z < r - 126 - log2 U + 60, a share below 2^-73 of that one's.  The output is off by 2^-50 max |V| at most, or 2^-93.  (With
// 2^-100 as the least scale of any list, zeros were lost beside scales of 2^26 and more.)
//
// Roundings: the query to fp16 (exact for magnitudes from 2^-17 to 65504, below that off by 2^-25 at most), a weight to
// fp16 for its product with V (2^-11 of it, or 2^-32 of the largest), the output to bf16 once; the rest is fp32.
//
// References (a head's running maximum, raised only when a weight would pass 2^15) are set at a piece's first tile from
// its largest weights.  That code is short, rolled loops over tensor memory: it runs once a piece, and unrolled over
// 64 heads in registers its first run in a launch took 16 k cycles of instruction fetches.
#include <cmath>

#include "decode4.cuh"
#include "tma.cuh"

namespace cai {
namespace {

constexpr int kSets = 2;
// Warpgroups: control (a producer and an issuer per set), two of converters, two of softmax.
constexpr int kConv0 = 4, kSoft0 = kConv0 + 4 * kSets;
constexpr int kThreads = 32 * (kSoft0 + 4 * kSets), kSetThreads = kThreads / kSets;
constexpr int kT = kDecodeTile;                      // 128 keys
constexpr int kTileBlks = kT / kBlk;                 // groups of 16 keys
constexpr int kCodeBytes8 = kT * 2 * kHeadDim;       // int8: code rows of a tile's pages, then their scales
constexpr int kInfo = 8;                             // ring of a set's tiles' key ranges, longer than any lag
constexpr float kRaise = kWeightLift + 8.0f;         // log2 units a weight may exceed its reference by

template <bool kFour, int HN>
struct Shape {
  // A stage belongs to a set, whose waits for it are then at most one phase behind.
  static constexpr int kTileBytes = kFour ? kTileBlks * kBlkBytes : kCodeBytes8 + kT * 8;  // 18432, 33792
  static constexpr int kStages = kFour ? (HN == 64 ? 3 : 4) : 2;     // raw tiles of a set
  static constexpr int kPBufs = !kFour && HN == 64 ? 1 : 2;          // P^T of a set
  static constexpr int kQBufs = HN == 64 ? 1 : 2;                    // Q^T of a set: pieces
  static constexpr int kPBytes = HN * kT * 2, kQBytes = HN * kHeadDim * 2;
  static constexpr int kOffP = kSets * kStages * kTileBytes;
  static constexpr int kOffQ = kOffP + kSets * kPBufs * kPBytes;
  static constexpr int kOffX = kOffQ + kSets * kQBufs * kQBytes;     // [set] exchange of the softmax warps, floats:
  // [4 quarters][HN] maxima, sums, references and factors of a raise (the latter two a copy per quarter)
  static constexpr int kXSum = 4 * HN, kXRef = 8 * HN, kXFac = 12 * HN, kXFloats = 16 * HN;
  static constexpr int kOffTok = kOffX + kSets * kXFloats * 4;       // int8: [set][2 tiles][key] K's scale (log2 units), V's
  static constexpr int kOffTop = kOffTok + (kFour ? 0 : kSets * 2 * kT * 8);  // int8: [set][quarter] V's largest scale in a tile
  static constexpr int kOffBars = kOffTop + (kFour ? 0 : kSets * 16);
  static constexpr int kSetBars = 2 * kStages + 16;
  static constexpr int kOffInfo = (kOffBars + kSets * kSetBars * 8 + 15) & ~15;  // [set] int4 per tile
  static constexpr int kOffScan = kOffInfo + kSets * kInfo * 16;     // start_lists'
  static constexpr int kOffWait = kOffScan + kThreads / 32 * 8;
  static constexpr int kOffSlot = kOffWait + 16;
  static constexpr int kOffPieces = kOffSlot + 16;                   // [set] pieces, then the list's state
  static constexpr int kPiecesBytes = (kPieces * (int)sizeof(Piece4) + (int)sizeof(List4) + 15) & ~15;
  static constexpr int kSmem = kOffPieces + kSets * kPiecesBytes;
  // int8: a set's first query is turned by the softmax warps, which have nothing else to do yet, later ones by the producer (64
  // rows of 4096 tokens, 64 heads: 36.0 us, without that 36.9; 4-bit chunks: 348 us, 335).
  static constexpr bool kSoftTurns = !kFour;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kTileBytes % 1024 == 0 || kFour, "swizzled rows");
  // Columns of a set: K 64, V^T 64 (two of them where they fit: V is then converted a tile ahead of its PV), S^T HN,
  // O^T HN.
  static constexpr int kVBufs = HN == 64 ? 1 : 2;
  static constexpr uint32_t kColV = 64, kColS = kColV + 64 * kVBufs, kColO = kColS + HN, kSetCols = kColO + HN;
  static_assert(kSets * kSetCols <= 512, "tensor memory columns");
  // Registers a thread: launched with 96 (five warps on a sub-partition: 15360 of 16384), then the control and
  // converting warpgroups give up what the softmax takes.  The host checks the launch count.
  static constexpr int kRegsLaunch = 96, kRegsCtl = HN == 64 ? 48 : 56, kRegsConv = HN == 64 ? 56 : 72, kRegsSoft = HN == 64 ? 160 : 136;
  static_assert(128 * kRegsCtl + 256 * kRegsConv + 256 * kRegsSoft <= kRegsLaunch * kThreads, "register split");
};

struct AttendArgs {
  Decode4Params p;
  CUtensorMap map[kMaxKvHeads];  // int8: each pool as rows of 128 bytes; a box is the code rows of a page
};

__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), CAI_W8(r, 0) : "memory");
}

// Sixteen int8 codes -> eight pairs of fp16, exact.
__device__ __forceinline__ void codes8(const uint4& w, uint32_t* r) {
  i8x4_to_f16x4(w.x, r[0], r[1]);
  i8x4_to_f16x4(w.y, r[2], r[3]);
  i8x4_to_f16x4(w.z, r[4], r[5]);
  i8x4_to_f16x4(w.w, r[6], r[7]);
}

// int8: the bound U of V's scales, as the bits of 2^-60 U, 2^-100 at a piece's start.
constexpr int kLeastScale = (127 - 100) << 23;
constexpr int kScaleRange = 60 << 23, kScaleRoom = 10 << 23;
constexpr float kSumUnit = 0x1p-12f;  // int8: sums are smaller by it: those of 2^24 weights over scales of 2^-100 stay below 2^128

__device__ __forceinline__ int piece_tiles(const Piece4& pc) {
  return pc.start < pc.end ? (pc.end - 1) / kT - pc.start / kT + 1 : 0;
}

template <bool kFour, int HN>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const __grid_constant__ AttendArgs args) {
  using S = Shape<kFour, HN>;
  constexpr int NS = S::kStages;
  constexpr bool kSoftTurns = S::kSoftTurns;
  const Decode4Params& p = args.p;
  extern __shared__ __align__(1024) uint8_t smem[];  // (aligned by hand, it would be addressed as generic memory)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // This warp's set: control warps in turn, then four warps of each kind.
  const int set = warp < kConv0 ? warp & 1 : (warp - kConv0) >> 2 & 1;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBars);
  uint64_t* raw_full = bars + set * S::kSetBars;  // [NS] producer -> converters (tx bytes)
  uint64_t* raw_empty = raw_full + NS;            // [NS] converters (4) -> producer
  uint64_t* k_full = raw_empty + NS;              // converters (4) -> issuer
  uint64_t* s_full = k_full + 1;                  // commit of S^T -> softmax, converters (K free)
  uint64_t* s_read = s_full + 1;                  // softmax (4) -> issuer: S^T free
  uint64_t* drain = s_read + 1;                   // the issuer's last commit
  uint64_t* v_full = drain + 1;                   // [2] converters (4) -> issuer
  uint64_t* p_full = v_full + 2;                  // [2] softmax (4) -> issuer
  uint64_t* pv_done = p_full + 2;                 // [2] commit of PV -> softmax (P^T free), converters (V^T free)
  uint64_t* q_full = pv_done + 2;                 // [2] producer -> issuer: a piece's Q^T
  uint64_t* q_raw = q_full + 2;                   // a query's bulk copy (tx bytes)
  uint64_t* q_room = q_raw + 1;                   // commit near a piece's end -> producer
  uint64_t* o_free = q_room + 1;                  // [2] softmax (4) -> issuer: a piece's O^T is read
  volatile int4* info = reinterpret_cast<volatile int4*>(smem + S::kOffInfo) + set * kInfo;  // tile: first and last + 1 key, groups landed
  volatile WaitState* wctl = reinterpret_cast<volatile WaitState*>(smem + S::kOffWait);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffSlot);
  float* xch = reinterpret_cast<float*>(smem + S::kOffX) + set * S::kXFloats;
  uint8_t* raw = smem + set * NS * S::kTileBytes;
  uint8_t* pt = smem + S::kOffP + set * S::kPBufs * S::kPBytes;
  uint8_t* qt = smem + S::kOffQ + set * S::kQBufs * S::kQBytes;
  Piece4* pieces = reinterpret_cast<Piece4*>(smem + S::kOffPieces + set * S::kPiecesBytes);
  List4& ls = *reinterpret_cast<List4*>(pieces + kPieces);

  // Blocks of one range but different head groups are neighbours: they read the same keys at the same time.
  const int G = p.num_heads / p.num_kv_heads;
  const int hgrp = blockIdx.x % p.head_groups, c0 = blockIdx.x / p.head_groups * kSets;  // the sets' ranges: c0, c0 + 1
  const int h0 = hgrp * HN, nh = min(G - h0, HN);  // this block's heads of the K/V head's group

  if (warp == 0) tmem_alloc(tmem_slot, 512);
  if (threadIdx.x < 32 * kSets && lane == 0) {  // warps 0 and 1: their sets'
    for (int s = 0; s < NS; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);
    }
    mbar_init(k_full, 4);
    mbar_init(s_full, 1);
    mbar_init(s_read, 4);
    mbar_init(drain, 1);
    mbar_init(q_raw, 1);
    mbar_init(q_room, 1);
    for (int k = 0; k < 2; ++k) {
      mbar_init(&v_full[k], 4);
      mbar_init(&p_full[k], 4);
      mbar_init(&pv_done[k], 1);
      mbar_init(&q_full[k], 1);
      mbar_init(&o_free[k], 4);
    }
    if (warp == 0) {
      wctl->abort = 0;
      wctl->limit_ns = p.wait_ns;
    }
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0) + set * S::kSetCols;
  grid_dependency_wait();
  grid_launch_dependents();
  start_lists<kThreads, kSets>(p, c0, reinterpret_cast<List4*>(smem + S::kOffPieces + kPieces * sizeof(Piece4)), S::kPiecesBytes,
                               reinterpret_cast<int64_t*>(smem + S::kOffScan));

  // Tiles (gt) and pieces with tiles (gp) of the set since the start; every role keeps its own count.
  int gt = 0, gp = 0;
  bool ok = true;  // no wait of this thread gave up
  int issued = 0;  // producer: tiles up to this one were started,
  int copies = 0;  // and copies of queries

  // A query's rows as they came -> Q^T, in the order of K's columns, by `step` threads.
  auto turn_query = [&](const uint8_t* src, uint8_t* dst, int first, int step) {
#pragma unroll 4
    for (int u = first; u < HN * 16; u += step) {
      if constexpr (kFour) {
        // Word t of 16-byte unit 4 j + i of a head holds channels 32 j + 8 t + 2 i, + 1.
        const int t = u & 3, j = u >> 5 & 3, h = (u >> 2 & 7) | (u >> 7 << 3);
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (h < nh) x = *reinterpret_cast<const uint4*>(src + h * 256 + 64 * j + 16 * t);
        uint32_t* y = reinterpret_cast<uint32_t*>(dst + (h >> 3) * 2048 + j * 512 + (h & 7) * 16 + t * 4);
        y[0] = bf16x2_to_f16x2(x.x);
        y[32] = bf16x2_to_f16x2(x.y);
        y[64] = bf16x2_to_f16x2(x.z);
        y[96] = bf16x2_to_f16x2(x.w);
      } else {
        // Eight channels a unit; eight lanes take a diagonal of heads and units (banks of both sides).
        const int h = (u & 7) | (u >> 7 << 3), c8 = ((u + (u >> 3)) & 7) | (u >> 3 & 8);
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (h < nh) x = *reinterpret_cast<const uint4*>(src + h * 256 + 16 * c8);
        *reinterpret_cast<uint4*>(dst + (h >> 3) * 2048 + c8 * 128 + (h & 7) * 16) =
            make_uint4(bf16x2_to_f16x2(x.x), bf16x2_to_f16x2(x.y), bf16x2_to_f16x2(x.z), bf16x2_to_f16x2(x.w));
      }
    }
  };

  // Every role goes through its set's lists of pieces; `work` is its part of one.  (The roles are the outermost branch:
  // the compiler gives each the registers that its setmaxnreg names.)  A wait that gave up, in either set, stops a set at
  // the end of a list: its warps agree there, by one barrier-reduction.
  auto lists = [&](auto&& work) {
    const uint32_t bar = 3 + set;
    bool more = ls.more != 0;  // (written before start_list's last barrier)
    while (more) {
      named_barrier_sync(bar, kSetThreads);
      if (warp == set) next_pieces(p, c0 + set, ls, pieces);
      named_barrier_sync(bar, kSetThreads);
      work(ls.count);
      more = ls.more != 0;
      if (bar_red_or(bar, kSetThreads, wctl->abort != 0)) break;
    }
  };

  if (warp < kConv0) {
    setmaxnreg_dec<S::kRegsCtl>();
    lists([&](int count) {
    if (warp < kSets) {
      // ------------------------------------------------------------------ producer
      // Lane l: page l of a tile.
      const int P = p.page_size, per = P / kBlk, in_tile = kT / P;
      // A piece's query as Q^T, in the order of K's columns.  One bulk copy brings its rows (by loads of one warp, which wait
      // 2000 cycles each beside the tiles' copies, 64 heads took 10 k cycles) to where the first tile's P^T will be, which
      // is not written before the S^T that needs this query.  That place and Q^T's buffer are free when the issuer says so
      // for the piece before, whose phase this warp has not passed: a parity names the last phase or the one before, so
      // the tiles' own barriers, of which several phases may pass between two pieces, would not do.
      auto ask_q = [&](const Piece4& pc) {
        if (gp > 0 && !mbar_wait_lean_warp(q_room, (gp - 1) & 1, wctl)) {
          ok = false;
          return;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(q_raw, (uint32_t)nh * kHeadDim * 2);
          bulk_g2s(pt + (S::kPBufs == 2 ? gt & 1 : 0) * S::kPBytes,
                   p.q + ((int64_t)pc.row * p.num_heads + (int64_t)pc.kvh * G + h0) * kHeadDim, (uint32_t)nh * kHeadDim * 2, q_raw);
        }
        __syncwarp();
        ++copies;
      };
      auto write_q = [&]() {
        if (kSoftTurns && gp == 0) return;
        if (!mbar_wait_lean_warp(q_raw, (copies - 1) & 1, wctl)) {
          ok = false;
          return;
        }
        turn_query(pt + (S::kPBufs == 2 ? gt & 1 : 0) * S::kPBytes, qt + (S::kQBufs == 2 ? gp & 1 : 0) * S::kQBytes, lane, 32);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[gp & 1]);
      };
      for (int pi = 0; pi < count && ok; ++pi) {
        const Piece4 pc = pieces[pi];
        const int nt = piece_tiles(pc);
        if (nt == 0) continue;
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
        int32_t id_next = load_id(0);
        // The first query is asked for first, later ones behind the copies of the tiles that have stages, two ahead of the
        // products.
        const int at_q = min(gp == 0 ? NS - 1 : NS - 2, nt - 1);
        if (gp == 0) ask_q(pc);
        for (int t = 0; t < nt; ++t) {
          const int x = gt + t, s = x % NS;
          const int32_t id = id_next;
          id_next = load_id(t + 1);
          if (x >= NS && !mbar_wait_lean_warp(&raw_empty[s], (x / NS - 1) & 1, wctl)) {
            ok = false;
            break;
          }
          int lo, hi;
          groups(t, lo, hi);
          const bool live = lo < hi, in_range = (uint32_t)id < (uint32_t)num_pages;
          if (live && !in_range && p.err) atomicOr(p.err, CAI_DEVERR_PAGE);
          // Groups that land: 4-bit, those that are needed; int8, a page's all.
          const uint32_t mine = kFour ? ((1u << hi) - 1) & ~((1u << lo) - 1) : ((1u << per) - 1) << (lane * per);
          const uint32_t okm = __reduce_or_sync(0xffffffffu, live && in_range ? mine : 0u);
          issued = x + 1;
          if (x != p.drop_stage) {  // (fault injection: never issued)
            if (lane == 0) {
              volatile int4* y = info + x % kInfo;
              const int base = (pc.start / kT + t) * kT;
              y->x = pc.start - base;
              y->y = pc.end - base;
              y->z = (int)okm;
              mbar_arrive_expect_tx(&raw_full[s], kFour ? (uint32_t)__popc(okm) * kBlkBytes : (uint32_t)(__popc(okm) / per) * page_bytes(P));
            }
            __syncwarp();
            if (live && in_range) {
              uint8_t* stage = raw + s * S::kTileBytes;
              if constexpr (kFour) {
                bulk_g2s(stage + lo * kBlkBytes, pages + ((int64_t)id * per + (lo - lane * per)) * kBlkBytes,
                         (uint32_t)(hi - lo) * kBlkBytes, &raw_full[s]);
              } else {
                tma_load_2d(stage + lane * (2 * P * kHeadDim), &args.map[pc.kvh], 0, id * (page_bytes(P) / 128), &raw_full[s]);
                bulk_g2s(stage + kCodeBytes8 + lane * (8 * P), pages + (int64_t)id * page_bytes(P) + 2 * P * kHeadDim, 8 * P, &raw_full[s]);
              }
            }
          }
          if (t == at_q) {
            if (gp > 0) ask_q(pc);
            if (ok) write_q();
            if (!ok) break;
          }
        }
        gt += nt;
        ++gp;
      }
    } else {
      // ------------------------------------------------------------------ issuer
      // S^T of the next tile goes out before PV of this one, so that its softmax need not wait.
      const uint64_t dq = smem_desc(smem_addr(qt), 128, 2048);
      const uint64_t dp = smem_desc(smem_addr(pt), 128, kT * 16);
      constexpr uint32_t idesc_s = idesc_f16_f32(kT, HN, 0, 0), idesc_o = idesc_f16_f32(kHeadDim, HN, 0, 1);
      auto issue_s = [&](int n, bool first) {
        ok = (!first || mbar_wait_lean_warp(&q_full[gp & 1], (gp >> 1) & 1, wctl)) && mbar_wait_lean_warp(k_full, n & 1, wctl) &&
             (n == 0 || mbar_wait_lean_warp(s_read, (n - 1) & 1, wctl));
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kHeadDim / 16; ++k)
            mma_f16_ts(tmem + S::kColS, tmem + k * 8, dq + (uint64_t)((S::kQBufs == 2 ? gp & 1 : 0) * (S::kQBytes >> 4) + k * 16), idesc_s,
                       k > 0 ? 1u : 0u);
          mma_commit(s_full);
        }
        __syncwarp();
      };
      auto say_room = [&]() {
        if (elect_one()) mma_commit(q_room);
        __syncwarp();
      };
      auto issue_pv = [&](int n, bool first) {
        const int k2 = n & 1;
        // (the piece's first PV starts the accumulator, once the last piece's has been read)
        ok = mbar_wait_lean_warp(&v_full[k2], (n >> 1) & 1, wctl) && mbar_wait_lean_warp(&p_full[k2], (n >> 1) & 1, wctl) &&
             (!first || gp == 0 || mbar_wait_lean_warp(&o_free[(gp - 1) & 1], ((gp - 1) >> 1) & 1, wctl));
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kT / 16; ++k)
            mma_f16_ts(tmem + S::kColO, tmem + S::kColV + (S::kVBufs == 2 ? k2 * 64 : 0) + k * 8,
                       dp + (uint64_t)((S::kPBufs == 2 ? k2 : 0) * (S::kPBytes >> 4) + k * 16), idesc_o, (!first || k > 0) ? 1u : 0u);
          mma_commit(&pv_done[k2]);
        }
        __syncwarp();
      };
      for (int pi = 0; pi < count && ok; ++pi) {
        const int nt = piece_tiles(pieces[pi]);
        if (nt == 0) continue;
        issue_s(gt, true);
        for (int t = 0; t < nt && ok; ++t) {
          if (t + 1 < nt) issue_s(gt + t + 1, false);
          // Once the products so far are done the next piece's query may come: all S^T of this piece are among them, and
          // every PV but the last, or (one P^T buffer) that, too.
          if (S::kPBufs == 2 && t == nt - 1 && ok) say_room();
          if (ok) issue_pv(gt + t, t == 0);
          if (S::kPBufs == 1 && t == nt - 1 && ok) say_room();
        }
        gt += nt;
        ++gp;
      }
    }
    });
  } else if (warp < kSoft0) {
    setmaxnreg_dec<S::kRegsConv>();
    lists([&](int count) {
      // ------------------------------------------------------------------ converters
      // K of the next tile goes before V of this one where V has one buffer and a third raw tile is on its way: V may have to
      // wait for the products that its softmax comes before.  The waits are tried a step ahead (a wait costs 150 cycles and more even when its phase is
      // over), and a step's stores are waited for after the next one's loads.
      // A lane whose wait gave up carries on (on garbage) and releases nothing that it did not see land; the
      // lanes agree on stopping after each tile.
      const int quarter = warp & 3;
      const uint32_t tm = tmem + ((uint32_t)(quarter * 32) << 16);
      const int g = lane >> 2, t4 = lane & 3;  // (4-bit)
      // (int8) this thread's key (K) and channel (V): its 128-byte row of K in a stage, the row and first chunk of its
      // channel in a page's V, and its scales.
      const int P = p.page_size, lg = P == 16 ? 4 : P == 32 ? 5 : 6, row = quarter * 32 + lane;
      const uint32_t k_at = (uint32_t)((row >> lg) * 2 * P + (row & (P - 1))) * 128, k_x = row & 7;
      const uint32_t v_at = (uint32_t)(P + (row << lg >> 7)) * 128, v_c = (row << lg & 127) >> 4, v_x = (row << lg >> 7) & 7;
      const uint32_t s_at = kCodeBytes8 + ((row >> lg) * 2 * P + (row & (P - 1))) * 4;
      float2* tok = reinterpret_cast<float2*>(smem + S::kOffTok) + set * 2 * kT;  // (a tile's is read before the S^T after the next goes out)
      int total = 0;
      for (int pi = 0; pi < count; ++pi) total += piece_tiles(pieces[pi]);
      const int end = gt + total;
      bool landed = false, raw_there = false;
      constexpr int kB = S::kVBufs;  // V^T's buffer was read by PV of tile n - kB
      // (n: the tile whose V is converted, n + kAhead: K.  Loops are kept rolled: the roles' instructions together pass the
      // cache's size soon, unrolled twice as far this cost 20%.)
      constexpr int kAhead = kB == 1 && NS > 2 ? 1 : 0;
      for (int n = gt - kAhead; n < end; ++n) {
        const int nk = n + kAhead;
        const bool has_k = nk < end, has_v = n >= gt;
        bool landed_next = false;
        if (has_k) {
          // ---- K, free once S^T of the last tile is done.
          const int s = nk % NS;
          const bool k_there = nk < 1 || mbar_test_wait(s_full, (nk - 1) & 1);
          landed_next = raw_there || mbar_wait_lean(&raw_full[s], (nk / NS) & 1, wctl);
          ok = ok && landed_next;
          if (!k_there) ok = mbar_wait_lean(s_full, (nk - 1) & 1, wctl) && ok;
          __syncwarp();
          tc_fence_after();
          const uint8_t* stage = raw + s * S::kTileBytes;
          if constexpr (kFour) {
            // Two 16-key groups, column 16 j + 4 i + t: channels 32 j + 8 t + 2 i, + 1.
            const uint8_t* blk = stage + 2 * quarter * kBlkBytes;
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
          } else {
            // This thread's key, column k: channels 2 k, 2 k + 1.
            const float* sc = reinterpret_cast<const float*>(stage + s_at);
            tok[(nk & 1) * kT + row] = make_float2(sc[0] * p.scale_log2, sc[P]);
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              uint32_t r[16];
#pragma unroll
              for (int e = 0; e < 2; ++e)
                codes8(*reinterpret_cast<const uint4*>(stage + k_at + (((2 * i + e) ^ k_x) << 4)), r + 8 * e);
              tmem_st_32x32b_x16(tm + i * 16, r);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(k_full);
        }
        if (has_v) {
          // ---- V of this quarter's 32 channels, column k: keys 2 k, 2 k + 1
          const int s = n % NS;
          const bool v_there = n < kB || mbar_test_wait(&pv_done[(n - kB) & 1], ((n - kB) >> 1) & 1);
          if (!v_there) ok = mbar_wait_lean(&pv_done[(n - kB) & 1], ((n - kB) >> 1) & 1, wctl) && ok;
          __syncwarp();
          tc_fence_after();
          const uint32_t col = S::kColV + (kB == 2 ? (n & 1) * 64 : 0);
          if constexpr (kFour) {
            const int lo = info[n % kInfo].x, hi = info[n % kInfo].y, okm = info[n % kInfo].z;
            const bool edge = lo > 0 || hi < kT || okm != 255;
            const uint8_t* blk = raw + s * S::kTileBytes;
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
                tmem_st_16x128b_x8(tm + ((uint32_t)(16 * m) << 16) + col + kh * 32, r);
              }
            }
          } else {
            // (codes are numbers whatever the slots hold: a masked key's weight of 0 is enough)
            const uint8_t* stage = raw + s * S::kTileBytes + v_at;
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              uint32_t r[16];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int t0 = 16 * (2 * i + e);  // 16 keys of one page
                codes8(*reinterpret_cast<const uint4*>(stage + (t0 >> lg) * (2 * P * kHeadDim) + (((v_c + ((t0 & (P - 1)) >> 4)) ^ v_x) << 4)),
                       r + 8 * e);
              }
              tmem_st_32x32b_x16(tm + col + i * 16, r);
            }
          }
          raw_there = nk + 1 < end && mbar_test_wait(&raw_full[(nk + 1) % NS], ((nk + 1) / NS) & 1);
          tmem_wait_st();
          tc_fence_before();
          ok = __all_sync(0xffffffffu, ok);
          if (lane == 0) {
            if (kAhead ? landed : landed_next) mbar_arrive(&raw_empty[s]);
            mbar_arrive(&v_full[n & 1]);
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
      // ------------------------------------------------------------------ softmax, epilogue
      // A thread whose wait gave up carries on with the same steps (on garbage) until the set's next barrier-reduction,
      // which stops its four warps.
      const int quarter = warp & 3;
      const uint32_t tm = tmem + ((uint32_t)(quarter * 32) << 16);
      const uint32_t bar = 1 + set;
      const int key = quarter * 32 + lane;         // this thread's key of a tile (and channel of O^T)
      float* wmax = xch;                           // [quarter][HN] maxima of a raise
      float* part = xch + S::kXSum + quarter * HN; // sums of a piece
      float* nref = xch + S::kXRef + quarter * HN; // negated references (log2 units)
      float* fac = xch + S::kXFac + quarter * HN;  // factors of a raise
      const float2* tok = reinterpret_cast<const float2*>(smem + S::kOffTok) + set * 2 * kT + key;
      int* tops = reinterpret_cast<int*>(smem + S::kOffTop) + set * 4;

      for (int pi = 0; pi < count; ++pi) {
        const int nt = piece_tiles(pieces[pi]);
        // The block's first head row.  (Read from the list where it is wanted: kept through the tiles it makes registers spill.)
        auto first_row = [&]() { return (int64_t)pieces[pi].row * p.num_heads + (int64_t)pieces[pi].kvh * G + h0; };
        if (nt == 0) {  // nothing to attend, or an invalid length (flagged): out = 0, lse = -inf
          const int64_t row0 = first_row();
          for (int i = key; i < nh * kHeadDim / 4; i += kT)
            reinterpret_cast<uint2*>(p.out + row0 * kHeadDim)[i] = make_uint2(0u, 0u);
          if (p.lse_out && key < nh) p.lse_out[row0 + key] = -INFINITY;
          continue;
        }
        if (kSoftTurns && gp == 0) {
          ok = mbar_wait_lean(q_raw, 0, wctl) && ok;
          __syncwarp();
          turn_query(pt, qt, key, 128);
          fence_proxy_async_smem();
          named_barrier_sync(bar, 128);
          if (key == 0) mbar_arrive(&q_full[0]);
        }
        if (lane < HN / 4) reinterpret_cast<float4*>(nref)[lane] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        __syncwarp();
        uint64_t l[HN / 2];     // this key's sums, per head pair
#pragma unroll
        for (int h = 0; h < HN / 2; ++h) l[h] = 0ull;
        bool have_ref = false;  // some key was attended (the same in the whole set)
        int least = kLeastScale;  // int8: what V's scales count as at least (the same in the whole set)
        for (int t = 0; t < nt; ++t) {
          const int n = gt + t;
          ok = mbar_wait_lean(s_full, n & 1, wctl) && ok;
          __syncwarp();
          tc_fence_after();
          const int lo = info[n % kInfo].x, hi = info[n % kInfo].y, okm = info[n % kInfo].z;
          const bool edge = lo > 0 || hi < kT || okm != 255;
          const bool valid = key >= lo && key < hi && ((okm >> (key / kBlk)) & 1);
          // int8: K's scale; V's as a power of two, and its inverse for the sums (what is not there may be anything).
          uint64_t ks2, lv2 = 0ull, iv2 = 0ull;
          if constexpr (kFour) {
            ks2 = f2(p.scale_log2, p.scale_log2);
          } else {
            const float2 sc = tok[(n & 1) * kT];
            const float v = fmaxf(sc.y, __int_as_float(least));
            const bool above = __float_as_int(v) - least > kScaleRange;  // (U has to be raised, and the references with it)
            const float ks = valid ? sc.x : 0.0f, lv = !valid ? 0.0f : above ? INFINITY : __log2f(v), iv = ex2_approx(-lv) * kSumUnit;
            ks2 = f2(ks, ks);
            lv2 = f2(lv, lv);
            iv2 = f2(iv, iv);
          }
          // Logits minus references of N heads, from S^T's columns r (S^T stays in tensor memory until the set says it is read).
          auto logits = [&](auto& r, int h1, float* z) {
            constexpr int N = sizeof(r) / 4;
#pragma unroll
            for (int h = 0; h < N; h += 4) {
              const float4 x4 = *reinterpret_cast<const float4*>(nref + h1 + h);
              uint64_t a = f2_fma(f2(__uint_as_float(r[h]), __uint_as_float(r[h + 1])), ks2, f2(x4.x, x4.y));
              uint64_t b = f2_fma(f2(__uint_as_float(r[h + 2]), __uint_as_float(r[h + 3])), ks2, f2(x4.z, x4.w));
              if constexpr (!kFour) {
                a = f2_add(a, lv2);
                b = f2_add(b, lv2);
              }
              f2_split(a, z[h], z[h + 1]);
              f2_split(b, z[h + 2], z[h + 3]);
            }
            if (edge) {
#pragma unroll
              for (int h = 0; h < N; ++h) z[h] = valid ? z[h] : -INFINITY;
            }
          };
          float sv[HN];
          // P^T's row of this key: heads 8 i .. 8 i + 7 at i * 2048 + key * 16.
          uint8_t* dst = pt + (S::kPBufs == 2 ? n & 1 : 0) * S::kPBytes + key * 16;
          bool raise = !have_ref, stop = false;
          while (true) {  // (one copy of the code: instruction cache)
            const bool raised = raise;
            if (raise) {
              if constexpr (!kFour) {
                const float x = valid ? tok[(n & 1) * kT].y : 0.0f;
                const int most = __reduce_max_sync(0xffffffffu, __float_as_int(fmaxf(x, 0.0f)));
                if (lane == 0) tops[quarter] = most;
                named_barrier_sync(bar, 128);
                const int4 t4 = *reinterpret_cast<const int4*>(tops);
                const int top = max(max(t4.x, t4.y), max(t4.z, t4.w));
                if (top - least > kScaleRange) least = top - (kScaleRange - kScaleRoom);
                const float lv = valid ? __log2f(fmaxf(x, __int_as_float(least))) : 0.0f, iv = ex2_approx(-lv) * kSumUnit;
                lv2 = f2(lv, lv);
                iv2 = f2(iv, iv);
              }
              // Raise the references that a weight passes by 2^15 (all of them at the first tile with a key).
#pragma unroll 1
              for (int h1 = 0; h1 < HN; h1 += 16) {
                float z[16], mine = -INFINITY;
                uint32_t r[16];
                tmem_ld_32x32b_x16(tm + S::kColS + h1, r);
                tmem_wait_ld();
                logits(r, h1, z);
#pragma unroll
                for (int h = 0; h < 16; ++h) {
                  float m;
                  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(z[h]));
                  mine = lane == h ? m : mine;
                }
                if (lane < 16) wmax[quarter * HN + h1 + lane] = mine;
              }
              if (bar_red_or(bar, 128, !ok)) {
                stop = true;  // (all four warps are here)
                break;
              }
              const bool any = okm != 0;  // some key of the tile is attended
#pragma unroll 1
              for (int h = lane; h < HN; h += 32) {
                const float* w = wmax + h;
                const float v = fmaxf(fmaxf(w[0], w[HN]), fmaxf(w[2 * HN], w[3 * HN]));
                const float up = any && (!have_ref || v > kRaise) ? v - kWeightLift : 0.0f;
                nref[h] -= up;
                // (int8: the sums so far, over scales of 2^-100, count after a raise by more than 126, too: by its third, three
                // times)
                fac[h] = ex2_approx(kFour ? -up : up * (-1.0f / 3.0f));
              }
              __syncwarp();
              if (have_ref) {
                // O^T holds earlier tiles of the piece: the last PV must be done before it is rescaled.
                ok = mbar_wait_lean(&pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, wctl) && ok;
                __syncwarp();
                tc_fence_after();
#pragma unroll 1
                for (int h1 = 0; h1 < HN; h1 += 8) {
                  const float4 fa = *reinterpret_cast<const float4*>(fac + h1), fb = *reinterpret_cast<const float4*>(fac + h1 + 4);
                  const float f[8] = {fa.x, fa.y, fa.z, fa.w, fb.x, fb.y, fb.z, fb.w};
                  uint32_t r[8];
                  tmem_ld_32x32b_x8(tm + S::kColO + h1, r);
                  tmem_wait_ld();
#pragma unroll
                  for (int e = 0; e < 8; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * (kFour ? f[e] : f[e] * f[e] * f[e]));
                  tmem_st_32x32b_x8(tm + S::kColO + h1, r);
                }
#pragma unroll 1
                for (int times = kFour ? 1 : 3; times > 0; --times) {
#pragma unroll
                  for (int h = 0; h < HN; h += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(fac + h);
                    l[h / 2] = f2_mul(l[h / 2], f2(f.x, f.y));
                    l[h / 2 + 1] = f2_mul(l[h / 2 + 1], f2(f.z, f.w));
                  }
                }
                tmem_wait_st();
              }
              have_ref = have_ref || any;
            }
            float mx = -INFINITY;
            {
              constexpr int N = HN < 32 ? HN : 32;
              uint32_t r[HN / N][N];
#pragma unroll
              for (int i = 0; i < HN / N; ++i) {
                if constexpr (N == 32) tmem_ld_32x32b_x32(tm + S::kColS + i * N, r[i]);
                else tmem_ld_32x32b_x16(tm + S::kColS + i * N, r[i]);
              }
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < HN / N; ++i) logits(r[i], i * N, sv + i * N);
            }
#pragma unroll
            for (int h = 0; h < HN; h += 2) mx = fmax3(mx, sv[h], sv[h + 1]);
            if (!raised) {
              raise = bar_red_or(bar, 128, !ok || mx > kRaise);
              if (raise) continue;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_read);  // the next S^T may come while these become weights
            // P^T's buffer is free once PV of tile n - kPBufs is done.
            constexpr int kB = S::kPBufs;
            if (n >= kB) ok = mbar_wait_lean(&pv_done[(n - kB) & 1], ((n - kB) >> 1) & 1, wctl) && ok;
            __syncwarp();
            // The weights, in place of the logits.
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
            break;
          }
          if (stop) {
            ok = false;
            break;
          }
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[n & 1]);
#pragma unroll
          for (int h = 0; h < HN; h += 2)
            l[h / 2] = kFour ? f2_add(l[h / 2], f2(sv[h], sv[h + 1])) : f2_fma(f2(sv[h], sv[h + 1]), iv2, l[h / 2]);
        }
        gt += nt;

        // ---- end of piece: sums over the keys, 16 heads at a time
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
          if (lane < 16) part[h1 + lane] = v[0];
        }
        if (bar_red_or(bar, 128, !ok)) {
          ok = false;
          break;
        }
        // The piece's last PV, then its heads over their sums (lane h: heads h and h + 32).
        ok = mbar_wait_lean(&pv_done[(gt - 1) & 1], ((gt - 1) >> 1) & 1, wctl) && ok;
        __syncwarp();
        tc_fence_after();
        const int slot = pieces[pi].slot;
        const int64_t row0 = first_row(), slot0 = (int64_t)slot * G + h0;
#pragma unroll 1
        for (int h = lane; h < HN; h += 32) {
          const float* y = xch + S::kXSum + h;
          const float sum = (y[0] + y[HN]) + (y[2 * HN] + y[3 * HN]);
          fac[h] = have_ref && sum > 0.0f ? 1.0f / sum : 0.0f;
          if (quarter == 0 && h < nh) {
            const float lse2 = have_ref && sum > 0.0f ? log2f(sum) + (kFour ? 0.0f : 12.0f) - nref[h] : -INFINITY;
            if (slot >= 0) p.ws_lse[slot0 + h] = lse2;
            else if (p.lse_out) p.lse_out[row0 + h] = lse2 * kLn2;
          }
        }
        __syncwarp();
        uint16_t* out = slot < 0 ? p.out + row0 * kHeadDim + key : nullptr;
        float* ws = p.ws_o + slot0 * kHeadDim + key;
#pragma unroll 1
        for (int h1 = 0; h1 < nh; h1 += 16) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(tm + S::kColO + h1, r);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < 16; h += 4) {
            const float4 f4 = *reinterpret_cast<const float4*>(fac + h1 + h);
            const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = f[e] != 0.0f ? __uint_as_float(r[h + e]) * (kFour ? 1.0f : kSumUnit) * f[e] : 0.0f;  // (nothing attended: whatever is there does not count)
              if (h1 + h + e < nh) {
                if (out) out[(h1 + h + e) * kHeadDim] = (uint16_t)pack_bf16x2(x, 0.0f);
                else ws[(h1 + h + e) * kHeadDim] = x;
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[gp & 1]);
        // (the next piece's references and sums: every reader of this one's sums has come to its first raise's barrier
        // before they are written)
        ++gp;
      }
    });
  }

  // What this block started has ended before it goes away: the producer's copies, the issuer's products.
  if (warp < kSets) {
    for (int x = max(0, issued - NS); x < issued; ++x)
      if (x != p.drop_stage) mbar_wait_drain(&raw_full[x % NS], (x / NS) & 1);
    if (copies > 0) mbar_wait_drain(q_raw, (copies - 1) & 1);
  } else if (warp < kConv0) {
    if (elect_one()) mma_commit(drain);
    __syncwarp();
    mbar_wait_drain(drain, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && wctl->abort && p.err) atomicOr(p.err, CAI_DEVERR_TIMEOUT);
  if (warp == 0) tmem_dealloc(tmem, 512);  // (set 0's is the first column)
}

// The pieces' normalised outputs merged by their log2-sum-exp: as combine4_kernel (at most one row and K/V head starts in a
// range and goes on into the next, so there is an item per range), for the few pieces that a list has: a warp takes two
// heads and all of their pieces, a block 16 heads.  (With its four warps a head and two heads a block 64 heads took 15 us
// here, most of it the start of 9728 blocks.)
constexpr int kMergeWarps = 8, kMergeHeads = 2;
__global__ void __launch_bounds__(32 * kMergeWarps) merge_kernel(const __grid_constant__ Decode4Params p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = p.num_heads / p.num_kv_heads, groups = (G + kMergeWarps * kMergeHeads - 1) / (kMergeWarps * kMergeHeads);
  const int item = blockIdx.x / groups, h0 = ((blockIdx.x - item * groups) * kMergeWarps + warp) * kMergeHeads;
  grid_dependency_wait();
  grid_launch_dependents();
  int unit = item, n = 0;
  if (p.chunk == 0) {
    const int2 m = p.meta[item];  // the unit, and the last range with a piece of it
    if (m.x < 0) return;
    unit = m.x;
    n = m.y - item + 1;
  }
  const int b = unit / p.num_kv_heads, kvh = unit - b * p.num_kv_heads;
  int32_t row;
  SeqSplits sp;
  if (!seq_keys(p, b, row, sp)) return;
  if (p.chunk > 0) n = sp.nsplit;
  if (n <= 1 || h0 >= G) return;  // written by the attention kernel
  auto slot = [&](int j) -> int64_t {
    return (p.chunk > 0 ? (int64_t)unit * p.splits + j : 2ll * (item + j) + (j == 0 ? 1 : 0)) * G + h0;
  };
  float M[kMergeHeads], sum[kMergeHeads];
  float4 acc[kMergeHeads];
#pragma unroll
  for (int k = 0; k < kMergeHeads; ++k) M[k] = -INFINITY, sum[k] = 0.0f, acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < n; j0 += 4) {
    float4 x[4][kMergeHeads];
    float l[4][kMergeHeads];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t at = j0 + u < n ? slot(j0 + u) : 0;
#pragma unroll
      for (int k = 0; k < kMergeHeads; ++k) {
        const bool have = j0 + u < n && h0 + k < G;
        l[u][k] = have ? p.ws_lse[at + k] : -INFINITY;
        x[u][k] = have ? reinterpret_cast<const float4*>(p.ws_o + (at + k) * kHeadDim)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
#pragma unroll
    for (int k = 0; k < kMergeHeads; ++k) {
      const float m = fmaxf(fmaxf(fmaxf(l[0][k], l[1][k]), fmaxf(l[2][k], l[3][k])), M[k]);
      if (m == -INFINITY) continue;
      const float f = ex2_approx(M[k] - m);
      M[k] = m;
      sum[k] *= f;
      acc[k] = make_float4(acc[k].x * f, acc[k].y * f, acc[k].z * f, acc[k].w * f);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float w = ex2_approx(l[u][k] - m);
        sum[k] += w;
        acc[k].x = fmaf(w, x[u][k].x, acc[k].x);
        acc[k].y = fmaf(w, x[u][k].y, acc[k].y);
        acc[k].z = fmaf(w, x[u][k].z, acc[k].z);
        acc[k].w = fmaf(w, x[u][k].w, acc[k].w);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kMergeHeads; ++k) {
    if (h0 + k >= G) break;
    const float inv = sum[k] > 0.0f ? 1.0f / sum[k] : 0.0f;
    const int64_t at = (int64_t)row * p.num_heads + kvh * G + h0 + k;
    reinterpret_cast<uint2*>(p.out + at * kHeadDim)[lane] =
        make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv), pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
    if (p.lse_out && lane == 0) p.lse_out[at] = sum[k] > 0.0f ? (M[k] + log2f(sum[k])) * kLn2 : -INFINITY;
  }
}

template <bool kFour, int HN>
cudaError_t launch_hn(const Decode4Params& p, cudaStream_t stream) {
  using S = Shape<kFour, HN>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_set[dev]) {
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, attend_kernel<kFour, HN>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != S::kRegsLaunch) return cudaErrorInvalidDeviceFunction;
    e = cudaFuncSetAttribute(attend_kernel<kFour, HN>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set[dev] = true;
  }
  AttendArgs a = {};
  a.p = p;
  for (int j = 0; !kFour && j < p.num_kv_heads; ++j)
    if (!encode_pool_map(&a.map[j], p.pages[j], p.num_pages[j], p.page_size)) return cudaErrorInvalidValue;
  const int blocks = p.head_groups * ((p.ranges + kSets - 1) / kSets);
  return launch_pdl(attend_kernel<kFour, HN>, dim3((unsigned)blocks), dim3(kThreads), S::kSmem, stream, a);
}

template <bool kFour>
cudaError_t launch_heads(const Decode4Params& p, cudaStream_t stream) {
  const int G = p.num_heads / p.num_kv_heads;
  return G <= 16 ? launch_hn<kFour, 16>(p, stream) : G <= 32 ? launch_hn<kFour, 32>(p, stream) : launch_hn<kFour, 64>(p, stream);
}

}  // namespace

cudaError_t launch_attend(const Decode4Params& p, cudaStream_t stream) {
  return p.eight ? launch_heads<false>(p, stream) : launch_heads<true>(p, stream);
}

cudaError_t launch_merge(const Decode4Params& p, cudaStream_t stream) {
  const int G = p.num_heads / p.num_kv_heads, groups = (G + kMergeWarps * kMergeHeads - 1) / (kMergeWarps * kMergeHeads);
  const int64_t items = p.chunk == 0 ? p.ranges : (int64_t)p.batch * p.num_kv_heads;
  return launch_pdl(merge_kernel, dim3((unsigned)(items * groups)), dim3(32 * kMergeWarps), 0, stream, p);
}

}  // namespace cai

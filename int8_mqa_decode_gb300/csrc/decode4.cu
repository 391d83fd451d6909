// Decode attention over the 4-bit paged cache (layout in kv4.cuh), grouped query heads, and the
// log-sum-exp merge of its splits.
//
// What it computes: for one query token per sequence and every query head, softmax over the attended
// positions of softmax_scale * <q, k> and the weighted sum of v, k and v being the values that the
// 4-bit codes stand for; query heads [j G, (j + 1) G) read K/V head j.
//
// How.  A block takes one (sequence, K/V head, group of up to 32 query heads, key range); its four
// warps take steps of 32 keys in turn, each with a ring of its own that its lane 0 fills by bulk
// copies, so no warp waits for another before the end.  Scores are computed transposed, S^T = K Q^T
// with mma.m16n8k16 (16 keys x 8 heads): the codes become the A operand in registers (two bit
// operations and one fused multiply-add per pair, exact), query heads fill the N side in units of 8,
// so a group of 4 or 8 heads wastes little.  A column of S^T is one head: the running maximum is a
// reference per head, raised only when a logit passes it by 2^8, so the common step has no reduction
// across lanes.  P^T goes to the B operand by an 8 x 8 transpose in registers, and O^T += V^T P^T
// accumulates 128 channels x heads in registers.  At the end the warps' parts are merged through the
// ring's shared memory.
//
// Why this tensor path: one decode step of G <= 16 heads is bound by HBM, and a key costs each
// sub-partition G / 8 * 16 m16n8k16 at 8 cycles per 16 keys (512 cycles at 32 heads, against 392
// that the keys' 144 bytes take at the copy bandwidth).  Going through tensor memory instead costs
// two 128-row operand writes, two reads and four hand-offs between warps per 128 keys, and 16 MMA
// issues of about 70 cycles whatever the head count.
#include <cmath>

#include "common.cuh"
#include "kv4.cuh"
#include "ptx.cuh"

namespace cai {
namespace {

constexpr int kWarps = 4;
constexpr int kStep = 32;                             // keys of one step of one warp
constexpr int kStepBytes = kStep / kBlk * kBlkBytes;  // 4608
constexpr int kORow = kHeadDim + 4;                   // floats of a head's row in the merge buffer (bank spread)
constexpr float kRaise4 = 8.0f;                       // log2 units a logit may exceed its reference by

// One piece of work: keys [start, end) of one sequence and K/V head (end = start: nothing to attend).
struct Piece4 {
  int32_t b, kvh, row;  // row: of q, out and lse_out
  int32_t start, end;
  int32_t slot;         // partial's slot, or -1: the piece is the whole attended range
};
constexpr int kPieces = 32;  // pieces listed at a time
// State of the list, in shared memory.
struct List4 {
  int32_t count, more;
  int32_t unit;           // next (sequence, K/V head) to list (or item, with fixed chunks)
  int64_t pos;            // its first position in the numbering of all tiles
  int64_t begin, end, total;  // this block's range of it, and its length
  int32_t ranges;         // blocks that share it: at most one per position
};

// Blocks per SM and stages per warp: about 220 KB in flight on an SM at every head count.
template <int NT>
struct Shape4 {
  static constexpr int kBlocks = NT == 1 ? 4 : NT == 2 ? 3 : 2;
  static constexpr int kStages = NT == 1 ? 3 : NT == 2 ? 4 : 5;
  static constexpr int kHeads = 8 * NT;
  static constexpr bool kQRegs = NT <= 2;       // the query's B operand in registers
  static constexpr bool kGroupSums = NT == 1;   // K scales applied to the scores of a channel group, not to K
  static constexpr int kRing = kWarps * kStages * kStepBytes;
  static constexpr int kMerge = kWarps * kHeads * kORow * 4;  // in the ring, drained by then
  static constexpr int kOffQ = kRing > kMerge ? kRing : kMerge;
  static constexpr int kOffBars = kOffQ + (kQRegs ? 0 : kHeads * kHeadDim * 2);
  static constexpr int kOffOk = kOffBars + kWarps * kStages * 8;
  static constexpr int kOffMl = kOffOk + kWarps * kStages * 4;  // [kWarps][kHeads] references, then sums
  static constexpr int kOffWait = (kOffMl + 2 * kWarps * kHeads * 4 + 15) & ~15;
  static constexpr int kOffPieces = kOffWait + 16;
  static constexpr int kSmem = kOffPieces + kPieces * (int)sizeof(Piece4) + 64;  // and the list's state
  static_assert(kBlocks * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t x) {
  return pack_f16x2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

__device__ __forceinline__ float half_of(uint32_t x, int hi) {
  return __half2float(__ushort_as_half((unsigned short)(hi ? x >> 16 : x)));
}

__device__ __forceinline__ uint2 pack_bf16x4(float a, float b, float c, float d) {
  return make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

// Sequence b's row in q / out / lse_out and its attended keys; false: not a row of this launch.
__device__ __forceinline__ bool seq_keys(const Decode4Params& p, int b, int32_t& row, SeqSplits& sp) {
  int32_t L = p.ctx_len[b];
  row = b;
  if (p.q_off) {
    const int32_t a = p.q_off[b], e = p.q_off[b + 1];
    if (!(a >= 0 && e == a + 1 && e <= p.total_rows)) return false;  // a chunk: the prefill kernel's
    row = a;
    L = L < 0 || L >= p.max_pages * p.page_size ? -1 : L + 1;        // the length before the new token was given
  }
  sp = seq_splits(L, p.window, p.max_pages * p.page_size, p.chunk > 0 ? p.chunk : 1);
  return true;
}

// Tiles of 128 keys that hold sequence b's attended keys (-1: not a row of this launch).  A tile is
// aligned to 128 positions of the sequence.
__device__ __forceinline__ int seq_tiles(const Decode4Params& p, int b) {
  int32_t row;
  SeqSplits sp;
  if (!seq_keys(p, b, row, sp)) return -1;
  return sp.hi > sp.lo ? (sp.hi - 1) / kDecodeTile - sp.lo / kDecodeTile + 1 : 0;
}

// Positions that a (sequence, K/V head) takes in the numbering that is cut into equal parts: its tiles,
// and one more for its start and merge (which cost about as much as a tile).
__device__ __forceinline__ int unit_weight(int tiles) { return tiles < 0 ? 0 : tiles + 1; }

// Block c's range is [c W / n, (c + 1) W / n), n <= W; the block whose range holds position x:
__device__ __forceinline__ int block_of(int64_t x, int64_t W, int n) { return (int)(((x + 1) * n - 1) / W); }

// The whole block: W, this block's range and the unit it starts in.
__device__ __forceinline__ void start_list(const Decode4Params& p, int c, List4& ls, int64_t* scan) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (p.chunk > 0) {
    if (tid == 0) {
      ls.unit = c;
      ls.more = 1;
    }
    __syncthreads();
    return;
  }
  const int per = (p.batch + kWarps * 32 - 1) / (kWarps * 32);
  const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) sum += unit_weight(seq_tiles(p, b));
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int64_t before = 0, W = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan[w];
    W += scan[w];
  }
  W *= p.num_kv_heads;
  const int n = (int)(W < p.ranges ? W : p.ranges);  // every block gets a position
  if (c >= n) {
    if (tid == 0) ls.more = 0;
    __syncthreads();
    return;
  }
  const int64_t begin = W * c / n, end = W * (c + 1) / n;
  const int64_t mine = (before + incl - sum) * p.num_kv_heads;
  if (begin >= mine && begin < mine + sum * p.num_kv_heads) {  // one thread
    int64_t pos = mine;
    int b = b0;
    for (;; ++b) {
      const int64_t w = (int64_t)unit_weight(seq_tiles(p, b)) * p.num_kv_heads;
      if (begin < pos + w) break;
      pos += w;
    }
    const int w = unit_weight(seq_tiles(p, b));
    const int kvh = (int)((begin - pos) / w);
    ls.unit = b * p.num_kv_heads + kvh;
    ls.pos = pos + (int64_t)kvh * w;
    ls.begin = begin;
    ls.end = end;
    ls.total = W;
    ls.ranges = n;
    ls.more = 1;
  }
  __syncthreads();
}

// Warp 0: the next pieces of this block, one unit (or item) per lane.
__device__ __forceinline__ void next_pieces(const Decode4Params& p, int c, List4& ls, Piece4* list) {
  const int lane = threadIdx.x & 31;
  Piece4 x = {};
  bool have = false;
  const int units = p.batch * p.num_kv_heads;
  if (p.chunk > 0) {
    const int64_t item = ls.unit + (int64_t)lane * p.ranges;
    const int64_t items = (int64_t)units * p.splits;
    if (item < items) {
      const int split = (int)(item / units), unit = (int)(item - (int64_t)split * units);
      x.b = unit / p.num_kv_heads;
      x.kvh = unit - x.b * p.num_kv_heads;
      SeqSplits sp;
      if (seq_keys(p, x.b, x.row, sp) && (split < sp.nsplit || split == 0)) {
        have = true;
        x.start = sp.lo + split * p.chunk;
        x.end = min(sp.hi, x.start + p.chunk);
        x.slot = sp.nsplit > 1 ? unit * p.splits + split : -1;
        if (sp.nsplit == 0) x.end = x.start;
        if (!sp.valid && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
      }
    }
    __syncwarp();
    if (lane == 0) {
      const int64_t next = ls.unit + 32ll * p.ranges;
      ls.more = next < items;
      ls.unit = (int)next;
    }
  } else {
    const int unit = ls.unit + lane;
    int tiles = -1;
    SeqSplits sp = {};
    if (unit < units) {
      x.b = unit / p.num_kv_heads;
      x.kvh = unit - x.b * p.num_kv_heads;
      if (seq_keys(p, x.b, x.row, sp)) tiles = sp.hi > sp.lo ? (sp.hi - 1) / kDecodeTile - sp.lo / kDecodeTile + 1 : 0;
    }
    const int w = unit_weight(tiles);
    int incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int64_t base = ls.pos, begin = ls.begin, end = ls.end, total = ls.total;
    const int64_t pos = base + incl - w;  // the unit's first position
    if (tiles >= 0 && pos < end) {
      const int t0 = (int)(begin > pos ? begin - pos : 0);
      const int t1 = (int)(end - pos < tiles ? end - pos : tiles);
      if (tiles == 0) {
        have = begin <= pos;
        if (!sp.valid && p.err) atomicOr(p.err, CAI_DEVERR_LENGTH);
      } else if (t0 < t1) {
        have = true;
        const int tile0 = sp.lo / kDecodeTile;
        x.start = max(sp.lo, (tile0 + t0) * kDecodeTile);
        x.end = min(sp.hi, (tile0 + t1) * kDecodeTile);
        x.slot = t0 == 0 && t1 == tiles ? -1 : 2 * c + (t0 == 0 ? 1 : 0);
      }
      if (have && t0 == 0) {
        const int last = tiles > 0 ? block_of(pos + tiles - 1, total, ls.ranges) : c;
        p.meta[unit] = make_int2(c, last);
      }
    }
    const int64_t after = base + __shfl_sync(0xffffffffu, incl, 31);
    __syncwarp();
    if (lane == 0) {
      ls.more = after < end && ls.unit + 32 < units;
      ls.unit += 32;
      ls.pos = after;
    }
  }
  const uint32_t m = __ballot_sync(0xffffffffu, have);
  if (have) list[__popc(m & ((1u << lane) - 1u))] = x;
  if (lane == 0) ls.count = __popc(m);
}

template <int NT>
__global__ void __launch_bounds__(kWarps * 32, Shape4<NT>::kBlocks) decode4_kernel(const __grid_constant__ Decode4Params p) {
  using S = Shape4<NT>;
  constexpr int NS = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBars);
  volatile uint32_t* ok_bits = reinterpret_cast<volatile uint32_t*>(smem + S::kOffOk);
  float* ml = reinterpret_cast<float*>(smem + S::kOffMl);
  volatile WaitState* wctl = reinterpret_cast<volatile WaitState*>(smem + S::kOffWait);
  Piece4* pieces = reinterpret_cast<Piece4*>(smem + S::kOffPieces);
  List4& ls = *reinterpret_cast<List4*>(smem + S::kOffPieces + kPieces * sizeof(Piece4));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  // Blocks of one range but different head groups are neighbours: they read the same keys at the same time.
  const int G = p.num_heads / p.num_kv_heads;
  const int hg = blockIdx.x % p.head_groups, c = blockIdx.x / p.head_groups;
  const int h0 = hg * S::kHeads;                 // first head of the group
  const int nh = min(G - h0, S::kHeads);         // heads in this block

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
  start_list(p, c, ls, reinterpret_cast<int64_t*>(ml));

  const int P = p.page_size;
  const int per_log2 = P == 16 ? 0 : P == 32 ? 1 : 2;  // blocks of 16 tokens in a page
  uint8_t* ring = smem + warp * NS * kStepBytes;
  uint64_t* full = bars + warp * NS;
  // This warp's next step lies in stage st, the step after the last one issued in stage st_in; phase bit s is
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
      const int64_t row0 = (int64_t)pc.row * p.num_heads + (int64_t)pc.kvh * G + h0;  // the block's first head row
      const int start = pc.start, end = pc.end;
      if (start >= end) {  // nothing to attend, or an invalid length (flagged): out = 0, lse = -inf
        for (int i = threadIdx.x; i < nh * kHeadDim / 4; i += kWarps * 32)
          reinterpret_cast<uint2*>(p.out + row0 * kHeadDim)[i] = make_uint2(0u, 0u);
        if (p.lse_out && threadIdx.x < nh) p.lse_out[row0 + threadIdx.x] = -INFINITY;
        continue;
      }
      const int blk0 = start / kBlk, nblk = (end - 1) / kBlk - blk0 + 1;
      const int steps = (nblk + 1) / 2;
      const int mine = (steps - warp + kWarps - 1) / kWarps;  // this warp's steps: warp, warp + 4, ...
      const uint8_t* pages = p.pages[pc.kvh];
      const int num_pages = p.num_pages[pc.kvh];
      const int32_t* table = p.table + (int64_t)pc.b * p.max_pages;
      const uint16_t* q = p.q + row0 * kHeadDim;
      __syncthreads();  // the last piece's merge has left the ring (and Q)

      // Page ids of this warp's blocks, 16 steps at a time: lane 2 i + h holds block h of step i of the batch.
      auto load_ids = [&](int i0) -> int32_t {
        const int i = i0 + (lane >> 1);
        const int blk = 2 * (warp + i * kWarps) + (lane & 1);
        return i < mine && blk < nblk ? __ldg(table + ((blk0 + blk) >> per_log2)) : -1;
      };
      int32_t ids = load_ids(0);
      int32_t ids_next = mine > 16 ? load_ids(16) : -1;
      int issued = 0;
      // Starts the copies of this warp's next step (both blocks), into stage st_in.
      auto issue = [&]() {
        const int i = issued++, s = st_in;
        st_in = s + 1 == NS ? 0 : s + 1;
        if ((i & 15) == 0 && i > 0) {
          ids = ids_next;
          ids_next = i + 16 < mine ? load_ids(i + 16) : -1;
        }
        const int blk = 2 * (warp + i * kWarps) + (lane & 1);
        const int32_t pid = __shfl_sync(0xffffffffu, ids, 2 * (i & 15) + (lane & 1));
        const bool live = lane < 2 && blk < nblk;
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

      // B operand of S^T: lane (g, t) holds, for head 8 n + g and channel group j, channels 32 j + 8 t ..
      // + 7 (one 16-byte load), two k steps of 16 whose channel order is that of the K words.
      uint4 qf[S::kQRegs ? NT : 1][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!S::kQRegs && j != warp) continue;  // 64 registers would not fit: shared memory, a warp a group
          const uint4 x = 8 * n + g < nh ? __ldg(reinterpret_cast<const uint4*>(q + (8 * n + g) * kHeadDim + 32 * j + 8 * t))
                                         : make_uint4(0u, 0u, 0u, 0u);
          const uint4 y = make_uint4(bf16x2_to_f16x2(x.x), bf16x2_to_f16x2(x.y), bf16x2_to_f16x2(x.z), bf16x2_to_f16x2(x.w));
          if constexpr (S::kQRegs) qf[n][j] = y;
          else reinterpret_cast<uint4*>(smem + S::kOffQ)[(n * 4 + j) * 32 + lane] = y;
        }
      if constexpr (!S::kQRegs) __syncthreads();

      float o[8][NT][4];  // O^T: channels 16 m + g, + 8 x heads 8 n + 2 t, + 1
#pragma unroll
      for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[m][n][e] = 0.0f;
      uint64_t mref[NT], l[NT];  // negated reference (log2 units) and this lane's part of the sum, per head pair
#pragma unroll
      for (int n = 0; n < NT; ++n) mref[n] = l[n] = 0ull;
      bool have_ref = false;  // some key was attended (the same in every lane)

      int i = 0;
      for (; ok && i < mine; ++i) {
        ok = mbar_wait_warp(&full[st], (phase >> st) & 1u, wctl);
        if (!ok) break;
        const uint8_t* stage = ring + st * kStepBytes;
        const uint32_t okm = ok_bits[warp * NS + st];
        const int first = (blk0 + 2 * (warp + i * kWarps)) * kBlk;  // position of the step's first key
        const bool edge = first < start || first + kStep > end || okm != 3u;

        // ---- S^T = K Q^T
        float sc[2][NT][4];
        uint4 kw[2][2];
        uint2 ks[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            kw[h][e] = *reinterpret_cast<const uint4*>(stage + h * kBlkBytes + e * 512 + lane * 16);
            ks[h][e] = *reinterpret_cast<const uint2*>(stage + h * kBlkBytes + kBlkKs + e * 64 + g * 8);
          }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 qq[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if constexpr (S::kQRegs) qq[n] = qf[n][j];
            else qq[n] = reinterpret_cast<const uint4*>(smem + S::kOffQ)[(n * 4 + j) * 32 + lane];
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t x[4], y[4];
            const uint32_t sa = j < 2 ? ks[h][0].x : ks[h][0].y, sb = j < 2 ? ks[h][1].x : ks[h][1].y;
            if constexpr (S::kGroupSums) {
              // A group's products are summed as codes (exact in fp16) and its scale applied to the sum.
              codes_f16(word(kw[h][0], j), x);
              codes_f16(word(kw[h][1], j), y);
              const float a = half_of(sa, j & 1), b = half_of(sb, j & 1);
              const uint64_t a2 = f2(a, a), b2 = f2(b, b);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                mma_16816(acc, x[0], y[0], x[1], y[1], qq[n].x, qq[n].y);
                mma_16816(acc, x[2], y[2], x[3], y[3], qq[n].z, qq[n].w);
                if (j == 0) {
                  f2_split(f2_mul(f2(acc[0], acc[1]), a2), sc[h][n][0], sc[h][n][1]);
                  f2_split(f2_mul(f2(acc[2], acc[3]), b2), sc[h][n][2], sc[h][n][3]);
                } else {
                  f2_split(f2_fma(f2(acc[0], acc[1]), a2, f2(sc[h][n][0], sc[h][n][1])), sc[h][n][0], sc[h][n][1]);
                  f2_split(f2_fma(f2(acc[2], acc[3]), b2, f2(sc[h][n][2], sc[h][n][3])), sc[h][n][2], sc[h][n][3]);
                }
              }
            } else {
              const uint32_t a = __byte_perm(sa, 0u, j & 1 ? 0x3232u : 0x1010u), b = __byte_perm(sb, 0u, j & 1 ? 0x3232u : 0x1010u);
              values_f16(word(kw[h][0], j), a, a, x);
              values_f16(word(kw[h][1], j), b, b, y);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                if (j == 0) sc[h][n][0] = sc[h][n][1] = sc[h][n][2] = sc[h][n][3] = 0.0f;
                mma_16816(sc[h][n], x[0], y[0], x[1], y[1], qq[n].x, qq[n].y);
              }
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_16816(sc[h][n], x[2], y[2], x[3], y[3], qq[n].z, qq[n].w);
            }
          }
        }

        // ---- logits minus reference, in log2 units
        if (edge) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = first + h * kBlk + e * 8 + g;
              if (!(key >= start && key < end && ((okm >> h) & 1u)))
#pragma unroll
                for (int n = 0; n < NT; ++n) sc[h][n][2 * e] = sc[h][n][2 * e + 1] = -INFINITY;
            }
        }
        float mx = -INFINITY;
        const uint64_t sl2 = f2(p.scale_log2, p.scale_log2);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              f2_split(f2_fma(f2(sc[h][n][e], sc[h][n][e + 1]), sl2, mref[n]), sc[h][n][e], sc[h][n][e + 1]);
              mx = fmax3(mx, sc[h][n][e], sc[h][n][e + 1]);
            }
        if (__any_sync(0xffffffffu, have_ref ? mx > kRaise4 : mx > -INFINITY)) {
          // Raise the references that a logit passes by 2^8 (all of them at the first key).
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float up[2], f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float v = fmaxf(fmaxf(sc[0][n][e], sc[0][n][2 + e]), fmaxf(sc[1][n][e], sc[1][n][2 + e]));
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, x));
              up[e] = !have_ref || v > kRaise4 ? v : 0.0f;
              f[e] = have_ref ? ex2_approx(-up[e]) : 0.0f;
#pragma unroll
              for (int m = 0; m < 8; ++m) {
                o[m][n][e] *= f[e];
                o[m][n][2 + e] *= f[e];
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                sc[h][n][e] -= up[e];
                sc[h][n][2 + e] -= up[e];
              }
            }
            mref[n] = f2_add(mref[n], f2(-up[0], -up[1]));
            l[n] = f2_mul(l[n], f2(f[0], f[1]));
          }
          have_ref = true;
        }
        // ---- P^T = 2^z, its sums, and its transpose into the B operand
        uint32_t pf[2][NT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float a = ex2_approx(sc[h][n][2 * e]), b = ex2_approx(sc[h][n][2 * e + 1]);
              l[n] = f2_add(l[n], f2(a, b));
              pf[h][n][e] = transpose8x8(pack_f16x2(a, b));
            }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* blk = stage + h * kBlkBytes;
          uint4 s0 = *reinterpret_cast<const uint4*>(blk + kBlkVs + t * 32);
          uint4 s1 = *reinterpret_cast<const uint4*>(blk + kBlkVs + t * 32 + 16);
          if (edge) {
            // Masked keys' scales become 0 (their slots may hold anything, NaN included).
            const int key = first + h * kBlk + 2 * t;
            const bool good = (okm >> h) & 1u;
            auto keep = [&](int k) { return good && k >= start && k < end; };
            const uint32_t ma = (keep(key) ? 0xFFFFu : 0u) | (keep(key + 1) ? 0xFFFF0000u : 0u);
            const uint32_t mb = (keep(key + 8) ? 0xFFFFu : 0u) | (keep(key + 9) ? 0xFFFF0000u : 0u);
            s0 = make_uint4(s0.x & ma, s0.y & ma, s0.z & ma, s0.w & ma);
            s1 = make_uint4(s1.x & mb, s1.y & mb, s1.z & mb, s1.w & mb);
          }
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const uint4 vw = *reinterpret_cast<const uint4*>(blk + kBlkV + hh * 512 + lane * 16);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int m = hh * 4 + u, j = m >> 1;
              uint32_t x[4];
              values_f16(word(vw, u), word(s0, j), word(s1, j), x);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_16816(o[m][n], x[0], x[1], x[2], x[3], pf[h][n][0], pf[h][n][1]);
            }
          }
        }
        phase ^= 1u << st;
        st = st + 1 == NS ? 0 : st + 1;
        __syncwarp();  // every lane has read the stage
        if (issued < mine) issue();
      }
      if (!ok && issued > i) {
        // A wait gave up: report it, and let this warp's own copies land; it issues no more.
        if (lane == 0 && p.err) atomicOr(p.err, CAI_DEVERR_TIMEOUT);
        for (; i < issued; ++i) {
          if (r + i != p.drop_stage) mbar_wait_drain(&full[st], (phase >> st) & 1u);
          st = st + 1 == NS ? 0 : st + 1;
        }
      }
      r += mine;

      // ---- merge of the warps: out = sum_w 2^(m_w - M) O_w / sum_w 2^(m_w - M) l_w
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float m2[2], l2[2];
        f2_split(mref[n], m2[0], m2[1]);
        f2_split(l[n], l2[0], l2[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l2[e] += __shfl_xor_sync(0xffffffffu, l2[e], x);
          if (g == 0) {
            ml[warp * S::kHeads + 8 * n + 2 * t + e] = have_ref ? -m2[e] : -INFINITY;
            ml[(kWarps + warp) * S::kHeads + 8 * n + 2 * t + e] = l2[e];
          }
        }
      }
      __syncthreads();  // every ring is read, too
      float* mo = reinterpret_cast<float*>(smem);
      if (mine > 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float* dst = mo + (warp * S::kHeads + 8 * n + 2 * t + e) * kORow + g;
#pragma unroll
            for (int m = 0; m < 8; ++m) {
              dst[16 * m] = o[m][n][e];
              dst[16 * m + 8] = o[m][n][2 + e];
            }
          }
      }
      __syncthreads();
      const int live = min(kWarps, steps);
      for (int h = warp; h < nh; h += kWarps) {
        float M = -INFINITY;
        for (int w = 0; w < live; ++w) M = fmaxf(M, ml[w * S::kHeads + h]);
        float sum = 0.0f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < live; ++w) {
          const float f = M == -INFINITY ? 0.0f : ex2_approx(ml[w * S::kHeads + h] - M);
          sum = fmaf(f, ml[(kWarps + w) * S::kHeads + h], sum);
          const float4 x = *reinterpret_cast<const float4*>(mo + (w * S::kHeads + h) * kORow + 4 * lane);
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
          const int64_t at = (int64_t)pc.slot * G + h0 + h;
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

// One block per (sequence, query head): the pieces' normalised outputs merged by their log2-sum-exp.
constexpr int kCombineWarps = 4;
__global__ void __launch_bounds__(kCombineWarps * 32) combine4_kernel(const __grid_constant__ Decode4Params p) {
  __shared__ float part[kCombineWarps][kHeadDim];
  __shared__ float pm[kCombineWarps], pl[kCombineWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x / p.num_heads, h = blockIdx.x - b * p.num_heads;
  const int G = p.num_heads / p.num_kv_heads, kvh = h / G, unit = b * p.num_kv_heads + kvh;
  grid_dependency_wait();
  grid_launch_dependents();
  int32_t row;
  SeqSplits sp;
  if (!seq_keys(p, b, row, sp)) return;
  int n, first = 0;
  if (p.chunk > 0) {
    n = sp.nsplit;
  } else {
    const int2 m = p.meta[unit];
    first = m.x;
    n = m.y - m.x + 1;
  }
  if (n <= 1) return;  // written by the decode kernel
  auto slot = [&](int j) -> int64_t {
    return (p.chunk > 0 ? (int64_t)unit * p.splits + j : 2ll * (first + j) + (j == 0 ? 1 : 0)) * G + (h - kvh * G);
  };
  // Warp w takes pieces w, w + 4, ..., four at a time so that their loads overlap.
  float M = -INFINITY, sum = 0.0f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = warp; j0 < n; j0 += 4 * kCombineWarps) {
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
  if (warp > 0) return;
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

template <int NT>
cudaError_t launch_nt(const Decode4Params& p, cudaStream_t stream) {
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(decode4_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape4<NT>::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set[dev] = true;
  }
  return launch_pdl(decode4_kernel<NT>, dim3((unsigned)(p.head_groups * p.ranges)), dim3(kWarps * 32), Shape4<NT>::kSmem,
                    stream, p);
}

// Heads per block: the group padded to 8, 16 or 32.
int head_tiles(int group) { return group <= 8 ? 1 : group <= 16 ? 2 : 4; }

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t plan_decode4(Decode4Params& p, int32_t num_splits) {
  const int G = p.num_heads / p.num_kv_heads, nt = head_tiles(G);
  const int blocks = num_sms() * (nt == 1 ? Shape4<1>::kBlocks : nt == 2 ? Shape4<2>::kBlocks : Shape4<4>::kBlocks);
  p.head_groups = (G + 8 * nt - 1) / (8 * nt);
  const int64_t units = (int64_t)p.batch * p.num_kv_heads;
  const int64_t cap = (int64_t)p.max_pages * p.page_size;
  const int64_t span = p.window > 0 && p.window < cap ? p.window : cap;
  int64_t ranges = blocks / p.head_groups, most, slots;
  p.chunk = 0;
  p.splits = 0;
  if (num_splits > 0) {
    p.chunk = (int32_t)(((span + num_splits - 1) / num_splits + kDecodeTile - 1) / kDecodeTile * kDecodeTile);
    p.splits = (int32_t)((span + p.chunk - 1) / p.chunk);
    most = units * p.splits;
    slots = p.splits > 1 ? most : 0;
  } else {
    most = units * ((span + kDecodeTile - 1) / kDecodeTile + 2);  // a window may start inside a tile
    slots = 1;
  }
  p.ranges = (int32_t)(ranges < most ? ranges : most);
  if (num_splits == 0) slots = 2 * p.ranges;
  const int64_t rows = slots * G;
  return (size_t)((num_splits == 0 ? up256(units * 8) : 0) + up256(rows * kHeadDim * 4) + up256(rows * 4));
}

void place_decode4(Decode4Params& p, void* workspace) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int64_t units = (int64_t)p.batch * p.num_kv_heads, G = p.num_heads / p.num_kv_heads;
  const int64_t slots = p.chunk == 0 ? 2ll * p.ranges : p.splits > 1 ? units * p.splits : 0;
  p.meta = reinterpret_cast<int2*>(ws);
  if (p.chunk == 0) ws += up256(units * 8);
  p.ws_o = reinterpret_cast<float*>(ws);
  p.ws_lse = reinterpret_cast<float*>(ws + up256(slots * G * kHeadDim * 4));
}

cudaError_t launch_decode4(const Decode4Params& p, cudaStream_t stream) {
  const int nt = head_tiles(p.num_heads / p.num_kv_heads);
  const cudaError_t e = nt == 1 ? launch_nt<1>(p, stream) : nt == 2 ? launch_nt<2>(p, stream) : launch_nt<4>(p, stream);
  if (e != cudaSuccess || (p.chunk > 0 && p.splits <= 1)) return e;
  return launch_pdl(combine4_kernel, dim3((unsigned)(p.batch * p.num_heads)), dim3(kCombineWarps * 32), 0, stream, p);
}

}  // namespace cai

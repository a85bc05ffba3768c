// Tree attention on the tensor cores: the split kernel (see tree_attention.cu
// for the operator).
//
// One CTA per SM, all 512 columns of tensor memory.  The work is the flat
// list of (sequence, KV head, 128-position tile), cut into one equal range
// per CTA; a range holds whole segments ((sequence, KV head) pairs) and at
// most two cut ones, whose rows go to the workspace for the merge.
//
// The 4 query heads of the GQA group times 32 nodes are the 128 rows of an
// MMA tile (row = node * 4 + head).  Two score tiles S_0, S_1 and two output
// tiles O_0, O_1 (128 columns each; P, fp16, over the first half of its S)
// let one tile's softmax overlap the other's MMAs:
//  * trees of up to 32 nodes: one row tile; KV tiles alternate between slots 0
//    and 1, each with its own running max, sum and O, joined at the end of the
//    piece.  K and V are read once and every MMA row block works on another
//    KV tile;
//  * wider trees: two row tiles, both over every KV tile.
// A unit is one (KV tile, slot): S = Q K^T, softmax, O += P V.  Where wide
// trees may be among the batch a unit is worked on in two parts of 64
// positions, each with half of the slot's S columns, so that one part's S and
// P V run under the other's softmax.
//
// Warp roles (16 warps): 0-3 / 4-7 softmax of slot 0 / 1, one thread per row;
// 8, 10, 11, 14 dequantise V (E4M3 pages -> fp16 MN-major half tiles); 15
// issues S = Q K^T and 9 O += P V; 13 loads Q and K pages (TMA); 12 loads the
// E4M3 pages (bulk copies), walks the CTA's pieces and hands them to the
// others.  Every hand-off is an mbarrier, every wait is bounded.
//
// What it is built around (cycles at 1.96 GHz, from time stamps of one CTA; a
// KV tile at the full memory rate takes 2,150):
//  * An S MMA with both operands in shared memory takes the whole 128 bytes a
//    cycle (64 cycles per 128 x 128 x 16), and everything else in shared memory
//    waits: the test of a barrier takes 140-300 cycles.  So the warps that issue
//    MMAs test all their barriers at once, one per lane, and keep what they
//    learned (174 -> 168 us on 16 x 64 nodes at 8K); S and P V are issued by a
//    warp each, because the issue of one unit takes ~1,000 cycles of one warp
//    (173 -> 167 us).  Parts of 64 positions cost S a third of its rate (55
//    cycles per 128 x 64 x 16) and still gain for two row tiles, where MMAs and
//    softmax alternate otherwise (173 / 155 us in one part and in two, 16 x 64
//    nodes at 8K); for one row tile they do not (44.7 / 45.3 us on 32 x 32 nodes at
//    1.1K, 100.6 / 101.1 at 8K) and are not used.
//  * Nothing is in local memory: what L1 has left beside the operand stages is
//    so little that a spilled register or an array indexed at run time costs a
//    trip to L2 (~700 cycles) each time (46.8 -> 41.4 us on 32 x 8 nodes at 1.1K).
//  * The maximum of a row comes with the load (tcgen05.ld.red), and 16 columns
//    are on their way while 16 are exponentiated (103 -> 100 us on 32 nodes at
//    128K).  The loops are kept rolled up: each warp runs its role's code once
//    per tile, and unrolled over the 128 columns that code came from the far
//    side of the instruction cache (4,000 cycles a tile, against 1,500).
//  * The whole MMA warp walks the units and one elected lane issues: operands
//    stay in uniform registers (3,030 -> 1,900 cycles a unit).
//  * A bulk or tensor copy takes its lane ~90 cycles to issue, so K and V have
//    a warp each, and asking L2 for pages ahead of time costs more than it
//    hides (143 against 131 us on 8 nodes at 128K).
//  * A copy lands ~2,000-3,000 cycles after it is issued: three stages each
//    (two of K for wide trees, whose tiles take longer).
//  * A piece's description may take memory round trips to work out (the next
//    sequence's lengths): that is done one piece ahead, behind the copies of
//    the piece's first tile.
//  * Slots do not wait for one another where they need not: two row tiles end
//    their pieces apart (163 -> 148 us on 256 x 64 nodes at 250 positions).
// What a call takes now: 8 nodes at 128K 90 us (5.6 TB/s of K and V), 16 x 8
// nodes at 8K 93 us, 16 x 64 nodes at 8K 152 us (1.1 PFLOP/s), 32 x 16 nodes at
// 1.1K 40 us, one tree of 5 at 1K 11.3 us, the merge included.
#pragma once

#include "k16v8_device.cuh"
#include "tc_sm100.cuh"
#include "tree_plan.cuh"

namespace k16v8 {
namespace tree {
namespace tcore {

constexpr unsigned kFull = 0xffffffffu;

constexpr int kNodes = 32;                   // nodes per row tile
constexpr int kRows = kNodes * kGroup;       // 128
constexpr int kKv = 128;                     // positions per KV tile
constexpr int kPagesPerTile = kKv / kPage;   // 8
constexpr int kThreads = 512;
constexpr int kOutWarp = 9, kLoadVWarp = 12, kLoadKWarp = 13, kScoreWarp = 15;
constexpr int kDequantWarps = 4;
constexpr int kDequantThreads = kDequantWarps * 32;
constexpr int kPieceRing = 4;
constexpr int kPieceReaders = 8 + kDequantWarps + 4;  // every warp

// Rank of a dequant warp among them, or -1.
__device__ __forceinline__ int dequant_rank(int warp) {
  return warp == 8 ? 0 : warp == 10 ? 1 : warp == 11 ? 2 : warp == 14 ? 3 : -1;
}

constexpr uint32_t kQBytes = kRows * 256;
constexpr uint32_t kKBlk = kKv * 128;          // [128 pos][64 dims] fp16
constexpr uint32_t kKStage = 2 * kKBlk;
constexpr uint32_t kVstStage = kKv * 128;      // [128 pos][128] E4M3
constexpr int kHalf = kKv / 2;                 // positions of a V half tile
constexpr uint32_t kVBlk = kHalf * 128;        // [64 pos][64 dims] fp16
constexpr uint32_t kVHalf = 2 * kVBlk;
constexpr uint32_t kTmemCols = 512;  // S_0 [0,128) S_1 [128,256) O_0 [256,384) O_1 [384,512)

constexpr uint32_t kBarBytes = 448;

// kWide: trees of more than 32 nodes may be among the batch.
template <bool kWide>
struct Smem {
  static constexpr int kParts = kWide ? 2 : 1;  // of a unit
  static constexpr int kQSlots = kWide ? 2 : 1;
  // stages: with two row tiles a V tile is held until both have read it, so
  // two whole ones are needed; else a half tile is free as soon as it is read
  static constexpr int kKStages = kWide ? 2 : 3;
  static constexpr int kVstStages = kWide ? 2 : 3;
  static constexpr int kVHalves = kWide ? 4 : 3;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + kQSlots * kQBytes;
  static constexpr uint32_t kVst = kK + kKStages * kKStage;
  static constexpr uint32_t kV = kVst + kVstStages * kVstStage;
  static constexpr uint32_t kBar = kV + kVHalves * kVHalf;
  static constexpr uint32_t kPieces = kBar + kBarBytes;
  static constexpr uint32_t kInfo = kPieces + kPieceRing * sizeof(Piece);
  static constexpr uint32_t kNan = kInfo + 16 * 4;   // tree nodes with NaN value codes
  static constexpr uint32_t kStat = kNan + 4 * 8;    // [slot][max, sum][row]
  static constexpr uint32_t kBytes = kStat + 2 * 2 * kRows * 4;
  static_assert(kBytes <= 227 * 1024, "one CTA's shared memory");
  static_assert(sizeof(int64_t) * (kMaxBatch + 1) <= kBar, "the scan's scratch");
  static_assert(sizeof(int64_t) * 33 <= kBytes - kStat, "the scan's warp sums");
  static_assert(kInfo % 8 == 0 && kNan % 8 == 0 && kStat % 16 == 0, "alignment");
};

enum {
  kBarQFull = 0,      // +slot
  kBarQEmpty = 2,     // +slot
  kBarKFull = 4,      // +stage
  kBarKEmpty = 7,     // +stage
  kBarVstFull = 10,   // +stage
  kBarVstEmpty = 13,  // +stage, kDequantThreads arrivals
  kBarVFull = 16,     // +half, kDequantThreads arrivals
  kBarVEmpty = 20,    // +half
  kBarSFull = 24,     // +slot + 2 * part
  kBarPFull = 28,     // +slot + 2 * part, 4 arrivals (one per warp)
  kBarPV = 32,        // +slot + 2 * part: the part's P V is done
  kBarODone = 36,     // +slot: the slot's last P V of a piece
  kBarOEmpty = 38,    // 8 arrivals: both O tiles have been read
  kBarJoin = 39,      // 8 arrivals (one per warp): both slots' statistics are in shared memory
  kBarPiece = 40,     // +ring entry: described
  kBarTaken = 44,     // +ring entry: kPieceReaders arrivals
  kBarDrain = 48,     // +0, 1: every S, every P V
  kNumBars = 50
};
static_assert(kNumBars * 8 + 16 <= kBarBytes, "barriers");

// A count for either slot.  (Arrays indexed at run time would live in local
// memory, behind the little L1 that the operand stages leave.)
struct Pair {
  uint32_t c0 = 0, c1 = 0;
  __device__ __forceinline__ uint32_t operator[](int w) const { return w ? c1 : c0; }
  __device__ __forceinline__ void add(int w, uint32_t n = 1) {
    if (w)
      c1 += n;
    else
      c0 += n;
  }
};

// Position in a ring of n stages: the stage, and the parity of its phase.
template <int n>
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  bool wrapped = false;  // every stage has been used once
  __device__ __forceinline__ void next() {
    if (++s == n) {
      s = 0;
      phase ^= 1;
      wrapped = true;
    }
  }
};

// As in prefill: a wait that runs out raises the CTA-wide abort flag, which
// the suspending waits poll; every role leaves its loops on a failed wait.
__device__ __forceinline__ bool cta_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                         int32_t *dev_error) {
  for (uint32_t i = 0; i < kMaxPolls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 1023u) == 0 && *abort_flag) return false;
  }
  *abort_flag = 1;
  flag_error(dev_error, K16V8_DEVERR_TIMEOUT);
  return false;
}

// The 128 columns of a tile, or 64 of one part, that a row sees.
struct Columns {
  uint64_t lo, hi;
};
__device__ __forceinline__ uint32_t word(const Columns &s, int c) {
  return static_cast<uint32_t>((c & 2 ? s.hi : s.lo) >> (c & 1) * 32);
}
// 64 columns from the one `rel` behind the first node, for a row with tree mask m.
__device__ __forceinline__ uint64_t visible(int rel, uint64_t m) {
  if (rel <= -64) return ~0ull;
  if (rel >= 64) return 0ull;
  if (rel < 0) return ((1ull << -rel) - 1) | m << -rel;
  return m >> rel;
}

// Page id of page `lane` of a piece's tile t: -1 outside the pool, -2 behind
// the last position (and for lanes without a page).
__device__ __forceinline__ int page_id(const Args &a, const Piece &p, int t, int lane) {
  const int page = t * kPagesPerTile + lane;
  if (lane >= kPagesPerTile || page * kPage >= p.L) return -2;
  const int pid = __ldg(a.block_table + static_cast<int64_t>(p.b) * a.maxp + page);
  return pid >= 0 && pid < a.num_pages ? pid : -1;
}

// An asynchronous load's registers stay its own until here.
__device__ __forceinline__ void keep(const uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" ::"r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]),
                 "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7]));
}

// A row's weights are held 2^7 times as large as against its maximum, which
// moves when it grows by more than 2^8, so they stay below 2^15.
constexpr float kLift = 7.f, kSlack = 8.f;

// p = 2^(s * scale - m) of 16 scores to tensor memory, their sum in fp32; m is
// kLift below a maximum of the row.  P is rounded to fp16, the type of V's
// tile: an MMA takes both operands in one type, and bf16 would round P eight
// times as coarsely.  That is 2^-11 of a weight down to 2^-21 of the row's
// largest; a smaller one is subnormal and off by up to 2^-32 of the largest,
// which the row's sum, in fp32, does not share: L positions put O off by at
// most L 2^-32 max|v|.  (Without the lift, L 2^-25: a score 17 above a flat tail
// of 131,072 positions loses 0.24% of the output; the lift takes no instruction
// per weight.)
template <bool kMask>
__device__ __forceinline__ void exp_chunk(uint32_t t_p, const uint32_t (&s)[16], uint32_t seen,
                                          float2 scale, float2 neg_m, float2 &sum) {
  uint32_t pk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 x = __ffma2_rn(
        make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), scale, neg_m);
    float2 p = make_float2(ex2(x.x), ex2(x.y));
    if (kMask) {
      if (!(seen >> (2 * e) & 1)) p.x = 0.f;
      if (!(seen >> (2 * e + 1) & 1)) p.y = 0.f;
    }
    sum = __fadd2_rn(sum, p);
    const __half2 h = __floats2half2_rn(p.x, p.y);
    pk[e] = *reinterpret_cast<const uint32_t *>(&h);
  }
  tc::tmem_st8(t_p, pk);
}

// kTest: the form of the bounded-wait test hook.  CTA 0 withholds K of its first
// tile (no arrival, nothing in flight), so the score warp's wait for it runs out
// after kTestSpins polls and every role takes the abort path.
template <bool kWide, bool kTest>
__global__ void __launch_bounds__(kThreads, 1) tree_tc_kernel(
    const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
    const Args a) {
  using M = Smem<kWide>;
  constexpr int kParts = M::kParts, kChunks = 4 / kParts;  // of a tile; of 32 columns
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *sQ = smem_raw + M::kQ;
  uint8_t *sK = smem_raw + M::kK;
  uint8_t *sVst = smem_raw + M::kVst;
  uint8_t *sV = smem_raw + M::kV;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem_raw + M::kBar);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kNumBars);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + kNumBars) + 1;
  Piece *pieces = reinterpret_cast<Piece *>(smem_raw + M::kPieces);
  // rejected pages of a tile: for the softmax (by tile, 8 of them) and for the
  // dequantisation (by stage)
  volatile uint32_t *info = reinterpret_cast<volatile uint32_t *>(smem_raw + M::kInfo);
  volatile uint32_t *info_v = info + 8;
  uint32_t *nan_nodes = reinterpret_cast<uint32_t *>(smem_raw + M::kNan);  // [4][2], by piece
  float *stat = reinterpret_cast<float *>(smem_raw + M::kStat);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hq = a.hkv * kGroup;
  if (smem_addr(smem_raw) & 1023u) {  // operand tiles need 1024-byte alignment
    pdl_wait();
    if (tid == 0) {
      a.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
      flag_error(a.dev_error, K16V8_DEVERR_INTERNAL);
    }
    return;
  }
  // ---- set-up that needs nothing of the preceding kernel ----
  if (warp == kLoadKWarp && lane == 0) {
    tc::prefetch_tensormap(&tmap_q);
    tc::prefetch_tensormap(&tmap_k);
  }
  if (warp == 0) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t count = 1;
      if (i >= kBarVstEmpty && i < kBarVEmpty) count = kDequantThreads;
      if (i >= kBarPFull && i < kBarPV) count = 4;
      if (i == kBarJoin) count = 8;
      if (i == kBarOEmpty) count = 8;
      if (i >= kBarTaken && i < kBarDrain) count = kPieceReaders;
      mbar_init(&bars[i], count);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  pdl_wait();
  if (tid == kLoadVWarp * 32) a.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
  // ---- this CTA's range of the work (scratch: the operand stages) ----
  constexpr Shape kShape{kKv, kNodes};
  const Range range = plan_range(a, kShape, kWide ? 2 : 1, reinterpret_cast<int64_t *>(smem_raw),
                                 reinterpret_cast<int64_t *>(smem_raw + M::kStat));
  const bool work = range.lo < range.hi;  // uniform over the CTA
  const bool withholds = kTest && blockIdx.x == 0;
  fence_proxy_async();  // the scan's scratch becomes operand stages
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  auto wait = [&](int bar, uint32_t parity) {
    return cta_wait(&bars[bar], parity, abort_flag, a.dev_error);
  };
  // The next piece, for a whole warp; false at the end (or after an abort).
  auto get_piece = [&](Piece &pc, Ring<kPieceRing> &r) {
    if (!__all_sync(kFull, wait(kBarPiece + r.s, r.phase))) return false;
    pc = pieces[r.s];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[kBarTaken + r.s]);
    r.next();
    return pc.tiles > 0;
  };

  if (!work) {
  } else if (warp < 8) {
    // ================= softmax of slot w =================
    const int w = warp >> 2;
    const int r = tid & 127;
    const float qk_scale = a.sm_scale * kLog2e;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + w * 128;
    const uint32_t tO = tmem + 256 + w * 128;
    const uint32_t tOther = tmem + 256 + (w ^ 1) * 128;
    Ring<kPieceRing> ring;
    uint32_t units = 0;             // of this slot so far
    Pair last;                      // pieces in which a slot had units, so far
    uint32_t tiles = 0;             // of the CTA so far
    uint32_t joins = 0;             // pieces with one row tile, so far
    bool ok = true;
    for (uint32_t p_idx = 0; ok; ++p_idx) {
      // the piece stays in shared memory: registers are short here
      if (!__all_sync(kFull, wait(kBarPiece + ring.s, ring.phase))) break;
      const Piece &pc = pieces[ring.s];
      if (pc.tiles == 0) break;
      const bool two = kWide && pc.n > kNodes;  // two row tiles
      const int node = (two ? w * kNodes : 0) + (r >> 2);
      const bool row_valid = node < pc.n;
      const bool warp_live = (two ? w * kNodes : 0) + (warp & 3) * 8 < pc.n;
      const uint64_t mask_word =
          row_valid ? __ldg(a.tree_mask + pc.q0 + node) & pc.node_bits() : 0;  // used late
      const float vs = __ldg(a.v_scale + pc.g);
      const int mine = two ? pc.tiles : (pc.tiles + 1 - w) / 2;
      const int n_tiles = pc.tiles, d0 = pc.base() - pc.t0 * kKv;
      const int theirs = two ? 0 : (pc.tiles + w) / 2;  // units of the other slot to join
      float m_used = -INFINITY, l = 0.f;
      for (int k = 0; ok && k < mine; ++k, ++units) {
#pragma unroll 1
        for (int part = 0; part < kParts; ++part) {
          if (!__all_sync(kFull, wait(kBarSFull + w + 2 * part, units & 1))) {
            ok = false;
            break;
          }
          if (!warp_live) {
            if (lane == 0) mbar_arrive(&bars[kBarPFull + w + 2 * part]);
            continue;
          }
          tc::fence_after_sync();
          const int tile = two ? k : 2 * k + w;
          const int d = d0 - tile * kKv;  // prefix columns of this tile
          const uint32_t bad = info[(tiles + tile) & 7];
          const uint32_t tSp = tS + lane_base + part * kChunks * 32;
          // pass 1: row max
          float rmax = -INFINITY;
          bool need_mask = d < kKv;
          if (!need_mask) {
#pragma unroll 1
            for (int c = kChunks - 2; c >= 0; c -= 2) {
              uint32_t s0[32], s1[32];
              float m0, m1;
              tc::tmem_ld32_max(tSp + c * 32 + 32, s1, m1);
              tc::tmem_ld32_max(tSp + c * 32, s0, m0);
              tc::tmem_wait_ld();
              keep(s1);
              keep(s0);
              rmax = fmaxf(rmax, fmaxf(m0, m1));
            }
            need_mask = bad != 0;  // (seldom; its load took place meanwhile)
          }
          Columns seen{0, 0};
          if (need_mask) {
            seen.lo = visible(part * 64 - d, mask_word);
            if (kParts == 1) seen.hi = visible(64 - d, mask_word);
            for (uint32_t pages = bad >> 4 * part; pages; pages &= pages - 1) {
              const int page = __ffs(static_cast<int>(pages)) - 1;
              const uint64_t out = 0xffffull << (page & 3) * 16;
              if (page < 4)
                seen.lo &= ~out;
              else if (kParts == 1)
                seen.hi &= ~out;
            }
            rmax = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
              uint32_t s0[32];
              tc::tmem_ld32(tSp + c * 32, s0);
              tc::tmem_wait_ld();
              const uint32_t v = word(seen, c);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (v >> e & 1) rmax = fmaxf(rmax, __uint_as_float(s0[e]));
            }
          }
          rmax *= qk_scale;
          float alpha = 1.f;
          if (rmax > m_used + (kLift + kSlack)) {
            alpha = ex2(m_used - (rmax - kLift));
            m_used = rmax - kLift;
          }
          if (k + part > 0 && __any_sync(kFull, alpha != 1.f)) {
            // S of this part was issued after the P V of the part kParts before it;
            // any in between have to be done as well
            if (kParts > 1) {
              if (!__all_sync(kFull, wait(kBarPV + w + 2 * (part ^ 1), (units + part + 1) & 1))) {
                ok = false;
                break;
              }
              tc::fence_after_sync();
            }
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tc::tmem_ld32(tO + lane_base + c * 32, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tc::tmem_st32(tO + lane_base + c * 32, o);
            }
          }
          // pass 2: p = 2^(s * scale - m), fp32 row sum, P (fp16) over the S columns read
          const float neg = m_used == -INFINITY ? 0.f : -m_used;
          const float2 sc2 = make_float2(qk_scale, qk_scale);
          const float2 nm2 = make_float2(neg, neg);
          float2 ps2 = make_float2(0.f, 0.f);
          uint32_t s0[16], s1[16];
          if (!need_mask) {  // 16 columns are on their way while 16 are worked on
            tc::tmem_ld16(tSp, s0);
            tc::tmem_wait_ld();
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
              tc::tmem_ld16(tSp + c * 32 + 16, s1);
              exp_chunk<false>(tSp + c * 16, s0, 0, sc2, nm2, ps2);
              tc::tmem_wait_ld();
              tc::tmem_ld16(tSp + ((c + 1) & (kChunks - 1)) * 32, s0);  // (the last is unused)
              exp_chunk<false>(tSp + c * 16 + 8, s1, 0, sc2, nm2, ps2);
              tc::tmem_wait_ld();
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < 2 * kChunks; ++c) {
              tc::tmem_ld16(tSp + c * 16, s0);
              tc::tmem_wait_ld();
              exp_chunk<true>(tSp + c * 8, s0, word(seen, c >> 1) >> ((c & 1) * 16), sc2, nm2, ps2);
            }
          }
          tc::tmem_wait_st();
          l = l * alpha + (ps2.x + ps2.y);
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kBarPFull + w + 2 * part]);
        }
      }
      if (!ok) break;
      tiles += n_tiles;
      // ---- end of the piece: this slot's O, and with one row tile the other's ----
      const bool second = two || pc.tiles > 1;  // slot 1 has units
      if (mine > 0) ok = __all_sync(kFull, wait(kBarODone + w, last[w] & 1));
      if (ok && theirs > 0) ok = __all_sync(kFull, wait(kBarODone + (w ^ 1), last[w ^ 1] & 1));
      if (!ok) break;
      last.add(0);
      last.add(1, second);
      tc::fence_after_sync();
      const int pn = (p_idx & 3) * 2;
      const uint64_t nan_mask = nan_nodes[pn] | static_cast<uint64_t>(nan_nodes[pn + 1]) << 32;
      float f_own = 1.f, f_other = 0.f;
      float m_all = m_used, l_all = l;
      if (!two) {
        // (the last piece's have been read: this one's O was written after that)
        stat[(w * 2 + 0) * kRows + r] = m_used;
        stat[(w * 2 + 1) * kRows + r] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kBarJoin]);
        ok = __all_sync(kFull, wait(kBarJoin, joins++ & 1));
        if (!ok) break;
        const float m_o = stat[((w ^ 1) * 2 + 0) * kRows + r];
        const float l_o = stat[((w ^ 1) * 2 + 1) * kRows + r];
        m_all = fmaxf(m_used, m_o);
        // (a slot whose scores were all NaN keeps max -inf: its NaN sum decides)
        f_own = m_used == -INFINITY ? (l != l ? l : 0.f) : ex2(m_used - m_all);
        f_other = m_o == -INFINITY ? (l_o != l_o ? l_o : 0.f) : ex2(m_o - m_all);
        l_all = f_own * l + f_other * l_o;
      }
      const bool dead = !(l_all > 0.f) && l_all == l_all;  // the row sees nothing
      const float inv = dead ? 0.f : __fdividef(vs, l_all);
      // (the lift is taken off the sum, whose logarithm is most accurate near 1)
      const float lse =
          dead ? -INFINITY : ((m_all + kLift) + lg2(l_all * 0x1p-7f)) * kLn2;
      static_assert(kLift == 7.f, "the factor of l_all");
      const float g_own = f_own * inv, g_other = f_other * inv;
      // with one row tile, slot w's warps write dims 64w .. 64w + 63 of every row
      const int c_lo = two ? 0 : 4 * w, c_hi = two ? 8 : 4 * w + 4;  // 16 dims each
      const int row = (two ? w * kRows : 0) + r;  // of the segment
      const int64_t orow = static_cast<int64_t>(pc.q0 + node) * hq + pc.g * kGroup + (r & 3);
      const bool whole = pc.whole;
      if (warp_live) {
        // (what the piece says is read once: shared memory is slow under the MMAs)
        __half *po = a.out + orow * kHeadDim;
        float4 *pp = a.part_o + static_cast<int64_t>(pc.slot) * 32 * a.max_rows + row;
#pragma unroll 1
        for (int c = c_lo; c < c_hi; ++c) {
          float o[16];
          {
            uint32_t x[16];
            if (mine > 0) {
              tc::tmem_ld16(tO + lane_base + c * 16, x);
              tc::tmem_wait_ld();
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = mine > 0 ? __uint_as_float(x[e]) * g_own : 0.f;
            if (theirs > 0) {
              tc::tmem_ld16(tOther + lane_base + c * 16, x);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = fmaf(__uint_as_float(x[e]), g_other, o[e]);
            }
          }
          // NaN value codes of nodes this row sees
          for (uint64_t nm = mask_word & nan_mask; nm; nm &= nm - 1) {
            const int pos = pc.base() + __ffsll(static_cast<long long>(nm)) - 1;
            const int page = __ldg(a.block_table + static_cast<int64_t>(pc.b) * a.maxp + pos / kPage);
            if (page < 0 || page >= a.num_pages) continue;
            const uint8_t *vr = a.v_cache + ((static_cast<int64_t>(page) * a.hkv + pc.g) * kPage +
                                             pos % kPage) * kHeadDim + c * 16;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if ((__ldg(vr + e) & 0x7f) == 0x7f) o[e] = NAN;
          }
          if (row_valid && whole) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t pk[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __half2 hh = __floats2half2_rn(o[q * 8 + 2 * e], o[q * 8 + 2 * e + 1]);
                pk[e] = *reinterpret_cast<const uint32_t *>(&hh);
              }
              reinterpret_cast<uint4 *>(po)[2 * c + q] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
          } else if (row_valid) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              pp[static_cast<int64_t>(4 * c + q) * a.max_rows] =
                  make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          }
        }
        if (row_valid && (two || w == 0)) {
          if (!whole)
            a.part_lse[static_cast<int64_t>(pc.slot) * a.max_rows + row] = lse;
          else if (a.lse)
            a.lse[orow] = lse;
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars[kBarOEmpty]);  // O is read: the next piece may write it
        mbar_arrive(&bars[kBarTaken + ring.s]);
      }
      ring.next();
    }
    pdl_launch_dependents();
  } else if (dequant_rank(warp) >= 0) {
    // ================= V dequantisation =================
    const int dt = dequant_rank(warp) * 32 + lane;
    Piece pc;
    Ring<kPieceRing> ring;
    Ring<M::kVstStages> src;
    Ring<M::kVHalves> dst;
    bool ok = true;
    for (uint32_t p_idx = 0; ok && get_piece(pc, ring); ++p_idx) {
      for (int t = pc.t0; ok && t < pc.t1; ++t) {
        ok = wait(kBarVstFull + src.s, src.phase);
        const int live = pc.L - t * kKv;       // positions of the tile in the sequence
        const int tree0 = pc.base() - t * kKv;  // those from here on are nodes
        const uint32_t bad = info_v[src.s];
        const uint8_t *vst = sVst + src.s * kVstStage;
#pragma unroll 1
        for (int h = 0; ok && h < 2; ++h) {
          if (dst.wrapped) ok = wait(kBarVEmpty + dst.s, dst.phase ^ 1);
          if (!ok) break;
          uint8_t *vdst = sV + dst.s * kVHalf;
          // chunk i of this thread: 16 E4M3 values, position hp of the half
          constexpr int kChunks = kHalf * 8 / kDequantThreads;
          auto put = [&](int hp, int c16, const uint4 &raw) {
            const uint32_t wv[4] = {raw.x, raw.y, raw.z, raw.w};
            uint32_t hv[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const __half2 u = e4m3x2_to_half2(static_cast<uint16_t>(wv[q] & 0xffffu));
              const __half2 v = e4m3x2_to_half2(static_cast<uint16_t>(wv[q] >> 16));
              hv[2 * q] = *reinterpret_cast<const uint32_t *>(&u);
              hv[2 * q + 1] = *reinterpret_cast<const uint32_t *>(&v);
            }
            const uint32_t off = hp * 128 + (c16 & 3) * 32;
            uint8_t *blk = vdst + (c16 >> 2) * kVBlk;
            *reinterpret_cast<uint4 *>(blk + tc::sw128(off)) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
            *reinterpret_cast<uint4 *>(blk + tc::sw128(off + 16)) =
                make_uint4(hv[4], hv[5], hv[6], hv[7]);
          };
          const int hp0 = dt >> 3, c16 = dt & 7;
          const uint8_t *from = vst + (h * kHalf + hp0) * 128 + c16 * 16;
          if (tree0 >= kKv && !bad) {  // prefix positions only: no tests, loads in flight together
            uint4 raw[kChunks];
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
              raw[i] = *reinterpret_cast<const uint4 *>(from + i * (kDequantThreads / 8) * 128);
#pragma unroll
            for (int i = 0; i < kChunks; ++i) put(hp0 + i * (kDequantThreads / 8), c16, raw[i]);
          } else {
#pragma unroll 1
            for (int i = 0; i < kChunks; ++i) {
              const int hp = hp0 + i * (kDequantThreads / 8), pos = h * kHalf + hp;
              uint4 raw = make_uint4(0, 0, 0, 0);
              if (pos < live && !(bad >> (pos >> 4) & 1)) {
                raw = *reinterpret_cast<const uint4 *>(from + i * (kDequantThreads / 8) * 128);
                if (pos >= tree0) {  // a node: NaN codes must not reach rows that do not see it
                  const uint32_t n0 = nan_bytes(raw.x), n1 = nan_bytes(raw.y),
                                 n2 = nan_bytes(raw.z), n3 = nan_bytes(raw.w);
                  if (n0 | n1 | n2 | n3) {
                    raw = make_uint4(raw.x & ~n0, raw.y & ~n1, raw.z & ~n2, raw.w & ~n3);
                    const int rel = pos - tree0;
                    atomicOr(&nan_nodes[(p_idx & 3) * 2 + (rel >> 5)], 1u << (rel & 31));
                  }
                }
              }
              put(hp, c16, raw);
            }
          }
          fence_proxy_async();
          mbar_arrive(&bars[kBarVFull + dst.s]);
          dst.next();
        }
        if (!ok) break;
        mbar_arrive(&bars[kBarVstEmpty + src.s]);
        src.next();
      }
    }
  } else if (warp == kLoadVWarp) {
    // ================= V loads, and the CTA's pieces =================
    // Lane 0 also walks the pieces: the first at the start, the next one behind
    // the copies of a piece's first tile.
    Walker walker;
    Ring<kPieceRing> out;
    bool more = true;
    if (lane == 0) walker.init(a, kShape, range);
    auto describe = [&]() {
      bool done = true;
      if (lane == 0 && more) {
        done = !out.wrapped || wait(kBarTaken + out.s, out.phase ^ 1);
        if (done) {
          Piece p;
          more = walker.next(a, kShape, range, p);
          if (!more) p.tiles = 0;  // the end
          pieces[out.s] = p;
          nan_nodes[2 * out.s] = nan_nodes[2 * out.s + 1] = 0;  // (a ring like the pieces')
          mbar_arrive(&bars[kBarPiece + out.s]);
          out.next();
        }
      }
      return __all_sync(kFull, done) != 0;
    };
    Piece pc;
    Ring<kPieceRing> ring;
    Ring<M::kVstStages> dst;
    uint32_t issued = 0;
    bool ok = describe();
    while (ok && get_piece(pc, ring)) {
      int pid = page_id(a, pc, pc.t0, lane);
      for (int t = pc.t0; t < pc.t1; ++t) {
        if (dst.wrapped) ok = __all_sync(kFull, wait(kBarVstEmpty + dst.s, dst.phase ^ 1));
        if (!ok) break;
        const uint32_t bad = __ballot_sync(kFull, pid == -1);
        const uint32_t bytes = __popc(__ballot_sync(kFull, pid >= 0)) * 2048u;
        if (lane == 0) {
          if (bad) flag_error(a.dev_error, K16V8_DEVERR_PAGE);
          info_v[dst.s] = bad;
          mbar_arrive_expect_tx(&bars[kBarVstFull + dst.s], bytes);
        }
        __syncwarp();
        if (pid >= 0)
          bulk_g2s(sVst + dst.s * kVstStage + lane * 2048,
                   a.v_cache + (static_cast<int64_t>(pid) * a.hkv + pc.g) * kPage * kHeadDim, 2048,
                   &bars[kBarVstFull + dst.s]);
        if (t + 1 < pc.t1) pid = page_id(a, pc, t + 1, lane);
        __syncwarp();
        dst.next();
        ++issued;
        if (t == pc.t0) ok = ok && describe();
        if (!ok) break;
      }
    }
    // let the copies issued last land before shared memory is released
    if (lane == 0)
      for (uint32_t n = M::kVstStages, i = issued < n ? 0 : issued - n; i < issued; ++i)
        mbar_wait_bounded(&bars[kBarVstFull + i % n], (i / n) & 1);
    __syncwarp();
  } else if (warp == kLoadKWarp) {
    // ================= Q and K loads =================
    Piece pc;
    Ring<kPieceRing> ring;
    Ring<M::kKStages> dst;
    uint32_t issued = 0;
    Pair uses;
    bool ok = true;
    for (uint32_t p_idx = 0; ok && get_piece(pc, ring); ++p_idx) {
      int pid = page_id(a, pc, pc.t0, lane);
      for (int t = pc.t0; ok && t < pc.t1; ++t) {
        if (dst.wrapped) ok = __all_sync(kFull, wait(kBarKEmpty + dst.s, dst.phase ^ 1));
        if (!ok) break;
        const uint32_t bad = __ballot_sync(kFull, pid == -1);
        const uint32_t bytes = __popc(__ballot_sync(kFull, pid >= 0)) * 4096u;
        const bool withheld = withholds && issued == 0;
        if (lane == 0) {
          info[issued & 7] = bad;
          if (!withheld) mbar_arrive_expect_tx(&bars[kBarKFull + dst.s], bytes);
        }
        __syncwarp();
        if (pid >= 0 && !withheld) {
          uint8_t *k_dst = sK + dst.s * kKStage + lane * 2048;
          const int row = (pid * a.hkv + pc.g) * kPage;
          tc::tma_load_2d(k_dst, &tmap_k, 0, row, &bars[kBarKFull + dst.s]);
          tc::tma_load_2d(k_dst + kKBlk, &tmap_k, 64, row, &bars[kBarKFull + dst.s]);
        }
        if (t + 1 < pc.t1) pid = page_id(a, pc, t + 1, lane);
        __syncwarp();
        dst.next();
        ++issued;
        if (t == pc.t0) {  // the query, behind the first tile's copies
          const bool two = kWide && pc.n > kNodes;
          for (int i = 0; ok && i < (two ? 2 : 1); ++i) {
            const int qs = two ? i : (kWide ? p_idx & 1 : 0);
            if (uses[qs] > 0) ok = __all_sync(kFull, wait(kBarQEmpty + qs, (uses[qs] - 1) & 1));
            if (!ok) break;
            uses.add(qs);
            if (lane == 0) {
              mbar_arrive_expect_tx(&bars[kBarQFull + qs], kQBytes);
              for (int h = 0; h < 2; ++h)
                tc::tma_load_3d(sQ + qs * kQBytes + h * (kQBytes / 2), &tmap_q, 64 * h,
                                pc.g * kGroup, pc.q0 + (two ? i * kNodes : 0),
                                &bars[kBarQFull + qs]);
            }
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) {
      constexpr uint32_t n = M::kKStages;
      for (uint32_t i = issued < n ? 0 : issued - n; i < issued; ++i)
        if (!(withholds && i == 0))
          mbar_wait_bounded(&bars[kBarKFull + i % n], (i / n) & 1);
      for (int s = 0; s < 2; ++s)
        if (uses[s] > 0) mbar_wait_bounded(&bars[kBarQFull + s], (uses[s] - 1) & 1);
    }
    __syncwarp();
  } else if (warp == kScoreWarp || warp == kOutWarp) {
    // ================= MMA issue: S = Q K^T by one warp, O += P V by the other =================
    // Each whole warp walks the units, so every operand stays uniform; one lane
    // issues.  Every lane tests one barrier, for the phase that its next use
    // needs, and a unit waits for those in a mask: a test takes ~140 cycles, and
    // what a unit's issue takes bounds the tile.
    const bool leader = tc::elect_one();
    uint64_t *bar = bars;  // this lane's
    uint32_t parity = 0;
    uint32_t ready = 0;  // lanes whose barrier is known to be there
    auto poll = [&](uint32_t need) {
      for (uint32_t i = 0; (ready & need) != need; ++i) {
        ready = __ballot_sync(kFull, mbar_test_wait(bar, parity));
        const uint32_t limit = withholds && warp == kScoreWarp ? kTestSpins : kMaxSpins;
        if ((i & 255u) == 255u && (i >= limit || *abort_flag)) {
          if (!*abort_flag) flag_error(a.dev_error, K16V8_DEVERR_TIMEOUT);
          *abort_flag = 1;
          return false;
        }
      }
      tc::fence_after_sync();
      return true;
    };
    auto used = [&](uint32_t lanes) {
      parity ^= lanes >> lane & 1u;
      ready &= ~lanes;
    };
    Piece pc;
    Ring<kPieceRing> ring;
    bool ok = true;
    if (warp == kScoreWarp) {
      constexpr uint32_t kIdesc = tc::idesc_f16_f32(kRows, kKv / kParts, false, false);
      const uint64_t dk = tc::smem_desc_sw128(smem_addr(sK), 16, 1024);
      const uint32_t dk_lo = static_cast<uint32_t>(dk), d_hi = static_cast<uint32_t>(dk >> 32);
      const uint32_t dq_lo = dk_lo + (M::kQ >> 4) - (M::kK >> 4);
      // lane 0: the K stage; 1 + slot + 2 * part: P V of the S tile's last use
      // (the first passes); 5, 6: the query
      constexpr uint32_t kK = 1u, kPV = 2u, kQ = 32u;
      Ring<M::kKStages> kr;
      bar += lane == 0 ? kBarKFull : lane <= 4 ? kBarPV + lane - 1 : kBarQFull + (lane == 6);
      parity = lane >= 1 && lane <= 4;
      for (uint32_t p_idx = 0; ok && get_piece(pc, ring); ++p_idx) {
        const bool two = kWide && pc.n > kNodes;
        const int slots = two ? 2 : 1;
        const int q0 = kWide && !two ? p_idx & 1 : 0;  // the first slot's query
        const int tiles = pc.tiles;
        for (int t = 0; ok && t < tiles; ++t) {
#pragma unroll 1
          for (int part = 0; part < kParts; ++part) {
#pragma unroll 1
            for (int i = 0; i < slots; ++i) {
              const int w = two ? i : t & 1;
              const int tile = w + 2 * part;
              uint32_t need = kPV << tile;
              if (part == 0 && i == 0) need |= kK;
              if (t == 0 && part == 0) need |= kQ << (q0 + i);
              ok = poll(need);
              if (!ok) break;
              used(kPV << tile);
              const uint32_t a0 = dq_lo + (q0 + i) * (kQBytes / 16);
              const uint32_t b0 = dk_lo + kr.s * (kKStage / 16) + part * (kKBlk / kParts / 16);
              const uint32_t d = tmem + w * 128 + part * (kKv / kParts);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                if (leader)
                  tc::mma_f16_ss(d, a0 + (kk >> 2) * (kQBytes / 2 / 16) + (kk & 3) * 2, d_hi,
                                 b0 + (kk >> 2) * (kKBlk / 16) + (kk & 3) * 2, d_hi, kIdesc, kk > 0);
              if (leader) tc::mma_commit(&bars[kBarSFull + tile]);
            }
            if (!ok) break;
          }
          // (a stage whose copy did not land is not to be filled again: its barrier's
          // phase is still open)
          if (!ok) break;
          if (leader) tc::mma_commit(&bars[kBarKEmpty + kr.s]);
          kr.next();
          ready &= ~kK;
          if (lane == 0) {
            bar = &bars[kBarKFull + kr.s];
            parity = kr.phase;
          }
        }
        if (!ok) break;
        if (leader) tc::mma_commit(&bars[kBarQEmpty + q0]);
        if (leader && two) tc::mma_commit(&bars[kBarQEmpty + 1]);
        used(two ? 3 * kQ : kQ << q0);
      }
    } else {
      constexpr uint32_t kIdesc = tc::idesc_f16_f32(kRows, kHeadDim, false, true);
      constexpr int kHalves = 2 / kParts;  // of V, per part
      const uint64_t dv = tc::smem_desc_sw128(smem_addr(sV), kVBlk, 1024);
      const uint32_t dv_lo = static_cast<uint32_t>(dv), d_hi = static_cast<uint32_t>(dv >> 32);
      // lanes 0, 1: the V halves; 2 + slot + 2 * part: P; 6: the last piece's O
      // tiles have been read (the first passes)
      constexpr uint32_t kV = 1u, kP = 4u, kO = 64u;
      Ring<M::kVHalves> vr;
      bar += lane < 2 ? kBarVFull + lane : lane < 6 ? kBarPFull + lane - 2 : kBarOEmpty;
      parity = lane == 6;
      while (ok && get_piece(pc, ring)) {
        const bool two = kWide && pc.n > kNodes;
        const int slots = two ? 2 : 1;
        const int tiles = pc.tiles;
        for (int t = 0; ok && t < tiles; ++t) {
#pragma unroll 1
          for (int part = 0; part < kParts; ++part) {
            Ring<M::kVHalves> v1 = vr;
            if (kHalves == 2) v1.next();
#pragma unroll 1
            for (int i = 0; i < slots; ++i) {
              const int w = two ? i : t & 1;
              const int tile = w + 2 * part;
              uint32_t need = kP << tile;
              if (i == 0) need |= kHalves == 2 ? 3 * kV : kV;
              if (t == 0 && part == 0) need |= kO;
              ok = poll(need);
              if (!ok) break;
              used(kP << tile);
              const bool more_o = (two ? t : t >> 1) + part > 0;  // O is added to
              const uint32_t p0 = tmem + w * 128 + part * (kKv / kParts);
#pragma unroll
              for (int h = 0; h < kHalves; ++h) {
                const uint32_t b0 = dv_lo + (h ? v1.s : vr.s) * (kVHalf / 16);
#pragma unroll
                for (int kk = 0; kk < kHalf / 16; ++kk)
                  if (leader)
                    tc::mma_f16_ts(tmem + 256 + w * 128, p0 + (h * (kHalf / 16) + kk) * 8,
                                   b0 + kk * 128, d_hi, kIdesc, more_o || h + kk > 0);
                if (leader && i + 1 == slots) tc::mma_commit(&bars[kBarVEmpty + (h ? v1.s : vr.s)]);
              }
              if (leader) tc::mma_commit(&bars[kBarPV + tile]);
              // the slot's last of the piece
              if (leader && part == kParts - 1 && t + (two ? 1 : 2) >= tiles)
                tc::mma_commit(&bars[kBarODone + w]);
            }
            if (!ok) break;
            vr = v1;
            vr.next();
            if (kHalves == 2) {
              v1 = vr;
              v1.next();
            }
            ready &= ~(3 * kV);
            if (lane < 2) {
              bar = &bars[kBarVFull + (lane ? v1.s : vr.s)];
              parity = lane ? v1.phase : vr.phase;
            }
          }
        }
        used(kO);
      }
    }
    // every MMA issued has to land before tensor memory is released
    const int drain = kBarDrain + (warp == kOutWarp);
    if (leader) tc::mma_commit(&bars[drain]);
    mbar_wait_bounded(&bars[drain], 0);
    __syncwarp();
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tmem, kTmemCols);
}

}  // namespace tcore
}  // namespace tree
}  // namespace k16v8

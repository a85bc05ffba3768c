// Attention of several query rows over the K8/V8 cache on the tensor cores: the
// split kernel (see attention_k8v8.cu for the operators).
//
// One CTA per SM, all 512 columns of tensor memory.  The work is the flat list of
// tiles of attention_k8v8_plan.cuh, an equal range per CTA.
//
// The 4 query heads of the GQA group times 32 tokens are the 128 rows of an MMA
// tile (row = token * 4 + head).  Two score tiles S_0, S_1 and two output tiles
// O_0, O_1 (128 columns each; P, fp16, over the first half of its S columns) let
// one slot's softmax overlap the other's MMAs:
//  * groups of up to 32 tokens: one row tile; KV tiles alternate between slots 0
//    and 1, each with its own running max, sum and O, joined at the end of the
//    piece;
//  * larger groups: two row tiles, both over every KV tile.
// A unit is one (KV tile, slot): S = Q K^T (128 x 128 x 128), the row maximum, the
// exponentials in two parts of 64 positions, O += P V of either part.  Each slot
// has a warp that issues both products: MMAs of one thread execute in the order
// of their issue, so the next S may follow the P V that reads its columns without
// a wait between them.  (One part's S under the other's softmax, 64 columns each:
// 159 against 151 us for 8 x 1024.)
//
// Keys and values arrive as codes (TMA boxes of 2 KB, a page and head) with
// their pages' scales (4-byte asynchronous copies on the same barrier) in half
// tiles of 64 positions, and are widened to fp16 in the layouts the MMAs read: a
// code times a power of two in the cache's range is an fp16 number, so the MMAs
// see the cache's values exactly and nothing is scaled afterwards.  (The e4m3 MMA
// would take the codes as they are, but wants one scale for all positions of P V
// and P itself in e4m3: 2^-4 of a weight instead of 2^-11.)
//
// Warp roles (16 warps): 0-3 / 4-7 softmax of slot 0 / 1, one thread per row; 9 / 13
// issue the MMAs of slot 0 / 1; 10, 11 widen keys, 14, 15 values; 12 loads Q (TMA)
// and key pages; 8 loads value pages, walks the CTA's pieces and hands them to the
// others.  Every hand-off is an mbarrier, every wait is bounded.
//
// What bounds it.  With two row tiles: hand-offs and shared memory, not arithmetic.
// 1,024 rows of 8,192 take 143 us (1.13 PFLOP/s, 0.59 of the cuBLAS rate, tensor pipe
// 51% active), 2,140 cycles a unit, in which operands, codes and widened tiles move
// some 160 KB through shared memory (1,280 cycles); without the exponentials' ex2 it
// is 140, without the row maxima 142, without the widening's arithmetic 138.  In short
// pieces their starts and ends come to that: 8 x 1024 causal 120.5 us (713 TFLOP/s),
// 16 x 283 to 448 rows over 945 to 1,500 171 us (871).  With one row tile: the widening warps, at
// work 0.6 of the time, and the hand-offs on either side of them: 8 rows at 128K 115
// us (2.9 TB/s of codes, 0.43 of the copy rate); 5 rows over 1,500 13.2 us, nearly all
// of it the latency of one piece and the merge.
// Code size matters throughout: the roles' loops together are about as large as
// the instruction cache near the SM, and every variant below that added code lost
// more than it won.
// Measured and left out (us, against what was kept at the time): a thread's 128
// scores held in registers between maximum and exponentials (156 / 133: 56
// registers are left to the other roles), two warps to a row with 64 scores each
// (145 / 121.5: exchanging the maxima takes 500 cycles a unit), an epilogue that turns
// rows through shuffles (151 / 146) or tensor memory (144 / 132) to fill the lines it
// stores, queries loaded without holding up the key tiles behind them (132 / 122),
// widening by four warps per side instead of two, as neighbouring rows or as
// alternate halves (122 / 116 for 8 rows at 128K), a ring of codes and fp16 tiles for
// either slot (127 / 116).
#pragma once

#include "k16v8_device.cuh"
#include "tc_sm100.cuh"
#include "attention_k8v8_plan.cuh"

namespace k16v8 {
namespace attn8 {

constexpr unsigned kFull = 0xffffffffu;

constexpr int kRows = kTileTokens * kGroup;  // 128
constexpr int kHalf = kKv / 2;               // positions of a half tile
constexpr int kPagesPerHalf = kHalf / kPage; // 4
constexpr int kThreads = 512;
// Warps i, i + 4, .. share a scheduler.  The loads' warps share one, the MMAs' another,
// a widening warp of keys and one of values each of the others: 8 x 1024 122.3 us (with
// a widening warp beside an MMA warp 127 to 137, loads beside the MMAs or the widening
// 125.7), 8 rows at 128K 113.6 (with widening beside softmax warp 0, which has all the
// rows then, 122 to 123).
constexpr int kMmaWarp0 = 9, kMmaWarp1 = 13, kLoadVWarp = 8, kLoadKWarp = 12;
constexpr int kWidenWarps = 2;               // for keys, and for values
constexpr int kPieceRing = 4;
constexpr int kPieceReaders = 16;            // every warp
constexpr int kKTiles = 2;                   // fp16 tiles of keys
constexpr int kVHalves = 3;                  // fp16 half tiles of values

constexpr uint32_t kQBytes = kRows * 256;
constexpr uint32_t kStage = kHalf * 128;     // [64 pos][128] codes
constexpr uint32_t kVBlk = kHalf * 128;      // [64 pos][64 dims] fp16
constexpr uint32_t kVBytes = 2 * kVBlk;
constexpr uint32_t kKBlk = kKv * 128;        // [128 pos][64 dims] fp16
constexpr uint32_t kKBytes = 2 * kKBlk;
// registers, together what the block was launched with; 136 + 120 and 152 + 104 are
// 0.5% slower or no faster
constexpr int kSoftmaxRegs = 144, kOtherRegs = 112;
static_assert(kSoftmaxRegs + kOtherRegs == 2 * (65536 / kThreads), "two warpgroups each");

constexpr uint32_t kTmemCols = 512;  // S_0 [0,128) S_1 [128,256) O_0 [256,384) O_1 [384,512)

constexpr uint32_t kBarBytes = 512;

// kWide: groups of more than 32 tokens may be among the work.
template <bool kWide>
struct Smem {
  static constexpr int kQSlots = kWide ? 2 : 1;
  // of codes, keys and values each; what is left beside Q.  (8 rows at 128K: 3 121.3 us,
  // 4 118.4, 5 116.0)
  static constexpr int kStages = kWide ? 3 : 5;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kKst = kQ + kQSlots * kQBytes;
  static constexpr uint32_t kVst = kKst + kStages * kStage;
  static constexpr uint32_t kK = kVst + kStages * kStage;
  static constexpr uint32_t kV = kK + kKTiles * kKBytes;
  static constexpr uint32_t kBar = kV + kVHalves * kVBytes;
  static constexpr uint32_t kPieces = kBar + kBarBytes;
  static constexpr uint32_t kInfo = kPieces + kPieceRing * 56;
  static constexpr uint32_t kNan = kInfo + 16 * 4;   // new tokens with NaN value codes
  static constexpr uint32_t kStat = kNan + 4 * 8;    // [slot][max, sum][row]
  static constexpr uint32_t kScale = kStat + 2 * 2 * kRows * 4;  // [keys, values][stage][page]
  static constexpr uint32_t kBytes = kScale + 2 * kStages * kPagesPerHalf * 4;
  static_assert(kBytes <= 227 * 1024, "one CTA's shared memory");
  static_assert(sizeof(int64_t) * (kMaxBatch + 1) <= kBar, "the scan's scratch");
  static_assert(sizeof(int64_t) * 33 <= kBytes - kStat, "the scan's warp sums");
  static_assert(sizeof(Piece) <= 56 && kInfo % 8 == 0 && kNan % 8 == 0 && kStat % 16 == 0,
                "alignment");
};

enum {
  kBarQFull = 0,      // +slot
  kBarQEmpty = 2,     // +slot, 2 arrivals: of either slot's MMAs
  kBarKstFull = 4,    // +stage, 33 arrivals: the bytes' and one per lane for the scales
  kBarKstEmpty = 9,   // +stage, kWidenWarps arrivals
  kBarVstFull = 14,   // +stage, as for keys
  kBarVstEmpty = 19,  // +stage
  kBarKFull = 24,     // +tile, kWidenWarps arrivals
  kBarVFull = 26,     // +half, kWidenWarps arrivals
  kBarKEmpty = 29,    // +tile, 2 arrivals: both slots' MMAs have read it
  kBarVEmpty = 31,    // +half, as for keys
  kBarSFull = 34,     // +slot
  kBarPFull = 36,     // +slot + 2 * part, 4 arrivals (one per warp)
  kBarODone = 40,     // +slot: the slot's last P V of a piece (or it has none)
  kBarJoin = 43,      // 8 arrivals (one per warp): both slots' statistics are in shared memory
  kBarPiece = 44,     // +ring entry: described
  kBarTaken = 48,     // +ring entry: kPieceReaders arrivals
  kBarDrain = 52,     // +slot: every MMA
  kBarTurn = 54,      // +slot, 4 arrivals: the other slot's exponentials of a tile are done
  kBarOEmpty = 56,    // +slot, 8 arrivals: the O tile has been read (two by each warp of its
                      // slot, or with one row tile one by every warp)
  kNumBars = 58
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
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  bool wrapped = false;  // every stage has been used once
  __device__ __forceinline__ void next(int n) {
    if (++s == n) {
      s = 0;
      phase ^= 1;
      wrapped = true;
    }
  }
};

// Barriers by their shared address: 32 bits, and no conversion at every use.  (The
// roles' code shares an instruction cache that is short of it: every instruction
// in here that is spared counts.)
__device__ __forceinline__ bool test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(bar)
      : "memory");
}

// A wait that runs out raises the CTA-wide abort flag, which the others poll; every
// role leaves its loops on a failed wait, and the flag becomes
// K16V8_DEVERR_TIMEOUT at the end of the kernel.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity,
                                              volatile int *abort_flag) {
  for (uint32_t i = 0; !try_wait(bar, parity); ++i) {
    if (i & 1023u) continue;
    if (*abort_flag) return false;
    if (i >= kMaxPolls) {
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

// 64 columns from the one `rel` behind the first new token, for a row that sees the
// new tokens of m.
__device__ __forceinline__ uint64_t visible(int rel, uint64_t m) {
  if (rel <= -64) return ~0ull;
  if (rel >= 64) return 0ull;
  if (rel < 0) return ((1ull << -rel) - 1) | m << -rel;
  return m >> rel;
}

// Entry `page` of a piece's block table (anything behind the last position).
__device__ __forceinline__ int table_entry(const Args &a, const Piece &p, int page) {
  int id = -1;
  if (page * kPage < p.L) id = __ldg(a.block_table + static_cast<int64_t>(p.b) * a.maxp + page);
  return id;
}

// Registers of a thread of this warpgroup from here on.
template <int n>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(n));
}
template <int n>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(n));
}

// A 4-byte asynchronous copy, and this thread's arrival when its copies so far are
// there (the barrier's count includes it).
__device__ __forceinline__ void copy4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void arrive_behind_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// 16 codes times a scale, as fp16.
__device__ __forceinline__ void widen16(const uint4 &raw, __half2 scale, uint4 &lo, uint4 &hi) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 a = __hmul2(e4m3x2_to_half2(static_cast<uint16_t>(w[i] & 0xffffu)), scale);
    const __half2 b = __hmul2(e4m3x2_to_half2(static_cast<uint16_t>(w[i] >> 16)), scale);
    h[2 * i] = *reinterpret_cast<const uint32_t *>(&a);
    h[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&b);
  }
  lo = make_uint4(h[0], h[1], h[2], h[3]);
  hi = make_uint4(h[4], h[5], h[6], h[7]);
}
// Where a lane of a widening warp finds and puts 16 codes.  Eight lanes take the
// same 16 dims of eight neighbouring positions: the codes are staged with the
// 128-byte swizzle and the fp16 tile has it too, so they meet in no bank on either
// side, and every step of eight positions is a constant further.
struct Lanes {
  uint32_t from, to0, to1;
  __device__ __forceinline__ Lanes(int rank, int lane, uint32_t blk) {
    const uint32_t row = lane & 7, c = rank * 4 + (lane >> 3);  // dims 16c .. 16c + 15
    from = row * 128 + ((c ^ row) << 4);
    const uint32_t to = (c >> 2) * blk + row * 128, pair = (c & 3) * 2;
    to0 = to + ((pair ^ row) << 4);
    to1 = to + (((pair + 1) ^ row) << 4);
  }
};

__device__ __forceinline__ void put16(uint8_t *half, const Lanes &at, int step, const uint4 &raw,
                                      float scale) {
  uint4 lo, hi;
  widen16(raw, __float2half2_rn(scale), lo, hi);
  *reinterpret_cast<uint4 *>(half + step * 1024 + at.to0) = lo;
  *reinterpret_cast<uint4 *>(half + step * 1024 + at.to1) = hi;
}
// A half tile, every position of it: scales of its four pages at sc.
__device__ __forceinline__ void widen_half(uint8_t *half, const uint8_t *from, const Lanes &at,
                                           const float *sc) {
#pragma unroll 1
  for (int i0 = 0; i0 < 8; i0 += 2) {  // two pages
    uint4 raw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) raw[i] = *reinterpret_cast<const uint4 *>(from + (i0 + i) * 1024);
#pragma unroll
    for (int i = 0; i < 2; ++i) put16(half, at, i0 + i, raw[i], sc[(i0 + i) >> 1]);
  }
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

// p = 2^(s * scale - m) of n scores to tensor memory, their sum in fp32; m is
// kLift below a maximum of the row.  P is rounded to fp16, the type of V's
// tile: an MMA takes both operands in one type, and bf16 would round P eight
// times as coarsely.  That is 2^-11 of a weight down to 2^-21 of the row's
// largest; a smaller one is subnormal and off by up to 2^-32 of the largest,
// which the row's sum, in fp32, does not share: L positions put O off by at
// most L 2^-32 max|v|.  (Without the lift, L 2^-25: a score 17 above a flat tail
// of 131,072 positions loses 0.24% of the output; the lift takes no instruction
// per weight.)
template <bool kMask, int n>
__device__ __forceinline__ void exp_chunk(uint32_t t_p, const uint32_t (&s)[n], uint32_t seen,
                                          float2 scale, float2 neg_m, float2 &sum) {
  uint32_t pk[n / 2];
#pragma unroll
  for (int e = 0; e < n / 2; ++e) {
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
  if constexpr (n == 32)
    tc::tmem_st16(t_p, pk);
  else
    tc::tmem_st8(t_p, pk);
}

// 32 bytes of a lane in one store where the address allows: every lane's row is a
// line of its own, so stores take the time of their lines.
__device__ __forceinline__ void store32(__half *p, const uint32_t (&x)[8]) {
  if (reinterpret_cast<uintptr_t>(p) & 31) {
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(x[4], x[5], x[6], x[7]);
  } else {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]),
                 "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  }
}

// kTest: the form of the bounded-wait test hook.  CTA 0 withholds K of its first
// tile (no arrival, nothing in flight), so the score warp's wait for it runs out
// after kTestSpins polls and every role takes the abort path.
template <bool kWide, bool kTest>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(
    const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
    const __grid_constant__ CUtensorMap tmap_v, const Args a) {
  using M = Smem<kWide>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *sQ = smem_raw + M::kQ;
  uint8_t *sKst = smem_raw + M::kKst;
  uint8_t *sVst = smem_raw + M::kVst;
  uint8_t *sK = smem_raw + M::kK;
  uint8_t *sV = smem_raw + M::kV;
  float *scale_k = reinterpret_cast<float *>(smem_raw + M::kScale);
  float *scale_v = scale_k + M::kStages * kPagesPerHalf;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem_raw + M::kBar);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kNumBars);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + kNumBars) + 1;
  Piece *pieces = reinterpret_cast<Piece *>(smem_raw + M::kPieces);
  // rejected pages of a tile: for the softmax (by tile, 8 of them) and for the
  // values (by stage)
  volatile uint32_t *info = reinterpret_cast<volatile uint32_t *>(smem_raw + M::kInfo);
  volatile uint32_t *info_v = info + 8;
  uint32_t *nan_rows = reinterpret_cast<uint32_t *>(smem_raw + M::kNan);  // [4][2], by piece
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
    tc::prefetch_tensormap(&tmap_v);
  }
  if (warp == 0) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  if (warp == 1) {
    for (int i = lane; i < kNumBars; i += 32) {
      uint32_t count = 1;
      if ((i >= kBarKstFull && i < kBarKstEmpty) || (i >= kBarVstFull && i < kBarVstEmpty)) count = 33;
      if ((i >= kBarKstEmpty && i < kBarVstFull) || (i >= kBarVstEmpty && i < kBarKEmpty))
        count = kWidenWarps;
      if (i >= kBarPFull && i < kBarODone) count = 4;
      if ((i >= kBarQEmpty && i < kBarKstFull) || (i >= kBarKEmpty && i < kBarSFull)) count = 2;
      if (i >= kBarTurn && i < kBarOEmpty) count = 4;
      if (i == kBarJoin) count = 8;
      if (i >= kBarOEmpty) count = 8;
      if (i >= kBarTaken && i < kBarDrain) count = kPieceReaders;
      mbar_init(&bars[i], count);
    }
    if (lane == 0) *abort_flag = 0;
    fence_barrier_init();
  }
  pdl_wait();
  if (tid == kLoadVWarp * 32) a.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
  // ---- this CTA's range of the work (scratch: the operand stages) ----
  const Range range = plan_range(a, reinterpret_cast<int64_t *>(smem_raw),
                                 reinterpret_cast<int64_t *>(smem_raw + M::kStat));
  const bool work = range.lo < range.hi;  // uniform over the CTA
  const bool withholds = kTest && blockIdx.x == 0;
  fence_proxy_async();  // the scan's scratch becomes operand stages
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  const uint32_t bar0 = smem_addr(bars);
  auto wait = [&](int bar, uint32_t parity) {
    return wait_or_abort(bar0 + 8 * bar, parity, abort_flag);
  };
  // The next piece, for a whole warp; false at the end (or after an abort).
  auto get_piece = [&](Piece &pc, Ring &r) {
    if (!__all_sync(kFull, wait(kBarPiece + r.s, r.phase))) return false;
    pc = pieces[r.s];
    __syncwarp();
    if (lane == 0) arrive(bar0 + 8 * (kBarTaken + r.s));
    r.next(kPieceRing);
    return pc.tiles > 0;
  };

  if (warp < 8)
    more_registers<kSoftmaxRegs>();
  else
    fewer_registers<kOtherRegs>();
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
    Ring ring;
    uint32_t units = 0;             // of this slot so far
    uint32_t tiles = 0;             // of the CTA so far
    uint32_t joins = 0;             // pieces with one row tile, so far
    uint32_t turns = 0;             // tiles with two row tiles, so far
    bool ok = true;
    for (uint32_t p_idx = 0; ok; ++p_idx) {
      // the piece stays in shared memory: registers are short here
      if (!__all_sync(kFull, wait(kBarPiece + ring.s, ring.phase))) break;
      const Piece &pc = pieces[ring.s];
      if (pc.tiles == 0) break;
      const bool two = kWide && pc.n > kTileTokens;  // two row tiles
      const int token = (two ? w * kTileTokens : 0) + (r >> 2);
      const bool row_valid = token < pc.n;
      const bool warp_live = (two ? w * kTileTokens : 0) + (warp & 3) * 8 < pc.n;
      // the new tokens this row sees: itself and those before it
      const uint64_t mask_word = a.causal && row_valid ? ~0ull >> (63 - token) : 0;
      const int after = two ? 0 : w ^ pc.turn;  // the slot's first tile
      const int mine = two ? pc.tiles : (pc.tiles + 1 - after) / 2;
      const int n_tiles = pc.tiles, d0 = pc.base - pc.t0 * kKv;
      const int theirs = two ? 0 : (pc.tiles + after) / 2;  // units of the other slot to join
      float m_used = -INFINITY, l = 0.f;
      for (int k = 0; k < mine; ++k, ++units) {
        ok = __all_sync(kFull, wait(kBarSFull + w, units & 1));
        if (!ok) break;
        const int tile = two ? k : 2 * k + after;
        const int parts = pc.halves(tile);
        if (!warp_live) {
          if (lane == 0) {
            arrive(bar0 + 8 * (kBarPFull + w));
            if (parts > 1) arrive(bar0 + 8 * (kBarPFull + w + 2));
          }
          if (two) {
            ok = __all_sync(kFull, wait(kBarTurn + w, (turns++ + 1 - w) & 1));
            if (!ok) break;
            if (lane == 0) arrive(bar0 + 8 * (kBarTurn + (w ^ 1)));
          }
          continue;
        }
        tc::fence_after_sync();
        const int d = d0 - tile * kKv;  // columns of this tile that every row sees
        const uint32_t bad = info[(tiles + tile) & 7];
        const uint32_t tSp = tS + lane_base;
        // pass 1: row max
        float rmax = -INFINITY;
        bool need_mask = d < kKv;
        if (!need_mask) {
#pragma unroll 1
          for (int c = 0; c < 4; c += 2) {
            uint32_t s0[32], s1[32];
            float m0, m1;
            tc::tmem_ld32_max(tSp + c * 32, s0, m0);
            tc::tmem_ld32_max(tSp + c * 32 + 32, s1, m1);
            tc::tmem_wait_ld();
            keep(s0);
            keep(s1);
            rmax = fmaxf(rmax, fmaxf(m0, m1));
          }
          need_mask = bad != 0;  // (seldom; its load took place meanwhile)
        }
        uint64_t seen_lo = 0, seen_hi = 0;
        if (need_mask) {
          seen_lo = visible(-d, mask_word);
          seen_hi = visible(kHalf - d, mask_word);
          for (uint32_t pages = bad; pages; pages &= pages - 1) {
            const int page = __ffs(static_cast<int>(pages)) - 1;
            const uint64_t out = 0xffffull << (page & 3) * 16;
            if (page < 4)
              seen_lo &= ~out;
            else
              seen_hi &= ~out;
          }
          rmax = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t s0[32];
            tc::tmem_ld32(tSp + c * 32, s0);
            tc::tmem_wait_ld();
            const uint32_t v = static_cast<uint32_t>((c & 2 ? seen_hi : seen_lo) >> (c & 1) * 32);
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
        // (S was issued behind the slot's P V so far: O is at rest)
        if (k > 0 && __any_sync(kFull, alpha != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            tc::tmem_ld16(tO + lane_base + c * 16, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc::tmem_st16(tO + lane_base + c * 16, o);
          }
        }
        // The slots of two row tiles exponentiate in turn, one under the other's MMAs,
        // or both would wait for both.  1,024 rows of 8,192 158.8 -> 143 us, 16 x 283
        // to 448 over 945 to 1,500 186.6 -> 178, 3,800 rows 201 -> 190; 64 x 20 to 40 of 150
        // to 300 42.6 -> 43.2.
        if (two) {
          ok = __all_sync(kFull, wait(kBarTurn + w, (turns++ + 1 - w) & 1));
          if (!ok) break;
        }
        // pass 2: p = 2^(s * scale - m), fp32 row sum, P (fp16) over the S columns read
        const float neg = m_used == -INFINITY ? 0.f : -m_used;
        const float2 sc2 = make_float2(qk_scale, qk_scale);
        const float2 nm2 = make_float2(neg, neg);
        float2 ps2 = make_float2(0.f, 0.f);
        auto hand_over = [&](int part) {
          tc::tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) arrive(bar0 + 8 * (kBarPFull + w + 2 * part));
        };
        if (!need_mask) {  // 32 columns are on their way while 32 are worked on
          uint32_t s0[32], s1[32];
          tc::tmem_ld32(tSp, s0);
          tc::tmem_wait_ld();
#pragma unroll 1
          for (int part = 0; part < 2; ++part) {
            const uint32_t at = tSp + part * kHalf;
            tc::tmem_ld32(at + 32, s1);
            exp_chunk<false>(at, s0, 0, sc2, nm2, ps2);
            tc::tmem_wait_ld();
            tc::tmem_ld32(tSp + kHalf, s0);  // (the second time unused)
            exp_chunk<false>(at + 16, s1, 0, sc2, nm2, ps2);
            tc::tmem_wait_ld();
            hand_over(part);
          }
        } else {
#pragma unroll 1
          for (int part = 0; part < parts; ++part) {
            const uint32_t at = tSp + part * kHalf;
            const uint64_t seen = part ? seen_hi : seen_lo;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t s0[16];
              tc::tmem_ld16(at + c * 16, s0);
              tc::tmem_wait_ld();
              exp_chunk<true>(at + c * 8, s0, static_cast<uint32_t>(seen >> c * 16), sc2, nm2, ps2);
            }
            hand_over(part);
          }
        }
        if (two && lane == 0) arrive(bar0 + 8 * (kBarTurn + (w ^ 1)));
        l = l * alpha + (ps2.x + ps2.y);
      }
      if (!ok) break;
      tiles += n_tiles;
      // ---- end of the piece: this slot's O, and with one row tile the other's ----
      ok = __all_sync(kFull, wait(kBarODone + w, p_idx & 1));
      if (!ok) break;
      tc::fence_after_sync();
      const int pn = (p_idx & 3) * 2;
      const uint64_t nan_mask = nan_rows[pn] | static_cast<uint64_t>(nan_rows[pn + 1]) << 32;
      float f_own = 1.f, f_other = 0.f;
      float m_all = m_used, l_all = l;
      if (!two) {
        // (the last piece's have been read: this one's O was written after that)
        stat[(w * 2 + 0) * kRows + r] = m_used;
        stat[(w * 2 + 1) * kRows + r] = l;
        __syncwarp();
        if (lane == 0) arrive(bar0 + 8 * (kBarJoin));
        // (the other slot's warps are in this piece, so its phase before is over)
        ok = __all_sync(kFull, wait(kBarJoin, joins++ & 1)) &&
             __all_sync(kFull, wait(kBarODone + (w ^ 1), p_idx & 1));
        if (!ok) break;
        tc::fence_after_sync();
        const float m_o = stat[((w ^ 1) * 2 + 0) * kRows + r];
        const float l_o = stat[((w ^ 1) * 2 + 1) * kRows + r];
        m_all = fmaxf(m_used, m_o);
        // (a slot whose scores were all NaN keeps max -inf: its NaN sum decides)
        f_own = m_used == -INFINITY ? (l != l ? l : 0.f) : ex2(m_used - m_all);
        f_other = m_o == -INFINITY ? (l_o != l_o ? l_o : 0.f) : ex2(m_o - m_all);
        l_all = f_own * l + f_other * l_o;
      }
      const bool dead = !(l_all > 0.f) && l_all == l_all;  // the row sees nothing
      const float inv = dead ? 0.f : __fdividef(1.f, l_all);
      // (the lift is taken off the sum, whose logarithm is most accurate near 1)
      const float lse =
          dead ? -INFINITY : ((m_all + kLift) + lg2(l_all * 0x1p-7f)) * kLn2;
      static_assert(kLift == 7.f, "the factor of l_all");
      const float g_own = f_own * inv, g_other = f_other * inv;
      // with one row tile, slot w's warps write dims 64w .. 64w + 63 of every row
      const int c_lo = two ? 0 : 4 * w, c_hi = two ? 8 : 4 * w + 4;  // 16 dims each
      const int row = (two ? w * kRows : 0) + r;  // of the segment
      const int64_t orow = static_cast<int64_t>(pc.q0 + token) * hq + pc.g * kGroup + (r & 3);
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
          if (row_valid && whole) {
            uint32_t pk[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const __half2 hh = __floats2half2_rn(o[2 * e], o[2 * e + 1]);
              pk[e] = *reinterpret_cast<const uint32_t *>(&hh);
            }
            store32(po + 16 * c, pk);
          } else if (row_valid) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              pp[static_cast<int64_t>(4 * c + q) * a.max_rows] =
                  make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          }
        }
        // (seldom) NaN value codes of new tokens this row sees, over what was stored
        for (uint64_t nm = row_valid ? mask_word & nan_mask : 0; nm; nm &= nm - 1) {
          const int pos = pc.base + __ffsll(static_cast<long long>(nm)) - 1;
          const int page = __ldg(a.block_table + static_cast<int64_t>(pc.b) * a.maxp + pos / kPage);
          if (page < 0 || page >= a.num_pages) continue;
          const uint8_t *vr = a.v_cache + ((static_cast<int64_t>(page) * a.hkv + pc.g) * kPage +
                                           pos % kPage) * kHeadDim;
#pragma unroll 1
          for (int d = 16 * c_lo; d < 16 * c_hi; ++d) {
            if ((__ldg(vr + d) & 0x7f) != 0x7f) continue;
            if (whole)
              po[d] = __ushort_as_half(0x7fff);
            else
              reinterpret_cast<float *>(pp + static_cast<int64_t>(d >> 2) * a.max_rows)[d & 3] = NAN;
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
        arrive(bar0 + 8 * (kBarOEmpty + w));  // O is read: the next piece may write it
        arrive(bar0 + 8 * (kBarOEmpty + (two ? w : w ^ 1)));
        arrive(bar0 + 8 * (kBarTaken + ring.s));
      }
      ring.next(kPieceRing);
    }
    pdl_launch_dependents();
  } else if (warp & 2) {
    // ================= codes to fp16: two warps for keys, two for values =================
    // (one code for both: the instruction cache holds little more than the roles' loops)
    const bool is_v = warp & 4;
    const Lanes at(warp & 1, lane, is_v ? kVBlk : kKBlk);
    const int bar_staged = is_v ? kBarVstFull : kBarKstFull, bar_read = is_v ? kBarVstEmpty : kBarKstEmpty;
    const int bar_full = is_v ? kBarVFull : kBarKFull, bar_empty = is_v ? kBarVEmpty : kBarKEmpty;
    const uint8_t *stages = is_v ? sVst : sKst;
    uint8_t *tiles = is_v ? sV : sK;
    const uint32_t tile_bytes = is_v ? kVBytes : kKBytes;
    const float *scales = is_v ? scale_v : scale_k;
    Piece pc;
    Ring ring, src, dst;
    bool ok = true;
    for (uint32_t p_idx = 0; ok && get_piece(pc, ring); ++p_idx) {
#pragma unroll 1
      for (int h = 2 * pc.t0; h < pc.h1; ++h) {
        ok = __all_sync(kFull, wait(bar_staged + src.s, src.phase));
        if (!ok) break;
        // a tile of keys is filled half by half, values are handed over by halves
        if ((is_v || !(h & 1)) && dst.wrapped)
          ok = __all_sync(kFull, wait(bar_empty + dst.s, dst.phase ^ 1));
        if (!ok) break;
        const int live = pc.L - h * kHalf;      // positions of the half that are seen
        const int fresh = pc.base - h * kHalf;  // those from here on are new tokens
        const uint32_t bad = is_v ? info_v[src.s] : 0;
        const float *sc = scales + src.s * kPagesPerHalf;
        uint8_t *half = tiles + dst.s * tile_bytes + (is_v ? 0 : (h & 1) * kVBlk);
        const uint8_t *from = stages + src.s * kStage + at.from;
        // (keys that are not seen are masked as scores, whatever is stored there)
        if (!is_v || (fresh >= kHalf && !bad)) {
          widen_half(half, from, at, sc);
        } else {
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            const int pos = 8 * i + (lane & 7), page = pos >> 4;
            uint4 raw = make_uint4(0, 0, 0, 0);  // what is not seen may hold anything, NaN too
            float scale = 0.f;
            if (pos < live && !(bad >> page & 1)) {
              raw = *reinterpret_cast<const uint4 *>(from + i * 1024);
              scale = sc[page];
              if (pos >= fresh) {  // NaN codes must not reach rows that do not see them
                const uint32_t n0 = nan_bytes(raw.x), n1 = nan_bytes(raw.y),
                               n2 = nan_bytes(raw.z), n3 = nan_bytes(raw.w);
                if (n0 | n1 | n2 | n3) {
                  raw = make_uint4(raw.x & ~n0, raw.y & ~n1, raw.z & ~n2, raw.w & ~n3);
                  const int rel = pos - fresh;
                  atomicOr(&nan_rows[(p_idx & 3) * 2 + (rel >> 5)], 1u << (rel & 31));
                }
              }
            }
            put16(half, at, i, raw, scale);
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) arrive(bar0 + 8 * (bar_read + src.s));
        src.next(M::kStages);
        if (is_v || (h & 1) || h + 1 == pc.h1) {
          if (lane == 0) arrive(bar0 + 8 * (bar_full + dst.s));
          dst.next(is_v ? kVHalves : kKTiles);
        }
      }
    }
  } else if (warp == kLoadVWarp || warp == kLoadKWarp) {
    // ================= loads; V's: the CTA's pieces, K's: the queries =================
    // V's lane 0 walks the pieces: the first at the start, the next one behind the
    // copies of a piece's first half tile.
    const bool is_v = warp == kLoadVWarp;
    const int bar_staged = is_v ? kBarVstFull : kBarKstFull, bar_read = is_v ? kBarVstEmpty : kBarKstEmpty;
    const CUtensorMap *map = is_v ? &tmap_v : &tmap_k;
    const uint32_t stages = smem_addr(is_v ? sVst : sKst);
    const uint32_t scales = smem_addr(is_v ? scale_v : scale_k);
    const float *pool_scales = a.kv_scale + is_v;
    Walker walker;
    Ring ring, dst, described;
    bool more = true;
    if (is_v && lane == 0) walker.init(a, range);
    Piece pc;
    uint32_t issued = 0;
    Pair uses;  // of the query buffers
    bool ok = true;
    uint32_t p_idx = 0, tiles = 0;
    int h = 0;
    // page ids of eight half tiles, a lane each, and of the eight behind: their loads
    // take longer than a step
    int ids = -1, ids_next = -1;
    pc.t0 = pc.h1 = 0;
    bool start = true;  // a description is due (V), at the start and behind a first tile
    while (true) {
      if (start) {
        bool done = true;
        if (is_v && lane == 0 && more) {
          done = !described.wrapped || wait(kBarTaken + described.s, described.phase ^ 1);
          if (done) {
            Piece p;
            more = walker.next(a, range, p);
            if (!more) p.tiles = 0;  // the end
            pieces[described.s] = p;
            nan_rows[2 * described.s] = nan_rows[2 * described.s + 1] = 0;  // (a ring like the pieces')
            arrive(bar0 + 8 * (kBarPiece + described.s));
            described.next(kPieceRing);
          }
        }
        start = false;
        ok = __all_sync(kFull, done);
        if (!ok) break;
      }
      if (h == pc.h1) {
        if (!get_piece(pc, ring)) break;
        h = 2 * pc.t0;
        ids = table_entry(a, pc, h * kPagesPerHalf + lane);
        ids_next = table_entry(a, pc, h * kPagesPerHalf + 32 + lane);
      }
      if (dst.wrapped) ok = __all_sync(kFull, wait(bar_read + dst.s, dst.phase ^ 1));
      if (!ok) break;
      const int at = (h - 2 * pc.t0) & 7;
      int pid = __shfl_sync(kFull, ids, at * kPagesPerHalf + (lane & 3));
      // -2: behind the last position (and lanes without a page), -1: outside the pool
      if (lane >= kPagesPerHalf || (h * kPagesPerHalf + lane) * kPage >= pc.L)
        pid = -2;
      else if (pid < 0 || pid >= a.num_pages)
        pid = -1;
      const uint32_t bad = __ballot_sync(kFull, pid == -1);
      const uint32_t bytes = __popc(__ballot_sync(kFull, pid >= 0)) * 2048u;
      const bool withheld = withholds && !is_v && issued == 0;
      if (lane == 0) {
        if (is_v) {
          if (bad) flag_error(a.dev_error, K16V8_DEVERR_PAGE);
          info_v[dst.s] = bad;
        } else if (h & 1) {
          if (bad) info[tiles & 7] |= bad << kPagesPerHalf;
        } else {
          info[tiles & 7] = bad;
        }
        if (!withheld) arrive_expect(bar0 + 8 * (bar_staged + dst.s), bytes);
      }
      __syncwarp();
      if (!withheld) {
        if (pid >= 0) {
          const int tile = pid * a.hkv + pc.g;
          load_box(stages + dst.s * kStage + lane * 2048, map, tile * kPage,
                   bar0 + 8 * (bar_staged + dst.s));
          copy4(scales + dst.s * (kPagesPerHalf * 4) + lane * 4,
                pool_scales + 2 * static_cast<int64_t>(tile));
        }
        arrive_behind_copies(bar0 + 8 * (bar_staged + dst.s));
      }
      // (K: the first tile's copies are out, whose loads do not wait for the queries')
      const bool first = h == (is_v ? 2 * pc.t0 : min(2 * pc.t0 + 1, pc.h1 - 1));
      ++h;
      if (!(h & 1) || h == pc.h1) ++tiles;
      if (at == 7) {
        ids = ids_next;
        ids_next = table_entry(a, pc, (h + 8) * kPagesPerHalf + lane);
      }
      __syncwarp();
      dst.next(M::kStages);
      ++issued;
      if (first) {
        start = true;
        if (!is_v) {  // the query, behind the first tile's copies
          const bool two = kWide && pc.n > kTileTokens;
          for (int i = 0; ok && i < (two ? 2 : 1); ++i) {
            const int qs = two ? i : (kWide ? p_idx & 1 : 0);
            if (uses[qs] > 0) ok = __all_sync(kFull, wait(kBarQEmpty + qs, (uses[qs] - 1) & 1));
            if (!ok) break;
            uses.add(qs);
            if (lane == 0) {
              arrive_expect(bar0 + 8 * (kBarQFull + qs), kQBytes);
              for (int h = 0; h < 2; ++h)
                tc::tma_load_3d(sQ + qs * kQBytes + h * (kQBytes / 2), &tmap_q, 64 * h,
                                pc.g * kGroup, pc.q0 + (two ? i * kTileTokens : 0),
                                &bars[kBarQFull + qs]);
            }
          }
          if (!ok) break;
          ++p_idx;
          __syncwarp();
        }
      }
    }
    // let the copies issued last land before shared memory is released
    if (lane == 0) {
      constexpr uint32_t n = M::kStages;
      for (uint32_t i = issued < n ? 0 : issued - n; i < issued; ++i)
        if (!(withholds && !is_v && i == 0))
          mbar_wait_bounded(&bars[bar_staged + i % n], (i / n) & 1);
      for (int s = 0; s < 2; ++s)
        if (uses[s] > 0) mbar_wait_bounded(&bars[kBarQFull + s], (uses[s] - 1) & 1);
    }
    __syncwarp();
  } else if (warp == kMmaWarp0 || warp == kMmaWarp1) {
    // ================= MMA issue for slot w: O += P V, then the next S = Q K^T =================
    // The MMAs of one thread execute in the order of their issue, so an S may follow
    // the P V that reads the same columns without waiting for it.  The whole warp
    // walks the units, so every operand stays uniform; one lane issues.  Every lane
    // tests one barrier, for the phase that its next use needs, and a unit waits for
    // those in a mask: a test takes ~140 cycles.
    // A test tells a phase from the one before or behind it by parity alone, so the
    // barrier must be in that phase or have completed it and no other.  Half tiles:
    // the slots take turns over tiles with one row tile, so of any two tiles in a
    // row one at least is the slot's, and a half implies those before it; its stage
    // is not filled again before the slot has released it.  Queries and O tiles: a
    // slot without a tile of a piece waits and arrives for that piece all the same.
    const int w = warp == kMmaWarp1;
    const bool leader = tc::elect_one();
    // lane 0: the K tile; 1: the V half; 2, 3: P of either part; 4, 5: the queries;
    // 6: the last piece's O tiles have been read (the first passes)
    constexpr uint32_t kK = 1u, kV = 2u, kP = 4u, kQ = 16u, kO = 64u;
    uint32_t bar = bar0 + 8 * (lane == 0   ? kBarKFull
                               : lane == 1 ? kBarVFull
                               : lane < 4  ? kBarPFull + w + 2 * (lane - 2)
                               : lane < 6  ? kBarQFull + lane - 4
                                           : kBarOEmpty + w);
    uint32_t parity = lane == 6;
    uint32_t ready = 0;  // lanes whose barrier is known to be there
    const uint32_t limit = withholds ? kTestSpins : kMaxSpins;
    auto poll = [&](uint32_t need) {
      for (uint32_t i = 0; (ready & need) != need; ++i) {
        ready = __ballot_sync(kFull, test_wait(bar, parity));
        if ((i & 255u) == 255u && (i >= limit || *abort_flag)) {
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
    // the tile of keys and the half of values to come, and on to the one behind
    int k_at = 0, v_at = 0;
    auto next_k = [&]() {
      if (lane == 0) {
        bar = k_at ? bar - 8 : bar + 8;
        parity ^= k_at;
      }
      k_at ^= 1;
      ready &= ~kK;
    };
    static_assert(kKTiles == 2, "next_k");
    auto next_v = [&]() {
      const bool wrap = v_at == kVHalves - 1;
      v_at = wrap ? 0 : v_at + 1;
      if (lane == 1) {
        bar = wrap ? bar - 8 * (kVHalves - 1) : bar + 8;
        parity ^= wrap;
      }
      ready &= ~kV;
    };
    constexpr uint32_t kIdescS = tc::idesc_f16_f32(kRows, kKv, false, false);
    constexpr uint32_t kIdescO = tc::idesc_f16_f32(kRows, kHeadDim, false, true);
    const uint64_t dk = tc::smem_desc_sw128(smem_addr(sK), 16, 1024);
    const uint64_t dv = tc::smem_desc_sw128(smem_addr(sV), kVBlk, 1024);
    const uint32_t dk_lo = static_cast<uint32_t>(dk), dk_hi = static_cast<uint32_t>(dk >> 32);
    const uint32_t dv_lo = static_cast<uint32_t>(dv), dv_hi = static_cast<uint32_t>(dv >> 32);
    const uint32_t dq_lo = dk_lo + (M::kQ >> 4) - (M::kK >> 4);
    const uint32_t tS = tmem + w * 128, tO = tmem + 256 + w * 128;

    // A step is the P V of a tile's two parts and the S of the slot's next tile: at
    // the start there is no P V, at the end no S, and where the next piece holds no
    // tile of the slot they are apart.
    Piece pc;
    Ring ring;
    uint32_t p_idx = 0;
    int t = 0, tiles = 0, t_first = 0, q = 0;  // of the piece whose S are issued
    uint32_t q_need = 0;
    bool two = false, more = true, pass = false;
    int v_skip = 0;       // halves of the other slot that do
    bool o_on = false, o_first = false, o_last = false, o_two = false;  // the tile before
    int o_skip = 0, o_parts = 0;
    bool ok = true;
    while (ok) {
      bool s_on = t < tiles;
      if (!s_on && more && !pass) {
        more = get_piece(pc, ring);
        if (more) {
          two = kWide && pc.n > kTileTokens;
          tiles = pc.tiles;
          t = t_first = two ? 0 : w ^ pc.turn;
          q = two ? w : kWide ? p_idx & 1 : 0;
          q_need = two ? 3 * kQ : kQ << q;
          ++p_idx;
          if (t_first) {
            next_k();
            v_skip += pc.halves(0);
          }
          s_on = t < tiles;
          pass = !s_on;  // one tile, the other slot's
        }
      }
      if (!s_on && !o_on && !pass) break;
      for (; o_skip > 0; --o_skip) next_v();
#pragma unroll 1
      for (int op = 0; op <= o_parts; ++op) {
        if (op < o_parts) {  // P V of a part
          const uint32_t need = kV | kP << op | (o_first && op == 0 ? kO : 0u);
          ok = poll(need);
          if (!ok) break;
          const uint32_t b0 = dv_lo + v_at * (kVBytes / 16), p0 = tS + op * kHalf;
          const bool add = !o_first || op > 0;  // else O is written
#pragma unroll
          for (int kk = 0; kk < kHalf / 16; ++kk)
            if (leader)
              tc::mma_f16_ts(tO, p0 + kk * 8, b0 + kk * 128, dv_hi, kIdescO, add || kk > 0);
          if (leader) {
            commit(bar0 + 8 * (kBarVEmpty + v_at));
            if (!o_two) arrive(bar0 + 8 * (kBarVEmpty + v_at));  // (the other slot does not read it)
            if (o_last && op + 1 == o_parts) commit(bar0 + 8 * (kBarODone + w));
          }
          used(need & ~kV);
          next_v();
        } else if (s_on) {
          ok = poll(t == t_first ? kK | q_need : kK);
          if (!ok) break;
          const uint32_t a0 = dq_lo + q * (kQBytes / 16), b0 = dk_lo + k_at * (kKBytes / 16);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            if (leader)
              tc::mma_f16_ss(tS, a0 + (kk >> 2) * (kQBytes / 2 / 16) + (kk & 3) * 2, dk_hi,
                             b0 + (kk >> 2) * (kKBlk / 16) + (kk & 3) * 2, dk_hi, kIdescS, kk > 0);
          if (leader) {
            commit(bar0 + 8 * (kBarSFull + w));
            commit(bar0 + 8 * (kBarKEmpty + k_at));
            if (!two) arrive(bar0 + 8 * (kBarKEmpty + k_at));
          }
          next_k();
        }
      }
      if (!ok) break;
      o_on = s_on;
      o_parts = 0;
      if (s_on) {
        o_two = two;
        o_first = t == t_first;
        o_parts = pc.halves(t);
        o_skip = v_skip;
        v_skip = 0;
        t += two ? 1 : 2;
        o_last = t >= tiles;
        if (!two && t <= tiles) {  // the other slot's tile behind it
          next_k();
          v_skip = pc.halves(t - 1);
        }
        if (o_last) {
          if (leader) {  // the queries have been read
            commit(bar0 + 8 * (kBarQEmpty + (two ? 0 : q)));
            if (two) commit(bar0 + 8 * (kBarQEmpty + 1));
          }
          used(q_need);
        }
      } else if (pass) {
        // (no wait with a P V due: the other slot's next pieces may depend on it)
        pass = false;
        tiles = 0;
        ok = poll(q_need);
        if (ok && leader) arrive(bar0 + 8 * (kBarQEmpty + q));
        ok = ok && poll(kO);
        used(q_need | kO);
        if (ok && leader) arrive(bar0 + 8 * (kBarODone + w));
      }
    }
    // every MMA issued has to land before tensor memory is released
    const int drain = kBarDrain + w;
    if (leader) commit(bar0 + 8 * (drain));
    mbar_wait_bounded(&bars[drain], 0);
    __syncwarp();
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tmem, kTmemCols);
  if (tid == 0 && *abort_flag) flag_error(a.dev_error, K16V8_DEVERR_TIMEOUT);
}

}  // namespace attn8
}  // namespace k16v8

// Load-balanced paged decode attention over the K8/V8 cache (E4M3 keys and
// values, a power-of-two scale per page and head for each).
//
// "Phi-4: quality transfer and interrupted throughput studies": the intro gives
// the geometry (40 query heads over 10 KV heads, d = 128) and the page pool;
// keys in 8 bits and scales per page are this library's.
//
// Mathematics.  With kappa, nu the scales of a page: scores sm_scale * kappa *
// (q . code_k), softmax over all positions, out = sum p * nu * code_v.  kappa is
// constant over a page, which is a warp's unit of work, and joins the score's
// factor.  nu multiplies the widened values, which is exact: a code times a scale
// of the cache's range is an fp16 number.  (It is not joined to the weight: in fp16
// the weights would have to be held against the largest nu of a run, and pages of
// small nu beside a page of large nu would lose their bits.  Pages' products scaled
// in fp32 behind the MMAs instead: registers spill, 1,024 sequences of 50 to 100
// positions 57 against 54 us.)
//
// The cut is that of the K16/V8 balanced decode (decode_balanced.cu): CTA i of one
// full wave takes flat (sequence, KV head, page) tiles [i W, (i + 1) W), and a merge
// joins the segments that were cut.  A warp takes a run of its CTA's tiles and writes
// the rows of segments that lie in it by itself; what warps share is joined once, at
// the end.
//
// HBM-bound: 4,096 bytes of codes and 8 of scales per tile.  What a tile costs in
// instructions decides whether the stream stays full (the K16/V8 kernel spends
// 544 on 6 KB), so both products are MMAs here:
//  * S = K q^T: the page's 16 tokens as M, the 4 heads padded to 8 as N, 16 dims
//    a step; codes are widened to fp16 pairs in registers.
//  * O^T += V^T p: 16 dims as M, the 16 tokens as K, heads as N.  A lane reads 16
//    dims of its 4 tokens, interleaves the bytes of two tokens (prmt) and widens
//    the pairs.  A weight, in fp16, is off by 2^-11 of itself, or by 2^-32 of the
//    row's largest where that is more, as in attention_k8v8.cuh.  The weights change
//    hands by two 8x8 transposes (movmatrix), and the accumulators' columns are the
//    heads whose scores the lane holds, so the rescale factors need no exchange.
//  * The running maximum moves only when a score exceeds it by 2^8: a tile
//    needs one vote instead of a reduction over its tokens.
// Tiles are staged by TMA with the 128-byte swizzle: a row is 128 bytes, and the
// lanes that read one column of 16-byte chunks would meet in the same banks.
// Both kernels: 16 sequences of 8.3K 58.5 us (5.8 TB/s of the bytes it cannot do
// without, 0.86 of the copy rate), one of 128K 58.2, 32 of 0.6K to 1.15K 18.9 (0.56),
// one of 1.1K 6.8, 1,024 of 50 to 100 54 (0.59; all of 100 70, 0.60), 8,192 of 20 to 40
// 273 (0.43; all of 40 304, 0.49).  Some 7 us are fixed: plan, first loads, the cut
// segments' merge.  (With value scales joined to the weights, which cost more than the
// products do now: warps that take a CTA's tiles in turn and join at the end of every
// segment 7.4 / 7.0 us for one of 1.1K, 70.6 / 54 for 1,024 of 50 to 100, 447 / 281 for
// 8,192 of 20 to 40, 0.5% less for the long ones.)
#include <math.h>

#include "k8v8_device.cuh"
#include "tensor_map.cuh"
#include "tc_sm100.cuh"

namespace k16v8 {
namespace decode8 {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr int kCtasPerSm = 4;
constexpr int kMinTiles = kWarps;   // at least one tile per warp
constexpr int kMaxBatch = 8192;     // the scan's page offsets live in the ring space
constexpr int kTile = k8v8::kTileBytes;
constexpr float kLift = 7.f, kSlack = 8.f;  // weights stay below 2^15

struct __align__(1024) Ring {  // one warp's
  uint8_t k[kStages][kTile];
  uint8_t v[kStages][kTile];
};
struct Stage {
  float4 o[kWarps - 1][8][16];     // [dims 16g + 2i, 2i + 1 of heads 2t, 2t + 1][2g + t]
  float m[kWarps - 1][kGroup], l[kWarps - 1][kGroup];
  uint64_t bar[kWarps][kStages];
  int32_t live[kWarps][kStages];   // slot holds a page (0: its id was rejected)
  int32_t aux[4];
};
constexpr size_t kSmemBytes = kWarps * sizeof(Ring) + sizeof(Stage);
static_assert(static_cast<size_t>(kMaxBatch + 1) * sizeof(int32_t) <= kWarps * sizeof(Ring),
              "scan scratch must fit in the ring space");

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t widen_lo(uint32_t w) {
  const __half2 h = e4m3x2_to_half2(static_cast<uint16_t>(w & 0xffffu));
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) {
  const __half2 h = e4m3x2_to_half2(static_cast<uint16_t>(w >> 16));
  return *reinterpret_cast<const uint32_t *>(&h);
}
// Two fp16 times a scale.
__device__ __forceinline__ uint32_t times(uint32_t x, __half2 s) {
  const __half2 h = __hmul2(*reinterpret_cast<const __half2 *>(&x), s);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void tma_load_evict_first(void *dst, const CUtensorMap *map, int y,
                                                     uint64_t *bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

__device__ __forceinline__ int clamped_len(const int32_t *seq_lens, int b, int cap) {
  return max(0, min(__ldg(seq_lens + b), cap));
}

// A warp's running state, lane 4g + t: heads 2t and 2t + 1 (t < 2; the padding
// heads of the others hold zeros).  m is kLift below a maximum of the scores so
// far, l the sum over the lane's tokens, o the 16 dims from 16g.
struct State {
  float m[2], l[2];
  float o[8][4];  // dims 16g + 2i (heads 2t, 2t + 1), 16g + 2i + 1
  __device__ __forceinline__ void reset() {
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  }
};

// Folds one staged page, its first `valid` tokens, into the state.  qf: lane 4g +
// t holds dims 32t .. 32t + 31 of head g; qs = sm_scale * log2(e) * kappa.
__device__ __forceinline__ void attend(const uint8_t *kp, const uint8_t *vp, int valid,
                                       const uint32_t (&qf)[16], float qs, float nu, State &st) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // ---- scores of tokens g, g + 8 ----
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = g * kHeadDim + (((2 * t + i) ^ g) << 4);  // chunk 2t + i of the row
    const uint4 a = *reinterpret_cast<const uint4 *>(kp + at);
    const uint4 b = *reinterpret_cast<const uint4 *>(kp + at + 8 * kHeadDim);
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int w = 0; w < 4; ++w)
      mma_16816(s, widen_lo(aw[w]), widen_lo(bw[w]), widen_hi(aw[w]), widen_hi(bw[w]),
                qf[8 * i + 2 * w], qf[8 * i + 2 * w + 1]);
  }
  // the value codes of tokens 2t, 2t + 1, 2t + 8, 2t + 9, dims 16g .. 16g + 15
  uint4 v0 = *reinterpret_cast<const uint4 *>(vp + 2 * t * kHeadDim + ((g ^ (2 * t)) << 4));
  uint4 v1 = *reinterpret_cast<const uint4 *>(vp + (2 * t + 1) * kHeadDim +
                                              ((g ^ (2 * t + 1)) << 4));
  uint4 v2 = *reinterpret_cast<const uint4 *>(vp + (2 * t + 8) * kHeadDim + ((g ^ (2 * t)) << 4));
  uint4 v3 = *reinterpret_cast<const uint4 *>(vp + (2 * t + 9) * kHeadDim +
                                              ((g ^ (2 * t + 1)) << 4));
#pragma unroll
  for (int e = 0; e < 4; ++e) s[e] *= qs;
  if (valid < kPage) {  // rows behind the last position may hold anything
    if (g >= valid) s[0] = s[1] = -INFINITY;
    if (g + 8 >= valid) s[2] = s[3] = -INFINITY;
    const uint4 none = make_uint4(0, 0, 0, 0);
    if (2 * t >= valid) v0 = none;
    if (2 * t + 1 >= valid) v1 = none;
    if (2 * t + 8 >= valid) v2 = none;
    if (2 * t + 9 >= valid) v3 = none;
  }
  // ---- the maximum moves seldom ----
  const bool up = fmaxf(s[0], s[2]) > st.m[0] + (kLift + kSlack) ||
                  fmaxf(s[1], s[3]) > st.m[1] + (kLift + kSlack);
  if (__any_sync(kFull, up)) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float top = fmaxf(s[e], s[e + 2]);
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 4));
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 8));
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 16));
      const float m_new = fmaxf(st.m[e], top - kLift);
      const float alpha = m_new == st.m[e] ? 1.f : ex2(st.m[e] - m_new);
      st.m[e] = m_new;
      st.l[e] *= alpha;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        st.o[i][e] *= alpha;
        st.o[i][e + 2] *= alpha;
      }
    }
  }
  float p[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = ex2(s[e] - st.m[e & 1]);
  st.l[0] += p[0] + p[2];
  st.l[1] += p[1] + p[3];
  const __half2 p01 = __floats2half2_rn(p[0], p[1]);
  const __half2 p23 = __floats2half2_rn(p[2], p[3]);
  const uint32_t b0 = transpose8x8(*reinterpret_cast<const uint32_t *>(&p01));
  const uint32_t b1 = transpose8x8(*reinterpret_cast<const uint32_t *>(&p23));
  // ---- values ----
  const __half2 sv = __float2half2_rn(nu);
  const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
  const uint32_t w2[4] = {v2.x, v2.y, v2.z, v2.w}, w3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo01 = __byte_perm(w0[j], w1[j], 0x5140), hi01 = __byte_perm(w0[j], w1[j], 0x7362);
    const uint32_t lo23 = __byte_perm(w2[j], w3[j], 0x5140), hi23 = __byte_perm(w2[j], w3[j], 0x7362);
    mma_16816(st.o[2 * j], times(widen_lo(lo01), sv), times(widen_hi(lo01), sv),
              times(widen_lo(lo23), sv), times(widen_hi(lo23), sv), b0, b1);
    mma_16816(st.o[2 * j + 1], times(widen_lo(hi01), sv), times(widen_hi(hi01), sv),
              times(widen_lo(hi23), sv), times(widen_hi(hi23), sv), b0, b1);
  }
}

// A (sequence, KV head) segment of the flat tile list: flat tiles [s0, s0 + np)
// are pages 0 .. np - 1 of sequence b under KV head g.
struct Segment {
  int b, g, s0, np, L;
  // The next non-empty segment, called only while there is one.
  __device__ __forceinline__ void next(const int32_t *seq_lens, int hkv, int cap) {
    s0 += np;
    if (++g == hkv) {
      g = 0;
      do {
        ++b;
        L = clamped_len(seq_lens, b, cap);
        np = (L + kPage - 1) / kPage;
      } while (np == 0);
    }
  }
};

__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) decode_k8v8_kernel(
    const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
    const __half *__restrict__ q, const float2 *__restrict__ kv_scale,
    const int32_t *__restrict__ block_table, int32_t maxp, const int32_t *__restrict__ seq_lens,
    int32_t batch, int32_t hkv, int32_t num_pages, float sm_scale, int32_t *__restrict__ plan,
    float *__restrict__ part_o, float *__restrict__ part_lse, __half *__restrict__ out,
    float *__restrict__ lse_out, int32_t *dev_error) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Stage &stg = *reinterpret_cast<Stage *>(smem_raw + kWarps * sizeof(Ring));
  int32_t *ps = reinterpret_cast<int32_t *>(smem_raw);  // scan scratch, before the rings run
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cap = maxp * kPage;
  const int hq = hkv * kGroup;
  uint64_t *bars = stg.bar[warp];
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) mbar_init(&bars[s], 1);
    fence_barrier_init();
    tc::prefetch_tensormap(&tmap_k);
    tc::prefetch_tensormap(&tmap_v);
  }
  pdl_wait();

  // ---- exclusive scan of the per-sequence page counts ----
  int carry = 0;
  for (int base = 0; base < batch; base += kWarps * 32) {
    const int b = base + threadIdx.x;
    int np = 0;
    if (b < batch) {
      int L = __ldg(seq_lens + b);
      if (L < 0 || L > cap) {
        if (blockIdx.x == 0) flag_error(dev_error, K16V8_DEVERR_SEQLEN);
        L = max(0, min(L, cap));
      }
      np = (L + kPage - 1) / kPage;
    }
    int x = np;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(kFull, x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31) stg.aux[warp] = x;
    __syncthreads();
    int pre = carry, tot = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int v = stg.aux[w];
      if (w < warp) pre += v;
      tot += v;
    }
    if (b < batch) ps[b] = pre + x - np;
    carry += tot;
    __syncthreads();
  }
  if (threadIdx.x == 0) ps[batch] = carry;
  __syncthreads();

  const int T = carry * hkv;
  const int G = gridDim.x;
  const int W = max((T + G - 1) / G, kMinTiles);
  const int a = static_cast<int>(blockIdx.x) * W;
  const int e = min(a + W, T);
  // of them a run of each warp
  const int run = e > a ? (e - a + kWarps - 1) / kWarps : 0;
  const int aw = a + warp * run, ew = min(aw + run, e);
  const int n_my = max(ew - aw, 0);

  auto segment_of = [&](int f) {  // largest b with ps[b] * hkv <= f
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (ps[mid] * hkv <= f) lo = mid; else hi = mid;
    }
    Segment sg;
    sg.b = lo;
    sg.np = ps[lo + 1] - ps[lo];
    sg.g = (f - ps[lo] * hkv) / sg.np;
    sg.s0 = ps[lo] * hkv + sg.g * sg.np;
    sg.L = 0;
    return sg;
  };
  // Lane l describes this warp's tile base + l: page id * hkv + g, -1 for a
  // rejected page id, -2 past the last; and the tile's scales, whose load is in
  // flight while the copies run.  `walk` goes from a segment at or before the
  // batch's first tile to that of its last.
  auto describe = [&](int base, Segment &walk, bool scratch_live, float2 &scale) {
    const int k = base + lane;
    int t = -2;
    scale = make_float2(0.f, 0.f);
    Segment sg = walk;
    if (k < n_my) {
      const int f = aw + k;
      if (scratch_live) {
        sg = segment_of(f);
      } else {
        while (f >= sg.s0 + sg.np) sg.next(seq_lens, hkv, cap);
      }
      const int pid = __ldg(block_table + static_cast<int64_t>(sg.b) * maxp + (f - sg.s0));
      if (pid < 0 || pid >= num_pages) {
        flag_error(dev_error, K16V8_DEVERR_PAGE);
        t = -1;
      } else {
        t = pid * hkv + sg.g;
        scale = __ldg(kv_scale + t);
      }
    }
    const int last = min(31, n_my - 1 - base);
    walk.b = __shfl_sync(kFull, sg.b, last);
    walk.g = __shfl_sync(kFull, sg.g, last);
    walk.s0 = __shfl_sync(kFull, sg.s0, last);
    walk.np = __shfl_sync(kFull, sg.np, last);
    walk.L = clamped_len(seq_lens, walk.b, cap);
    return t;
  };

  Segment seg0{0, 0, 0, 0, 0};
  if (n_my > 0) {
    seg0 = segment_of(aw);
    seg0.L = clamped_len(seq_lens, seg0.b, cap);
  }
  Segment walk = seg0;
  // descriptors of the batch of 32 tiles that is issued and of the next one;
  // scales of the batch that is consumed, of those that are issued, of the next
  int desc_cur = -2, desc_nxt = -2;
  float2 sc_use = make_float2(0.f, 0.f), sc_cur = sc_use, sc_nxt = sc_use;
  if (n_my > 0) {
    desc_cur = describe(0, walk, true, sc_cur);
    if (n_my > 32) desc_nxt = describe(32, walk, false, sc_nxt);
  }
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i <= batch; i += blockDim.x) plan[2 + i] = ps[i];
    if (threadIdx.x == 0) {
      plan[0] = T;
      plan[1] = W;
    }
  }
  fence_proxy_async();  // the scan scratch becomes ring space
  __syncthreads();
  if (a >= T) return;  // no tiles for this CTA

  Ring &ring = reinterpret_cast<Ring *>(smem_raw)[warp];
  int32_t *live = stg.live[warp];
  const uint64_t policy = l2_policy_evict_first();

  int ki = 0, si = 0;  // tiles issued; the next one's slot
  auto issue = [&]() {
    if (lane == (ki & 31)) {  // the lane that knows the page
      fence_proxy_async();    // after the warp's reads of the slot
      const int t = desc_cur;
      live[si] = t >= 0;
      if (t < 0) {
        mbar_arrive(&bars[si]);  // nothing to load: the phase completes empty
      } else {
        mbar_arrive_expect_tx(&bars[si], 2 * kTile);
        tma_load_evict_first(ring.k[si], &tmap_k, t * kPage, &bars[si], policy);
        tma_load_evict_first(ring.v[si], &tmap_v, t * kPage, &bars[si], policy);
      }
    }
    if (++si == kStages) si = 0;
    if ((++ki & 31) == 0 && ki < n_my) {  // the next batch of descriptors
      desc_cur = desc_nxt;
      sc_cur = sc_nxt;
      if (ki + 32 < n_my) desc_nxt = describe(ki + 32, walk, false, sc_nxt);
    }
  };
  for (int k = 0; k < min(kStages, n_my); ++k) issue();
  sc_use = sc_cur;  // (kStages < 32: still the first batch)

  const int g = lane >> 2, t = lane & 3;
  const float qs = sm_scale * kLog2e;
  Segment cs = seg0;  // of the current piece
  int fc = aw;        // this warp's next flat tile to consume
  int kc = 0, sc = 0;
  uint32_t phase = 0;
  int fail_k = -1;    // first tile whose wait gave up
  bool ok = true;
  State st;
  // Writes the rows of segment cs: this warp's state, joined with those staged by the
  // warps behind it up to w_end.
  auto finish = [&](int w_end) {
    if (t >= 2) return;
    const bool whole = cs.s0 >= a && cs.s0 + cs.np <= e;
    float f[kWarps][2], lse[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float M = st.m[h];
#pragma unroll
      for (int w = 1; w < kWarps; ++w)
        if (w > warp && w < w_end) M = fmaxf(M, stg.m[w - 1][2 * t + h]);
      // a warp without a finite score counts for nothing, unless its sum is NaN
      auto factor = [&](float m, float l) {
        return m == -INFINITY ? (l != l ? l : 0.f) : ex2(m - M);
      };
      f[0][h] = factor(st.m[h], st.l[h]);
      float sum = f[0][h] * st.l[h];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        f[w][h] = 0.f;
        if (w > warp && w < w_end) {
          const float l = stg.l[w - 1][2 * t + h];
          f[w][h] = factor(stg.m[w - 1][2 * t + h], l);
          sum += f[w][h] * l;
        }
      }
      const bool none = sum == 0.f;  // no live page
      const float inv = none ? 0.f : 1.f / sum;
      // (the lift comes off the sum, whose logarithm is most accurate near 1)
      lse[h] = none ? -INFINITY : (M + kLift + lg2(sum * 0x1p-7f)) * kLn2;
      static_assert(kLift == 7.f, "the factor of the sum");
#pragma unroll
      for (int w = 0; w < kWarps; ++w) f[w][h] *= inv;
    }
    float r[2][16];  // of either head
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        r[h][2 * i] = f[0][h] * st.o[i][h];
        r[h][2 * i + 1] = f[0][h] * st.o[i][h + 2];
      }
    }
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      if (w <= warp || w >= w_end) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 x = stg.o[w - 1][i][2 * g + t];
        r[0][2 * i] = fmaf(f[w][0], x.x, r[0][2 * i]);
        r[1][2 * i] = fmaf(f[w][1], x.y, r[1][2 * i]);
        r[0][2 * i + 1] = fmaf(f[w][0], x.z, r[0][2 * i + 1]);
        r[1][2 * i + 1] = fmaf(f[w][1], x.w, r[1][2 * i + 1]);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (whole) {
        const int64_t row = static_cast<int64_t>(cs.b) * hq + cs.g * kGroup + 2 * t + h;
        uint4 *po = reinterpret_cast<uint4 *>(out + row * kHeadDim + 16 * g);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __half2 x = __floats2half2_rn(r[h][8 * i + 2 * j], r[h][8 * i + 2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t *>(&x);
          }
          po[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (g == 0 && lse_out) lse_out[row] = lse[h];
      } else {  // slot 0: of the segment that the CTA begins in
        const int64_t row =
            (static_cast<int64_t>(blockIdx.x) * 2 + (cs.s0 > a ? 1 : 0)) * kGroup + 2 * t + h;
        float4 *po = reinterpret_cast<float4 *>(part_o + row * kHeadDim + 16 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          po[i] = make_float4(r[h][4 * i], r[h][4 * i + 1], r[h][4 * i + 2], r[h][4 * i + 3]);
        if (g == 0) part_lse[row] = lse[h];
      }
    }
  };

  bool lead = false;  // the warp's last segment goes on in the next warp
  while (n_my > 0) {
    uint32_t qf[16];
    {
      const __half *qrow =
          q + (static_cast<int64_t>(cs.b) * hq + cs.g * kGroup + (g & 3)) * kHeadDim + 32 * t;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (g < kGroup) raw = __ldg(reinterpret_cast<const uint4 *>(qrow) + i);
        qf[4 * i + 0] = raw.x;
        qf[4 * i + 1] = raw.y;
        qf[4 * i + 2] = raw.z;
        qf[4 * i + 3] = raw.w;
      }
    }
    st.reset();
    const int seg_end = cs.s0 + cs.np;
    const int pe = min(seg_end, ew);
    for (; fc < pe; ++fc) {
      if (ok) {
        ok = __all_sync(kFull, mbar_wait_bounded(&bars[sc], phase));
        if (!ok) fail_k = kc;
      }
      if (ok) {
        const float kappa = __shfl_sync(kFull, sc_use.x, kc & 31);
        const float nu = __shfl_sync(kFull, sc_use.y, kc & 31);
        if (live[sc])
          attend(ring.k[sc], ring.v[sc], min(kPage, cs.L - (fc - cs.s0) * kPage), qf, qs * kappa,
                 nu, st);
        __syncwarp();
        if (ki < n_my) issue();
      }
      if (++sc == kStages) {
        sc = 0;
        phase ^= 1;
      }
      if ((++kc & 31) == 0) sc_use = sc_cur;  // (the issue side is in that batch by now)
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      st.l[h] += __shfl_xor_sync(kFull, st.l[h], 4);
      st.l[h] += __shfl_xor_sync(kFull, st.l[h], 8);
      st.l[h] += __shfl_xor_sync(kFull, st.l[h], 16);
    }
    if (max(cs.s0, a) < aw) {  // begun by a warp before this one, which joins it
      if (t < 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          stg.o[warp - 1][i][2 * g + t] = make_float4(st.o[i][0], st.o[i][1], st.o[i][2], st.o[i][3]);
        if (g == 0) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            stg.m[warp - 1][2 * t + h] = st.m[h];
            stg.l[warp - 1][2 * t + h] = st.l[h];
          }
        }
      }
    } else if (min(seg_end, e) > ew) {
      lead = true;
    } else {
      finish(0);
    }
    if (pe >= ew) break;
    cs.next(seq_lens, hkv, cap);
  }
  pdl_launch_dependents();
  __syncthreads();
  if (lead) finish((min(cs.s0 + cs.np, e) - a + run - 1) / run);

  if (!ok) {
    // let the copies in flight land (bounded) before the CTA's memory is released
    if (lane == 0) {
      flag_error(dev_error, K16V8_DEVERR_TIMEOUT);
      for (int kk = fail_k; kk < ki; ++kk)
        mbar_wait_bounded(&bars[kk % kStages], (kk / kStages) & 1);
    }
    __syncwarp();
  }
}

// Joins the pieces of the segments that were cut: o = sum_p e^(lse_p - lse) o_p, lse
// = log sum_p e^lse_p.  A CTA takes a (sequence, KV head), kSplit warps one of its
// query heads, a lane 4 dims; kFlight pieces of a warp are in flight.
constexpr int kFlight = 8;

struct Joined {
  float M = -INFINITY, S = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ float scale_to(float top) {  // 2^(M - top) of the state
    const float fade = M == -INFINITY ? (S != S ? S : 0.f) : ex2((M - top) * kLog2e);
    return fade;
  }
};

template <int kSplit>
__global__ void __launch_bounds__(kGroup * kSplit * 32) merge_k8v8_kernel(
    const float *__restrict__ part_o, const float *__restrict__ part_lse,
    const int32_t *__restrict__ plan, int32_t hkv, __half *__restrict__ out,
    float *__restrict__ lse_out) {
  __shared__ float4 s_o[kSplit][kGroup][32];
  __shared__ float2 s_ms[kSplit][kGroup];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = warp % kGroup, part = warp / kGroup;
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.x / hkv, g = blockIdx.x - b * hkv;
  const int W = __ldg(plan + 1), pb = __ldg(plan + 2 + b), np = __ldg(plan + 3 + b) - pb;
  Joined st;
  if (np > 0) {
    const int s0 = pb * hkv + g * np;
    const int i0 = s0 / W, i1 = (s0 + np - 1) / W;
    if (i0 == i1) return;  // held whole by one CTA, which wrote the rows
    const int n = i1 - i0 + 1;
    auto row_of = [&](int p) {  // the first piece's slot, the first slot of the CTAs behind
      return (static_cast<int64_t>(i0 + p) * 2 + (p == 0 && s0 != i0 * W ? 1 : 0)) * kGroup + head;
    };
    for (int p0 = part * kFlight; p0 < n; p0 += kSplit * kFlight) {
      float4 x[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {  // (asked for in one go, the last one again: no branch)
        const float *p = part_o + row_of(min(p0 + u, n - 1)) * kHeadDim + lane * 4;
        asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(x[u].x), "=f"(x[u].y), "=f"(x[u].z), "=f"(x[u].w)
                     : "l"(p));
      }
      const float l_own =
          lane < kFlight && p0 + lane < n ? __ldg(part_lse + row_of(p0 + lane)) : -INFINITY;
      float top = fmaxf(st.M, l_own);  // (NaN counts as nothing here and makes the sum NaN)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      const float fade = st.scale_to(top);
      st.M = top;
      st.S *= fade;
      st.o = make_float4(st.o.x * fade, st.o.y * fade, st.o.z * fade, st.o.w * fade);
      const float w_own = l_own == -INFINITY ? 0.f : ex2((l_own - top) * kLog2e);
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const float w = __shfl_sync(kFull, w_own, u);
        st.S += w;
        st.o.x = fmaf(w, x[u].x, st.o.x);
        st.o.y = fmaf(w, x[u].y, st.o.y);
        st.o.z = fmaf(w, x[u].z, st.o.z);
        st.o.w = fmaf(w, x[u].w, st.o.w);
      }
    }
  }
  if constexpr (kSplit > 1) {
    s_o[part][head][lane] = st.o;
    if (lane == 0) s_ms[part][head] = make_float2(st.M, st.S);
    __syncthreads();
    if (part > 0) return;
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kSplit; ++k) top = fmaxf(top, s_ms[k][head].x);
    Joined all;
    all.M = top;
#pragma unroll
    for (int k = 0; k < kSplit; ++k) {
      Joined one;
      one.M = s_ms[k][head].x;
      one.S = s_ms[k][head].y;
      one.o = s_o[k][head][lane];
      const float w = one.scale_to(top);
      all.S = fmaf(w, one.S, all.S);
      all.o.x = fmaf(w, one.o.x, all.o.x);
      all.o.y = fmaf(w, one.o.y, all.o.y);
      all.o.z = fmaf(w, one.o.z, all.o.z);
      all.o.w = fmaf(w, one.o.w, all.o.w);
    }
    st = all;
  }
  // S = 0: no position, or no live page
  const float inv = st.S == 0.f ? 0.f : 1.f / st.S;
  const __half2 h[2] = {__floats2half2_rn(st.o.x * inv, st.o.y * inv),
                        __floats2half2_rn(st.o.z * inv, st.o.w * inv)};
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kGroup + head;
  *reinterpret_cast<uint2 *>(out + row * kHeadDim + lane * 4) = *reinterpret_cast<const uint2 *>(h);
  if (lane == 0 && lse_out) lse_out[row] = st.S == 0.f ? -INFINITY : st.M + lg2(st.S) * kLn2;
}

// Workspace: plan int32 [T, W, P(0 .. batch)], partial rows fp32 [CTA][2][4][128], their
// LSEs fp32 [CTA][2][4], each on 256 bytes.
struct Layout {
  int ctas;
  size_t o_off, lse_off, total;
};

static bool layout(int32_t batch, Layout *w) {
  const int sms = k16v8_sm_count();
  if (sms <= 0) return false;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  w->ctas = sms * kCtasPerSm;
  const size_t rows = static_cast<size_t>(w->ctas) * 2 * kGroup;
  w->o_off = up((static_cast<size_t>(batch) + 3) * sizeof(int32_t));
  w->lse_off = w->o_off + up(rows * kHeadDim * sizeof(float));
  w->total = w->lse_off + up(rows * sizeof(float));
  return true;
}

template <int kSplit>
static int32_t launch_merge(int32_t batch, int32_t hkv, const uint8_t *ws, const Layout &w,
                            void *out, float *lse, cudaStream_t s) {
  return k16v8_launch_pdl(merge_k8v8_kernel<kSplit>, dim3(static_cast<unsigned>(batch) * hkv),
                          dim3(kGroup * kSplit * 32), 0, s,
                          reinterpret_cast<const float *>(ws + w.o_off),
                          reinterpret_cast<const float *>(ws + w.lse_off),
                          reinterpret_cast<const int32_t *>(ws), hkv, static_cast<__half *>(out),
                          lse);
}

}  // namespace decode8
}  // namespace k16v8

using namespace k16v8;

extern "C" size_t k16v8_decode_workspace_size_k8v8(int32_t batch, int32_t num_qo_heads,
                                                   int32_t head_dim) {
  decode8::Layout w;
  if (batch < 0 || batch > decode8::kMaxBatch || num_qo_heads <= 0 || num_qo_heads % kGroup ||
      head_dim != kHeadDim || !decode8::layout(batch, &w))
    return 0;
  return w.total;
}

extern "C" int32_t k16v8_paged_decode_attention_k8v8(
    const void *q, const uint8_t *k_cache, const uint8_t *v_cache, const float *kv_scale,
    const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens, int32_t batch,
    int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim, int32_t num_pages,
    float sm_scale, void *workspace, size_t workspace_bytes, void *out, float *lse,
    int32_t *dev_error, void *stream) {
  if (num_qo_heads <= 0 || num_kv_heads <= 0) return K16V8_ERR_INVALID_ARG;
  if (head_dim != kHeadDim || num_qo_heads / kGroup != num_kv_heads || num_qo_heads % kGroup)
    return K16V8_ERR_UNSUPPORTED_SHAPE;
  if (batch < 0 || batch > decode8::kMaxBatch || num_pages <= 0 || max_pages_per_seq < 0)
    return K16V8_ERR_INVALID_ARG;
  // a larger score times the scale has to be a larger scaled score
  if (!(sm_scale >= 0.f && sm_scale - sm_scale == 0.f)) return K16V8_ERR_INVALID_ARG;
  // rows of the pool and flat tile indices are int32
  if (static_cast<int64_t>(num_pages) * num_kv_heads * kPage >= (1LL << 31) ||
      static_cast<int64_t>(batch) * max_pages_per_seq * num_kv_heads >= (1LL << 31) - 8192 ||
      static_cast<int64_t>(max_pages_per_seq) * kPage >= (1LL << 31))
    return K16V8_ERR_INVALID_ARG;
  if (batch == 0) return K16V8_OK;
  if (!q || !k_cache || !v_cache || !kv_scale || (!block_table && max_pages_per_seq > 0) ||
      !seq_lens || !workspace || !out)
    return K16V8_ERR_INVALID_ARG;
  if (!k16v8_aligned(q, 16) || !k16v8_aligned(k_cache, 16) || !k16v8_aligned(v_cache, 16) ||
      !k16v8_aligned(kv_scale, 8) || !k16v8_aligned(workspace, 256) ||
      !k16v8_aligned(block_table, 4) || !k16v8_aligned(seq_lens, 4) || !k16v8_aligned(out, 16) ||
      (lse && !k16v8_aligned(lse, 4)))
    return K16V8_ERR_INVALID_ARG;
  decode8::Layout w;
  if (!decode8::layout(batch, &w)) return K16V8_ERR_CUDA;
  if (workspace_bytes < w.total) return K16V8_ERR_WORKSPACE_TOO_SMALL;
  uint8_t *ws = static_cast<uint8_t *>(workspace);

  CUtensorMap mk, mv;
  const uint64_t rows = static_cast<uint64_t>(num_pages) * num_kv_heads * kPage;
  if (!map_codes(&mk, k_cache, rows) || !map_codes(&mv, v_cache, rows)) return K16V8_ERR_CUDA;
  static bool configured[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return K16V8_ERR_CUDA;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    if (cudaFuncSetAttribute(decode8::decode_k8v8_kernel,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(decode8::kSmemBytes)) != cudaSuccess)
      return K16V8_ERR_CUDA;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  const int32_t st = k16v8_launch_pdl(
      decode8::decode_k8v8_kernel, dim3(w.ctas), dim3(decode8::kWarps * 32), decode8::kSmemBytes,
      static_cast<cudaStream_t>(stream), mk, mv, static_cast<const __half *>(q),
      reinterpret_cast<const float2 *>(kv_scale), block_table, max_pages_per_seq, seq_lens, batch,
      num_kv_heads, num_pages, sm_scale, reinterpret_cast<int32_t *>(ws),
      reinterpret_cast<float *>(ws + w.o_off), reinterpret_cast<float *>(ws + w.lse_off),
      static_cast<__half *>(out), lse, dev_error);
  if (st != K16V8_OK) return st;
  // Few segments are cut by many CTAs each (61 for one sequence of 128K and 10 heads),
  // many by a few.  4 warps a row and 1, both kernels: one of 1.1K 6.7 and 7.6 us, one of
  // 128K 58.4 and 60.4; 32 of 0.6K to 1.15K 20.2 and 18.9, 256 of 250 to 500 54.2 and 48.5.
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return batch * num_kv_heads <= 64
             ? decode8::launch_merge<4>(batch, num_kv_heads, ws, w, out, lse, s)
             : decode8::launch_merge<1>(batch, num_kv_heads, ws, w, out, lse, s);
}

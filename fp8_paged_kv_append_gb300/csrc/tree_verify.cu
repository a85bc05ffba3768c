// tree_verify: which drafted tokens of a tree the target model's
// probabilities accept, and the token that follows the accepted path, from
// given random numbers.
//
// "Phi-4: quality transfer and interrupted throughput studies": the decode
// step this library serves emits one token per sequence ("Fixed throughput
// studies"); drafted trees let one step emit several without changing the
// target's distribution.
//
// Mathematics (rejection sampling, one candidate after another).  At a node
// with target row p, draft row q and children x_1, x_2, ... (drawn from q),
// the weights start as r_0 = p with mass Z_0 = 1.  Child x is accepted when
// u q[x] Z_k < r_k[x]; a rejected one leaves r_{k+1} = max(r_k - Z_k q, 0),
// Z_{k+1} = sum r_{k+1}.  As every subtraction is of the same q,
// r_k = max(p - C_k q, 0) with C_k = Z_0 + ... + Z_{k-1}: any r_k comes
// straight from p and q and one scalar.  Without a draft row a candidate is
// certain to be proposed (q is 1 at it): its weight is set to 0.  The walk
// goes on at an accepted child; where no child is left the next token is
// drawn from r_k by inversion, the smallest j with r_0 + .. + r_j > u Z.
//
// Sums are whole numbers: a weight p - C q is formed as an unevaluated sum of
// two fp32 numbers and counted in units of 2^-44.  Integer sums do not depend
// on their order, so every split of the vocabulary gives the same masses, the
// same accepted path and the same token.  The conversion is two additions of
// a magic number (whose mantissa then holds the digits) with the remainder
// carried over: every step runs at full rate, while a conversion instruction
// to 64 bits does not (97 against 46 us at 64 sequences x 128,000).  For the
// same reason no thread but one does arithmetic in fp64, and only for a
// sibling that is tried after a rejection.
//
// Bound by one pass over the last row of p and q, and by the chain of memory
// round trips and cluster barriers around it (about 5 us of the kernel).  A
// cluster of CTAs shares a sequence: each sums its slice of the vocabulary,
// the slices' masses are exchanged through distributed shared memory, and
// every CTA takes the same decisions from the same integers.  The walk itself
// reads one p and one q per node, fetched for all nodes at once.  The CTA that
// holds the drawn number scans the run of its warp that holds it with all its
// threads.  GB300: 6.8 us for one sequence of 32,000 tokens, 10.1 us for 32 of
// 50,257 (no draft rows), 22.0 us for 64 chains of 8 nodes over 128,000 (65.5 MB:
// 9.7 us at the copy rate), 32.3 us for trees with two children a node, some of
// which pass over their row two or three times.
#include <cooperative_groups.h>

#include "k16v8_device.cuh"

namespace k16v8 {
namespace verify {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kNodes = K16V8_MAX_TREE_NODES;
constexpr int kFlush = 128;  // terms that fit the 32-bit digit sums
constexpr int kUnitBits = 44;
constexpr double kUnit = 0x1p-44;
constexpr int64_t kOne = 1ll << kUnitBits;
// x + kMagicHi has the mantissa digits of x in units of 2^-22, the remainder
// plus kMagicLo those in units of 2^-44
constexpr float kMagicHi = 3.0f;
constexpr float kMagicLo = 0x1.8p-21f;

__device__ __forceinline__ float prob(float x) { return __saturatef(x); }  // NaN: 0

// The two digits of x + rest (0 <= x <= 1, rest at most an ulp of x), still
// biased by the magic numbers' bit patterns.
__device__ __forceinline__ void digits(float x, float rest, uint32_t &hi, uint32_t &lo) {
  const float y = x + kMagicHi;
  const float z = ((x - (y - kMagicHi)) + rest) + kMagicLo;
  hi = __float_as_uint(y);
  lo = __float_as_uint(z);
}

// Units of n terms from the wrapped sums of their digits.
__device__ __forceinline__ int64_t units(uint32_t hi, uint32_t lo, uint32_t n) {
  const int32_t h = static_cast<int32_t>(hi - n * 0x40400000u);  // bits of kMagicHi
  const int32_t l = static_cast<int32_t>(lo - n * 0x35400000u);  // bits of kMagicLo
  return static_cast<int64_t>(h) * (1 << 22) + l;
}

// C (in units, below 64) as a sum of two fp32 numbers.  Rows that sum to 1 keep
// it there: 63 children leave masses of at most 1 each.  A larger one's high part
// would not be exact (and from 2^14 on not fit), so the walk ends with an error.
constexpr int64_t kMaxC = 64 * kOne;
// A mass that ends the walk so; also what 2^19 weights of 1 add up to.
constexpr int64_t kTooLarge = INT64_MIN;
__device__ __forceinline__ float c_high(int64_t C) {
  return static_cast<float>(static_cast<uint32_t>(C >> 26)) * 0x1p-18f;
}
__device__ __forceinline__ float c_low(int64_t C) {
  return static_cast<float>(static_cast<uint32_t>(C) & 0x3ffffffu) * 0x1p-44f;
}

// max(p - C q, 0), C = ch + cl, as digits.
__device__ __forceinline__ void weight(float p, float q, float ch, float cl, uint32_t &hi,
                                       uint32_t &lo) {
  const float h = __fmul_rn(ch, q);              // (not to be contracted below)
  const float l = fmaf(cl, q, fmaf(ch, q, -h));  // C q = h + l
  const float s = p - h;
  const float e = (p - s) - h;  // exact where p >= h; elsewhere the weight is 0
  const float r = e - l;
  const bool some = s + r > 0.f;
  digits(some ? s : 0.f, some ? r : 0.f, hi, lo);
}

__device__ __forceinline__ int64_t units_of(float p) {
  uint32_t hi, lo;
  digits(p, 0.f, hi, lo);
  return units(hi, lo, 1);
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
  uint64_t s = static_cast<uint64_t>(v);  // (2^63 units come out as kTooLarge)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return static_cast<int64_t>(s);
}

// The two halves of a cluster barrier: the first says that this CTA runs.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct Shared {
  int64_t cta_mass[2][kMaxCluster];  // every CTA's slice, by pass parity
  int64_t warp_mass[kWarps];
  uint64_t u63;                      // the last draw's number times 2^63
  float p[kNodes], q[kNodes], u[kNodes];
  int32_t token[kNodes], path[kNodes];
  uint32_t child[kNodes][2];         // bit masks of each node's children
  uint32_t first[2];                 // nodes accepted if tried first
  int32_t later[kNodes];             // the same for one tried after rejections
};

// Digits of the weights of tokens j, j + 1, ... (four in x, and in y of the
// draft row), added up.
template <bool kDraft>
__device__ __forceinline__ void add4(const float4 &p, const float4 &q, float ch, float cl,
                                     uint32_t &hs, uint32_t &ls) {
  const float x[4] = {p.x, p.y, p.z, p.w}, y[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t hi, lo;
    if constexpr (kDraft)
      weight(prob(x[i]), prob(y[i]), ch, cl, hi, lo);
    else
      digits(prob(x[i]), 0.f, hi, lo);
    hs += hi;
    ls += lo;
  }
}

// Mass of this lane's tokens of the run [w0, w1): blocks of four from w0 + 4
// lane in steps of 128; w0 is a 16-byte boundary of pr's memory (and of qr's
// if kVecQ) and may lie up to three tokens before the row.  The whole
// blocks' loop has no branch, so its loads are in flight together.
template <bool kDraft, bool kVecQ>
__device__ __forceinline__ int64_t run_mass(const float *pr, const float *qr, int w0, int w1,
                                            float ch, float cl) {
  const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
  int64_t sum = 0;
  auto edge = [&](int j) {  // a block that reaches beyond the row or the run
    for (int i = max(j, 0); i < min(j + 4, w1); ++i) {
      uint32_t hi, lo;
      if constexpr (kDraft)
        weight(prob(__ldg(pr + i)), prob(__ldg(qr + i)), ch, cl, hi, lo);
      else
        digits(prob(__ldg(pr + i)), 0.f, hi, lo);
      sum += units(hi, lo, 1);
    }
  };
  int j = w0 + 4 * static_cast<int>(threadIdx.x & 31);
  if (j < 0) {
    edge(j);
    j += 128;
  }
  while (j + 3 < w1) {
    const int end = min(w1, j + 32 * kFlush);
    uint32_t hs = 0, ls = 0, terms = 0;
#pragma unroll 8
    for (; j + 3 < end; j += 128) {
      const float4 p = __ldg(reinterpret_cast<const float4 *>(pr + j));
      float4 q = none;
      if constexpr (kDraft) {
        if constexpr (kVecQ)
          q = __ldg(reinterpret_cast<const float4 *>(qr + j));
        else
          q = make_float4(__ldg(qr + j), __ldg(qr + j + 1), __ldg(qr + j + 2), __ldg(qr + j + 3));
      }
      add4<kDraft>(p, q, ch, cl, hs, ls);
      terms += 4;
    }
    sum += units(hs, ls, terms);
  }
  if (j < w1) edge(j);
  return sum;
}

__global__ void __launch_bounds__(kThreads, 2) tree_verify_kernel(
    const float *__restrict__ target, int64_t target_stride, const float *__restrict__ draft,
    int64_t draft_stride, const int32_t *__restrict__ tokens, const int32_t *__restrict__ parents,
    const int32_t *__restrict__ qo_indptr, int32_t total_q, int32_t max_nodes,
    const float *__restrict__ uniforms, int32_t vocab, int32_t *__restrict__ path_out,
    int32_t *__restrict__ path_len, int32_t *__restrict__ next_token, int32_t *dev_error) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ Shared sh;
  const int rank = static_cast<int>(cluster.block_rank());
  const int csize = static_cast<int>(cluster.num_blocks());
  const int b = blockIdx.x / csize;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  cluster_arrive();
  // Slices in coordinates x = j + skew that start on the row's 16-byte
  // boundary before token 0: CTA slices and warp runs are whole 128s.
  const int per_cta = (vocab + 3 + csize * 128 - 1) / (csize * 128) * 128;
  const int per_warp = (per_cta + kWarps * 128 - 1) / (kWarps * 128) * 128;

  if (tid < kNodes) sh.child[tid][0] = sh.child[tid][1] = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();

  const int q0 = __ldg(qo_indptr + b);
  const int n = __ldg(qo_indptr + b + 1) - q0;
  auto no_result = [&](int32_t error) {
    if (rank != 0) return;
    if (tid == 0) {
      if (error) flag_error(dev_error, error);
      path_len[b] = 0;
      next_token[b] = -1;
    }
    for (int i = tid; i < max_nodes; i += kThreads)
      path_out[static_cast<int64_t>(b) * max_nodes + i] = -1;
  };
  if (q0 < 0 || n <= 0 || n > max_nodes || q0 > total_q - n) {  // the whole cluster leaves
    no_result(q0 < 0 || n != 0 ? K16V8_DEVERR_SEQLEN : 0);
    cluster_wait();
    return;
  }
  if (warp < kNodes / 32) {  // one thread per node
    bool first = false;
    if (tid < n) {
      const float u = __ldg(uniforms + q0 + tid);
      float p = 0.f, q = 1.f;
      int x = -1;
      if (tid == 0) {
        sh.u63 = __float2ull_rz(prob(u) * 0x1p63f);
      } else {
        const int par = __ldg(parents + q0 + tid);
        x = __ldg(tokens + q0 + tid);
        if (par < 0 || par >= tid || x < 0 || x >= vocab) {
          if (rank == 0) flag_error(dev_error, K16V8_DEVERR_TREE);  // no node reaches it
        } else {
          p = prob(__ldg(target + (q0 + par) * target_stride + x));
          if (draft) q = prob(__ldg(draft + (q0 + par) * draft_stride + x));
          atomicOr(&sh.child[par][tid >> 5], 1u << lane);
          // u q < p, with the product's rounding error
          const float h = __fmul_rn(u, q);
          first = h < p || (h == p && fmaf(u, q, -h) < 0.f);
        }
      }
      sh.token[tid] = x;
      sh.p[tid] = p;
      sh.q[tid] = q;
      sh.u[tid] = u;
    }
    const unsigned m = __ballot_sync(0xffffffffu, first);
    if (lane == 0) sh.first[warp] = m;
  }
  __syncthreads();
  cluster_wait();  // every CTA runs: their shared memory can be written from now on

  int passes = 0, skew = 0;
  // Mass of row `cur` with the weights max(p - C q, 0) (C = 0: p alone); the
  // warps' shares stay in sh.warp_mass, the CTAs' in sh.cta_mass[parity].
  auto mass_of = [&](int cur, int64_t C) -> int64_t {
    const float *pr = target + (q0 + cur) * target_stride;
    skew = static_cast<int>((reinterpret_cast<uintptr_t>(pr) >> 2) & 3);
    const int c0 = rank * per_cta;
    const int w0 = c0 + warp * per_warp - skew;
    const int w1 = min(vocab, min(c0 + per_cta, c0 + (warp + 1) * per_warp) - skew);
    int64_t sum = 0;
    if (C == 0) {
      sum = run_mass<false, false>(pr, nullptr, w0, w1, 0.f, 0.f);
    } else {
      const float *qr = draft + (q0 + cur) * draft_stride;
      const float ch = c_high(C), cl = c_low(C);
      if (((reinterpret_cast<uintptr_t>(qr) >> 2) & 3) == skew)
        sum = run_mass<true, true>(pr, qr, w0, w1, ch, cl);
      else
        sum = run_mass<true, false>(pr, qr, w0, w1, ch, cl);
    }
    sum = warp_sum(sum);
    __syncthreads();  // the last pass's shares have been read
    if (lane == 0) sh.warp_mass[warp] = sum;
    __syncthreads();
    const int par = passes & 1;
    if (warp == 0) {
      static_assert(kWarps <= 32, "one lane per warp");
      const int64_t cta = warp_sum(lane < kWarps ? sh.warp_mass[lane] : 0);
      if (lane < csize) cluster.map_shared_rank(&sh, lane)->cta_mass[par][rank] = cta;
    }
    cluster.sync();
    ++passes;
    uint64_t all = 0;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) all += r < csize ? sh.cta_mass[par][r] : 0;
    return static_cast<int64_t>(all);
  };
  auto mask64 = [](const uint32_t (&m)[2]) { return m[0] | static_cast<uint64_t>(m[1]) << 32; };

  // ---- the walk: the same decisions in every thread of the cluster ----
  int cur = 0, len = 1;
  int64_t C = 0;        // in units, of r_k at the current node
  int64_t mass = -1;    // of r_k, once a pass has been made
  uint64_t out_of = 0;  // no draft row: the rejected children
  const uint64_t first = mask64(sh.first);
  if (tid == 0) sh.path[0] = 0;
  for (bool down = true; down;) {
    down = false;
    bool tried = false;
    for (uint64_t m = mask64(sh.child[cur]); m && !down; m &= m - 1) {
      const int i = __ffsll(static_cast<long long>(m)) - 1;
      bool gone = false;  // a sibling with this token was rejected before
      if (!draft)
        for (uint64_t o = out_of; o; o &= o - 1)
          gone |= sh.token[__ffsll(static_cast<long long>(o)) - 1] == sh.token[i];
      if (!tried) {
        down = first >> i & 1;
      } else if (!gone) {
        // seldom taken, and in 64 bits, whose rate is low: one thread's
        if (tid == 0) {
          const double p = sh.p[i], q = sh.q[i];
          const double r = draft ? fmax(p - static_cast<double>(C) * kUnit * q, 0.0) : p;
          sh.later[i] = static_cast<double>(sh.u[i]) * q * (static_cast<double>(mass) * kUnit) < r;
        }
        __syncthreads();
        down = sh.later[i] != 0;
      }
      if (down) {
        cur = i;
        if (tid == 0) sh.path[len] = i;
        ++len;
        C = 0;
        mass = -1;
        out_of = 0;
        break;
      }
      if (draft) {
        C += tried ? mass : kOne;
        if (C >= kMaxC || C < 0) {
          mass = kTooLarge;
          break;
        }
        mass = mass_of(cur, C);
      } else {
        if (mass < 0) mass = mass_of(cur, 0);
        if (mass < 0) break;
        if (!gone) {
          mass -= units_of(sh.p[i]);
          out_of |= 1ull << i;
        }
      }
      tried = true;
    }
  }
  if (mass == -1) mass = mass_of(cur, 0);
  if (mass <= 0 && mass != kTooLarge) {  // nothing left but rounding: the target's row itself
    if (C != 0) mass = mass_of(cur, 0);
    for (uint64_t m = out_of; m; m &= m - 1)
      mass += units_of(sh.p[__ffsll(static_cast<long long>(m)) - 1]);
    C = 0;
    out_of = 0;
  }
  if (mass == kTooLarge) {  // the whole cluster leaves
    no_result(K16V8_DEVERR_PROBS);
    return;
  }
  if (rank == 0) {
    if (tid == 0) path_len[b] = len;
    for (int i = tid; i < max_nodes; i += kThreads)
      path_out[static_cast<int64_t>(b) * max_nodes + i] = i < len ? sh.path[i] : -1;
  }

  // ---- the next token: smallest j whose running sum exceeds floor(u * mass) ----
  if (mass <= 0) {  // a row without any weight
    if (rank == 0 && tid == 0) next_token[b] = -1;
    return;
  }
  const int last = (passes - 1) & 1;
  const uint64_t u63 = sh.u63;
  int64_t t = static_cast<int64_t>((__umul64hi(static_cast<uint64_t>(mass), u63) << 1) |
                                   ((static_cast<uint64_t>(mass) * u63) >> 63));
  t = min(t, mass - 1);
  if (out_of) {  // the removed tokens' weights leave the shares that hold them
    __syncthreads();  // the shares have been read
    if (tid < kNodes && (out_of >> tid & 1)) {
      const int x = sh.token[tid] + skew, r = x / per_cta, w = (x - r * per_cta) / per_warp;
      const unsigned long long u = static_cast<unsigned long long>(-units_of(sh.p[tid]));
      atomicAdd(reinterpret_cast<unsigned long long *>(&sh.cta_mass[last][r]), u);
      if (r == rank) atomicAdd(reinterpret_cast<unsigned long long *>(&sh.warp_mass[w]), u);
    }
    __syncthreads();
  }
  int owner = 0;
  for (; owner < csize - 1; ++owner) {
    const int64_t m = sh.cta_mass[last][owner];
    if (t < m) break;
    t -= m;
  }
  if (owner != rank) return;
  int a = 0, z = 0;  // the run of the owning warp
  for (int w = 0; w < kWarps; ++w) {
    const int c0 = rank * per_cta;
    a = c0 + w * per_warp - skew;
    z = min(vocab, min(c0 + per_cta, c0 + (w + 1) * per_warp) - skew);
    const int64_t m = sh.warp_mass[w];
    if (t < m || w == kWarps - 1) break;
    t -= m;
  }
  a = max(a, 0);
  // all threads scan the run, a few neighbouring tokens each
  const float *pr = target + (q0 + cur) * target_stride;
  const float *qr = C == 0 ? nullptr : draft + (q0 + cur) * draft_stride;
  const float ch = c_high(C), cl = c_low(C);
  auto weight_of = [&](int j) -> int64_t {
    const float p = prob(__ldg(pr + j));
    uint32_t hi, lo;
    if (qr)
      weight(p, prob(__ldg(qr + j)), ch, cl, hi, lo);
    else
      digits(p, 0.f, hi, lo);
    for (uint64_t m = out_of; m; m &= m - 1)
      if (sh.token[__ffsll(static_cast<long long>(m)) - 1] == j) return 0;
    return units(hi, lo, 1);
  };
  const int each = max(0, z - a + kThreads - 1) / kThreads;
  const int j0 = min(z, a + tid * each), j1 = min(z, j0 + each);
  int64_t own = 0;
  if (out_of) {
    for (int j = j0; j < j1; ++j) own += weight_of(j);
  } else {  // loads in flight together
    uint32_t hs = 0, ls = 0;
#pragma unroll 4
    for (int j = j0; j < j1; ++j) {
      uint32_t hi, lo;
      const float p = prob(__ldg(pr + j));
      if (qr)
        weight(p, prob(__ldg(qr + j)), ch, cl, hi, lo);
      else
        digits(p, 0.f, hi, lo);
      hs += hi;
      ls += lo;
    }
    own = units(hs, ls, j1 - j0);
  }
  int64_t run = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += up;
  }
  __syncthreads();  // the warps' shares have been read
  if (lane == 31) sh.warp_mass[warp] = run;
  __syncthreads();
  for (int w = 0; w < warp; ++w) run += sh.warp_mass[w];
  if (t >= run - own && t < run) {  // one thread of the CTA
    int64_t before = run - own;
    int j = j0;
    for (; j < j1 - 1; ++j) {
      before += weight_of(j);
      if (t < before) break;
    }
    next_token[b] = j;
  }
}

}  // namespace verify
}  // namespace k16v8

using namespace k16v8;

extern "C" int32_t k16v8_tree_verify(const float *target_probs, int64_t target_row_stride,
                                     const float *draft_probs, int64_t draft_row_stride,
                                     const int32_t *tokens, const int32_t *parents,
                                     const int32_t *qo_indptr, int32_t total_q, int32_t max_nodes,
                                     const float *uniforms, int32_t vocab_size, int32_t batch,
                                     int32_t *path, int32_t *path_len, int32_t *next_token,
                                     int32_t *dev_error, void *stream) {
  if (batch < 0 || total_q < 0 || max_nodes < 0 || vocab_size <= 0) return K16V8_ERR_INVALID_ARG;
  if (max_nodes > K16V8_MAX_TREE_NODES || vocab_size > K16V8_MAX_VOCAB)
    return K16V8_ERR_UNSUPPORTED_SHAPE;
  if (target_row_stride == 0) target_row_stride = vocab_size;
  if (draft_row_stride == 0) draft_row_stride = vocab_size;
  if (target_row_stride < vocab_size || draft_row_stride < vocab_size)
    return K16V8_ERR_INVALID_ARG;
  if (batch == 0) return K16V8_OK;
  if (!qo_indptr || !path_len || !next_token || (max_nodes > 0 && !path))
    return K16V8_ERR_INVALID_ARG;
  if (total_q > 0 && (!target_probs || !tokens || !parents || !uniforms))
    return K16V8_ERR_INVALID_ARG;
  if (!k16v8_aligned(target_probs, 4) || !k16v8_aligned(draft_probs, 4) ||
      !k16v8_aligned(tokens, 4) || !k16v8_aligned(parents, 4) || !k16v8_aligned(qo_indptr, 4) ||
      !k16v8_aligned(uniforms, 4) || !k16v8_aligned(path, 4) || !k16v8_aligned(path_len, 4) ||
      !k16v8_aligned(next_token, 4))
    return K16V8_ERR_INVALID_ARG;
  if (batch > 0x7fffffff / verify::kMaxCluster) return K16V8_ERR_INVALID_ARG;
  // CTAs per sequence: as many as keep the whole batch on the SMs at once, two
  // CTAs each.  64 chains over 128,000: 4 CTAs each 22.0 us, 8 (two waves) 28.7.
  const int sms = k16v8_sm_count();
  if (sms <= 0) return K16V8_ERR_CUDA;
  int cluster = verify::kMaxCluster;
  while (cluster > 1 && static_cast<int64_t>(batch) * cluster > 2LL * sms) cluster /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(batch) * cluster);
  cfg.blockDim = dim3(verify::kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify::tree_verify_kernel, target_probs, target_row_stride,
                            draft_probs, draft_row_stride, tokens, parents, qo_indptr, total_q,
                            max_nodes, uniforms, vocab_size, path, path_len, next_token,
                            dev_error) == cudaSuccess
             ? K16V8_OK
             : K16V8_ERR_CUDA;
}

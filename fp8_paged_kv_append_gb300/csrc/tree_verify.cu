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
// Sums are whole numbers: a weight is p - C q as an unevaluated sum of two
// fp32 numbers, in units of 2^-60.  Integer sums do not depend on their
// order, so every split of the vocabulary gives the same masses, the same
// accepted path and the same token.
//
// Bound by the latency of one row of p and q.  A cluster of CTAs shares a
// sequence: each sums its slice of the vocabulary, the slices' masses are
// exchanged through distributed shared memory, and every CTA takes the same
// decisions from the same integers.  The walk itself reads one p and one q
// per node, fetched for all nodes at once.
#include <cooperative_groups.h>

#include "k16v8_device.cuh"

namespace k16v8 {
namespace verify {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kNodes = K16V8_MAX_TREE_NODES;
constexpr float kUnit = 0x1p60f;  // weights are counted in units of 2^-60

__device__ __forceinline__ float prob(float x) { return fminf(fmaxf(x, 0.f), 1.f); }  // NaN: 0

__device__ __forceinline__ int64_t units(float x) { return __float2ll_rz(x * kUnit); }

// max(p - C q, 0) in units, C = ch + cl.
__device__ __forceinline__ int64_t residual(float p, float q, float ch, float cl) {
  const float h = ch * q;
  const float l = fmaf(ch, q, -h) + cl * q;  // C q = h + l
  const float s = p - h;
  const float bb = s - p;
  const float e = (p - (s - bb)) + (-h - bb);  // p - h = s + e exactly
  const int64_t r = units(fmaxf(s, -1.f)) + units(e - l);
  return r > 0 ? r : 0;
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct Shared {
  int64_t cta_mass[2][kMaxCluster];  // every CTA's slice, by pass parity
  int64_t warp_mass[kWarps];
  float p[kNodes], q[kNodes], u[kNodes];
  int32_t parent[kNodes], token[kNodes];
  int32_t path[kNodes];
};

__global__ void __launch_bounds__(kThreads) tree_verify_kernel(
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
  pdl_wait();
  pdl_launch_dependents();

  const int q0 = __ldg(qo_indptr + b);
  const int n = __ldg(qo_indptr + b + 1) - q0;
  if (q0 < 0 || n <= 0 || n > max_nodes || q0 > total_q - n) {  // the whole cluster leaves
    if (rank == 0) {
      if (tid == 0) {
        if (q0 < 0 || n != 0) flag_error(dev_error, K16V8_DEVERR_SEQLEN);
        path_len[b] = 0;
        next_token[b] = -1;
      }
      for (int i = tid; i < max_nodes; i += kThreads)
        path_out[static_cast<int64_t>(b) * max_nodes + i] = -1;
    }
    return;
  }
  if (tid < n) {
    int par = -1, x = -1;
    float p = 0.f, q = 1.f;
    const float u = __ldg(uniforms + q0 + tid);
    if (tid > 0) {
      par = __ldg(parents + q0 + tid);
      x = __ldg(tokens + q0 + tid);
      if (par < 0 || par >= tid || x < 0 || x >= vocab) {
        if (rank == 0) flag_error(dev_error, K16V8_DEVERR_TREE);
        par = -1;  // no node reaches it
      } else {
        p = prob(__ldg(target + (q0 + par) * target_stride + x));
        if (draft) q = prob(__ldg(draft + (q0 + par) * draft_stride + x));
      }
    }
    sh.parent[tid] = par;
    sh.token[tid] = x;
    sh.p[tid] = p;
    sh.q[tid] = q;
    sh.u[tid] = u;
  }
  cluster.sync();  // every CTA runs: their shared memory can be written from now on

  // this CTA's slice, and each warp's run of it
  const int per_cta = (vocab + csize - 1) / csize;
  const int c0 = min(vocab, rank * per_cta), c1 = min(vocab, c0 + per_cta);
  const int per_warp = ((c1 - c0 + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int w0 = min(c1, c0 + warp * per_warp), w1 = min(c1, w0 + per_warp);

  int passes = 0;
  // Mass of row `cur` with the weights max(p - C q, 0) (C = 0: p alone); the
  // warps' shares stay in sh.warp_mass, the CTAs' in sh.cta_mass[parity].
  auto mass_of = [&](int cur, double C) -> int64_t {
    const float *pr = target + (q0 + cur) * target_stride;
    int64_t sum = 0;
    if (C == 0.0) {
#pragma unroll 8
      for (int j = w0 + lane; j < w1; j += 32) sum += units(prob(__ldg(pr + j)));
    } else {
      const float *qr = draft + (q0 + cur) * draft_stride;
      const float ch = static_cast<float>(C);
      const float cl = static_cast<float>(C - static_cast<double>(ch));
#pragma unroll 4
      for (int j = w0 + lane; j < w1; j += 32)
        sum += residual(prob(__ldg(pr + j)), prob(__ldg(qr + j)), ch, cl);
    }
    sum = warp_sum(sum);
    __syncthreads();  // the last pass's shares have been read
    if (lane == 0) sh.warp_mass[warp] = sum;
    __syncthreads();
    const int par = passes & 1;
    if (tid < csize) {
      int64_t cta = 0;
      for (int w = 0; w < kWarps; ++w) cta += sh.warp_mass[w];
      cluster.map_shared_rank(&sh, tid)->cta_mass[par][rank] = cta;
    }
    cluster.sync();
    ++passes;
    int64_t all = 0;
    for (int r = 0; r < csize; ++r) all += sh.cta_mass[par][r];
    return all;
  };

  // ---- the walk: the same decisions in every thread of the cluster ----
  int cur = 0, len = 1;
  double C = 0.0, Z = 1.0;       // scalars of r_k at the current node
  int64_t mass = -1;             // Z in units once a pass has been made
  uint64_t out_of = 0;           // no draft row: the rejected children
  if (tid == 0) sh.path[0] = 0;
  for (int i = 1; i < n; ++i) {
    if (sh.parent[i] != cur) continue;
    const double p = sh.p[i], q = sh.q[i];
    bool gone = false;  // a sibling with this token was rejected before
    if (!draft)
      for (uint64_t m = out_of; m; m &= m - 1) gone |= sh.token[__ffsll(m) - 1] == sh.token[i];
    const double r = gone ? 0.0 : (draft ? fmax(p - C * q, 0.0) : p);
    if (static_cast<double>(sh.u[i]) * q * Z < r) {
      cur = i;
      if (tid == 0) sh.path[len] = i;
      ++len;
      C = 0.0;
      Z = 1.0;
      mass = -1;
      out_of = 0;
      continue;
    }
    if (draft) {
      C += Z;
      mass = mass_of(cur, C);
    } else {
      if (mass < 0) mass = mass_of(cur, 0.0);
      if (!gone) {
        mass -= units(sh.p[i]);
        out_of |= 1ull << i;
      }
    }
    Z = static_cast<double>(mass) * 0x1p-60;
  }
  if (mass < 0) mass = mass_of(cur, 0.0);
  if (mass <= 0 && (C != 0.0 || out_of)) {  // nothing left but rounding: the target's row itself
    if (C != 0.0) {
      mass = mass_of(cur, 0.0);
    } else {
      for (uint64_t m = out_of; m; m &= m - 1) mass += units(sh.p[__ffsll(m) - 1]);
    }
    C = 0.0;
    out_of = 0;
  }

  // ---- the next token ----
  const int last = (passes - 1) & 1;
  int token = -1;
  bool mine = false;
  if (mass > 0) {
    // smallest j whose running sum exceeds floor(u * mass)
    const double ud = static_cast<double>(prob(sh.u[0]));
    int64_t t = static_cast<int64_t>(
        __umul64hi(static_cast<uint64_t>(mass), __double2ull_rz(ud * 0x1p63)) << 1);
    t |= static_cast<int64_t>(
        (static_cast<uint64_t>(mass) * __double2ull_rz(ud * 0x1p63)) >> 63);
    t = min(t, mass - 1);
    // weight of the removed tokens inside [a, z)
    auto removed = [&](int a, int z) {
      int64_t s = 0;
      for (uint64_t m = out_of; m; m &= m - 1) {
        const int i = __ffsll(m) - 1;
        if (sh.token[i] >= a && sh.token[i] < z) s += units(sh.p[i]);
      }
      return s;
    };
    int64_t before = 0;
    int owner = 0;
    for (int r = 0; r < csize; ++r) {
      const int a = min(vocab, r * per_cta), z = min(vocab, a + per_cta);
      const int64_t m = sh.cta_mass[last][r] - removed(a, z);
      if (t < before + m) {
        owner = r;
        break;
      }
      before += m;
    }
    if (owner == rank) {
      int w = 0;
      for (; w < kWarps - 1; ++w) {
        const int a = min(c1, c0 + w * per_warp), z = min(c1, a + per_warp);
        const int64_t m = sh.warp_mass[w] - removed(a, z);
        if (t < before + m) break;
        before += m;
      }
      if (w == warp) {
        mine = true;
        const float *pr = target + (q0 + cur) * target_stride;
        const float *qr = draft ? draft + (q0 + cur) * draft_stride : nullptr;
        const float ch = static_cast<float>(C);
        const float cl = static_cast<float>(C - static_cast<double>(ch));
        for (int j0 = w0; j0 < w1; j0 += 32) {
          const int j = j0 + lane;
          int64_t v = 0;
          if (j < w1) {
            const float p = prob(__ldg(pr + j));
            v = C == 0.0 ? units(p) : residual(p, prob(__ldg(qr + j)), ch, cl);
            for (uint64_t m = out_of; m; m &= m - 1)
              if (sh.token[__ffsll(m) - 1] == j) v = 0;
          }
          int64_t run = v;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += up;
          }
          const unsigned hit = __ballot_sync(0xffffffffu, t < before + run);
          if (hit) {
            token = j0 + __ffs(hit) - 1;
            break;
          }
          before += __shfl_sync(0xffffffffu, run, 31);
        }
      }
    }
  } else if (rank == 0 && warp == 0) {
    mine = true;  // a row without any weight
  }
  if (mine && lane == 0) next_token[b] = token;
  if (rank == 0) {
    if (tid == 0) path_len[b] = len;
    for (int i = tid; i < max_nodes; i += kThreads)
      path_out[static_cast<int64_t>(b) * max_nodes + i] = i < len ? sh.path[i] : -1;
  }
  cluster.sync();  // no CTA leaves while another may still write its shared memory
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
  const int cluster = verify::kMaxCluster;
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

// Attention of drafted token trees over the paged K16/V8 cache: the calls
// and the merge of cut segments (the split kernel: tree_tc.cuh, the cut: tree_plan.cuh).
//
// "Phi-4: quality transfer and interrupted throughput studies": the intro
// gives the format (FP16 K, E4M3 V with per-head scales) and the geometry (40
// query heads over 10 KV heads, d = 128); a tree of drafted tokens lets one
// pass over the cache serve several query tokens of a sequence.
//
// Mathematics.  The n nodes of a sequence are its last n cached positions
// (base .. base + n - 1).  Node i sees every position below base, and
// position base + j exactly when bit j of its mask is set; softmax attention
// over what it sees, a row that sees nothing gives 0 and LSE -inf.
#include <algorithm>

#include "tensor_map.cuh"
#include "tree_tc.cuh"

namespace k16v8 {
namespace tree {

// Joins the pieces of the segment that begins in CTA blockIdx.x and is cut:
// o = sum_p e^(lse_p - lse) o_p, lse = log sum_p e^lse_p.  A block takes 32
// rows x 32 dims: a lane per row, a warp per 8 dims, so a warp's loads are
// 512-byte runs.  Bound by latency: the first pieces' rows are asked for
// before the LSEs are in hand, and eight pieces are in flight at a time.
constexpr int kMergeFlight = 8;
__global__ void __launch_bounds__(128) tree_merge_kernel(const Args a) {
  extern __shared__ float lse_of[];  // [piece][32 rows]
  pdl_wait();
  pdl_launch_dependents();
  const int4 cut = __ldg(a.cut + blockIdx.x);
  if (cut.x < 0) return;
  const int first = blockIdx.x, pieces = cut.z - first + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.y * 32 + lane, chunk = (blockIdx.z * 4 + warp) * 2;
  auto slot = [&](int p) { return 2 * static_cast<int64_t>(first + p) + (p == 0 ? 1 : 0); };
  float4 x[kMergeFlight][2];
  auto load = [&](int p0) {
#pragma unroll
    for (int u = 0; u < kMergeFlight; ++u) {
      if (p0 + u >= pieces) continue;
      const float4 *po = a.part_o + (slot(p0 + u) * 32 + chunk) * a.max_rows + row;
      x[u][0] = __ldg(po);
      x[u][1] = __ldg(po + a.max_rows);
    }
  };
  load(0);
  for (int p = warp; p < pieces; p += 4)
    lse_of[p * 32 + lane] = __ldg(a.part_lse + slot(p) * a.max_rows + row);
  const int q0 = __ldg(a.qo_indptr + cut.x), n = __ldg(a.qo_indptr + cut.x + 1) - q0;
  __syncthreads();
  float M = -INFINITY;
  for (int p = 0; p < pieces; ++p) M = fmaxf(M, lse_of[p * 32 + lane]);
  float S = 0.f;
  float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int p0 = 0; p0 < pieces; p0 += kMergeFlight) {
    if (p0 > 0) load(p0);
#pragma unroll
    for (int u = 0; u < kMergeFlight; ++u) {
      if (p0 + u >= pieces) continue;
      const float l = lse_of[(p0 + u) * 32 + lane];
      if (l == -INFINITY) continue;
      const float w = ex2((l - M) * kLog2e);
      S += w;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        acc[i].x = fmaf(w, x[u][i].x, acc[i].x);
        acc[i].y = fmaf(w, x[u][i].y, acc[i].y);
        acc[i].z = fmaf(w, x[u][i].z, acc[i].z);
        acc[i].w = fmaf(w, x[u][i].w, acc[i].w);
      }
    }
  }
  if (row >= n * kGroup) return;
  const bool dead = S == 0.f;  // the row sees nothing
  const float inv = dead ? 0.f : 1.f / S;
  const int64_t orow =
      static_cast<int64_t>(q0 + row / kGroup) * a.hkv * kGroup + cut.y * kGroup + row % kGroup;
  const __half2 h[4] = {__floats2half2_rn(acc[0].x * inv, acc[0].y * inv),
                        __floats2half2_rn(acc[0].z * inv, acc[0].w * inv),
                        __floats2half2_rn(acc[1].x * inv, acc[1].y * inv),
                        __floats2half2_rn(acc[1].z * inv, acc[1].w * inv)};
  *reinterpret_cast<uint4 *>(a.out + orow * kHeadDim + chunk * 4) =
      *reinterpret_cast<const uint4 *>(h);
  if (chunk == 0 && a.lse) a.lse[orow] = dead ? -INFINITY : M + lg2(S) * kLn2;
}

// ---- host side ------------------------------------------------------------

struct Layout {
  int ctas, max_rows;
  size_t lse_off, o_off, total;  // cut segments first
};

static bool layout(int32_t max_nodes, Layout *w) {
  const int sms = k16v8_sm_count();
  if (sms <= 0) return false;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  w->ctas = sms;
  w->max_rows = max_nodes <= tcore::kNodes ? tcore::kRows : 2 * tcore::kRows;
  const size_t rows = 2 * static_cast<size_t>(w->ctas) * w->max_rows;
  w->lse_off = up(w->ctas * sizeof(int4));
  w->o_off = w->lse_off + up(rows * sizeof(float));
  w->total = w->o_off + rows * kHeadDim * sizeof(float);
  return true;
}

template <bool kWide>
static int32_t launch_tc(const CUtensorMap &mq, const CUtensorMap &mk, const Args &a, int ctas,
                         cudaStream_t s) {
  static bool configured[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return K16V8_ERR_CUDA;
  constexpr uint32_t smem = tcore::Smem<kWide>::kBytes;
  if (dev >= 64 || !configured[dev]) {
    if (cudaFuncSetAttribute(tcore::tree_tc_kernel<kWide>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess)
      return K16V8_ERR_CUDA;
    if (dev < 64) configured[dev] = true;
  }
  return k16v8_launch_pdl(tcore::tree_tc_kernel<kWide>, dim3(ctas), dim3(tcore::kThreads), smem, s,
                          mq, mk, a);
}

}  // namespace tree
}  // namespace k16v8

using namespace k16v8;

static int32_t check_tree_shape(int32_t total_q, int32_t batch, int32_t max_nodes, int32_t hq,
                                int32_t hkv, int32_t head_dim, int32_t max_len) {
  if (total_q < 0 || batch < 0 || max_nodes < 0 || hq <= 0 || hkv <= 0 || max_len < 0)
    return K16V8_ERR_INVALID_ARG;
  if (head_dim != kHeadDim || hq != kGroup * hkv || max_nodes > K16V8_MAX_TREE_NODES)
    return K16V8_ERR_UNSUPPORTED_SHAPE;
  if (batch > tree::kMaxBatch || hkv > 4095 || max_len > tree::kMaxLen)
    return K16V8_ERR_INVALID_ARG;
  return K16V8_OK;
}

extern "C" size_t k16v8_tree_workspace_size(int32_t total_q, int32_t batch, int32_t max_nodes,
                                            int32_t num_qo_heads, int32_t num_kv_heads,
                                            int32_t head_dim, int32_t max_seq_len) {
  tree::Layout w;
  if (check_tree_shape(total_q, batch, max_nodes, num_qo_heads, num_kv_heads, head_dim,
                       max_seq_len) != K16V8_OK ||
      !tree::layout(max_nodes, &w))
    return 0;
  return w.total;
}

extern "C" int32_t k16v8_paged_tree_attention(
    const void *q, const int32_t *qo_indptr, int32_t total_q, int32_t max_nodes,
    const uint64_t *tree_mask, const void *k_cache, const uint8_t *v_cache, const float *v_scale,
    const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
    int32_t max_seq_len, int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t num_pages, float sm_scale, void *workspace, size_t workspace_bytes,
    void *out, float *lse, int32_t *dev_error, void *stream) {
  int32_t st = check_tree_shape(total_q, batch, max_nodes, num_qo_heads, num_kv_heads, head_dim,
                                max_seq_len);
  if (st != K16V8_OK) return st;
  if (num_pages <= 0 || max_pages_per_seq < 0) return K16V8_ERR_INVALID_ARG;
  // a row's largest score times the scale has to be its largest scaled score
  if (!(sm_scale >= 0.f && sm_scale - sm_scale == 0.f)) return K16V8_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_pages_per_seq) * kPage < max_seq_len) return K16V8_ERR_INVALID_ARG;
  if (batch == 0 || total_q == 0 || max_nodes == 0 || max_seq_len == 0) return K16V8_OK;
  if (!q || !qo_indptr || !tree_mask || !k_cache || !v_cache || !v_scale || !block_table ||
      !seq_lens || !workspace || !out)
    return K16V8_ERR_INVALID_ARG;
  if (!k16v8_aligned(q, 16) || !k16v8_aligned(k_cache, 16) || !k16v8_aligned(v_cache, 16) ||
      !k16v8_aligned(out, 16) || !k16v8_aligned(tree_mask, 8) || !k16v8_aligned(qo_indptr, 4) ||
      !k16v8_aligned(seq_lens, 4) || !k16v8_aligned(block_table, 4) ||
      !k16v8_aligned(v_scale, 4) || (lse && !k16v8_aligned(lse, 4)) ||
      !k16v8_aligned(workspace, 256))
    return K16V8_ERR_INVALID_ARG;
  const uint64_t k_rows = static_cast<uint64_t>(num_pages) * num_kv_heads * kPage;
  if (k_rows >= (1ull << 31)) return K16V8_ERR_INVALID_ARG;
  tree::Layout w;
  if (!tree::layout(max_nodes, &w)) return K16V8_ERR_CUDA;
  if (workspace_bytes < w.total) return K16V8_ERR_WORKSPACE_TOO_SMALL;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const tree::Args a{static_cast<const __half *>(q),
                     qo_indptr,
                     total_q,
                     max_nodes,
                     tree_mask,
                     static_cast<const __half *>(k_cache),
                     v_cache,
                     v_scale,
                     block_table,
                     max_pages_per_seq,
                     seq_lens,
                     max_seq_len,
                     batch,
                     num_kv_heads,
                     num_pages,
                     sm_scale,
                     reinterpret_cast<int4 *>(ws),
                     reinterpret_cast<float *>(ws + w.lse_off),
                     reinterpret_cast<float4 *>(ws + w.o_off),
                     w.max_rows,
                     static_cast<__half *>(out),
                     lse,
                     dev_error};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CUtensorMap mq, mk;
  if (!map_rows(&mq, q, num_qo_heads, total_q) || !map_keys(&mk, k_cache, k_rows))
    return K16V8_ERR_CUDA;
  st = max_nodes > tree::tcore::kNodes ? tree::launch_tc<true>(mq, mk, a, w.ctas, s)
                                       : tree::launch_tc<false>(mq, mk, a, w.ctas, s);
  if (st != K16V8_OK) return st;
  return k16v8_launch_pdl(tree::tree_merge_kernel,
                          dim3(w.ctas, (max_nodes * kGroup + 31) / 32, 4), dim3(128),
                          static_cast<size_t>(w.ctas) * 32 * sizeof(float), s, a);
}

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
// o = sum_p e^(lse_p - lse) o_p, lse = log sum_p e^lse_p, with a running
// maximum.  A warp takes 32 rows, a lane each (so its loads are 512-byte runs),
// by kChunks chunks of 4 dims, and has kFlight pieces in flight.
template <int kChunks, int kFlight>
__device__ __forceinline__ void merge_rows(const Args &a, const int4 &cut, int first, int row,
                                           int chunk) {
  const int pieces = cut.z - first + 1;
  float M = -INFINITY, S = 0.f;
  float4 acc[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int q0 = __ldg(a.qo_indptr + cut.x), n = __ldg(a.qo_indptr + cut.x + 1) - q0;
  for (int p0 = 0; p0 < pieces; p0 += kFlight) {
    float4 x[kFlight][kChunks];
    float l[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int p = min(p0 + u, pieces - 1);  // (the last one again: no branch)
      const int64_t slot = 2 * static_cast<int64_t>(first + p) + (p == 0 ? 1 : 0);
      const float4 *po = a.part_o + (slot * 32 + chunk) * a.max_rows + row;
      l[u] = __ldg(a.part_lse + slot * a.max_rows + row);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) x[u][c] = __ldg(po + static_cast<int64_t>(c) * a.max_rows);
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      if (p0 + u >= pieces) l[u] = -INFINITY;
      top = fmaxf(top, l[u]);
    }
    const float fade = M == -INFINITY ? 0.f : ex2((M - top) * kLog2e);
    M = top;
    S *= fade;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      acc[c] = make_float4(acc[c].x * fade, acc[c].y * fade, acc[c].z * fade, acc[c].w * fade);
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      if (l[u] == -INFINITY) continue;
      const float w = ex2((l[u] - M) * kLog2e);
      S += w;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        acc[c].x = fmaf(w, x[u][c].x, acc[c].x);
        acc[c].y = fmaf(w, x[u][c].y, acc[c].y);
        acc[c].z = fmaf(w, x[u][c].z, acc[c].z);
        acc[c].w = fmaf(w, x[u][c].w, acc[c].w);
      }
    }
  }
  if (row >= n * kGroup) return;
  const bool dead = S == 0.f;  // the row sees nothing
  const float inv = dead ? 0.f : 1.f / S;
  const int64_t orow =
      static_cast<int64_t>(q0 + row / kGroup) * a.hkv * kGroup + cut.y * kGroup + row % kGroup;
  uint4 *po = reinterpret_cast<uint4 *>(a.out + orow * kHeadDim + chunk * 4);
#pragma unroll
  for (int c = 0; c < kChunks; c += 2) {
    const __half2 h[4] = {__floats2half2_rn(acc[c].x * inv, acc[c].y * inv),
                          __floats2half2_rn(acc[c].z * inv, acc[c].w * inv),
                          __floats2half2_rn(acc[c + 1].x * inv, acc[c + 1].y * inv),
                          __floats2half2_rn(acc[c + 1].z * inv, acc[c + 1].w * inv)};
    po[c / 2] = *reinterpret_cast<const uint4 *>(h);
  }
  if (chunk == 0 && a.lse) a.lse[orow] = dead ? -INFINITY : M + lg2(S) * kLn2;
}

// One CTA: 32 rows by 16 kChunks dims (32 dims for trees of up to 16 nodes, 64
// beyond: launch_merge).  Latency-bound: three round trips (the cut, lengths
// and rows, stores) for up to 2 pieces or 16 / kChunks (8 and 4), no
// shared memory; about 3 us of a call, and 8 where all 152 CTAs' segments are
// cut and have 256 rows (40 MB).  LSEs through shared memory ahead of the
// rows: 95.9 against 91.8 us on 5 nodes at 128K.
constexpr int kMergeWarps = 4;
template <int kChunks>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const Args a) {
  pdl_wait();
  pdl_launch_dependents();
  const int4 cut = __ldg(a.cut + blockIdx.x);
  if (cut.x < 0) return;
  const int row = blockIdx.y * 32 + (threadIdx.x & 31);
  const int chunk = (blockIdx.z * kMergeWarps + (threadIdx.x >> 5)) * kChunks;
  if (cut.z - static_cast<int>(blockIdx.x) + 1 <= 2)
    merge_rows<kChunks, 2>(a, cut, blockIdx.x, row, chunk);
  else
    merge_rows<kChunks, 16 / kChunks>(a, cut, blockIdx.x, row, chunk);
}

template <int kChunks>
static int32_t launch_merge(const Args &a, int ctas, cudaStream_t s) {
  const dim3 grid(ctas, (a.max_nodes * kGroup + 31) / 32, kHeadDim / 4 / (kMergeWarps * kChunks));
  return k16v8_launch_pdl(tree_merge_kernel<kChunks>, grid, dim3(kMergeWarps * 32), 0, s, a);
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

template <bool kWide, bool kTest>
static int32_t launch_tc(const CUtensorMap &mq, const CUtensorMap &mk, const Args &a, int ctas,
                         cudaStream_t s) {
  static bool configured[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return K16V8_ERR_CUDA;
  constexpr uint32_t smem = tcore::Smem<kWide>::kBytes;
  if (dev >= 64 || !configured[dev]) {
    if (cudaFuncSetAttribute(tcore::tree_tc_kernel<kWide, kTest>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess)
      return K16V8_ERR_CUDA;
    if (dev < 64) configured[dev] = true;
  }
  return k16v8_launch_pdl(tcore::tree_tc_kernel<kWide, kTest>, dim3(ctas), dim3(tcore::kThreads),
                          smem, s, mq, mk, a);
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

template <bool kTest>
static int32_t tree_attention(
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
  const tree::Args a{qo_indptr,
                     total_q,
                     max_nodes,
                     tree_mask,
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
  st = max_nodes > tree::tcore::kNodes ? tree::launch_tc<true, kTest>(mq, mk, a, w.ctas, s)
                                       : tree::launch_tc<false, kTest>(mq, mk, a, w.ctas, s);
  if (st != K16V8_OK) return st;
  // Wide trees have row groups enough, and every CTA costs its launch whether its
  // segment is cut or not.  2 and 4 chunks per warp, both calls together, us: 5
  // nodes at 1K 11.5 / 12.0, at 128K 91.8 / 94.8; 16 nodes 12.1 / 12.4, 93.3 /
  // 94.3 and 32 x 1.1K 41.4 / 40.8; 32 nodes at 128K 95.4 / 95.9, 32 x 1.1K 45.7 /
  // 44.9, one short sequence 12.2 / 11.0; 64 nodes, 16 x 8K 160.3 / 154.8 (8: 154.6),
  // 1 x 128K 149 / 146.7 (8: 149.1).
  return max_nodes > 16 ? tree::launch_merge<4>(a, w.ctas, s)
                        : tree::launch_merge<2>(a, w.ctas, s);
}

extern "C" int32_t k16v8_paged_tree_attention(
    const void *q, const int32_t *qo_indptr, int32_t total_q, int32_t max_nodes,
    const uint64_t *tree_mask, const void *k_cache, const uint8_t *v_cache, const float *v_scale,
    const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
    int32_t max_seq_len, int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t num_pages, float sm_scale, void *workspace, size_t workspace_bytes,
    void *out, float *lse, int32_t *dev_error, void *stream) {
  return tree_attention<false>(q, qo_indptr, total_q, max_nodes, tree_mask, k_cache, v_cache, v_scale,
                               block_table, max_pages_per_seq, seq_lens, max_seq_len, batch,
                               num_qo_heads, num_kv_heads, head_dim, num_pages, sm_scale, workspace,
                               workspace_bytes, out, lse, dev_error, stream);
}

extern "C" int32_t k16v8_paged_tree_attention_wait_test(
    const void *q, const int32_t *qo_indptr, int32_t total_q, int32_t max_nodes,
    const uint64_t *tree_mask, const void *k_cache, const uint8_t *v_cache, const float *v_scale,
    const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
    int32_t max_seq_len, int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t num_pages, float sm_scale, void *workspace, size_t workspace_bytes,
    void *out, float *lse, int32_t *dev_error, void *stream) {
  return tree_attention<true>(q, qo_indptr, total_q, max_nodes, tree_mask, k_cache, v_cache, v_scale,
                               block_table, max_pages_per_seq, seq_lens, max_seq_len, batch,
                               num_qo_heads, num_kv_heads, head_dim, num_pages, sm_scale, workspace,
                               workspace_bytes, out, lse, dev_error, stream);
}

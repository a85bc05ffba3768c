// Attention of several query rows over the K8/V8 cache: causal prefill and cross
// attention to an encoder's states, and the merge of cut segments (the split
// kernel: attention_k8v8.cuh, the cut: attention_k8v8_plan.cuh).
//
// "Phi-4: quality transfer and interrupted throughput studies": the intro gives
// the geometry (40 query heads over 10 KV heads, d = 128) and the page pool;
// keys in 8 bits and scales per page are this library's.
//
// Mathematics.  Keys and values are scale * code of their page and head.  Prefill:
// the n query rows of a sequence are its last n cached positions, row i sees
// positions 0 .. L - n + i.  Cross attention: every row sees all L positions, n
// and L are unrelated.  Softmax attention over what a row sees; one that sees
// nothing gives 0 and LSE -inf.
#include <algorithm>

#include "tensor_map.cuh"
#include "attention_k8v8.cuh"

namespace k16v8 {
namespace attn8 {

// Joins the pieces of the segment that begins in CTA blockIdx.x and is cut:
// o = sum_p e^(lse_p - lse) o_p, lse = log sum_p e^lse_p, with a running
// maximum.  A warp takes 32 rows, a lane each (so its loads are 512-byte runs),
// by kChunks chunks of 4 dims, and has kFlight pieces in flight.
template <int kMerge, int kFlight>
__device__ __forceinline__ void merge_rows(const Args &a, const int4 &cut, int first, int row,
                                           int chunk) {
  const int pieces = cut.w - first + 1;
  float M = -INFINITY, S = 0.f;
  float4 acc[kMerge];
#pragma unroll
  for (int c = 0; c < kMerge; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = 0; p0 < pieces; p0 += kFlight) {
    float4 x[kFlight][kMerge];
    float l[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int p = min(p0 + u, pieces - 1);  // (the last one again: no branch)
      const int64_t slot = 2 * static_cast<int64_t>(first + p) + (p == 0 ? 1 : 0);
      const float4 *po = a.part_o + (slot * 32 + chunk) * a.max_rows + row;
      l[u] = __ldg(a.part_lse + slot * a.max_rows + row);
#pragma unroll
      for (int c = 0; c < kMerge; ++c) x[u][c] = __ldg(po + static_cast<int64_t>(c) * a.max_rows);
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
    for (int c = 0; c < kMerge; ++c)
      acc[c] = make_float4(acc[c].x * fade, acc[c].y * fade, acc[c].z * fade, acc[c].w * fade);
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      if (l[u] == -INFINITY) continue;
      const float w = ex2((l[u] - M) * kLog2e);
      S += w;
#pragma unroll
      for (int c = 0; c < kMerge; ++c) {
        acc[c].x = fmaf(w, x[u][c].x, acc[c].x);
        acc[c].y = fmaf(w, x[u][c].y, acc[c].y);
        acc[c].z = fmaf(w, x[u][c].z, acc[c].z);
        acc[c].w = fmaf(w, x[u][c].w, acc[c].w);
      }
    }
  }
  if (row >= cut.y * kGroup) return;
  const bool dead = S == 0.f;  // the row sees nothing
  const float inv = dead ? 0.f : 1.f / S;
  const int64_t orow =
      static_cast<int64_t>(cut.x + row / kGroup) * a.hkv * kGroup + cut.z * kGroup + row % kGroup;
  uint4 *po = reinterpret_cast<uint4 *>(a.out + orow * kHeadDim + chunk * 4);
#pragma unroll
  for (int c = 0; c < kMerge; c += 2) {
    const __half2 h[4] = {__floats2half2_rn(acc[c].x * inv, acc[c].y * inv),
                          __floats2half2_rn(acc[c].z * inv, acc[c].w * inv),
                          __floats2half2_rn(acc[c + 1].x * inv, acc[c + 1].y * inv),
                          __floats2half2_rn(acc[c + 1].z * inv, acc[c + 1].w * inv)};
    po[c / 2] = *reinterpret_cast<const uint4 *>(h);
  }
  if (chunk == 0 && a.lse) a.lse[orow] = dead ? -INFINITY : M + lg2(S) * kLn2;
}

// One CTA: 32 rows by 16 kMerge dims.  Latency-bound: the cut, then LSEs and rows
// together, then stores.
constexpr int kMergeWarps = 4;
template <int kMerge>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_kernel(const Args a) {
  pdl_wait();
  pdl_launch_dependents();
  const int4 cut = __ldg(a.cut + blockIdx.x);
  if (cut.x < 0) return;
  const int row = blockIdx.y * 32 + (threadIdx.x & 31);
  const int chunk = (blockIdx.z * kMergeWarps + (threadIdx.x >> 5)) * kMerge;
  if (cut.w - static_cast<int>(blockIdx.x) + 1 <= 2)
    merge_rows<kMerge, 2>(a, cut, blockIdx.x, row, chunk);
  else
    merge_rows<kMerge, 16 / kMerge>(a, cut, blockIdx.x, row, chunk);
}

template <int kMerge>
static int32_t launch_merge(const Args &a, int ctas, cudaStream_t s) {
  const dim3 grid(ctas, (std::min(a.max_q, kGroupTokens) * kGroup + 31) / 32, kHeadDim / 4 / (kMergeWarps * kMerge));
  return k16v8_launch_pdl(merge_kernel<kMerge>, grid, dim3(kMergeWarps * 32), 0, s, a);
}

// ---- host side ------------------------------------------------------------

struct Layout {
  int ctas, max_rows;
  size_t lse_off, o_off, total;  // cut segments first
};

static bool layout(int32_t max_q, Layout *w) {
  const int sms = k16v8_sm_count();
  if (sms <= 0) return false;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  w->ctas = sms;
  w->max_rows = max_q <= kTileTokens ? kRows : 2 * kRows;
  const size_t rows = 2 * static_cast<size_t>(w->ctas) * w->max_rows;
  w->lse_off = up(w->ctas * sizeof(int4));
  w->o_off = w->lse_off + up(rows * sizeof(float));
  w->total = w->o_off + rows * kHeadDim * sizeof(float);
  return true;
}

template <bool kWide, bool kTest>
static int32_t launch_split(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                            const Args &a, int ctas, cudaStream_t s) {
  static bool configured[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return K16V8_ERR_CUDA;
  constexpr uint32_t smem = Smem<kWide>::kBytes;
  if (dev >= 64 || !configured[dev]) {
    if (cudaFuncSetAttribute(attention_kernel<kWide, kTest>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess)
      return K16V8_ERR_CUDA;
    if (dev < 64) configured[dev] = true;
  }
  return k16v8_launch_pdl(attention_kernel<kWide, kTest>, dim3(ctas), dim3(kThreads), smem, s, mq,
                          mk, mv, a);
}

}  // namespace attn8
}  // namespace k16v8

using namespace k16v8;

static int32_t check_attention_shape(int32_t max_q, int32_t hq, int32_t hkv, int32_t head_dim) {
  if (max_q < 0 || hq <= 0 || hkv <= 0) return K16V8_ERR_INVALID_ARG;
  if (head_dim != kHeadDim || hq / kGroup != hkv || hq % kGroup) return K16V8_ERR_UNSUPPORTED_SHAPE;
  return hkv > 4095 ? K16V8_ERR_INVALID_ARG : K16V8_OK;
}

extern "C" size_t k16v8_attention_workspace_size_k8v8(int32_t max_qlen, int32_t num_qo_heads,
                                                      int32_t num_kv_heads, int32_t head_dim) {
  attn8::Layout w;
  if (check_attention_shape(max_qlen, num_qo_heads, num_kv_heads, head_dim) != K16V8_OK ||
      !attn8::layout(max_qlen, &w))
    return 0;
  return w.total;
}

template <bool kTest>
static int32_t attention_k8v8(bool causal, const void *q, const int32_t *qo_indptr,
                              int32_t total_q, int32_t max_qlen, const uint8_t *k_cache,
                              const uint8_t *v_cache, const float *kv_scale,
                              const int32_t *block_table, int32_t max_pages_per_seq,
                              const int32_t *seq_lens, int32_t max_seq_len, int32_t batch,
                              int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                              int32_t num_pages, float sm_scale, void *workspace,
                              size_t workspace_bytes, void *out, float *lse, int32_t *dev_error,
                              void *stream) {
  int32_t st = check_attention_shape(max_qlen, num_qo_heads, num_kv_heads, head_dim);
  if (st != K16V8_OK) return st;
  if (total_q < 0 || batch < 0 || batch > attn8::kMaxBatch || num_pages <= 0 ||
      max_pages_per_seq < 0 || max_seq_len < 0 || max_seq_len > attn8::kMaxLen)
    return K16V8_ERR_INVALID_ARG;
  // a row's largest score times the scale has to be its largest scaled score
  if (!(sm_scale >= 0.f && sm_scale - sm_scale == 0.f)) return K16V8_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_pages_per_seq) * kPage < max_seq_len) return K16V8_ERR_INVALID_ARG;
  if (static_cast<int64_t>(num_pages) * num_kv_heads * kPage >= (1LL << 31))
    return K16V8_ERR_INVALID_ARG;
  if (batch == 0 || total_q == 0 || max_qlen == 0) return K16V8_OK;
  if (!q || !qo_indptr || !k_cache || !v_cache || !kv_scale ||
      (!block_table && max_pages_per_seq > 0) || !seq_lens || !workspace || !out)
    return K16V8_ERR_INVALID_ARG;
  if (!k16v8_aligned(q, 16) || !k16v8_aligned(k_cache, 16) || !k16v8_aligned(v_cache, 16) ||
      !k16v8_aligned(out, 16) || !k16v8_aligned(kv_scale, 8) || !k16v8_aligned(qo_indptr, 4) ||
      !k16v8_aligned(seq_lens, 4) || !k16v8_aligned(block_table, 4) ||
      (lse && !k16v8_aligned(lse, 4)) || !k16v8_aligned(workspace, 256))
    return K16V8_ERR_INVALID_ARG;
  attn8::Layout w;
  if (!attn8::layout(max_qlen, &w)) return K16V8_ERR_CUDA;
  if (workspace_bytes < w.total) return K16V8_ERR_WORKSPACE_TOO_SMALL;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const attn8::Args a{qo_indptr,
                      total_q,
                      max_qlen,
                      causal ? 1 : 0,
                      v_cache,
                      kv_scale,
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
  CUtensorMap mq, mk, mv;
  const uint64_t pool = static_cast<uint64_t>(num_pages) * num_kv_heads * kPage;
  if (!map_rows(&mq, q, num_qo_heads, total_q) || !map_codes(&mk, k_cache, pool) ||
      !map_codes(&mv, v_cache, pool))
    return K16V8_ERR_CUDA;
  st = max_qlen > attn8::kTileTokens ? attn8::launch_split<true, kTest>(mq, mk, mv, a, w.ctas, s)
                                     : attn8::launch_split<false, kTest>(mq, mk, mv, a, w.ctas, s);
  if (st != K16V8_OK) return st;
  // Short segments are cut by many CTAs each and want pieces in flight (8), tall ones
  // fewer CTAs (8 per 32 rows or 2).  64 and 32 dims to a CTA, both kernels: 5 rows over
  // 1,500 13.8 and 13.3 us, 8 rows at 128K 117.2 and 116.0; 20 over 8,000 121.7 and
  // 122.3, 64 x 20 to 40 of 150 to 300 42.4 and 43.1, 8 x 1024 131.9 and 133.4.
  return max_qlen > 16 ? attn8::launch_merge<4>(a, w.ctas, s)
                       : attn8::launch_merge<2>(a, w.ctas, s);
}

extern "C" int32_t k16v8_paged_prefill_attention_k8v8(
    const void *q, const int32_t *qo_indptr, int32_t total_q, int32_t max_qlen,
    const uint8_t *k_cache, const uint8_t *v_cache, const float *kv_scale,
    const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
    int32_t max_seq_len, int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t num_pages, float sm_scale, void *workspace, size_t workspace_bytes,
    void *out, float *lse, int32_t *dev_error, void *stream) {
  return attention_k8v8<false>(true, q, qo_indptr, total_q, max_qlen, k_cache, v_cache, kv_scale,
                               block_table, max_pages_per_seq, seq_lens, max_seq_len, batch,
                               num_qo_heads, num_kv_heads, head_dim, num_pages, sm_scale, workspace,
                               workspace_bytes, out, lse, dev_error, stream);
}

extern "C" int32_t k16v8_paged_cross_attention_k8v8(
    const void *q, const int32_t *qo_indptr, int32_t total_q, int32_t max_qlen,
    const uint8_t *k_cache, const uint8_t *v_cache, const float *kv_scale,
    const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
    int32_t max_seq_len, int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t num_pages, float sm_scale, void *workspace, size_t workspace_bytes,
    void *out, float *lse, int32_t *dev_error, void *stream) {
  return attention_k8v8<false>(false, q, qo_indptr, total_q, max_qlen, k_cache, v_cache, kv_scale,
                               block_table, max_pages_per_seq, seq_lens, max_seq_len, batch,
                               num_qo_heads, num_kv_heads, head_dim, num_pages, sm_scale, workspace,
                               workspace_bytes, out, lse, dev_error, stream);
}

extern "C" int32_t k16v8_paged_prefill_attention_k8v8_wait_test(
    const void *q, const int32_t *qo_indptr, int32_t total_q, int32_t max_qlen,
    const uint8_t *k_cache, const uint8_t *v_cache, const float *kv_scale,
    const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
    int32_t max_seq_len, int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t num_pages, float sm_scale, void *workspace, size_t workspace_bytes,
    void *out, float *lse, int32_t *dev_error, void *stream) {
  return attention_k8v8<true>(true, q, qo_indptr, total_q, max_qlen, k_cache, v_cache, kv_scale,
                              block_table, max_pages_per_seq, seq_lens, max_seq_len, batch,
                              num_qo_heads, num_kv_heads, head_dim, num_pages, sm_scale, workspace,
                              workspace_bytes, out, lse, dev_error, stream);
}

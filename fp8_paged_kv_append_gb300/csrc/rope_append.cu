// Rotary positions fused with the compressed-cache write: queries and keys
// are turned by their positions, keys go to the fp16 pages, values to the
// E4M3 pages, queries to the fp16 rows that the attention calls take.
//
// "Phi-4: quality transfer and interrupted throughput studies": the intro
// fixes the cache format; "Matched diagnostic profiles" names the
// compressed-cache write that this call extends.
//
// Mathematics.  Pair i of a head at position p is turned by the angle
// p * inv_freq[i]:  (a, b) -> f * (a cos - b sin, b cos + a sin), f the
// attention factor of a scaled context.  A far position times a frequency
// does not fit fp32 (at 2^17 one fp32 ulp of the angle is 2^-7 rad), so the
// angle is formed in revolutions as an unevaluated sum of two fp32 numbers,
// t = p * (inv_freq / 2pi): both products keep their rounding error through
// an FMA, whole revolutions are dropped exactly, and sincospi gets the
// fraction.  For |p| < 2^24 the fraction is off by less than 2^-25 of a
// revolution per unit frequency.
//
// HBM-bound: 43.4 us for 8,192 bf16 tokens of 40 + 10 heads, 5.56 TB/s of the
// bytes it cannot do without (0.82 of the copy rate), 28.6 us for 4,096 fp32
// tokens (0.95); with three axes 44.6 and 31.7.  A unit is 16 elements of one
// row: in the half layout dims [8c, 8c+8) and their partners half a rotary width
// on, in the interleaved layout 16 neighbouring dims -- either way frequencies
// 8c..8c+7, so one table serves both.  A CTA takes a run of units; its threads
// load their units first, compute the run's cosines and sines into shared memory
// (each once) while those loads are in flight, and then turn and store.
#include "rope_device.cuh"

namespace k16v8 {
namespace rope {

constexpr int kThreads = 128;

// kUnits units per thread.  Rows of a token: hq query heads, hkv key heads,
// hkv value heads.  kAxes: positions [axes.count][num_tokens], pair f turned by row axes[f].
template <typename T, bool kInterleaved, int kUnits, bool kAxes>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(
    const T *q, int64_t q_ts, const T *k, int64_t k_ts, const T *v, int64_t v_ts,
    const int32_t *__restrict__ positions, const PairAxes axes,
    const float *__restrict__ inv_freq, int32_t rotary, float factor,
    const int64_t *__restrict__ slot_mapping, int32_t num_tokens,
    const float *__restrict__ v_scale, __half *q_out, __half *k_cache, uint8_t *v_cache,
    int32_t num_pages, int32_t hq, int32_t hkv, int32_t *dev_error) {
  // cos, sin of the run's tokens: pair 8c + 2i + e of a token at [i][c][e], so
  // the eight lanes of a row read neighbouring 16 bytes
  extern __shared__ __align__(16) float2 table[];
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t upt = static_cast<uint32_t>(hq + 2 * hkv) * kUnitsPerRow;  // units per token
  const int64_t total = static_cast<int64_t>(num_tokens) * upt;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnits);
  const int32_t t0 = static_cast<int32_t>(first / upt);
  const uint32_t rem = static_cast<uint32_t>(first - static_cast<int64_t>(t0) * upt);
  const uint32_t run =
      static_cast<uint32_t>(min(static_cast<int64_t>(kThreads * kUnits), total - first));
  const int n_tok = (rem + run - 1) / upt + 1;
  const int half = rotary >> 1;

  // The data first: nothing of it depends on slots or positions.
  Raw<T> raw[kUnits];
  int row[kUnits], tok[kUnits], c[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const uint32_t u = j * kThreads + threadIdx.x;
    row[j] = -1;
    if (u >= run) continue;
    tok[j] = (rem + u) / upt;
    const int in_tok = rem + u - tok[j] * upt;
    row[j] = in_tok / kUnitsPerRow;
    c[j] = in_tok % kUnitsPerRow;
    const int64_t t = t0 + tok[j];
    const T *src;
    if (row[j] < hq)
      src = q + t * q_ts + row[j] * kHeadDim;
    else if (row[j] < hq + hkv)
      src = k + t * k_ts + (row[j] - hq) * kHeadDim;
    else
      src = v + t * v_ts + (row[j] - hq - hkv) * kHeadDim;
    const bool apart = !kInterleaved && row[j] < hq + hkv && 16 * c[j] < rotary;
    load8(src + (apart ? 8 : 16) * c[j], raw[j].w);
    load8(src + (apart ? 8 * c[j] + half : 16 * c[j] + 8), raw[j].w + sizeof(T) / 2);
  }
  int64_t slot[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j)
    slot[j] = row[j] >= 0 ? __ldg(slot_mapping + t0 + tok[j]) : -1;

  // (of several axes a token's positions are checked once, not by each of its units:
  // 46.3 -> 44.6 us at 8,192 tokens)
  __shared__ bool s_ok[kAxes ? kThreads * kUnits / (2 * kUnitsPerRow) + 2 : 1];
  if (kAxes && threadIdx.x < n_tok)
    s_ok[threadIdx.x] = positions_ok(positions, num_tokens, axes.count, t0 + threadIdx.x);
  for (int i = threadIdx.x; i < n_tok * half; i += kThreads) {
    const int t = i / half, f = i - t * half;
    table[t * half + ((f & 7) >> 1) * (half >> 2) + (f >> 3) * 2 + (f & 1)] =
        turn(__ldg(positions + (kAxes ? static_cast<int64_t>(axes[f]) * num_tokens : 0) + t0 + t),
             __ldg(inv_freq + f), factor);
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    if (slot[j] < 0) {  // a padding token: nothing is written for it
      row[j] = -1;
      continue;
    }
    const bool bad_slot = slot[j] >= static_cast<int64_t>(num_pages) * kPage;
    if (bad_slot || (!kAxes && !positions_ok(positions, num_tokens, 1, t0 + tok[j]))) {
      if (row[j] == 0) flag_error(dev_error, bad_slot ? K16V8_DEVERR_SLOT : K16V8_DEVERR_POSITION);
      row[j] = -1;
    }
  }
  __syncthreads();

#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    if (row[j] < 0) continue;
    if (kAxes && !s_ok[tok[j]]) {
      if (row[j] == 0) flag_error(dev_error, K16V8_DEVERR_POSITION);
      continue;
    }
    float x[8], y[8];
    widen8(raw[j].w, x, static_cast<const T *>(nullptr));
    widen8(raw[j].w + sizeof(T) / 2, y, static_cast<const T *>(nullptr));
    const uint32_t page = static_cast<uint32_t>(slot[j] >> 4), off = slot[j] & (kPage - 1);
    static_assert(kPage == 16, "slot = page * 16 + offset");
    // row of head 0 of the slot in the pool
    const int64_t pool = static_cast<int64_t>(page) * hkv * kPage + off;
    if (row[j] >= hq + hkv) {  // value: IEEE divide by the head's scale, round to E4M3
      const int h = row[j] - hq - hkv;
      const float s = __ldg(v_scale + h);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float *z = i < 2 ? x + 4 * i : y + 4 * (i - 2);
        w[i] = static_cast<uint32_t>(e4m3x2_from_f32(__fdiv_rn(z[0], s), __fdiv_rn(z[1], s))) |
               (static_cast<uint32_t>(e4m3x2_from_f32(__fdiv_rn(z[2], s), __fdiv_rn(z[3], s)))
                << 16);
      }
      *reinterpret_cast<uint4 *>(v_cache + (pool + h * kPage) * kHeadDim + 16 * c[j]) =
          make_uint4(w[0], w[1], w[2], w[3]);
      continue;
    }
    const bool rotated = 16 * c[j] < rotary;
    if (rotated) {
      const float4 *cs =
          reinterpret_cast<const float4 *>(table + tok[j] * half) + c[j];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 t2 = cs[i * (half >> 3)];  // cos, sin of two frequencies
        float &a0 = kInterleaved ? (i < 2 ? x[4 * i] : y[4 * i - 8]) : x[2 * i];
        float &b0 = kInterleaved ? (i < 2 ? x[4 * i + 1] : y[4 * i - 7]) : y[2 * i];
        float &a1 = kInterleaved ? (i < 2 ? x[4 * i + 2] : y[4 * i - 6]) : x[2 * i + 1];
        float &b1 = kInterleaved ? (i < 2 ? x[4 * i + 3] : y[4 * i - 5]) : y[2 * i + 1];
        const float ra0 = fmaf(a0, t2.x, -(b0 * t2.y)), rb0 = fmaf(b0, t2.x, a0 * t2.y);
        const float ra1 = fmaf(a1, t2.z, -(b1 * t2.w)), rb1 = fmaf(b1, t2.z, a1 * t2.w);
        a0 = ra0;
        b0 = rb0;
        a1 = ra1;
        b1 = rb1;
      }
    }
    __half *dst = row[j] < hq ? q_out + (static_cast<int64_t>(t0 + tok[j]) * hq + row[j]) * kHeadDim
                              : k_cache + (pool + (row[j] - hq) * kPage) * kHeadDim;
    const bool apart = !kInterleaved && rotated;
    *reinterpret_cast<uint4 *>(dst + (apart ? 8 : 16) * c[j]) = narrow8(x);
    *reinterpret_cast<uint4 *>(dst + (apart ? 8 * c[j] + half : 16 * c[j] + 8)) = narrow8(y);
  }
}

struct Args {
  const void *q, *k, *v;
  int64_t q_ts, k_ts, v_ts;
  const int32_t *positions;
  PairAxes axes;
  const float *inv_freq;
  int32_t rotary;
  float factor;
  const int64_t *slots;
  int32_t num_tokens;
  const float *v_scale;
  void *q_out, *k_cache;
  uint8_t *v_cache;
  int32_t num_pages, hq, hkv;
  int32_t *dev_error;
};

template <typename T, bool kInterleaved, int kUnits, bool kAxes>
static int32_t launch(const Args &a, cudaStream_t stream) {
  const int upt = (a.hq + 2 * a.hkv) * kUnitsPerRow;
  const int64_t total = static_cast<int64_t>(a.num_tokens) * upt;
  const int64_t blocks = (total + kThreads * kUnits - 1) / (kThreads * kUnits);
  if (blocks > 0x7fffffffLL) return K16V8_ERR_INVALID_ARG;
  // a run of units touches at most this many tokens
  const int toks = (kThreads * kUnits - 2) / upt + 2;
  const size_t smem = static_cast<size_t>(toks) * (a.rotary / 2) * sizeof(float2);
  return k16v8_launch_pdl(rope_append_kernel<T, kInterleaved, kUnits, kAxes>,
                          dim3(static_cast<unsigned>(blocks)), dim3(kThreads), smem, stream,
                          static_cast<const T *>(a.q), a.q_ts, static_cast<const T *>(a.k), a.k_ts,
                          static_cast<const T *>(a.v), a.v_ts, a.positions, a.axes, a.inv_freq,
                          a.rotary, a.factor, a.slots, a.num_tokens, a.v_scale,
                          static_cast<__half *>(a.q_out), static_cast<__half *>(a.k_cache),
                          a.v_cache, a.num_pages, a.hq, a.hkv, a.dev_error);
}

// 64 bytes of a thread's input in flight: one fp32 unit or two 16-bit ones,
// except where that leaves SMs without a CTA.  Two 16-bit units against one,
// GB300: 43.4 against 47.2 us at 8,192 tokens of 40 + 10 heads, 3.6 against 4.1
// at 256, 3.1 against 2.5 at 32 (60 CTAs); two fp32 units against one: 29.2
// against 28.6 us at 4,096 tokens.  (CTAs of 256 threads: 45.0 and 29.4 us.)
template <typename T, bool kAxes>
static int32_t dispatch(const Args &a, bool interleaved, cudaStream_t stream) {
  if constexpr (sizeof(T) == 2) {
    const int64_t units = static_cast<int64_t>(a.num_tokens) * (a.hq + 2 * a.hkv) * kUnitsPerRow;
    const int sms = k16v8_sm_count();
    if (sms <= 0) return K16V8_ERR_CUDA;
    if (units >= static_cast<int64_t>(sms) * 2 * kThreads)
      return interleaved ? launch<T, true, 2, kAxes>(a, stream) : launch<T, false, 2, kAxes>(a, stream);
  }
  return interleaved ? launch<T, true, 1, kAxes>(a, stream) : launch<T, false, 1, kAxes>(a, stream);
}

}  // namespace rope
}  // namespace k16v8

using namespace k16v8;

template <bool kAxes>
static int32_t rope_kv_append(
    const void *q, int64_t q_token_stride, const void *k, int64_t k_token_stride, const void *v,
    int64_t v_token_stride, int32_t x_dtype, const int32_t *positions,
    int32_t num_axes, const int8_t *pair_axis, const float *inv_freq,
    int32_t rotary_dim, int32_t interleaved, float attn_factor, const int64_t *slot_mapping,
    int32_t num_tokens, const float *v_scale, void *q_out, void *k_cache, uint8_t *v_cache,
    int32_t num_pages, int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t *dev_error, void *stream) {
  if (num_tokens < 0 || num_qo_heads < 0 || num_kv_heads <= 0 || num_pages <= 0)
    return K16V8_ERR_INVALID_ARG;
  if (num_qo_heads > 65535 || num_kv_heads > 65535) return K16V8_ERR_INVALID_ARG;
  if (head_dim != kHeadDim) return K16V8_ERR_UNSUPPORTED_SHAPE;
  if (rotary_dim < 16 || rotary_dim > kHeadDim || rotary_dim % 16)
    return K16V8_ERR_UNSUPPORTED_SHAPE;
  if (x_dtype != K16V8_F16 && x_dtype != K16V8_F32 && x_dtype != K16V8_BF16)
    return K16V8_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return K16V8_ERR_INVALID_ARG;
  if (!(attn_factor - attn_factor == 0.f)) return K16V8_ERR_INVALID_ARG;  // finite
  rope::PairAxes axes{0, 0, 1};
  if (kAxes && (num_axes < 1 || num_axes > K16V8_MAX_ROPE_AXES || !pair_axis ||
                !rope::pack_axes(pair_axis, rotary_dim / 2, num_axes, &axes)))
    return K16V8_ERR_INVALID_ARG;
  if (num_tokens == 0) return K16V8_OK;
  if ((num_qo_heads > 0 && (!q || !q_out)) || !k || !v || !positions || !inv_freq ||
      !slot_mapping || !v_scale || !k_cache || !v_cache)
    return K16V8_ERR_INVALID_ARG;
  const int64_t q_row = static_cast<int64_t>(num_qo_heads) * head_dim;
  const int64_t kv_row = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (q_token_stride == 0) q_token_stride = q_row;
  if (k_token_stride == 0) k_token_stride = kv_row;
  if (v_token_stride == 0) v_token_stride = kv_row;
  if (q_token_stride < q_row || k_token_stride < kv_row || v_token_stride < kv_row)
    return K16V8_ERR_INVALID_ARG;
  const int64_t per16 = x_dtype == K16V8_F32 ? 4 : 8;  // elements of a 16-byte access
  if (q_token_stride % per16 || k_token_stride % per16 || v_token_stride % per16)
    return K16V8_ERR_INVALID_ARG;
  if ((num_qo_heads > 0 && (!k16v8_aligned(q, 16) || !k16v8_aligned(q_out, 16))) ||
      !k16v8_aligned(k, 16) || !k16v8_aligned(v, 16) || !k16v8_aligned(k_cache, 16) ||
      !k16v8_aligned(v_cache, 16) || !k16v8_aligned(slot_mapping, 8) ||
      !k16v8_aligned(positions, 4) || !k16v8_aligned(inv_freq, 4) || !k16v8_aligned(v_scale, 4))
    return K16V8_ERR_INVALID_ARG;
  const rope::Args a{q,           k,         v,       q_token_stride, k_token_stride,
                     v_token_stride, positions, axes, inv_freq, rotary_dim, attn_factor,
                     slot_mapping, num_tokens, v_scale, q_out,          k_cache,
                     v_cache,     num_pages, num_qo_heads, num_kv_heads, dev_error};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (x_dtype == K16V8_F32) return rope::dispatch<float, kAxes>(a, interleaved != 0, s);
  if (x_dtype == K16V8_BF16) return rope::dispatch<__nv_bfloat16, kAxes>(a, interleaved != 0, s);
  return rope::dispatch<__half, kAxes>(a, interleaved != 0, s);
}

extern "C" int32_t k16v8_rope_kv_append(
    const void *q, int64_t q_token_stride, const void *k, int64_t k_token_stride, const void *v,
    int64_t v_token_stride, int32_t x_dtype, const int32_t *positions, const float *inv_freq,
    int32_t rotary_dim, int32_t interleaved, float attn_factor, const int64_t *slot_mapping,
    int32_t num_tokens, const float *v_scale, void *q_out, void *k_cache, uint8_t *v_cache,
    int32_t num_pages, int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t *dev_error, void *stream) {
  return rope_kv_append<false>(q, q_token_stride, k, k_token_stride, v, v_token_stride, x_dtype,
                               positions, 1, nullptr, inv_freq, rotary_dim, interleaved,
                               attn_factor, slot_mapping, num_tokens, v_scale, q_out, k_cache,
                               v_cache, num_pages, num_qo_heads, num_kv_heads, head_dim, dev_error,
                               stream);
}

extern "C" int32_t k16v8_rope_axes_kv_append(
    const void *q, int64_t q_token_stride, const void *k, int64_t k_token_stride, const void *v,
    int64_t v_token_stride, int32_t x_dtype, const int32_t *positions, int32_t num_axes,
    const int8_t *pair_axis, const float *inv_freq, int32_t rotary_dim, int32_t interleaved,
    float attn_factor, const int64_t *slot_mapping, int32_t num_tokens, const float *v_scale,
    void *q_out, void *k_cache, uint8_t *v_cache, int32_t num_pages, int32_t num_qo_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t *dev_error, void *stream) {
  return rope_kv_append<true>(q, q_token_stride, k, k_token_stride, v, v_token_stride, x_dtype,
                              positions, num_axes, pair_axis, inv_freq, rotary_dim, interleaved,
                              attn_factor, slot_mapping, num_tokens, v_scale, q_out, k_cache,
                              v_cache, num_pages, num_qo_heads, num_kv_heads, head_dim, dev_error,
                              stream);
}

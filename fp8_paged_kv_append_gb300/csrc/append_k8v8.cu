// The cache write of the K8/V8 cache, with rotary positions of one or several
// axes on the way: queries to fp16 rows, keys and values to E4M3 pages whose
// scales it chooses.
//
// "Phi-4: quality transfer and interrupted throughput studies": the cache
// write and the page pool; a scale per page and head in place of one per head
// is this library's.
//
// Mathematics.  With x the rows that the call puts into a page (keys turned by
// their positions, in fp32), s = 2^e the smallest power of two with
// max |x| <= 448 s, within [2^-15, 2^7]; not below the page's scale where it
// holds rows of earlier calls.  code = E4M3(x / s): the division is exact, so a
// code is one rounding from x.  Where s has grown, the rows that were there are
// rounded again: code' = E4M3(code * s_old / s), which changes nothing but codes
// that become subnormal.  Infinities and NaN do not take part in max |x|.
//
// A call says which sequences get how many new last positions, so the rows of a
// page are known from the lengths: a page and head belong to one warp, which
// holds all new rows in registers between the maximum and the rounding.  No
// row is read twice, nothing depends on an order.
//
// A task is up to 16 rows of one page and head (of K, V or a query head), a
// lane holding four units of 16 elements.  A CTA takes the tasks of one page
// and some KV heads (with their share of the query heads) and shares the
// cosines and sines of the page's tokens.
//
// HBM-bound where there are many tokens: 41.7 us for 8,192 bf16 tokens of 40 + 10
// heads, 5.5 TB/s of the bytes it cannot do without (0.81 of the copy rate; without
// rotation 37.3, 0.91), 45 for as many fp16 ones (0.75), 34.6 for 4,096 fp32 ones
// (0.76); 24,000 bf16 states without queries and rotation 33.1 (0.82).  A step of 32
// sequences takes 4.8 us, one launch with four dependent loads (rows, table entry,
// positions, held scale), of 8,192 66 (0.51 of the copy rate).  A step in which every
// page's scales grow codes the held rows again one after another, a load and a store
// each: 32 sequences 11.3 us, 256 12.1, 1,024 23.6 (4.7, 5.6 and 10.4 without).
#include <algorithm>

#include "k8v8_device.cuh"
#include "rope_device.cuh"

namespace k16v8 {
namespace append8 {

using rope::kUnitsPerRow;
using rope::load8;
using rope::narrow8;
using rope::Raw;
using rope::widen8;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// 16-bit rows: 80 registers and 24 warps per SM, 41.7 us for 8,192 tokens of 40 + 10
// heads (5: 43.5, 7: 44.2; the turned rows kept in registers, 128 of them, 4 us more;
// the next task's rows loaded into each unit's registers as it is stored 48.0).  In 80,
// fp16 prompts spill 28 to 36 bytes of a thread and interleaved bf16 ones 24; steps take
// 96 (256 sequences 5.6 us, with 6 per SM 5.8; the bf16 form of apart halves spills 4
// bytes in them).  fp32 rows take 162 to 168 (2 to 4 per SM alike).
template <typename T, bool kStep>
constexpr int kCtasPerSm = sizeof(T) == 2 ? (kStep ? 5 : 6) : 3;
constexpr int kUnits = kPage * kUnitsPerRow / 32;  // of a lane and task

struct Args {
  const void *q, *k, *v;
  int64_t q_ts, k_ts, v_ts;
  const int32_t *qo_indptr;
  int32_t num_tokens;
  const int32_t *positions;
  rope::PairAxes axes;
  const float *inv_freq;
  int32_t rotary;
  float factor;
  const int32_t *block_table;
  int32_t maxp;
  const int32_t *seq_lens;
  int32_t batch;
  __half *q_out;
  uint8_t *k_cache, *v_cache;
  float *kv_scale;
  int32_t num_pages, hq, hkv;
  int32_t *dev_error;
};

// New rows and length of sequence b; false for what is out of range.
__device__ __forceinline__ bool sequence(const Args &a, int b, int &q0, int &n, int &L) {
  q0 = __ldg(a.qo_indptr + b);
  L = __ldg(a.seq_lens + b);
  const int64_t rows = static_cast<int64_t>(__ldg(a.qo_indptr + b + 1)) - q0;
  n = static_cast<int>(rows);
  return q0 >= 0 && rows >= 0 && rows <= a.num_tokens - q0 && rows <= L &&
         L <= static_cast<int64_t>(a.maxp) * kPage;
}

// Turns a unit: frequencies 8c .. 8c + 7 of a row whose table is cs.
template <bool kInterleaved>
__device__ __forceinline__ void turn_unit(float (&x)[8], float (&y)[8], const float4 *cs,
                                          int half) {
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

// Makes the compiler read these words again, in place of what it computed from them.
template <typename T>
__device__ __forceinline__ void keep(Raw<T> &r) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)); ++i)
    asm volatile("" : "+r"(r.w[i].x), "+r"(r.w[i].y), "+r"(r.w[i].z), "+r"(r.w[i].w));
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = static_cast<uint32_t>(e4m3x2_from_f32(x[4 * i] * inv, x[4 * i + 1] * inv)) |
           (static_cast<uint32_t>(e4m3x2_from_f32(x[4 * i + 2] * inv, x[4 * i + 3] * inv)) << 16);
  return make_uint2(w[0], w[1]);
}

// Four codes times a power of two, rounded again.
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float ratio) {
  const float2 a = __half22float2(e4m3x2_to_half2(static_cast<uint16_t>(w & 0xffffu)));
  const float2 b = __half22float2(e4m3x2_to_half2(static_cast<uint16_t>(w >> 16)));
  return static_cast<uint32_t>(e4m3x2_from_f32(a.x * ratio, a.y * ratio)) |
         (static_cast<uint32_t>(e4m3x2_from_f32(b.x * ratio, b.y * ratio)) << 16);
}

// Items: the pages that sequences may write, an upper bound.  Those of sequence b start
// at item
//   qo_indptr[b] / 16 + 2b  -- room for every page that its rows can touch, or
//   qo_indptr[b]            -- kStep: a page per token, for calls of about one each.
template <bool kStep>
__device__ __forceinline__ int first_item(const Args &a, int b) {
  const int q0 = __ldg(a.qo_indptr + b);
  return kStep ? q0 : (q0 >> 4) + 2 * b;
}

// grid: (items; parts of the heads).  kStep: a part is kStepTasks tasks, which pages of
// one new row take at once, 8 lanes each.
constexpr int kStepTasks = kWarps * 4 * kUnits;

template <typename T, bool kInterleaved, bool kStep>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<T, kStep>)
    append_k8v8_kernel(const Args a, int kv_per_cta, int q_per_cta) {
  extern __shared__ __align__(16) float2 table[];  // pair 8c + 2i + e of a token at [i][c][e]
  __shared__ int s_last[2][kWarps];
  __shared__ int s_seq[3][kThreads];  // q0, n, L of the sequences looked at
  __shared__ uint32_t s_live;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int item = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();

  if (blockIdx.y == 0 && item <= a.batch / kThreads && item * kThreads + tid < a.batch) {
    int q0, n, L;
    if (!sequence(a, item * kThreads + tid, q0, n, L)) flag_error(a.dev_error, K16V8_DEVERR_SEQLEN);
  }
  // The item's sequence is the last (of those in range) that starts at or before it: by
  // the start alone down to as many as there are threads, then among those in range.
  int low = 0, count = a.batch, round = 0;
  auto last_of = [&](bool before) {  // the last thread for which it holds, -1: none
    const int mine = __reduce_max_sync(kFull, before ? tid : -1);
    if (lane == 0) s_last[round & 1][warp] = mine;
    __syncthreads();
    int last = -1;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) last = max(last, s_last[round & 1][w]);
    ++round;
    return last;
  };
  while (count > kThreads) {
    const int step = (count + kThreads - 1) / kThreads, at = tid * step;
    const int last = last_of(at < count && first_item<kStep>(a, low + at) <= item);
    if (last < 0) return;
    low += last * step;
    count = min(step, count - last * step);
  }
  bool before = false;
  if (tid < count) {
    int q0, n, L;
    before = sequence(a, low + tid, q0, n, L) && first_item<kStep>(a, low + tid) <= item;
    s_seq[0][tid] = q0;
    s_seq[1][tid] = n;
    s_seq[2][tid] = L;
  }
  const int at = last_of(before);
  if (at < 0) return;
  const int b = low + at;
  const int q0 = s_seq[0][at], n = s_seq[1][at], L = s_seq[2][at];
  if (n == 0) return;
  const int first = L - n;  // the first new position
  const int page = first / kPage + (item - (kStep ? q0 : (q0 >> 4) + 2 * b));
  if (page > (L - 1) / kPage || page < first / kPage) return;
  const int p0 = max(page * kPage, first), p1 = min(page * kPage + kPage, L);
  const int rows = p1 - p0, lo = p0 - page * kPage;  // new rows, from this offset on
  const int64_t t0 = q0 + (p0 - first);
  const int pid = __ldg(a.block_table + static_cast<int64_t>(b) * a.maxp + page);

  // Tasks: keys and values of the part's KV heads, then its query heads.
  const int h0 = kStep ? 0 : blockIdx.y * kv_per_cta, nh = min(kStep ? a.hkv : kv_per_cta, a.hkv - h0);
  const int qh0 = kStep ? 0 : blockIdx.y * q_per_cta;
  const int nq = max(0, min(kStep ? a.hq : q_per_cta, a.hq - qh0));
  const int all = 2 * max(nh, 0) + nq;
  // of this warp
  const int task0 = kStep ? blockIdx.y * kStepTasks + warp * (kStepTasks / kWarps) : warp;
  const int task1 = kStep ? min(all, task0 + kStepTasks / kWarps) : all;
  const int stride = kStep ? 1 : kWarps;
  const int half = a.rotary >> 1;
  const int c = lane % kUnitsPerRow, r0 = lane / kUnitsPerRow;  // rows r0, r0 + 4, ...
  const bool turned_unit = 16 * c < a.rotary;

  Raw<T> raw[kUnits];
  // row 0 of a task's 16 dims c (and, where a pair's halves are apart, their partners)
  auto rows_of = [&](int task, const T *&src, int64_t &ts, bool &apart) {
    const bool is_v = task >= nh && task < 2 * nh;
    if (task < nh) {
      src = static_cast<const T *>(a.k) + (h0 + task) * kHeadDim;
      ts = a.k_ts;
    } else if (is_v) {
      src = static_cast<const T *>(a.v) + (h0 + task - nh) * kHeadDim;
      ts = a.v_ts;
    } else {
      src = static_cast<const T *>(a.q) + (qh0 + task - 2 * nh) * kHeadDim;
      ts = a.q_ts;
    }
    apart = !kInterleaved && !is_v && turned_unit;
  };
  auto load = [&](int task) {
    const T *src;
    int64_t ts;
    bool apart;
    rows_of(task, src, ts, apart);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int r = r0 + 4 * i;
      if (r >= rows) continue;
      const T *p = src + (t0 + r) * ts;
      load8(p + (apart ? 8 : 16) * c, raw[i].w);
      load8(p + (apart ? 8 * c + half : 16 * c + 8), raw[i].w + sizeof(T) / 2);
    }
  };
  const bool single = kStep && rows == 1;  // unit i of a lane: task task0 + 4i + r0
  if (single) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if (task0 + 4 * i + r0 >= task1) continue;
      const T *src;
      int64_t ts;
      bool apart;
      rows_of(task0 + 4 * i + r0, src, ts, apart);
      src += t0 * ts;
      load8(src + (apart ? 8 : 16) * c, raw[i].w);
      load8(src + (apart ? 8 * c + half : 16 * c + 8), raw[i].w + sizeof(T) / 2);
    }
  } else if (task0 < task1) {
    load(task0);
  }
  if (pid < 0 || pid >= a.num_pages) {
    if (tid == 0 && blockIdx.y == 0) flag_error(a.dev_error, K16V8_DEVERR_PAGE);
    return;
  }

  if (warp == 0) {  // rows whose positions are in range
    bool ok = lane < rows;
    if (ok && half > 0 && !rope::positions_ok(a.positions, a.num_tokens, a.axes.count, t0 + lane)) {
      if (blockIdx.y == 0) flag_error(a.dev_error, K16V8_DEVERR_POSITION);
      ok = false;
    }
    const uint32_t live = __ballot_sync(kFull, ok);
    if (lane == 0) s_live = live;
  }
  if (half > 0) {  // a thread's frequency stays (half <= 64: a pass takes two tokens or more)
    const int per_pass = kThreads / half, f = tid % half;
    if (tid < per_pass * half) {
      const int32_t *pos = a.positions + static_cast<int64_t>(a.axes[f]) * a.num_tokens + t0;
      const float freq = __ldg(a.inv_freq + f);
      float2 *to = table + ((f & 7) >> 1) * (half >> 2) + (f >> 3) * 2 + (f & 1);
#pragma unroll 2
      for (int t = tid / half; t < rows; t += per_pass)
        to[t * half] = rope::turn(__ldg(pos + t), freq, a.factor);
    }
  }
  __syncthreads();
  const uint32_t live = s_live;
  if (live == 0) return;

  if (single) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int task = task0 + 4 * i + r0;
      const bool is_v = task >= nh && task < 2 * nh, turns = !is_v && turned_unit;
      const bool apart = !kInterleaved && turns, on = task < task1;
      float x[8], y[8], top = 0.f;
      if (on) {
        widen8(raw[i].w, x, static_cast<const T *>(nullptr));
        widen8(raw[i].w + sizeof(T) / 2, y, static_cast<const T *>(nullptr));
        if (turns) turn_unit<kInterleaved>(x, y, reinterpret_cast<const float4 *>(table) + c, half);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float ax = fabsf(x[e]), ay = fabsf(y[e]);
          top = fmaxf(top, fmaxf(ax < INFINITY ? ax : 0.f, ay < INFINITY ? ay : 0.f));
        }
      }
#pragma unroll
      for (int o = kUnitsPerRow / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      const bool cached = on && task < 2 * nh;
      const int64_t tile = static_cast<int64_t>(pid) * a.hkv + (is_v ? task - nh : task);
      float *scale = a.kv_scale + tile * 2 + (is_v ? 1 : 0);
      const float held = cached && lo > 0 ? *scale : 0.f;
      __syncwarp();  // every lane of the row has read the old scale
      if (on && !cached) {
        __half *dst = a.q_out + (t0 * a.hq + task - 2 * nh) * kHeadDim;
        *reinterpret_cast<uint4 *>(dst + (apart ? 8 : 16) * c) = narrow8(x);
        *reinterpret_cast<uint4 *>(dst + (apart ? 8 * c + half : 16 * c + 8)) = narrow8(y);
      }
      if (!cached) continue;
      uint8_t *codes = (is_v ? a.v_cache : a.k_cache) + tile * k8v8::kTileBytes;
      int e = k8v8::scale_exponent(top);
      if (lo > 0) {
        e = max(e, k8v8::stored_exponent(held));
        const float ratio = held / k8v8::exp2_int(e);
        if (ratio != 1.f) {
          for (int r = 0; r < lo; ++r) {
            uint4 *p = reinterpret_cast<uint4 *>(codes + r * kHeadDim) + c;
            const uint4 w = *p;
            *p = make_uint4(rescaled(w.x, ratio), rescaled(w.y, ratio), rescaled(w.z, ratio),
                            rescaled(w.w, ratio));
          }
        }
      }
      if (c == 0) *scale = k8v8::exp2_int(e);
      const float inv = k8v8::exp2_int(-e);
      uint8_t *dst = codes + lo * kHeadDim;
      const uint2 cx = codes8(x, inv), cy = codes8(y, inv);
      if (apart) {
        *reinterpret_cast<uint2 *>(dst + 8 * c) = cx;
        *reinterpret_cast<uint2 *>(dst + 8 * c + half) = cy;
      } else {
        *reinterpret_cast<uint4 *>(dst + 16 * c) = make_uint4(cx.x, cx.y, cy.x, cy.y);
      }
    }
    return;
  }

  for (int task = task0; task < task1; task += stride) {
    if (task != task0) load(task);
    const bool is_k = task < nh, is_v = !is_k && task < 2 * nh;
    const bool turns = !is_v && turned_unit;
    const bool apart = !kInterleaved && turns;
    // a unit of this lane, turned; 16-bit rows stay as they were loaded and are turned
    // again for the codes, which costs less than the registers of their turned form
    auto unit = [&](int i, float (&x)[8], float (&y)[8]) {
      widen8(raw[i].w, x, static_cast<const T *>(nullptr));
      widen8(raw[i].w + sizeof(T) / 2, y, static_cast<const T *>(nullptr));
      if (turns)
        turn_unit<kInterleaved>(
            x, y, reinterpret_cast<const float4 *>(table + (r0 + 4 * i) * half) + c, half);
    };
    if (!is_k && !is_v) {  // a query head
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int r = r0 + 4 * i;
        if (!(live >> r & 1)) continue;
        float x[8], y[8];
        unit(i, x, y);
        __half *dst = a.q_out + ((t0 + r) * a.hq + qh0 + task - 2 * nh) * kHeadDim;
        *reinterpret_cast<uint4 *>(dst + (apart ? 8 : 16) * c) = narrow8(x);
        *reinterpret_cast<uint4 *>(dst + (apart ? 8 * c + half : 16 * c + 8)) = narrow8(y);
      }
      continue;
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if (!(live >> (r0 + 4 * i) & 1)) continue;
      float x[8], y[8];
      unit(i, x, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fmaxf(fabsf(x[e]), fabsf(y[e])));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    if (top == INFINITY) {  // (seldom) the largest finite value
      top = 0.f;
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        if (!(live >> (r0 + 4 * i) & 1)) continue;
        float x[8], y[8];
        unit(i, x, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float ax = fabsf(x[e]), ay = fabsf(y[e]);
          top = fmaxf(top, fmaxf(ax < INFINITY ? ax : 0.f, ay < INFINITY ? ay : 0.f));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    }
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < kUnits; ++i) keep(raw[i]);
    }
    const int h = is_k ? h0 + task : h0 + task - nh;
    const int64_t tile = static_cast<int64_t>(pid) * a.hkv + h;
    float *scale = a.kv_scale + tile * 2 + (is_v ? 1 : 0);
    uint8_t *codes = (is_v ? a.v_cache : a.k_cache) + tile * k8v8::kTileBytes;
    int e = k8v8::scale_exponent(top);
    if (lo > 0) {
      const float held = *scale;
      e = max(e, k8v8::stored_exponent(held));
      const float ratio = held / k8v8::exp2_int(e);
      if (ratio != 1.f) {  // the rows that were there take the new scale
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
          const int r = r0 + 4 * i;
          if (r >= lo) continue;
          uint4 *p = reinterpret_cast<uint4 *>(codes + r * kHeadDim) + c;
          const uint4 w = *p;
          *p = make_uint4(rescaled(w.x, ratio), rescaled(w.y, ratio), rescaled(w.z, ratio),
                          rescaled(w.w, ratio));
        }
      }
      __syncwarp();  // every lane has read the old scale
    }
    if (lane == 0) *scale = k8v8::exp2_int(e);
    const float inv = k8v8::exp2_int(-e);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int r = r0 + 4 * i;
      if (!(live >> r & 1)) continue;
      float x[8], y[8];
      unit(i, x, y);
      uint8_t *dst = codes + (lo + r) * kHeadDim;
      const uint2 cx = codes8(x, inv), cy = codes8(y, inv);
      if (apart) {
        *reinterpret_cast<uint2 *>(dst + 8 * c) = cx;
        *reinterpret_cast<uint2 *>(dst + 8 * c + half) = cy;
      } else {
        *reinterpret_cast<uint4 *>(dst + 16 * c) = make_uint4(cx.x, cx.y, cy.x, cy.y);
      }
    }
  }
}

template <typename T, bool kInterleaved>
static int32_t launch(const Args &a, cudaStream_t stream) {
  const int sms = k16v8_sm_count();
  if (sms <= 0) return K16V8_ERR_CUDA;
  const size_t smem = static_cast<size_t>(kPage) * (a.rotary / 2) * sizeof(float2);
  const int checks = (a.batch + kThreads - 1) / kThreads;  // CTAs that look for bad sequences
  // Calls of about a token per sequence: a CTA holds all heads of a token's page.  So and
  // by pages with parts of the heads: 32 sequences 4.8 and 5.1 us, 256 5.6 and 12.0, 1,024
  // 13.2 and 42, 8,192 66 and 321; two tokens each, where its rows wait for one another,
  // 256 26.7 and 13.8, 1,024 53 and 46.  (The average decides: 256 single rows beside a
  // chunk of 512 tokens go by pages, 15.7 us, alone they take 5.6 and 7.2.)
  if (4LL * a.num_tokens <= 5LL * a.batch) {
    const int parts = (2 * a.hkv + a.hq + kStepTasks - 1) / kStepTasks;
    return k16v8_launch_pdl(append_k8v8_kernel<T, kInterleaved, true>,
                            dim3(static_cast<unsigned>(std::max(a.num_tokens, checks)), parts),
                            dim3(kThreads), smem, stream, a, 0, 0);
  }
  const int64_t items = a.num_tokens / kPage + 2LL * a.batch;
  // Two KV heads share a table where there are pages enough.  Two and one: 8,192 bf16
  // tokens 41.7 and 48.7 us, 64 of 32 to 64 fp16 20.5 and 22.5; 5 x 300 fp32 of 2 heads (about 100
  // items) 7.7 and 6.6.  (Three to five: 44 to 51 for the first.)
  const int kv_per_cta = items * a.hkv >= 8LL * sms ? 2 : 1;
  const int parts = (a.hkv + kv_per_cta - 1) / kv_per_cta;
  const int q_per_cta = (a.hq + parts - 1) / parts;
  return k16v8_launch_pdl(append_k8v8_kernel<T, kInterleaved, false>,
                          dim3(static_cast<unsigned>(items), parts), dim3(kThreads), smem, stream,
                          a, kv_per_cta, q_per_cta);
}

template <typename T>
static int32_t dispatch(const Args &a, bool interleaved, cudaStream_t s) {
  return interleaved ? launch<T, true>(a, s) : launch<T, false>(a, s);
}

}  // namespace append8
}  // namespace k16v8

using namespace k16v8;

extern "C" int32_t k16v8_rope_kv_append_k8v8(
    const void *q, int64_t q_token_stride, const void *k, int64_t k_token_stride, const void *v,
    int64_t v_token_stride, int32_t x_dtype, const int32_t *qo_indptr, int32_t num_tokens,
    const int32_t *positions, int32_t num_axes, const int8_t *pair_axis, const float *inv_freq,
    int32_t rotary_dim, int32_t interleaved, float attn_factor, const int32_t *block_table,
    int32_t max_pages_per_seq, const int32_t *seq_lens, int32_t batch, void *q_out,
    uint8_t *k_cache, uint8_t *v_cache, float *kv_scale, int32_t num_pages, int32_t num_qo_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t *dev_error, void *stream) {
  if (num_tokens < 0 || batch < 0 || num_qo_heads < 0 || num_kv_heads <= 0 || num_pages <= 0 ||
      max_pages_per_seq < 0)
    return K16V8_ERR_INVALID_ARG;
  if (num_qo_heads > 65535 || num_kv_heads > 65535 || batch > 65535) return K16V8_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_pages_per_seq) * kPage >= (1LL << 31)) return K16V8_ERR_INVALID_ARG;
  if (head_dim != kHeadDim) return K16V8_ERR_UNSUPPORTED_SHAPE;
  if (rotary_dim < 0 || rotary_dim > kHeadDim || rotary_dim % 16)
    return K16V8_ERR_UNSUPPORTED_SHAPE;
  if (x_dtype != K16V8_F16 && x_dtype != K16V8_F32 && x_dtype != K16V8_BF16)
    return K16V8_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return K16V8_ERR_INVALID_ARG;
  if (!(attn_factor - attn_factor == 0.f)) return K16V8_ERR_INVALID_ARG;  // finite
  rope::PairAxes axes{0, 0, 1};
  if (rotary_dim > 0 && (num_axes < 1 || num_axes > K16V8_MAX_ROPE_AXES || !pair_axis ||
                         !rope::pack_axes(pair_axis, rotary_dim / 2, num_axes, &axes)))
    return K16V8_ERR_INVALID_ARG;
  if (num_tokens == 0 || batch == 0) return K16V8_OK;
  if ((num_qo_heads > 0 && (!q || !q_out)) || !k || !v || !qo_indptr ||
      (!block_table && max_pages_per_seq > 0) || !seq_lens || !k_cache || !v_cache || !kv_scale ||
      (rotary_dim > 0 && (!positions || !inv_freq)))
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
      !k16v8_aligned(v_cache, 16) || !k16v8_aligned(kv_scale, 8) ||
      !k16v8_aligned(qo_indptr, 4) || !k16v8_aligned(block_table, 4) ||
      !k16v8_aligned(seq_lens, 4) ||
      (rotary_dim > 0 && (!k16v8_aligned(positions, 4) || !k16v8_aligned(inv_freq, 4))))
    return K16V8_ERR_INVALID_ARG;
  const append8::Args a{q,
                        k,
                        v,
                        q_token_stride,
                        k_token_stride,
                        v_token_stride,
                        qo_indptr,
                        num_tokens,
                        positions,
                        axes,
                        inv_freq,
                        rotary_dim,
                        attn_factor,
                        block_table,
                        max_pages_per_seq,
                        seq_lens,
                        batch,
                        static_cast<__half *>(q_out),
                        k_cache,
                        v_cache,
                        kv_scale,
                        num_pages,
                        num_qo_heads,
                        num_kv_heads,
                        dev_error};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (x_dtype == K16V8_F32) return append8::dispatch<float>(a, interleaved != 0, s);
  if (x_dtype == K16V8_BF16) return append8::dispatch<__nv_bfloat16>(a, interleaved != 0, s);
  return append8::dispatch<__half>(a, interleaved != 0, s);
}

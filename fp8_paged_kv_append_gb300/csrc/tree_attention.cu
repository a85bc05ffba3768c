// Attention of drafted token trees over the paged K16/V8 cache.
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
//
// Design.  As in decode, a warp streams pages (16 tokens of K and V) through
// a private ring of bulk-async copies, and the four query heads of a GQA group
// share every page.  The rows of an MMA tile are 4 nodes x 4 heads (row =
// node * 4 + head): S = Q K^T and O += P V on m16n8k16 with fp32
// accumulators, kTiles row tiles per warp.
//  * Q.K: a dot product does not depend on which dims an MMA's K index
//    stands for as long as both operands agree, so a lane owns the same 32 dims
//    of its two query rows and of its two key rows (tokens g and g + 8).
//  * P.V: the score accumulators are the P operand as they stand.  A V
//    operand pairs two tokens of one dim: two rows' bytes are interleaved
//    (prmt) and widened E4M3 -> fp16 pairs.  Which dims an MMA's columns
//    stand for is free as well: lane group g owns dims [16g, 16g + 16).
//  * The running max moves only when a row's max grows by more than 2^8
//    (exact: the final division uses the same max), so O is seldom rescaled.
//  * Masks are looked at only in pages that reach into the tree; there a NaN
//    value code counts only in rows that see its token (a second MMA over
//    indicators, taken only when a code is NaN).
#include <math.h>

#include <algorithm>

#include "decode_page.cuh"

namespace k16v8 {
namespace tree {

constexpr int kTreeStages = 4;

struct __align__(128) Ring {
  uint8_t k[kTreeStages][kKPageBytes];
  uint8_t v[kTreeStages][kVPageBytes];
};

// Shared memory: the rings (the warps' states are joined over them), every
// warp's barriers (apart: memory of a live mbarrier takes no other writes),
// the page ids of the chunk.
constexpr size_t kBarOffset = kWarps * sizeof(Ring);
constexpr size_t kIdsOffset = kBarOffset + kWarps * kTreeStages * sizeof(uint64_t);

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Two tokens' bytes of 4 neighbouring dims -> 4 fp16 pairs (token a low).
__device__ __forceinline__ void pair_tokens(uint32_t a, uint32_t b, uint32_t (&out)[4]) {
  const uint32_t lo = __byte_perm(a, b, 0x5140), hi = __byte_perm(a, b, 0x7362);
  const __half2 h0 = e4m3x2_to_half2(static_cast<uint16_t>(lo & 0xffffu));
  const __half2 h1 = e4m3x2_to_half2(static_cast<uint16_t>(lo >> 16));
  const __half2 h2 = e4m3x2_to_half2(static_cast<uint16_t>(hi & 0xffffu));
  const __half2 h3 = e4m3x2_to_half2(static_cast<uint16_t>(hi >> 16));
  out[0] = *reinterpret_cast<const uint32_t *>(&h0);
  out[1] = *reinterpret_cast<const uint32_t *>(&h1);
  out[2] = *reinterpret_cast<const uint32_t *>(&h2);
  out[3] = *reinterpret_cast<const uint32_t *>(&h3);
}

// 0xff in every byte of w that is an E4M3 NaN (0x7f or 0xff).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

// One CTA: a chunk of positions of sequence b, KV head g, kTiles * 4 nodes.
template <int kTiles>
__global__ void __launch_bounds__(kWarps * 32, 2) tree_split_kernel(
    const __half *__restrict__ q, const int32_t *__restrict__ qo_indptr, int32_t total_q,
    int32_t max_nodes, const uint64_t *__restrict__ tree_mask, const __half *__restrict__ k_cache,
    const uint8_t *__restrict__ v_cache, const float *__restrict__ v_scale,
    const int32_t *__restrict__ block_table, int32_t maxp, const int32_t *__restrict__ seq_lens,
    int32_t max_len, int32_t hkv, int32_t num_pages, float sm_scale, int32_t chunk,
    int32_t max_chunks, float *__restrict__ part_o, float *__restrict__ part_lse,
    __half *__restrict__ out, float *__restrict__ lse_out, int32_t *dev_error) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Ring *rings = reinterpret_cast<Ring *>(smem_raw);
  int *page_ids = reinterpret_cast<int *>(smem_raw + kIdsOffset);
  const int c = blockIdx.x, g = blockIdx.y % hkv, block = blockIdx.y / hkv, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gr = lane >> 2, t = lane & 3;
  const int hq = hkv * kGroup;
  pdl_wait();
  pdl_launch_dependents();

  const int q0 = __ldg(qo_indptr + b);
  const int n = __ldg(qo_indptr + b + 1) - q0;
  const int L = __ldg(seq_lens + b);
  if (q0 < 0 || n < 0 || n > max_nodes || q0 > total_q - n || n > L || L > max_len) {
    if (threadIdx.x == 0 && c == 0 && blockIdx.y == 0) flag_error(dev_error, K16V8_DEVERR_SEQLEN);
    return;
  }
  const int node0 = block * 4 * kTiles;
  const int start = c * chunk;
  if (node0 >= n || start >= L) return;
  const int base = L - n;
  const int n_tok = min(chunk, L - start);
  const int n_pages = (n_tok + kPage - 1) / kPage;
  const int32_t *bt = block_table + static_cast<int64_t>(b) * maxp + start / kPage;
  for (int i = threadIdx.x; i < n_pages; i += blockDim.x) {
    int pid = __ldg(bt + i);
    if (pid < 0 || pid >= num_pages) {
      flag_error(dev_error, K16V8_DEVERR_PAGE);
      pid = -1;
    }
    page_ids[i] = pid;
  }
  Ring &ring = rings[warp];
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem_raw + kBarOffset) + warp * kTreeStages;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < kTreeStages; ++s) mbar_init(&bar[s], 1);
    fence_barrier_init();
  }
  __syncthreads();

  const int n_my = warp < n_pages ? (n_pages - warp + kWarps - 1) / kWarps : 0;
  const int64_t head_tile = static_cast<int64_t>(kPage) * kHeadDim;
  auto issue = [&](int k) {
    const int s = k % kTreeStages;
    const int pid = page_ids[warp + k * kWarps];
    if (pid < 0) {
      mbar_arrive(&bar[s]);  // nothing to load
      return;
    }
    const int64_t tile = (static_cast<int64_t>(pid) * hkv + g) * head_tile;
    mbar_arrive_expect_tx(&bar[s], kKPageBytes + kVPageBytes);
    bulk_g2s(ring.k[s], k_cache + tile, kKPageBytes, &bar[s]);
    bulk_g2s(ring.v[s], v_cache + tile, kVPageBytes, &bar[s]);
  };
  if (lane == 0)
    for (int k = 0; k < min(kTreeStages, n_my); ++k) issue(k);

  // query rows gr and gr + 8 of every tile: node = node0 + 4 tile + row / 4, head = row % 4
  uint32_t qa[kTiles][2][16];
  uint64_t mask[kTiles][2];
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int node = node0 + 4 * m + 2 * r + (gr >> 2);
      const bool live = node < n;
      mask[m][r] = live ? __ldg(tree_mask + q0 + node) : 0;
      const uint4 *src = reinterpret_cast<const uint4 *>(
          q + (static_cast<int64_t>(q0 + node) * hq + g * kGroup + (gr & 3)) * kHeadDim);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 raw = live ? __ldg(src + qk_chunk(i, t)) : make_uint4(0, 0, 0, 0);
        qa[m][r][4 * i] = raw.x;
        qa[m][r][4 * i + 1] = raw.y;
        qa[m][r][4 * i + 2] = raw.z;
        qa[m][r][4 * i + 3] = raw.w;
      }
    }

  const float qs = sm_scale * kLog2e;
  float mx[kTiles][2], sum[kTiles][2];
  float o[kTiles][16][4];
#pragma unroll
  for (int m = 0; m < kTiles; ++m) {
    mx[m][0] = mx[m][1] = -INFINITY;
    sum[m][0] = sum[m][1] = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[m][i][e] = 0.f;
  }

  bool ok = true;
  int k = 0;
  for (; k < n_my; ++k) {
    const int s = k % kTreeStages;
    ok = __all_sync(kFull, mbar_wait_bounded(&bar[s], (k / kTreeStages) & 1));
    if (!ok) break;
    const int page = warp + k * kWarps;
    const int pos0 = start + page * kPage;
    const bool in_tree = pos0 + kPage > base;  // the page reaches into the tree
    if (page_ids[page] >= 0) {
      // ---- scores ----
      float sc[kTiles][2][4];
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[m][h][e] = 0.f;
      const uint8_t *kp = ring.k[s];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 kw =
              *reinterpret_cast<const uint4 *>(kp + (gr + 8 * h) * 256 + qk_chunk(i, t) * 16);
#pragma unroll
          for (int m = 0; m < kTiles; ++m) {
            mma_16816(sc[m][h], qa[m][0][4 * i], qa[m][1][4 * i], qa[m][0][4 * i + 1],
                      qa[m][1][4 * i + 1], kw.x, kw.y);
            mma_16816(sc[m][h], qa[m][0][4 * i + 2], qa[m][1][4 * i + 2], qa[m][0][4 * i + 3],
                      qa[m][1][4 * i + 3], kw.z, kw.w);
          }
        }
      }
      // ---- softmax: element e of half h is row gr + 8 (e / 2), token 8h + 2t + (e & 1) ----
      uint32_t pa[kTiles][4];
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = sc[m][h][e] * qs;
            if (in_tree) {
              const int rel = pos0 + 8 * h + 2 * t + (e & 1) - base;
              const bool see = rel < 0 || (rel < n && ((mask[m][e >> 1] >> rel) & 1));
              if (!see) x = -INFINITY;
            }
            sc[m][h][e] = x;
            top[e >> 1] = fmaxf(top[e >> 1], x);
          }
        bool grow = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          top[r] = fmaxf(top[r], __shfl_xor_sync(kFull, top[r], 1));
          top[r] = fmaxf(top[r], __shfl_xor_sync(kFull, top[r], 2));
          grow |= top[r] > mx[m][r] + 8.f;
        }
        if (__any_sync(kFull, grow)) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float now = top[r] > mx[m][r] + 8.f ? top[r] : mx[m][r];
            const float alpha = now == -INFINITY ? 1.f : ex2(mx[m][r] - now);
            mx[m][r] = now;
            sum[m][r] *= alpha;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              o[m][i][2 * r] *= alpha;
              o[m][i][2 * r + 1] *= alpha;
            }
          }
        }
        float p[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // a row that has seen nothing yet keeps max -inf: its weights are 0
            const float ref = mx[m][e >> 1] == -INFINITY ? 0.f : mx[m][e >> 1];
            p[h][e] = ex2(sc[m][h][e] - ref);
          }
#pragma unroll
        for (int r = 0; r < 2; ++r)
          sum[m][r] += (p[0][2 * r] + p[0][2 * r + 1]) + (p[1][2 * r] + p[1][2 * r + 1]);
        pa[m][0] = pack_half2(p[0][0], p[0][1]);
        pa[m][1] = pack_half2(p[0][2], p[0][3]);
        pa[m][2] = pack_half2(p[1][0], p[1][1]);
        pa[m][3] = pack_half2(p[1][2], p[1][3]);
      }
      // ---- O += P V: dims 16 gr + i, tokens 2t, 2t + 1, 2t + 8, 2t + 9 ----
      const uint8_t *vp = ring.v[s] + 16 * gr;
      uint4 vr[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        vr[x] = *reinterpret_cast<const uint4 *>(vp + (2 * t + (x & 1) + 8 * (x >> 1)) * kHeadDim);
      uint32_t bad = 0;
      if (in_tree) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          bad |= nan_bytes(vr[x].x) | nan_bytes(vr[x].y) | nan_bytes(vr[x].z) | nan_bytes(vr[x].w);
      }
      const bool any_nan = in_tree && __any_sync(kFull, bad != 0);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t word[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          word[x] = w == 0 ? vr[x].x : (w == 1 ? vr[x].y : (w == 2 ? vr[x].z : vr[x].w));
        if (any_nan) {
          // rows that see a NaN code become NaN, the others do not
          uint32_t one[4];  // E4M3 1.0 where the code is NaN
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t nb = nan_bytes(word[x]);
            one[x] = nb & 0x38383838u;
            word[x] &= ~nb;
          }
          uint32_t lo[4], hi[4];
          pair_tokens(one[0], one[1], lo);
          pair_tokens(one[2], one[3], hi);
#pragma unroll
          for (int m = 0; m < kTiles; ++m) {
            uint32_t va[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {  // visibility in the layout of pa
              float f[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int rel = pos0 + 8 * (x >> 1) + 2 * t + e - base;
                f[e] = rel < 0 || (rel < n && ((mask[m][x & 1] >> rel) & 1)) ? 1.f : 0.f;
              }
              va[x] = pack_half2(f[0], f[1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float hit[4] = {0.f, 0.f, 0.f, 0.f};
              mma_16816(hit, va[0], va[1], va[2], va[3], lo[i], hi[i]);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (hit[e] > 0.f) o[m][4 * w + i][e] = NAN;
            }
          }
        }
        uint32_t lo[4], hi[4];
        pair_tokens(word[0], word[1], lo);
        pair_tokens(word[2], word[3], hi);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int m = 0; m < kTiles; ++m)
            mma_16816(o[m][4 * w + i], pa[m][0], pa[m][1], pa[m][2], pa[m][3], lo[i], hi[i]);
      }
    }
    __syncwarp();
    if (lane == 0 && k + kTreeStages < n_my) {
      fence_proxy_async();
      issue(k + kTreeStages);
    }
  }
  if (!ok) {
    if (lane == 0) {
      flag_error(dev_error, K16V8_DEVERR_TIMEOUT);
      for (int kk = k; kk < min(k + kTreeStages, n_my); ++kk)
        mbar_wait_bounded(&bar[kk % kTreeStages], (kk / kTreeStages) & 1);
    }
    __syncwarp();
  }
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sum[m][r] += __shfl_xor_sync(kFull, sum[m][r], 1);
      sum[m][r] += __shfl_xor_sync(kFull, sum[m][r], 2);
    }

  // ---- the warps' states, one row tile at a time, joined in shared memory ----
  float *wo = reinterpret_cast<float *>(smem_raw);           // [warp][16][128]
  float *wm = wo + kWarps * 16 * kHeadDim;                   // [warp][16]
  float *wl = wm + kWarps * 16;
  const float vs = __ldg(v_scale + g);
#pragma unroll
  for (int m = 0; m < kTiles; ++m) {
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float *row = wo + (warp * 16 + gr + 8 * r) * kHeadDim;
      // accumulator column e & 1 is lane column 2t + (e & 1): dim 16 (2t + (e & 1)) + i
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<float4 *>(row + 16 * (2 * t + e) + i) =
              make_float4(o[m][i][2 * r + e], o[m][i + 1][2 * r + e], o[m][i + 2][2 * r + e],
                          o[m][i + 3][2 * r + e]);
      if (t == 0) {
        wm[warp * 16 + gr + 8 * r] = mx[m][r];
        wl[warp * 16 + gr + 8 * r] = sum[m][r];
      }
    }
    __syncthreads();
    for (int row = warp; row < 16; row += kWarps) {
      const int node = node0 + 4 * m + (row >> 2);
      if (node >= n) continue;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w * 16 + row]);
      float total = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = wm[w * 16 + row];
        if (mw == -INFINITY) continue;
        const float f = ex2(mw - M);
        total += f * wl[w * 16 + row];
        const float4 x =
            *reinterpret_cast<const float4 *>(wo + (w * 16 + row) * kHeadDim + lane * 4);
        acc.x += f * x.x;
        acc.y += f * x.y;
        acc.z += f * x.z;
        acc.w += f * x.w;
      }
      float lse = -INFINITY;
      if (total > 0.f || total != total) {
        const float inv = vs / total;
        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        lse = (M + lg2(total)) * kLn2;
      }
      const int64_t r = static_cast<int64_t>(q0 + node) * hq + g * kGroup + (row & 3);
      if (max_chunks == 1) {
        *reinterpret_cast<uint2 *>(out + r * kHeadDim + lane * 4) =
            make_uint2(pack_half2(acc.x, acc.y), pack_half2(acc.z, acc.w));
        if (lane == 0 && lse_out) lse_out[r] = lse;
      } else {
        *reinterpret_cast<float4 *>(part_o + (r * max_chunks + c) * kHeadDim + lane * 4) = acc;
        if (lane == 0) part_lse[r * max_chunks + c] = lse;
      }
    }
  }
}

// One warp per row: the log-sum-exp join of a row's chunks.
__global__ void __launch_bounds__(128) tree_merge_kernel(
    const float *__restrict__ part_o, const float *__restrict__ part_lse,
    const int32_t *__restrict__ qo_indptr, int32_t total_q, int32_t max_nodes,
    const int32_t *__restrict__ seq_lens, int32_t max_len, int32_t hq, int32_t chunk,
    int32_t max_chunks, __half *__restrict__ out, float *__restrict__ lse_out) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int i = blockIdx.x * 4 + (threadIdx.x >> 5);  // node * hq + head
  pdl_wait();
  pdl_launch_dependents();
  const int q0 = __ldg(qo_indptr + b), n = __ldg(qo_indptr + b + 1) - q0;
  const int L = __ldg(seq_lens + b);
  if (q0 < 0 || n < 0 || n > max_nodes || q0 > total_q - n || n > L || L > max_len) return;
  if (i >= n * hq) return;
  const int64_t row = static_cast<int64_t>(q0) * hq + i;
  const int nc = (L + chunk - 1) / chunk;
  const float *pl = part_lse + row * max_chunks;
  const float *po = part_o + row * max_chunks * kHeadDim + lane * 4;
  float M = -INFINITY;
  for (int c = lane; c < nc; c += 32) M = fmaxf(M, __ldg(pl + c));
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, x));
  float S = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = 0; c < nc; ++c) {
    const float lc = __ldg(pl + c);
    const float4 x = __ldg(reinterpret_cast<const float4 *>(po + static_cast<int64_t>(c) * kHeadDim));
    if (lc == -INFINITY) continue;
    const float w = ex2((lc - M) * kLog2e);
    S += w;
    acc.x = fmaf(w, x.x, acc.x);
    acc.y = fmaf(w, x.y, acc.y);
    acc.z = fmaf(w, x.z, acc.z);
    acc.w = fmaf(w, x.w, acc.w);
  }
  float lse = -INFINITY;
  if (S > 0.f || S != S) {
    const float inv = 1.f / S;
    acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    lse = M + lg2(S) * kLn2;
  }
  *reinterpret_cast<uint2 *>(out + row * kHeadDim + lane * 4) =
      make_uint2(pack_half2(acc.x, acc.y), pack_half2(acc.z, acc.w));
  if (lane == 0 && lse_out) lse_out[row] = lse;
}

// ---- host side ------------------------------------------------------------

constexpr int kMinChunk = 64;  // one page per warp
constexpr int kMaxChunk = 8192;

struct Plan {
  int tiles, blocks, chunk, chunks;
  size_t lse_off, total;
};

// Row tiles per CTA, and the chunk that gives the SMs about four CTAs each
// (the fewest chunks that do, as every chunk costs a partial row).
static bool make_plan(int32_t total_q, int32_t batch, int32_t max_nodes, int32_t hkv,
                      int32_t max_len, Plan *p) {
  const int sms = k16v8_sm_count();
  if (sms <= 0) return false;
  p->tiles = max_nodes <= 4 ? 1 : 2;
  p->blocks = (max_nodes + 4 * p->tiles - 1) / (4 * p->tiles);
  const int64_t items = std::max<int64_t>(1, static_cast<int64_t>(batch) * hkv * p->blocks);
  const int64_t want = std::max<int64_t>(1, (4LL * sms + items - 1) / items);
  int64_t chunk = (max_len + want - 1) / want;
  chunk = (chunk + kMinChunk - 1) / kMinChunk * kMinChunk;
  p->chunk = static_cast<int>(std::min<int64_t>(kMaxChunk, std::max<int64_t>(kMinChunk, chunk)));
  p->chunks = std::max(1, (max_len + p->chunk - 1) / p->chunk);
  p->lse_off = p->total = 0;
  if (p->chunks > 1) {
    const size_t rows = static_cast<size_t>(total_q) * hkv * kGroup * p->chunks;
    p->lse_off = (rows * kHeadDim * 4 + 255) / 256 * 256;
    p->total = p->lse_off + (rows * 4 + 255) / 256 * 256;
  }
  return true;
}

template <int kTiles>
static int32_t set_smem(size_t bytes) {
  static size_t configured[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return K16V8_ERR_CUDA;
  if (dev < 64 && configured[dev] >= bytes) return K16V8_OK;
  if (cudaFuncSetAttribute(tree_split_kernel<kTiles>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes)) != cudaSuccess)
    return K16V8_ERR_CUDA;
  if (dev < 64) configured[dev] = bytes;
  return K16V8_OK;
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
  if (batch > 65535 || hkv > 4095) return K16V8_ERR_INVALID_ARG;
  return K16V8_OK;
}

extern "C" size_t k16v8_tree_workspace_size(int32_t total_q, int32_t batch, int32_t max_nodes,
                                            int32_t num_qo_heads, int32_t num_kv_heads,
                                            int32_t head_dim, int32_t max_seq_len) {
  tree::Plan p;
  if (check_tree_shape(total_q, batch, max_nodes, num_qo_heads, num_kv_heads, head_dim,
                       max_seq_len) != K16V8_OK ||
      !tree::make_plan(total_q, batch, max_nodes, num_kv_heads, max_seq_len, &p))
    return 0;
  return p.total;
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
  if (static_cast<int64_t>(max_pages_per_seq) * kPage < max_seq_len) return K16V8_ERR_INVALID_ARG;
  if (batch == 0 || total_q == 0 || max_nodes == 0 || max_seq_len == 0) return K16V8_OK;
  if (!q || !qo_indptr || !tree_mask || !k_cache || !v_cache || !v_scale || !block_table ||
      !seq_lens || !out)
    return K16V8_ERR_INVALID_ARG;
  if (!k16v8_aligned(q, 16) || !k16v8_aligned(k_cache, 16) || !k16v8_aligned(v_cache, 16) ||
      !k16v8_aligned(out, 16) || !k16v8_aligned(tree_mask, 8) || !k16v8_aligned(qo_indptr, 4) ||
      !k16v8_aligned(seq_lens, 4) || !k16v8_aligned(block_table, 4) ||
      !k16v8_aligned(v_scale, 4) || (lse && !k16v8_aligned(lse, 4)))
    return K16V8_ERR_INVALID_ARG;
  tree::Plan p;
  if (!tree::make_plan(total_q, batch, max_nodes, num_kv_heads, max_seq_len, &p))
    return K16V8_ERR_CUDA;
  if (p.total) {
    if (!workspace || !k16v8_aligned(workspace, 256)) return K16V8_ERR_INVALID_ARG;
    if (workspace_bytes < p.total) return K16V8_ERR_WORKSPACE_TOO_SMALL;
  }
  float *po = static_cast<float *>(workspace);
  float *pl = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + p.lse_off);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t smem = tree::kIdsOffset + p.chunk / kPage * sizeof(int);
  st = p.tiles == 1 ? tree::set_smem<1>(smem) : tree::set_smem<2>(smem);
  if (st != K16V8_OK) return st;
  const dim3 grid(p.chunks, num_kv_heads * p.blocks, batch);
  st = k16v8_launch_pdl(
      p.tiles == 1 ? tree::tree_split_kernel<1> : tree::tree_split_kernel<2>, grid,
      dim3(kWarps * 32), smem, s, static_cast<const __half *>(q), qo_indptr, total_q, max_nodes,
      tree_mask, static_cast<const __half *>(k_cache), v_cache, v_scale, block_table,
      max_pages_per_seq, seq_lens, max_seq_len, num_kv_heads, num_pages, sm_scale, p.chunk,
      p.chunks, po, pl, static_cast<__half *>(out), lse, dev_error);
  if (st != K16V8_OK || p.chunks == 1) return st;
  const dim3 mgrid((max_nodes * num_qo_heads + 3) / 4, batch);
  return k16v8_launch_pdl(tree::tree_merge_kernel, mgrid, dim3(128), 0, s, po, pl, qo_indptr,
                          total_q, max_nodes, seq_lens, max_seq_len, num_qo_heads, p.chunk,
                          p.chunks, static_cast<__half *>(out), lse);
}

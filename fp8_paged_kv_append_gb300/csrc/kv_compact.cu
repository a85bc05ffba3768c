// kv_compact: the cache rows of an accepted path move to the front of their
// tree's slots, in every layer at once.
//
// "Phi-4: quality transfer and interrupted throughput studies": the intro
// fixes the cache format and the 40-layer geometry; a verified tree of
// drafted tokens leaves its accepted rows scattered over the last positions
// of each sequence, and the next step needs them in order.
//
// For sequence b with n nodes at positions base .. base + n - 1 and an
// accepted path of m nodes, row base + path[j] goes to base + j.  A path
// increases strictly, so path[j] >= j: rows only move down, and a warp that
// moves them in order of j, reading a group of rows whole before it writes
// them, never overwrites a row that is still to be read (a later row j' sits
// at path[j'] >= j' > every j written so far).
//
// HBM-bound copy of scattered rows (256 and 128 bytes), and on small calls a
// chain of four memory round trips (lengths, path, block table, rows).  One
// warp per (layer, sequence, KV head); a row is 24 pieces of 16 bytes (16 of
// K, 8 of V).  The lanes resolve the addresses of a group of rows in parallel
// and hand them round by shuffles; a group of 4 rows is 3 loads in flight per
// lane.  GB300, 40 layers x 10 heads, 64 sequences with 8 rows each to move:
// 28.7 us, 5.5 TB/s read and written (0.81 of the copy rate); groups of 8 rows
// 42.6 us (more registers, fewer warps), CTAs of 1 / 2 / 8 warps 29.6 / 28.6 /
// 29.5 us, a lane resolving its own pieces' addresses 37.2 us.  One sequence
// with 3 rows to move: 2.2 us for all 40 layers.
#include "k16v8_device.cuh"

namespace k16v8 {
namespace compact {

constexpr int kWarpsPerCta = 4;
constexpr int kPieces = kHeadDim * 3 / 16;  // 24 pieces of 16 bytes per row
constexpr int kGroupRows = 4;
constexpr int kPerLane = kPieces * kGroupRows / 32;
constexpr unsigned kFull = 0xffffffffu;

// The base position and node count of sequence b, or false (nothing to do).
__device__ __forceinline__ bool sequence(const int32_t *qo_indptr, const int32_t *seq_lens, int b,
                                         int32_t maxp, int32_t max_path, int &base, int &n) {
  const int q0 = __ldg(qo_indptr + b), L = __ldg(seq_lens + b);
  n = __ldg(qo_indptr + b + 1) - q0;
  base = L - n;
  return q0 >= 0 && n >= 0 && n <= L && n <= max_path && L <= maxp * kPage;
}

__global__ void __launch_bounds__(kWarpsPerCta * 32) kv_compact_kernel(
    const uint64_t *__restrict__ k_ptrs, const uint64_t *__restrict__ v_ptrs, int32_t layers,
    const int32_t *__restrict__ block_table, int32_t maxp, const int32_t *__restrict__ seq_lens,
    const int32_t *__restrict__ qo_indptr, const int32_t *__restrict__ path, int32_t max_path,
    const int32_t *__restrict__ path_len, int32_t batch, int32_t hkv, int32_t num_pages,
    int32_t *__restrict__ new_lens, int32_t *dev_error) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t item = blockIdx.x * static_cast<int64_t>(kWarpsPerCta) + (threadIdx.x >> 5);
  const int64_t per_layer = static_cast<int64_t>(batch) * hkv;
  const int layer = static_cast<int>(item / per_layer);
  if (layer >= layers) return;
  const int in_layer = static_cast<int>(item - layer * per_layer);  // below 2^31 (checked)
  const int b = in_layer / hkv, g = in_layer - b * hkv;
  const bool report = layer == 0 && g == 0;  // one warp per sequence
  int base, n;
  const int m = __ldg(path_len + b);
  // the path, two nodes per lane: strictly increasing nodes of this tree
  const int32_t *pb = path + static_cast<int64_t>(b) * max_path;
  const int p0 = lane < max_path ? __ldg(pb + lane) : 0;
  const int p1 = lane + 32 < max_path ? __ldg(pb + lane + 32) : 0;
  if (!sequence(qo_indptr, seq_lens, b, maxp, max_path, base, n)) {
    if (report && lane == 0) {
      flag_error(dev_error, K16V8_DEVERR_SEQLEN);
      if (new_lens) new_lens[b] = __ldg(seq_lens + b);
    }
    return;
  }
  const int before0 = __shfl_up_sync(kFull, p0, 1), wrap = __shfl_sync(kFull, p0, 31);
  const int before1 = __shfl_up_sync(kFull, p1, 1);
  bool good = m >= 0 && m <= n;
  if (lane < m) good &= p0 > (lane > 0 ? before0 : -1) && p0 < n;
  if (lane + 32 < m) good &= p1 > (lane > 0 ? before1 : wrap) && p1 < n;
  good = __all_sync(kFull, good);
  if (report && lane == 0) {
    if (!good) flag_error(dev_error, K16V8_DEVERR_TREE);
    if (new_lens) new_lens[b] = good ? base + m : __ldg(seq_lens + b);
  }
  if (!good) return;
  // rows at the front of the path are in place; from the first that is not on,
  // none is
  const unsigned away0 = __ballot_sync(kFull, lane < m && p0 != lane);
  const unsigned away1 = __ballot_sync(kFull, lane + 32 < m && p1 != lane + 32);
  const int first = away0 ? __ffs(away0) - 1 : (away1 ? __ffs(away1) + 31 : m);
  if (first >= m) return;
  uint8_t *kc = reinterpret_cast<uint8_t *>(__ldg(k_ptrs + layer));
  uint8_t *vc = reinterpret_cast<uint8_t *>(__ldg(v_ptrs + layer));
  const uint64_t low = reinterpret_cast<uint64_t>(kc) | reinterpret_cast<uint64_t>(vc);
  if (!kc || !vc || (low & 15)) {
    if (lane == 0) flag_error(dev_error, K16V8_DEVERR_PAGE);
    return;
  }
  const int32_t *bt = block_table + static_cast<int64_t>(b) * maxp;
  for (int j0 = first; j0 < m; j0 += kGroupRows) {
    // lane 2r + d: the offset of row j0 + r's source (d = 0) or destination
    // (d = 1) in a cache of one-byte elements, -1 for none
    const int r = lane >> 1, j = j0 + r;
    const int node = __shfl_sync(kFull, p0, j & 31), node1 = __shfl_sync(kFull, p1, j & 31);
    int64_t at = -1;
    if (r < kGroupRows && j < m) {
      const int pos = base + (lane & 1 ? j : (j < 32 ? node : node1));
      const int page = __ldg(bt + pos / kPage);
      if (page < 0 || page >= num_pages)
        flag_error(dev_error, K16V8_DEVERR_PAGE);
      else
        at = ((static_cast<int64_t>(page) * hkv + g) * kPage + pos % kPage) * kHeadDim;
    }
    uint4 piece[kPerLane];
    uint4 *to[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int x = i * 32 + lane, row = x / kPieces, c = x - row * kPieces;
      const int64_t src = __shfl_sync(kFull, at, 2 * row), dst = __shfl_sync(kFull, at, 2 * row + 1);
      to[i] = nullptr;
      if (src < 0 || dst < 0) continue;
      uint8_t *cache = c < 16 ? kc : vc;
      const int shift = c < 16 ? 1 : 0;  // bytes per element: 2 or 1
      const int off = 16 * (c < 16 ? c : c - 16);
      piece[i] = *reinterpret_cast<const uint4 *>(cache + (src << shift) + off);
      to[i] = reinterpret_cast<uint4 *>(cache + (dst << shift) + off);
    }
    __syncwarp();  // a group is read whole before any of it is written
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (to[i]) *to[i] = piece[i];
    __syncwarp();
  }
}

}  // namespace compact
}  // namespace k16v8

using namespace k16v8;

extern "C" int32_t k16v8_kv_compact(const uint64_t *k_caches, const uint64_t *v_caches,
                                    int32_t num_layers, const int32_t *block_table,
                                    int32_t max_pages_per_seq, const int32_t *seq_lens,
                                    const int32_t *qo_indptr, const int32_t *path,
                                    int32_t max_nodes, const int32_t *path_len, int32_t batch,
                                    int32_t num_kv_heads, int32_t head_dim, int32_t num_pages,
                                    int32_t *new_seq_lens, int32_t *dev_error, void *stream) {
  if (num_layers < 0 || batch < 0 || max_nodes < 0 || max_pages_per_seq < 0 ||
      num_kv_heads <= 0 || num_pages <= 0)
    return K16V8_ERR_INVALID_ARG;
  if (max_pages_per_seq > 0x7fffffff / kPage) return K16V8_ERR_INVALID_ARG;
  if (head_dim != kHeadDim || max_nodes > K16V8_MAX_TREE_NODES)
    return K16V8_ERR_UNSUPPORTED_SHAPE;
  if (batch == 0 || num_layers == 0) return K16V8_OK;
  if (!k_caches || !v_caches || !block_table || !seq_lens || !qo_indptr || !path_len ||
      (max_nodes > 0 && !path))
    return K16V8_ERR_INVALID_ARG;
  if (!k16v8_aligned(k_caches, 8) || !k16v8_aligned(v_caches, 8) ||
      !k16v8_aligned(block_table, 4) || !k16v8_aligned(seq_lens, 4) ||
      !k16v8_aligned(qo_indptr, 4) || !k16v8_aligned(path, 4) || !k16v8_aligned(path_len, 4) ||
      (new_seq_lens && !k16v8_aligned(new_seq_lens, 4)))
    return K16V8_ERR_INVALID_ARG;
  // other warps still read the inputs when the new lengths are written
  auto over = [&](const int32_t *in, int64_t n) {
    return new_seq_lens && n > 0 && new_seq_lens < in + n && in < new_seq_lens + batch;
  };
  if (over(seq_lens, batch) || over(path_len, batch) || over(qo_indptr, batch + 1ll) ||
      over(path, static_cast<int64_t>(batch) * max_nodes) ||
      over(block_table, static_cast<int64_t>(batch) * max_pages_per_seq))
    return K16V8_ERR_INVALID_ARG;
  if (static_cast<int64_t>(batch) * num_kv_heads > 0x7fffffffLL) return K16V8_ERR_INVALID_ARG;
  const int64_t items = static_cast<int64_t>(num_layers) * batch * num_kv_heads;
  const int64_t blocks = (items + compact::kWarpsPerCta - 1) / compact::kWarpsPerCta;
  if (blocks > 0x7fffffffLL) return K16V8_ERR_INVALID_ARG;
  return k16v8_launch_pdl(compact::kv_compact_kernel, dim3(static_cast<unsigned>(blocks)),
                          dim3(compact::kWarpsPerCta * 32), 0, static_cast<cudaStream_t>(stream),
                          k_caches, v_caches, num_layers, block_table, max_pages_per_seq, seq_lens,
                          qo_indptr, path, max_nodes, path_len, batch, num_kv_heads, num_pages,
                          new_seq_lens, dev_error);
}

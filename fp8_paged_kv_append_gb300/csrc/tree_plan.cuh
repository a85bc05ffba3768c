// How tree attention cuts its work: shared by the split kernels and the
// merge.
//
// A segment is one (sequence, KV head) pair; its KV range is nt tiles of a
// fixed number of positions.  All tiles form one flat list, sequence-major,
// then head, then tile; a tile costs `weight` units (2 for trees that need
// two row tiles of the tensor cores, else 1).  With a total of T units and G
// CTAs, CTA i owns the tiles that start in [i W, (i + 1) W), W = ceil(T / G):
// equal ranges whatever the mix of lengths, at most two cut segments per CTA
// (the one it begins in and the one it ends in).  A whole segment's rows go
// straight to the output; a cut one's go to the workspace, slot 2i + 1 of the
// CTA the segment begins in and slot 2i of every later one, and cut[i] tells
// the merge which segment that is.
#pragma once

#include "k16v8_device.cuh"

namespace k16v8 {
namespace tree {

constexpr int kMaxBatch = 8192;  // the scan's prefix lives in shared memory
constexpr int kMaxLen = 1 << 30;  // positions round up to tiles in 32 bits

struct Args {  // (queries and keys come through their tensor maps)
  const int32_t *qo_indptr;
  int32_t total_q, max_nodes;
  const uint64_t *tree_mask;
  const uint8_t *v_cache;
  const float *v_scale;
  const int32_t *block_table;
  int32_t maxp;
  const int32_t *seq_lens;
  int32_t max_len, batch, hkv, num_pages;
  float sm_scale;
  int4 *cut;          // [G] segment that begins in the CTA and is cut: b, g, last CTA
  float *part_lse;    // [2 G][max_rows]
  float4 *part_o;     // [2 G][32 chunks of 4 dims][max_rows], normalised rows
  int32_t max_rows;   // rows of a segment, at most: node * 4 + head
  __half *out;
  float *lse;
  int32_t *dev_error;
};

// Rows and length of sequence b; false where there is nothing to do.
__device__ __forceinline__ bool sequence(const Args &a, int b, int &q0, int &n, int &L,
                                         bool &bad) {
  q0 = __ldg(a.qo_indptr + b);
  n = __ldg(a.qo_indptr + b + 1) - q0;
  L = __ldg(a.seq_lens + b);
  bad = q0 < 0 || n < 0 || n > a.max_nodes || q0 > a.total_q - n || n > L || L > a.max_len;
  return !bad && n > 0;
}

// x / y of numbers >= 0, in 32 bits where they fit (64-bit division is a
// hundred instructions).
__device__ __forceinline__ int64_t divide(int64_t x, int64_t y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// The shape of a split kernel's tiles.
struct Shape {
  int positions;   // per KV tile
  int wide_nodes;  // trees beyond cost two units per tile
  __device__ __forceinline__ int tiles(int L) const { return (L + positions - 1) / positions; }
  __device__ __forceinline__ int weight(int n) const { return n > wide_nodes ? 2 : 1; }
};

struct Range {
  int64_t lo, hi, width;  // units
  int64_t start;          // of sequence b's first segment
  int b, cta;
};

// The CTA's range of units, at least `least` (no less than the largest
// weight, so that a CTA between two cuts has a tile); every thread of the block
// calls it.  `prefix`: scratch of batch + 1 entries, `aux`: of 33.
__device__ __forceinline__ Range plan_range(const Args &a, const Shape &shape, int least,
                                            int64_t *prefix, int64_t *aux) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  int64_t carry = 0;
  for (int b0 = 0; b0 < a.batch; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int64_t cost = 0;
    if (b < a.batch) {
      int q0, n, L;
      bool bad;
      if (sequence(a, b, q0, n, L, bad))
        cost = static_cast<int64_t>(shape.tiles(L)) * shape.weight(n) * a.hkv;
      if (bad && blockIdx.x == 0) flag_error(a.dev_error, K16V8_DEVERR_SEQLEN);
    }
    int64_t x = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) aux[warp] = x;
    __syncthreads();
    int64_t before = carry, all = 0;
    const int busy = min(warps, (a.batch - b0 + 31) >> 5);  // warps with sequences
    for (int w = 0; w < busy; ++w) {
      const int64_t v = aux[w];
      if (w < warp) before += v;
      all += v;
    }
    if (b < a.batch) prefix[b] = before + x - cost;
    carry += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) prefix[a.batch] = carry;
  __syncthreads();
  Range r;
  r.width = divide(carry + gridDim.x - 1, gridDim.x);
  if (r.width < least) r.width = least;
  r.cta = blockIdx.x;
  r.lo = r.width * r.cta;
  r.hi = min(r.lo + r.width, carry);
  int b = 0, e = a.batch;  // largest b with prefix[b] <= lo
  while (e - b > 1) {
    const int mid = (b + e) >> 1;
    if (prefix[mid] <= r.lo) b = mid; else e = mid;
  }
  r.b = b;
  r.start = r.lo < r.hi ? prefix[b] : 0;
  return r;
}

// The part [t0, t1) of a segment's tiles that a CTA owns.
struct Piece {
  int32_t b, g, q0, n, L, t0, t1;
  int32_t whole;  // all of the segment
  int32_t slot;   // workspace slot of a cut piece
  int32_t tiles;  // t1 - t0, 0: the end of the CTA's pieces

  __device__ __forceinline__ int base() const { return L - n; }
  __device__ __forceinline__ uint64_t node_bits() const {
    return n >= 64 ? ~0ull : (1ull << n) - 1;
  }
};

// Walks the pieces of a range in order.  Of a cut segment that begins in the
// CTA it tells the merge.
struct Walker {
  Piece p;
  int nt, shift;  // the segment's tiles and the weight's logarithm
  int64_t start;  // of the segment, in units

  __device__ __forceinline__ bool load(const Args &a, const Shape &shape) {
    bool bad;
    if (!sequence(a, p.b, p.q0, p.n, p.L, bad)) return false;
    nt = shape.tiles(p.L);
    shift = shape.weight(p.n) - 1;
    return true;
  }
  __device__ __forceinline__ void init(const Args &a, const Shape &shape, const Range &r) {
    p.b = r.b;
    load(a, shape);  // it holds the range's first unit, so it has tiles
    const int64_t seg = static_cast<int64_t>(nt) << shift;
    p.g = static_cast<int>(divide(r.lo - r.start, seg));
    start = r.start + p.g * seg;
    p.t0 = static_cast<int>((r.lo - start + (1 << shift) - 1) >> shift);
  }
  // The next piece, false at the end of the range.
  __device__ __forceinline__ bool next(const Args &a, const Shape &shape, const Range &r,
                                       Piece &out) {
    bool found = false;
    while (!found && p.b < a.batch) {
      if (p.t0 < nt) {  // else the range begins inside the segment's last tile
        if (start + (static_cast<int64_t>(p.t0) << shift) >= r.hi) {
          p.b = a.batch;
          break;
        }
        p.t1 = static_cast<int>(
            min(static_cast<int64_t>(nt), (r.hi - start + (1 << shift) - 1) >> shift));
        p.tiles = p.t1 - p.t0;
        p.whole = p.t0 == 0 && p.t1 == nt;
        p.slot = 2 * r.cta + (start >= r.lo ? 1 : 0);
        if (start >= r.lo && p.t1 < nt)
          a.cut[r.cta] = make_int4(
              p.b, p.g,
              static_cast<int>(divide(start + (static_cast<int64_t>(nt - 1) << shift), r.width)),
              0);
        out = p;
        found = true;
      }
      start += static_cast<int64_t>(nt) << shift;
      p.t0 = 0;
      if (++p.g == a.hkv) {
        p.g = 0;
        do {
          ++p.b;
        } while (p.b < a.batch && !load(a, shape));
      }
    }
    return found;
  }
};

// 0xff in every byte of w that is an E4M3 NaN (0x7f or 0xff).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

}  // namespace tree
}  // namespace k16v8

// How attention of several query rows over the K8/V8 cache cuts its work: shared
// by the split kernel and the merge.
//
// A segment is one KV head with up to 64 query tokens of a sequence (a token
// group: two row tiles of 32 tokens x 4 heads); its KV range is the tiles of 128
// positions that any of its tokens sees.  All tiles form one flat list --
// sequence, head, token group, tile -- and a tile costs 2 units where the group
// has more than 32 tokens, else 1.  With a total of T units and G CTAs, CTA i
// owns the tiles that start in [i W, (i + 1) W), W = ceil(T / G): equal ranges
// whatever the mix of lengths, at most two cut segments per CTA (the one it
// begins in and the one it ends in).  A whole segment's rows go straight to the
// output; a cut one's go to the workspace, slot 2i + 1 of the CTA the segment
// begins in and slot 2i of every later one, and cut[i] tells the merge.
//
// Under a causal mask the groups of a sequence see more and more tiles, so what
// comes before a group has to be summed.  With base positions before the first
// new token, full group p sees floor((base + 64 (p + 1) + 127) / 128) tiles;
// writing base + 191 = 64 a + r this is floor((a + p) / 2), and sum_{i < k}
// floor(i / 2) = floor((k - 1)^2 / 4).
#pragma once

#include "k8v8_device.cuh"

namespace k16v8 {
namespace attn8 {

constexpr int kMaxBatch = 8192;  // the scan's prefix lives in shared memory
constexpr int kMaxLen = 1 << 30;
constexpr int kKv = 128;         // positions per tile
constexpr int kTileTokens = 32;  // query tokens per row tile
constexpr int kGroupTokens = 2 * kTileTokens;

struct Args {  // (queries come through their tensor map)
  const int32_t *qo_indptr;
  int32_t total_q, max_q, causal;
  const uint8_t *v_cache;  // (codes come through their tensor maps; NaN ones are looked up)
  const float *kv_scale;
  const int32_t *block_table;
  int32_t maxp;
  const int32_t *seq_lens;
  int32_t max_len, batch, hkv, num_pages;
  float sm_scale;
  int4 *cut;        // [G] segment that begins in the CTA and is cut: row, tokens, head, last CTA
  float *part_lse;  // [2 G][max_rows]
  float4 *part_o;   // [2 G][32 chunks of 4 dims][max_rows], normalised rows
  int32_t max_rows; // of a segment: token * 4 + head
  __half *out;
  float *lse;
  int32_t *dev_error;
};

// x / y of numbers >= 0, in 32 bits where they fit (64-bit division is a hundred
// instructions).
__device__ __forceinline__ int64_t divide(int64_t x, int64_t y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// A sequence: its n query rows from q0 on, L cached positions.
struct Sequence {
  int q0, n, L;

  // False where there is nothing to do; bad: out of range.
  __device__ __forceinline__ bool load(const Args &a, int b, bool &bad) {
    q0 = __ldg(a.qo_indptr + b);
    const int64_t rows = static_cast<int64_t>(__ldg(a.qo_indptr + b + 1)) - q0;
    n = static_cast<int>(rows);
    L = __ldg(a.seq_lens + b);
    bad = q0 < 0 || rows < 0 || rows > a.max_q || rows > a.total_q - q0 || L < 0 || L > a.max_len ||
          (a.causal && n > L);
    return !bad && n > 0;
  }
  __device__ __forceinline__ int groups() const { return (n + kGroupTokens - 1) / kGroupTokens; }
  __device__ __forceinline__ int tokens(int p) const { return min(kGroupTokens, n - p * kGroupTokens); }
  __device__ __forceinline__ int seen(bool causal, int p) const {  // positions, of the group's last token
    return causal ? L - n + p * kGroupTokens + tokens(p) : L;
  }
  __device__ __forceinline__ int tiles(bool causal, int p) const {
    return max(1, (seen(causal, p) + kKv - 1) / kKv);  // (one where there is nothing to see)
  }
  __device__ __forceinline__ int shift(int p) const { return tokens(p) > kTileTokens; }
  // units of the groups before group p, all of them full
  __device__ __forceinline__ int64_t before(bool causal, int p) const {
    if (!causal) return 2ll * p * tiles(false, 0);
    const int64_t a = (L - n + 191) >> 6;
    auto sum = [](int64_t k) { return ((k - 1) * (k - 1)) >> 2; };
    return 2 * (sum(a + p) - sum(a));
  }
  __device__ __forceinline__ int64_t units(bool causal) const {  // of a head
    const int p = groups() - 1;
    return before(causal, p) + (static_cast<int64_t>(tiles(causal, p)) << shift(p));
  }
};

struct Range {
  int64_t lo, hi, width;  // units
  int64_t start;          // of sequence b
  int b, cta;
};

// The CTA's range of units; every thread of the block calls it.  `prefix`:
// scratch of batch + 1 entries, `aux`: of 33.
__device__ __forceinline__ Range plan_range(const Args &a, int64_t *prefix, int64_t *aux) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  int64_t carry = 0;
  for (int b0 = 0; b0 < a.batch; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int64_t cost = 0;
    if (b < a.batch) {
      Sequence s;
      bool bad;
      if (s.load(a, b, bad)) cost = s.units(a.causal) * a.hkv;
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
  // no less than the largest weight: a CTA between two cuts has a tile
  if (r.width < 2) r.width = 2;
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
  int32_t b, g;
  int32_t q0, n;   // the group's first row, its tokens
  int32_t L, base; // positions seen; those below base are seen by every token
  int32_t t0, h1;  // the first tile; the end, in half tiles of 64 positions
  int32_t whole;   // all of the segment
  int32_t slot;    // workspace slot of a cut piece
  int32_t tiles;   // t1 - t0, 0: the end of the CTA's pieces
  int32_t turn;    // of one row tile: the slot of the first KV tile, such that the
                   // slots take turns over all such tiles of the CTA

  // Halves of the piece's tile t (from 0 on) that hold positions: one where the last
  // tile ends in its first half.
  __device__ __forceinline__ int halves(int t) const { return 2 * (t0 + t) + 1 < h1 ? 2 : 1; }
};

// Walks the pieces of a range in order.  Of a cut segment that begins in the CTA
// it tells the merge.
struct Walker {
  Sequence s;
  Piece p;
  int group, nt, shift, turn;
  int64_t start;  // of the segment, in units

  __device__ __forceinline__ void set_group(const Args &a, int k) {
    group = k;
    nt = s.tiles(a.causal, k);
    shift = s.shift(k);
    p.q0 = s.q0 + k * kGroupTokens;
    p.n = s.tokens(k);
    p.L = s.seen(a.causal, k);
    p.base = a.causal ? p.L - p.n : p.L;
  }
  __device__ __forceinline__ void init(const Args &a, const Range &r) {
    bool bad;
    turn = 0;
    p.b = r.b;
    s.load(a, r.b, bad);  // it holds the range's first unit, so it has tiles
    const int64_t head = s.units(a.causal);
    p.g = static_cast<int>(divide(r.lo - r.start, head));
    start = r.start + p.g * head;
    int lo = 0, hi = s.groups();  // the last group that starts at or before the range
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start + s.before(a.causal, mid) <= r.lo) lo = mid; else hi = mid;
    }
    set_group(a, lo);
    start += s.before(a.causal, lo);
    p.t0 = static_cast<int>((r.lo - start + (1 << shift) - 1) >> shift);
  }
  // The next piece, false at the end of the range.
  __device__ __forceinline__ bool next(const Args &a, const Range &r, Piece &out) {
    bool found = false;
    while (!found && p.b < a.batch) {
      if (p.t0 < nt) {  // else the range begins inside the segment's last tile
        if (start + (static_cast<int64_t>(p.t0) << shift) >= r.hi) {
          p.b = a.batch;
          break;
        }
        const int t1 = static_cast<int>(
            min(static_cast<int64_t>(nt), (r.hi - start + (1 << shift) - 1) >> shift));
        p.tiles = t1 - p.t0;
        p.h1 = max(2 * t1 - 1, min(2 * t1, (p.L + kKv / 2 - 1) / (kKv / 2)));
        p.whole = p.t0 == 0 && t1 == nt;
        p.slot = 2 * r.cta + (start >= r.lo ? 1 : 0);
        if (start >= r.lo && t1 < nt)
          a.cut[r.cta] = make_int4(
              p.q0, p.n, p.g,
              static_cast<int>(divide(start + (static_cast<int64_t>(nt - 1) << shift), r.width)));
        p.turn = turn;
        if (shift == 0) turn ^= p.tiles & 1;
        out = p;
        found = true;
      }
      start += static_cast<int64_t>(nt) << shift;
      p.t0 = 0;
      if (group + 1 < s.groups()) {
        set_group(a, group + 1);
      } else {
        bool more = ++p.g < a.hkv, bad;
        if (!more) {
          p.g = 0;
          do {
            ++p.b;
            more = p.b < a.batch && s.load(a, p.b, bad);
          } while (!more && p.b < a.batch);
        }
        if (more) set_group(a, 0);
      }
    }
    return found;
  }
};

// 0xff in every byte of w that is an E4M3 NaN (0x7f or 0xff).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

}  // namespace attn8
}  // namespace k16v8

// Device code shared by the kernels that turn rows by their positions: units of
// 16 elements of a row, their widening and rounding, the angle of a pair, and
// which axis of a several-axis position turns it.
#pragma once

#include <cuda_bf16.h>

#include "k16v8_device.cuh"

namespace k16v8 {
namespace rope {

constexpr int kUnitsPerRow = kHeadDim / 16;
constexpr int32_t kMaxPosition = 1 << 24;  // positions below are exact in fp32
// 1 / 2pi as a sum of two fp32 numbers
constexpr float kInv2PiHi = 0x1.45f306p-3f;
constexpr float kInv2PiLo = 0x1.b9391p-28f;

template <typename T>
struct Raw {  // 16 elements
  uint4 w[sizeof(T)];
};

// Elements [e, e + 8) of a row.
template <typename T>
__device__ __forceinline__ void load8(const T *p, uint4 *w) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
    w[i] = reinterpret_cast<const uint4 *>(p)[i];
}

__device__ __forceinline__ void widen8(const uint4 *w, float (&x)[8], const __half *) {
  const __half2 *h = reinterpret_cast<const __half2 *>(w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(h[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void widen8(const uint4 *w, float (&x)[8], const __nv_bfloat16 *) {
  const uint32_t u[4] = {w->x, w->y, w->z, w->w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen8(const uint4 *w, float (&x)[8], const float *) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(w[i].x);
    x[4 * i + 1] = __uint_as_float(w[i].y);
    x[4 * i + 2] = __uint_as_float(w[i].z);
    x[4 * i + 3] = __uint_as_float(w[i].w);
  }
}

__device__ __forceinline__ uint4 narrow8(const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// cos and sin of position * freq, times factor.
__device__ __forceinline__ float2 turn(int32_t position, float freq, float factor) {
  const float p = static_cast<float>(position);
  const float rh = __fmul_rn(freq, kInv2PiHi);  // products that are not to be contracted
  const float rl = fmaf(freq, kInv2PiLo, fmaf(freq, kInv2PiHi, -rh));
  const float th = __fmul_rn(p, rh);
  const float tl = fmaf(p, rl, fmaf(p, rh, -th));
  const float frac = (th - rintf(th)) + tl;
  float s, c;
  sincospif(2.f * frac, &s, &c);
  return make_float2(c * factor, s * factor);
}

// The axis of every pair, two bits each, by value: pairs 0-31 in lo.
struct PairAxes {
  uint64_t lo, hi;
  int32_t count;  // axes of a position
  __host__ __device__ __forceinline__ int operator[](int pair) const {
    return static_cast<int>((pair & 32 ? hi : lo) >> (2 * (pair & 31))) & 3;
  }
};

// From the host array of the C ABI; false where an entry is no axis.
static inline bool pack_axes(const int8_t *pair_axis, int32_t pairs, int32_t count, PairAxes *out) {
  *out = PairAxes{0, 0, count};
  for (int32_t i = 0; i < pairs; ++i) {
    if (pair_axis[i] < 0 || pair_axis[i] >= count) return false;
    (i & 32 ? out->hi : out->lo) |= static_cast<uint64_t>(pair_axis[i]) << (2 * (i & 31));
  }
  return true;
}

// Token t's positions [count][num_tokens] are all in range.
__device__ __forceinline__ bool positions_ok(const int32_t *positions, int64_t num_tokens,
                                             int32_t count, int64_t t) {
  uint32_t top = 0;
#pragma unroll
  for (int a = 0; a < K16V8_MAX_ROPE_AXES; ++a)
    if (a < count) top |= static_cast<uint32_t>(__ldg(positions + a * num_tokens + t));
  return top < static_cast<uint32_t>(kMaxPosition);
}

}  // namespace rope
}  // namespace k16v8

// The K8/V8 cache: E4M3 keys and values with one power-of-two scale per page
// and KV head for each of them.
//
// A scale is in [2^-15, 2^7].  With four significant bits to a code and 2^-9
// the smallest, every code times every such scale is an fp16 number (2^-24 the
// smallest, 57,344 the largest), so a kernel may widen pages to fp16 exactly,
// and a page that takes a larger scale keeps its codes' bits but for those that
// fall below the smallest code.
#pragma once

#include "k16v8_device.cuh"

namespace k16v8 {
namespace k8v8 {

constexpr int kMinExp = -15, kMaxExp = 7;
constexpr int kTileBytes = kPage * kHeadDim;  // codes of one page and head

// Exponent of the smallest power of two s with amax <= 448 s, within the range.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);  // amax >= 0 and finite
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
  static_assert(K16V8_E4M3_MAX == 448, "448 = 1.75 * 2^8");
  return max(kMinExp, min(e, kMaxExp));
}

// Exponent of the scale that a page has, or of the next power of two above one
// that is none, within the range.
__device__ __forceinline__ int stored_exponent(float scale) {
  const uint32_t bits = __float_as_uint(scale);
  const int e = static_cast<int>(bits >> 23) - 127 + ((bits & 0x7fffffu) != 0);
  return max(kMinExp, min(e, kMaxExp));
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((e + 127) << 23); }

}  // namespace k8v8
}  // namespace k16v8

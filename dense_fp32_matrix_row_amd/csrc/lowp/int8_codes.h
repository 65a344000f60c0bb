// int8_codes.h -- elements into 8-bit integers with a scale for each row, as the
// quantiser (int8_quantize.hip) and the linear layer of few tokens (int8_gemm.hip)
// make them (not installed).
#pragma once

#include "lowp.h"

namespace sgemm {
namespace int8 {

constexpr uint32_t kAmaxFloor = (127u - 100u) << 23;  // 2^-100
constexpr uint32_t kInfBits = 0x7f800000u;

// s, and its float reciprocal; r is 0 where a row holds an infinity or a NaN.
struct Scale {
  float s, r;
};

__device__ __forceinline__ Scale make_scale(uint32_t top) {
  if (top >= kInfBits) return Scale{__uint_as_float(0x7fc00000u), 0.0f};
  const float a = __uint_as_float(top < kAmaxFloor ? kAmaxFloor : top), s = a / 127.0f;
  return Scale{s, 1.0f / s};
}

// x / s rounded once, ties to even.  t = |x| r is within 127 * 2^-22 of the
// quotient, so the quotient lies within half a step and that of floor(t) + 1/2,
// the one border between integers that can decide: on which side of it |x| / s
// lies is the sign of |x| - border * s, which fma gives as it is (border has 8
// bits and s 24, so the difference, where it is small, is a float).  A tie goes to the even
// of the two.
__device__ __forceinline__ int code(float x, Scale q) {
  const float a = q.r == 0.0f ? 0.0f : fabsf(x), f = floorf(a * q.r), rest = fmaf(-(f + 0.5f), q.s, a);
  int k = static_cast<int>(f);
  k += rest > 0.0f || (rest == 0.0f && (k & 1)) ? 1 : 0;
  return x < 0.0f ? -k : k;
}

template <class X>
__device__ __forceinline__ Pack<8, int8_t> codes8(const Pack<8, X>& x, Scale q) {
  Pack<8, int8_t> c;
#pragma unroll
  for (int i = 0; i < 8; ++i) c.v[i] = static_cast<int8_t>(code(to_float(x.v[i]), q));
  return c;
}

struct Max {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};

template <class X>
__device__ __forceinline__ uint32_t top8(uint32_t top, const Pack<8, X>& x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, magnitude(to_float(x.v[i])));
  return top;
}

}  // namespace int8
}  // namespace sgemm

// lowp.h -- element types of the low-precision operators, read and written
// from float (not installed).
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include "../sgemm_internal.h"

namespace sgemm {

// bfloat16 by its bits: the conversions are exact in one direction and round
// to nearest even, NaN kept quiet, in the other.
struct bf16 {
  uint16_t bits;
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(bf16 x) { return __uint_as_float(uint32_t(x.bits) << 16); }
__device__ __forceinline__ float to_float(_Float16 x) { return static_cast<float>(x); }

__device__ __forceinline__ void from_float(float v, float& x) { x = v; }
__device__ __forceinline__ void from_float(float v, _Float16& x) { x = static_cast<_Float16>(v); }
__device__ __forceinline__ void from_float(float v, bf16& x) {
  const __bf16 b = static_cast<__bf16>(v);
  __builtin_memcpy(&x, &b, 2);
}

// N neighbours at once; any alignment of the element type.
template <int N, class T>
struct Pack {
  T v[N];
};
template <int N, class T>
__device__ __forceinline__ Pack<N, T> load_pack(const T* p) {
  Pack<N, T> r;
  __builtin_memcpy(&r, p, sizeof(r));
  return r;
}
template <int N, class T>
__device__ __forceinline__ void store_pack(T* p, const Pack<N, T>& r) {
  __builtin_memcpy(p, &r, sizeof(r));
}

}  // namespace sgemm

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

// The bits of |x|: as unsigned integers magnitudes order like their values, with
// infinities and then NaNs above.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Maximum over the 16 lanes of a group: with the neighbour, the next pair, the
// other half of eight and of sixteen.
template <int CONTROL>
__device__ __forceinline__ uint32_t max_with(uint32_t v) {
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CONTROL, 0xf, 0xf, true)));
}
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  return max_with<0x140>(max_with<0x141>(max_with<0x4e>(max_with<0xb1>(v))));
}

}  // namespace sgemm

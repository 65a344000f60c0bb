// rows.h -- rows held in registers, as the integer quantiser (int8_quantize.hip)
// and the layer norm (layernorm.hip) take them: LANES threads a row, COUNT chunks
// of eight neighbours each, chunk c of thread t at column (c LANES + t) 8.
#pragma once

#include <type_traits>

#include "lowp.h"

namespace sgemm {

template <int LANES_, int COUNT_, int THREADS_ = (LANES_ < 256 ? 256 : LANES_)>
struct RowShape {
  static constexpr int LANES = LANES_, COUNT = COUNT_;
  static constexpr int threads = THREADS_;          // of a block
  static constexpr int rows = threads / LANES;      // a block's at a time
  static constexpr int width = LANES * COUNT * 8;   // longest row
  static constexpr int waves = (LANES + 63) / 64;   // that share a row
  static_assert(threads % LANES == 0 && (LANES == 16 || LANES == 32 || LANES % 64 == 0));
};
constexpr int kRowWidth = 16384;  // the widest shape's

// Eight neighbours of a row from column `col`, zeros past `cols` (whose end is
// compared as cols - 8: col + 8 passes 2^31 in the widest row).
template <class X>
__device__ __forceinline__ Pack<8, X> load_row8(const X* row, int col, int cols) {
  if (col <= cols - 8) return load_pack<8>(row + col);
  Pack<8, X> p{};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col + i < cols) p.v[i] = row[col + i];
  return p;
}
// The same of a row of at least eight, without a branch around the load, behind which
// the compiler would wait for it: where fewer than eight are left, the row's last eight.
template <class X>
__device__ __forceinline__ Pack<8, X> load_last8(const X* row, int col, int cols) {
  return load_pack<8>(row + min(col, cols - 8));
}
// Those inside of eight neighbours of a row.
template <class X>
__device__ __forceinline__ void store_row8(X* row, int col, int cols, const Pack<8, X>& p) {
  if (col <= cols - 8) {
    store_pack(row + col, p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < cols) row[col + i] = p.v[i];
  }
}

// Of eight that load_last8 takes, those that no lane before has.
template <class X>
__device__ __forceinline__ void store_last8(X* row, int col, int cols, const Pack<8, X>& p) {
  const int before = col - (cols - 8);
  if (before <= 0) {
    store_pack(row + col, p);
  } else {
#pragma unroll
    for (int i = 1; i < 8; ++i)
      if (i >= before) row[cols - 8 + i] = p.v[i];
  }
}

// Another lane's value: the neighbour's, the next pair's, the other half of eight's
// and of sixteen's.
template <int CONTROL, class T>
__device__ __forceinline__ T from_lane(T v) {
  constexpr int words = sizeof(T) / 4;
  int w[words];
  __builtin_memcpy(w, &v, sizeof(T));
#pragma unroll
  for (int i = 0; i < words; ++i) w[i] = __builtin_amdgcn_update_dpp(0, w[i], CONTROL, 0xf, 0xf, true);
  __builtin_memcpy(&v, w, sizeof(T));
  return v;
}

// v joined over the lanes of a row, the same in each: within the wavefront, then
// by LDS in the wavefronts' order.  Where wavefronts share a row all threads of the
// block call it; a `meet` may be used again once all have met in another call.
template <class S, int N, class T, class F>
__device__ __forceinline__ void join_row(T (&v)[N], T (&meet)[S::threads / 64][N], const F& f) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = f(v[i], from_lane<0xb1>(v[i]));
    v[i] = f(v[i], from_lane<0x4e>(v[i]));
    v[i] = f(v[i], from_lane<0x141>(v[i]));
    v[i] = f(v[i], from_lane<0x140>(v[i]));
    if constexpr (S::LANES > 16) v[i] = f(v[i], __shfl_xor(v[i], 16));
    if constexpr (S::LANES > 32) v[i] = f(v[i], __shfl_xor(v[i], 32));
  }
  if constexpr (S::waves > 1) {
    if (threadIdx.x % 64 == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) meet[threadIdx.x / 64][i] = v[i];
    __syncthreads();
    const int first = S::rows > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / S::LANES) * S::waves : 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      T all = meet[first][i];
#pragma unroll
      for (int w = 1; w < S::waves; ++w) all = f(all, meet[first + w][i]);
      v[i] = all;
    }
  }
}

}  // namespace sgemm

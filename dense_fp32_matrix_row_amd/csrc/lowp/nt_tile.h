// nt_tile.h -- what the tiles of the block-scaled 8-bit product (fp8_gemm.hip)
// and of the orthogonalised update (orthogonal.hip) share: D = A * B^T over
// operands whose rows are contiguous along K.  nt_direct.h has the small tiles,
// nt_loop.h the large ones.
//
// Both operands are rows of bytes, taken 128 bytes a step: 128 e4m3 codes, or
// 32 numbers as halfs hi and lo (64 bytes each).  A step is eight 16-byte
// chunks of a row; lane group g = lane / 16 of a wavefront takes chunks g and
// 4 + g of row lane % 16.  For the 8-bit matrix instruction that is some
// permutation of the block's 128 k, the same one on both sides, which leaves
// the sum's terms as they are.
//
// B's rows go in as the instruction's first operand, A's as its second, so that
// a lane ends up with D[m][n .. n+3], m = lane % 16, n = 4 (lane / 16): four
// neighbours in a row of D, stored at once.
#pragma once

#include "../sgemm_internal.h"

namespace sgemm {
namespace nt {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kStep = 128;  // bytes of a row per step

// One operand: `rows` rows of K bytes, ld bytes apart (a multiple of 16, as
// the base), and a scale for each 1 << shift rows of each step.
struct Side {
  const uint8_t* p;
  int64_t ld;
  int rows;
  const void* s;
  int64_t s_row, s_col;
  int shift;
  int64_t batch;  // bytes between the matrices of a batch
};

struct Frag {
  v4i lo, hi;  // chunks g and 4 + g
};

// Where a block's tile lies in D.
struct Place {
  int tm, tn;
};

// Blocks in the order of their ids within an XCD walk columns of tiles `group`
// high, so that the tiles an XCD runs together share A and B panels in its L2.
__device__ __forceinline__ Place place_of(int64_t id, int tiles_m, int tiles_n, int group) {
  const int64_t per = int64_t(group) * tiles_n;
  const int first = static_cast<int>(id / per) * group;
  const int high = min(group, tiles_m - first);
  const int64_t in = id % per;
  return Place{first + static_cast<int>(in % high), static_cast<int>(in / high)};
}

// Zeroes the bytes of a chunk from byte `keep` on.
__device__ __forceinline__ v4i mask_chunk(v4i v, int keep) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int k = keep - 4 * w;
    v[w] = k >= 4 ? v[w] : k <= 0 ? 0 : v[w] & ((1 << (8 * k)) - 1);
  }
  return v;
}

__device__ __forceinline__ Frag mask_frag(Frag f, int g, int left) {
  f.lo = mask_chunk(f.lo, left - 16 * g);
  f.hi = mask_chunk(f.hi, left - 16 * (4 + g));
  return f;
}

// --- what a step does with two fragments -----------------------------------
//
// A policy's Op is a fragment as its matrix instructions take it; mac adds the
// product of B's fragment n and A's fragment m; kScaleBytes is what a scale has
// in memory, kRowScales whether mac takes the scales of the four D columns
// (floats, in sn) or B's row's own (bits, in sn[0]).

__device__ __forceinline__ v8i join(const Frag& f) {
  return __builtin_shufflevector(f.lo, f.hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// A scale as float: its bits, or 2^(e - 127) of an e8m0 byte (255 is NaN, 0 is
// subnormal).
template <int BYTES>
__device__ __forceinline__ float scale_value(uint32_t s) {
  if constexpr (BYTES == 4) return __uint_as_float(s);
  return __uint_as_float(s == 255 ? 0x7fc00000u : s == 0 ? 0x00400000u : s << 23);
}

// The 8-bit matrix instruction, as its rounding was measured: the products of
// eight neighbours along k are lined up with the largest of them and cut 13
// bits below it, and only the sums of eight are added as floats.  On normal
// data that is 1.5e-5 of the result, far below the half step of a 16-bit
// result (2^-8, 2^-11 of it), and far above a float's: float results use Widened.

// Float scales: a block of 128 is summed from zero and added times its scales
// (the matrix instruction can apply powers of two only).  UNIFORM: all B rows of a
// wavefront share a scale, so the scales' product is formed once a row of A and a
// step, and a result costs one vector instruction instead of two (beside an 8-bit
// product five fit: 13.7 ns; eight make 19).  It loses bits below 2^-126, where
// scaling one after the other would not; the header says so.
template <bool UNIFORM>
struct Fp8F32 {
  static constexpr int kScaleBytes = 4;
  static constexpr bool kUniform = UNIFORM, kRowScales = true;
  using Acc = v4f;
  using Op = v8i;
  static __device__ __forceinline__ Op prepare(const Frag& f) { return join(f); }
  static __device__ __forceinline__ void zero(Acc& a) { a = v4f{0, 0, 0, 0}; }
  static __device__ __forceinline__ void mac(Acc& acc, const Op& n, const Op& m, v4f sn, float sm) {
    const v4f z = {0, 0, 0, 0};
    add(acc, __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(n, m, z, 0, 0, 0, 0, 0, 0), sn, sm);
  }
  static __device__ __forceinline__ void add(Acc& acc, v4f t, v4f sn, float sm) {
    if constexpr (UNIFORM) {
      const float s = sm * sn[0];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(t[i], s, acc[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(t[i] * sm, sn[i], acc[i]);  // as the large tiles' loops do
    }
  }
  static __device__ __forceinline__ v4f value(const Acc& a) { return a; }
};

// Power-of-two scales, which the matrix instruction applies: lane l gives the
// scale of row l % 16, the same for all of the block's 128 k.
struct Fp8E8M0 {
  static constexpr int kScaleBytes = 1;
  static constexpr bool kUniform = false, kRowScales = false;
  using Acc = v4f;
  using Op = v8i;
  static __device__ __forceinline__ Op prepare(const Frag& f) { return join(f); }
  static __device__ __forceinline__ void zero(Acc& a) { a = v4f{0, 0, 0, 0}; }
  static __device__ __forceinline__ void mac(Acc& acc, const Op& n, const Op& m, uint32_t sn, uint32_t sm) {
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(n, m, acc, 0, 0, 0, sn, 0, sm);
  }
  static __device__ __forceinline__ v4f value(const Acc& a) { return a; }
};

// The codes widened to halfs, which is exact, and multiplied by the half
// instruction, whose sums keep a float's bits: half the 8-bit rate.
template <bool UNIFORM, int BYTES>
struct Widened {
  static constexpr int kScaleBytes = BYTES;
  static constexpr bool kUniform = UNIFORM, kRowScales = true;
  using Acc = v4f;
  struct Op {
    v8h k[4];
  };
  static __device__ __forceinline__ Op prepare(const Frag& f) {
    typedef _Float16 v2h __attribute__((ext_vector_type(2)));
    Op o;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t c = static_cast<uint32_t>(q < 2 ? f.lo[2 * q + w] : f.hi[2 * (q - 2) + w]);
        const v2h x = __builtin_bit_cast(v2h, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, false));
        const v2h y = __builtin_bit_cast(v2h, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, true));
        o.k[q][4 * w] = x[0];
        o.k[q][4 * w + 1] = x[1];
        o.k[q][4 * w + 2] = y[0];
        o.k[q][4 * w + 3] = y[1];
      }
    return o;
  }
  static __device__ __forceinline__ void zero(Acc& a) { a = v4f{0, 0, 0, 0}; }
  static __device__ __forceinline__ void mac(Acc& acc, const Op& n, const Op& m, v4f sn, float sm) {
    v4f t = {0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q) t = __builtin_amdgcn_mfma_f32_16x16x32_f16(n.k[q], m.k[q], t, 0, 0, 0);
    Fp8F32<UNIFORM>::add(acc, t, sn, sm);
  }
  static __device__ __forceinline__ v4f value(const Acc& a) { return a; }
};

// Pairs of halfs, x = hi + lo: hi hi' + hi lo' + lo hi'; lo lo' (2^-22 of the
// product) is left out, as small as the pair's own rounding.
struct HalfPair {
  static constexpr int kScaleBytes = 0;
  static constexpr bool kUniform = false, kRowScales = false;
  using Acc = v4f;
  using Op = Frag;
  static __device__ __forceinline__ Op prepare(const Frag& f) { return f; }
  static __device__ __forceinline__ void zero(Acc& a) { a = v4f{0, 0, 0, 0}; }
  static __device__ __forceinline__ void mac(Acc& acc, const Op& n, const Op& m, uint32_t, uint32_t) {
    const v8h nh = __builtin_bit_cast(v8h, n.lo), nl = __builtin_bit_cast(v8h, n.hi);
    const v8h mh = __builtin_bit_cast(v8h, m.lo), ml = __builtin_bit_cast(v8h, m.hi);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(nh, mh, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(nh, ml, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(nl, mh, acc, 0, 0, 0);
  }
  static __device__ __forceinline__ v4f value(const Acc& a) { return a; }
};

}  // namespace nt
}  // namespace sgemm

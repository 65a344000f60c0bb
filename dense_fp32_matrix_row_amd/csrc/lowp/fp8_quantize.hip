// fp8_quantize.hip -- hip_fp8_quantize: a matrix into e4m3 codes with a scale
// for each block of 1 x 128 or 128 x 128, as it lies, transposed, or both from
// one read.
//
// Bound by memory: e bytes read and one written per element and orientation,
// against some fifteen vector instructions per element and orientation.
#include "../../../include/blockfp8.h"
#include "lowp.h"

namespace sgemm {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr uint32_t kAmaxFloor = (127u - 100u) << 23;  // 2^-100
constexpr uint32_t kInfBits = 0x7f800000u;

// What a block's elements are multiplied by, and m as codes4 has it.
struct Factor {
  float f;
  uint32_t m;
};
// That and the bits of the scale that is stored.
struct Scale {
  Factor by;
  uint32_t stored;
};

__device__ __forceinline__ uint32_t round4(float a, float b, float c, float d) {
  const int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}

// x / s as a float whose rounding to e4m3 is that of the exact quotient.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  // The remainder x - t s is exact (t is within two units of the quotient),
  // so one correction with it rounds the quotient correctly.  Then the only
  // wrong roundings left are of quotients that fall on a border between two
  // codes by their float rounding alone: borders have at most five
  // significant bits, and the new remainder says to which side to step.
  float t = x * r;
  t = fmaf(fmaf(-t, s, x), r, t);
  const uint32_t b = __float_as_uint(t);
  if ((b & 0x7ffffu) == 0 && (b << 1) != 0) {
    const float rem = fmaf(-t, s, x);
    const float out = __uint_as_float(__float_as_uint(rem) ^ (b & 0x80000000u));  // > 0: away from zero
    t = __uint_as_float(b + (out > 0.0f ? 1 : 0) - (out < 0.0f ? 1 : 0));
  }
  return t;
}

// The codes of four elements x / s, each the exact quotient rounded once.
//
// Power-of-two scales: the product with 1 / s is exact.
//
// Float scales, 16-bit x: with a the block's largest magnitude, 448 x / a is
// either a border between two codes (of five bits) or at least 2^-16 of it away,
// x and a having 11 bits at most.  s = a / 448 (1 + e), |e| <= 2^-24, so the
// quotients that matter are all off their borders to the same side, by e's
// sign: f = 1 / s is moved 2^-19 to that side, past all rounding errors
// (2^-22 together), and the product rounds as the quotient does.  Where e is 0
// a border is met exactly, and the tie goes to the even code: the product is
// rounded to 18 bits first, which gives a border that is 2^-22 away itself and
// keeps all else on its side.  m is the mask of that rounding, or of none.
// One element in 200 of bf16 data is such a border.
//
// Float scales, float x: the exact quotient lies between the products with
// 1 / s less and more three units (at least 3 x 2^-24 off, x r within 2 x 2^-24),
// so where both round to the same code that is it.  Elsewhere, one element in
// 10^5 of ordinary data, the quotient is looked at closely.  m holds s.
template <int KIND, class X>
__device__ __forceinline__ uint32_t codes4(X a, X b, X c, X d, Factor q) {
  const float x[4] = {to_float(a), to_float(b), to_float(c), to_float(d)};
  if constexpr (KIND == HIP_FP8_SCALE_E8M0) {
    return round4(x[0] * q.f, x[1] * q.f, x[2] * q.f, x[3] * q.f);
  } else if constexpr (sizeof(X) == 2) {
    const uint32_t half = (0u - q.m) >> 1;
    const auto t = [&](float v) { return __uint_as_float((__float_as_uint(v * q.f) + half) & q.m); };
    return round4(t(x[0]), t(x[1]), t(x[2]), t(x[3]));
  } else {
    const float less = __uint_as_float(__float_as_uint(q.f) - 3), more = __uint_as_float(__float_as_uint(q.f) + 3);
    uint32_t v = round4(x[0] * less, x[1] * less, x[2] * less, x[3] * less);
    if (v != round4(x[0] * more, x[1] * more, x[2] * more, x[3] * more)) {
      const float s = __uint_as_float(q.m);
      v = round4(quotient(x[0], s, q.f), quotient(x[1], s, q.f), quotient(x[2], s, q.f), quotient(x[3], s, q.f));
    }
    return v;
  }
}

// From the bits of the largest |x|: as unsigned integers magnitudes order like
// their values, with infinities and then NaNs above, so that neither is lost
// in the maximum.  A block that holds one has a NaN for a factor, which makes
// every code NaN.
template <int KIND, class X>
__device__ __forceinline__ Scale make_scale(uint32_t top) {
  Scale q;
  const bool bad = top >= kInfBits;
  if (top < kAmaxFloor) top = kAmaxFloor;
  if constexpr (KIND == HIP_FP8_SCALE_F32) {
    const float a = __uint_as_float(top), s = a / kE4m3Max, r = 1.0f / s;
    if constexpr (sizeof(X) == 2) {
      const float e = fmaf(-s, kE4m3Max, a);  // exact; > 0: s is less than a / 448, the quotients more
      q.by.f = e > 0.0f ? r * (1.0f + 0x1p-19f) : e < 0.0f ? r * (1.0f - 0x1p-19f) : r;
      q.by.m = e == 0.0f ? ~0x3fu : ~0u;
    } else {
      q.by.f = r;
      q.by.m = __float_as_uint(s);
    }
    q.stored = bad ? 0x7fc00000u : __float_as_uint(s);
  } else {
    // a = f 2^p with 1 <= f < 2, 448 = 1.75 2^8: 2^(p-8), or twice that for f > 1.75
    const uint32_t e = (top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    q.by.f = __uint_as_float((254 - e) << 23);
    q.by.m = 0;
    q.stored = bad ? 0xffu : e;
  }
  if (bad) q.by.f = __uint_as_float(0x7fc00000u);
  return q;
}

template <int KIND>
__device__ __forceinline__ void store_scale(void* s, int64_t at, const Scale& q) {
  if constexpr (KIND == HIP_FP8_SCALE_F32) static_cast<uint32_t*>(s)[at] = q.stored;
  else static_cast<uint8_t*>(s)[at] = static_cast<uint8_t>(q.stored);
}

// Eight neighbours of a row from column `col`, zeros past `cols` (whose end is
// compared as cols - 8: col + 8 passes 2^31 in the widest row).
template <class X>
__device__ __forceinline__ Pack<8, X> load8(const X* row, int col, int cols) {
  if (col <= cols - 8) return load_pack<8>(row + col);
  Pack<8, X> p{};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col + i < cols) p.v[i] = row[col + i];
  return p;
}

// The codes of eight neighbours.
template <int KIND, class X>
__device__ __forceinline__ uint2 codes8(const Pack<8, X>& p, Factor q) {
  return make_uint2(codes4<KIND>(p.v[0], p.v[1], p.v[2], p.v[3], q), codes4<KIND>(p.v[4], p.v[5], p.v[6], p.v[7], q));
}

// Eight codes of a row from column `col`, none past `cols`.
__device__ __forceinline__ void store8(uint8_t* row, int col, int cols, uint2 c) {
  if (col <= cols - 8) {
    __builtin_memcpy(row + col, &c, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < cols) row[col + i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i % 4)));
  }
}

// Makes the compiler forget what it made of the elements so far, lest it keep
// them as floats beside the halves that they come as: twice the registers.
template <class X>
__device__ __forceinline__ void forget(Pack<8, X>& p) {
  if constexpr (sizeof(X) == 2) {
    uint4 w = __builtin_bit_cast(uint4, p);
    asm volatile("" : "+v"(w.x), "+v"(w.y), "+v"(w.z), "+v"(w.w));
    p = __builtin_bit_cast(Pack<8, X>, w);
  }
}

struct Args {
  int rows, cols;
  int64_t ldx;
  uint8_t* q;
  int64_t ldq;
  void* s;
  int64_t s_row, s_col;
  uint8_t* qt;
  int64_t ldqt;
  void* st;
  int64_t st_row, st_col;
};

// Blocks of 1 x 128 as the matrix lies: sixteen lanes a block, eight neighbours
// each, nothing shared, so that a few rows still spread over many CUs.  16 x 1024
// in 2.9 us, all of it a launch; 8192 x 8192 bf16 in 41 us (4.9 TB/s), floats in 56.
template <class X, int KIND>
__global__ __launch_bounds__(256) void k_rows(const X* __restrict__ x, Args a, int64_t items, int blocks) {
  const int lane = threadIdx.x % 16;
  for (int64_t it = int64_t(blockIdx.x) * 16 + threadIdx.x / 16; it < items; it += int64_t(gridDim.x) * 16) {
    const int64_t row = it / blocks;
    const int kb = static_cast<int>(it % blocks), col = kb * 128 + lane * 8;
    const Pack<8, X> v = load8(x + row * a.ldx, col, a.cols);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, magnitude(to_float(v.v[i])));
    const Scale q = make_scale<KIND, X>(max16(top));
    store8(a.q + row * a.ldq, col, a.cols, codes8<KIND>(v, q.by));
    if (lane == 0) store_scale<KIND>(a.s, row * a.s_row + kb * a.s_col, q);
  }
}

// 128 x 128 tiles, a thread holding 8 x 8 of it: rows 8 rg .., columns 8 cg ...
// Blocks of 128 x 128 have one scale for the tile; blocks of 1 x 128 one for
// each row (a maximum over 16 lanes) and, transposed, one for each column (a
// maximum through LDS); a thread each works out those 256 scales.  Transposed
// codes go through LDS too, so that they leave in 128-byte rows: column c's eight
// bytes of row group rg lie in slot rg ^ (c / 8) of 16, which spreads both sides
// over the banks.  Bound by memory: 8192 x 8192 bf16 both ways, 260 MiB, in 61-62 us
// (4.4 TB/s; a copy reaches 4.9), one way in 40 (5.0).  Rows of an odd number of
// floats begin off the 16 bytes that a load takes and lie over one more cache line:
// 4096 x 2048 in 9.7 us (5.2 TB/s), 4097 x 2048 in 10.3, 4096 x 2049 in 14.2, 4097 x
// 2049 in 14.7-15.0 (3.4); 8192 x 4096 32.2, 8193 x 4097 41.5.  A tile a block, so
// few tokens leave CUs idle: 256 x 1024 bf16 both ways on 16 blocks in 6.7-7.4.
template <class X, int KIND, int BR, bool AS_IS, bool TRANS>
__global__ __launch_bounds__(256, 2) void k_tile(const X* __restrict__ x, Args a, int tiles_c, int64_t tiles) {
  __shared__ uint32_t part[16][128];
  __shared__ Factor cscale[128], rscale[128];  // of column 8 c + i at 16 i + c, of rows as they are
  __shared__ alignas(16) uint32_t row_top[128];
  __shared__ alignas(16) uint8_t tr[TRANS ? 128 * 128 : 16];
  const int cg = threadIdx.x % 16, rg = threadIdx.x / 16;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t tr_i = tile / tiles_c, tc_i = tile % tiles_c;
    const int64_t r0 = tr_i * 128, c0 = tc_i * 128;
    const int rows = static_cast<int>(min(int64_t(128), a.rows - r0));
    const int cols = static_cast<int>(min(int64_t(128), a.cols - c0));
    const int col = cg * 8;

    Pack<8, X> v[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int row = rg * 8 + p;
      v[p] = row < rows ? load8(x + (r0 + row) * a.ldx + c0, col, cols) : Pack<8, X>{};
    }

    uint32_t rtop[8], ctop[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      rtop[p] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) rtop[p] = max(rtop[p], magnitude(to_float(v[p].v[i])));
    }

#pragma unroll
    for (int p = 0; p < 8; ++p) forget(v[p]);
    Factor whole;
    if constexpr (BR == 128) {
      uint32_t top = 0;
#pragma unroll
      for (int p = 0; p < 8; ++p) top = max(top, rtop[p]);
      part[rg][cg] = top;
      __syncthreads();
      top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, part[(threadIdx.x % 64) / 16 * 4 + i][cg]);
      top = max16(top);
      top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16)));
      top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
      const Scale q = make_scale<KIND, X>(top);
      whole = q.by;
      if (threadIdx.x == 0) {
        if constexpr (AS_IS) store_scale<KIND>(a.s, tr_i * a.s_row + tc_i * a.s_col, q);
        if constexpr (TRANS) store_scale<KIND>(a.st, tc_i * a.st_row + tr_i * a.st_col, q);
      }
    } else if constexpr (TRANS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ctop[i] = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) ctop[i] = max(ctop[i], magnitude(to_float(v[p].v[i])));
        part[rg][col + i] = ctop[i];
      }
      if constexpr (AS_IS) {
#pragma unroll
        for (int p = 0; p < 8; ++p) rtop[p] = max16(rtop[p]);
        if (cg == 0) {
          *reinterpret_cast<uint4*>(&row_top[rg * 8]) = make_uint4(rtop[0], rtop[1], rtop[2], rtop[3]);
          *reinterpret_cast<uint4*>(&row_top[rg * 8 + 4]) = make_uint4(rtop[4], rtop[5], rtop[6], rtop[7]);
        }
      }
      __syncthreads();
      if (AS_IS && threadIdx.x >= 128) {
        const int row = threadIdx.x - 128;
        const Scale q = make_scale<KIND, X>(row_top[row]);
        rscale[row] = q.by;
        if (row < rows) store_scale<KIND>(a.s, (r0 + row) * a.s_row + tc_i * a.s_col, q);
      }
      if (threadIdx.x < 128) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max(top, part[i][threadIdx.x]);
        const Scale q = make_scale<KIND, X>(top);
        cscale[threadIdx.x % 8 * 16 + threadIdx.x / 8] = q.by;
        if (static_cast<int>(threadIdx.x) < cols)
          store_scale<KIND>(a.st, (c0 + threadIdx.x) * a.st_row + tr_i * a.st_col, q);
      }
      __syncthreads();
    }

#pragma unroll
    for (int p = 0; p < 8; ++p) forget(v[p]);
    if constexpr (AS_IS) {
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const int row = rg * 8 + p;
        Factor by = whole;
        if constexpr (BR == 1) by = rscale[row];
        if (row < rows)
          store8(a.q + (r0 + row) * a.ldq + c0, col, cols, codes8<KIND>(v[p], by));
      }
    }
    if constexpr (TRANS) {
#pragma unroll
      for (int p = 0; p < 8; ++p) forget(v[p]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        Factor by = whole;
        if constexpr (BR == 1) by = cscale[16 * i + cg];
        Pack<8, X> column;
#pragma unroll
        for (int p = 0; p < 8; ++p) column.v[p] = v[p].v[i];
        *reinterpret_cast<uint2*>(&tr[(col + i) * 128 + 8 * (rg ^ cg)]) = codes8<KIND>(column, by);
      }
      __syncthreads();
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int c = p * 32 + threadIdx.x / 8, h = threadIdx.x % 8, x8 = c / 8;  // 16 bytes: row groups 2h, 2h + 1
        uint4 w = *reinterpret_cast<const uint4*>(&tr[c * 128 + 16 * (h ^ (x8 / 2))]);
        if (x8 & 1) w = make_uint4(w.z, w.w, w.x, w.y);
        if (c < cols) {
          uint8_t* out = a.qt + (c0 + c) * a.ldqt + r0;
          if (16 * h + 16 <= rows) {
            __builtin_memcpy(out + 16 * h, &w, 16);
          } else {
            store8(out, 16 * h, rows, make_uint2(w.x, w.y));
            store8(out, 16 * h + 8, rows, make_uint2(w.z, w.w));
          }
        }
      }
    }
    if constexpr (TRANS || BR == 128) __syncthreads();  // the next tile writes the same LDS
  }
}

template <class X, int KIND, int BR>
void launch_kind(const void* x, const Args& a, hipStream_t stream) {
  const X* p = static_cast<const X*>(x);
  const int blocks = static_cast<int>(ceil_div(a.cols, 128));
  const int64_t cap = kMaxWorkItems / 256;
  if constexpr (BR == 1) {
    if (!a.qt) {
      const int64_t items = int64_t(a.rows) * blocks;
      const int64_t grid = ceil_div(items, 16) < cap ? ceil_div(items, 16) : cap;
      hipLaunchKernelGGL((k_rows<X, KIND>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, stream, p, a, items,
                         blocks);
      return;
    }
  }
  const int64_t tiles = ceil_div(a.rows, 128) * blocks;
  const dim3 grid(static_cast<unsigned>(tiles < cap ? tiles : cap));
  if (a.q && a.qt) hipLaunchKernelGGL((k_tile<X, KIND, BR, true, true>), grid, dim3(256), 0, stream, p, a, blocks, tiles);
  else if (a.qt) hipLaunchKernelGGL((k_tile<X, KIND, BR, false, true>), grid, dim3(256), 0, stream, p, a, blocks, tiles);
  else if constexpr (BR == 128) hipLaunchKernelGGL((k_tile<X, KIND, BR, true, false>), grid, dim3(256), 0, stream, p, a, blocks, tiles);
}

template <class X>
void launch_type(const void* x, int block_rows, int kind, const Args& a, hipStream_t stream) {
  if (kind == HIP_FP8_SCALE_F32) {
    if (block_rows == 1) launch_kind<X, HIP_FP8_SCALE_F32, 1>(x, a, stream);
    else launch_kind<X, HIP_FP8_SCALE_F32, 128>(x, a, stream);
  } else {
    if (block_rows == 1) launch_kind<X, HIP_FP8_SCALE_E8M0, 1>(x, a, stream);
    else launch_kind<X, HIP_FP8_SCALE_E8M0, 128>(x, a, stream);
  }
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" {

int hip_fp8_quantize(int rows, int cols, const void* X, int x_type, int ldx, int block_rows, int scale_type,
                     void* Q, int ldq, void* S, long long s_row, long long s_col,
                     void* QT, int ldqt, void* ST, long long st_row, long long st_col, hipStream_t stream) {
  if (rows < 0) return -1;
  if (cols < 0) return -2;
  if (x_type != HIP_FP8_F32 && x_type != HIP_FP8_BF16 && x_type != HIP_FP8_F16) return -4;
  if (ldx < (cols > 1 ? cols : 1)) return -5;
  if (block_rows != 1 && block_rows != 128) return -6;
  if (scale_type != HIP_FP8_SCALE_F32 && scale_type != HIP_FP8_SCALE_E8M0) return -7;
  const bool n = Q != nullptr || S != nullptr, t = QT != nullptr || ST != nullptr;
  if (rows > 0 && cols > 0) {
    if (X == nullptr) return -3;
    if (!n && !t) return -8;
    if (n && Q == nullptr) return -8;
    if (n && S == nullptr) return -10;
    if (t && QT == nullptr) return -13;
    if (t && ST == nullptr) return -15;
  }
  if (n && ldq < (cols > 1 ? cols : 1)) return -9;
  if (n && s_row < 0) return -11;
  if (n && s_col < 0) return -12;
  if (t && ldqt < (rows > 1 ? rows : 1)) return -14;
  if (t && st_row < 0) return -16;
  if (t && st_col < 0) return -17;
  if (rows == 0 || cols == 0) return 0;
  const Args a{rows, cols, ldx, static_cast<uint8_t*>(Q), ldq, S, s_row, s_col,
               static_cast<uint8_t*>(QT), ldqt, ST, st_row, st_col};
  if (x_type == HIP_FP8_F32) launch_type<float>(X, block_rows, scale_type, a, stream);
  else if (x_type == HIP_FP8_BF16) launch_type<bf16>(X, block_rows, scale_type, a, stream);
  else launch_type<_Float16>(X, block_rows, scale_type, a, stream);
  return static_cast<int>(hipGetLastError());
}

const char* hip_fp8_quantize_status_string(int status) {
  switch (status) {
    case 0: return "success";
    case -1: return "argument 1 (rows) is negative";
    case -2: return "argument 2 (cols) is negative";
    case -3: return "argument 3 (X) is NULL";
    case -4: return "argument 4 (x_type) is not a known type";
    case -5: return "argument 5 (ldx) is smaller than max(1, cols)";
    case -6: return "argument 6 (block_rows) is not 1 or 128";
    case -7: return "argument 7 (scale_type) is not a known type";
    case -8: return "argument 8 (Q) is NULL but S is given, or neither Q nor QT is given";
    case -9: return "argument 9 (ldq) is smaller than max(1, cols)";
    case -10: return "argument 10 (S) is NULL but Q is given";
    case -11: return "argument 11 (s_row) is negative";
    case -12: return "argument 12 (s_col) is negative";
    case -13: return "argument 13 (QT) is NULL but ST is given";
    case -14: return "argument 14 (ldqt) is smaller than max(1, rows)";
    case -15: return "argument 15 (ST) is NULL but QT is given";
    case -16: return "argument 16 (st_row) is negative";
    case -17: return "argument 17 (st_col) is negative";
    default: break;
  }
  if (status > 0) return hipGetErrorString(static_cast<hipError_t>(status));
  return "unknown status";
}

}  // extern "C"

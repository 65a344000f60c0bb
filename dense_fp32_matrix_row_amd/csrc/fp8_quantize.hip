// fp8_quantize.hip -- hip_fp8_quantize: a matrix into e4m3 codes with a scale
// for each block of 1 x 128 or 128 x 128, as it lies, transposed, or both from
// one read.
//
// Bound by memory: e bytes read and one written per element and orientation,
// against some fifteen vector instructions per element and orientation.
#include "../../include/blockfp8.h"
#include "lowp.h"

namespace sgemm {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr uint32_t kAmaxFloor = (127u - 100u) << 23;  // 2^-100
constexpr uint32_t kInfBits = 0x7f800000u;

// A block's scale: s and 1 / s, for float scales also three units less and more
// of 1 / s, and what is stored for it.
struct Scale {
  float s, r, less, more;
  uint32_t stored;
  bool bad;  // the block holds an infinity or a NaN
};

// From the bits of the largest |x|: as unsigned integers magnitudes order like
// their values, with infinities and then NaNs above, so that neither is lost
// in the maximum.
template <int KIND>
__device__ __forceinline__ Scale make_scale(uint32_t top) {
  Scale q;
  q.bad = top >= kInfBits;
  if (top < kAmaxFloor) top = kAmaxFloor;
  if constexpr (KIND == HIP_FP8_SCALE_F32) {
    q.s = __uint_as_float(top) / kE4m3Max;
    q.r = 1.0f / q.s;
    q.less = __uint_as_float(__float_as_uint(q.r) - 3);
    q.more = __uint_as_float(__float_as_uint(q.r) + 3);
    q.stored = q.bad ? 0x7fc00000u : __float_as_uint(q.s);
  } else {
    // a = f 2^p with 1 <= f < 2, 448 = 1.75 2^8: 2^(p-8), or twice that for f > 1.75
    const uint32_t e = (top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    q.s = __uint_as_float(e << 23);
    q.r = __uint_as_float((254 - e) << 23);
    q.stored = q.bad ? 0xffu : e;
  }
  return q;
}

// x / s as a float whose rounding to e4m3 is that of the exact quotient.
template <int KIND>
__device__ __forceinline__ float quotient(float x, const Scale& q) {
  float t = x * q.r;
  if constexpr (KIND == HIP_FP8_SCALE_F32) {
    // The remainder x - t s is exact (t is within two units of the quotient),
    // so one correction with it rounds the quotient correctly.  Then the only
    // wrong roundings left are of quotients that fall on a border between two
    // codes by their float rounding alone: borders have at most five
    // significant bits, and the new remainder says to which side to step.
    t = fmaf(fmaf(-t, q.s, x), q.r, t);
    const uint32_t b = __float_as_uint(t);
    if ((b & 0x7ffffu) == 0 && (b << 1) != 0) {
      const float rem = fmaf(-t, q.s, x);
      const float out = __uint_as_float(__float_as_uint(rem) ^ (b & 0x80000000u));  // > 0: away from zero
      t = __uint_as_float(b + (out > 0.0f ? 1 : 0) - (out < 0.0f ? 1 : 0));
    }
  }
  return t;
}

__device__ __forceinline__ uint32_t round4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}

// The codes of four quotients.  For float scales the exact quotient lies
// between the products with `less` and `more` (x r is within 2^-24 of it from
// r's rounding and 2^-24 from its own, three units are 3 x 2^-24 at least), so
// where both round to the same code that is it.  Elsewhere, one element in
// 10^5 of ordinary data, the quotient is looked at closely; all together 4
// instructions an element instead of 12.
template <int KIND>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, const Scale& q) {
  uint32_t v;
  if constexpr (KIND == HIP_FP8_SCALE_F32) {
    v = round4(a * q.less, b * q.less, c * q.less, d * q.less);
    if (v != round4(a * q.more, b * q.more, c * q.more, d * q.more))
      v = round4(quotient<KIND>(a, q), quotient<KIND>(b, q), quotient<KIND>(c, q), quotient<KIND>(d, q));
  } else {
    v = round4(quotient<KIND>(a, q), quotient<KIND>(b, q), quotient<KIND>(c, q), quotient<KIND>(d, q));
  }
  return q.bad ? 0x7f7f7f7fu : v;
}

template <int KIND>
__device__ __forceinline__ void store_scale(void* s, int64_t at, const Scale& q) {
  if constexpr (KIND == HIP_FP8_SCALE_F32) static_cast<uint32_t*>(s)[at] = q.stored;
  else static_cast<uint8_t*>(s)[at] = static_cast<uint8_t>(q.stored);
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Eight neighbours of a row from column `col`, zeros past `cols`.
template <class X>
__device__ __forceinline__ void load8(const X* row, int col, int cols, float (&v)[8]) {
  if (col + 8 <= cols) {
    const Pack<8, X> p = load_pack<8>(row + col);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_float(p.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = col + i < cols ? to_float(row[col + i]) : 0.0f;
  }
}

// Eight codes of a row from column `col`, none past `cols`.
__device__ __forceinline__ void store8(uint8_t* row, int col, int cols, uint2 c) {
  if (col + 8 <= cols) {
    __builtin_memcpy(row + col, &c, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < cols) row[col + i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i % 4)));
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

// Maximum over the 16 lanes of a group.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 16; d *= 2) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), d)));
  return v;
}

// Blocks of 1 x 128 as the matrix lies: sixteen lanes a block, eight neighbours
// each, nothing shared, so that a few rows still spread over many CUs.
template <class X, int KIND>
__global__ __launch_bounds__(256) void k_rows(const X* __restrict__ x, Args a, int64_t items, int blocks) {
  const int lane = threadIdx.x % 16;
  for (int64_t it = int64_t(blockIdx.x) * 16 + threadIdx.x / 16; it < items; it += int64_t(gridDim.x) * 16) {
    const int64_t row = it / blocks;
    const int kb = static_cast<int>(it % blocks), col = kb * 128 + lane * 8;
    float v[8];
    load8(x + row * a.ldx, col, a.cols, v);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, magnitude(v[i]));
    const Scale q = make_scale<KIND>(max16(top));
    store8(a.q + row * a.ldq, col, a.cols,
           make_uint2(codes4<KIND>(v[0], v[1], v[2], v[3], q), codes4<KIND>(v[4], v[5], v[6], v[7], q)));
    if (lane == 0) store_scale<KIND>(a.s, row * a.s_row + kb * a.s_col, q);
  }
}

// 128 x 128 tiles, a thread holding 8 x 8 of it: rows 8 rg .., columns 8 cg ...
// Blocks of 128 x 128 have one scale for the tile; blocks of 1 x 128 one for
// each row (a maximum over 16 lanes) and, transposed, one for each column (a
// maximum through LDS).  Transposed codes go through LDS too, so that they
// leave in 128-byte rows: column c's eight bytes of row group rg lie in slot
// rg ^ (c / 8) of 16, which spreads both sides over the banks.
template <class X, int KIND, int BR, bool AS_IS, bool TRANS>
__global__ __launch_bounds__(256) void k_tile(const X* __restrict__ x, Args a, int tiles_c, int64_t tiles) {
  __shared__ uint32_t part[16][128];
  __shared__ Scale cscale[128];
  __shared__ alignas(16) uint8_t tr[TRANS ? 128 * 128 : 16];
  const int cg = threadIdx.x % 16, rg = threadIdx.x / 16;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t tr_i = tile / tiles_c, tc_i = tile % tiles_c;
    const int64_t r0 = tr_i * 128, c0 = tc_i * 128;
    const int rows = static_cast<int>(min(int64_t(128), a.rows - r0));
    const int cols = static_cast<int>(min(int64_t(128), a.cols - c0));
    const int col = cg * 8;

    float v[8][8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int row = rg * 8 + p;
      if (row < rows) {
        load8(x + (r0 + row) * a.ldx + c0, col, cols, v[p]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[p][i] = 0.0f;
      }
    }

    uint32_t rtop[8], ctop[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      rtop[p] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) rtop[p] = max(rtop[p], magnitude(v[p][i]));
    }

    Scale whole;
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
      whole = make_scale<KIND>(top);
      if (threadIdx.x == 0) {
        if constexpr (AS_IS) store_scale<KIND>(a.s, tr_i * a.s_row + tc_i * a.s_col, whole);
        if constexpr (TRANS) store_scale<KIND>(a.st, tc_i * a.st_row + tr_i * a.st_col, whole);
      }
    } else if constexpr (TRANS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ctop[i] = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) ctop[i] = max(ctop[i], magnitude(v[p][i]));
        part[rg][col + i] = ctop[i];
      }
      __syncthreads();
      if (threadIdx.x < 128) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max(top, part[i][threadIdx.x]);
        const Scale q = make_scale<KIND>(top);
        cscale[threadIdx.x] = q;
        if (static_cast<int>(threadIdx.x) < cols)
          store_scale<KIND>(a.st, (c0 + threadIdx.x) * a.st_row + tr_i * a.st_col, q);
      }
      __syncthreads();
    }

    if constexpr (AS_IS) {
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const int row = rg * 8 + p;
        Scale q = whole;
        if constexpr (BR == 1) {
          q = make_scale<KIND>(max16(rtop[p]));
          if (cg == 0 && row < rows) store_scale<KIND>(a.s, (r0 + row) * a.s_row + tc_i * a.s_col, q);
        }
        if (row < rows)
          store8(a.q + (r0 + row) * a.ldq + c0, col, cols,
                 make_uint2(codes4<KIND>(v[p][0], v[p][1], v[p][2], v[p][3], q),
                            codes4<KIND>(v[p][4], v[p][5], v[p][6], v[p][7], q)));
      }
    }
    if constexpr (TRANS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        Scale q = whole;
        if constexpr (BR == 1) q = cscale[col + i];
        const uint2 c = make_uint2(codes4<KIND>(v[0][i], v[1][i], v[2][i], v[3][i], q),
                                   codes4<KIND>(v[4][i], v[5][i], v[6][i], v[7][i], q));
        *reinterpret_cast<uint2*>(&tr[(col + i) * 128 + 8 * (rg ^ cg)]) = c;
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
  else hipLaunchKernelGGL((k_tile<X, KIND, BR, true, false>), grid, dim3(256), 0, stream, p, a, blocks, tiles);
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

// orthogonal.hip -- hip_orthogonalize: Newton-Schulz products on the matrix
// cores with operands as pairs of halfs.
//
// A number x of a matrix is kept as hi + lo with halfs hi = RN(s x), lo =
// RN(s x - hi) for a power of two s: 22 significant bits while |s x| is between
// 2^-3 and 65504, an absolute 2^-25 below (a half's least step is 2^-24).  The sums
// are float.  Three half products an element (hi hi', hi lo', lo hi') run at a
// third of the half rate, three times the float matrix rate (4096 x 4096: 425
// TFLOP/s of the products asked for, against 150), and err no more than float
// products do (4096 x 4096, five steps: 3.3e-6 of the norm against 4.8e-6).
//
// So that rows and columns much smaller than the rest keep their bits, X is kept
// as X^ = D^-1 X and X~ = D^-1 X E^-1 with powers of two D (rows) and E (columns)
// near the square roots of the rows' and columns' norms.  An element is at most the
// smaller of its row's and its column's norm, so at most the product of the roots:
// nothing leaves the range, and a row 2^-40 of the largest is 2^-20 of it here (512 x 1024,
// five steps, one row in 16 smaller by 1e-4, 1e-6, 1e-9: those rows off by 5e-7,
// 5e-7, 6e-6 of their norm, with D = E = 1 by 3e-5, 3e-3 and all; float products
// 8e-7).  It costs 3 % at 4096 x 4096, about half of it power: more bits are set.
// The roots come from the largest elements, norm <= sqrt(n) max |x|, and grow with
// the steps as the polynomial lets a norm grow at most; s of each matrix is the
// largest power of two that its bound allows (schedule()).
//
// Per step, with m <= n the sides of the iterate X and X^T kept beside it, all
// operands have their K side contiguous:
//   U = D^-1 S = X^ X^^T D            (m x m, K = n; X^ X^^T is symmetric: the lower
//                                     tiles, mirrored)
//   P~ = D^-1 P D = a + (b U + c U U^T D) D  with P = a + b S + c S S
//                                     (m x m, K = m; U U^T is symmetric)
//   D^-1 X' E^-1 = P~ X~              (m x n, K = m; X~^T is the other operand),
//                                     written as X^' over X^, which is not read,
//                                     and as X~'^T into the other of two buffers.
#include "../../../include/orthogonal.h"
#include "lowp.h"
#include "nt_direct.h"
#include "nt_loop.h"

#include <cmath>

namespace sgemm {
namespace {

using nt::Side;
using nt::v4f;

// The norms' pass: a block takes kNormRows x 256 elements at a time.  Of each side as
// many parts as that needs, but columns at most 64, rows at most 256 and such that
// all are about 1024: what follows reads all parts of 64 rows and columns in every
// block.
constexpr int kNormRows = 16, kMaxColParts = 64, kMaxRowParts = 256, kNormBlocks = 1024;
constexpr int kLeastExponent = -120;  // of a row's or column's norm: its root's inverse stays a float

__host__ __device__ inline int64_t pad32(int64_t n) { return (n + 31) / 32 * 32; }

// A matrix of pairs: row r, element k at r * ld + (k / 32) * 128 + 2 (k % 32),
// hi there and lo 64 bytes on; rows padded to 32 elements with zeros.
struct Pairs {
  uint8_t* p;
  int64_t ld;     // bytes
  int64_t batch;  // bytes between matrices
};

__device__ __forceinline__ int64_t pair_at(int64_t k) { return k / 32 * 128 + 2 * (k % 32); }

__device__ __forceinline__ void split(float v, _Float16& hi, _Float16& lo) {
  hi = static_cast<_Float16>(v);
  lo = static_cast<_Float16>(v - static_cast<float>(hi));
}

__device__ __forceinline__ void store_pair(uint8_t* row, int64_t k, float v) {
  _Float16 hi, lo;
  split(v, hi, lo);
  uint8_t* at = row + pair_at(k);
  *reinterpret_cast<_Float16*>(at) = hi;
  *reinterpret_cast<_Float16*>(at + 64) = lo;
}

// From a matrix that the kernel does not write: such loads need not wait for the
// stores before them.
template <class V>
__device__ __forceinline__ V load_unwritten(const uint8_t* at) {
  return *reinterpret_cast<const __attribute__((address_space(4))) V*>(reinterpret_cast<uintptr_t>(at));
}

__device__ __forceinline__ float load_pair(const uint8_t* row, int64_t k) {
  const uint8_t* at = row + pair_at(k);
  return static_cast<float>(load_unwritten<_Float16>(at)) + static_cast<float>(load_unwritten<_Float16>(at + 64));
}

// Four neighbours from k, a multiple of 4.
__device__ __forceinline__ void store_pairs(uint8_t* row, int64_t k, v4f v) {
  Pack<4, _Float16> hi, lo;
#pragma unroll
  for (int i = 0; i < 4; ++i) split(v[i], hi.v[i], lo.v[i]);
  uint8_t* at = row + pair_at(k);
  *reinterpret_cast<uint2*>(at) = __builtin_bit_cast(uint2, hi);
  *reinterpret_cast<uint2*>(at + 64) = __builtin_bit_cast(uint2, lo);
}

// Eight neighbours from k, a multiple of 8: two stores of 16 bytes.
__device__ __forceinline__ void store_pairs8(uint8_t* row, int64_t k, const float (&v)[8]) {
  Pack<8, _Float16> hi, lo;
#pragma unroll
  for (int i = 0; i < 8; ++i) split(v[i], hi.v[i], lo.v[i]);
  uint8_t* at = row + pair_at(k);
  *reinterpret_cast<uint4*>(at) = __builtin_bit_cast(uint4, hi);
  *reinterpret_cast<uint4*>(at + 64) = __builtin_bit_cast(uint4, lo);
}

__device__ __forceinline__ v4f load_pairs(const uint8_t* row, int64_t k) {
  const uint8_t* at = row + pair_at(k);
  typedef _Float16 v4h __attribute__((ext_vector_type(4)));
  const v4h hi = load_unwritten<v4h>(at), lo = load_unwritten<v4h>(at + 64);
  return __builtin_convertvector(hi, v4f) + __builtin_convertvector(lo, v4f);
}

// Eight, from a multiple of 8.
typedef float v8f __attribute__((ext_vector_type(8)));
__device__ __forceinline__ v8f load_pairs8(const uint8_t* row, int64_t k) {
  const uint8_t* at = row + pair_at(k);
  const nt::v8h hi = load_unwritten<nt::v8h>(at), lo = load_unwritten<nt::v8h>(at + 64);
  return __builtin_convertvector(hi, v8f) + __builtin_convertvector(lo, v8f);
}

struct Source {
  const void* g;
  int64_t ld, batch;
  int rows, cols;
};

// The sum of v over a block of 256 threads, in a fixed order; s is not in use.
__device__ __forceinline__ double block_sum(double v, double (&s)[4]) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  if (threadIdx.x % 64 == 0) s[threadIdx.x / 64] = v;
  __syncthreads();
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// The sums of squares of a matrix's parts, in doubles, and of each row within a
// part's columns, and each column within its rows, the largest magnitude's upper
// sixteen bits, rounded up (as integers they order like the values, infinities and
// NaNs above; all of the latter become 0x7f81).
struct Lines {
  double* sum;                  // [batch][parts_r][parts_c]
  uint16_t *row_top, *col_top;  // [batch][parts_c][rows], [batch][parts_r][cols]
  int parts_r, parts_c, span_r, span_c;
};
__device__ __forceinline__ uint16_t top16(uint32_t top) { return static_cast<uint16_t>(min((top + 0xffffu) >> 16, 0x7f81u)); }

// No atomics, so the same sums every time.  Bound by memory: 4096 x 4096 floats in
// 16.6 us, 4.0 TB/s (13.6 for the sums alone); 256 x 256 in 3.8.
template <class T>
__global__ __launch_bounds__(256) void k_norm(Source src, Lines lines) {
  __shared__ uint32_t col_top[8][256];
  const T* g = static_cast<const T*>(src.g) + blockIdx.y * src.batch;
  const int pr = blockIdx.x / lines.parts_c, pc = blockIdx.x % lines.parts_c;
  const int row0 = pr * lines.span_r, rows = min(lines.span_r, src.rows - row0);
  const int col0 = pc * lines.span_c, cols = min(lines.span_c, src.cols - col0);
  const int lane = threadIdx.x % 32, rg = threadIdx.x / 32;
  uint16_t* const to_rows = lines.row_top + (int64_t(blockIdx.y) * lines.parts_c + pc) * src.rows + row0;
  uint16_t* const to_cols = lines.col_top + (int64_t(blockIdx.y) * lines.parts_r + pr) * src.cols + col0;
  double sum = 0;
  for (int c0 = 0; c0 < cols; c0 += 256) {
    const int c = c0 + lane * 8, have = cols - c;  // this thread's columns
    uint32_t ctop[8] = {};
    for (int r0 = 0; r0 < rows; r0 += kNormRows) {
      constexpr int kEach = kNormRows / 8;
      Pack<8, T> v[kEach];
#pragma unroll
      for (int p = 0; p < kEach; ++p) {
        const int r = r0 + 8 * p + rg;
        const T* from = g + (row0 + r) * src.ld + col0 + c;
        v[p] = Pack<8, T>{};
        if (r < rows && have >= 8) {
          v[p] = load_pack<8>(from);
        } else if (r < rows) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < have) v[p].v[i] = from[i];
        }
      }
#pragma unroll
      for (int p = 0; p < kEach; ++p) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float f = to_float(v[p].v[i]);
          const uint32_t m = magnitude(f);
          const double x = f;
          sum = fma(x, x, sum);
          top = max(top, m);
          ctop[i] = max(ctop[i], m);
        }
        top = max16(top);
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16)));
        const int r = r0 + 8 * p + rg;  // always this half wavefront's
        if (lane == 0 && r < rows) to_rows[r] = c0 ? max(to_rows[r], top16(top)) : top16(top);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) col_top[rg][lane * 8 + i] = ctop[i];
    __syncthreads();
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, col_top[i][threadIdx.x]);
    if (c0 + static_cast<int>(threadIdx.x) < cols) to_cols[c0 + threadIdx.x] = top16(top);
    __syncthreads();
  }
  __shared__ double s[4];
  sum = block_sum(sum, s);
  if (threadIdx.x == 0) lines.sum[int64_t(blockIdx.y) * gridDim.x + blockIdx.x] = sum;
}

// 1 / (|G|_F + eps) from the parts; all threads of a 256-thread block call it.  In
// double, and x times it too: the norm of finite floats can pass a float's largest
// number or lie below its normal ones.
__device__ __forceinline__ double factor(const Lines& lines, float eps, double (&s)[4]) {
  const int parts = lines.parts_r * lines.parts_c;
  double sum = 0;
#pragma unroll 4
  for (int p = threadIdx.x; p < parts; p += 256) sum += lines.sum[int64_t(blockIdx.y) * parts + p];
  return 1.0 / (sqrt(block_sum(sum, s)) + eps);
}

// 2^e of an exponent within a float's normal ones.
__device__ __forceinline__ float power(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// The exponent of a row's or column's root: half its norm's, p at the start and
// `grown` more by now, rounded up, at most 0.
__device__ __forceinline__ int root(int p, int grown) { return min((p + grown + 1) >> 1, 0); }

// The largest of a line's parts, `stride` apart, that this wavefront of four takes.
__device__ __forceinline__ uint32_t top_of(const uint16_t* from, int64_t stride, int parts, int wave) {
  uint32_t top = 0;
  for (int p0 = wave; p0 < parts; p0 += 32) {
    uint32_t v[8];  // together: one trip to memory
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int p = min(p0 + 4 * i, parts - 1);
      v[i] = from[p * stride];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, v[i]);
  }
  return top;
}

// An exponent e with n elements of at most `top` times `by` below 2^e in the 2-norm;
// root_n: sqrt(n).
__device__ __forceinline__ int norm_exponent(uint32_t top, double by, double root_n) {
  const double v = __uint_as_float(top << 16) * by * root_n;
  if (!(v < 1.0)) return 0;  // NaN among them: all is lost anyway
  return v > 0.0 ? max(__builtin_amdgcn_frexp_exp(v), kLeastExponent) : kLeastExponent;
}

// X_0 as pairs, as G lies (`direct`: rows of G) and transposed (`across`), a
// 64 x 64 tile a block through LDS; both padded with zeros.  The one that is X^
// (across for a tall G) is divided by its rows' roots, the one that is X~^T by both
// sides'.  The first tiles of a row or column leave its exponent for what follows.
// Bound by memory: 4096 x 4096 floats, 192 MiB, in 37 us (5.4 TB/s; 46 with the
// tops' parts loaded one after the other), 256 x 256 in 6.3.
template <class T>
__global__ __launch_bounds__(256) void k_start(Source src, Lines lines, float eps, float scale, Pairs direct, Pairs across,
                                               int* row_exponent, int* col_exponent, int64_t row_batch, int64_t col_batch,
                                               double root_rows, double root_cols, int tiles_c) {
  __shared__ double s[4];
  __shared__ float t[64][65];
  __shared__ uint32_t top[2][4][64];
  __shared__ float line[2][64];  // 1 / root of the rows, of the columns
  const T* g = static_cast<const T*>(src.g) + blockIdx.y * src.batch;
  const int r0 = blockIdx.x / tiles_c * 64, c0 = blockIdx.x % tiles_c * 64;
  const int at = threadIdx.x % 64, wave = threadIdx.x / 64;
  T x[16];  // under way while the norm's parts are added
#pragma unroll
  for (int p = 0; p < 16; ++p) {
    const int r = p * 4 + wave, c = at;
    x[p] = T{};
    if (r0 + r < src.rows && c0 + c < src.cols) x[p] = g[(r0 + r) * src.ld + c0 + c];
  }
  const int row = min(r0 + at, src.rows - 1), col = min(c0 + at, src.cols - 1);
  top[0][wave][at] = top_of(lines.row_top + int64_t(blockIdx.y) * lines.parts_c * src.rows + row, src.rows, lines.parts_c, wave);
  top[1][wave][at] = top_of(lines.col_top + int64_t(blockIdx.y) * lines.parts_r * src.cols + col, src.cols, lines.parts_r, wave);
  const double by = factor(lines, eps, s);  // which waits for all threads
  if (wave < 2) {
    const uint32_t most = max(max(top[wave][0][at], top[wave][1][at]), max(top[wave][2][at], top[wave][3][at]));
    const int e = norm_exponent(most, by, wave ? root_rows : root_cols);
    line[wave][at] = power(-root(e, 0));
    if (wave == 0 && c0 == 0 && r0 + at < src.rows) row_exponent[blockIdx.y * row_batch + r0 + at] = e;
    if (wave == 1 && r0 == 0 && c0 + at < src.cols) col_exponent[blockIdx.y * col_batch + c0 + at] = e;
  }
  __syncthreads();
  const bool tall = src.rows > src.cols;
  // x by in floats: a power of two first, which brings x near its place exactly (but
  // what lies 2^-126 below the norm), then what is left of the factor, rounded
  const double first = __builtin_amdgcn_ldexp(1.0, min(max(__builtin_amdgcn_frexp_exp(by), -120), 120));
  const float to_place = static_cast<float>(first), left = static_cast<float>(by / first) * scale;
#pragma unroll
  for (int p = 0; p < 16; ++p) {
    const int r = p * 4 + wave;
    t[r][at] = to_float(x[p]) * to_place * (left * (tall ? line[1][at] : line[0][r]));
  }
  __syncthreads();
  uint8_t* dp = direct.p + blockIdx.y * direct.batch;
  uint8_t* ap = across.p + blockIdx.y * across.batch;
  const int64_t dpad = pad32(src.cols), apad = pad32(src.rows);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int r = p * 16 + threadIdx.x / 16, c = threadIdx.x % 16 * 4;
    const float d = tall ? line[0][r] : 1.0f, a = tall ? 1.0f : line[1][r];
    if (r0 + r < src.rows && c0 + c < dpad)
      store_pairs(dp + (r0 + r) * direct.ld, c0 + c, v4f{t[r][c] * d, t[r][c + 1] * d, t[r][c + 2] * d, t[r][c + 3] * d});
    if (c0 + r < src.cols && r0 + c < apad)
      store_pairs(ap + (c0 + r) * across.ld, r0 + c, v4f{t[c][r] * a, t[c + 1][r] * a, t[c + 2][r] * a, t[c + 3][r] * a});
  }
}

// steps == 0: G / (|G|_F + eps).
template <class T>
__global__ __launch_bounds__(256) void k_divide(Source src, Lines lines, float eps, T* x, int64_t ldx, int64_t batch_x) {
  __shared__ double s[4];
  const double by = factor(lines, eps, s);
  const T* g = static_cast<const T*>(src.g) + blockIdx.y * src.batch;
  const int64_t items = int64_t(src.rows) * src.cols;
  for (int64_t it = int64_t(blockIdx.x) * 256 + threadIdx.x; it < items; it += int64_t(gridDim.x) * 256) {
    const int64_t r = it / src.cols, c = it % src.cols;
    from_float(static_cast<float>(to_float(g[r * src.ld + c]) * by), x[blockIdx.y * batch_x + r * ldx + c]);
  }
}

// The exponents of the norms of X_0's rows (or columns) and by how much they have
// grown.
struct Norms {
  const int* p;
  int64_t batch;
  int size, grown;
  __device__ __forceinline__ int at(int matrix, int line) const { return p[matrix * batch + min(line, size - 1)]; }
};

// What a tile's sums are multiplied by, of each of its rows and columns, in LDS: in
// a row-wise result and in a column-wise one.  The exponents are loaded before the
// sum, a line a thread, and become factors behind it.
template <int ROWS, int COLS>
struct alignas(16) Factors {
  static constexpr int kLines = ROWS + COLS;
  float row[ROWS], col[COLS], across[COLS];
};
template <int THREADS, int ROWS, int COLS>
struct Held {
  static constexpr int kEach = (ROWS + COLS + THREADS - 1) / THREADS;
  int e[kEach];
  template <class O>
  __device__ __forceinline__ Held(const O& out, int r0, int c0) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int l = threadIdx.x + i * THREADS;
      e[i] = l < ROWS ? out.row_norms().at(out.batch, r0 + l) : out.col_norms().at(out.batch, c0 + l - ROWS);
    }
  }
  template <class O>
  __device__ __forceinline__ void put(const O& out, Factors<ROWS, COLS>& f) const {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int l = threadIdx.x + i * THREADS;
      int x = e[i];
      asm volatile("" : "+v"(x));  // here, and not where it is loaded, is it waited for
      if (l < ROWS) {
        f.row[l] = out.by_row(x);
      } else if (l < ROWS + COLS) {
        f.col[l - ROWS] = out.by_col(x);
        f.across[l - ROWS] = out.by_col_across(x);
      }
    }
  }
};

// What becomes of the sums v of a symmetric m x m matrix at row r, column c: with
// the root d_c of row c of X
//   U:   scale v d_c
//   P~:  (scale v d_c + b U_rc) d_c, and `diagonal` on the diagonal
// written as pairs at its place and, off the diagonal tiles, at the mirrored one
// (with d_r, U_cr).  Both indexes run on past m to the padding, where zeros go.
struct SymmetricOut {
  Pairs out, add;  // add: U, for P~
  int m;
  float scale, b, diagonal;
  Norms rows;
  int batch;
  bool mirror;
  __device__ __forceinline__ const Norms& row_norms() const { return rows; }
  __device__ __forceinline__ const Norms& col_norms() const { return rows; }
  __device__ __forceinline__ float by_row(int e) const { return power(root(e, rows.grown)); }
  __device__ __forceinline__ float by_col(int e) const { return by_row(e); }
  __device__ __forceinline__ float by_col_across(int) const { return 0.0f; }
  __device__ __forceinline__ float value(float v, float old, float d) const {
    const float x = v * scale * d;
    return add.p ? fmaf(b, old, x) * d : x;
  }
  __device__ __forceinline__ float value(int r, int c, float v, float old, float d) const {
    return r < m && c < m ? value(v, old, d) + (r == c ? diagonal : 0.0f) : 0.0f;
  }
  // four neighbours of a row; dr, dc: the roots of row r and of columns c ..
  __device__ __forceinline__ void four(int r, int c, v4f v, float dr, v4f dc, v4f) const {
    if (r >= pad32(m) || c >= pad32(m)) return;
    uint8_t* base = out.p + batch * out.batch;
    const uint8_t* from = add.p + batch * add.batch;
    v4f old = {}, across = {};
    if (add.p) {
      old = load_pairs(from + min(r, m - 1) * add.ld, c);
      across = old;  // U_rc = U_cr where the roots are alike
      if (mirror && !(dr == dc[0] && dr == dc[1] && dr == dc[2] && dr == dc[3])) {
#pragma unroll
        for (int i = 0; i < 4; ++i) across[i] = load_pair(from + min(c + i, m - 1) * add.ld, r);
      }
    }
    if (r < m) {
      v4f x;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = value(r, c + i, v[i], old[i], dc[i]);
      store_pairs(base + r * out.ld, c, x);
    }
    if (mirror) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < m) store_pair(base + (c + i) * out.ld, r, value(c + i, r, v[i], across[i], dr));
    }
  }
  // eight neighbours of row r, wherever their sums lay (past m these are 0: the large
  // tiles read zeros there); d: their roots
  __device__ __forceinline__ void eight(int r, int c, const float (&v)[8], const float* d) const {
    if (r >= m || c >= pad32(m)) return;
    v8f old = {};
    if (add.p) old = load_pairs8(add.p + batch * add.batch + r * add.ld, c);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = value(v[i], old[i], d[i]);
    if (!mirror) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] += r == c + i ? diagonal : 0.0f;
    }
    store_pairs8(out.p + batch * out.batch + r * out.ld, c, x);
  }
  // 64 rows of a tile, from row r0 and column c0
  template <int THREADS, int COLS>
  __device__ __forceinline__ void sheet(nt::Sheet<COLS>& s, int r0, int c0, const float* dr, const float* dc,
                                        const float*) const {
    s.template out<THREADS>(mirror, [&](int r, int c, const float (&v)[8]) { eight(r0 + r, c0 + c, v, dc + c); },
                            [&](int c, int r, const float (&v)[8]) { eight(c0 + c, r0 + r, v, dr + r); });
  }
};

// P~ X~ = D^-1 X' E^-1: as pairs X^' and X~'^T under the roots of the next step, or
// at the last step as the result X'.
template <class T>
struct IterateOut {
  Pairs x, xt;
  T* out;  // not NULL at the last step
  int64_t ldo, batch_o;
  int m, n;
  float scale;  // the sums' scale to the next step's, or to 1
  Norms rows, cols;
  int next;  // `grown` of the next step
  int batch;
  bool tall;
  __device__ __forceinline__ const Norms& row_norms() const { return rows; }
  __device__ __forceinline__ const Norms& col_norms() const { return cols; }
  // D over the next step's (over 1 for the result); E, and for X~' over the next step's
  __device__ __forceinline__ float by_row(int e) const {
    return power(root(e, rows.grown) - (out ? 0 : root(e, next))) * scale;
  }
  __device__ __forceinline__ float by_col(int e) const { return power(root(e, cols.grown)); }
  __device__ __forceinline__ float by_col_across(int e) const {
    return power(root(e, cols.grown) - (out ? 0 : root(e, next)));
  }
  // four neighbours of a row; d, e, f: the factors of row r, of columns c .. in X^', in X~'
  __device__ __forceinline__ void four(int r, int c, v4f v, float d, v4f e, v4f f) const {
    if (r >= pad32(m) || c >= pad32(n)) return;
    v4f y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = r < m && c + i < n ? v[i] * d : 0.0f;
    if (out) {
      if (r >= m) return;
      T* o = out + batch * batch_o;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < n) from_float(y[i] * e[i], tall ? o[(c + i) * ldo + r] : o[r * ldo + c + i]);
    } else {
      uint8_t* t = xt.p + batch * xt.batch;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < n) store_pair(t + (c + i) * xt.ld, r, y[i] * f[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] *= e[i];
      if (r < m) store_pairs(x.p + batch * x.batch + r * x.ld, c, y);
    }
  }
  // `count` of eight neighbours of the result, from `at`
  __device__ __forceinline__ void result(T* at, int count, const float (&v)[8]) const {
    Pack<8, T> p;
#pragma unroll
    for (int i = 0; i < 8; ++i) from_float(v[i], p.v[i]);
    if (count >= 8) {
      store_pack(at, p);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < count) at[i] = p.v[i];
    }
  }
  template <int THREADS, int COLS>
  __device__ __forceinline__ void sheet(nt::Sheet<COLS>& s, int r0, int c0, const float* d, const float* e,
                                        const float* f) const {
    T* o = out + batch * batch_o;
    uint8_t *xp = x.p + batch * x.batch, *tp = xt.p + batch * xt.batch;
    s.template out<THREADS>(
        !out || tall,
        [&](int r, int c, const float (&v)[8]) {
          const int row = r0 + r, col = c0 + c;
          if (row >= m || col >= (out ? n : pad32(n)) || (out && tall)) return;
          const float k = d[r];
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = v[i] * k * e[c + i];  // past n: 0, as the sums there
          if (out) result(o + row * ldo + col, n - col, y);
          else store_pairs8(xp + row * x.ld, col, y);
        },
        [&](int c, int r, const float (&v)[8]) {
          const int row = r0 + r, col = c0 + c;
          if (col >= n || row >= (out ? m : pad32(m))) return;
          const float k = f[c];
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = v[i] * k * d[r + i];
          if (out) result(o + col * ldo + row, m - row, y);
          else store_pairs8(tp + col * xt.ld, row, y);
        });
  }
};

// The lower triangle's tiles, row by row.
__device__ __forceinline__ nt::Place triangle(int id) {
  int i = static_cast<int>((sqrtf(8.0f * id + 1.0f) - 1.0f) * 0.5f);
  while ((i + 1) * (i + 2) / 2 <= id) ++i;
  while (i * (i + 1) / 2 > id) --i;
  return nt::Place{i, id - i * (i + 1) / 2};
}

// Small tiles, K split over the wavefronts.
template <int T>
struct Small : nt::Direct<nt::HalfPair, T, T, 8> {
  static constexpr bool kDirect = true;
  static constexpr int kMinWaves = 2;
};
// Large ones, with their loop in assembly; LDS holds one block a CU, so of four
// wavefronts one a SIMD, of eight two.
template <int MT, int NT, int WM, int WN, int STAGES>
struct Assembled : nt::Loop<nt::Kind::kPair, MT, NT, WM, WN, STAGES> {
  static constexpr bool kDirect = false;
  static constexpr int kMinWaves = WM * WN / 4;
};

template <class T, class E>
__device__ __forceinline__ void product(const Side& A, const Side& B, int m0, int n0, int K, const E& epi) {
  __shared__ Factors<T::BM, T::BN> by;
  const Held<T::threads, T::BM, T::BN> held(epi, m0, n0);
  if constexpr (T::kDirect) {
    __shared__ typename T::Meet meet;
    T::run(meet, A, B, m0, n0, K * 4,
           [&](int r, int c, v4f v) {
             float d = by.row[r - m0];
             v4f e = *reinterpret_cast<const v4f*>(&by.col[c - n0]), f = *reinterpret_cast<const v4f*>(&by.across[c - n0]);
             asm volatile("" : "+v"(d), "+v"(e), "+v"(f));  // read together, not one by one where they are used
             epi.four(r, c, v, d, e, f);
           },
           [&] { held.put(epi, by); });
  } else {
    __shared__ alignas(16) uint8_t smem[T::kLds];
    nt::v16f acc[T::kAcc];
    nt::loop_sum<T>(smem, A, B, m0, n0, K * 4, acc);
    held.put(epi, by);
    using Sheet = nt::Sheet<T::BN>;
    static_assert(sizeof(Sheet) <= T::kLds, "a sheet fits");
    Sheet& sheet = *reinterpret_cast<Sheet*>(smem);
    __syncthreads();  // all wavefronts have left the loop
    nt::loop_sheets<T>(sheet, acc, [&](int top) {
      epi.template sheet<T::threads>(sheet, m0 + top, n0, by.row + top, by.col, by.across);
    });
  }
}

// S = X X^T and P = a + b S + c S S: the lower tiles, mirrored.  Bound by the
// matrix rate where the tiles fill the CUs: 4096 x 4096 in 174-187 us on 253 tiles
// of 192 x 192 (136 of 256 x 256 would leave half the CUs idle), MfmaUtil 65 %; by
// the latency of one trip to memory where they are few: 256 x 256 in 4.4-5.0 us.
template <class T>
__global__ __launch_bounds__(T::threads, T::kMinWaves) void k_symmetric(Side A, int K, SymmetricOut out) {
  out.batch = blockIdx.y;
  A.p += blockIdx.y * A.batch;
  const nt::Place at = triangle(static_cast<int>(xcd_contiguous(blockIdx.x, gridDim.x)));
  out.mirror = at.tm != at.tn;
  product<T>(A, A, at.tm * T::BM, at.tn * T::BN, K, out);
}

// X' = P X.  Bound by the matrix rate: 4096 x 4096 in 281-292 us on 256 tiles of
// 256 x 256, 1440 TFLOP/s of half products, MfmaUtil 75 %; 1024 x 1024 x 4096 in
// 29 us on 256 tiles of 128 x 128, whose 32 steps hardly outlast the first loads
// and the results' way out.
template <class T, class O>
__global__ __launch_bounds__(T::threads, T::kMinWaves) void k_iterate(Side A, Side B, int K, IterateOut<O> out,
                                                                      int col0, int tiles_m, int tiles_n) {
  out.batch = blockIdx.y;
  A.p += blockIdx.y * A.batch;
  B.p += blockIdx.y * B.batch;
  const nt::Place at = nt::place_of(xcd_contiguous(blockIdx.x, gridDim.x), tiles_m, tiles_n, 8);
  product<T>(A, B, at.tm * T::BM, col0 + at.tn * T::BN, K, out);
}

// One of `splits` parts of the K of a symmetric product's tiles: the sums as the
// wavefronts hold them, 16 bytes a lane side by side.  For where the tiles are
// far fewer than the CUs: S of 1024 x 4097 in 17.2 us on 36 tiles by 7 parts, with
// 5.6 us for the parts' sum, against about 80 us on 36 blocks.
template <class T>
__global__ __launch_bounds__(T::threads, T::kMinWaves) void k_partial(Side A, int K, float* sums, int tiles, int splits) {
  __shared__ alignas(16) uint8_t smem[T::kLds];
  const int64_t id = xcd_contiguous(blockIdx.x, gridDim.x);  // an XCD's blocks share a part of K
  const int tile = static_cast<int>(id % tiles), part = static_cast<int>(id / tiles), steps = K / 32;
  const int k0 = static_cast<int>(int64_t(steps) * part / splits), k1 = static_cast<int>(int64_t(steps) * (part + 1) / splits);
  const nt::Place at = triangle(tile);
  A.p += blockIdx.y * A.batch + int64_t(k0) * nt::kStep;
  nt::v16f acc[T::kAcc];
  nt::loop_sum<T>(smem, A, A, at.tm * T::BM, at.tn * T::BN, (k1 - k0) * nt::kStep, acc);
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  float* to = sums + ((int64_t(blockIdx.y) * splits + part) * tiles + tile) * (T::BM * T::BN) + wave * (T::MT * T::NT * 256) + lane * 4;
#pragma unroll
  for (int f = 0; f < T::MT * T::NT; ++f)
#pragma unroll
    for (int r = 0; r < 4; ++r) to[f * 256 + r] = acc[f / 4][f % 4 * 4 + r];
}

// The parts added in their order, a wavefront's share of a tile a block.
template <class T>
__global__ __launch_bounds__(256) void k_finish(const float* sums, int tiles, int splits, SymmetricOut out) {
  static_assert(T::MT == 4 && T::NT == 2, "a sheet of 64 rows, two fragments each of four wavefronts");
  __shared__ nt::Sheet<16 * T::NT> sheet;
  __shared__ Factors<64, 16 * T::NT> by;
  const int tile = blockIdx.x / T::waves, share = blockIdx.x % T::waves, lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const nt::Place at = triangle(tile);
  out.batch = blockIdx.y;
  out.mirror = at.tm != at.tn;
  const int r0 = at.tm * T::BM + share % T::WM * 64, c0 = at.tn * T::BN + share / T::WM * 16 * T::NT;
  const Held<256, 64, 16 * T::NT> held(out, r0, c0);
  const float* from = sums + (int64_t(blockIdx.y) * splits * tiles + tile) * (T::BM * T::BN) + share * (T::MT * T::NT * 256) + wave * 512 + lane * 4;
  v4f v[2] = {};
#pragma unroll 4
  for (int p = 0; p < splits; ++p) {
    const float* at_p = from + int64_t(p) * tiles * (T::BM * T::BN);
    v[0] += *reinterpret_cast<const v4f*>(at_p);
    v[1] += *reinterpret_cast<const v4f*>(at_p + 256);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int f = 2 * wave + i;  // fragment j MT + i of the wavefront
    sheet.put(f % T::MT * 16 + lane % 16, f / T::MT * 16 + 4 * (lane / 16), v[i]);
  }
  held.put(out, by);
  out.sheet<256>(sheet, r0, c0, by.row, by.col, by.across);
}

// Which tile takes the products of `batch` matrices, by estimates of the time in
// us: of the small ones what a launch, a step of a wavefront alone and a step of
// one block among many take; of the large ones what a step takes alone and with
// all 256 CUs at it.  Measured from 256 x 256 to 4096 x 4096, which they meet
// within a quarter.
enum class Way { kSmall32, kSmall64, kLoop128, kLoop192, kLoop256, kSplit, kColumns };
struct Choice {
  Way way;
  int at;  // kSplit: parts of K; kColumns: where the result is cut in two
  double us;
};
constexpr int kMaxParts = 16;

Choice choose(int batch, int rows, int cols, int K, bool symmetric, bool cut) {
  const double steps = K / 32, each = static_cast<double>(ceil_div(K / 32, 8));
  const auto tiles_of = [&](int t) {
    const int64_t tm = ceil_div(rows, t), tn = ceil_div(cols, t);
    return batch * (symmetric ? tm * (tm + 1) / 2 : tm * tn);
  };
  Choice best{Way::kSmall32, 0, 1e30};
  const auto offer = [&](Way w, int at, double us) {
    if (us < best.us) best = Choice{w, at, us};
  };
  const auto small = [&](Way w, int t, double base, double alone, double among) {
    const double blocks = static_cast<double>(tiles_of(t));
    offer(w, 0, base + each * (alone > among * blocks ? alone : among * blocks));
  };
  const auto loop = [&](Way w, int t, double base, double alone, double full) {
    const int64_t tiles = tiles_of(t), rest = tiles % 256;
    offer(w, 0, base + steps * (tiles / 256 * full + (rest ? alone + (full - alone) * rest / 256 : 0)));
  };
  small(Way::kSmall32, 32, 2.5, 1.4, 0.0085);
  small(Way::kSmall64, 64, 3.0, 3.4, 0.018);
  loop(Way::kLoop128, 128, 5.0, 0.45, 0.65);
  loop(Way::kLoop192, 192, 8.0, 1.0, 1.35);
  loop(Way::kLoop256, 256, 10.0, 1.45, 2.3);
  if (symmetric) {
    const int64_t tiles = tiles_of(128);
    const int64_t most = steps / 2 < kMaxParts ? static_cast<int64_t>(steps / 2) : kMaxParts;
    // a part's sums are written and read, and there is a second launch
    for (int64_t parts = 2; parts <= most && parts * tiles <= 256; ++parts)
      offer(Way::kSplit, static_cast<int>(parts), 8.0 + static_cast<double>(ceil_div(K / 32, parts)) * 0.6 + 0.025 * tiles * parts);
  }
  for (int t = 128; cut && !symmetric && t <= 256; t += 64)  // columns that hardly fill their tiles apart from the rest
    if (cols > t && cols % t) {
      const int at = cols - cols % t;
      offer(Way::kColumns, at, choose(batch, rows, at, K, false, false).us + choose(batch, rows, cols - at, K, false, false).us);
    }
  return best;
}

// A step's three products: S and P, which are alike at every step, and P X, whose
// columns from `cut` on (0: none) may have a launch of their own.
struct Plan {
  Choice s, p, x;
  int cut;
  Way rest;
};

Plan plan(int batch, int m, int n) {
  const int km = static_cast<int>(pad32(m)), kn = static_cast<int>(pad32(n));
  Plan l;
  l.s = choose(batch, m, m, kn, true, false);
  l.p = choose(batch, m, m, km, true, false);
  l.x = choose(batch, m, n, km, false, true);
  l.cut = 0;
  l.rest = Way::kSmall32;
  if (l.x.way == Way::kColumns) {
    l.cut = l.x.at;
    l.rest = choose(batch, m, n - l.cut, km, false, false).way;
    l.x = choose(batch, m, l.cut, km, false, false);
  }
  return l;
}

int tile_of(Way way) {
  switch (way) {
    case Way::kSmall32: return 32;
    case Way::kSmall64: return 64;
    case Way::kLoop192: return 192;
    case Way::kLoop256: return 256;
    default: return 128;
  }
}

using Loop128 = Assembled<4, 2, 2, 4, 4>;

// Calls f with the tile.
template <class F>
void with_tile(Way way, const F& f) {
  switch (way) {
    case Way::kSmall32: return f(Small<2>{});
    case Way::kSmall64: return f(Small<4>{});
    case Way::kLoop128: return f(Loop128{});
    case Way::kLoop192: return f(Assembled<6, 6, 2, 2, 3>{});
    default: return f(Assembled<8, 4, 2, 4, 2>{});
  }
}

// The workspace: parts of the norms, the rows' and columns' exponents, then X^, X~^T
// twice, U and P~, and the parts of the symmetric products' sums.
struct Layout {
  int m, n, parts_r, parts_c, span_r, span_c;
  int64_t sum, row_top, col_top, p, q, x, xt[2], s, ps, sums, bytes;
  int64_t ldx, ldm;  // bytes of a row of X^, and of the others
  int64_t lm, ln;    // exponents of a matrix
};

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

Layout layout_of(int batch, int rows, int cols) {
  Layout l;
  l.m = rows < cols ? rows : cols;
  l.n = rows < cols ? cols : rows;
  l.ldx = pad32(l.n) * 4;
  l.ldm = pad32(l.m) * 4;
  const auto split = [](int size, int unit, int most, int& span) {
    span = static_cast<int>(ceil_div(ceil_div(size, unit), most)) * unit;
    return static_cast<int>(ceil_div(size, span > 0 ? span : unit));
  };
  const auto rows_of = [&](int size, int parts_c, int& span) {
    const int most = parts_c > 0 ? kNormBlocks / parts_c : kMaxRowParts;  // 16 to 1024
    return split(size, kNormRows, most < kMaxRowParts ? most : kMaxRowParts, span);
  };
  l.parts_c = split(cols, 256, kMaxColParts, l.span_c);
  l.parts_r = rows_of(rows, l.parts_c, l.span_r);
  // as many bytes for G as for its transpose
  int across_span;
  const int across_c = split(rows, 256, kMaxColParts, across_span), across_r = rows_of(cols, across_c, across_span);
  const auto most = [](int64_t a, int64_t b) { return a > b ? a : b; };
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += up256(bytes);
    return here;
  };
  l.sum = take(batch * most(l.parts_r * l.parts_c, across_r * across_c) * 8);
  l.row_top = take(batch * most(int64_t(l.parts_c) * rows, int64_t(across_c) * cols) * 2);
  l.col_top = take(batch * most(int64_t(l.parts_r) * cols, int64_t(across_r) * rows) * 2);
  l.lm = up256(l.m);
  l.ln = up256(l.n);
  l.p = take(batch * l.lm * 4);
  l.q = take(batch * l.ln * 4);
  l.x = take(batch * (l.m * l.ldx));
  l.xt[0] = take(batch * (l.n * l.ldm));
  l.xt[1] = take(batch * (l.n * l.ldm));
  l.s = take(batch * (l.m * l.ldm));
  l.ps = take(batch * (l.m * l.ldm));
  const int64_t t = ceil_div(l.m, Loop128::BM), tiles = batch * (t * (t + 1) / 2);
  l.sums = take(tiles > 0 && tiles <= 128 ? (256 / tiles < kMaxParts ? 256 / tiles : kMaxParts) * tiles * (Loop128::BM * Loop128::BN * 4) : 0);
  l.bytes = at;
  return l;
}

// What bounds a step's matrices, from the polynomials a + b x + c x^2 so far: the
// largest singular value is at most `sigma`, and norms have grown by 2^grown at most.
struct Step {
  float x, s, p;  // the scales of X^ and X~, U, P~
  int grown;
};

// The largest power of two that keeps numbers up to `bound`, with some room for
// rounding, within a half.
float scale_for(double bound) {
  if (!(bound < 0x1p60)) return 0x1p-60f;
  return static_cast<float>(std::exp2(std::floor(std::log2(61000.0 / std::fmax(bound, 1.0)))));
}

// steps + 1 of them; the last one for what a next step would find.
void schedule(int steps, const float* co, Step* out) {
  double sigma = 1.0, grown = 0.0;
  for (int i = 0; i <= steps; ++i) {
    const double most = std::fmax(sigma, 1.0), square = most * most;
    // |X^|, |X~| <= most; |U| = |S| over a row's root <= most^2, |U U^T| <= most^4
    const double a = i < steps ? co[3 * i] : 0, b = i < steps ? co[3 * i + 1] : 0, c = i < steps ? co[3 * i + 2] : 0;
    out[i].x = scale_for(most);
    out[i].s = scale_for(square);
    out[i].p = scale_for(std::fabs(a) + std::fabs(b) * square + std::fabs(c) * square * square);
    out[i].grown = grown < 1000 ? static_cast<int>(std::ceil(grown)) : 1000;
    // the largest |p(x)| and sqrt(x) |p(x)| over 0 <= x <= sigma^2: at the ends or where they are flat
    const auto poly = [&](double x) { return std::fabs(a + b * x + c * x * x); };
    const double end = sigma * sigma;
    double grow = std::fmax(poly(0), poly(end)), next = sigma * poly(end);
    const auto flat = [&](double x, bool root) {
      if (!(x > 0 && x < end)) return;
      if (root) next = std::fmax(next, std::sqrt(x) * poly(x));
      else grow = std::fmax(grow, poly(x));
    };
    if (c != 0) flat(-b / (2 * c), false);
    const double disc = 9 * b * b - 20 * a * c;  // of a + 3 b x + 5 c x^2
    if (c != 0 && disc >= 0) {
      flat((-3 * b + std::sqrt(disc)) / (10 * c), true);
      flat((-3 * b - std::sqrt(disc)) / (10 * c), true);
    } else if (c == 0 && b != 0) {
      flat(-a / (3 * b), true);
    }
    if (grow > 1) grown += std::log2(grow);
    sigma = next;
  }
}

int check_sizes(int batch, int rows, int cols, int type) {
  if (batch < 0 || batch > 65535) return -1;
  if (rows < 0 || rows > HIP_ORTHOGONAL_MAX_SIZE) return -2;
  if (cols < 0 || cols > HIP_ORTHOGONAL_MAX_SIZE) return -3;
  if (type != HIP_ORTHOGONAL_F32 && type != HIP_ORTHOGONAL_BF16 && type != HIP_ORTHOGONAL_F16) return -4;
  return 0;
}

template <class T>
hipError_t launch(int batch, const Source& src, int steps, const float* co, float eps, T* x, int64_t ldx,
                  int64_t batch_x, uint8_t* ws, hipStream_t stream) {
  const Layout l = layout_of(batch, src.rows, src.cols);
  const Lines lines{reinterpret_cast<double*>(ws + l.sum), reinterpret_cast<uint16_t*>(ws + l.row_top),
                    reinterpret_cast<uint16_t*>(ws + l.col_top), l.parts_r, l.parts_c, l.span_r, l.span_c};
  hipLaunchKernelGGL((k_norm<T>), dim3(l.parts_r * l.parts_c, batch), dim3(256), 0, stream, src, lines);
  if (steps == 0) {
    const int64_t blocks = ceil_div(int64_t(src.rows) * src.cols, 256);
    hipLaunchKernelGGL((k_divide<T>), dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096), batch), dim3(256), 0,
                       stream, src, lines, eps, x, ldx, batch_x);
    return hipGetLastError();
  }
  const bool tall = src.rows > src.cols;
  const Pairs X{ws + l.x, l.ldx, l.m * l.ldx};
  Pairs XT{ws + l.xt[0], l.ldm, l.n * l.ldm}, XT2{ws + l.xt[1], l.ldm, l.n * l.ldm};
  const Pairs S{ws + l.s, l.ldm, l.m * l.ldm}, P{ws + l.ps, l.ldm, l.m * l.ldm};
  int *const p = reinterpret_cast<int*>(ws + l.p), *const q = reinterpret_cast<int*>(ws + l.q);
  Step step[HIP_ORTHOGONAL_MAX_STEPS + 1];
  schedule(steps, co, step);
  // 64-wide tiles: both paddings (to 32) lie inside them
  const int64_t tr = ceil_div(src.rows, 64), tc = ceil_div(src.cols, 64);
  hipLaunchKernelGGL((k_start<T>), dim3(static_cast<unsigned>(tr * tc), batch), dim3(256), 0, stream, src, lines, eps,
                     step[0].x, tall ? XT : X, tall ? X : XT, tall ? q : p, tall ? p : q, tall ? l.ln : l.lm,
                     tall ? l.lm : l.ln, std::sqrt(static_cast<double>(src.rows)), std::sqrt(static_cast<double>(src.cols)),
                     static_cast<int>(tc));
  const auto side = [](const Pairs& p, int rows) { return Side{p.p, p.ld, rows, nullptr, 0, 0, 0, p.batch}; };
  const int km = static_cast<int>(pad32(l.m)), kn = static_cast<int>(pad32(l.n));
  const Plan choice = plan(batch, l.m, l.n);
  const auto symmetric = [&](const Choice& c, const Side& a, int K, const SymmetricOut& out) {
    if (c.way == Way::kSplit) {
      const int t = static_cast<int>(ceil_div(l.m, Loop128::BM)), tiles = t * (t + 1) / 2;
      float* sums = reinterpret_cast<float*>(ws + l.sums);
      hipLaunchKernelGGL((k_partial<Loop128>), dim3(tiles * c.at, batch), dim3(Loop128::threads), 0, stream, a, K, sums, tiles, c.at);
      hipLaunchKernelGGL((k_finish<Loop128>), dim3(tiles * Loop128::waves, batch), dim3(256), 0, stream, sums, tiles, c.at, out);
      return;
    }
    with_tile(c.way, [&](auto tile) {
      using Tile = decltype(tile);
      const unsigned t = static_cast<unsigned>(ceil_div(l.m, Tile::BM));
      hipLaunchKernelGGL((k_symmetric<Tile>), dim3(t * (t + 1) / 2, batch), dim3(Tile::threads), 0, stream, a, K, out);
    });
  };
  // columns col0 .. col0 + cols - 1 of P X
  const auto iterate = [&](const Side& p, const Side& xt, int col0, int cols, Way way, const IterateOut<T>& out) {
    with_tile(way, [&](auto tile) {
      using Tile = decltype(tile);
      const unsigned tm = static_cast<unsigned>(ceil_div(l.m, Tile::BM)), tn = static_cast<unsigned>(ceil_div(cols, Tile::BN));
      hipLaunchKernelGGL((k_iterate<Tile, T>), dim3(tm * tn, batch), dim3(Tile::threads), 0, stream, p, xt, km, out, col0,
                         static_cast<int>(tm), static_cast<int>(tn));
    });
  };
  for (int i = 0; i < steps; ++i) {
    const float a = co[3 * i], b = co[3 * i + 1], c = co[3 * i + 2];
    const Step &now = step[i], &next = step[i + 1];
    const Norms rows{p, l.lm, l.m, now.grown}, cols{q, l.ln, l.n, now.grown};
    symmetric(choice.s, side(X, l.m), kn,
              SymmetricOut{S, Pairs{nullptr, 0, 0}, l.m, now.s / (now.x * now.x), 0.0f, 0.0f, rows, 0, false});
    symmetric(choice.p, side(S, l.m), km,
              SymmetricOut{P, S, l.m, c * (now.p / (now.s * now.s)), b * (now.p / now.s), a * now.p, rows, 0, false});
    const bool last = i + 1 == steps;
    const IterateOut<T> out{X, XT2, last ? x : nullptr, ldx, batch_x, l.m, l.n, (last ? 1.0f : next.x) / (now.p * now.x),
                            rows, cols, next.grown, 0, tall};
    iterate(side(P, l.m), side(XT, l.n), 0, choice.cut ? choice.cut : l.n, choice.x.way, out);
    if (choice.cut) iterate(side(P, l.m), side(XT, l.n), choice.cut, l.n - choice.cut, choice.rest, out);
    const Pairs t = XT;
    XT = XT2;
    XT2 = t;
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" {

int hip_orthogonalize_workspace(int batch, int rows, int cols, int type, long long* bytes) {
  const int bad = check_sizes(batch, rows, cols, type);
  if (bad) return bad;
  if (bytes) *bytes = layout_of(batch, rows, cols).bytes;
  return 0;
}

int hip_orthogonalize(int batch, int rows, int cols, int type, const void* G, int ldg, long long stride_g, int steps,
                      const float* coefficients, float eps, void* X, int ldx, long long stride_x, void* workspace,
                      long long workspace_bytes, hipStream_t stream) {
  const int bad = check_sizes(batch, rows, cols, type);
  if (bad) return bad;
  const bool some = batch > 0 && rows > 0 && cols > 0;
  if (some && G == nullptr) return -5;
  if (ldg < (cols > 1 ? cols : 1)) return -6;
  if (stride_g < 0) return -7;
  if (steps < 0 || steps > HIP_ORTHOGONAL_MAX_STEPS) return -8;
  if (some && steps > 0 && coefficients == nullptr) return -9;
  if (!(eps >= 0.0f)) return -10;
  if (some && X == nullptr) return -11;
  if (ldx < (cols > 1 ? cols : 1)) return -12;
  if (stride_x < 0 || (batch > 1 && stride_x < int64_t(rows) * ldx)) return -13;
  if (!some) return 0;
  if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return -14;
  if (workspace_bytes < layout_of(batch, rows, cols).bytes) return -15;
  const Source src{G, ldg, stride_g, rows, cols};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  hipError_t e;
  if (type == HIP_ORTHOGONAL_F32)
    e = launch(batch, src, steps, coefficients, eps, static_cast<float*>(X), ldx, stride_x, ws, stream);
  else if (type == HIP_ORTHOGONAL_BF16)
    e = launch(batch, src, steps, coefficients, eps, static_cast<bf16*>(X), ldx, stride_x, ws, stream);
  else
    e = launch(batch, src, steps, coefficients, eps, static_cast<_Float16*>(X), ldx, stride_x, ws, stream);
  return static_cast<int>(e);
}

int hip_orthogonalize_plan(int batch, int rows, int cols, hip_orthogonalize_product* products) {
  const int bad = check_sizes(batch, rows, cols, HIP_ORTHOGONAL_F32);
  if (bad) return bad;
  if (!products) return 0;
  for (int i = 0; i < 3; ++i) products[i] = hip_orthogonalize_product{0, 0, 0, 0};
  if (batch == 0 || rows == 0 || cols == 0) return 0;
  const Plan p = plan(batch, rows < cols ? rows : cols, rows < cols ? cols : rows);
  const auto product = [](const Choice& c) {
    return hip_orthogonalize_product{tile_of(c.way), c.way == Way::kSplit ? c.at : 1, 0, 0};
  };
  products[0] = product(p.s);
  products[1] = product(p.p);
  products[2] = product(p.x);
  products[2].cut = p.cut;
  products[2].cut_tile = p.cut ? tile_of(p.rest) : 0;
  return 0;
}

const char* hip_orthogonalize_status_string(int status) {
  switch (status) {
    case 0: return "success";
    case -1: return "argument 1 (batch) is negative or above 65535";
    case -2: return "argument 2 (rows) is negative or above HIP_ORTHOGONAL_MAX_SIZE";
    case -3: return "argument 3 (cols) is negative or above HIP_ORTHOGONAL_MAX_SIZE";
    case -4: return "argument 4 (type) is not a known type";
    case -5: return "argument 5 (G) is NULL";
    case -6: return "argument 6 (ldg) is smaller than max(1, cols)";
    case -7: return "argument 7 (stride_g) is negative";
    case -8: return "argument 8 (steps) is negative or above HIP_ORTHOGONAL_MAX_STEPS";
    case -9: return "argument 9 (coefficients) is NULL";
    case -10: return "argument 10 (eps) is negative or NaN";
    case -11: return "argument 11 (X) is NULL";
    case -12: return "argument 12 (ldx) is smaller than max(1, cols)";
    case -13: return "argument 13 (stride_x) is negative or lets the batch's matrices overlap";
    case -14: return "argument 14 (workspace) is NULL or not 256-byte aligned";
    case -15: return "argument 15 (workspace_bytes) is smaller than hip_orthogonalize_workspace says";
    default: break;
  }
  if (status > 0) return hipGetErrorString(static_cast<hipError_t>(status));
  return "unknown status";
}

}  // extern "C"

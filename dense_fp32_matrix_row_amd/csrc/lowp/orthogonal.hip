// orthogonal.hip -- hip_orthogonalize: Newton-Schulz products on the matrix
// cores with operands as pairs of halfs.
//
// A number x of the iterate is kept as hi + lo with halfs hi = RN(s x), lo =
// RN(s x - hi) for a fixed power of two s: 22 significant bits while |s x| is
// between 2^-3 and 65504, an absolute 2^-25 below (a half's least step is
// 2^-24).  That is 2^-37 of |X_0|_F = 1, whose elements are 2^-12 in the mean for
// 4096 x 4096.  The sums are float.  Three half products an element (hi hi',
// hi lo', lo hi') run at a third of the half rate, three times the float matrix
// rate (4096 x 4096: 443 TFLOP/s of the products asked for, against 150), and
// err no more than float products do.
//
// Per step, with m <= n the sides of the iterate X and X^T kept beside it, all
// operands have their K side contiguous:
//   S = X X^T               (m x m, K = n; symmetric: the lower tiles, mirrored)
//   P = a + b S + c S S     (m x m, K = m; S is its own transpose; symmetric)
//   X' = P X                (m x n, K = m; X^T is the other operand), written
//                           as X' over X, which is not read, and as X'^T into
//                           the other of two buffers.
#include "../../../include/orthogonal.h"
#include "lowp.h"
#include "nt_direct.h"
#include "nt_loop.h"

namespace sgemm {
namespace {

using nt::Side;
using nt::v4f;

constexpr float kScaleX = 0x1p12f;  // |X| < 16
constexpr float kScaleS = 0x1p8f;   // |S|, |P| < 255
constexpr int kNormBlocks = 1024;

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

// Four neighbours from k, a multiple of 4.
__device__ __forceinline__ void store_pairs(uint8_t* row, int64_t k, v4f v) {
  Pack<4, _Float16> hi, lo;
#pragma unroll
  for (int i = 0; i < 4; ++i) split(v[i], hi.v[i], lo.v[i]);
  uint8_t* at = row + pair_at(k);
  *reinterpret_cast<uint2*>(at) = __builtin_bit_cast(uint2, hi);
  *reinterpret_cast<uint2*>(at + 64) = __builtin_bit_cast(uint2, lo);
}

__device__ __forceinline__ v4f load_pairs(const uint8_t* row, int64_t k) {
  const uint8_t* at = row + pair_at(k);
  const auto hi = __builtin_bit_cast(Pack<4, _Float16>, *reinterpret_cast<const uint2*>(at));
  const auto lo = __builtin_bit_cast(Pack<4, _Float16>, *reinterpret_cast<const uint2*>(at + 64));
  v4f v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = static_cast<float>(hi.v[i]) + static_cast<float>(lo.v[i]);
  return v;
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

// The sum of squares of a matrix, in doubles: every block a part, in a fixed
// order (no atomics).  Bound by memory: 4096 x 4096 floats in 13.8 us, 4.9 TB/s.
template <class T>
__global__ __launch_bounds__(256) void k_norm(Source src, double* part, int parts) {
  const T* g = static_cast<const T*>(src.g) + blockIdx.y * src.batch;
  // sixteen neighbours a thread and turn
  const int groups = static_cast<int>(ceil_div(src.cols, 16));
  const int64_t items = int64_t(src.rows) * groups;
  double sum = 0;
  for (int64_t it = int64_t(blockIdx.x) * 256 + threadIdx.x; it < items; it += int64_t(parts) * 256) {
    const int64_t row = it / groups;
    const int col = static_cast<int>(it % groups) * 16;
    const T* p = g + row * src.ld + col;
    if (col + 16 <= src.cols) {
      const Pack<16, T> v = load_pack<16>(p);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const double x = to_float(v.v[i]);
        sum = fma(x, x, sum);
      }
    } else {
      for (int i = 0; i < src.cols - col; ++i) {
        const double x = to_float(p[i]);
        sum = fma(x, x, sum);
      }
    }
  }
  __shared__ double s[4];
  sum = block_sum(sum, s);
  if (threadIdx.x == 0) part[int64_t(blockIdx.y) * kNormBlocks + blockIdx.x] = sum;
}

// 1 / (|G|_F + eps) from the parts; all threads of a 256-thread block call it.  In
// double, and x times it too: the norm of finite floats can pass a float's largest
// number or lie below its normal ones.
__device__ __forceinline__ double factor(const double* part, int parts, float eps, double (&s)[4]) {
  double sum = 0;
  for (int p = threadIdx.x; p < parts; p += 256) sum += part[int64_t(blockIdx.y) * kNormBlocks + p];
  return 1.0 / (sqrt(block_sum(sum, s)) + eps);
}

// X_0 as pairs, as G lies (`direct`: rows of G) and transposed (`across`), a
// 64 x 64 tile a block through LDS; both padded with zeros.  Bound by memory:
// 4096 x 4096 floats, 192 MiB, in 38.5 us (5.2 TB/s; 44.9 with the loads behind
// the norm), 256 x 256 in 4.8 us (7.0).
template <class T>
__global__ __launch_bounds__(256) void k_start(Source src, const double* part, int parts, float eps, Pairs direct,
                                               Pairs across, int tiles_c) {
  __shared__ double s[4];
  __shared__ float t[64][65];
  const T* g = static_cast<const T*>(src.g) + blockIdx.y * src.batch;
  const int r0 = blockIdx.x / tiles_c * 64, c0 = blockIdx.x % tiles_c * 64;
  T x[16];  // under way while the norm's parts are added
#pragma unroll
  for (int p = 0; p < 16; ++p) {
    const int r = p * 4 + threadIdx.x / 64, c = threadIdx.x % 64;
    x[p] = T{};
    if (r0 + r < src.rows && c0 + c < src.cols) x[p] = g[(r0 + r) * src.ld + c0 + c];
  }
  const double by = factor(part, parts, eps, s) * kScaleX;
#pragma unroll
  for (int p = 0; p < 16; ++p) t[p * 4 + threadIdx.x / 64][threadIdx.x % 64] = static_cast<float>(to_float(x[p]) * by);
  __syncthreads();
  uint8_t* dp = direct.p + blockIdx.y * direct.batch;
  uint8_t* ap = across.p + blockIdx.y * across.batch;
  const int64_t dpad = pad32(src.cols), apad = pad32(src.rows);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int r = p * 16 + threadIdx.x / 16, c = threadIdx.x % 16 * 4;
    if (r0 + r < src.rows && c0 + c < dpad)
      store_pairs(dp + (r0 + r) * direct.ld, c0 + c, v4f{t[r][c], t[r][c + 1], t[r][c + 2], t[r][c + 3]});
    if (c0 + r < src.cols && r0 + c < apad)
      store_pairs(ap + (c0 + r) * across.ld, r0 + c, v4f{t[c][r], t[c + 1][r], t[c + 2][r], t[c + 3][r]});
  }
}

// steps == 0: G / (|G|_F + eps).
template <class T>
__global__ __launch_bounds__(256) void k_divide(Source src, const double* part, int parts, float eps, T* x,
                                                int64_t ldx, int64_t batch_x) {
  __shared__ double s[4];
  const double by = factor(part, parts, eps, s);
  const T* g = static_cast<const T*>(src.g) + blockIdx.y * src.batch;
  const int64_t items = int64_t(src.rows) * src.cols;
  for (int64_t it = int64_t(blockIdx.x) * 256 + threadIdx.x; it < items; it += int64_t(gridDim.x) * 256) {
    const int64_t r = it / src.cols, c = it % src.cols;
    from_float(static_cast<float>(to_float(g[r * src.ld + c]) * by), x[blockIdx.y * batch_x + r * ldx + c]);
  }
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

// What becomes of the sums of a symmetric m x m matrix: scaled, `b` times `add`
// added (if there is one) and `diagonal` on the diagonal, written as pairs at
// its place and, off the diagonal tiles, mirrored.  Both indexes run on past m
// to the padding, where zeros go.
struct SymmetricOut {
  Pairs out, add;
  int m;
  float scale, b, diagonal;
  int batch;
  bool mirror;
  __device__ __forceinline__ float value(int r, int c, float v, float old) const {
    return r < m && c < m ? fmaf(v, scale, b * old) + (r == c ? diagonal : 0.0f) : 0.0f;
  }
  // four neighbours of a row
  __device__ __forceinline__ void operator()(int r, int c, v4f v) const {
    if (r >= pad32(m) || c >= pad32(m)) return;
    uint8_t* base = out.p + batch * out.batch;
    v4f x = {0, 0, 0, 0};
    if (r < m) {
      const v4f old = add.p ? load_pairs(add.p + batch * add.batch + r * add.ld, c) : x;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = value(r, c + i, v[i], old[i]);
      store_pairs(base + r * out.ld, c, x);
    }
    if (mirror) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < m) store_pair(base + (c + i) * out.ld, r, x[i]);
    }
  }
  // 64 rows of a tile, from row r0 and column c0
  template <int THREADS, int COLS>
  __device__ __forceinline__ void sheet(nt::Sheet<COLS>& s, int r0, int c0) const {
    uint8_t* base = out.p + batch * out.batch;
    s.template out<THREADS>(
        mirror,
        [&](int r, int c, float (&v)[8]) {
          r += r0, c += c0;
          if (c >= pad32(m)) return;
          v4f old[2] = {};
          if (add.p && r < m) {
            old[0] = load_pairs(add.p + batch * add.batch + r * add.ld, c);
            old[1] = load_pairs(add.p + batch * add.batch + r * add.ld, c + 4);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = value(r, c + i, v[i], old[i / 4][i % 4]);
          if (r < m) store_pairs8(base + r * out.ld, c, v);
        },
        [&](int c, int r, const float (&v)[8]) {
          if (c0 + c < m && r0 + r < pad32(m)) store_pairs8(base + (c0 + c) * out.ld, r0 + r, v);
        });
  }
};

// P X: as pairs and transposed pairs, or at the last step as the result.
template <class T>
struct IterateOut {
  Pairs x, xt;
  T* out;  // not NULL at the last step
  int64_t ldo, batch_o;
  int m, n;
  int batch;
  bool tall;
  __device__ __forceinline__ void operator()(int r, int c, v4f v) const {
    if (r >= pad32(m) || c >= pad32(n)) return;
    v4f y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = r < m && c + i < n ? v[i] * (1.0f / kScaleS) : 0.0f;
    if (out) {
      if (r >= m) return;
      T* o = out + batch * batch_o;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < n) from_float(y[i] * (1.0f / kScaleX), tall ? o[(c + i) * ldo + r] : o[r * ldo + c + i]);
    } else {
      if (r < m) store_pairs(x.p + batch * x.batch + r * x.ld, c, y);
      uint8_t* t = xt.p + batch * xt.batch;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < n) store_pair(t + (c + i) * xt.ld, r, y[i]);
    }
  }
  // `count` of eight neighbours of the result, from `at`
  __device__ __forceinline__ void result(T* at, int count, const float (&v)[8]) const {
    Pack<8, T> p;
#pragma unroll
    for (int i = 0; i < 8; ++i) from_float(v[i] * (1.0f / (kScaleS * kScaleX)), p.v[i]);
    if (count >= 8) {
      store_pack(at, p);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < count) at[i] = p.v[i];
    }
  }
  template <int THREADS, int COLS>
  __device__ __forceinline__ void sheet(nt::Sheet<COLS>& s, int r0, int c0) const {
    T* o = out + batch * batch_o;
    uint8_t *xp = x.p + batch * x.batch, *tp = xt.p + batch * xt.batch;
    s.template out<THREADS>(
        !out || tall,
        [&](int r, int c, float (&v)[8]) {
          r += r0, c += c0;
          if (out) {
            if (!tall && r < m && c < n) result(o + r * ldo + c, n - c, v);
            return;
          }
          if (c >= pad32(n)) return;
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = r < m && c + i < n ? v[i] * (1.0f / kScaleS) : 0.0f;
          if (r < m) store_pairs8(xp + r * x.ld, c, v);
        },
        [&](int c, int r, const float (&v)[8]) {
          r += r0, c += c0;
          if (c >= n) return;
          if (!out) {
            if (r < pad32(m)) store_pairs8(tp + c * xt.ld, r, v);
          } else if (r < m) {
            result(o + c * ldo + r, m - r, v);
          }
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
// Large ones, with their loop in assembly; several wavefronts a SIMD where registers allow.
template <int MT, int NT, int WM, int WN, int STAGES>
struct Assembled : nt::Loop<nt::Kind::kPair, MT, NT, WM, WN, STAGES> {
  static constexpr bool kDirect = false;
  static constexpr int kMinWaves = 2;
};

template <class T, class E>
__device__ __forceinline__ void product(const Side& A, const Side& B, int m0, int n0, int K, const E& epi) {
  if constexpr (T::kDirect) {
    __shared__ typename T::Meet meet;
    T::run(meet, A, B, m0, n0, K * 4, epi);
  } else {
    __shared__ alignas(16) uint8_t smem[T::kLds];
    nt::v16f acc[T::kAcc];
    nt::loop_sum<T>(smem, A, B, m0, n0, K * 4, acc);
    using Sheet = nt::Sheet<T::BN>;
    static_assert(sizeof(Sheet) <= T::kLds, "a sheet fits");
    Sheet& sheet = *reinterpret_cast<Sheet*>(smem);
    __syncthreads();  // all wavefronts have left the loop
    nt::loop_sheets<T>(sheet, acc, [&](int top) { epi.template sheet<T::threads>(sheet, m0 + top, n0); });
  }
}

// S = X X^T and P = a + b S + c S S: the lower tiles, mirrored.  Bound by the
// matrix rate where the tiles fill the CUs: 4096 x 4096 in 165-175 us on 253 tiles
// of 192 x 192 (136 of 256 x 256 would leave half the CUs idle), MfmaUtil 65 %; by
// the latency of one trip to memory where they are few: 256 x 256 in 4.4 us.
template <class T>
__global__ __launch_bounds__(T::threads, T::kMinWaves) void k_symmetric(Side A, int K, SymmetricOut out) {
  out.batch = blockIdx.y;
  A.p += blockIdx.y * A.batch;
  const nt::Place at = triangle(static_cast<int>(xcd_contiguous(blockIdx.x, gridDim.x)));
  out.mirror = at.tm != at.tn;
  product<T>(A, A, at.tm * T::BM, at.tn * T::BN, K, out);
}

// X' = P X.  Bound by the matrix rate: 4096 x 4096 in 278 us on 256 tiles of
// 256 x 256, 1483 TFLOP/s of half products, MfmaUtil 75 %; 1024 x 1024 x 4096 in
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
  const int tile = blockIdx.x / T::waves, share = blockIdx.x % T::waves, lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const nt::Place at = triangle(tile);
  out.batch = blockIdx.y;
  out.mirror = at.tm != at.tn;
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
  out.sheet<256>(sheet, at.tm * T::BM + share % T::WM * 64, at.tn * T::BN + share / T::WM * 16 * T::NT);
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

// The workspace: per-block parts of the norms, then X, X^T twice, S and P, and the
// parts of the symmetric products' sums.
struct Layout {
  int m, n;
  int64_t part, x, xt[2], s, p, sums, bytes;
  int64_t ldx, ldm;  // bytes of a row of X, and of the others
};

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

Layout layout_of(int batch, int rows, int cols) {
  Layout l;
  l.m = rows < cols ? rows : cols;
  l.n = rows < cols ? cols : rows;
  l.ldx = pad32(l.n) * 4;
  l.ldm = pad32(l.m) * 4;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += up256(bytes);
    return here;
  };
  l.part = take(int64_t(batch) * kNormBlocks * 8);
  l.x = take(batch * (l.m * l.ldx));
  l.xt[0] = take(batch * (l.n * l.ldm));
  l.xt[1] = take(batch * (l.n * l.ldm));
  l.s = take(batch * (l.m * l.ldm));
  l.p = take(batch * (l.m * l.ldm));
  const int64_t t = ceil_div(l.m, Loop128::BM), tiles = batch * (t * (t + 1) / 2);
  l.sums = take(tiles > 0 && tiles <= 128 ? (256 / tiles < kMaxParts ? 256 / tiles : kMaxParts) * tiles * (Loop128::BM * Loop128::BN * 4) : 0);
  l.bytes = at;
  return l;
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
  double* part = reinterpret_cast<double*>(ws + l.part);
  const int64_t groups = int64_t(src.rows) * ceil_div(src.cols, 16);
  const int parts = static_cast<int>(ceil_div(groups, 256) < kNormBlocks ? ceil_div(groups, 256) : kNormBlocks);
  hipLaunchKernelGGL((k_norm<T>), dim3(parts, batch), dim3(256), 0, stream, src, part, parts);
  if (steps == 0) {
    const int64_t blocks = ceil_div(int64_t(src.rows) * src.cols, 256);
    hipLaunchKernelGGL((k_divide<T>), dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096), batch), dim3(256), 0,
                       stream, src, part, parts, eps, x, ldx, batch_x);
    return hipGetLastError();
  }
  const bool tall = src.rows > src.cols;
  const Pairs X{ws + l.x, l.ldx, l.m * l.ldx};
  Pairs XT{ws + l.xt[0], l.ldm, l.n * l.ldm}, XT2{ws + l.xt[1], l.ldm, l.n * l.ldm};
  const Pairs S{ws + l.s, l.ldm, l.m * l.ldm}, P{ws + l.p, l.ldm, l.m * l.ldm};
  // 64-wide tiles: both paddings (to 32) lie inside them
  const int64_t tr = ceil_div(src.rows, 64), tc = ceil_div(src.cols, 64);
  hipLaunchKernelGGL((k_start<T>), dim3(static_cast<unsigned>(tr * tc), batch), dim3(256), 0, stream, src, part, parts,
                     eps, tall ? XT : X, tall ? X : XT, static_cast<int>(tc));
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
    symmetric(choice.s, side(X, l.m), kn,
              SymmetricOut{S, Pairs{nullptr, 0, 0}, l.m, kScaleS / (kScaleX * kScaleX), 0.0f, 0.0f, 0, false});
    symmetric(choice.p, side(S, l.m), km, SymmetricOut{P, S, l.m, c / kScaleS, b, a * kScaleS, 0, false});
    const bool last = i + 1 == steps;
    const IterateOut<T> out{X, XT2, last ? x : nullptr, ldx, batch_x, l.m, l.n, 0, tall};
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

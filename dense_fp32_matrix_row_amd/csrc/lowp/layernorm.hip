// layernorm.hip -- hip_layernorm_forward and hip_layernorm_backward.
//
// Bound by memory: the forward pass reads x and writes y, the backward pass reads
// x and dy and writes dx, each once, against some ten vector instructions an
// element; rows lie in registers (rows.h) from the sums to the results.
//
// One MI355X, kernels alone, forward and backward: 16 x 1024 bf16 3.5 and 2.8 us, 8192 x
// 1024 9.0 and 17, 8192 x 4096 27 (4.9 TB/s) and 51 (3.9 TB/s, and 25 MB of parts written
// and read), 8192 x 8192 57 and 95, 4096 x 16384 65 and 121, 65536 x 512 28 and 45; 4097 x
// 2049 float32 14 and 29; 2048 x 32768, past what registers hold, 95 and 200.
#include <algorithm>

#include "../../../include/layernorm.h"
#include "rows.h"

namespace sgemm {
namespace {

static_assert(HIP_LAYERNORM_ROW == kRowWidth);

struct Sum {
  template <class T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};

// w or b: numbers side by side, of X's type or floats, or (NULL) one number for all.
template <class W>
__device__ __forceinline__ void load_param(float (&v)[8], const W* p, float fill, int col, int cols) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fill;
    return;
  }
  const Pack<8, W> r = load_row8(p, col, cols);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_float(r.v[i]);
}

// A row's mean, what its rounding to float left over, and rstd.
struct Stats {
  float mean, rest, rstd;
};
__device__ __forceinline__ Stats load_stats(const float* stats, int64_t row, int64_t rows) {
  return Stats{stats[row], stats[rows + row], stats[2 * rows + row]};
}
__device__ __forceinline__ void store_stats(float* stats, int64_t row, int64_t rows, const Stats& s) {
  stats[row] = s.mean;
  stats[rows + row] = s.rest;
  stats[2 * rows + row] = s.rstd;
}
// (x - mean) rstd: x - mean is exact where x is near the mean, and the rest small.
__device__ __forceinline__ float normalised(float x, const Stats& s) { return ((x - s.mean) - s.rest) * s.rstd; }

// Where chunk c of a lane lies: WIDE (load_last8), the row's last eight if it would reach
// over its end.
template <bool WIDE, class S>
__device__ __forceinline__ int place(int c, int lane, int cols) {
  const int col = (c * S::LANES + lane) * 8;
  return WIDE ? min(col, cols - 8) : col;
}

// Adds g h to the backward pass's second sum; `inside`: of an element of the row.  Past its end
// dy, and so g, is zero, but a zero's (x - mean) rstd may pass a float's range where the
// row's own do not, and 0 inf is NaN.  (Not of halfs: no mean of theirs times an rstd does.)
template <class X, class T>
__device__ __forceinline__ void add_inside(T& sum, T g, T h, bool inside) {
  const T v = fma(g, h, sum);
  sum = std::is_same_v<X, _Float16> || inside ? v : sum;
}

// A lane's share of a row, zeros past its end.
template <class S, class X>
struct Share {
  Pack<8, X> v[S::COUNT];
  __device__ __forceinline__ void load(const X* row, int lane, int cols) {
#pragma unroll
    for (int c = 0; c < S::COUNT; ++c) v[c] = load_row8(row, (c * S::LANES + lane) * 8, cols);
  }
  // Without branches around the loads: of a row of whole eights; the same with the row's last
  // eight past its end; of any row (at least eight), zeros also for those of its last eight
  // that the lane before has.
  __device__ __forceinline__ void load_even(const X* row, int lane, int cols) {
    load_any(row, lane, cols);
#pragma unroll
    for (int c = 0; c < S::COUNT; ++c)
      if ((c * S::LANES + lane) * 8 >= cols) v[c] = Pack<8, X>{};
  }
  __device__ __forceinline__ void load_any(const X* row, int lane, int cols) {
#pragma unroll
    for (int c = 0; c < S::COUNT; ++c) v[c] = load_last8(row, (c * S::LANES + lane) * 8, cols);
  }
  __device__ __forceinline__ void load_wide(const X* row, int lane, int cols) {
#pragma unroll
    for (int c = 0; c < S::COUNT; ++c) v[c] = load_last8(row, (c * S::LANES + lane) * 8, cols);
#pragma unroll
    for (int c = 0; c < S::COUNT; ++c) {
      const int before = (c * S::LANES + lane) * 8 - (cols - 8);
      if (before > 0)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < before) v[c].v[i] = X{};
    }
  }
  // Makes the compiler forget what it made of the elements so far, lest it keep them
  // as floats beside the halves that they come as.
  __device__ __forceinline__ void forget() {
    if constexpr (sizeof(X) == 2) {
#pragma unroll
      for (int c = 0; c < S::COUNT; ++c) {
        uint4 r = __builtin_bit_cast(uint4, v[c]);
        asm volatile("" : "+v"(r.x), "+v"(r.y), "+v"(r.z), "+v"(r.w));
        v[c] = __builtin_bit_cast(Pack<8, X>, r);
      }
    }
  }
};

// Blocks walk the rows, with w and b in registers (read for each row, floats of them
// would be twice the bytes of 16-bit x and y: 8192 x 4096 39 us instead of 27).
//
// The mean rounded to float is off by up to 2^-24 of itself, which for a row far
// off zero is much of its differences, so their own mean is taken beside their
// squares': with d = x - mean, the mean is mean + avg d and the variance
// avg d^2 - (avg d)^2.
//
// Where the squares' sum passes a float's range (rows of 10^18; equal values of 10^26, whose
// mean is some steps off them; never halfs), the differences from the whole mean are squared
// again, times 2^-80, behind a branch that is hardly taken (0.2 us of code to fetch; squares
// of scaled differences throughout cost 2-6 %: 8192 x 4096 bf16 26.4 -> 28.1 us).  Where eps is
// below kLeastEps (0 as a rule) and squares below a float's normal numbers would count, the
// differences and their squares are summed in double.
constexpr float kLeastEps = 0x1p-100f;
template <bool WIDE, class D, class S, class X, class W>
__global__ __launch_bounds__(S::threads, S::LANES <= 256 ? 5 : 4) void k_forward(
    const X* x, int64_t ldx, const W* __restrict__ w, const W* __restrict__ b, float eps, X* y, int64_t ldy,
    float* __restrict__ stats, int rows, int cols) {
  __shared__ float first[S::threads / 64][1], third[S::threads / 64][1];
  __shared__ D second[S::threads / 64][2];
  const int lane = threadIdx.x % S::LANES;
  const int64_t steps = ceil_div(rows, S::rows);
  const float n = static_cast<float>(cols);
  float wv[S::COUNT][8], bv[S::COUNT][8];
#pragma unroll
  for (int c = 0; c < S::COUNT; ++c) {
    load_param(wv[c], w, 1.0f, place<WIDE, S>(c, lane, cols), cols);
    load_param(bv[c], b, 0.0f, place<WIDE, S>(c, lane, cols), cols);
  }
  for (int64_t step = blockIdx.x; step < steps; step += gridDim.x) {
    const int64_t row = step * S::rows + threadIdx.x / S::LANES;
    const bool live = S::rows == 1 || row < rows;
    Share<S, X> now{};
    if (live) {
      if constexpr (WIDE) now.load_wide(x + row * ldx, lane, cols);
      else now.load(x + row * ldx, lane, cols);
    }
    float sum[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < S::COUNT; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0] += to_float(now.v[c].v[i]);
    join_row<S>(sum, first, Sum{});
    Stats s{sum[0] / n, 0.0f, 0.0f};
    D d[2] = {0, 0};
#pragma unroll
    for (int c = 0; c < S::COUNT; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool inside = WIDE ? i >= (c * S::LANES + lane) * 8 - (cols - 8) : (c * S::LANES + lane) * 8 < cols - i;
        const float t = inside ? to_float(now.v[c].v[i]) - s.mean : 0.0f;
        d[0] += t;
        d[1] = fma(static_cast<D>(t), static_cast<D>(t), d[1]);
      }
    join_row<S>(d, second, Sum{});
    now.forget();
    if constexpr (sizeof(D) == 8) {
      const double rest = d[0] / cols;
      s.rest = static_cast<float>(rest);
      s.rstd = static_cast<float>(1.0 / sqrt(fmax(d[1] / cols - rest * rest, 0.0) + static_cast<double>(eps)));
    } else {
      s.rest = d[0] / n;
      s.rstd = 1.0f / sqrtf(fmaxf(d[1] / n - s.rest * s.rest, 0.0f) + eps);
    }
    const bool past = !(d[1] < static_cast<D>(INFINITY));
    if constexpr (sizeof(D) == 8 || std::is_same_v<X, _Float16>) {
      if (past) s.rstd = __uint_as_float(0x7fc00000u);  // fmax takes no NaN over
    } else {
      bool again = past;  // the same in all threads that meet
      if constexpr (S::waves > 1 && S::rows > 1)
#pragma unroll
        for (int i = 0; i < S::threads / 64; ++i) again = again || !(second[i][1] < 0x1p126f);
      if (__builtin_expect(__ballot(again) != 0, 0)) {
        float e[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < S::COUNT; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const bool inside = WIDE ? i >= (c * S::LANES + lane) * 8 - (cols - 8) : (c * S::LANES + lane) * 8 < cols - i;
            const float t = inside ? ((to_float(now.v[c].v[i]) - s.mean) - s.rest) * 0x1p-80f : 0.0f;
            e[0] = fmaf(t, t, e[0]);
          }
        join_row<S>(e, third, Sum{});
        now.forget();
        const float v = e[0] / n;  // 2^-160 of the variance
        if (past) s.rstd = v < 0x1p-60f ? 1.0f / sqrtf(v * 0x1p80f * 0x1p80f + eps) : 0x1p-80f / sqrtf(v + eps * 0x1p-80f * 0x1p-80f);
      }
    }
    if (live) {
#pragma unroll
      for (int c = 0; c < S::COUNT; ++c) {
        Pack<8, X> r;
#pragma unroll
        for (int i = 0; i < 8; ++i) from_float(fmaf(normalised(to_float(now.v[c].v[i]), s), wv[c][i], bv[c][i]), r.v[i]);
        if constexpr (WIDE) store_last8(y + row * ldy, (c * S::LANES + lane) * 8, cols, r);
        else store_row8(y + row * ldy, (c * S::LANES + lane) * 8, cols, r);
      }
      if (stats && lane == 0) store_stats(stats, row, rows, s);
    }
  }
}

// Rows longer than registers hold: read three times, sums in double.
template <class X, class W>
__global__ __launch_bounds__(1024) void k_forward_long(const X* x, int64_t ldx, const W* __restrict__ w,
                                                       const W* __restrict__ b, float eps, X* y, int64_t ldy,
                                                       float* __restrict__ stats, int rows, int cols) {
  using S = RowShape<1024, 1>;
  __shared__ double first[S::threads / 64][1], second[S::threads / 64][2];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const X* const from = x + row * ldx;
    double sum[1] = {0.0};
    for (int64_t c = threadIdx.x * 8; c < cols; c += S::width) {
      const Pack<8, X> v = load_row8(from, static_cast<int>(c), cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0] += static_cast<double>(to_float(v.v[i]));
    }
    join_row<S>(sum, first, Sum{});
    const double mean = sum[0] / cols;
    double d[2] = {0.0, 0.0};
    for (int64_t c = threadIdx.x * 8; c < cols; c += S::width) {
      const Pack<8, X> v = load_row8(from, static_cast<int>(c), cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double t = c + i < cols ? static_cast<double>(to_float(v.v[i])) - mean : 0.0;
        d[0] += t;
        d[1] = fma(t, t, d[1]);
      }
    }
    join_row<S>(d, second, Sum{});
    Stats s;
    s.mean = static_cast<float>(mean);
    s.rest = static_cast<float>(mean - static_cast<double>(s.mean));
    s.rstd = static_cast<float>(1.0 / sqrt(d[1] / cols + static_cast<double>(eps)));
    for (int64_t c = threadIdx.x * 8; c < cols; c += S::width) {
      const Pack<8, X> v = load_row8(from, static_cast<int>(c), cols);
      float wv[8], bv[8];
      load_param(wv, w, 1.0f, static_cast<int>(c), cols);
      load_param(bv, b, 0.0f, static_cast<int>(c), cols);
      Pack<8, X> r;
#pragma unroll
      for (int i = 0; i < 8; ++i) from_float(fmaf(normalised(to_float(v.v[i]), s), wv[i], bv[i]), r.v[i]);
      store_row8(y + row * ldy, static_cast<int>(c), cols, r);
    }
    if (stats && threadIdx.x == 0) store_stats(stats, row, rows, s);
  }
}

// dw and db of a block's rows lie in its threads' registers, a thread's columns
// being the same in every row, and leave once, into the block's part of the
// workspace; k_join adds the parts in their order.  The next row's loads ahead of this
// one's sums take more registers than they hide (8192 x 4096 51 -> 54 us, 4097 x 2049
// float32 29 -> 40); blocks of 1024 threads, two rows and a third fewer parts, 51 and 43.
template <bool EVEN, class S, class X, class W>
__global__ __launch_bounds__(S::threads, S::COUNT == 1 && S::LANES <= 512 ? 6 : 4) void k_backward(
    const X* dy, int64_t lddy, const X* x, int64_t ldx, const float* __restrict__ stats, const W* __restrict__ w, X* dx,
    int64_t lddx, float* __restrict__ parts, int rows, int cols) {
  __shared__ float meet[2][S::threads / 64][2];
  const int lane = threadIdx.x % S::LANES;
  const int64_t steps = ceil_div(rows, S::rows);
  const float n = static_cast<float>(cols);
  // w too, but in the widest rows, whose threads have 128 registers (4096 x 16384 bf16:
  // with some of them spilled 159 us, with w read in each row 120), and where it is
  // fp16 and two chunks a lane, which the compiler spills as well (8192 x 8192 248, 107)
  constexpr bool kHold = S::LANES < 1024 && !(S::COUNT == 2 && std::is_same_v<W, _Float16>);
  float wv[S::COUNT][8], pw[S::COUNT][8], pb[S::COUNT][8];
  const auto load_w = [&](int c) { load_param(wv[c], w, 1.0f, (c * S::LANES + lane) * 8, cols); };
#pragma unroll
  for (int c = 0; c < S::COUNT; ++c) {
    if (kHold) load_w(c);
#pragma unroll
    for (int i = 0; i < 8; ++i) pw[c][i] = pb[c][i] = 0.0f;
  }
  Share<S, X> xv, gv;
  Stats s;
  const auto load = [&](int64_t step) {  // rows past the last repeat it
    const int64_t row = min(step * S::rows + threadIdx.x / S::LANES, int64_t(rows) - 1);
    if constexpr (EVEN) {
      xv.load_any(x + row * ldx, lane, cols);
      gv.load_even(dy + row * lddy, lane, cols);
    } else {
      xv.load(x + row * ldx, lane, cols);
      gv.load(dy + row * lddy, lane, cols);
    }
    s = load_stats(stats, row, rows);
  };
  load(blockIdx.x);
  int turn = 0;
  for (int64_t step = blockIdx.x; step < steps; step += gridDim.x, turn ^= 1) {
    const int64_t row = step * S::rows + threadIdx.x / S::LANES;
    const bool live = S::rows == 1 || row < rows;
    float sum[2] = {0.0f, 0.0f};
    if (live) {
#pragma unroll
      for (int c = 0; c < S::COUNT; ++c) {
        if (!kHold) load_w(c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // past the row's end dy is zero
          const float t = to_float(gv.v[c].v[i]), g = t * wv[c][i], h = normalised(to_float(xv.v[c].v[i]), s);
          pw[c][i] = fmaf(t, h, pw[c][i]);
          pb[c][i] += t;
          sum[0] += g;
          add_inside<X>(sum[1], g, h, EVEN || c < S::COUNT - 1 || (c * S::LANES + lane) * 8 < cols - i);
        }
      }
    }
    if (dx) {
      join_row<S>(sum, meet[turn], Sum{});
      xv.forget();
      gv.forget();
      const float c1 = sum[0] / n, c2 = sum[1] / n;
      if (live) {
#pragma unroll
        for (int c = 0; c < S::COUNT; ++c) {
          if (!kHold) load_w(c);
          Pack<8, X> r;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float g = fmaf(to_float(gv.v[c].v[i]), wv[c][i], -c1), h = normalised(to_float(xv.v[c].v[i]), s);
            from_float((g - h * c2) * s.rstd, r.v[i]);
          }
          store_row8(dx + row * lddx, (c * S::LANES + lane) * 8, cols, r);
        }
      }
    }
    if (step + gridDim.x < steps) load(step + gridDim.x);
  }
  if (!parts) return;
  float* const to = parts + int64_t(blockIdx.x) * 2 * cols;
  if constexpr (S::rows > 1) {  // the block's rows first
    __shared__ float all[S::rows][S::width];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < S::COUNT; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) all[threadIdx.x / S::LANES][(c * S::LANES + lane) * 8 + i] = k ? pb[c][i] : pw[c][i];
      __syncthreads();
      for (int at = threadIdx.x; at < cols; at += S::threads) {
        float v = all[0][at];
#pragma unroll
        for (int r = 1; r < S::rows; ++r) v += all[r][at];
        to[k * cols + at] = v;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int c = 0; c < S::COUNT; ++c) {
        Pack<8, float> v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v.v[i] = k ? pb[c][i] : pw[c][i];
        store_row8(to + k * cols, (c * S::LANES + lane) * 8, cols, v);
      }
  }
}

// Few rows: dx a row of threads each, as above, and beside them in the same launch dw
// and db, a block for 64 columns, whose wavefronts take every so many-th row with four
// loads under way: no parts, no second launch to join them (16 x 1000 bf16 6.9 -> 3.2 us,
// 128 x 4000 9.6 -> 5.0, 256 x 1000 7.7 -> 6.5; 512 x 1000 would take 14.0 against 8.1).  x
// and dy are read twice, so where dx is written over one of them there are two
// launches, the columns' first: the same sums.
template <class S, class X, class W>
__global__ __launch_bounds__(S::threads, S::COUNT == 1 && S::LANES <= 512 ? 6 : 4) void k_few(
    const X* dy, int64_t lddy, const X* x, int64_t ldx, const float* __restrict__ stats, const W* __restrict__ w, X* dx,
    int64_t lddx, float* dw, float* db, int accumulate, int rows, int cols, int row_blocks) {
  constexpr int kWaves = S::threads / 64;
  __shared__ float meet[kWaves][2], all[2][kWaves][64];
  const float n = static_cast<float>(cols);
  if (static_cast<int>(blockIdx.x) < row_blocks) {
    const int lane = threadIdx.x % S::LANES, row = blockIdx.x * S::rows + threadIdx.x / S::LANES, from = min(row, rows - 1);
    Share<S, X> xv, gv;
    xv.load(x + from * ldx, lane, cols);
    gv.load(dy + from * lddy, lane, cols);
    const Stats s = load_stats(stats, from, rows);
    float wv[S::COUNT][8], sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < S::COUNT; ++c) {
      load_param(wv[c], w, 1.0f, (c * S::LANES + lane) * 8, cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = to_float(gv.v[c].v[i]) * wv[c][i];
        sum[0] += g;
        add_inside<X>(sum[1], g, normalised(to_float(xv.v[c].v[i]), s), c < S::COUNT - 1 || (c * S::LANES + lane) * 8 < cols - i);
      }
    }
    join_row<S>(sum, meet, Sum{});
    const float c1 = sum[0] / n, c2 = sum[1] / n;
    if (row >= rows) return;
#pragma unroll
    for (int c = 0; c < S::COUNT; ++c) {
      Pack<8, X> r;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = fmaf(to_float(gv.v[c].v[i]), wv[c][i], -c1), h = normalised(to_float(xv.v[c].v[i]), s);
        from_float((g - h * c2) * s.rstd, r.v[i]);
      }
      store_row8(dx + row * lddx, (c * S::LANES + lane) * 8, cols, r);
    }
    return;
  }
  constexpr int kLoads = 4;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, col = (blockIdx.x - row_blocks) * 64 + lane;
  const int at = min(col, cols - 1);
  float pw = 0.0f, pb = 0.0f;
  for (int r0 = wave; r0 < rows; r0 += kLoads * kWaves) {
    X xv[kLoads], gv[kLoads];
    Stats s[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int row = min(r0 + u * kWaves, rows - 1);
      xv[u] = x[row * ldx + at];
      gv[u] = dy[row * lddy + at];
      s[u] = load_stats(stats, row, rows);
    }
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      if (r0 + u * kWaves < rows) {
        const float t = to_float(gv[u]);
        pw = fmaf(t, normalised(to_float(xv[u]), s[u]), pw);
        pb += t;
      }
  }
  all[0][wave][lane] = pw;
  all[1][wave][lane] = pb;
  __syncthreads();
  if (wave > 1 || col >= cols) return;
  float* const out = wave ? db : dw;
  if (!out) return;
  float v = all[wave][0][lane];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) v += all[wave][i][lane];
  out[col] = accumulate ? out[col] + v : v;
}

// Rows longer than registers hold: first dw and db (dx may be written over dy), a
// block for 2048 columns of a share of the rows; then dx, a block a row, read twice.
template <class X>
__global__ __launch_bounds__(256) void k_params_long(const X* __restrict__ dy, int64_t lddy, const X* __restrict__ x,
                                                     int64_t ldx, const float* __restrict__ stats,
                                                     float* __restrict__ parts, int rows, int cols, int strips) {
  const int64_t strip = blockIdx.x % strips, part = blockIdx.x / strips, count = gridDim.x / strips;
  const int64_t at = strip * 2048 + threadIdx.x * 8;
  if (at >= cols) return;
  const int col = static_cast<int>(at);
  Pack<8, float> pw{}, pb{};
  for (int64_t row = part; row < rows; row += count) {
    const Pack<8, X> xv = load_row8(x + row * ldx, col, cols), gv = load_row8(dy + row * lddy, col, cols);
    const Stats s = load_stats(stats, row, rows);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = to_float(gv.v[i]);
      pw.v[i] = fmaf(t, normalised(to_float(xv.v[i]), s), pw.v[i]);
      pb.v[i] += t;
    }
  }
  store_row8(parts + part * 2 * cols, col, cols, pw);
  store_row8(parts + part * 2 * cols + cols, col, cols, pb);
}

template <class X, class W>
__global__ __launch_bounds__(1024) void k_backward_long(const X* dy, int64_t lddy, const X* x, int64_t ldx,
                                                        const float* __restrict__ stats, const W* __restrict__ w, X* dx,
                                                        int64_t lddx, int rows, int cols) {
  using S = RowShape<1024, 1>;
  __shared__ double meet[2][S::threads / 64][2];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
    const Stats s = load_stats(stats, row, rows);
    double sum[2] = {0.0, 0.0};
    for (int64_t c = threadIdx.x * 8; c < cols; c += S::width) {
      const int col = static_cast<int>(c);
      const Pack<8, X> xv = load_row8(x + row * ldx, col, cols), gv = load_row8(dy + row * lddy, col, cols);
      float wv[8];
      load_param(wv, w, 1.0f, col, cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = to_float(gv.v[i]) * wv[i];
        sum[0] += static_cast<double>(g);
        add_inside<X>(sum[1], static_cast<double>(g), static_cast<double>(normalised(to_float(xv.v[i]), s)), col < cols - i);
      }
    }
    join_row<S>(sum, meet[turn], Sum{});
    const float c1 = static_cast<float>(sum[0] / cols), c2 = static_cast<float>(sum[1] / cols);
    for (int64_t c = threadIdx.x * 8; c < cols; c += S::width) {
      const int col = static_cast<int>(c);
      const Pack<8, X> xv = load_row8(x + row * ldx, col, cols), gv = load_row8(dy + row * lddy, col, cols);
      float wv[8];
      load_param(wv, w, 1.0f, col, cols);
      Pack<8, X> r;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        from_float((fmaf(to_float(gv.v[i]), wv[i], -c1) - normalised(to_float(xv.v[i]), s) * c2) * s.rstd, r.v[i]);
      store_row8(dx + row * lddx, col, cols, r);
    }
  }
}

// dw (blockIdx.y 0) and db (1): the sums of the parts' columns, 32 columns a block (a
// cache line of each part; 16 read the lines twice, 8192 x 4096 51 -> 60 us), 32
// shares of the parts, each in its order with twelve loads under way, then the shares.
// (Eight shares and one load after another took 25 of 8192 x 1024's 34 us.)
__global__ __launch_bounds__(1024) void k_join(const float* __restrict__ parts, int count, float* dw, float* db, int cols,
                                               int accumulate) {
  constexpr int kShares = 32, kLoads = 12;
  __shared__ float meet[kShares][33];
  float* const out = blockIdx.y ? db : dw;
  if (!out) return;
  const int share = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int64_t tile = blockIdx.x; tile < ceil_div(cols, 32); tile += gridDim.x) {
    const int64_t col = tile * 32 + lane;
    const float* const from = parts + int64_t(blockIdx.y) * cols + min(col, int64_t(cols) - 1);
    float v = 0.0f;
    for (int p = share; p < count; p += kShares * kLoads) {
      float t[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) t[i] = p + i * kShares < count ? from[int64_t(p + i * kShares) * 2 * cols] : 0.0f;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) v += t[i];
    }
    meet[share][lane] = v;
    __syncthreads();
    if (share == 0 && col < cols) {
#pragma unroll
      for (int i = 1; i < kShares; ++i) v += meet[i][lane];
      out[col] = accumulate ? out[col] + v : v;
    }
    __syncthreads();  // the next columns write the same LDS
  }
}
constexpr int64_t kJoinBlocks = int64_t(1) << 20;

// Calls f with the shape of rows of `cols` (at most kRowWidth).
template <class F>
void with_forward_shape(int cols, const F& f) {
  if (cols <= 128) f(RowShape<16, 1>{});
  else if (cols <= 256) f(RowShape<32, 1>{});
  else if (cols <= 512) f(RowShape<64, 1>{});
  else if (cols <= 1024) f(RowShape<64, 2>{});
  else if (cols <= 2048) f(RowShape<128, 2>{});
  else if (cols <= 4096) f(RowShape<256, 2>{});
  else if (cols <= 8192) f(RowShape<512, 2>{});
  else f(RowShape<1024, 2>{});
}
// Several rows a block, which share its part of dw and db.
template <class F>
void with_backward_shape(int cols, const F& f) {
  if (cols <= 128) f(RowShape<16, 1, 512>{});
  else if (cols <= 256) f(RowShape<32, 1, 512>{});
  else if (cols <= 512) f(RowShape<64, 1, 512>{});
  else if (cols <= 1024) f(RowShape<128, 1, 512>{});
  else if (cols <= 2048) f(RowShape<256, 1, 512>{});
  else if (cols <= 4096) f(RowShape<512, 1, 512>{});
  else if (cols <= 8192) f(RowShape<512, 2, 512>{});
  else f(RowShape<1024, 2>{});
}

constexpr int kFewRows = HIP_LAYERNORM_FEW;
bool few_rows(int rows, int cols) { return rows <= kFewRows && cols <= kRowWidth; }

// Blocks of the backward pass, each with a part of dw and db in the workspace; few rows
// have none.
int64_t parts_of(int rows, int cols) {
  if (few_rows(rows, cols)) return 0;
  if (cols > kRowWidth) {
    const int64_t share = 2048 / ceil_div(cols, 2048), most = share < 1 ? 1 : share < 64 ? share : 64;
    return rows < most ? rows : most;
  }
  int64_t parts = 0;
  with_backward_shape(cols, [&](auto shape) {
    using S = decltype(shape);
    const int64_t steps = ceil_div(rows, S::rows), cap = 256 * (S::COUNT == 1 ? 1536 : 1024) / S::threads;
    // two turns of a block from 128 blocks on: parts of one turn each would be as much to
    // write and read as x and dy (500 x 4000 16.3 -> 13.6 us, 300 x 2500 12.1 -> 10.5)
    const int64_t few = ceil_div(steps, 2) > 128 ? ceil_div(steps, 2) : 128;
    parts = std::min({steps, cap, few});
  });
  return parts;
}
struct Forward {
  int rows, cols;
  const void* x;
  int64_t ldx;
  const void *w, *b;
  float eps;
  void* y;
  int64_t ldy;
  float* stats;
};
struct Backward {
  int rows, cols;
  const void* dy;
  int64_t lddy;
  const void* x;
  int64_t ldx;
  const float* stats;
  const void* w;
  void* dx;
  int64_t lddx;
  float *dw, *db;
  int accumulate;
  float* parts;
  int count;
};

// Rows of two chunks a lane are loaded without branches (8192 x 8192 bf16 forward 61 ->
// 57 us, backward 103 -> 96; 4096 x 16384 72 -> 65, 125 -> 120), in the forward pass ragged ones
// too (8192 x 8191 79 -> 65; in the backward pass dropping what the lane before has costs
// more: 8192 x 8192 122); rows of one chunk are not (8192 x 4096 backward 51 -> 53, 65536 x
// 512 forward 29 -> 30).
template <class S>
bool even(int cols) { return S::COUNT == 2 && cols % 8 == 0; }

template <class X, class W>
void launch(const Forward& a, hipStream_t stream) {
  const X* const x = static_cast<const X*>(a.x);
  const W *const w = static_cast<const W*>(a.w), *const b = static_cast<const W*>(a.b);
  X* const y = static_cast<X*>(a.y);
  if (a.cols > kRowWidth) {
    const int64_t cap = kMaxWorkItems / 1024;
    hipLaunchKernelGGL((k_forward_long<X, W>), dim3(static_cast<unsigned>(a.rows < cap ? a.rows : cap)), dim3(1024), 0,
                       stream, x, a.ldx, w, b, a.eps, y, a.ldy, a.stats, a.rows, a.cols);
    return;
  }
  with_forward_shape(a.cols, [&](auto shape) {
    using S = decltype(shape);
    const int64_t steps = ceil_div(a.rows, S::rows), cap = 256 * (S::COUNT == 2 && S::LANES <= 256 ? 1280 : 2048) / S::threads;
    const dim3 grid(static_cast<unsigned>(steps < cap ? steps : cap));
    const auto kernel = a.eps < kLeastEps ? k_forward<S::COUNT == 2, double, S, X, W> : k_forward<S::COUNT == 2, float, S, X, W>;
    hipLaunchKernelGGL(kernel, grid, dim3(S::threads), 0, stream, x, a.ldx, w, b, a.eps, y, a.ldy, a.stats, a.rows,
                       a.cols);
  });
}

template <class X, class W>
void launch(const Backward& a, hipStream_t stream) {
  const X *const dy = static_cast<const X*>(a.dy), *const x = static_cast<const X*>(a.x);
  const W* const w = static_cast<const W*>(a.w);
  X* const dx = static_cast<X*>(a.dx);
  if (a.cols > kRowWidth) {
    const int strips = static_cast<int>(ceil_div(a.cols, 2048));
    if (a.parts)
      hipLaunchKernelGGL((k_params_long<X>), dim3(static_cast<unsigned>(strips * a.count)), dim3(256), 0, stream, dy,
                         a.lddy, x, a.ldx, a.stats, a.parts, a.rows, a.cols, strips);
    const int64_t cap = kMaxWorkItems / 1024;
    if (dx)
      hipLaunchKernelGGL((k_backward_long<X, W>), dim3(static_cast<unsigned>(a.rows < cap ? a.rows : cap)), dim3(1024), 0,
                         stream, dy, a.lddy, x, a.ldx, a.stats, w, dx, a.lddx, a.rows, a.cols);
    return;
  }
  with_backward_shape(a.cols, [&](auto shape) {
    using S = decltype(shape);
    if (few_rows(a.rows, a.cols)) {
      const int rows = dx ? static_cast<int>(ceil_div(a.rows, S::rows)) : 0;
      const int columns = a.dw || a.db ? static_cast<int>(ceil_div(a.cols, 64)) : 0;
      const auto go = [&](int row_blocks, int blocks) {
        if (blocks > 0)
          hipLaunchKernelGGL((k_few<S, X, W>), dim3(blocks), dim3(S::threads), 0, stream, dy, a.lddy, x, a.ldx, a.stats, w,
                             dx, a.lddx, a.dw, a.db, a.accumulate, a.rows, a.cols, row_blocks);
      };
      if (dx != dy && dx != x) {
        go(rows, rows + columns);
      } else {
        go(0, columns);
        go(rows, rows);
      }
      return;
    }
    const auto kernel = even<S>(a.cols) ? k_backward<S::COUNT == 2, S, X, W> : k_backward<false, S, X, W>;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(a.count)), dim3(S::threads), 0, stream, dy,
                       a.lddy, x, a.ldx, a.stats, w, dx, a.lddx, a.parts, a.rows, a.cols);
  });
}

// w and b of X's type, or floats.
template <class A>
void launch_type(int type, int w_type, const A& a, hipStream_t stream) {
  const bool wide = w_type == HIP_LAYERNORM_F32;
  if (type == HIP_LAYERNORM_F32) launch<float, float>(a, stream);
  else if (type == HIP_LAYERNORM_BF16 && wide) launch<bf16, float>(a, stream);
  else if (type == HIP_LAYERNORM_BF16) launch<bf16, bf16>(a, stream);
  else if (wide) launch<_Float16, float>(a, stream);
  else launch<_Float16, _Float16>(a, stream);
}

bool bad_param(int t, int type) { return t != HIP_LAYERNORM_F32 && t != type; }
bool bad_type(int t) { return t != HIP_LAYERNORM_F32 && t != HIP_LAYERNORM_BF16 && t != HIP_LAYERNORM_F16; }

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" {

int hip_layernorm_forward(int rows, int cols, int type, const void* X, int ldx, const void* w, const void* b, int w_type,
                          float eps, void* Y, int ldy, float* stats, hipStream_t stream) {
  if (rows < 0) return -1;
  if (cols < 0) return -2;
  const bool some = rows > 0 && cols > 0;
  if (bad_type(type)) return -3;
  if (some && X == nullptr) return -4;
  if (ldx < (cols > 1 ? cols : 1)) return -5;
  const bool params = w != nullptr || b != nullptr;
  if (params && bad_param(w_type, type)) return -8;
  if (!(eps >= 0.0f)) return -9;
  if (some && Y == nullptr) return -10;
  if (ldy < (cols > 1 ? cols : 1)) return -11;
  if (!some) return 0;
  launch_type(type, params ? w_type : HIP_LAYERNORM_F32, Forward{rows, cols, X, ldx, w, b, eps, Y, ldy, stats}, stream);
  return static_cast<int>(hipGetLastError());
}

int hip_layernorm_backward_workspace(int rows, int cols, long long* bytes) {
  if (rows < 0) return -1;
  if (cols < 0) return -2;
  if (bytes) *bytes = rows > 0 && cols > 0 ? parts_of(rows, cols) * 2 * cols * 4 : 0;
  return 0;
}

int hip_layernorm_backward(int rows, int cols, int type, const void* DY, int lddy, const void* X, int ldx,
                           const float* stats, const void* w, int w_type, void* DX, int lddx, float* dw, float* db,
                           int accumulate, void* workspace, long long workspace_bytes, hipStream_t stream) {
  if (rows < 0) return -1;
  if (cols < 0) return -2;
  const bool some = rows > 0 && cols > 0, params = dw != nullptr || db != nullptr;
  if (bad_type(type)) return -3;
  if (some && DY == nullptr) return -4;
  if (lddy < (cols > 1 ? cols : 1)) return -5;
  if (some && X == nullptr) return -6;
  if (ldx < (cols > 1 ? cols : 1)) return -7;
  if (some && stats == nullptr) return -8;
  if (w != nullptr && bad_param(w_type, type)) return -10;
  if (DX != nullptr && lddx < (cols > 1 ? cols : 1)) return -12;
  if (dw != nullptr && db != nullptr) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(dw), b = reinterpret_cast<uintptr_t>(db);
    if ((a < b ? b - a : a - b) < static_cast<uintptr_t>(cols) * 4) return -14;
  }
  if (accumulate != 0 && accumulate != 1) return -15;
  const int64_t count = some ? parts_of(rows, cols) : 0;
  if (some && params && count > 0 && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 16 != 0)) return -16;
  if (some && params && workspace_bytes < count * 2 * cols * 4) return -17;
  if (cols == 0 || (!params && (rows == 0 || DX == nullptr))) return 0;
  if (rows > 0) {
    launch_type(type, w != nullptr ? w_type : HIP_LAYERNORM_F32,
                Backward{rows, cols, DY, lddy, X, ldx, stats, w, DX, lddx, dw, db, accumulate,
                         params ? static_cast<float*>(workspace) : nullptr, static_cast<int>(count)},
                stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return static_cast<int>(e);
  }
  if (params && (rows == 0 || count > 0))
    hipLaunchKernelGGL(k_join, dim3(static_cast<unsigned>(min(ceil_div(cols, 32), kJoinBlocks)), 2), dim3(1024), 0, stream,
                       static_cast<const float*>(workspace), static_cast<int>(count), dw, db, cols, accumulate);
  return static_cast<int>(hipGetLastError());
}

const char* hip_layernorm_forward_status_string(int status) {
  switch (status) {
    case 0: return "success";
    case -1: return "argument 1 (rows) is negative";
    case -2: return "argument 2 (cols) is negative";
    case -3: return "argument 3 (type) is not a known type";
    case -4: return "argument 4 (X) is NULL";
    case -5: return "argument 5 (ldx) is smaller than max(1, cols)";
    case -8: return "argument 8 (w_type) is neither HIP_LAYERNORM_F32 nor the type of X";
    case -9: return "argument 9 (eps) is negative or NaN";
    case -10: return "argument 10 (Y) is NULL";
    case -11: return "argument 11 (ldy) is smaller than max(1, cols)";
    default: break;
  }
  if (status > 0) return hipGetErrorString(static_cast<hipError_t>(status));
  return "unknown status";
}

const char* hip_layernorm_backward_status_string(int status) {
  switch (status) {
    case 0: return "success";
    case -1: return "argument 1 (rows) is negative";
    case -2: return "argument 2 (cols) is negative";
    case -3: return "argument 3 (type) is not a known type";
    case -4: return "argument 4 (DY) is NULL";
    case -5: return "argument 5 (lddy) is smaller than max(1, cols)";
    case -6: return "argument 6 (X) is NULL";
    case -7: return "argument 7 (ldx) is smaller than max(1, cols)";
    case -8: return "argument 8 (stats) is NULL";
    case -10: return "argument 10 (w_type) is neither HIP_LAYERNORM_F32 nor the type of X";
    case -12: return "argument 12 (lddx) is smaller than max(1, cols)";
    case -14: return "argument 14 (db) overlaps argument 13 (dw)";
    case -15: return "argument 15 (accumulate) is not 0 or 1";
    case -16: return "argument 16 (workspace) is NULL or not 16-byte aligned";
    case -17: return "argument 17 (workspace_bytes) is less than hip_layernorm_backward_workspace says";
    default: break;
  }
  if (status > 0) return hipGetErrorString(static_cast<hipError_t>(status));
  return "unknown status";
}

}  // extern "C"

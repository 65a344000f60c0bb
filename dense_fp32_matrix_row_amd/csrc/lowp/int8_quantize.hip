// int8_quantize.hip -- hip_int8_quantize: the rows of a matrix into 8-bit integers
// with a scale each.
//
// Bound by memory: e bytes read and one written per element, against some twelve
// vector instructions.
#include "../../../include/int8.h"
#include "int8_codes.h"
#include "int8_internal.h"
#include "rows.h"

namespace sgemm {
namespace {

using namespace int8;

using Narrowest = RowShape<16, 1>;

// Calls f with the shape that takes rows of `cols` (at most kRowWidth).  Lanes that
// share a row in a wavefront need no barrier, and more rows in a block keep more
// loads under way; longer rows take more lanes before more registers, up to 512 (8192 x
// 8192 bf16 with 256 lanes and four chunks 45 us, with 512 and two 42; 4096 x 16384 with
// 1024 and two 49, with 512 and four 42).
template <class F>
void with_row_shape(int cols, const F& f) {
  if (cols <= 128) f(Narrowest{});
  else if (cols <= 256) f(RowShape<32, 1>{});
  else if (cols <= 512) f(RowShape<64, 1>{});
  else if (cols <= 1024) f(RowShape<64, 2>{});
  else if (cols <= 2048) f(RowShape<256, 1>{});
  else if (cols <= 4096) f(RowShape<256, 2>{});
  else if (cols <= 8192) f(RowShape<512, 2>{});
  else f(RowShape<512, 4>{});
}

// A row in the registers of its lanes: read once.  The lane that reaches over the row's
// end takes the last eight instead (WIDE), codes that its neighbour has too and writes
// alike, so that no load has a branch around it, behind which the compiler would wait; a
// row of fewer than eight, of the narrowest shape only, has none.
// One MI355X, kernels alone: 16 x 1024 bf16 2.9 us, 8192 x 8192 42 us (4.8 TB/s, what a
// large copy reaches; with branches 46), 8192 x 8191 42 (55), float32 63 (5.3 TB/s), 65536
// x 256 12.4, 4097 x 2049 float32 9.9 (13).  Blocks that walk the rows with the next one's
// loads under way take no less (42-45, float32 65-69).
template <bool WIDE, class S, class X>
__global__ __launch_bounds__(S::threads) void k_rows(const X* __restrict__ x, int64_t ldx, int8_t* __restrict__ q,
                                                     int64_t ldq, float* __restrict__ s, int rows, int cols) {
  __shared__ uint32_t meet[S::threads / 64][1];
  const int lane = threadIdx.x % S::LANES;
  const int64_t steps = ceil_div(rows, S::rows);
  for (int64_t step = blockIdx.x; step < steps; step += gridDim.x) {
    const int64_t row = step * S::rows + threadIdx.x / S::LANES;
    if (S::waves == 1 && row >= rows) return;
    Pack<8, X> v[S::COUNT];
    uint32_t top[1] = {0};
#pragma unroll
    for (int c = 0; c < S::COUNT; ++c) {
      const int col = (c * S::LANES + lane) * 8;
      v[c] = WIDE ? load_last8(x + row * ldx, col, cols) : load_row8(x + row * ldx, col, cols);
    }
#pragma unroll
    for (int c = 0; c < S::COUNT; ++c) top[0] = top8(top[0], v[c]);
    join_row<S>(top, meet, Max{});
    const Scale by = make_scale(top[0]);
#pragma unroll
    for (int c = 0; c < S::COUNT; ++c) {
      const int col = (c * S::LANES + lane) * 8;
      if constexpr (!WIDE) store_row8(q + row * ldq, col, cols, codes8(v[c], by));
      else if (col < cols) store_pack(q + row * ldq + min(col, cols - 8), codes8(v[c], by));
    }
    if (lane == 0) s[row] = by.s;
    if constexpr (S::waves > 1) __syncthreads();  // the next row writes the same LDS
  }
}

// Rows longer than registers hold: read twice (2048 x 32768 bf16 56 us).
template <class X>
__global__ __launch_bounds__(1024) void k_long(const X* __restrict__ x, int64_t ldx, int8_t* __restrict__ q,
                                               int64_t ldq, float* __restrict__ s, int rows, int cols) {
  using S = RowShape<1024, 1>;
  __shared__ uint32_t meet[S::threads / 64][1];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    uint32_t top[1] = {0};
    for (int64_t c = threadIdx.x * 8; c < cols; c += S::width)
      top[0] = top8(top[0], load_row8(x + row * ldx, static_cast<int>(c), cols));
    join_row<S>(top, meet, Max{});
    const Scale by = make_scale(top[0]);
    for (int64_t c = threadIdx.x * 8; c < cols; c += S::width)
      store_row8(q + row * ldq, static_cast<int>(c), cols, codes8(load_row8(x + row * ldx, static_cast<int>(c), cols), by));
    if (threadIdx.x == 0) s[row] = by.s;
    __syncthreads();
  }
}

template <class X>
void launch_type(int rows, int cols, const void* x, int64_t ldx, int8_t* q, int64_t ldq, float* s, hipStream_t stream) {
  const X* p = static_cast<const X*>(x);
  if (cols > kRowWidth) {
    const int64_t cap = kMaxWorkItems / 1024;
    const dim3 grid(static_cast<unsigned>(rows < cap ? rows : cap));
    hipLaunchKernelGGL((k_long<X>), grid, dim3(1024), 0, stream, p, ldx, q, ldq, s, rows, cols);
    return;
  }
  const auto go = [&](auto shape, const auto& kernel) {
    using S = decltype(shape);
    const int64_t steps = ceil_div(rows, S::rows), cap = kMaxWorkItems / S::threads;
    const dim3 grid(static_cast<unsigned>(steps < cap ? steps : cap));
    hipLaunchKernelGGL(kernel, grid, dim3(S::threads), 0, stream, p, ldx, q, ldq, s, rows, cols);
  };
  if (cols < 8) go(Narrowest{}, k_rows<false, Narrowest, X>);
  else with_row_shape(cols, [&](auto shape) { go(shape, k_rows<true, decltype(shape), X>); });
}

}  // namespace

void launch_int8_quantize(int rows, int cols, const void* x, int x_type, int64_t ldx, int8_t* q, int64_t ldq, float* s,
                          hipStream_t stream) {
  if (x_type == HIP_INT8_F32) launch_type<float>(rows, cols, x, ldx, q, ldq, s, stream);
  else if (x_type == HIP_INT8_BF16) launch_type<bf16>(rows, cols, x, ldx, q, ldq, s, stream);
  else launch_type<_Float16>(rows, cols, x, ldx, q, ldq, s, stream);
}

}  // namespace sgemm

using namespace sgemm;

extern "C" {

int hip_int8_quantize(int rows, int cols, const void* X, int x_type, int ldx, void* Q, int ldq, float* S,
                      hipStream_t stream) {
  if (rows < 0) return -1;
  if (cols < 0) return -2;
  const bool some = rows > 0 && cols > 0;
  if (some && X == nullptr) return -3;
  if (x_type != HIP_INT8_F32 && x_type != HIP_INT8_BF16 && x_type != HIP_INT8_F16) return -4;
  if (ldx < (cols > 1 ? cols : 1)) return -5;
  if (some && Q == nullptr) return -6;
  if (ldq < (cols > 1 ? cols : 1)) return -7;
  if (some && S == nullptr) return -8;
  if (!some) return 0;
  launch_int8_quantize(rows, cols, X, x_type, ldx, static_cast<int8_t*>(Q), ldq, S, stream);
  return static_cast<int>(hipGetLastError());
}

const char* hip_int8_quantize_status_string(int status) {
  switch (status) {
    case 0: return "success";
    case -1: return "argument 1 (rows) is negative";
    case -2: return "argument 2 (cols) is negative";
    case -3: return "argument 3 (X) is NULL";
    case -4: return "argument 4 (x_type) is not a known type";
    case -5: return "argument 5 (ldx) is smaller than max(1, cols)";
    case -6: return "argument 6 (Q) is NULL";
    case -7: return "argument 7 (ldq) is smaller than max(1, cols)";
    case -8: return "argument 8 (S) is NULL";
    default: break;
  }
  if (status > 0) return hipGetErrorString(static_cast<hipError_t>(status));
  return "unknown status";
}

}  // extern "C"

// fp8_gemm.hip -- hip_fp8_gemm: D = alpha A B^T + beta C over e4m3 operands with
// a scale for each block of 128 along K.
#include "../../../include/blockfp8.h"
#include "lowp.h"
#include "nt_loop.h"
#include "nt_plan.h"

namespace sgemm {
namespace {

using nt::Plan;
using nt::Side;
using nt::v4f;
using nt::Way;

template <class O>
struct Out {
  O* d;
  const O* c;
  int64_t ldd, ldc;
  int M, N;
  float alpha, beta;
  // C's COUNT neighbours of row m from column n, those inside; WHOLE: all are.
  // (Ends are compared as N - COUNT: n + COUNT passes 2^31 for the widest D.)
  template <bool WHOLE, int COUNT>
  __device__ __forceinline__ Pack<COUNT, O> old(int m, int n) const {
    Pack<COUNT, O> o{};
    if (!WHOLE && (m >= M || n >= N)) return o;
    const O* const from = c + m * ldc + n;
    if (WHOLE || n <= N - COUNT) return load_pack<COUNT>(from);
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
      if (n + i < N) o.v[i] = from[i];
    return o;
  }
  // D's, of their sums and of C's where ADD.
  template <bool WHOLE, bool ADD, int COUNT>
  __device__ __forceinline__ void put(int m, int n, const float (&v)[COUNT], const Pack<COUNT, O>& o) const {
    if (!WHOLE && (m >= M || n >= N)) return;
    O* const to = d + m * ldd + n;
    Pack<COUNT, O> r;
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      float x = alpha * v[i];
      if (ADD) x = fmaf(beta, to_float(o.v[i]), x);
      from_float(x, r.v[i]);
    }
    if (WHOLE || n <= N - COUNT) {
      store_pack(to, r);
    } else {
#pragma unroll
      for (int i = 0; i < COUNT; ++i)
        if (n + i < N) to[i] = r.v[i];
    }
  }
  template <bool WHOLE, bool ADD, int COUNT>
  __device__ __forceinline__ void row(int m, int n, const float (&v)[COUNT]) const {
    Pack<COUNT, O> o{};
    if (ADD) o = old<WHOLE, COUNT>(m, n);
    put<WHOLE, ADD>(m, n, v, o);
  }
  __device__ __forceinline__ void operator()(int m, int n, v4f v) const {
    const float x[4] = {v[0], v[1], v[2], v[3]};
    if (beta == 0.0f) row<false, false>(m, n, x);
    else row<false, true>(m, n, x);
  }
  // f with what of a rows x cols tile at m0, n0 is known beforehand.
  template <class F>
  __device__ __forceinline__ void tile(int m0, int n0, int rows, int cols, const F& f) const {
    const bool whole = m0 <= M - rows && n0 <= N - cols;
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    if (beta == 0.0f) {
      if (whole) f(yes, no);
      else f(no, no);
    } else {
      if (whole) f(yes, yes);
      else f(no, yes);
    }
  }
};

// Large tiles.  On one MI355X, kernels alone: 4096^3 with float scales 58-61 us
// (2300 TFLOP/s; each product's vector instructions of scaling take issue slots
// beside the matrix instruction; 68 where B has a scale a row, two instructions a
// result), 8192^3 with power-of-two scales, which need none, 381-476 us (2310-2890
// TFLOP/s, the clock down to about 1.75 GHz: power; MfmaUtil 77 %), 4096^3 with a
// float result 117-134 us (1030-1170 TFLOP/s; 276 vector instructions a wavefront and
// step widen and scale beside 64 matrix ones, and more than two a matrix instruction
// take its time: four make 7.5 ns 11.8).
template <class L, class O>
__global__ __launch_bounds__(L::threads, 2) void k_loop(Side A, Side B, int K, Out<O> out, int tiles_m, int tiles_n) {
  __shared__ alignas(16) uint8_t smem[L::kLds];
  const nt::Place at = nt::place_of(xcd_contiguous(blockIdx.x, gridDim.x), tiles_m, tiles_n, 8);
  const int m0 = at.tm * L::BM, n0 = at.tn * L::BN;
  nt::v16f acc[L::kAcc];
  nt::loop_sum<L>(smem, A, B, m0, n0, K, acc);
  // By way of LDS, so that whole lines are written (16-bit results of 4096^3: 61 ->
  // 60 us; float ones with C read, 4097^3 159 -> 153, 8000 x 8000 x 1000 205 -> 191).
  using Sheet = nt::Sheet<L::BN>;
  static_assert(sizeof(Sheet) <= L::kLds, "a sheet fits");
  Sheet& sheet = *reinterpret_cast<Sheet*>(smem);
  __syncthreads();  // all wavefronts have left the loop
  if constexpr (sizeof(O) == 4) {
    constexpr int kRow = L::BN / 4, kTurns = 64 * kRow / L::threads;
    out.tile(m0, n0, L::BM, L::BN, [&](auto whole, auto add) {
      nt::loop_sheets<L>(sheet, acc, [&](int top) {
        // all of C first: it may be D, so a load would wait for the stores before it
        // (8000 x 8000 x 1000 223 -> 200 us)
        Pack<4, O> old[kTurns];
        if (add.value) {
#pragma unroll
          for (int i = 0; i < kTurns; ++i) {
            const int t = threadIdx.x + i * L::threads;
            old[i] = out.template old<whole.value, 4>(m0 + top + t / kRow, n0 + t % kRow * 4);
          }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
          const int t = threadIdx.x + i * L::threads;
          float x[4];
          __builtin_memcpy(x, &sheet.v[t / kRow * Sheet::kLd + t % kRow * 4], 16);
          out.template put<whole.value, add.value>(m0 + top + t / kRow, n0 + t % kRow * 4, x, old[i]);
        }
        __syncthreads();
      });
    });
  } else {
    out.tile(m0, n0, L::BM, L::BN, [&](auto whole, auto add) {
      nt::loop_sheets<L>(sheet, acc, [&](int top) {
        sheet.template out<L::threads>(
            false, [&](int r, int c, const float (&v)[8]) { out.template row<whole.value, add.value>(m0 + top + r, n0 + c, v); },
            [](int, int, const float (&)[8]) {});
      });
    });
  }
}

template <class L, class O>
void launch_loop(const Side& A, const Side& B, int K, const Out<O>& out, unsigned blocks, hipStream_t s) {
  const int64_t tm = ceil_div(out.M, L::BM), tn = ceil_div(out.N, L::BN);
  hipLaunchKernelGGL((k_loop<L, O>), dim3(blocks), dim3(L::threads), 0, s, A, B, K, out, static_cast<int>(tm),
                     static_cast<int>(tn));
}

// Small tiles.  Bound by a launch and one trip to memory, or the weight's read:
// 1 x 4096 x 4096 in 4.4-5.3 us (3.2-3.8 TB/s; 16 x 16 tiles, 256 blocks), 256 x
// 1024 x 1024 in 4.3-5.1 us (32 x 32, 256 blocks).  The 64 x 64 tile is short of
// registers: with a scale for each row of B, and for float results with any, some
// of 13 to 73 registers that do not fit come and go in the loop (1024 x 1024 x 4096
// bf16 15 us with one scale for B's rows or powers of two, 22 with a float each;
// float 19-21, 31 and 46).
//
// Which tile takes a product, by estimates of the time in us: of a small tile
// what a launch takes, what one of its wavefronts' steps takes alone, and what a
// step of one block takes among many; of a large one what a step takes alone and
// in a full round over the 256 CUs.  The constants are fitted.  Of 160 products
// measured since (20 sizes from 1 x 4096 x 4096 to 8192^3, 16-bit and float
// results, both scales, B in blocks of 1 and 128) four in five took between 0.8
// and 1.25 of the estimate; 1024 x 1024 x 32768 mostly less (from 0.46), 64 x 64
// tiles with scales for rows of B more (up to 1.8).
struct Model {
  bool wide;  // a float result

  nt::SmallCost small(int i) const {
    if (i == 0) return {2.8, 0.45, 0.003};
    if (i == 1) return {2.3, 1.3, wide ? 0.007 : 0.0056};
    if (wide) return {2.0, 4.5, 0.024};
    return {3.0, 2.2, 0.0135};
  }
  template <class F>
  void loops(int M, int N, double steps, const F& offer) const {
    const auto loop = [&](Way w, int bn, double base, double alone, double full) {
      const int64_t tiles = ceil_div(M, 256) * ceil_div(N, bn), rest = tiles % 256;
      if (tiles > kMaxWorkItems / 512) return;  // a block a tile: more than a launch takes
      offer(w, base + steps * (tiles / 256 * full + (rest ? alone + (full - alone) * rest / 256 : 0)));
    };
    if (wide) {  // two blocks a CU: with one each, a step takes little more than half the time
      const int64_t tiles = ceil_div(M, 128) * ceil_div(N, 128), rest = tiles % 512;
      if (tiles <= kMaxWorkItems / 256)
        offer(Way::kLoop128, 5.0 + steps * (tiles / 512 * 1.92 + (rest == 0 ? 0 : rest <= 256 ? 1.09 : 1.92)));
    } else {
      loop(Way::kLoop128, 128, 6.0, 0.65, 0.98);
      loop(Way::kLoop256, 256, 7.0, 1.0, 1.6);
    }
  }
  bool cuts_rows(int t) const { return wide || t == 256; }
  constexpr nt::TileShape shape(Way way) const {
    switch (way) {
      case Way::kSmall16: return {16, 16, 512};
      case Way::kSmall32: return {32, 32, 512};
      case Way::kSmall64: return {64, 64, 512};
      case Way::kLoop128: return wide ? nt::TileShape{128, 128, 256} : nt::TileShape{256, 128, 512};
      default: return {256, 256, 512};
    }
  }
};

template <class P, nt::Kind KIND, class O>
void launch(const Side& A, const Side& B, int K, const Out<O>& out, hipStream_t s) {
  constexpr bool wide = sizeof(O) == 4;
  // 256 x 128 of eight wavefronts; for float results 128 x 128 of four, two blocks a
  // CU, so that one widens while the other multiplies and results leave meanwhile:
  // as fast as 256 x 128 where there are many (4096^3 127 and 130 us, 8000 x 8000 x
  // 1000 167 and 156), and fewer are needed (2048 x 2048 x 4096 55 and 39, 1500 x
  // 1500 x 4096 84 and 41).  With 8-bit instructions the loads to LDS, a third more
  // a product, would bound it.
  using Loop128 = nt::Loop<KIND, 4, 4, wide ? 2 : 4, 2, wide ? 2 : 3>;
  using Loop256 = nt::Loop<KIND, 8, 4, 2, 4, 2>;
  constexpr Model model{wide};
  using nt::is_shape;
  static_assert(is_shape<Loop128>(model.shape(Way::kLoop128)) && is_shape<Loop256>(model.shape(Way::kLoop256)) &&
                is_shape<nt::Direct<P, 1, 1, 8>>(model.shape(Way::kSmall16)) &&
                is_shape<nt::Direct<P, 2, 2, 8>>(model.shape(Way::kSmall32)) &&
                is_shape<nt::Direct<P, 4, 4, 8>>(model.shape(Way::kSmall64)));
  Plan p;
  plan(model, p, 0, 0, out.M, out.N, K, K > 0 && Loop128::fits(A) && Loop128::fits(B), nt::kCuts);
  for (int i = 0; i < p.count; ++i) {
    const nt::Piece& at = p.piece[i];
    Out<O> part = out;
    part.M = at.M;
    part.N = at.N;
    part.d += at.m0 * out.ldd + at.n0;
    if (out.beta != 0.0f) part.c += at.m0 * out.ldc + at.n0;
    const Side a = from_row(A, at.m0, P::kScaleBytes), b = from_row(B, at.n0, P::kScaleBytes);
    const unsigned blocks = static_cast<unsigned>(blocks_of(model, at));
    if (at.way <= Way::kSmall64) nt::launch_small<P>(at.way, a, b, K, part, at.skip_m, at.skip_n, blocks, s);
    else if (at.way == Way::kLoop128) launch_loop<Loop128>(a, b, K, part, blocks, s);
    else if constexpr (!wide) launch_loop<Loop256>(a, b, K, part, blocks, s);
  }
}

template <class O>
void launch_out(const Side& A, const Side& B, int K, int scale_type, const Out<O>& out, hipStream_t s) {
  using nt::Kind;
  const bool bytes = scale_type == HIP_FP8_SCALE_E8M0, uniform = B.shift != 0;
  if constexpr (sizeof(O) == 4) {
    // a float result: sums with a float's bits
    if (bytes && uniform) launch<nt::Widened<true, 1>, Kind::kWideE8M0Uniform>(A, B, K, out, s);
    else if (bytes) launch<nt::Widened<false, 1>, Kind::kWideE8M0Rows>(A, B, K, out, s);
    else if (uniform) launch<nt::Widened<true, 4>, Kind::kWideF32Uniform>(A, B, K, out, s);
    else launch<nt::Widened<false, 4>, Kind::kWideF32Rows>(A, B, K, out, s);
  } else if (bytes) {
    launch<nt::Fp8E8M0, Kind::kE8M0>(A, B, K, out, s);
  } else if (uniform) {
    launch<nt::Fp8F32<true>, Kind::kF32Uniform>(A, B, K, out, s);
  } else {
    launch<nt::Fp8F32<false>, Kind::kF32Rows>(A, B, K, out, s);
  }
}

bool bad_ld(int ld, int K) { return ld < (K > 1 ? K : 1) || ld % 16 != 0 || ld > HIP_FP8_MAX_LD; }
bool off16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" {

int hip_fp8_gemm(int M, int N, int K, float alpha, const void* A, int lda, const void* SA, long long sa_row,
                 long long sa_col, int a_block_rows, const void* B, int ldb, const void* SB, long long sb_row,
                 long long sb_col, int b_block_rows, int scale_type, float beta, const void* C, int ldc, void* D,
                 int ldd, int c_type, hipStream_t stream) {
  if (M < 0) return -1;
  if (N < 0) return -2;
  if (K < 0) return -3;
  const bool product = M > 0 && N > 0 && K > 0 && alpha != 0.0f;
  if (product && (A == nullptr || off16(A))) return -5;
  if (bad_ld(lda, K)) return -6;
  if (product && SA == nullptr) return -7;
  if (sa_row < 0) return -8;
  if (sa_col < 0) return -9;
  if (a_block_rows != 1 && a_block_rows != 128) return -10;
  if (product && (B == nullptr || off16(B))) return -11;
  if (bad_ld(ldb, K)) return -12;
  if (product && SB == nullptr) return -13;
  if (sb_row < 0) return -14;
  if (sb_col < 0) return -15;
  if (b_block_rows != 1 && b_block_rows != 128) return -16;
  if (scale_type != HIP_FP8_SCALE_F32 && scale_type != HIP_FP8_SCALE_E8M0) return -17;
  const bool some = M > 0 && N > 0;
  if (some && beta != 0.0f && C == nullptr) return -19;
  if (beta != 0.0f && ldc < (N > 1 ? N : 1)) return -20;
  if (some && D == nullptr) return -21;
  if (ldd < (N > 1 ? N : 1)) return -22;
  if (c_type != HIP_FP8_F32 && c_type != HIP_FP8_BF16 && c_type != HIP_FP8_F16) return -23;
  if (!some) return 0;
  const int k = product ? K : 0;
  if (k == 0) alpha = 0.0f;  // an empty sum times an infinity would be NaN
  const Side a{static_cast<const uint8_t*>(A), lda, M, SA, sa_row, sa_col, a_block_rows == 128 ? 7 : 0, 0};
  const Side b{static_cast<const uint8_t*>(B), ldb, N, SB, sb_row, sb_col, b_block_rows == 128 ? 7 : 0, 0};
  if (c_type == HIP_FP8_F32)
    launch_out(a, b, k, scale_type,
               Out<float>{static_cast<float*>(D), static_cast<const float*>(C), ldd, ldc, M, N, alpha, beta}, stream);
  else if (c_type == HIP_FP8_BF16)
    launch_out(a, b, k, scale_type,
               Out<bf16>{static_cast<bf16*>(D), static_cast<const bf16*>(C), ldd, ldc, M, N, alpha, beta}, stream);
  else
    launch_out(a, b, k, scale_type,
               Out<_Float16>{static_cast<_Float16*>(D), static_cast<const _Float16*>(C), ldd, ldc, M, N, alpha, beta},
               stream);
  return static_cast<int>(hipGetLastError());
}

int hip_fp8_gemm_plan(int M, int N, int K, int c_type, hip_fp8_gemm_launch* launches, int* count) {
  if (M < 0) return -1;
  if (N < 0) return -2;
  if (K < 0) return -3;
  if (c_type != HIP_FP8_F32 && c_type != HIP_FP8_BF16 && c_type != HIP_FP8_F16) return -23;
  Plan p;
  const bool wide = c_type == HIP_FP8_F32;
  const Model model{wide};
  if (M > 0 && N > 0) plan(model, p, 0, 0, M, N, K, K > 0, nt::kCuts);
  for (int i = 0; launches && i < p.count; ++i) {
    const nt::Piece& at = p.piece[i];
    const nt::TileShape t = model.shape(at.way);
    launches[i] = hip_fp8_gemm_launch{t.rows, t.cols, at.m0, at.n0, at.M, at.N, at.skip_m, at.skip_n, t.threads,
                                      blocks_of(model, at)};
  }
  if (count) *count = p.count;
  return 0;
}

const char* hip_fp8_gemm_status_string(int status) {
  switch (status) {
    case 0: return "success";
    case -1: return "argument 1 (M) is negative";
    case -2: return "argument 2 (N) is negative";
    case -3: return "argument 3 (K) is negative";
    case -5: return "argument 5 (A) is NULL or not 16-byte aligned";
    case -6: return "argument 6 (lda) is smaller than max(1, K), no multiple of 16, or above HIP_FP8_MAX_LD";
    case -7: return "argument 7 (SA) is NULL";
    case -8: return "argument 8 (sa_row) is negative";
    case -9: return "argument 9 (sa_col) is negative";
    case -10: return "argument 10 (a_block_rows) is not 1 or 128";
    case -11: return "argument 11 (B) is NULL or not 16-byte aligned";
    case -12: return "argument 12 (ldb) is smaller than max(1, K), no multiple of 16, or above HIP_FP8_MAX_LD";
    case -13: return "argument 13 (SB) is NULL";
    case -14: return "argument 14 (sb_row) is negative";
    case -15: return "argument 15 (sb_col) is negative";
    case -16: return "argument 16 (b_block_rows) is not 1 or 128";
    case -17: return "argument 17 (scale_type) is not a known type";
    case -19: return "argument 19 (C) is NULL but beta is not 0";
    case -20: return "argument 20 (ldc) is smaller than max(1, N)";
    case -21: return "argument 21 (D) is NULL";
    case -22: return "argument 22 (ldd) is smaller than max(1, N)";
    case -23: return "argument 23 (c_type) is not a known type";
    default: break;
  }
  if (status > 0) return hipGetErrorString(static_cast<hipError_t>(status));
  return "unknown status";
}

}  // extern "C"

// fp8_gemm.hip -- hip_fp8_gemm: D = alpha A B^T + beta C over e4m3 operands with
// a scale for each block of 128 along K.
#include "../../include/blockfp8.h"
#include "lowp.h"
#include "nt_loop.h"

namespace sgemm {
namespace {

using nt::Side;
using nt::v4f;

template <class O>
struct Out {
  O* d;
  const O* c;
  int64_t ldd, ldc;
  int M, N;
  float alpha, beta;
  template <bool ADD>
  __device__ __forceinline__ Pack<4, O> value(v4f v, const Pack<4, O>& o) const {
    Pack<4, O> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x = alpha * v[i];
      if (ADD) x = fmaf(beta, to_float(o.v[i]), x);
      from_float(x, r.v[i]);
    }
    return r;
  }
  // Four neighbours inside D, or across its edge.
  template <bool ADD>
  __device__ __forceinline__ void inside(int m, int n, v4f v) const {
    Pack<4, O> o{};
    if (ADD) o = load_pack<4>(c + m * ldc + n);
    store_pack(d + m * ldd + n, value<ADD>(v, o));
  }
  template <bool ADD>
  __device__ __forceinline__ void edge(int m, int n, v4f v) const {
    if (m >= M) return;
    Pack<4, O> o{};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (ADD && n + i < N) o.v[i] = c[m * ldc + n + i];
    const Pack<4, O> r = value<ADD>(v, o);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) d[m * ldd + n + i] = r.v[i];
  }
  // each: calls its argument with (m, n, v) for all that a thread holds of the
  // rows x cols tile at m0, n0.
  template <class F>
  __device__ __forceinline__ void tile(int m0, int n0, int rows, int cols, const F& each) const {
    const bool whole = m0 + rows <= M && n0 + cols <= N;
    if (beta == 0.0f) {
      if (whole) each([&](int m, int n, v4f v) { inside<false>(m, n, v); });
      else each([&](int m, int n, v4f v) { edge<false>(m, n, v); });
    } else {
      if (whole) each([&](int m, int n, v4f v) { inside<true>(m, n, v); });
      else each([&](int m, int n, v4f v) { edge<true>(m, n, v); });
    }
  }
};

template <class P, class T, class O>
__global__ __launch_bounds__(T::threads, T::WPS) void k_gemm(Side A, Side B, int K, Out<O> out, int tiles_m,
                                                             int tiles_n, int64_t tiles) {
  __shared__ nt::Shared<P, T> sh;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const nt::Place at = nt::place_of(xcd_contiguous(t, tiles), tiles_m, tiles_n, 8);
    nt::Sums<P, T> acc;
    nt::TileOp<P, T>::sum(sh, A, B, at.tm * T::BM, at.tn * T::BN, K, 0, static_cast<int>(ceil_div(K, nt::kStep)), acc);
    const int m0 = at.tm * T::BM, n0 = at.tn * T::BN;
    out.tile(m0, n0, T::BM, T::BN, [&](const auto& epi) { nt::TileOp<P, T>::out(acc, m0, n0, epi); });
    __syncthreads();  // the next tile writes the same LDS
  }
}

template <class P, class T, class O>
void launch_tile(const Side& A, const Side& B, int K, const Out<O>& out, hipStream_t s) {
  const int64_t tm = ceil_div(out.M, T::BM), tn = ceil_div(out.N, T::BN), tiles = tm * tn;
  const int64_t cap = kMaxWorkItems / T::threads;
  hipLaunchKernelGGL((k_gemm<P, T, O>), dim3(static_cast<unsigned>(tiles < cap ? tiles : cap)), dim3(T::threads), 0,
                     s, A, B, K, out, static_cast<int>(tm), static_cast<int>(tn), tiles);
}

template <class L, class O>
__global__ __launch_bounds__(L::threads, 2) void k_loop(Side A, Side B, int K, Out<O> out, int tiles_m, int tiles_n) {
  __shared__ alignas(16) uint8_t smem[L::kLds];
  const nt::Place at = nt::place_of(xcd_contiguous(blockIdx.x, gridDim.x), tiles_m, tiles_n, 8);
  const int m0 = at.tm * L::BM, n0 = at.tn * L::BN;
  nt::v16f acc[L::kAcc];
  nt::loop_sum<L>(smem, A, B, m0, n0, K, acc);
  out.tile(m0, n0, L::BM, L::BN, [&](const auto& epi) { nt::loop_out<L>(acc, m0, n0, epi); });
}

template <class L, class O>
void launch_loop(const Side& A, const Side& B, int K, const Out<O>& out, hipStream_t s) {
  const int64_t tm = ceil_div(out.M, L::BM), tn = ceil_div(out.N, L::BN);
  hipLaunchKernelGGL((k_loop<L, O>), dim3(static_cast<unsigned>(tm * tn)), dim3(L::threads), 0, s, A, B, K, out,
                     static_cast<int>(tm), static_cast<int>(tn));
}

template <class P, class O>
void launch_policy(const Side& A, const Side& B, int K, const Out<O>& out, hipStream_t s) {
  using Small = nt::Tile<64, 64, 2, 2, 2>;
  using Large = nt::Tile<128, 128, 2, 2, 2>;
  if (ceil_div(out.M, 128) * ceil_div(out.N, 128) >= 256) launch_tile<P, Large>(A, B, K, out, s);
  else launch_tile<P, Small>(A, B, K, out, s);
}

template <class P, class L, class O>
void launch(const Side& A, const Side& B, int K, const Out<O>& out, hipStream_t s) {
  if (K > 0 && L::fits(A) && L::fits(B) && ceil_div(out.M, 128) * ceil_div(out.N, 128) >= 256)
    launch_loop<L>(A, B, K, out, s);
  else launch_policy<P>(A, B, K, out, s);
}

template <class O>
void launch_out(const Side& A, const Side& B, int K, int scale_type, const Out<O>& out, hipStream_t s) {
  using nt::Kind;
  if constexpr (sizeof(O) == 4) {
    // a float result: sums with a float's bits
    if (scale_type == HIP_FP8_SCALE_E8M0) {
      if (B.shift) launch<nt::Widened<true, 1>, nt::Loop<Kind::kWideE8M0Uniform, 4, 4, 4, 2>>(A, B, K, out, s);
      else launch<nt::Widened<false, 1>, nt::Loop<Kind::kWideE8M0Rows, 4, 4, 4, 2>>(A, B, K, out, s);
    } else {
      if (B.shift) launch<nt::Widened<true, 4>, nt::Loop<Kind::kWideF32Uniform, 4, 4, 4, 2>>(A, B, K, out, s);
      else launch<nt::Widened<false, 4>, nt::Loop<Kind::kWideF32Rows, 4, 4, 4, 2>>(A, B, K, out, s);
    }
  } else if (scale_type == HIP_FP8_SCALE_E8M0) launch<nt::Fp8E8M0, nt::Loop<Kind::kE8M0, 8, 4, 2, 4>>(A, B, K, out, s);
  else if (B.shift) launch<nt::Fp8F32<true>, nt::Loop<Kind::kF32Uniform, 8, 4, 2, 4>>(A, B, K, out, s);
  else launch<nt::Fp8F32<false>, nt::Loop<Kind::kF32Rows, 8, 4, 2, 4>>(A, B, K, out, s);
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

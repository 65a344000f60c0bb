// fp8_gemm.hip -- hip_fp8_gemm: D = alpha A B^T + beta C over e4m3 operands with
// a scale for each block of 128 along K.
#include "../../../include/blockfp8.h"
#include "lowp.h"
#include "nt_direct.h"
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

// The tiles from column n0, all rows; then those from row m0 left of it.
struct Part {
  int tiles_m, n0;
  int64_t tiles;
  int low_m, m0;
};

// Small tiles.  Bound by a launch and one trip to memory, or the weight's read:
// 1 x 4096 x 4096 in 4.4-5.3 us (3.2-3.8 TB/s; 16 x 16 tiles, 256 blocks), 256 x
// 1024 x 1024 in 4.3-5.1 us (32 x 32, 256 blocks).  The 64 x 64 tile is short of
// registers: with a scale for each row of B, and for float results with any, some
// of 13 to 73 registers that do not fit come and go in the loop (1024 x 1024 x 4096
// bf16 15 us with one scale for B's rows or powers of two, 22 with a float each;
// float 19-21, 31 and 46).
template <class D, class O>
__global__ __launch_bounds__(D::threads, 2) void k_direct(Side A, Side B, int K, Out<O> out, Part part, int64_t tiles) {
  __shared__ typename D::Meet meet;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t id = xcd_contiguous(t, tiles), low = id - part.tiles;
    const int m0 = low < 0 ? static_cast<int>(id % part.tiles_m) * D::BM : part.m0 + static_cast<int>(low % part.low_m) * D::BM;
    const int n0 = low < 0 ? part.n0 + static_cast<int>(id / part.tiles_m) * D::BN : static_cast<int>(low / part.low_m) * D::BN;
    D::run(meet, A, B, m0, n0, K, out);
    __syncthreads();  // the next tile writes the same LDS
  }
}

// Of D, what is neither left of column n0 nor above row m0, one launch for both
// edges (2050 x 2049 x 4096, float result: 51 -> 47 us); all of it for 0, 0.
template <class D, class O>
void launch_direct(const Side& A, const Side& B, int K, const Out<O>& out, int m0, int n0, unsigned blocks,
                   hipStream_t s) {
  Part part;
  const int64_t tm = ceil_div(out.M, D::BM), low = ceil_div(out.M - m0, D::BM);
  part.tiles_m = static_cast<int>(tm);
  part.n0 = n0;
  part.tiles = tm * ceil_div(out.N - n0, D::BN);
  part.low_m = static_cast<int>(low);
  part.m0 = m0;
  const int64_t tiles = part.tiles + low * (n0 / D::BN);
  hipLaunchKernelGGL((k_direct<D, O>), dim3(blocks), dim3(D::threads), 0, s, A, B, K, out, part, tiles);
}

// Which tile takes a product, by estimates of the time in us: of a small tile
// (16, 32 or 64 square) what a launch takes, what one of its wavefronts' steps
// takes alone, and what a step of one block takes among many; of a large one
// what a step takes alone and in a full round over the 256 CUs.  The constants are
// fitted.  Of 160 products measured since (20 sizes from 1 x 4096 x 4096 to 8192^3,
// 16-bit and float results, both scales, B in blocks of 1 and 128) four in five took
// between 0.8 and 1.25 of the estimate; 1024 x 1024 x 32768 mostly less (from 0.46),
// 64 x 64 tiles with scales for rows of B more (up to 1.8).
enum class Way { kSmall16, kSmall32, kSmall64, kLoop128, kLoop256, kRows, kColumns };
struct Choice {
  Way way;
  int at;  // kRows, kColumns: where D is cut in two
  double us;
};

Choice choose(int M, int N, int K, bool wide, bool loops, int cuts) {
  const double steps = static_cast<double>(ceil_div(K, nt::kStep)), each = static_cast<double>(ceil_div(K, 8 * nt::kStep));
  const auto small = [&](int t, double base, double alone, double among) {
    const double blocks = static_cast<double>(ceil_div(M, t) * ceil_div(N, t));
    return base + each * (alone > among * blocks ? alone : among * blocks);
  };
  Choice best{Way::kSmall16, 0, small(16, 2.8, 0.45, 0.003)};
  const auto offer = [&](Way w, int at, double us) {
    if (us < best.us) best = Choice{w, at, us};
  };
  const auto loop = [&](Way w, int bn, double base, double alone, double full) {
    const int64_t tiles = ceil_div(M, 256) * ceil_div(N, bn), rest = tiles % 256;
    if (tiles > kMaxWorkItems / 512) return;  // a block a tile: more than a launch takes
    offer(w, 0, base + steps * (tiles / 256 * full + (rest ? alone + (full - alone) * rest / 256 : 0)));
  };
  offer(Way::kSmall32, 0, small(32, 2.3, 1.3, wide ? 0.007 : 0.0056));
  offer(Way::kSmall64, 0, wide ? small(64, 2.0, 4.5, 0.024) : small(64, 3.0, 2.2, 0.0135));
  if (!loops) return best;
  if (wide) {  // two blocks a CU: with one each, a step takes little more than half the time
    const int64_t tiles = ceil_div(M, 128) * ceil_div(N, 128), rest = tiles % 512;
    if (tiles <= kMaxWorkItems / 256)
      offer(Way::kLoop128, 0, 5.0 + steps * (tiles / 512 * 1.92 + (rest == 0 ? 0 : rest <= 256 ? 1.09 : 1.92)));
  } else {
    loop(Way::kLoop128, 128, 6.0, 0.65, 0.98);
    loop(Way::kLoop256, 256, 7.0, 1.0, 1.6);
  }
  // rows or columns that hardly fill their tiles apart from the rest
  for (int t = 128; cuts > 0 && t <= 256; t *= 2) {
    if (N > t && N % t) {
      const int at = N - N % t;
      offer(Way::kColumns, at, choose(M, at, K, wide, loops, cuts - 1).us + choose(M, N - at, K, wide, loops, 0).us);
    }
    if ((wide || t == 256) && M > t && M % t) {
      const int at = M - M % t;
      offer(Way::kRows, at, choose(at, N, K, wide, loops, cuts - 1).us + choose(M - at, N, K, wide, loops, 0).us);
    }
  }
  return best;
}

// One launch: tiles of one kind (small or large) over rows m0 .. m0 + M - 1 and
// columns n0 .. n0 + N - 1 of D but, of small tiles, the first skip_m rows of the
// first skip_n columns.
struct Piece {
  Way way;
  int m0, n0, M, N, skip_m, skip_n;
};
// A product's launches; two cuts make three of them.
struct Plan {
  Piece piece[3];
  int count = 0;
};

void plan(Plan& p, int m0, int n0, int M, int N, int K, bool wide, bool loops, int cuts) {
  const Choice c = choose(M, N, K, wide, loops, cuts);
  if (c.way != Way::kRows && c.way != Way::kColumns) {
    p.piece[p.count++] = Piece{c.way, m0, n0, M, N, 0, 0};
    return;
  }
  const bool rows = c.way == Way::kRows;
  const Choice inner = choose(rows ? c.at : M, rows ? N : c.at, K, wide, loops, cuts - 1);
  if (inner.way == (rows ? Way::kColumns : Way::kRows)) {  // both edges, with small tiles of one size: these in one launch
    const int m = rows ? c.at : inner.at, n = rows ? inner.at : c.at;
    const Way right = choose(M, N - n, K, wide, loops, 0).way, low = choose(M - m, n, K, wide, loops, 0).way;
    if (right == low && right <= Way::kSmall64) {
      plan(p, m0, n0, m, n, K, wide, loops, 0);
      p.piece[p.count++] = Piece{right, m0, n0, M, N, m, n};
      return;
    }
  }
  if (rows) {
    plan(p, m0, n0, c.at, N, K, wide, loops, cuts - 1);
    plan(p, m0 + c.at, n0, M - c.at, N, K, wide, loops, 0);
  } else {
    plan(p, m0, n0, M, c.at, K, wide, loops, cuts - 1);
    plan(p, m0, n0 + c.at, M, N - c.at, K, wide, loops, 0);
  }
}
constexpr int kCuts = 2;

// Tile and block of a way.
struct TileShape {
  int rows, cols, threads;
};
constexpr TileShape shape_of(Way way, bool wide) {
  switch (way) {
    case Way::kSmall16: return TileShape{16, 16, 512};
    case Way::kSmall32: return TileShape{32, 32, 512};
    case Way::kSmall64: return TileShape{64, 64, 512};
    case Way::kLoop128: return wide ? TileShape{128, 128, 256} : TileShape{256, 128, 512};
    default: return TileShape{256, 256, 512};
  }
}

template <class T>
constexpr bool is_shape(Way way, bool wide) {
  const TileShape t = shape_of(way, wide);
  return t.rows == T::BM && t.cols == T::BN && t.threads == T::threads;
}

// Blocks of a launch: one a tile, but small tiles past what a launch takes, which
// the blocks walk.
int64_t blocks_of(const Piece& p, bool wide) {
  const TileShape t = shape_of(p.way, wide);
  const int64_t tiles = ceil_div(p.M, t.rows) * ceil_div(p.N - p.skip_n, t.cols) +
                        ceil_div(p.M - p.skip_m, t.rows) * (p.skip_n / t.cols);
  const int64_t cap = kMaxWorkItems / t.threads;
  return tiles < cap ? tiles : cap;
}

Side from_row(Side o, int row, int scale_bytes) {  // row: a multiple of 128
  o.p += row * o.ld;
  o.s = static_cast<const uint8_t*>(o.s) + (row >> o.shift) * o.s_row * scale_bytes;
  o.rows -= row;
  return o;
}

// The small tiles of a way, over the part of D that launch_direct takes.
template <class P, class O>
void launch_small(Way way, const Side& A, const Side& B, int K, const Out<O>& out, int m0, int n0, unsigned blocks,
                  hipStream_t s) {
  using nt::Direct;
  if (way == Way::kSmall16) launch_direct<Direct<P, 1, 1, 8>>(A, B, K, out, m0, n0, blocks, s);
  else if (way == Way::kSmall32) launch_direct<Direct<P, 2, 2, 8>>(A, B, K, out, m0, n0, blocks, s);
  else launch_direct<Direct<P, 4, 4, 8>>(A, B, K, out, m0, n0, blocks, s);
}

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
  static_assert(is_shape<Loop128>(Way::kLoop128, wide) && is_shape<Loop256>(Way::kLoop256, wide) &&
                is_shape<nt::Direct<P, 1, 1, 8>>(Way::kSmall16, wide) && is_shape<nt::Direct<P, 2, 2, 8>>(Way::kSmall32, wide) &&
                is_shape<nt::Direct<P, 4, 4, 8>>(Way::kSmall64, wide));
  Plan p;
  plan(p, 0, 0, out.M, out.N, K, wide, K > 0 && Loop128::fits(A) && Loop128::fits(B), kCuts);
  for (int i = 0; i < p.count; ++i) {
    const Piece& at = p.piece[i];
    Out<O> part = out;
    part.M = at.M;
    part.N = at.N;
    part.d += at.m0 * out.ldd + at.n0;
    if (out.beta != 0.0f) part.c += at.m0 * out.ldc + at.n0;
    const Side a = from_row(A, at.m0, P::kScaleBytes), b = from_row(B, at.n0, P::kScaleBytes);
    const unsigned blocks = static_cast<unsigned>(blocks_of(at, wide));
    if (at.way <= Way::kSmall64) launch_small<P>(at.way, a, b, K, part, at.skip_m, at.skip_n, blocks, s);
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
  if (M > 0 && N > 0) plan(p, 0, 0, M, N, K, wide, K > 0, kCuts);
  for (int i = 0; launches && i < p.count; ++i) {
    const Piece& at = p.piece[i];
    const TileShape t = shape_of(at.way, wide);
    launches[i] = hip_fp8_gemm_launch{t.rows, t.cols, at.m0, at.n0, at.M, at.N, at.skip_m, at.skip_n, t.threads,
                                      blocks_of(at, wide)};
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

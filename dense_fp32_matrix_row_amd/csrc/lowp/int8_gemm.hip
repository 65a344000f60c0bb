// int8_gemm.hip -- hip_int8_gemm: D = A B^T, scaled by a float for each row of A
// and of B, plus a bias, over 8-bit integers; hip_int8_linear: the quantiser and
// that product.
#include "../../../include/int8.h"
#include "int8_codes.h"
#include "int8_internal.h"
#include "lowp.h"
#include "nt_loop.h"
#include "nt_plan.h"
#include "rows.h"

namespace sgemm {
namespace {

using nt::Plan;
using nt::Side;
using nt::v4f;
using nt::v4i;
using nt::Way;

// The bias of COUNT neighbours from column n; those inside.
struct Bias {
  const void* p;
  int type;
  template <class T, int COUNT>
  __device__ __forceinline__ void load(float (&b)[COUNT], int n, int N) const {
    const T* const from = static_cast<const T*>(p) + n;
    if (n <= N - COUNT) {
      const Pack<COUNT, T> v = load_pack<COUNT>(from);
#pragma unroll
      for (int i = 0; i < COUNT; ++i) b[i] = to_float(v.v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < COUNT; ++i) b[i] = n < N - i ? to_float(from[i]) : 0.0f;
    }
  }
  template <int COUNT>
  __device__ __forceinline__ void get(float (&b)[COUNT], int n, int N) const {
    if (type == HIP_INT8_F32) load<float>(b, n, N);
    else if (type == HIP_INT8_BF16) load<bf16>(b, n, N);
    else load<_Float16>(b, n, N);
  }
  Bias from(int n) const {
    if (!p) return *this;
    return Bias{static_cast<const uint8_t*>(p) + int64_t(n) * (type == HIP_INT8_F32 ? 4 : 2), type};
  }
};

template <class O>
struct Out {
  O* d;
  int64_t ldd;
  int M, N;
  const float* sa;
  int64_t sa_inc;
  const float* sb;
  int64_t sb_inc;
  Bias bias;

  // What COUNT neighbours of a row from column n take: their scales and biases, those
  // inside.  (Ends are compared as N - COUNT: n + COUNT passes 2^31 for the widest D.)
  template <int COUNT>
  struct Columns {
    float scale[COUNT], bias[COUNT];
  };
  template <int COUNT>
  __device__ __forceinline__ Columns<COUNT> columns(int n) const {
    Columns<COUNT> c;
    if (sb_inc == 1 && n <= N - COUNT) {
      __builtin_memcpy(c.scale, sb + n, sizeof(c.scale));
    } else {
#pragma unroll
      for (int i = 0; i < COUNT; ++i) c.scale[i] = n < N - i ? sb[(n + i) * sb_inc] : 0.0f;
    }
    if (bias.p && n < N) {
      bias.get(c.bias, n, N);
    } else {
#pragma unroll
      for (int i = 0; i < COUNT; ++i) c.bias[i] = 0.0f;
    }
    return c;
  }
  // D's COUNT neighbours of row m, whose scale is s, from column n, those inside, of their sums.
  template <int COUNT>
  __device__ __forceinline__ void row(int m, int n, const float (&v)[COUNT], float s, const Columns<COUNT>& c) const {
    if (m >= M || n >= N) return;
    Pack<COUNT, O> r;
    if (bias.p) {
#pragma unroll
      for (int i = 0; i < COUNT; ++i) from_float(fmaf(v[i] * s, c.scale[i], c.bias[i]), r.v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < COUNT; ++i) from_float(v[i] * s * c.scale[i], r.v[i]);
    }
    O* const to = d + m * ldd + n;
    if (n <= N - COUNT) {
      store_pack(to, r);
    } else {
#pragma unroll
      for (int i = 0; i < COUNT; ++i)
        if (n < N - i) to[i] = r.v[i];
    }
  }
  __device__ __forceinline__ float row_scale(int m) const { return m < M ? sa[m * sa_inc] : 0.0f; }
  __device__ __forceinline__ void operator()(int m, int n, v4i v) const {
    if (m >= M || n >= N) return;
    const float x[4] = {static_cast<float>(v[0]), static_cast<float>(v[1]), static_cast<float>(v[2]),
                        static_cast<float>(v[3])};
    row(m, n, x, row_scale(m), columns<4>(n));
  }
  Out from(int m0, int n0, int rows, int cols) const {
    Out o = *this;
    o.d += m0 * ldd + n0;
    o.M = rows;
    o.N = cols;
    o.sa += m0 * sa_inc;
    o.sb += n0 * sb_inc;
    o.bias = bias.from(n0);
    return o;
  }
};

// Large tiles.  On one MI355X, kernels alone: 4096^3 61.5 us (2230 TOP/s), 8192^3 434-444
// (2480-2530; the library's int8 product 63.5 and 441), 2048^3 15 (128 x 128 tiles, 256 of
// them; 256 x 128 19), 512 x 4096 x 4096 18.7 (27).  A step of 256 x 256 takes 1.53 us,
// 1.05 without its loads to LDS, 1.39 without its matrix instructions: 64 KB a step and
// CU, with two stages to be under way in, bound it, and power (the clock at 1.7 GHz,
// matrix pipes 67 % busy at 8192^3).  32 x 32 x 32 instructions give less at the same
// power (from registers alone 3500 TOP/s against 4120).
//
// The K loop in assembly, results by way of LDS as floats, so that whole
// lines are written.  A thread stores the same columns of every row, so their scales
// and biases, and its rows' scales, are read once, all together, behind the loop (read
// for each eight results they cost a trip to memory each: 4096 x 4096 x 1024 31 -> 27 us).
template <class L, class O>
__global__ __launch_bounds__(L::threads, 2) void k_loop(Side A, Side B, int K, Out<O> out, int tiles_m, int tiles_n) {
  __shared__ alignas(16) uint8_t smem[L::kLds];
  const nt::Place at = nt::place_of(xcd_contiguous(blockIdx.x, gridDim.x), tiles_m, tiles_n, 8);
  const int m0 = at.tm * L::BM, n0 = at.tn * L::BN;
  nt::v16f acc[L::kAcc];
  nt::loop_sum<L>(smem, A, B, m0, n0, K, acc);
  constexpr int kRow = L::BN / 8, kStep = L::threads / kRow, kTurns = 64 / kStep;
  static_assert(L::threads % kRow == 0 && 64 % kStep == 0);
  const int col = threadIdx.x % kRow * 8, first = threadIdx.x / kRow;
  float scale[L::BM / 64][kTurns];
#pragma unroll
  for (int s = 0; s < L::BM / 64; ++s)
#pragma unroll
    for (int t = 0; t < kTurns; ++t) scale[s][t] = out.row_scale(m0 + 64 * s + first + t * kStep);
  const typename Out<O>::template Columns<8> columns = out.template columns<8>(n0 + col);
#pragma unroll
  for (int i = 0; i < L::kAcc; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][r] = static_cast<float>(__float_as_int(acc[i][r]));
  using Sheet = nt::Sheet<L::BN>;
  static_assert(sizeof(Sheet) <= L::kLds, "a sheet fits");
  Sheet& sheet = *reinterpret_cast<Sheet*>(smem);
  __syncthreads();  // all wavefronts have left the loop
  nt::loop_sheets<L>(sheet, acc, [&](int top) {
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
      const int r = first + t * kStep;
      float x[8];
      __builtin_memcpy(x, &sheet.v[r * Sheet::kLd + col], 32);
      out.row(m0 + top + r, n0 + col, x, scale[top / 64][t], columns);
    }
    __syncthreads();
  });
}

template <class L, class O>
void launch_loop(const Side& A, const Side& B, int K, const Out<O>& out, unsigned blocks, hipStream_t s) {
  const int64_t tm = ceil_div(out.M, L::BM), tn = ceil_div(out.N, L::BN);
  hipLaunchKernelGGL((k_loop<L, O>), dim3(blocks), dim3(L::threads), 0, s, A, B, K, out, static_cast<int>(tm),
                     static_cast<int>(tn));
}

// Which tile takes a product, by estimates of the time in us, whose constants are
// fitted to 64 sizes from 16 x 4096 x 4096 to 8192^3: of a small tile as SmallCost
// has it, of a large one a launch, and of each round over the 256 CUs what its tiles'
// start and end take, which nothing hides, and its steps, a round of few tiles
// sharing the loads' way with fewer.
struct Model {
  nt::SmallCost small(int i) const {
    if (i == 0) return {2.8, 0.45, 0.003};
    if (i == 1) return {3.0, 1.25, 0.0046};
    return {4.0, 2.7, 0.011};
  }
  template <class F>
  void loops(int M, int N, double steps, const F& offer) const {
    struct Cost {
      double ends, step;  // of a full round
      double few_ends, few_step, share;  // of one of less than `share` of the CUs
    };
    const auto loop = [&](Way w, const Cost& c) {
      const nt::TileShape t = shape(w);
      const int64_t tiles = ceil_div(M, t.rows) * ceil_div(N, t.cols), rest = tiles % 256;
      if (tiles > kMaxWorkItems / t.threads) return;  // a block a tile: more than a launch takes
      double us = 2.5 + tiles / 256 * (c.ends + c.step * steps);
      if (rest) {
        const double more = rest > c.share * 256 ? (rest / 256.0 - c.share) / (1 - c.share) : 0.0;
        us += c.few_ends + (c.ends - c.few_ends) * more + (c.few_step + (c.step - c.few_step) * more) * steps;
      }
      offer(w, us);
    };
    loop(Way::kLoopSquare, {6.0, 0.44, 5.5, 0.33, 0.25});
    loop(Way::kLoop128, {9.2, 0.77, 7.0, 0.56, 0.5});
    loop(Way::kLoop256, {13.2, 1.43, 11.0, 1.02, 0.0});
  }
  bool cuts_rows(int) const { return true; }
  constexpr nt::TileShape shape(Way way) const {
    switch (way) {
      case Way::kSmall16: return {16, 16, 512};
      case Way::kSmall32: return {32, 32, 512};
      case Way::kSmall64: return {64, 64, 512};
      case Way::kLoopSquare: return {128, 128, 256};
      case Way::kLoop128: return {256, 128, 512};
      default: return {256, 256, 512};
    }
  }
};

template <class O>
void launch(const Side& A, const Side& B, int K, const Out<O>& out, hipStream_t s) {
  using LoopSquare = nt::Loop<nt::Kind::kInt8, 4, 4, 2, 2, 4>;
  using Loop128 = nt::Loop<nt::Kind::kInt8, 4, 4, 4, 2, 3>;
  using Loop256 = nt::Loop<nt::Kind::kInt8, 8, 4, 2, 4, 2>;
  using P = nt::Int8;
  constexpr Model model{};
  using nt::is_shape;
  static_assert(is_shape<LoopSquare>(model.shape(Way::kLoopSquare)) && is_shape<Loop128>(model.shape(Way::kLoop128)) &&
                is_shape<Loop256>(model.shape(Way::kLoop256)) &&
                is_shape<nt::Direct<P, 1, 1, 8>>(model.shape(Way::kSmall16)) &&
                is_shape<nt::Direct<P, 2, 2, 8>>(model.shape(Way::kSmall32)) &&
                is_shape<nt::Direct<P, 4, 4, 8>>(model.shape(Way::kSmall64)));
  Plan p;
  plan(model, p, 0, 0, out.M, out.N, K, K > 0, nt::kCuts);
  for (int i = 0; i < p.count; ++i) {
    const nt::Piece& at = p.piece[i];
    const Out<O> part = out.from(at.m0, at.n0, at.M, at.N);
    const Side a = from_row(A, at.m0, 0), b = from_row(B, at.n0, 0);
    const unsigned blocks = static_cast<unsigned>(blocks_of(model, at));
    if (at.way <= Way::kSmall64) nt::launch_small<P>(at.way, a, b, K, part, at.skip_m, at.skip_n, blocks, s);
    else if (at.way == Way::kLoopSquare) launch_loop<LoopSquare>(a, b, K, part, blocks, s);
    else if (at.way == Way::kLoop128) launch_loop<Loop128>(a, b, K, part, blocks, s);
    else launch_loop<Loop256>(a, b, K, part, blocks, s);
  }
}

// The sum is empty: D is the bias.
template <class O>
__global__ __launch_bounds__(256) void k_bias(Out<O> out, int64_t items, int per_row) {
  for (int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x; t < items; t += int64_t(gridDim.x) * 256) {
    const int64_t m = t / per_row;
    const int n = static_cast<int>(t % per_row) * 4;
    float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (out.bias.p) out.bias.get(b, n, out.N);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n < out.N - i) from_float(b[i], out.d[m * out.ldd + n + i]);
  }
}

template <class O>
void launch_out(const Int8Product& p, hipStream_t stream) {
  const Out<O> out{static_cast<O*>(p.d), p.ldd, p.M, p.N, p.sa, p.sa_inc, p.sb, p.sb_inc, Bias{p.bias, p.bias_type}};
  if (p.K == 0) {
    const int64_t per = ceil_div(p.N, 4), items = per * p.M, blocks = ceil_div(items, 256), cap = kMaxWorkItems / 256;
    hipLaunchKernelGGL((k_bias<O>), dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)), dim3(256), 0, stream, out,
                       items, static_cast<int>(per));
    return;
  }
  const Side a{static_cast<const uint8_t*>(p.a), p.lda, p.M, nullptr, 0, 0, 0, 0};
  const Side b{static_cast<const uint8_t*>(p.b), p.ldb, p.N, nullptr, 0, 0, 0, 0};
  launch<O>(a, b, p.K, out, stream);
}

// A linear layer of few tokens in one launch: each block quantises all of them for
// itself, with its first loads of the weight under way, into LDS, and sums 16 x 16
// results from there, its wavefronts taking every eighth step along K as Direct's do.
// Bound by a launch, a trip to memory for x and the weight's read: 1 x 1024 x 1024 4.6 us
// (quantiser and product in two launches 5.9), 1 x 4096 x 4096 6.2 (8.7), 16 x 1024 x
// 4096 5.6 (6.4), 4 x 4096 x 16384 14.6 (16.9); where many blocks quantise many tokens
// the second launch would be worth it on the device, 16 x 1024 x 16384 10.6 (9.4), but
// costs the host 4 us.
// At most 32 elements a thread, held in registers from the maximum to the codes.
constexpr int kTokenThreads = 512, kTokenElements = 32 * kTokenThreads, kMostTokens = 16;
constexpr int64_t kTokenBlocks = 512;  // at most: two a CU, as many as run at a time (4 x 4096 x 16384 with 1024 19 us, 14.6)
// tokens rounded up to a power of two, so that each takes as many lanes
__host__ __device__ constexpr int token_rows(int tokens) {
  int r = 1;
  while (r < tokens) r *= 2;
  return r;
}
bool few_tokens(int tokens, int inputs) {
  return tokens <= kMostTokens && int64_t(token_rows(tokens)) * ceil_div(inputs, 8) * 8 <= kTokenElements;
}

// Eight neighbours of a row, of at least eight or none: the words of the last eight
// inside where fewer are left, moved to the front when they are looked at.  The load
// has no branch around it, behind which the compiler would wait for it by itself
// (1 x 4096 x 4096 8.0 -> 6.2 us).
template <class X>
struct Raw8 {
  static constexpr int kWords = 2 * sizeof(X);
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const X* row, int col, int cols) {
    if (cols >= 8) {
      __builtin_memcpy(w, row + min(col, cols - 8), sizeof(w));
      return;
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < 7; ++i)  // uniform: a row shorter than that
      if (col + i < cols) {
        if constexpr (sizeof(X) == 4) w[i] = reinterpret_cast<const uint32_t*>(row)[col + i];
        else w[i / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(row)[col + i]) << (16 * (i % 2));
      }
  }
  __device__ __forceinline__ Pack<8, X> settled(int col, int cols) const {
    Raw8 r = *this;
    if (cols >= 8 && col > cols - 8) {
      const int off = min(col - (cols - 8), 8);
      const auto down = [&](bool on, int by) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) r.w[i] = !on ? r.w[i] : i + by < kWords ? r.w[i + by] : 0;
      };
      down(off & 8, kWords);
      down(off & 4, kWords / 2);
      down(off & 2, kWords / 4);
      if constexpr (sizeof(X) == 4) {
        down(off & 1, 1);
      } else if (off & 1) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) r.w[i] = r.w[i] >> 16 | (i + 1 < kWords ? r.w[i + 1] << 16 : 0);
      }
    }
    return __builtin_bit_cast(Pack<8, X>, r);
  }
};

template <int ROWS, class X, class O>
__global__ __launch_bounds__(kTokenThreads) void k_tokens(const X* __restrict__ x, int64_t ldx, int tokens, Side B, int K,
                                                          Out<O> out) {
  constexpr int kLanes = kTokenThreads / ROWS, kChunks = 4, kWaves = kTokenThreads / 64, kAhead = 4;
  using S = RowShape<kLanes, kChunks, kTokenThreads>;
  // rows of codes 16 bytes more than a multiple of 128 apart, the last step's filled up with zeros
  constexpr int kLdMost = kTokenElements / ROWS + 16;
  __shared__ alignas(16) int8_t codes[ROWS * kLdMost];
  __shared__ uint32_t meet[kWaves][1];
  __shared__ float scales[ROWS];
  __shared__ v4i sums[2][kWaves][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int row = lane % 16, g = lane / 16;
  const int64_t tiles = ceil_div(out.N, 16);
  const int steps = static_cast<int>(ceil_div(K, nt::kStep)), ld = steps * nt::kStep + 16;
  const int last = (K - 1) / 16 * 16;  // the last 16 bytes of a row; what they hold past K meets zeros
  const auto read = [&](nt::Frag& f, int64_t tile, int k) {
    const uint8_t* const b = B.p + min(tile * 16 + row, int64_t(B.rows) - 1) * B.ld;
    f.lo = *reinterpret_cast<const v4i*>(b + min(k * nt::kStep + 16 * g, last));
    f.hi = *reinterpret_cast<const v4i*>(b + min(k * nt::kStep + 16 * (4 + g), last));
  };
  // x before the weight: loads arrive in order
  const int token = threadIdx.x / kLanes, place = threadIdx.x % kLanes;
  Raw8<X> raw[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) raw[c].load(x + int64_t(min(token, tokens - 1)) * ldx, (c * kLanes + place) * 8, K);
  // the wavefront's steps wave + 8 u of every 32 pass through fragment u (those past
  // the end read a row's last bytes: with a branch around them all loads would have to
  // arrive before x is looked at)
  nt::Frag f[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) read(f[u], blockIdx.x, wave + u * kWaves);
  {
    Pack<8, X> v[kChunks];
    uint32_t top[1] = {0};
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      v[c] = raw[c].settled((c * kLanes + place) * 8, K);
      top[0] = int8::top8(top[0], v[c]);
    }
    join_row<S>(top, meet, int8::Max{});
    const int8::Scale by = int8::make_scale(top[0]);
    if (place == 0) scales[token] = by.s;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int col = (c * kLanes + place) * 8;
      if (col < ld - 16) {  // past K codes of zeros are zeros
        const Pack<8, int8_t> q = int8::codes8(v[c], by);
        __builtin_memcpy(&codes[token * ld + col], &q, 8);
      }
    }
  }
  __syncthreads();
  Out<O> o = out;
  o.sa = scales;
  o.sa_inc = 1;
  const int8_t* const a = &codes[min(row, tokens - 1) * ld + 16 * g];
  int turn = 0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, turn ^= 1) {
    v4i acc = {0, 0, 0, 0};
    for (int k0 = wave; k0 < steps; k0 += kAhead * kWaves) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = k0 + u * kWaves;
        if (k >= steps) break;
        nt::Frag m;
        m.lo = *reinterpret_cast<const v4i*>(a + k * nt::kStep);
        m.hi = *reinterpret_cast<const v4i*>(a + k * nt::kStep + 64);
        nt::Int8::mac(acc, f[u], m, 0, 0);
        if (k + kAhead * kWaves < steps) read(f[u], tile, k + kAhead * kWaves);
        else if (tile + gridDim.x < tiles) read(f[u], tile + gridDim.x, wave + u * kWaves);
      }
    }
    sums[turn][wave][lane] = acc;
    __syncthreads();  // sums[turn] is free again when all have met in the next tile
    if (wave == 0) {
      v4i v = sums[turn][0][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += sums[turn][w][lane];
      o(row, static_cast<int>(tile * 16) + 4 * g, v);
    }
  }
}

template <class X, class O>
void launch_tokens(const void* x, int64_t ldx, const Int8Product& p, hipStream_t stream) {
  const Out<O> out{static_cast<O*>(p.d), p.ldd, p.M, p.N, nullptr, 1, p.sb, p.sb_inc, Bias{p.bias, p.bias_type}};
  const Side b{static_cast<const uint8_t*>(p.b), p.ldb, p.N, nullptr, 0, 0, 0, 0};
  const int64_t tiles = ceil_div(p.N, 16);
  const dim3 grid(static_cast<unsigned>(tiles < kTokenBlocks ? tiles : kTokenBlocks));
  const auto go = [&](auto rows) {
    hipLaunchKernelGGL((k_tokens<rows.value, X, O>), grid, dim3(kTokenThreads), 0, stream, static_cast<const X*>(x), ldx,
                       p.M, b, p.K, out);
  };
  switch (token_rows(p.M)) {
    case 1: return go(std::integral_constant<int, 1>{});
    case 2: return go(std::integral_constant<int, 2>{});
    case 4: return go(std::integral_constant<int, 4>{});
    case 8: return go(std::integral_constant<int, 8>{});
    default: return go(std::integral_constant<int, 16>{});
  }
}
template <class X>
void launch_tokens(const void* x, int64_t ldx, const Int8Product& p, hipStream_t stream) {
  if (p.d_type == HIP_INT8_F32) launch_tokens<X, float>(x, ldx, p, stream);
  else if (p.d_type == HIP_INT8_BF16) launch_tokens<X, bf16>(x, ldx, p, stream);
  else launch_tokens<X, _Float16>(x, ldx, p, stream);
}

bool bad_type(int t) { return t != HIP_INT8_F32 && t != HIP_INT8_BF16 && t != HIP_INT8_F16; }
bool bad_ld(int ld, int K) { return ld < (K > 1 ? K : 1) || ld % 16 != 0 || ld > HIP_INT8_MAX_LD; }
bool off16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }
// of the codes of a linear layer's tokens in the workspace, long ones in whole cache
// lines (a product 4096 x 4096 x 4097 of rows of 4112 bytes 70 us, of 4224 62), and what they take there
int64_t code_stride(int inputs) {
  if (inputs >= 512) return ceil_div(inputs, 128) * 128;
  return inputs > 0 ? ceil_div(inputs, 16) * 16 : 16;
}
int64_t linear_bytes(int tokens, int inputs) {
  return tokens == 0 || inputs == 0 || few_tokens(tokens, inputs) ? 0 : tokens * (code_stride(inputs) + 4);
}

}  // namespace

void launch_int8_gemm(const Int8Product& p, hipStream_t stream) {
  if (p.d_type == HIP_INT8_F32) launch_out<float>(p, stream);
  else if (p.d_type == HIP_INT8_BF16) launch_out<bf16>(p, stream);
  else launch_out<_Float16>(p, stream);
}

}  // namespace sgemm

using namespace sgemm;

extern "C" {

int hip_int8_gemm(int M, int N, int K, const void* A, int lda, const float* SA, long long sa_inc, const void* B, int ldb,
                  const float* SB, long long sb_inc, const void* bias, int bias_type, void* D, int ldd, int d_type,
                  hipStream_t stream) {
  if (M < 0) return -1;
  if (N < 0) return -2;
  if (K < 0 || K > HIP_INT8_MAX_K) return -3;
  const bool some = M > 0 && N > 0, product = some && K > 0;
  if (product && (A == nullptr || off16(A))) return -4;
  if (bad_ld(lda, K)) return -5;
  if (product && SA == nullptr) return -6;
  if (sa_inc < 0) return -7;
  if (product && (B == nullptr || off16(B))) return -8;
  if (bad_ld(ldb, K)) return -9;
  if (product && SB == nullptr) return -10;
  if (sb_inc < 0) return -11;
  if (bias != nullptr && bad_type(bias_type)) return -13;
  if (some && D == nullptr) return -14;
  if (ldd < (N > 1 ? N : 1)) return -15;
  if (bad_type(d_type)) return -16;
  if (!some) return 0;
  launch_int8_gemm(Int8Product{M, N, K, A, lda, SA, sa_inc, B, ldb, SB, sb_inc, bias, bias_type, D, ldd, d_type}, stream);
  return static_cast<int>(hipGetLastError());
}

int hip_int8_gemm_plan(int M, int N, int K, hip_int8_gemm_launch* launches, int* count) {
  if (M < 0) return -1;
  if (N < 0) return -2;
  if (K < 0 || K > HIP_INT8_MAX_K) return -3;
  Plan p;
  const Model model{};
  if (M > 0 && N > 0 && K > 0) plan(model, p, 0, 0, M, N, K, true, nt::kCuts);
  for (int i = 0; launches && i < p.count; ++i) {
    const nt::Piece& at = p.piece[i];
    const nt::TileShape t = model.shape(at.way);
    launches[i] = hip_int8_gemm_launch{t.rows, t.cols, at.m0, at.n0, at.M, at.N, at.skip_m, at.skip_n, t.threads,
                                       blocks_of(model, at)};
  }
  if (count) *count = p.count;
  return 0;
}

int hip_int8_linear_workspace(int tokens, int inputs, long long* bytes) {
  if (tokens < 0) return -1;
  if (inputs < 0 || inputs > HIP_INT8_MAX_K) return -2;
  if (bytes) *bytes = linear_bytes(tokens, inputs);
  return 0;
}

int hip_int8_linear(int tokens, int inputs, int outputs, const void* X, int x_type, int ldx, const void* W, int ldw,
                    const float* SW, long long sw_inc, const void* bias, int bias_type, void* Y, int ldy, int y_type,
                    void* workspace, long long workspace_bytes, hipStream_t stream) {
  if (tokens < 0) return -1;
  if (inputs < 0 || inputs > HIP_INT8_MAX_K) return -2;
  if (outputs < 0) return -3;
  const bool some = tokens > 0 && outputs > 0, product = some && inputs > 0;
  if (product && X == nullptr) return -4;
  if (bad_type(x_type)) return -5;
  if (ldx < (inputs > 1 ? inputs : 1)) return -6;
  if (product && (W == nullptr || off16(W))) return -7;
  if (bad_ld(ldw, inputs)) return -8;
  if (product && SW == nullptr) return -9;
  if (sw_inc < 0) return -10;
  if (bias != nullptr && bad_type(bias_type)) return -12;
  if (some && Y == nullptr) return -13;
  if (ldy < (outputs > 1 ? outputs : 1)) return -14;
  if (bad_type(y_type)) return -15;
  const int64_t bytes = product ? linear_bytes(tokens, inputs) : 0;
  if (bytes > 0 && (workspace == nullptr || off16(workspace))) return -16;
  if (workspace_bytes < bytes) return -17;
  if (!some) return 0;
  Int8Product p{tokens, outputs, inputs, workspace, code_stride(inputs), nullptr, 1, W, ldw, SW, sw_inc, bias, bias_type, Y,
                ldy, y_type};
  if (product && bytes == 0) {
    if (x_type == HIP_INT8_F32) launch_tokens<float>(X, ldx, p, stream);
    else if (x_type == HIP_INT8_BF16) launch_tokens<bf16>(X, ldx, p, stream);
    else launch_tokens<_Float16>(X, ldx, p, stream);
    return static_cast<int>(hipGetLastError());
  }
  if (product) {
    int8_t* const q = static_cast<int8_t*>(workspace);
    float* const s = reinterpret_cast<float*>(q + tokens * p.lda);
    launch_int8_quantize(tokens, inputs, X, x_type, ldx, q, p.lda, s, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return static_cast<int>(e);
    p.sa = s;
  }
  launch_int8_gemm(p, stream);
  return static_cast<int>(hipGetLastError());
}

const char* hip_int8_gemm_status_string(int status) {
  switch (status) {
    case 0: return "success";
    case -1: return "argument 1 (M) is negative";
    case -2: return "argument 2 (N) is negative";
    case -3: return "argument 3 (K) is negative or above HIP_INT8_MAX_K";
    case -4: return "argument 4 (A) is NULL or not 16-byte aligned";
    case -5: return "argument 5 (lda) is smaller than max(1, K), no multiple of 16, or above HIP_INT8_MAX_LD";
    case -6: return "argument 6 (SA) is NULL";
    case -7: return "argument 7 (sa_inc) is negative";
    case -8: return "argument 8 (B) is NULL or not 16-byte aligned";
    case -9: return "argument 9 (ldb) is smaller than max(1, K), no multiple of 16, or above HIP_INT8_MAX_LD";
    case -10: return "argument 10 (SB) is NULL";
    case -11: return "argument 11 (sb_inc) is negative";
    case -13: return "argument 13 (bias_type) is not a known type";
    case -14: return "argument 14 (D) is NULL";
    case -15: return "argument 15 (ldd) is smaller than max(1, N)";
    case -16: return "argument 16 (d_type) is not a known type";
    default: break;
  }
  if (status > 0) return hipGetErrorString(static_cast<hipError_t>(status));
  return "unknown status";
}

const char* hip_int8_linear_status_string(int status) {
  switch (status) {
    case 0: return "success";
    case -1: return "argument 1 (tokens) is negative";
    case -2: return "argument 2 (inputs) is negative or above HIP_INT8_MAX_K";
    case -3: return "argument 3 (outputs) is negative";
    case -4: return "argument 4 (X) is NULL";
    case -5: return "argument 5 (x_type) is not a known type";
    case -6: return "argument 6 (ldx) is smaller than max(1, inputs)";
    case -7: return "argument 7 (W) is NULL or not 16-byte aligned";
    case -8: return "argument 8 (ldw) is smaller than max(1, inputs), no multiple of 16, or above HIP_INT8_MAX_LD";
    case -9: return "argument 9 (SW) is NULL";
    case -10: return "argument 10 (sw_inc) is negative";
    case -12: return "argument 12 (bias_type) is not a known type";
    case -13: return "argument 13 (Y) is NULL";
    case -14: return "argument 14 (ldy) is smaller than max(1, outputs)";
    case -15: return "argument 15 (y_type) is not a known type";
    case -16: return "argument 16 (workspace) is NULL or not 16-byte aligned";
    case -17: return "argument 17 (workspace_bytes) is less than hip_int8_linear_workspace says";
    default: break;
  }
  if (status > 0) return hipGetErrorString(static_cast<hipError_t>(status));
  return "unknown status";
}

}  // extern "C"

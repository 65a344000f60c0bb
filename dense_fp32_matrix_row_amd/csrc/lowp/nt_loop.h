// nt_loop.h -- the large tiles of the block-scaled 8-bit product and the
// orthogonalised update: D = A * B^T over operands whose rows are contiguous
// along K (nt_tile.h has the operands' form), with the K loop in assembly
// (nt_loop.inc, written by gen_nt_loop.py).
#pragma once

#include "nt_loop.inc"
#include "nt_tile.h"

namespace sgemm {
namespace nt {

typedef float v16f __attribute__((ext_vector_type(16)));

// What a loop multiplies and how it scales (gen_nt_loop.py).
enum class Kind { kE8M0, kF32Uniform, kF32Rows, kWideF32Uniform, kWideF32Rows, kWideE8M0Uniform, kWideE8M0Rows, kPair };

// Block tile of WM x WN wavefronts of 16 MT x 16 NT, at most 256 registers each.
template <Kind KIND_, int MT_, int NT_, int WM_, int WN_, int STAGES_>
struct Loop {
  static constexpr Kind KIND = KIND_;
  static constexpr int MT = MT_, NT = NT_, WM = WM_, WN = WN_, STAGES = STAGES_;
  static constexpr int kPositions = STAGES % 2 ? 2 * STAGES : STAGES;  // steps that the loop is unrolled over
  static constexpr int BM = 16 * MT * WM, BN = 16 * NT * WN, waves = WM * WN, threads = 64 * waves;
  static constexpr bool kScaled = KIND != Kind::kPair;
  static constexpr bool kBytes = KIND == Kind::kWideE8M0Uniform || KIND == Kind::kWideE8M0Rows;
  static constexpr bool kUniform =
      KIND == Kind::kF32Uniform || KIND == Kind::kWideF32Uniform || KIND == Kind::kWideE8M0Uniform;
  static constexpr int kScaleBytes = KIND == Kind::kE8M0 || kBytes ? 1 : 4;
  static constexpr int kStage = (BM + BN) * kStep;
  static constexpr int kScaleLoads = kScaled ? ((BM + BN) / 64 + waves - 1) / waves : 0;
  static constexpr int kScaleStage = 256 * waves * kScaleLoads;
  static constexpr int kLds = STAGES * (kStage + kScaleStage);
  static constexpr int kA = BM / 8 / waves, kB = BN / 8 / waves;  // loads a wavefront and step
  static constexpr int kAcc = MT * NT / 4;
  static_assert(kScaleLoads <= 1 && kA % 2 == 0 && kB % 2 == 0, "one scale a thread, rows of chunks in turn");

  // Whether every scale of a tile lies within 32 bits of the first.
  static bool fits(const Side& o) { return !kScaled || o.s_row <= (int64_t(1) << 30) / 256 / kScaleBytes; }
};

#define NT_LOOP_RUN(NAME, SUMS, MORE_OUT, MORE_IN)                                                                 \
  asm volatile(NT_LOOP_##NAME                                                                                      \
               : SUMS, "+{s[60:63]}"(ra), "+{s[64:67]}"(rb), [left] "+s"(left), [turns] "+s"(turns), [aLo] "+v"(aLo), \
                 [aHi] "+v"(aHi), [bLo] "+v"(bLo), [bHi] "+v"(bHi) MORE_OUT                                        \
               : [aEven] "v"(aEven), [aOdd] "v"(aOdd), [bEven] "v"(bEven), [bOdd] "v"(bOdd), [ldsA] "s"(lds_a),    \
                 [ldsB] "s"(lds_b), [oA] "s"(oa), [eA] "s"(ea), [oB] "s"(ob), [eB] "s"(eb), [first] "s"(first),     \
                 [single] "s"(single) MORE_IN                                                                      \
               : NT_CLOBBERS_##NAME, "memory", "scc")
#define NT_SUMS_2 "=&{v[0:15]}"(acc[0]), "=&{v[16:31]}"(acc[1])
#define NT_SUMS_4 NT_SUMS_2, "=&{v[32:47]}"(acc[2]), "=&{v[48:63]}"(acc[3])
#define NT_SUMS_8                                                                                                  \
  NT_SUMS_4, "=&{v[64:79]}"(acc[4]), "=&{v[80:95]}"(acc[5]), "=&{v[96:111]}"(acc[6]), "=&{v[112:127]}"(acc[7])
#define NT_SUMS_9 NT_SUMS_8, "=&{v[128:143]}"(acc[8])
#define NT_SCALES_OUT , "+{s[68:71]}"(rs), [aS] "+v"(aS), [bS] "+v"(bS)
#define NT_SCALES_IN                                                                                               \
  , "{s[86:87]}"(ss), [gS] "v"(gs), [maskLo0] "v"(mask[0]), [maskLo1] "v"(mask[1]), [maskLo2] "v"(mask[2]),       \
      [maskLo3] "v"(mask[3]), [maskHi0] "v"(mask[4]), [maskHi1] "v"(mask[5]), [maskHi2] "v"(mask[6]),              \
      [maskHi3] "v"(mask[7])
#define NT_DIRECT_IN NT_SCALES_IN, [ldsS] "s"(lds_s)
#define NT_PARTIAL_IN NT_DIRECT_IN, [partial] "s"(partial)
#define NT_BYTES_OUT NT_SCALES_OUT, [tmp] "=&v"(tmp)
#define NT_BYTES_IN NT_SCALES_IN, [wS] "v"(wS), [half] "v"(0x400000)
#define NT_NONE

// A value that all lanes of a wavefront share, in a scalar register.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(static_cast<int>(v)); }
__device__ __forceinline__ uint64_t uniform(uint64_t v) {
  return uniform(static_cast<uint32_t>(v)) | static_cast<uint64_t>(uniform(static_cast<uint32_t>(v >> 32))) << 32;
}

// Sums the tile at rows m0 of A and n0 of B over K > 0 bytes.  LDS (L::kLds
// bytes) must not be in use.
template <class L>
__device__ __forceinline__ void loop_sum(uint8_t* smem, const Side& A, const Side& B, int m0, int n0, int K,
                                         v16f (&acc)[L::kAcc]) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int wm = wave % L::WM, wn = wave / L::WM, row = lane % 16, g = lane / 16;
  const uint32_t lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)smem));

  // The panels end with their last row: what lies past it, or past the last row's end, is read as zeros.
  const auto resource = [&](const Side& o, int row0, int rows) {
    const uint64_t at = reinterpret_cast<uint64_t>(o.p + row0 * o.ld);
    const uint32_t bytes = static_cast<uint32_t>(min(o.rows - row0, rows) - 1) * static_cast<uint32_t>(o.ld) + (K + 15) / 16 * 16;
    return v4i{static_cast<int>(uniform(static_cast<uint32_t>(at))),
               static_cast<int>(uniform(static_cast<uint32_t>(at >> 32) & 0xffff)), static_cast<int>(uniform(bytes)), 0x00020000};
  };
  v4i ra = resource(A, m0, L::BM), rb = resource(B, n0, L::BN);
  // Load i of a wavefront takes rows (wave kA + i) 8 ..: every other one has its chunks 64 bytes off.
  const uint32_t lda = static_cast<uint32_t>(A.ld), ldb = static_cast<uint32_t>(B.ld);
  const uint32_t chunk = 16 * ((lane % 8) ^ (lane / 16));
  const uint32_t aEven = lane / 8 * lda + chunk, aOdd = lane / 8 * lda + (chunk ^ 64);
  const uint32_t bEven = lane / 8 * ldb + chunk, bOdd = lane / 8 * ldb + (chunk ^ 64);
  const uint32_t ea = uniform(8 * lda), eb = uniform(8 * ldb);
  const uint32_t oa = uniform(wave * L::kA * 8 * lda), ob = uniform(wave * L::kB * 8 * ldb);
  const uint32_t lds_a = uniform(lds + wave * L::kA * 1024), lds_b = uniform(lds + wave * L::kB * 1024);

  const uint32_t steps = uniform(static_cast<uint32_t>(K - 1) / kStep + 1);
  // the position of the first step, so that the last one is in the last position
  const uint32_t first = uniform((L::kPositions - steps % L::kPositions) % L::kPositions);
  uint32_t left = steps, turns = uniform((steps - 1) / L::kPositions - (first == L::kPositions - 1 ? 1 : 0));
  const uint32_t single = uniform(static_cast<uint32_t>(steps == 1)), stage = first % L::STAGES;

  const uint32_t at = stage * L::kStage + row * kStep + 16 * (g ^ ((row / 2) % 8));
  uint32_t aLo = lds + wm * L::MT * 16 * kStep + at, aHi = lds + wm * L::MT * 16 * kStep + (at ^ 64);
  uint32_t bLo = lds + (L::BM + wn * L::NT * 16) * kStep + at, bHi = lds + (L::BM + wn * L::NT * 16) * kStep + (at ^ 64);

  if constexpr (L::kScaled) {
    // A wavefront loads 64 rows' scales, all of one side; the wavefronts past the last row's repeat it.
    const bool on_a = wave * 64 < L::BM;
    const Side& o = on_a ? A : B;
    const int row0 = on_a ? m0 : n0, r = min(on_a ? wave * 64 + lane : wave * 64 - L::BM + lane, (on_a ? L::BM : L::BN) - 1);
    const uint64_t s0 = reinterpret_cast<uint64_t>(o.s) + (row0 >> o.shift) * o.s_row * L::kScaleBytes;
    v4i rs = {static_cast<int>(uniform(static_cast<uint32_t>(s0))), static_cast<int>(uniform(static_cast<uint32_t>(s0 >> 32) & 0xffff)),
              -1, 0x00020000};
    const uint64_t ss = uniform(static_cast<uint64_t>(o.s_col * L::kScaleBytes));
    const uint32_t gs = static_cast<uint32_t>(((min(row0 + r, o.rows - 1) >> o.shift) - (row0 >> o.shift)) * o.s_row * L::kScaleBytes);
    const uint32_t lds_s = uniform(lds + wave * 256);
    const uint32_t s = lds + L::STAGES * L::kStage;
    uint32_t aS = s + stage * L::kScaleStage + 4 * (wm * L::MT * 16 + row);
    uint32_t bS = s + stage * L::kScaleStage + 4 * (L::BM + wn * L::NT * 16 + (L::KIND == Kind::kE8M0 ? row : L::kUniform ? 0 : 4 * g));
    const int last = K - (static_cast<int>(steps) - 1) * kStep;  // bytes of the last step
    const uint32_t partial = uniform(static_cast<uint32_t>(last < kStep));
    int mask[8];
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const int keep = last - 16 * (w < 4 ? g : 4 + g) - 4 * (w % 4);
      mask[w] = keep >= 4 ? -1 : keep <= 0 ? 0 : (1 << (8 * keep)) - 1;
    }
    [[maybe_unused]] uint32_t tmp;
    [[maybe_unused]] const uint32_t wS = s + 4 * threadIdx.x;
#define NT_LOOP_BOTH(KIND)                                                                             \
  if constexpr (L::BN == 256) NT_LOOP_RUN(KIND##_256x256, NT_SUMS_8, NT_SCALES_OUT, NT_PARTIAL_IN);    \
  else NT_LOOP_RUN(KIND##_256x128, NT_SUMS_4, NT_SCALES_OUT, NT_PARTIAL_IN)
    if constexpr (L::KIND == Kind::kE8M0) { NT_LOOP_BOTH(e8m0); }
    else if constexpr (L::KIND == Kind::kF32Uniform) { NT_LOOP_BOTH(f32u); }
    else if constexpr (L::KIND == Kind::kF32Rows) { NT_LOOP_BOTH(f32n); }
    else if constexpr (L::KIND == Kind::kWideF32Uniform) NT_LOOP_RUN(w32u_128x128, NT_SUMS_4, NT_SCALES_OUT, NT_DIRECT_IN);
    else if constexpr (L::KIND == Kind::kWideF32Rows) NT_LOOP_RUN(w32n_128x128, NT_SUMS_4, NT_SCALES_OUT, NT_DIRECT_IN);
    else if constexpr (L::KIND == Kind::kWideE8M0Uniform) NT_LOOP_RUN(w8u_128x128, NT_SUMS_4, NT_BYTES_OUT, NT_BYTES_IN);
    else NT_LOOP_RUN(w8n_128x128, NT_SUMS_4, NT_BYTES_OUT, NT_BYTES_IN);
  } else if constexpr (L::BM == 256) {
    NT_LOOP_RUN(pair_256x256, NT_SUMS_8, NT_NONE, NT_NONE);
  } else if constexpr (L::BM == 192) {
    NT_LOOP_RUN(pair_192x192, NT_SUMS_9, NT_NONE, NT_NONE);
  } else {
    NT_LOOP_RUN(pair_128x128, NT_SUMS_2, NT_NONE, NT_NONE);
  }
}

// The way out, through LDS, for what is stored by rows and by columns: 64
// rows of sums at a time lie in LDS, COLS + 4 floats apart (four columns of 16
// rows at once, as fragments come, then fall in different banks).
template <int COLS>
struct alignas(16) Sheet {
  static constexpr int kLd = COLS + 4;
  float v[64 * kLd];

  __device__ __forceinline__ void put(int r, int c, v4f x) { *reinterpret_cast<v4f*>(&v[r * kLd + c]) = x; }

  // rows(r, c, x): eight neighbours of row r from column c; columns(c, r, x): eight
  // of column c from row r, if `both`.  All threads of the block call it, with the
  // sheet written.
  template <int THREADS, class R, class C>
  __device__ __forceinline__ void out(bool both, const R& rows, const C& columns) {
    __syncthreads();
#pragma unroll 2
    for (int t = threadIdx.x; t < 64 * COLS / 8; t += THREADS) {
      float x[8];
      __builtin_memcpy(x, &v[t / (COLS / 8) * kLd + t % (COLS / 8) * 8], 32);
      rows(t / (COLS / 8), t % (COLS / 8) * 8, x);
    }
    if (!both) {
      __syncthreads();
      return;
    }
    // four lanes take 32 rows of a column, whose pairs lie side by side
#pragma unroll 2
    for (int t = threadIdx.x; t < 64 * COLS / 8; t += THREADS) {
      const int c = t / 4 % COLS, r = (t % 4 + t / (4 * COLS) * 4) * 8;
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = v[(r + i) * kLd + c];
      columns(c, r, x);
    }
    __syncthreads();
  }
};

// Puts a block's sums on sheets, 64 rows after another, and calls each(first
// row) with each one written.  LDS must hold a sheet and be free.
template <class L, class F>
__device__ __forceinline__ void loop_sheets(Sheet<L::BN>& sheet, const v16f (&acc)[L::kAcc], const F& each) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int wm = wave % L::WM, wn = wave / L::WM;
#pragma unroll
  for (int top = 0; top < L::BM; top += 64) {
#pragma unroll
    for (int i = 0; i < L::MT; ++i) {
      const int r = (wm * L::MT + i) * 16;
      if (r < top || r >= top + 64) continue;
#pragma unroll
      for (int j = 0; j < L::NT; ++j) {
        const int at = j * L::MT + i;
        const v16f& a = acc[at / 4];
        sheet.put(r - top + lane % 16, (wn * L::NT + j) * 16 + 4 * (lane / 16),
                  v4f{a[at % 4 * 4], a[at % 4 * 4 + 1], a[at % 4 * 4 + 2], a[at % 4 * 4 + 3]});
      }
    }
    each(top);
  }
}

}  // namespace nt
}  // namespace sgemm

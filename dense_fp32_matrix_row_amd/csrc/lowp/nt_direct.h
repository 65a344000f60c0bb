// nt_direct.h -- tiles for products with few rows or columns: D = A * B^T over
// operands whose rows are contiguous along K (nt_tile.h has the operands' form
// and what is done with them).
//
// The wavefronts of a block share one small tile and split its K: each takes
// every WAVES-th step straight from memory into registers, in the matrix
// instructions' order, with the next one of its steps under way, and their sums
// meet in LDS.  Nothing is staged and nobody waits for anybody before the end,
// so that a short K costs one trip to memory, and a long one keeps 2 WAVES
// steps of every block under way.  Each block reads its rows from the L2 for
// itself; the first-level cache's 64 bytes a clock and CU hold a 64 x 64 tile of
// pairs to three quarters of the matrix rate, one of 8-bit codes to half.
#pragma once

#include "nt_tile.h"

namespace sgemm {
namespace nt {

template <class P_, int MT_, int NT_, int WAVES_>
struct Direct {
  using P = P_;
  static constexpr int MT = MT_, NT = NT_, WAVES = WAVES_;
  static constexpr int BM = 16 * MT, BN = 16 * NT, threads = 64 * WAVES;
  static constexpr int kFrags = MT * NT;
  static constexpr int kChunk = kFrags < 8 ? kFrags : 8;     // fragments that meet at a time
  static constexpr bool kScaled = P::kScaleBytes > 0;
  static constexpr int kSn = !kScaled ? 0 : !P::kRowScales || P::kUniform ? 1 : 4;  // scales a lane takes of 16 rows of B

  using Meet = v4f[WAVES][kChunk][64];

  struct Raw {
    Frag a[MT], b[NT];
    uint32_t sa[MT], sb[NT][kSn ? kSn : 1];
  };

  // Where a lane's rows begin; rows past the end repeat the last one.  Of a step's
  // 128 bytes of a row a lane takes two times 16, 64 apart.  Where all rows begin
  // in the same half of the cache's 128-byte lines, odd rows take the second
  // first, so that a load takes both halves of the lines alike (256 x 1024 x 1024
  // with rows of 1024 bytes back to back: 4.9 -> 4.1 us).
  struct Reader {
    const uint8_t *a, *b;
    uint32_t ra[MT], rb[NT];
    const uint8_t *sa[MT], *sb[NT][kSn ? kSn : 1];
    int64_t ca, cb;  // bytes from one step's scales to the next's
    uint32_t last;   // the last 16 bytes of a row
    bool turn_a, turn_b;
    int g;

    __device__ __forceinline__ Reader(const Side& A, const Side& B, int m0, int n0, int K, int row, int g_)
        : a(A.p + int64_t(m0) * A.ld), b(B.p + int64_t(n0) * B.ld), ca(A.s_col * P::kScaleBytes),
          cb(B.s_col * P::kScaleBytes), last(static_cast<uint32_t>(K - 1) / 16 * 16), turn_a(row % 2 != 0 && A.ld / 64 % 2 == 0),
          turn_b(row % 2 != 0 && B.ld / 64 % 2 == 0), g(g_) {
      const auto scale = [](const Side& o, int at) {
        return static_cast<const uint8_t*>(o.s) + (int64_t(min(at, o.rows - 1) >> o.shift) * o.s_row) * P::kScaleBytes;
      };
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        ra[i] = static_cast<uint32_t>(min(16 * i + row, A.rows - 1 - m0)) * static_cast<uint32_t>(A.ld);
        if constexpr (kScaled) sa[i] = scale(A, m0 + 16 * i + row);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        rb[j] = static_cast<uint32_t>(min(16 * j + row, B.rows - 1 - n0)) * static_cast<uint32_t>(B.ld);
        if constexpr (kScaled)
#pragma unroll
          for (int r = 0; r < kSn; ++r) sb[j][r] = scale(B, n0 + 16 * j + (P::kRowScales ? P::kUniform ? 0 : 4 * g + r : row));
      }
    }
    static __device__ __forceinline__ uint32_t scale_at(const uint8_t* p) {
      if constexpr (P::kScaleBytes == 4) return *reinterpret_cast<const uint32_t*>(p);
      return *p;
    }
    __device__ __forceinline__ void read(Raw& r, int k) const {
      const uint32_t first = static_cast<uint32_t>(k) * kStep + 16 * g, lo = min(first, last), hi = min(first + 64, last);
      const uint32_t alo = turn_a ? hi : lo, ahi = turn_a ? lo : hi, blo = turn_b ? hi : lo, bhi = turn_b ? lo : hi;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        r.a[i].lo = *reinterpret_cast<const v4i*>(a + ra[i] + alo);
        r.a[i].hi = *reinterpret_cast<const v4i*>(a + ra[i] + ahi);
        if constexpr (kScaled) r.sa[i] = scale_at(sa[i] + k * ca);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        r.b[j].lo = *reinterpret_cast<const v4i*>(b + rb[j] + blo);
        r.b[j].hi = *reinterpret_cast<const v4i*>(b + rb[j] + bhi);
        if constexpr (kScaled)
#pragma unroll
          for (int s = 0; s < kSn; ++s) r.sb[j][s] = scale_at(sb[j][s] + k * cb);
      }
    }
  };

  // What was read the other way round.
  static __device__ __forceinline__ void turn(Frag& f, bool other) {
    const v4i lo = f.lo;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      f.lo[w] = other ? f.hi[w] : lo[w];
      f.hi[w] = other ? lo[w] : f.hi[w];
    }
  }
  static __device__ __forceinline__ void turn(Raw& r, const Reader& rd) {
#pragma unroll
    for (int i = 0; i < MT; ++i) turn(r.a[i], rd.turn_a);
#pragma unroll
    for (int j = 0; j < NT; ++j) turn(r.b[j], rd.turn_b);
  }

  static __device__ __forceinline__ void mac(typename P::Acc (&acc)[NT][MT], const Raw& r) {
    typename P::Op mo[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) mo[i] = P::prepare(r.a[i]);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const typename P::Op no = P::prepare(r.b[j]);
      if constexpr (P::kRowScales) {
        v4f sn;
#pragma unroll
        for (int s = 0; s < kSn; ++s) sn[s] = scale_value<P::kScaleBytes>(r.sb[j][s]);
#pragma unroll
        for (int i = 0; i < MT; ++i) P::mac(acc[j][i], no, mo[i], sn, scale_value<P::kScaleBytes>(r.sa[i]));
      } else {
#pragma unroll
        for (int i = 0; i < MT; ++i) P::mac(acc[j][i], no, mo[i], r.sb[j][0], r.sa[i]);
      }
    }
  }

  // Zeroes what lies past K's end, of the last step.
  static __device__ __forceinline__ void mask(Raw& r, int left, int g) {
#pragma unroll
    for (int i = 0; i < MT; ++i) r.a[i] = mask_frag(r.a[i], g, left);
#pragma unroll
    for (int j = 0; j < NT; ++j) r.b[j] = mask_frag(r.b[j], g, left);
  }

  // Sums the tile at rows m0 of A and n0 of B over K bytes and calls
  // epi(m, n, v) for every four neighbours D[m][n .. n+3], also past D's edges;
  // the block's wavefronts take a share each.  started() is called by all threads
  // with the first loads under way, a barrier before epi.
  struct Nothing {
    __device__ __forceinline__ void operator()() const {}
  };
  template <class E, class S = Nothing>
  static __device__ __forceinline__ void run(Meet& meet, const Side& A, const Side& B, int m0, int n0, int K,
                                             const E& epi, const S& started = S{}) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int row = lane % 16, g = lane / 16;
    typename P::Acc acc[NT][MT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) P::zero(acc[j][i]);

    const int steps = static_cast<int>(ceil_div(K, kStep));
    if (wave < steps) {
      const Reader rd(A, B, m0, n0, K, row, g);
      Raw now, next;
      rd.read(now, wave);
      started();
      int k = wave;
      for (; k + WAVES < steps; k += WAVES) {
        rd.read(next, k + WAVES);
        turn(now, rd);
        mac(acc, now);
        now = next;
      }
      turn(now, rd);
      if (K - k * kStep < kStep) mask(now, K - k * kStep, g);
      mac(acc, now);
    } else {
      started();
    }

#pragma unroll
    for (int c = 0; c < kFrags; c += kChunk) {
      if (c) __syncthreads();
#pragma unroll
      for (int f = c; f < c + kChunk && f < kFrags; ++f) meet[wave][f - c][lane] = P::value(acc[f / MT][f % MT]);
      __syncthreads();
#pragma unroll
      for (int o = 0; o < kChunk; o += WAVES) {
        const int f = o + wave;  // in the order of the wavefronts, whoever adds
        if (f < kChunk && c + f < kFrags) {
          v4f v = meet[0][f][lane];
#pragma unroll
          for (int w = 1; w < WAVES; ++w) v += meet[w][f][lane];
          epi(m0 + 16 * ((c + f) % MT) + row, n0 + 16 * ((c + f) / MT) + 4 * g, v);
        }
      }
    }
  }
};

}  // namespace nt
}  // namespace sgemm

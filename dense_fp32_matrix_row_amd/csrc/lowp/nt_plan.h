// nt_plan.h -- which tiles take an 8-bit product D = A * B^T (fp8_gemm.hip,
// int8_gemm.hip), and the launches of the small ones.  Host-side, from the sizes
// alone; what a tile costs is a model's, one for each kind of product.
#pragma once

#include "nt_direct.h"

namespace sgemm {
namespace nt {

enum class Way { kSmall16, kSmall32, kSmall64, kLoopSquare, kLoop128, kLoop256, kRows, kColumns };
struct Choice {
  Way way;
  int at;  // kRows, kColumns: where D is cut in two
  double us;
};

// Tile and block of a way.
struct TileShape {
  int rows, cols, threads;
};
template <class T>
constexpr bool is_shape(TileShape t) {
  return t.rows == T::BM && t.cols == T::BN && t.threads == T::threads;
}

// Of a small tile (16, 32 or 64 square), in us: what a launch takes, what one of
// its wavefronts' steps takes alone, and what a step of one block takes among many.
struct SmallCost {
  double base, alone, among;
};

// A model has
//   SmallCost small(int i): of the tile of 16 << i;
//   void loops(M, N, steps, offer): offer(way, us) for each large tile;
//   bool cuts_rows(t): whether rows beyond a multiple of t may be taken apart;
//   TileShape shape(way).
template <class Model>
Choice choose(const Model& model, int M, int N, int K, bool loops, int cuts) {
  const double steps = static_cast<double>(ceil_div(K, kStep)), each = static_cast<double>(ceil_div(K, 8 * kStep));
  Choice best{};
  const auto offer = [&](Way w, int at, double us) {
    if (us < best.us) best = Choice{w, at, us};
  };
  for (int i = 0; i < 3; ++i) {
    const SmallCost c = model.small(i);
    const double blocks = static_cast<double>(ceil_div(M, 16 << i) * ceil_div(N, 16 << i));
    const double us = c.base + each * (c.alone > c.among * blocks ? c.alone : c.among * blocks);
    if (i == 0) best = Choice{Way::kSmall16, 0, us};
    else offer(i == 1 ? Way::kSmall32 : Way::kSmall64, 0, us);
  }
  if (!loops) return best;
  model.loops(M, N, steps, [&](Way w, double us) { offer(w, 0, us); });
  // rows or columns that hardly fill their tiles apart from the rest
  for (int t = 128; cuts > 0 && t <= 256; t *= 2) {
    if (N > t && N % t) {
      const int at = N - N % t;
      offer(Way::kColumns, at, choose(model, M, at, K, loops, cuts - 1).us + choose(model, M, N - at, K, loops, 0).us);
    }
    if (model.cuts_rows(t) && M > t && M % t) {
      const int at = M - M % t;
      offer(Way::kRows, at, choose(model, at, N, K, loops, cuts - 1).us + choose(model, M - at, N, K, loops, 0).us);
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
constexpr int kCuts = 2;

template <class Model>
void plan(const Model& model, Plan& p, int m0, int n0, int M, int N, int K, bool loops, int cuts) {
  const Choice c = choose(model, M, N, K, loops, cuts);
  if (c.way != Way::kRows && c.way != Way::kColumns) {
    p.piece[p.count++] = Piece{c.way, m0, n0, M, N, 0, 0};
    return;
  }
  const bool rows = c.way == Way::kRows;
  const Choice inner = choose(model, rows ? c.at : M, rows ? N : c.at, K, loops, cuts - 1);
  if (inner.way == (rows ? Way::kColumns : Way::kRows)) {  // both edges, with small tiles of one size: these in one launch
    const int m = rows ? c.at : inner.at, n = rows ? inner.at : c.at;
    const Way right = choose(model, M, N - n, K, loops, 0).way, low = choose(model, M - m, n, K, loops, 0).way;
    if (right == low && right <= Way::kSmall64) {
      plan(model, p, m0, n0, m, n, K, loops, 0);
      p.piece[p.count++] = Piece{right, m0, n0, M, N, m, n};
      return;
    }
  }
  if (rows) {
    plan(model, p, m0, n0, c.at, N, K, loops, cuts - 1);
    plan(model, p, m0 + c.at, n0, M - c.at, N, K, loops, 0);
  } else {
    plan(model, p, m0, n0, M, c.at, K, loops, cuts - 1);
    plan(model, p, m0, n0 + c.at, M, N - c.at, K, loops, 0);
  }
}

// Blocks of a launch: one a tile, but small tiles past what a launch takes, which
// the blocks walk.
template <class Model>
int64_t blocks_of(const Model& model, const Piece& p) {
  const TileShape t = model.shape(p.way);
  const int64_t tiles = ceil_div(p.M, t.rows) * ceil_div(p.N - p.skip_n, t.cols) +
                        ceil_div(p.M - p.skip_m, t.rows) * (p.skip_n / t.cols);
  const int64_t cap = kMaxWorkItems / t.threads;
  return tiles < cap ? tiles : cap;
}

inline Side from_row(Side o, int row, int scale_bytes) {  // row: a multiple of 128
  o.p += row * o.ld;
  o.s = static_cast<const uint8_t*>(o.s) + (row >> o.shift) * o.s_row * scale_bytes;
  o.rows -= row;
  return o;
}

// The tiles from column n0, all rows; then those from row m0 left of it.
struct Part {
  int tiles_m, n0;
  int64_t tiles;
  int low_m, m0;
};

// Small tiles, whose blocks walk them; out(m, n, v) takes four neighbours' sums.
template <class D, class E>
__global__ __launch_bounds__(D::threads, 2) void k_direct(Side A, Side B, int K, E out, Part part, int64_t tiles) {
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
// edges (8-bit floats, 2050 x 2049 x 4096, float result: 51 -> 47 us); all of it for 0, 0.
template <class D, class E>
void launch_direct(const Side& A, const Side& B, int K, const E& out, int m0, int n0, unsigned blocks, hipStream_t s) {
  Part part;
  const int64_t tm = ceil_div(out.M, D::BM), low = ceil_div(out.M - m0, D::BM);
  part.tiles_m = static_cast<int>(tm);
  part.n0 = n0;
  part.tiles = tm * ceil_div(out.N - n0, D::BN);
  part.low_m = static_cast<int>(low);
  part.m0 = m0;
  const int64_t tiles = part.tiles + low * (n0 / D::BN);
  hipLaunchKernelGGL((k_direct<D, E>), dim3(blocks), dim3(D::threads), 0, s, A, B, K, out, part, tiles);
}

// The small tiles of a way, over the part of D that launch_direct takes.
template <class P, class E>
void launch_small(Way way, const Side& A, const Side& B, int K, const E& out, int m0, int n0, unsigned blocks,
                  hipStream_t s) {
  if (way == Way::kSmall16) launch_direct<Direct<P, 1, 1, 8>>(A, B, K, out, m0, n0, blocks, s);
  else if (way == Way::kSmall32) launch_direct<Direct<P, 2, 2, 8>>(A, B, K, out, m0, n0, blocks, s);
  else launch_direct<Direct<P, 4, 4, 8>>(A, B, K, out, m0, n0, blocks, s);
}

}  // namespace nt
}  // namespace sgemm

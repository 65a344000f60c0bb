// gradients.hip -- hip_gradient_norm, hip_gradient_clip and hip_gradient_clip_by: the
// norm over many tensors, and scaling by it.
//
// Bound by memory: every element is read for the norm, and again, and written,
// where it is scaled.  All tensors' elements are cut into chunks of one size, which
// a grid of blocks walks, whatever the tensors' own sizes; a table says which
// tensor a chunk lies in.  (But rows shorter than a chunk, of strided tensors, are taken an
// element at a time, with a division each: a fifth to a third of that rate.)  The norm's launch leaves a sum for each block, and each
// block of the next launch adds them up for itself in the same order: no atomics,
// no third launch.
//
// One MI355X, kernels alone: the norm of 1 GiB of floats in 48 tensors 188 us (5.7
// TB/s), scaled into others 629 us in all (a copy alone takes 441); 200 tensors, 64M
// elements of mixed types, in place and within the limit, 51 us (205 MB at 5.4 TB/s, a
// launch each for the table's two parts and 5 us to find that nothing is to be
// written); 4 tensors with 1M floats in all 6.8 us, two launches.  Scaled in place: the 1
// GiB in 48 tensors 642 us, the 200 tensors of bf16 72.  Strided and in place: 48 tensors of
// 4096 rows of 4000 bf16, 4096 apart, 3.23 ms (norm 1.49; 1.1 TB/s), of floats 3.70 (1.61; 2.0).
#include <algorithm>
#include <limits>
#include <vector>

#include "../../../include/gradients.h"
#include "rows.h"

namespace sgemm {
namespace {

// A tensor in the table: where it lies, its first chunk of all tensors', and its type;
// one of several rows has a second slot behind it, of the same first chunk.
struct Slot {
  int64_t x, y, cols;  // addresses; or rows, ldx, ldy
  uint32_t first;
  int32_t kind;  // the type, with kRows where a slot follows; kSecond
};
constexpr int32_t kRows = 4, kSecond = 8;
static_assert(sizeof(Slot) == 32);

constexpr int kInline = 120;  // slots that fit a launch's arguments (4 KiB)
struct Table {
  Slot e[kInline];
};
constexpr int kThreads = 256;
constexpr int64_t kBlocks = 2048;  // at most, of a launch: eight for each CU
constexpr int64_t kPartBytes = kBlocks * 8;

// The slot of the tensor that a chunk lies in: the last whose first chunk is not behind
// it (or the one before), found 64 at a time.
__device__ __forceinline__ int find(const Slot* e, int count, uint32_t chunk) {
  int lo = 0, n = count;
  while (n > 1) {
    const int lane = threadIdx.x % 64, step = (n + 63) / 64;
    const bool before = lane * step < n && e[lo + min(lane * step, n - 1)].first <= chunk;
    const int at = (__popcll(__ballot(before)) - 1) * step;
    lo += at;
    n = min(step, n - at);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  return e[lo].kind == kSecond ? lo - 1 : lo;
}

// 16 bytes of elements.
template <class T>
using Wide = Pack<16 / sizeof(T), T>;

// Calls one(i) for every element i < n and wide(i) for those that lie in whole 16
// bytes from `p` on, four at a time, spread over the block's threads.
template <class T, class W, class O>
__device__ __forceinline__ void walk(const T* p, int n, const W& wide, const O& one) {
  constexpr int kWide = 16 / sizeof(T);
  const int head = min(n, static_cast<int>((16 - reinterpret_cast<uintptr_t>(p) % 16) % 16 / sizeof(T)));
  const int count = (n - head) / kWide;
  int t = threadIdx.x;
  for (; t + 3 * kThreads < count; t += 4 * kThreads) wide(head + t * kWide, std::integral_constant<int, 4>{});
  for (; t < count; t += kThreads) wide(head + t * kWide, std::integral_constant<int, 1>{});
  const int rest = n - head - count * kWide;  // before and behind
  for (int i = threadIdx.x; i < head + rest; i += kThreads) one(i < head ? i : head + count * kWide + (i - head));
}

template <class T>
__device__ __forceinline__ double square(T x) {
  const double d = static_cast<double>(to_float(x));
  return d * d;
}

// In double: a float's square fits, no sum of 2^60 of them passes its range, and the
// instructions hide behind the loads.
struct Squares {
  double sum = 0.0;
  template <class T>
  __device__ __forceinline__ void flat(const T* x, T*, int n) {
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    walk(
        x, n,
        [&](int i, auto many) {
          Wide<T> v[many.value];
#pragma unroll
          for (int k = 0; k < many.value; ++k) v[k] = load_pack<16 / sizeof(T)>(x + i + k * (kThreads * (16 / sizeof(T))));
#pragma unroll
          for (int k = 0; k < many.value; ++k)
#pragma unroll
            for (int j = 0; j < 16 / int(sizeof(T)); ++j) {
              const double d = static_cast<double>(to_float(v[k].v[j]));
              s[j % 4] = fma(d, d, s[j % 4]);
            }
        },
        [&](int i) { s[0] += square(x[i]); });
    sum += (s[0] + s[1]) + (s[2] + s[3]);
  }
  template <class T>
  __device__ __forceinline__ void one(const T* x, T*) { sum += square(*x); }
};

// x c, with c = f 2^-64 where c is too small for a float's bits (a norm past 10^38),
// f and 1 elsewhere.
struct Scale {
  float f, shift;
  __device__ __forceinline__ explicit Scale(double c)
      : f(static_cast<float>(c < 0x1p-64 ? c * 0x1p64 : c)), shift(c < 0x1p-64 ? 0x1p-64f : 1.0f) {}
  __device__ __forceinline__ float operator()(float x) const { return x * f * shift; }
  template <class T>
  __device__ __forceinline__ void flat(const T* x, T* y, int n) {
    walk(
        x, n,
        [&](int i, auto many) {
          constexpr int kWide = 16 / sizeof(T);
          Wide<T> v[many.value];
#pragma unroll
          for (int k = 0; k < many.value; ++k) v[k] = load_pack<kWide>(x + i + k * (kThreads * kWide));
#pragma unroll
          for (int k = 0; k < many.value; ++k) {
#pragma unroll
            for (int j = 0; j < kWide; ++j) from_float((*this)(to_float(v[k].v[j])), v[k].v[j]);
            store_pack(y + i + k * (kThreads * kWide), v[k]);
          }
        },
        [&](int i) { one(x + i, y + i); });
  }
  template <class T>
  __device__ __forceinline__ void one(const T* x, T* y) { from_float((*this)(to_float(*x)), *y); }
};

// Chunk k of a tensor: a piece of a row, or several rows shorter than a chunk.
template <class T, class F>
__device__ __forceinline__ void do_chunk(const Slot* e, uint32_t k, int chunk, F& f) {
  const T* const x = reinterpret_cast<const T*>(e->x);
  T* const y = reinterpret_cast<T*>(e->y);
  const int64_t cols = e->cols;
  if (!(e->kind & kRows)) {
    const int64_t at = int64_t(k) * chunk;
    f.flat(x + at, y + at, static_cast<int>(min(int64_t(chunk), cols - at)));
    return;
  }
  const int64_t rows = e[1].x, ldx = e[1].y, ldy = e[1].cols;
  if (cols >= chunk) {
    const int64_t per = ceil_div(cols, chunk), row = k / per, at = (k - row * per) * chunk;
    f.flat(x + row * ldx + at, y + row * ldy + at, static_cast<int>(min(int64_t(chunk), cols - at)));
  } else {
    const int few = static_cast<int>(cols), per = chunk / few;
    const int64_t row = int64_t(k) * per;
    const int count = static_cast<int>(min(int64_t(per), rows - row)) * few;
    for (int i = threadIdx.x; i < count; i += kThreads)
      f.one(x + (row + i / few) * ldx + i % few, y + (row + i / few) * ldy + i % few);
  }
}

// The chunks of a block, in order.
template <class F>
__device__ __forceinline__ void do_chunks(const Slot* table, int count, uint32_t chunks, int chunk, bool skip_in_place, F& f) {
  for (int64_t at = blockIdx.x; at < chunks; at += gridDim.x) {
    const uint32_t k = static_cast<uint32_t>(at);
    const Slot* const e = table + find(table, count, k);
    if (skip_in_place && e->x == e->y) continue;
    const int type = e->kind & 3;
    if (type == HIP_GRADIENT_F32) do_chunk<float>(e, k - e->first, chunk, f);
    else if (type == HIP_GRADIENT_BF16) do_chunk<bf16>(e, k - e->first, chunk, f);
    else do_chunk<_Float16>(e, k - e->first, chunk, f);
  }
}

struct Add {
  __device__ __forceinline__ double operator()(double a, double b) const { return a + b; }
};

__device__ __forceinline__ void norm_body(const Slot* table, int count, uint32_t chunks, int chunk, double* parts) {
  using S = RowShape<kThreads, 1>;
  __shared__ double meet[S::threads / 64][1];
  Squares f;
  do_chunks(table, count, chunks, chunk, false, f);
  double sum[1] = {f.sum};
  join_row<S>(sum, meet, Add{});
  if (threadIdx.x == 0) parts[blockIdx.x] = sum[0];
}
__global__ __launch_bounds__(kThreads) void k_norm(Table t, int count, uint32_t chunks, int chunk, double* parts) {
  norm_body(t.e, count, chunks, chunk, parts);
}
__global__ __launch_bounds__(kThreads) void k_norm_long(const Slot* __restrict__ table, int count, uint32_t chunks, int chunk,
                                                        double* parts) {
  norm_body(table, count, chunks, chunk, parts);
}

// The norm from the blocks' sums, the same in every thread of every block (2048 of
// them at most, 16 KB that the L2 holds: a launch between would cost more).
__device__ __forceinline__ double join_parts(const double* parts, int count) {
  using S = RowShape<kThreads, 1>;
  __shared__ double meet[S::threads / 64][1];
  double sum[1] = {0.0};
  for (int i = threadIdx.x; i < count; i += kThreads) sum[0] += parts[i];
  join_row<S>(sum, meet, Add{});
  return sqrt(sum[0]);
}
__global__ __launch_bounds__(kThreads) void k_finish(const double* parts, int count, float* norm) {
  const double v = join_parts(parts, count);
  if (threadIdx.x == 0) *norm = static_cast<float>(v);
}

struct Limit {
  const double* parts;  // the blocks' sums, or NULL:
  int count;
  const float* given;  // the norm
  float* norm;         // where it goes, or NULL
  double max_norm, eps;
  bool all_in_place;
};
__device__ __forceinline__ void clip_body(const Slot* table, int count, uint32_t chunks, int chunk, const Limit& l) {
  const double norm = l.given ? static_cast<double>(*l.given) : join_parts(l.parts, l.count);
  if (l.norm && blockIdx.x == 0 && threadIdx.x == 0) *l.norm = static_cast<float>(norm);
  const double all = norm + l.eps, most = l.max_norm;
  const bool same = all <= most;  // not for a NaN
  Scale f(same ? 1.0 : most / all);
  if (same && l.all_in_place) return;
  do_chunks(table, count, chunks, chunk, same, f);
}
__global__ __launch_bounds__(kThreads) void k_clip(Table t, int count, uint32_t chunks, int chunk, Limit l) {
  clip_body(t.e, count, chunks, chunk, l);
}
__global__ __launch_bounds__(kThreads) void k_clip_long(const Slot* __restrict__ table, int count, uint32_t chunks, int chunk,
                                                        Limit l) {
  clip_body(table, count, chunks, chunk, l);
}

// Slots that come as arguments into memory.
__global__ __launch_bounds__(64) void k_table(Table t, int count, Slot* to) {
  for (int i = threadIdx.x; i < count; i += 64) to[i] = t.e[i];
}

// What a call works on: the tensors that have elements.
struct Tensor {
  uintptr_t x, y;
  int64_t rows, cols, ldx, ldy;
  int type;
};
struct Work {
  std::vector<Tensor> tensors;
  std::vector<Slot> slots;
  uint32_t chunks = 0;
  int chunk = 0;
  bool all_in_place = true;
};

// Sizes and strides below 2^40 and no tensor that reaches over 2^44 elements: more than
// memory, less than what overflows below.
bool valid(const hip_gradient& g, bool clip) {
  constexpr int64_t kSide = int64_t(1) << 40;
  if (g.rows < 0 || g.cols < 0 || g.rows > kSide || g.cols > kSide || g.type < 0 || g.type > HIP_GRADIENT_F16) return false;
  if (g.rows == 0 || g.cols == 0) return true;
  const uintptr_t align = g.type == HIP_GRADIENT_F32 ? 4 : 2;
  const auto bad = [&](const void* p, int64_t ld) {
    if (!p || reinterpret_cast<uintptr_t>(p) % align) return true;
    return g.rows > 1 && (ld < g.cols || ld > kSide || static_cast<double>(g.rows) * static_cast<double>(ld) > 0x1p44);
  };
  return !bad(g.x, g.ldx) && !(clip && bad(g.y, g.ldy));
}

// False where there are more chunks than a number of 32 bits counts.
bool collect(Work& w, int count, const hip_gradient* tensors, bool clip) {
  w.tensors.reserve(count);
  w.slots.reserve(count);
  double total = 0.0;
  for (int i = 0; i < count; ++i) {
    const hip_gradient& g = tensors[i];
    if (g.rows == 0 || g.cols == 0) continue;
    Tensor t{reinterpret_cast<uintptr_t>(g.x), reinterpret_cast<uintptr_t>(clip ? g.y : g.x), g.rows, g.cols, g.ldx,
             clip ? g.ldy : g.ldx, static_cast<int>(g.type)};
    total += static_cast<double>(t.rows) * static_cast<double>(t.cols);
    if (t.rows > 1 && t.ldx == t.cols && t.ldy == t.cols && t.rows < (int64_t(1) << 40) / t.cols) {  // dense
      t.cols *= t.rows;
      t.rows = 1;
    }
    w.all_in_place = w.all_in_place && t.x == t.y;
    w.tensors.push_back(t);
  }
  // two chunks or more for each block where there is that much, down to four 16-byte
  // loads a thread, and eight for an even end where there is more
  w.chunk = 4096;
  while (w.chunk < 16384 && total / w.chunk > 2 * kBlocks) w.chunk *= 2;
  uint64_t chunks = 0;
  for (const Tensor& t : w.tensors) {
    const uint32_t first = static_cast<uint32_t>(chunks);
    w.slots.push_back(Slot{static_cast<int64_t>(t.x), static_cast<int64_t>(t.y), t.cols, first, t.type | (t.rows > 1 ? kRows : 0)});
    if (t.rows > 1) w.slots.push_back(Slot{t.rows, t.ldx, t.ldy, first, kSecond});
    const double many = static_cast<double>(t.rows) * static_cast<double>(ceil_div(t.cols, w.chunk));
    if (t.rows > 1 && t.cols < w.chunk) chunks += ceil_div(t.rows, w.chunk / t.cols);
    else if (many < 1e10) chunks += t.rows * ceil_div(t.cols, w.chunk);
    else return false;
    if (chunks > std::numeric_limits<uint32_t>::max()) return false;
  }
  w.chunks = static_cast<uint32_t>(chunks);
  return true;
}

// The sum of floor((a i + b) / m) over i < n, modulo 2^64.  Whole multiples of m in a and b
// come out; what is left counts the points under a line, which as many columns of its
// inverse hold.
uint64_t sum_of_floors(uint64_t n, uint64_t m, uint64_t a, uint64_t b) {
  const uint64_t pairs = n % 2 ? n * (n / 2) : n / 2 * (n - 1), whole = a / m * pairs + b / m * n;
  const uint64_t top = a % m * n + b % m;
  return top < m ? whole : whole + sum_of_floors(top / m, a % m, m, top % m);
}

// Whether what a clipping call writes overlaps anything else that it touches.
struct Range {
  int64_t from, to;       // bytes
  int64_t row, ld, rows;  // `rows` of `row` bytes, ld apart
  bool writes;
};
// How many of a's rows begin before `at`.
int64_t rows_before(const Range& a, int64_t at) {
  if (at <= a.from) return 0;
  return std::min(a.rows, ceil_div(at - a.from, a.ld));
}
bool meet(const Range& a, const Range& b) {
  if (!(a.writes || b.writes) || a.to <= b.from || b.to <= a.from) return false;
  if (a.ld == b.ld) {  // two sets of columns of one matrix (a division instead of a dozen)
    const int64_t off = a.from <= b.from ? (b.from - a.from) % a.ld : (a.ld - (a.from - b.from) % a.ld) % a.ld;
    return off < a.row || off + b.row > a.ld;
  }
  const int64_t last = b.from + (b.rows - 1) * b.ld;  // b's last row
  // a's rows that begin before b's first or within its last; and those between, which meet a
  // row of b where its begin less b's, modulo b.ld, is less than b.row or more than b.ld - a.row
  const int64_t first = rows_before(a, b.from), past = rows_before(a, last);
  if (rows_before(a, b.from - a.row + 1) < first || past < rows_before(a, last + b.row)) return true;
  if (first == past) return false;
  const int64_t near = a.row + b.row - 1;  // as many of the b.ld places
  if (near >= b.ld) return true;
  const uint64_t n = past - first, at = a.from + first * a.ld - b.from + a.row - 1 + b.ld;
  return sum_of_floors(n, b.ld, a.ld, at) != sum_of_floors(n, b.ld, a.ld, at - near);
}
bool overlaps(const Work& w, const float* norm, bool writes_norm) {
  std::vector<Range> ranges;
  ranges.reserve(2 * w.tensors.size() + 1);
  for (const Tensor& t : w.tensors) {
    const int64_t size = t.type == HIP_GRADIENT_F32 ? 4 : 2, row = t.cols * size;
    const auto add = [&](uintptr_t p, int64_t ld, bool writes) {
      const int64_t at = static_cast<int64_t>(p), step = t.rows > 1 ? ld * size : row;
      ranges.push_back(Range{at, at + (t.rows - 1) * step + row, row, step, t.rows, writes});
    };
    add(t.y, t.ldy, true);
    if (t.x != t.y || (t.rows > 1 && t.ldx != t.ldy)) add(t.x, t.ldx, false);
  }
  if (norm) {
    const int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(norm));
    ranges.push_back(Range{at, at + 4, 4, 4, 1, writes_norm});
  }
  const auto before = [](const Range& a, const Range& b) { return a.from < b.from; };
  if (!std::is_sorted(ranges.begin(), ranges.end(), before)) std::sort(ranges.begin(), ranges.end(), before);
  std::vector<const Range*> open;  // those that reach past the present one's begin
  for (const Range& r : ranges) {
    size_t kept = 0;
    for (const Range* o : open) {
      if (o->to <= r.from) continue;
      if (meet(*o, r)) return true;
      open[kept++] = o;
    }
    open.resize(kept);
    open.push_back(&r);
  }
  return false;
}

// The slots into memory.
void put_table(const Work& w, Slot* to, hipStream_t stream) {
  const int n = static_cast<int>(w.slots.size());
  for (int at = 0; at < n; at += kInline) {
    Table t;
    const int some = std::min(kInline, n - at);
    std::copy_n(w.slots.begin() + at, some, t.e);
    hipLaunchKernelGGL(k_table, dim3(1), dim3(64), 0, stream, t, some, to + at);
  }
}
Table inline_table(const Work& w) {
  Table t;
  std::copy(w.slots.begin(), w.slots.end(), t.e);
  return t;
}

struct Memory {
  double* parts;
  Slot* table;
};
Memory memory(void* workspace) {
  uint8_t* const p = static_cast<uint8_t*>(workspace);
  return Memory{reinterpret_cast<double*>(p), reinterpret_cast<Slot*>(p + kPartBytes)};
}
int64_t bytes_for(int count) { return kPartBytes + (2 * count > kInline ? 2 * int64_t(count) * int64_t(sizeof(Slot)) : 0); }

unsigned blocks_for(const Work& w) { return static_cast<unsigned>(std::min(int64_t(w.chunks), kBlocks)); }

void launch_norm(const Work& w, const Memory& m, hipStream_t stream) {
  const int n = static_cast<int>(w.slots.size());
  if (n == 0) return;
  if (n <= kInline)
    hipLaunchKernelGGL(k_norm, dim3(blocks_for(w)), dim3(kThreads), 0, stream, inline_table(w), n, w.chunks, w.chunk, m.parts);
  else
    hipLaunchKernelGGL(k_norm_long, dim3(blocks_for(w)), dim3(kThreads), 0, stream, m.table, n, w.chunks, w.chunk, m.parts);
}
void launch_clip(const Work& w, const Memory& m, const Limit& l, hipStream_t stream) {
  const int n = static_cast<int>(w.slots.size());
  const dim3 grid(std::max(1u, blocks_for(w)));
  if (n <= kInline) hipLaunchKernelGGL(k_clip, grid, dim3(kThreads), 0, stream, inline_table(w), n, w.chunks, w.chunk, l);
  else hipLaunchKernelGGL(k_clip_long, grid, dim3(kThreads), 0, stream, m.table, n, w.chunks, w.chunk, l);
}

bool bad_count(int count) { return count < 0 || count > HIP_GRADIENT_MAX_COUNT; }
bool off256(const void* p) { return reinterpret_cast<uintptr_t>(p) % 256 != 0; }

// What the three calls share, their arguments' numbers being the same but the
// norm's: 0, or a status.
int begin(Work& w, int count, const hip_gradient* tensors, bool clip, const float* norm, bool writes_norm, void* workspace,
          long long workspace_bytes, int workspace_at, hipStream_t stream) {
  if (bad_count(count)) return -1;
  if (count > 0 && tensors == nullptr) return -2;
  for (int i = 0; i < count; ++i)
    if (!valid(tensors[i], clip)) return -2;
  if (workspace == nullptr || off256(workspace)) return -workspace_at;
  if (workspace_bytes < bytes_for(count)) return -(workspace_at + 1);
  if (!collect(w, count, tensors, clip)) return -2;
  if (clip && overlaps(w, norm, writes_norm)) return -2;
  if (static_cast<int>(w.slots.size()) > kInline) put_table(w, memory(workspace).table, stream);
  return 0;
}

int clip(int count, const hip_gradient* tensors, double max_norm, double eps, float* norm, const float* given,
         void* workspace, long long workspace_bytes, hipStream_t stream) {
  if (!(max_norm >= 0.0)) return -3;
  if (!(eps >= 0.0) || eps == std::numeric_limits<double>::infinity()) return -4;
  Work w;
  const int status = begin(w, count, tensors, true, given ? given : norm, !given, workspace, workspace_bytes, 6, stream);
  if (status != 0) return status;
  const Memory m = memory(workspace);
  if (!given) launch_norm(w, m, stream);
  if (w.chunks > 0 || norm)
    launch_clip(w, m, Limit{m.parts, static_cast<int>(blocks_for(w)), given, norm, max_norm, eps, w.all_in_place}, stream);
  return static_cast<int>(hipGetLastError());
}

// No exception leaves a C function.
template <class F>
int guarded(const F& f) {
  try {
    return f();
  } catch (...) {
    return static_cast<int>(hipErrorOutOfMemory);
  }
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" {

int hip_gradient_workspace(int count, long long* bytes) {
  if (bad_count(count)) return -1;
  if (bytes) *bytes = bytes_for(count);
  return 0;
}

int hip_gradient_norm(int count, const hip_gradient* tensors, float* norm, void* workspace, long long workspace_bytes,
                      hipStream_t stream) {
  return guarded([&] {
    if (norm == nullptr) return -3;
    Work w;
    const int status = begin(w, count, tensors, false, nullptr, false, workspace, workspace_bytes, 4, stream);
    if (status != 0) return status;
    const Memory m = memory(workspace);
    launch_norm(w, m, stream);
    hipLaunchKernelGGL(k_finish, dim3(1), dim3(kThreads), 0, stream, m.parts, static_cast<int>(blocks_for(w)), norm);
    return static_cast<int>(hipGetLastError());
  });
}

int hip_gradient_clip(int count, const hip_gradient* tensors, double max_norm, double eps, float* norm, void* workspace,
                      long long workspace_bytes, hipStream_t stream) {
  return guarded([&] { return clip(count, tensors, max_norm, eps, norm, nullptr, workspace, workspace_bytes, stream); });
}

int hip_gradient_clip_by(int count, const hip_gradient* tensors, double max_norm, double eps, const float* norm,
                         void* workspace, long long workspace_bytes, hipStream_t stream) {
  return guarded([&] {
    if (norm == nullptr) return -5;
    return clip(count, tensors, max_norm, eps, nullptr, norm, workspace, workspace_bytes, stream);
  });
}

const char* hip_gradient_norm_status_string(int status) {
  switch (status) {
    case 0: return "success";
    case -1: return "argument 1 (count) is negative or above HIP_GRADIENT_MAX_COUNT";
    case -2: return "argument 2 (tensors) is NULL, or has a bad size, stride, type or pointer";
    case -3: return "argument 3 (norm) is NULL";
    case -4: return "argument 4 (workspace) is NULL or not 256-byte aligned";
    case -5: return "argument 5 (workspace_bytes) is less than hip_gradient_workspace says";
    default: break;
  }
  if (status > 0) return hipGetErrorString(static_cast<hipError_t>(status));
  return "unknown status";
}

const char* hip_gradient_clip_status_string(int status) {
  switch (status) {
    case 0: return "success";
    case -1: return "argument 1 (count) is negative or above HIP_GRADIENT_MAX_COUNT";
    case -2: return "argument 2 (tensors) is NULL, has a bad size, stride, type or pointer, or what is written overlaps";
    case -3: return "argument 3 (max_norm) is negative or NaN";
    case -4: return "argument 4 (eps) is negative, infinite or NaN";
    case -5: return "argument 5 (norm) is NULL";
    case -6: return "argument 6 (workspace) is NULL or not 256-byte aligned";
    case -7: return "argument 7 (workspace_bytes) is less than hip_gradient_workspace says";
    default: break;
  }
  if (status > 0) return hipGetErrorString(static_cast<hipError_t>(status));
  return "unknown status";
}

}  // extern "C"

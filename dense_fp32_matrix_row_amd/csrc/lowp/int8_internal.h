// int8_internal.h -- the integer operators' kernels by their checked arguments
// (not installed; the public interface is include/int8.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sgemm {

// rows > 0, cols > 0
void launch_int8_quantize(int rows, int cols, const void* x, int x_type, int64_t ldx, int8_t* q, int64_t ldq, float* s,
                          hipStream_t stream);

struct Int8Product {
  int M, N, K;  // M > 0, N > 0
  const void* a;
  int64_t lda;
  const float* sa;
  int64_t sa_inc;
  const void* b;
  int64_t ldb;
  const float* sb;
  int64_t sb_inc;
  const void* bias;
  int bias_type;
  void* d;
  int64_t ldd;
  int d_type;
};
void launch_int8_gemm(const Int8Product& p, hipStream_t stream);

}  // namespace sgemm

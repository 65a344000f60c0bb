/*
 * int8.h -- products of 8-bit integers with a scale for each row of both
 * operands (each token and each channel), on the AMD Instinct MI355X (gfx950),
 * as linear layers are served.  Part of libsgemm; the conventions of sgemm.h hold
 * (device pointers, row-major storage, work enqueued on `stream` without
 * synchronising, argument errors found on the host before anything is
 * enqueued, no state kept between calls).
 *
 * A quantised matrix is a pair (Q, S): codes Q, rows x cols, one signed byte
 * each, row i from Q + i*ldq; and a float scale for each row, S[i * s_inc]
 * (s_inc 0: one for all).  It stands for Q[i][j] * S[i * s_inc].
 *
 * Status codes: 0 enqueued; -i the i-th argument is invalid; > 0 the
 * hipError_t of a failed launch.  hip_int8_*_status_string name them.
 */
#ifndef LIBSGEMM_INT8_H
#define LIBSGEMM_INT8_H

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* element types of the matrices that are not quantised */
#define HIP_INT8_F32 0
#define HIP_INT8_BF16 1
#define HIP_INT8_F16 2

/* longest sum: 131071 products of -128 by -128 fit 32 bits */
#define HIP_INT8_MAX_K 131071
/* largest row stride (bytes) of an operand of a product */
#define HIP_INT8_MAX_LD (1 << 23)

/*
 * Quantises the rows of X (rows x cols, row stride ldx elements).  With
 * a = max(largest |x| of the row, 2^-100):
 *   S_i = a / 127, rounded to float;
 *   code = x / S_i rounded once to an integer, ties to even (the exact
 *   quotient is rounded, not its float approximation): -127 .. 127.
 * A row that holds an infinity or a NaN gets a NaN scale and codes of 0.  Bytes of
 * a row of Q past cols are not written.  Pointers need the alignment of their
 * element type; Q and S must not overlap X.  rows == 0 or cols == 0: nothing is done.
 *
 * Arguments are numbered from 1: rows, cols, X, x_type, ldx, Q, ldq, S, stream.
 */
int hip_int8_quantize(int rows, int cols, const void *X, int x_type, int ldx, void *Q, int ldq, float *S,
                      hipStream_t stream);

/*
 * D <- A * B^T of quantised A (M x K) and B (N x K), plus a bias for each column:
 *   D_ij = (sum over k of A_ik B_jk) * SA_i * SB_j + bias_j.
 * The sum is exact; it is rounded to float, multiplied by SA_i and by SB_j as
 * floats, the bias added in the second multiplication's rounding, and the result
 * rounded to D's type.  Any code is allowed, -128 too.
 *   K: at most HIP_INT8_MAX_K.
 *   lda, ldb: multiples of 16 bytes (best of 128, the cache's lines), at most
 *   HIP_INT8_MAX_LD; A and B 16-byte aligned; a row is read up to the next multiple
 *   of 16 bytes (what lies past K has no influence).
 *   bias: N numbers of bias_type side by side, or NULL for none.
 *   D: M x N of type d_type, row stride ldd; element alignment suffices.  It must
 *   not overlap anything that is read.
 *   M == 0 or N == 0: nothing is done.  K == 0: D <- bias; A, B and their scales
 *   are not read.
 *
 * Arguments are numbered from 1: M, N, K, A, lda, SA, sa_inc, B, ldb, SB, sb_inc,
 * bias, bias_type, D, ldd, d_type, stream.
 */
int hip_int8_gemm(int M, int N, int K, const void *A, int lda, const float *SA, long long sa_inc,
                  const void *B, int ldb, const float *SB, long long sb_inc, const void *bias, int bias_type,
                  void *D, int ldd, int d_type, hipStream_t stream);

/*
 * What hip_int8_gemm enqueues for a shape, decided on the host from the sizes
 * alone without launching anything: *count launches over disjoint parts of D, at
 * most HIP_INT8_GEMM_MAX_LAUNCHES, described in launches[0 .. *count).  Either
 * pointer may be NULL.  0, or -1, -2, -3 as hip_int8_gemm.
 */
#define HIP_INT8_GEMM_MAX_LAUNCHES 3
typedef struct {
  int tile_m, tile_n;         /* of D a block sums at a time */
  int row0, col0, rows, cols; /* the part of D ... */
  int skip_rows, skip_cols;   /* ... but its first skip_rows rows of its first skip_cols columns */
  int threads;                /* of a block */
  long long workgroups;       /* workgroups * threads <= 2^31 */
} hip_int8_gemm_launch;
int hip_int8_gemm_plan(int M, int N, int K, hip_int8_gemm_launch *launches, int *count);

/*
 * Bytes of workspace that hip_int8_linear needs (host only, launches nothing).
 * 0, or -1, -2 for bad tokens or inputs.
 */
int hip_int8_linear_workspace(int tokens, int inputs, long long *bytes);

/*
 * Y <- X * W^T + bias of tokens X (tokens x inputs), quantised on the way as
 * hip_int8_quantize does, and a quantised weight W (outputs x inputs): what
 * hip_int8_quantize and hip_int8_gemm give, bit for bit.
 *   workspace: device memory of at least the bytes above (none for few tokens: then it
 *   may be NULL), 16-byte aligned; calls that overlap in time need workspaces of their
 *   own.
 * The rest as in hip_int8_quantize and hip_int8_gemm.
 *
 * Arguments are numbered from 1: tokens, inputs, outputs, X, x_type, ldx, W, ldw,
 * SW, sw_inc, bias, bias_type, Y, ldy, y_type, workspace, workspace_bytes, stream.
 */
int hip_int8_linear(int tokens, int inputs, int outputs, const void *X, int x_type, int ldx,
                    const void *W, int ldw, const float *SW, long long sw_inc, const void *bias, int bias_type,
                    void *Y, int ldy, int y_type, void *workspace, long long workspace_bytes, hipStream_t stream);

const char *hip_int8_quantize_status_string(int status);
const char *hip_int8_gemm_status_string(int status);
const char *hip_int8_linear_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* LIBSGEMM_INT8_H */

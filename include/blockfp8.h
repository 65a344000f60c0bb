/*
 * blockfp8.h -- 8-bit floating-point products with a scale for every block of
 * 128 elements, on the AMD Instinct MI355X (gfx950).  Part of libsgemm; the
 * conventions of sgemm.h hold (device pointers, row-major storage, work
 * enqueued on `stream` without synchronising, argument errors found on the
 * host before anything is enqueued, no state kept between calls).
 *
 * A quantised matrix is a pair (Q, S):
 *   Q  rows x cols codes, one byte each, OCP e4m3 (largest value 448, no
 *      infinity, NaN 0x7f / 0xff); row i starts at Q + i*ldq.
 *   S  one scale for each block of block_rows x 128 elements, block_rows 1
 *      or 128: the scale of element (i, j) is S[(i / block_rows) * s_row +
 *      (j / 128) * s_col] (s_row, s_col: strides in scales, any sign-free
 *      layout; the kernels read s_row == 1 fastest).
 *      HIP_FP8_SCALE_F32: a float s.  HIP_FP8_SCALE_E8M0: a byte e, the
 *      scale 2^(e - 127), 0xff NaN.
 * and stands for Q[i][j] * scale(i, j).  Blocks at the right and lower edge
 * may be partial.
 *
 * Status codes: 0 enqueued; -i the i-th argument is invalid; > 0 the
 * hipError_t of a failed launch.  hip_fp8_quantize_status_string and
 * hip_fp8_gemm_status_string name them.
 */
#ifndef LIBSGEMM_BLOCKFP8_H
#define LIBSGEMM_BLOCKFP8_H

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* element types of the matrices that are not quantised */
#define HIP_FP8_F32 0
#define HIP_FP8_BF16 1
#define HIP_FP8_F16 2

#define HIP_FP8_SCALE_F32 0
#define HIP_FP8_SCALE_E8M0 1

/* largest row stride (bytes) of an operand of hip_fp8_gemm */
#define HIP_FP8_MAX_LD (1 << 23)

/*
 * Quantises X (rows x cols, row stride ldx elements) and / or its transpose,
 * reading X once.
 *   (Q, S): X in blocks of block_rows x 128.
 *   (QT, ST): X^T (cols x rows) in blocks of block_rows x 128 of X^T, so with
 *   block_rows 1 each scale covers 128 rows of one column of X; with
 *   block_rows 128 the codes are Q's transposed.
 * Either pair may be NULL (both members), not both pairs.
 *
 * With a = max(largest |x| of the block, 2^-100):
 *   F32:  s = a / 448, rounded to float;
 *   E8M0: s = the smallest power of two with a <= 448 s;
 *   code = x / s rounded once to e4m3, ties to even (the exact quotient is
 *   rounded, not its float approximation).
 * A block that holds an infinity or a NaN gets a NaN scale and NaN codes.
 * Bytes of a row of Q past cols are not written.  Pointers need the alignment
 * of their element type; QT rows 4-byte alignment is faster, not required.
 *
 * Arguments are numbered from 1: rows, cols, X, x_type, ldx, block_rows,
 * scale_type, Q, ldq, S, s_row, s_col, QT, ldqt, ST, st_row, st_col, stream.
 */
int hip_fp8_quantize(int rows, int cols, const void *X, int x_type, int ldx,
                     int block_rows, int scale_type,
                     void *Q, int ldq, void *S, long long s_row, long long s_col,
                     void *QT, int ldqt, void *ST, long long st_row, long long st_col,
                     hipStream_t stream);

/*
 * D <- alpha * A * B^T + beta * C with A (M x K) and B (N x K) quantised:
 *   D_ij = alpha * sum over k of A_ik s_A(i, k) B_jk s_B(j, k) + beta * C_ij.
 * Both operands have the same scale_type, each its own block rows.  Sums are
 * float.  A 16-bit D is summed by the 8-bit matrix instructions, which cut the
 * products of eight neighbours along k 13 bits below the largest of them (an
 * error of 1.5e-5 on normal data, 2^-10 of the sum of magnitudes at most); a
 * float D is summed at half that rate with a float's bits throughout.
 * Where a partial sum or a block's s_A s_B passes float's range, D_ij is an
 * infinity or a NaN as the order of the sum, which depends on the sizes, has it.
 * Float scales, and scales of either type of a float D, multiply a block's sum as
 * floats: with b_block_rows 1 by s_A and then by s_B; with 128 by s_A s_B, rounded
 * to float first, which costs half the multiplications and, where s_A s_B is below
 * 2^-126, bits: an error of up to 2^-150 times the block's sum of code products.
 *   lda, ldb: multiples of 16 bytes, at most HIP_FP8_MAX_LD; A and B 16-byte
 *   aligned; a row is read up to the next multiple of 16 bytes (what lies
 *   past K has no influence).
 *   C, D: M x N of type c_type (HIP_FP8_F32 / BF16 / F16), row strides ldc,
 *   ldd; element alignment suffices.  C is not read if beta == 0 (may be
 *   NULL) and may be D itself (same ldc), but must not overlap it otherwise.
 *   M == 0 or N == 0: nothing is done.  K == 0 or alpha == 0: D <- beta * C,
 *   A and B are not read.
 *
 * Arguments are numbered from 1: M, N, K, alpha, A, lda, SA, sa_row, sa_col,
 * a_block_rows, B, ldb, SB, sb_row, sb_col, b_block_rows, scale_type, beta,
 * C, ldc, D, ldd, c_type, stream.
 */
int hip_fp8_gemm(int M, int N, int K, float alpha,
                 const void *A, int lda, const void *SA, long long sa_row, long long sa_col,
                 int a_block_rows,
                 const void *B, int ldb, const void *SB, long long sb_row, long long sb_col,
                 int b_block_rows, int scale_type,
                 float beta, const void *C, int ldc, void *D, int ldd, int c_type,
                 hipStream_t stream);

/*
 * What hip_fp8_gemm enqueues for a shape (alpha != 0, scales whose s_row is
 * small, as the quantiser lays them out), decided on the host from M, N, K and
 * c_type alone without launching anything: *count launches over disjoint parts
 * of D, at most HIP_FP8_GEMM_MAX_LAUNCHES, described in launches[0 .. *count).
 * Either pointer may be NULL.  0, or -1, -2, -3, -23 as hip_fp8_gemm.
 */
#define HIP_FP8_GEMM_MAX_LAUNCHES 3
typedef struct {
  int tile_m, tile_n;         /* of D a block sums at a time */
  int row0, col0, rows, cols; /* the part of D ... */
  int skip_rows, skip_cols;   /* ... but its first skip_rows rows of its first skip_cols columns */
  int threads;                /* of a block */
  long long workgroups;       /* workgroups * threads <= 2^31 */
} hip_fp8_gemm_launch;
int hip_fp8_gemm_plan(int M, int N, int K, int c_type, hip_fp8_gemm_launch *launches, int *count);

const char *hip_fp8_quantize_status_string(int status);
const char *hip_fp8_gemm_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* LIBSGEMM_BLOCKFP8_H */

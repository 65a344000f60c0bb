/*
 * orthogonal.h -- orthogonalising a matrix by Newton-Schulz products, as
 * optimisers that update a weight by the nearest semi-orthogonal matrix to its
 * momentum do.  Part of libsgemm; the conventions of sgemm.h hold (device
 * pointers, row-major storage, work enqueued on `stream` without
 * synchronising, argument errors found on the host first, no state kept).
 *
 *     X_0 = G / (|G|_F + eps)
 *     X_{i+1} = a_i X_i + (b_i S + c_i S^2) X_i,   S = X_i X_i^T
 *
 * for i < steps, with the polynomial's coefficients a_i, b_i, c_i given per
 * step.  A tall G (rows > cols) is iterated as G^T, the same result with the
 * smaller of the two S.
 */
#ifndef LIBSGEMM_ORTHOGONAL_H
#define LIBSGEMM_ORTHOGONAL_H

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define HIP_ORTHOGONAL_F32 0
#define HIP_ORTHOGONAL_BF16 1
#define HIP_ORTHOGONAL_F16 2

/* limits of one call */
#define HIP_ORTHOGONAL_MAX_SIZE (1 << 20) /* rows, cols */
#define HIP_ORTHOGONAL_MAX_STEPS 64

/*
 * Bytes of workspace that hip_orthogonalize needs for a batch of rows x cols
 * matrices of a type (host only, launches nothing).  0, or -1 .. -4 for a bad
 * batch, rows, cols or type.
 */
int hip_orthogonalize_workspace(int batch, int rows, int cols, int type, long long *bytes);

/*
 * X <- the Newton-Schulz iterate of G, for `batch` matrices.
 *   G, X  rows x cols of `type`, row strides ldg, ldx, matrix strides
 *         stride_g, stride_x (elements; not read for batch 1); element
 *         alignment suffices.  X may be G itself (same strides) and must not
 *         overlap it otherwise.
 *   coefficients  HOST array of 3 * steps floats a_0 b_0 c_0 a_1 ...; read
 *         before the call returns.
 *   workspace  device memory of at least the bytes above, 256-byte aligned;
 *         calls that overlap in time need workspaces of their own.
 * steps 0 gives G / (|G|_F + eps).  A zero matrix gives zeros (eps > 0).  A
 * matrix with an infinity or NaN gives NaN throughout; for steps 0 a NaN makes
 * all elements NaN, an infinity only the infinite ones (finite ones become 0).
 *
 * The norm is summed, and divided by, in double.  The products' operands are
 * kept as pairs of halfs and multiplied on the matrix cores with float sums.  A
 * pair has 22 significant bits of numbers down to 2^-18 of its matrix's range and
 * an absolute 2^-40 of the range below; each row and each column of X_i is
 * scaled by the root of its norm first, so that a row or column is computed as
 * float products would compute it, relative to its own norm, while that is above
 * 1e-7 of the largest, and loses a bit for each factor of 4 below.  The ranges
 * follow the polynomials' bounds on the singular values, which in X_0 are at most
 * 1: a polynomial may let them grow, until a float sum overflows (infinities, NaN).
 *
 * Status codes: 0 enqueued; -i the i-th argument is invalid (numbered from 1:
 * batch, rows, cols, type, G, ldg, stride_g, steps, coefficients, eps, X, ldx,
 * stride_x, workspace, workspace_bytes, stream); > 0 the hipError_t of a
 * failed launch.
 */
int hip_orthogonalize(int batch, int rows, int cols, int type,
                      const void *G, int ldg, long long stride_g,
                      int steps, const float *coefficients, float eps,
                      void *X, int ldx, long long stride_x,
                      void *workspace, long long workspace_bytes,
                      hipStream_t stream);

/*
 * Which tiles the three products of a step take, S = X X^T, P = a + b S + c S^2
 * and P X, decided on the host from the sizes alone without launching anything.
 * 0, or -1 .. -3 for a bad batch, rows or cols; all zeros where there is nothing
 * to do.
 */
typedef struct {
  int tile;          /* rows and columns of a block's tile */
  int parts;         /* of the sums' long side, joined by a second launch if > 1 */
  int cut, cut_tile; /* P X: the column from which on a launch of its own computes it, and its tile; 0: none */
} hip_orthogonalize_product;
int hip_orthogonalize_plan(int batch, int rows, int cols, hip_orthogonalize_product products[3]);

const char *hip_orthogonalize_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* LIBSGEMM_ORTHOGONAL_H */

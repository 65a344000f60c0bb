/*
 * layernorm.h -- layer norm's forward and backward pass on the AMD Instinct MI355X
 * (gfx950).  Part of libsgemm; the conventions of sgemm.h hold (device pointers,
 * row-major storage, work enqueued on `stream` without synchronising, argument
 * errors found on the host before anything is enqueued, no state kept between
 * calls).
 *
 * For each row x of X (rows x cols), with w and b a number for each column:
 *     mean = sum x / cols,  rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps),
 *     h = (x - mean) rstd,  y = h w + b.
 * And from the loss's derivative dy by y, with g = dy w:
 *     dx = rstd (g - sum g / cols - h sum (g h) / cols),
 *     dw = sum over rows of dy h,  db = sum over rows of dy.
 *
 * Sums are float, or double for rows of more than HIP_LAYERNORM_ROW; the mean is kept
 * with what its rounding to float left over, so that a row far off zero keeps its
 * differences, and the squared differences may be larger or smaller than a float holds.
 * An infinity or NaN in a row of x, or a sum of the row or a difference past a float's range,
 * makes that row of y and dx NaN, and dw.  A row without differences has h 0 if eps > 0.
 * rstd is a float: infinite, with y and dx, where eps is 0 and the root of the squared
 * differences' mean below 2^-128.
 *
 * Status codes: 0 enqueued; -i the i-th argument is invalid; > 0 the
 * hipError_t of a failed launch.  hip_layernorm_*_status_string name them.
 */
#ifndef LIBSGEMM_LAYERNORM_H
#define LIBSGEMM_LAYERNORM_H

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
#define HIP_LAYERNORM_F32 0
#define HIP_LAYERNORM_BF16 1
#define HIP_LAYERNORM_F16 2

#define HIP_LAYERNORM_ROW 16384
/* the backward pass of at most so many rows of at most HIP_LAYERNORM_ROW needs no workspace */
#define HIP_LAYERNORM_FEW 256

/*
 * Y <- the layer norm of X's rows.
 *   X, Y: rows x cols of `type`, row strides ldx, ldy; element alignment suffices.  Y
 *   may be X itself (same stride) and must not overlap it otherwise.
 *   w, b: cols numbers of w_type (`type`, or HIP_LAYERNORM_F32) side by side; either
 *   may be NULL (1 and 0).
 *   eps: at least 0.  stats: NULL, or 3 * rows floats that the backward pass takes:
 *   the means, what their rounding left over, and rstd.
 *   rows == 0 or cols == 0: nothing is done.
 *
 * Arguments are numbered from 1: rows, cols, type, X, ldx, w, b, w_type, eps, Y, ldy,
 * stats, stream.
 */
int hip_layernorm_forward(int rows, int cols, int type, const void *X, int ldx, const void *w, const void *b,
                          int w_type, float eps, void *Y, int ldy, float *stats, hipStream_t stream);

/*
 * Bytes of workspace that hip_layernorm_backward needs (host only, launches
 * nothing).  0, or -1, -2 for bad rows or cols.
 */
int hip_layernorm_backward_workspace(int rows, int cols, long long *bytes);

/*
 * DX <- the gradient by X; dw and db <- (accumulate 0) or += (1) the gradients by w
 * and b, in an order of summation that depends on the sizes alone.
 *   DY, X, DX: rows x cols of `type`, row strides lddy, ldx, lddx.  DX may be DY or X
 *   itself (same stride), and must not overlap them otherwise; NULL: not wanted.
 *   stats: hip_layernorm_forward's.  w: as there (NULL: 1).
 *   dw, db: cols floats; either may be NULL (not wanted).  They must not overlap each
 *   other, nor anything else that is read or written.
 *   workspace: device memory of at least the bytes above, 16-byte aligned; calls
 *   that overlap in time need workspaces of their own.
 *   rows == 0: dw and db <- 0 without accumulate.  cols == 0: nothing is done.
 *
 * Arguments are numbered from 1: rows, cols, type, DY, lddy, X, ldx, stats, w, w_type,
 * DX, lddx, dw, db, accumulate, workspace, workspace_bytes, stream.
 */
int hip_layernorm_backward(int rows, int cols, int type, const void *DY, int lddy, const void *X, int ldx,
                           const float *stats, const void *w, int w_type, void *DX, int lddx, float *dw, float *db,
                           int accumulate, void *workspace, long long workspace_bytes, hipStream_t stream);

const char *hip_layernorm_forward_status_string(int status);
const char *hip_layernorm_backward_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* LIBSGEMM_LAYERNORM_H */

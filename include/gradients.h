/*
 * gradients.h -- the global norm of many gradients, and clipping by it, on the AMD
 * Instinct MI355X (gfx950).  Part of libsgemm; the conventions of sgemm.h hold
 * (device pointers, work enqueued on `stream` without synchronising, argument
 * errors found on the host before anything is enqueued, no state kept between
 * calls).
 *
 *     norm = sqrt(sum over all tensors and elements of x^2)
 *     y = x * c,  c = 1 if norm + eps <= max_norm, else max_norm / (norm + eps)
 *
 * Squares are summed in double, in an order that depends on the sizes alone, and c
 * is worked out in double; it is rounded to float, the product x c to float and then to
 * y's type.
 * A NaN anywhere makes the norm and every y NaN (also for an infinite max_norm); an
 * infinity makes the norm infinite and, unless max_norm is infinite too, c 0: what is
 * finite becomes 0, what is not NaN.  The norm that is written is rounded to float (an
 * infinity past its range, which c does not see).
 *
 * Status codes: 0 enqueued; -i the i-th argument is invalid; > 0 the
 * hipError_t of a failed launch.  hip_gradient_*_status_string name them.
 */
#ifndef LIBSGEMM_GRADIENTS_H
#define LIBSGEMM_GRADIENTS_H

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define HIP_GRADIENT_F32 0
#define HIP_GRADIENT_BF16 1
#define HIP_GRADIENT_F16 2

#define HIP_GRADIENT_MAX_COUNT (1 << 20) /* tensors of a call */

/*
 * One tensor: rows x cols elements of `type` at x, row stride ldx, and where the
 * clipped ones go, y with row stride ldy (strides are not read where rows is 1);
 * element alignment suffices.  Dense tensors of any shape are one row.  y may be x
 * itself (same stride).
 */
typedef struct {
  const void *x;
  void *y;
  long long rows, cols, ldx, ldy;
  long long type;
} hip_gradient;

/*
 * Bytes of workspace that the functions below need for `count` tensors (host only,
 * launches nothing).  0, or -1 for a bad count.
 */
int hip_gradient_workspace(int count, long long *bytes);

/*
 * norm <- the norm of `count` tensors; y, ldy are not read.  A tensor that is given
 * twice counts twice.
 *   tensors: HOST array, read before the call returns.
 *   norm: one float on the device.
 *   workspace: device memory of at least the bytes above, 256-byte aligned; calls
 *   that overlap in time need workspaces of their own.
 *
 * Arguments are numbered from 1: count, tensors, norm, workspace, workspace_bytes,
 * stream.
 */
int hip_gradient_norm(int count, const hip_gradient *tensors, float *norm, void *workspace, long long workspace_bytes,
                      hipStream_t stream);

/*
 * norm <- the norm, and y <- c x for each tensor.  Where c is 1 a tensor whose y is x
 * is not written.  What a call writes must not overlap anything else it reads or
 * writes: the call is refused where the tensors' memory says it does.
 *   max_norm: at least 0 (an infinity: no limit).  eps: at least 0.
 *   norm: one float on the device, may be NULL.
 *
 * Arguments are numbered from 1: count, tensors, max_norm, eps, norm, workspace,
 * workspace_bytes, stream.
 */
int hip_gradient_clip(int count, const hip_gradient *tensors, double max_norm, double eps, float *norm, void *workspace,
                      long long workspace_bytes, hipStream_t stream);

/*
 * The same by a norm that is there, one float on the device: what hip_gradient_norm
 * gave, or the root of several ranks' summed squares.
 *
 * Arguments are numbered from 1: count, tensors, max_norm, eps, norm, workspace,
 * workspace_bytes, stream.
 */
int hip_gradient_clip_by(int count, const hip_gradient *tensors, double max_norm, double eps, const float *norm,
                         void *workspace, long long workspace_bytes, hipStream_t stream);

const char *hip_gradient_norm_status_string(int status);
const char *hip_gradient_clip_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* LIBSGEMM_GRADIENTS_H */

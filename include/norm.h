/*
 * Root-mean-square norm of rows with the residual's addition: its output in the
 * input's type, or in 8-bit integers with a scale a row (the left operand of
 * i8gemm), and its gradients. In the same library as sgemm.h.
 *
 *   h[m,k] = X[m,k] + R[m,k]              (in fp32, rounded once to the type)
 *   t[m,k] = h[m,k] * weight[k]           (in fp32, one rounding)
 *   rstd[m] = 1 / sqrt(mean_k h[m,k]^2 + eps)             (in fp32)
 *
 * Matrices are row-major with element strides (leading dimensions) and hold one
 * type a call (an sgemm_type: F32, F16 or BF16); weight is K floats. All
 * pointers are DEVICE pointers owned by the caller and need no alignment beyond
 * their elements'. Calls are asynchronous on `stream`, never synchronise the
 * host, allocate nothing, use no atomics and are deterministic. They launch on
 * the current device, which has to be the stream's. Outputs must not overlap
 * inputs, but where it says that one may be an input itself: the same address
 * and leading dimension.
 *
 * The squares are added in fp32 before they are divided by K. A sum beyond its
 * range (a root mean square of 2^64 / sqrt(K) and more) makes rstd 0, and an
 * infinity in h does: its own element of Y is NaN then, the row's others are 0. A
 * NaN in h makes the row NaN. With eps 0, a sum that is 0 (a row of zeros, or of
 * nothing but elements below 2^-75) makes rstd infinite: Y is NaN where h is 0
 * and infinite elsewhere, the scale of rms_norm_i8 is infinite, and rms_norm_grad
 * gives no finite number in that row of dX nor in dweight. (With rstd 0 and a
 * finite row its dX is dH.)
 *
 * Status codes: 0 success, a positive hipError_t, or minus (a base for the
 * call + the position of the first invalid argument): 1000 for rms_norm, 1100
 * for rms_norm_i8, 1200 for rms_norm_grad. Nothing is launched on error.
 * sgemm_status_string() gives the message.
 */
#ifndef PRECISION_GEMM_AMD_NORM_H
#define PRECISION_GEMM_AMD_NORM_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Longest row rms_norm_grad takes. */
#define RMS_NORM_GRAD_MAX_K 16384

/*
 * Y[m,k] = t[m,k] * rstd[m], rounded once more. R may be NULL (none); H may be
 * NULL (h is not kept), X or R.
 * Positions: M 1, K 2, X 3, type 4, ldx 5 (>= max(1, K), as every leading
 * dimension of a matrix that is there), R 6, ldr 7, weight 8, eps 9 (>= 0), H
 * 10, ldh 11, Y 12, ldy 13.
 */
int rms_norm(int M, int K, const void *X, int type, int ldx, const void *R, int ldr,
             const float *weight, float eps, void *H, int ldh, void *Y, int ldy,
             sgemm_stream_t stream);

/*
 * The same in 8-bit integers, as i8_quantize_rows makes them of t:
 *   s[m] = max(max_k |t[m,k]| / 127, 2^-126)             (fp32 division)
 *   Q[m,k] = the integer nearest to t[m,k] / s[m], ties to even
 *   scale[m] = s[m] * rstd[m]
 * so Q[m,k] * scale[m] is the norm's output. The quotient is that of the real
 * numbers and rstd is no part of it: Q does not depend on how the sum of
 * squares, the root or a division rounds. A row of t with an infinity or NaN has
 * Q = 0 and scale NaN. K == 0: scale[m] = 2^-126.
 * Positions: as rms_norm up to ldh 11; Q 12, ldq 13, scale 14.
 */
int rms_norm_i8(int M, int K, const void *X, int type, int ldx, const void *R, int ldr,
                const float *weight, float eps, void *H, int ldh, signed char *Q, int ldq,
                float *scale, sgemm_stream_t stream);

/*
 * The gradients of rms_norm, given those of Y and (or NULL: none) of H, which
 * went on beside it:
 *   dX[m,k] = dH[m,k] + rstd[m] * (weight[k] dY[m,k]
 *             - h[m,k] rstd[m]^2 mean_j(weight[j] dY[m,j] h[m,j]))
 *   dweight[k] = sum_m dY[m,k] h[m,k] rstd[m]           (fp32)
 * dX, in fp32 and rounded once, is the gradient of X and of R alike; it may be
 * dY or dH. dweight may be NULL. workspace: at least
 * rms_norm_grad_workspace_size() bytes, 16-byte aligned, in use until the work
 * completes on `stream`: calls that overlap (two streams, two captured graphs)
 * need one each. M == 0 sets dweight to 0.
 * Positions: M 1, K 2 (at most RMS_NORM_GRAD_MAX_K), dY 3, type 4, lddy 5, H 6,
 * ldh 7, weight 8, eps 9, dH 10, lddh 11, dX 12, lddx 13, dweight 14, workspace
 * 15, workspace_bytes 16.
 */
int rms_norm_grad(int M, int K, const void *dY, int type, int lddy, const void *H, int ldh,
                  const float *weight, float eps, const void *dH, int lddh, void *dX, int lddx,
                  float *dweight, void *workspace, size_t workspace_bytes, sgemm_stream_t stream);

/* Bytes of workspace of rms_norm_grad with a dweight; without one it needs none.
   (0 for invalid arguments too.) */
size_t rms_norm_grad_workspace_size(int M, int K, int type);

#ifdef __cplusplus
}
#endif

#endif /* PRECISION_GEMM_AMD_NORM_H */

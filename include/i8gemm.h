/*
 * 8-bit integer products with a scale for each row of A (token) and each row
 * of B (channel), next to the fp32 products of sgemm.h and in the same
 * library: the row quantization that makes A, the product, and the product
 * over rows sorted by expert.
 *
 * Storage is row-major with element strides. A holds one token a row, B one
 * output channel a row (the layout weights are kept in), so both are
 * contiguous in k:
 *   acc[m,n] = sum_k A[m*lda + k] * B[n*ldb + k]            (exact, 32-bit integers)
 *   C[m*ldc + n] = (float(acc) * scaleA[m]) * scaleB[n] + bias[n]
 * in fp32 (the last product and sum with one rounding), rounded once to C's
 * type. The integer sum is exact for every order
 * of its terms, so results do not depend on how a kernel splits K.
 *
 * Ownership, execution (asynchronous on `stream`, no host synchronisation, no
 * allocation, deterministic) and thread safety are those of sgemm.h. The calls
 * launch on the current device, which has to be the stream's. Outputs must not
 * overlap inputs.
 *
 * Alignment: none is required beyond the element types' own. Rows that start on
 * 16-byte boundaries (A and B 16-byte aligned, lda, ldb and strideB multiples of
 * 16) with K a multiple of 16 and lda and ldb below 2^22 run the fast kernels.
 *
 * Status codes: 0 success, a positive hipError_t, or minus (a base for the
 * call + the position of the first invalid argument): 100 for
 * i8_quantize_rows, 200 for i8gemm, 300 for i8gemm_grouped; e.g. -205 is a bad
 * lda of i8gemm; -22 for a product of more output tiles than a launch (2^32 - 1
 * work-items) holds, whichever kernel runs.
 * Nothing is launched on error. sgemm_status_string() gives the message.
 */
#ifndef PRECISION_GEMM_AMD_I8GEMM_H
#define PRECISION_GEMM_AMD_I8GEMM_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest K: the sum of K products of at most 2^14 each stays below 2^31. */
#define I8GEMM_MAX_K 131071

/*
 * Rows to 8-bit integers, one scale a row:
 *   scale[m] = max(max_k |X[m*ldx + k]| / 127, 2^-126)      (fp32 division)
 *   Q[m*ldq + k] = the integer nearest to X[m*ldx + k] / scale[m], ties to even
 * The quotient is that of the real numbers: Q never depends on how a division
 * rounds. Values lie in [-127, 127]; a row of zeros has scale 2^-126. A row
 * holding an infinity or NaN has scale infinity or NaN and Q = 0, so products
 * with it are NaN. K == 0: scale[m] = 2^-126.
 * Positions: M 1, K 2, X 3, x_type 4 (an sgemm_type: F32, F16 or BF16), ldx 5
 * (>= max(1, K)), Q 6, ldq 7 (>= max(1, K)), scale 8.
 */
int i8_quantize_rows(int M, int K, const void *X, int x_type, int ldx, signed char *Q, int ldq,
                     float *scale, sgemm_stream_t stream);

/*
 * C = (A B^T) * scaleA[m] * scaleB[n] + bias[n]: A is M x K, B is N x K, C is
 * M x N of type c_type (F32, F16 or BF16); scaleA has M entries, scaleB N, and
 * bias N or is NULL (none). K == 0 gives C = bias (or 0); A and B are not read
 * then. M == 0 or N == 0: nothing is launched.
 * Positions: M 1, N 2, K 3 (at most I8GEMM_MAX_K), A 4, lda 5 (>= max(1, K)),
 * scaleA 6, B 7, ldb 8, scaleB 9, C 11, c_type 12, ldc 13 (>= max(1, N)).
 */
int i8gemm(int M, int N, int K, const signed char *A, int lda, const float *scaleA,
           const signed char *B, int ldb, const float *scaleB, const float *bias, void *C,
           int c_type, int ldc, sgemm_stream_t stream);

/*
 * The same with rows sorted by group (expert): rows offsets[g] <= m <
 * offsets[g+1] of A and C use B + g*strideB, scaleB + g*N and bias + g*N.
 * offsets is a DEVICE array of groups + 1 nondecreasing ints within [0, M]
 * (expert_sort writes one); the host never reads it. Groups may be empty. Rows
 * of C before offsets[0] and from offsets[groups] on are left as they were.
 * Values outside [0, M] are brought into that range, and a group whose end
 * lies before its start is empty; rows that decreasing values put into two
 * groups get either's values or stay as they were.
 * Positions: M 1 (rows of A and C), N 2, K 3, groups 4, offsets 5, A 6, lda 7,
 * scaleA 8, B 9, ldb 10, strideB 11 (>= 0; 0 shares one B), scaleB 12, C 14,
 * c_type 15, ldc 16. groups == 0: nothing is launched.
 * At most 65536 groups; every workgroup reads all offsets.
 */
int i8gemm_grouped(int M, int N, int K, int groups, const int *offsets, const signed char *A,
                   int lda, const float *scaleA, const signed char *B, int ldb, long long strideB,
                   const float *scaleB, const float *bias, void *C, int c_type, int ldc,
                   sgemm_stream_t stream);

/*
 * Kernels the two calls choose among (see i8gemm_select_kernel): the tile of C
 * one workgroup owns. Results do not depend on the kernel.
 */
enum i8gemm_kernel {
    /* B streams from memory into registers, K split over the waves */
    I8GEMM_KERNEL_S16x16 = 0,     /* 8 waves */
    I8GEMM_KERNEL_S16x16_W16 = 1, /* 16 waves */
    I8GEMM_KERNEL_S16x32 = 2,     /* 4 waves */
    I8GEMM_KERNEL_S32x16 = 3,     /* 8 waves */
    I8GEMM_KERNEL_S32x32 = 4,     /* 8 waves */
    I8GEMM_KERNEL_S32x64 = 5,     /* 4 waves */
    /* K-steps through registers to LDS: rows of any alignment */
    I8GEMM_KERNEL_T64x64 = 6,
    I8GEMM_KERNEL_T128x128 = 7,
    /* K-steps straight into LDS: the fast kernels (see Alignment above) */
    I8GEMM_KERNEL_L32x64 = 8,
    I8GEMM_KERNEL_L64x64_R4 = 9,  /* four stages of LDS instead of three */
    I8GEMM_KERNEL_L64x64 = 10,
    I8GEMM_KERNEL_L64x128 = 11,
    I8GEMM_KERNEL_L128x128 = 12,
    I8GEMM_KERNEL_L128x256 = 13,
    I8GEMM_KERNEL_L256x256 = 14,
    I8GEMM_KERNEL_COUNT = 15
};

/*
 * Host-side dispatch decision, exposed for tests and tuning (no device call):
 * the kernel that i8gemm (groups == 0) or i8gemm_grouped launches for this
 * shape, given whether rows start on 16-byte boundaries (`aligned`; leading
 * dimensions are taken to be below 2^22) and the device's compute-unit count.
 * Returns an i8gemm_kernel, -22 for more output tiles than a launch of any
 * kernel that takes the call holds, or a negative status for invalid sizes.
 */
int i8gemm_select_kernel(int M, int N, int K, int groups, int aligned, int num_cus);

#ifdef __cplusplus
}
#endif

#endif /* PRECISION_GEMM_AMD_I8GEMM_H */

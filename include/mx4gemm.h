/*
 * Microscaled 4-bit floating point: rows to 4 bits and back, and products of
 * such rows, next to the 8-bit ones of i8gemm.h and in the same library.
 *
 * A row's elements are taken 32 at a time; a block of 32 shares one scale, a
 * power of two, and an element is one of
 *   0, 0.5, 1, 1.5, 2, 3, 4, 6 (codes 0 to 7), or their negatives (8 to 15)
 * times that (E2M1 elements and E8M0 scales, as the microscaling formats of the
 * Open Compute Project define them). Layout:
 *   elements: row m at Q + m*ldq, ldq in BYTES; element k is the low (k even) or
 *     high (k odd) half of byte k/2. A row takes (K + 1)/2 bytes; the high half
 *     of an odd row's last byte is written as 0 and never taken into account.
 *   scales: four neighbouring blocks' bytes stand together, then the rows, then
 *     the next four blocks: block b of row m has the byte
 *       scale[((b/4) * lds + m) * 4 + b%4],  lds >= rows,
 *     and stands for 2^(byte - 127), or NaN for 255. Bytes of blocks from
 *     (K + 31)/32 on are written as 0 and never taken into account. The array
 *     is 4-byte aligned and holds (((K + 127)/128 - 1) * lds + rows) * 4 bytes.
 *     (Rows that run through a matrix tile have their scales side by side; a
 *     row-major array [rows, K/32] is brought into this order by a transpose of
 *     its groups of four.)
 *
 * Ownership, execution (asynchronous on `stream`, no host synchronisation, no
 * allocation, deterministic) and thread safety are those of sgemm.h. The calls
 * launch on the current device, which has to be the stream's. Outputs must not
 * overlap inputs.
 *
 * Alignment: none is required beyond the scales'. Rows that start on 16-byte
 * boundaries (A and B 16-byte aligned, lda, ldb and strideB multiples of 16)
 * with K a multiple of 32 and lda and ldb below 2^22 run the fast kernels.
 *
 * Status codes: 0 success, a positive hipError_t, or minus (a base for the
 * call + the position of the first invalid argument): 1300 for
 * mx4_quantize_rows, 1400 for mx4_dequantize_rows, 1500 for mx4gemm, 1600 for
 * mx4gemm_grouped; -22 for a product of more output tiles than a launch (2^32 -
 * 1 work-items) holds. Nothing is launched on error. sgemm_status_string()
 * gives the message.
 */
#ifndef PRECISION_GEMM_AMD_MX4GEMM_H
#define PRECISION_GEMM_AMD_MX4GEMM_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Rows to 4 bits. For each block, e = max(floor(log2(max |x|)) - 2, -127), or
 * -127 for a block of zeros; the scale is 2^e, and an element the value nearest
 * to x / 2^e (ties to the even code, beyond 6: 6), with x's sign. A block
 * holding an infinity or NaN has the scale NaN and elements 0. Every step is
 * exact but the one rounding.
 * Positions: M 1, K 2, X 3, x_type 4 (an sgemm_type: F32, F16 or BF16), ldx 5
 * (>= max(1, K)), Q 6, ldq 7 (bytes, >= max(1, (K + 1)/2)), scale 8, lds 9
 * (>= max(1, M)).
 */
int mx4_quantize_rows(int M, int K, const void *X, int x_type, int ldx, unsigned char *Q, int ldq,
                      unsigned char *scale, int lds, sgemm_stream_t stream);

/*
 * And back: Y[m,k] = element * scale, rounded once to Y's type: exact in F32 and
 * BF16, but infinite beyond the type's range (of F32 and BF16: elements of 4 and
 * more with the byte 253, of 2 and more with 254, which the rounding never writes).
 * Positions: M 1, K 2, Q 3, ldq 4, scale 5, lds 6, Y 7, y_type 8, ldy 9.
 */
int mx4_dequantize_rows(int M, int K, const unsigned char *Q, int ldq, const unsigned char *scale,
                        int lds, void *Y, int y_type, int ldy, sgemm_stream_t stream);

/*
 * C[m,n] = sum_k a[m,k] b[n,k] + bias[n]: A has M rows of K elements, B N rows
 * (one output channel each), C is M x N of type c_type (F32, F16 or BF16); bias
 * is N floats or NULL (none). Sums run in fp32 in the matrix units, which add
 * the products of up to 128 k at a time to a sum at once, dropping what lies
 * below 2^-22 of the largest of them; the result is rounded once to C's type. A
 * block with the scale NaN makes its whole row (of B: column) of C NaN. K == 0
 * gives C = bias (or 0); A, B and the scales are not read then. M == 0 or N ==
 * 0: nothing is launched.
 * Positions: M 1, N 2, K 3, A 4, lda 5 (bytes, >= max(1, (K + 1)/2)), scaleA 6,
 * ldsa 7 (>= M), B 8, ldb 9, scaleB 10, ldsb 11 (>= N), C 13, c_type 14, ldc 15
 * (>= max(1, N)).
 */
int mx4gemm(int M, int N, int K, const unsigned char *A, int lda, const unsigned char *scaleA,
            int ldsa, const unsigned char *B, int ldb, const unsigned char *scaleB, int ldsb,
            const float *bias, void *C, int c_type, int ldc, sgemm_stream_t stream);

/*
 * The same with rows sorted by group (expert): rows offsets[g] <= m <
 * offsets[g+1] of A and C use B + g*strideB, scaleB + g*strideSB (both in
 * bytes) and bias + g*N. offsets is a DEVICE array of groups + 1 nondecreasing
 * ints within [0, M] (expert_sort writes one); the host never reads it. Groups
 * may be empty. Rows of C before offsets[0] and from offsets[groups] on are left
 * as they were. Values outside [0, M] are brought into that range, and a group
 * whose end lies before its start is empty; rows that decreasing values put
 * into two groups get either's values or stay as they were.
 * Positions: M 1 (rows of A and C), N 2, K 3, groups 4 (at most 65536), offsets
 * 5, A 6, lda 7, scaleA 8, ldsa 9, B 10, ldb 11, strideB 12 (>= 0; 0 shares one
 * B), scaleB 13, ldsb 14, strideSB 15 (>= 0, a multiple of 4), C 17, c_type 18,
 * ldc 19. groups == 0: nothing is launched. Every workgroup reads all offsets.
 */
int mx4gemm_grouped(int M, int N, int K, int groups, const int *offsets, const unsigned char *A,
                    int lda, const unsigned char *scaleA, int ldsa, const unsigned char *B, int ldb,
                    long long strideB, const unsigned char *scaleB, int ldsb, long long strideSB,
                    const float *bias, void *C, int c_type, int ldc, sgemm_stream_t stream);

/*
 * Kernels the two calls choose among (see mx4gemm_select_kernel): the tile of C
 * one workgroup owns. The order of a sum, and with it its last bits, depends on
 * the kernel.
 */
enum mx4gemm_kernel {
    /* B streams from memory into registers, K split over the waves */
    MX4GEMM_KERNEL_S16x16 = 0, /* 8 waves */
    MX4GEMM_KERNEL_S16x32 = 1, /* 4 waves */
    MX4GEMM_KERNEL_S32x16 = 2, /* 8 waves */
    MX4GEMM_KERNEL_S32x32 = 3, /* 8 waves */
    MX4GEMM_KERNEL_S32x64 = 4, /* 4 waves */
    /* K-steps through registers to LDS: rows of any alignment */
    MX4GEMM_KERNEL_T64x64 = 5,
    MX4GEMM_KERNEL_T128x128 = 6,
    /* K-steps straight into LDS: the fast kernels (see Alignment above) */
    MX4GEMM_KERNEL_L64x64 = 7,
    MX4GEMM_KERNEL_L64x128 = 8,
    MX4GEMM_KERNEL_L128x128 = 9,
    MX4GEMM_KERNEL_L128x128_R2 = 10, /* two stages of LDS instead of four */
    MX4GEMM_KERNEL_L128x256 = 11,
    MX4GEMM_KERNEL_L256x256 = 12,
    MX4GEMM_KERNEL_COUNT = 13
};

/*
 * Host-side dispatch decision, exposed for tests and tuning (no device call):
 * the kernel that mx4gemm (groups == 0) or mx4gemm_grouped launches for this
 * shape, given whether rows start on 16-byte boundaries (`aligned`; leading
 * dimensions are taken to be below 2^22) and the device's compute-unit count.
 * Returns an mx4gemm_kernel, -22 for more output tiles than a launch of any
 * kernel that takes the call holds, or a negative status for invalid sizes.
 */
int mx4gemm_select_kernel(int M, int N, int K, int groups, int aligned, int num_cus);

#ifdef __cplusplus
}
#endif

#endif /* PRECISION_GEMM_AMD_MX4GEMM_H */

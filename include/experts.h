/*
 * Tokens sorted by expert and back, with the gradients: what stands before and
 * after the grouped products (i8gemm_grouped, sgemm_grouped) of a layer whose
 * router sends every token to `topk` of `experts` experts.
 *
 * Token t's slot j (of topk) goes to expert ids[t*topk + j]. An id outside
 * [0, experts) is a slot without an expert (a padding token, an expert held
 * elsewhere): it takes part in nothing. The sorted rows are ordered by expert
 * and, within one, by slot t*topk + j:
 *   offsets[e] = number of slots with an expert below e   (experts + 1 ints)
 *   row_of_slot[t*topk + j] = the slot's sorted row, or -1
 *
 * Matrices are row-major with element strides (leading dimensions) and hold
 * one type a call (an sgemm_type); sorted matrices have tokens*topk rows, of
 * which the last ones, from offsets[experts] on, belong to no slot: what they
 * hold is not used, and they are not written. All pointers are DEVICE pointers
 * owned by the caller. Calls are asynchronous on `stream`, never synchronise the
 * host, allocate nothing, use no floating-point atomics and are deterministic.
 * They launch on the current device, which has to be the stream's. Outputs must not
 * overlap inputs. Matrices need no alignment beyond their elements'. Entries of
 * row_of_slot outside [0, tokens*topk) count as -1; the others have to differ
 * from each other, as expert_sort makes them, where rows are written
 * (expert_gather, expert_combine_grad).
 *
 * tokens*topk is at most 2^31 - 1. Status codes: 0 success, a positive
 * hipError_t, or minus (a base for the call + the position of the first
 * invalid argument): 400 for expert_sort, 500 for expert_gather, 600 for
 * expert_combine, 700 for expert_combine_grad, 1700 for expert_layer; -22 for more
 * rows than a launch holds (over 2^23 tokens with rows of more than 2048 bytes,
 * twice as many for each halving of that; expert_layer: where F, or H / 2, times the
 * experts that the slots can name and a 16th of the other slots passes some 2^30,
 * with weights off its fast path). Nothing is launched on error.
 * sgemm_status_string() gives the message.
 */
#ifndef PRECISION_GEMM_AMD_EXPERTS_H
#define PRECISION_GEMM_AMD_EXPERTS_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of experts expert_sort takes. */
#define EXPERT_SORT_MAX_EXPERTS 1024

/*
 * offsets and row_of_slot of the ids (id_bytes 4: int32, 8: int64; contiguous).
 * workspace: at least expert_sort_workspace_size() bytes, 4-byte aligned, in
 * use until the work completes on `stream`: calls that overlap (two streams,
 * two captured graphs) need one each.
 * Positions: tokens 1, topk 2 (>= 1), experts 3 (1 to
 * EXPERT_SORT_MAX_EXPERTS), ids 4, id_bytes 5, offsets 6, row_of_slot 7,
 * workspace 8, workspace_bytes 9. tokens == 0 writes offsets only.
 */
int expert_sort(int tokens, int topk, int experts, const void *ids, int id_bytes, int *offsets,
                int *row_of_slot, void *workspace, size_t workspace_bytes, sgemm_stream_t stream);

/* Bytes of workspace of expert_sort (0: none; 0 for invalid arguments too). */
size_t expert_sort_workspace_size(int tokens, int topk, int experts);

/*
 * Y[row_of_slot[t*topk + j], :] = X[t, :] for every slot with an expert: X is
 * tokens x cols, Y tokens*topk x cols. Any type, 8-bit integers among them
 * (the rows of i8_quantize_rows; their scales are a matrix of cols = 1).
 * Its gradient is expert_combine without weights.
 * Positions: tokens 1, topk 2, cols 3, X 4, type 5 (F32, F16, BF16 or I8), ldx
 * 6, row_of_slot 7, Y 8, ldy 9.
 */
int expert_gather(int tokens, int topk, int cols, const void *X, int type, int ldx,
                  const int *row_of_slot, void *Y, int ldy, sgemm_stream_t stream);

/*
 * out[t, :] = sum_j weights[t*topk + j] * Y[row_of_slot[t*topk + j], :], over
 * the slots with an expert, in fp32 in the order of j, rounded once; 0 for a
 * token that has none. weights: tokens*topk floats, or NULL for 1 everywhere
 * (the gradient of expert_gather).
 * Positions: tokens 1, topk 2, cols 3, Y 4, type 5 (F32, F16 or BF16), ldy 6,
 * row_of_slot 7, weights 8, out 9, ldo 10.
 */
int expert_combine(int tokens, int topk, int cols, const void *Y, int type, int ldy,
                   const int *row_of_slot, const float *weights, void *out, int ldo,
                   sgemm_stream_t stream);

/*
 * The gradient of expert_combine: for every slot with an expert, r its row,
 *   dY[r, :] = weights[t*topk + j] * dout[t, :]          (rounded once)
 *   dweights[t*topk + j] = sum_h dout[t, h] * Y[r, h]    (in fp32)
 * and dweights = 0 for a slot without. dweights may be NULL (Y is not read
 * then and may be NULL too); weights may be NULL, as above.
 * Positions: tokens 1, topk 2, cols 3, dout 4, type 5, ldo 6, Y 7, ldy 8,
 * row_of_slot 9, weights 10, dY 11, lddy 12, dweights 13.
 */
int expert_combine_grad(int tokens, int topk, int cols, const void *dout, int type, int ldo,
                        const void *Y, int ldy, const int *row_of_slot, const float *weights,
                        void *dY, int lddy, float *dweights, sgemm_stream_t stream);

/* Most slots (tokens * topk) and experts expert_layer takes. */
#define EXPERT_LAYER_MAX_SLOTS 2048
#define EXPERT_LAYER_MAX_EXPERTS 1024

/*
 * A whole layer of experts for a few tokens, without a sort, sorted copies or a
 * launch for each step: with e = ids[t*topk + j],
 *   g = W1_e[0:F] X[t],  u = W1_e[F:2F] X[t],  a = silu(g) * u  (silu(x) = x / (1 + exp(-x)))
 *   out[t] = sum_j weights[t*topk + j] * (W2_e a)
 * W1_e is 2F x H (first the rows of the gate, then those it multiplies) and W2_e
 * H x F, both with the products' sums along a row: W1 + e*strideW1 with rows ldw1
 * apart, W2 + e*strideW2 with rows ldw2 apart. X and out are tokens x H of `type`
 * (F32, F16 or BF16). w_type is the weights':
 *   - `type` itself; scale1 and scale2 are not used and may be NULL;
 *   - SGEMM_I8, one fp32 scale a row: scale1[e*2F + i], scale2[e*H + i];
 *   - SGEMM_MX4, 4-bit blocks as mx4gemm.h lays them out: leading dimensions and
 *     strides are BYTES, and expert e's scales stand at scale1 + e*((H + 127)/128
 *     * 2F * 4) with 2F rows, scale2 + e*((F + 127)/128 * H * 4) with H rows.
 * Slots whose id is outside [0, experts) take part in nothing; a token without
 * any gets 0. A token may name an expert twice. weights may be NULL (1
 * everywhere).
 * Sums run in fp32, and so are tokens and a held and multiplied, in all their bits
 * (24 of F32 tokens and of a, with narrower weights down to 2^-133); out is rounded
 * once, after the sum over j in its order. An infinity among the weights or the
 * values of a may give NaN where it would give an infinity; a 4-bit weight of 2^128
 * or more (scale bytes 253 and 254, which mx4_quantize_rows never writes) counts as
 * one, and a block with the scale NaN makes what it is part of NaN.
 * Only the experts that the tokens name are read, each once for up to 16 of its
 * slots; beyond that the sorted path of expert_sort to expert_combine is the
 * faster one. Rows on 16-byte boundaries that hold a multiple of 16 bytes (MX4:
 * of 32 elements) run the fast kernels.
 * workspace: at least expert_layer_workspace_size() bytes, 16-byte aligned, in
 * use until the work completes on `stream`: calls that overlap (two streams, two
 * captured graphs) need one each. Its contents need no preparation.
 * Positions: tokens 1 (tokens*topk at most EXPERT_LAYER_MAX_SLOTS), topk 2 (>=
 * 1), experts 3 (1 to EXPERT_LAYER_MAX_EXPERTS), H 4, F 5 (each at most 2^20), X 6, type 7, ldx 8,
 * ids 9, id_bytes 10 (4: int32, 8: int64; contiguous), W1 12, w_type 13, ldw1 14,
 * strideW1 15 (>= 0), scale1 16, W2 17, ldw2 18, strideW2 19, scale2 20, out 21,
 * ldo 22, workspace 23, workspace_bytes 24. tokens == 0 or H == 0: nothing is
 * launched; F == 0 sets out to 0.
 */
int expert_layer(int tokens, int topk, int experts, int H, int F, const void *X, int type, int ldx,
                 const void *ids, int id_bytes, const float *weights, const void *W1, int w_type,
                 int ldw1, long long strideW1, const void *scale1, const void *W2, int ldw2,
                 long long strideW2, const void *scale2, void *out, int ldo, void *workspace,
                 size_t workspace_bytes, sgemm_stream_t stream);

/* Bytes of workspace of expert_layer (0 for invalid arguments). */
size_t expert_layer_workspace_size(int tokens, int topk, int H, int F, int type);

#ifdef __cplusplus
}
#endif

#endif /* PRECISION_GEMM_AMD_EXPERTS_H */

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
 * expert_combine, 700 for expert_combine_grad; -22 for more rows than a launch
 * holds (over 2^23 tokens with rows of more than 2048 bytes, twice as many for
 * each halving of that). Nothing is launched on error. sgemm_status_string()
 * gives the message.
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

#ifdef __cplusplus
}
#endif

#endif /* PRECISION_GEMM_AMD_EXPERTS_H */

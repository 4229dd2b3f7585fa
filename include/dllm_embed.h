/*
 * dllm_embed.h -- C ABI of the token embedding of a masked diffusion LLM on
 * AMD Instinct MI355X (gfx950), with its gradient.
 *
 *   out[t] = scale * table[tokens[t]]
 *   d_table[v] = scale * sum of d_out[t] over the t with tokens[t] = v
 * bf16 in and out, products and sums in fp32, rounded once.  A token outside
 * 0 .. V - 1 has no row: its output is zero and it adds to no gradient.
 *
 * In a masked diffusion model one token, the mask, may be most of a batch:
 * the gradient sorts the tokens and splits long runs, so no token's share is
 * one workgroup's, and no sum depends on the order in which workgroups end.
 *
 * Memory: every pointer is a DEVICE pointer; bf16 is passed as uint16_t bit
 * patterns; arrays are row-major, contiguous and, tokens apart, 16-byte
 * aligned.  The caller owns everything; nothing is allocated.  Work is queued
 * on `stream` (a hipStream_t, NULL = the default stream), whose device must be
 * the current one, and the calls return without waiting.  Argument errors
 * return before anything is queued.  Calls queue kernels only and may be
 * captured in HIP graphs; two calls that may overlap in time need a workspace
 * each.  Results do not change from run to run.  The status codes are those
 * of dllm_readout.h.
 */
#ifndef DLLM_EMBED_H
#define DLLM_EMBED_H

#include <stddef.h>
#include <stdint.h>

#include "dllm_readout.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * out [T, d] = scale * table[tokens].
 *   table   [V, d] bf16, 1 <= V < 2^31 - 1024, d a multiple of 8, d < 2^20
 *   tokens  [T] int32, any values; 0 <= T < 2^31 - 1024.  T = 0 queues nothing
 *   scale   finite; 1 copies rows as they are
 *   out     [T, d] bf16, no overlap with table or tokens
 */
dllm_status dllm_embed(const uint16_t *table, int64_t V, int64_t d, const int32_t *tokens, int64_t T, float scale,
                       uint16_t *out, void *stream);

/* Bytes of workspace dllm_embed_backward needs (host-only arithmetic).  0 if a size is invalid. */
size_t dllm_embed_backward_workspace_bytes(int64_t V, int64_t d, int64_t T);

/*
 * The gradient of the table, of T < 2^30 tokens.
 *   d_out       [T, d] bf16
 *   d_table     [V, d] bf16, no overlap with tokens or d_out (nor has the
 *               workspace)
 *   accumulate  0: every row is written (zero where no token is).
 *               1: added to what d_table holds, once and rounded once; rows
 *               of no token are not touched (a table tied to the LM head takes
 *               the head's gradient first)
 *   workspace   256-byte aligned
 * With T = 0, accumulate = 0 clears d_table and accumulate = 1 queues nothing.
 */
dllm_status dllm_embed_backward(const int32_t *tokens, int64_t T, const uint16_t *d_out, int64_t V, int64_t d,
                                float scale, int32_t accumulate, uint16_t *d_table, void *workspace,
                                size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* DLLM_EMBED_H */

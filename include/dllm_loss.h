/*
 * dllm_loss.h -- C ABI of the training loss of a masked diffusion LLM on AMD
 * Instinct MI355X (gfx950): softmax cross entropy of the masked positions
 * over the whole vocabulary, with the gradients of the hidden states and of
 * the LM head, without the L x V logits.
 *
 * A position i counts if mask[i] != 0 and 0 <= targets[i] < V.  For those
 *   z_iv   = hidden[i] . W_lm[v]
 *   lse_i  = ln sum_v exp(z_iv)
 *   l_i    = lse_i - z_i,targets[i]
 *   loss   = sum_i w_i l_i              (w_i = weights[i], 1 without weights)
 *   dz_iv  = grad w_i (exp(z_iv - lse_i) - [v = targets[i]])
 *   d_hidden[i] = sum_v dz_iv W_lm[v],   d_W[v] = sum_i dz_iv hidden[i]
 * bf16 inputs, fp32 products' sums and softmax statistics.
 * A NaN logit makes the position's lse, loss and gradients NaN, and with them
 * d_W; logits of +inf make lse infinite and the gradients NaN.
 *
 * The vocabulary is taken in pieces.  Forward keeps a running maximum and sum
 * for each row; backward computes a piece's logits again, turns them into dz
 * in the workspace and multiplies that by the piece's rows of W_lm and by the
 * hidden states before the next piece takes its place.  dz is rounded to bf16
 * once, as the operand of those two products; their sums are fp32 over the
 * whole vocabulary and over all rows, and the gradients are rounded once.
 *
 * Memory: every pointer is a DEVICE pointer; bf16 is passed as uint16_t bit
 * patterns; arrays are row-major and contiguous, the bf16 ones 16-byte
 * aligned.  The caller owns everything; nothing is allocated.  Work is queued
 * on `stream` (a hipStream_t, NULL = the default stream), whose device must be
 * the current one, and the calls return without waiting; the number of
 * counted rows stays on the device.  Argument errors return before anything is
 * queued.  Calls queue kernels only and may be captured in HIP graphs; two
 * calls that may overlap in time need a workspace each.  Results do not
 * change from run to run.  The status codes are those of dllm_readout.h.
 */
#ifndef DLLM_LOSS_H
#define DLLM_LOSS_H

#include <stddef.h>
#include <stdint.h>

#include "dllm_readout.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * One set of positions against one LM head (host struct), shared by both
 * directions.
 *   W_lm     [V, d] bf16; 1 <= V < 2^31 - 1024; d a multiple of 8, d < 2^20
 *            (the forward pass is fastest where d is a multiple of 32)
 *   hidden   [L, d] bf16; 1 <= L < 2^31 - 1024
 *   mask     [L] u8: nonzero = the position holds the mask token
 *   targets  [L] int32: the tokens to predict; any other value = no target
 *   weights  [L] float32, or NULL = all 1
 */
typedef struct {
  const uint16_t *W_lm;
  const uint16_t *hidden;
  const uint8_t *mask;
  const int32_t *targets;
  const float *weights;
  int64_t V;
  int64_t d;
  int64_t L;
} dllm_loss;

/* Bytes of workspace dllm_loss_forward needs (host-only arithmetic).  0 if a size is invalid. */
size_t dllm_loss_forward_workspace_bytes(int64_t V, int64_t d, int64_t L);

/*
 *   loss    [1] float32
 *   losses  [L] float32: l_i, never below 0, and 0 where a position does not count
 *   lse     [L] float32: lse_i, and 0 where a position does not count
 *   workspace  256-byte aligned
 * Outputs overlap no input and not each other.
 */
dllm_status dllm_loss_forward(const dllm_loss *p, float *loss, float *losses, float *lse, void *workspace,
                              size_t workspace_bytes, void *stream);

/*
 * Bytes of workspace dllm_loss_backward needs for pieces of `piece`
 * vocabulary entries (host-only arithmetic).  0 if a size is invalid.
 * piece: a multiple of 256, or 0 for the default: as many as make the piece's
 * gradient of the logits about 1 GiB, at least 8192.
 */
size_t dllm_loss_backward_workspace_bytes(int64_t V, int64_t d, int64_t L, int64_t piece);

/*
 *   lse         [L] float32 as dllm_loss_forward wrote it for the same inputs
 *   grad        [1] float32: gradient of the loss, NULL = 1
 *   d_hidden    [L, d] bf16, every row written (zero where a position does not
 *               count); NULL = not wanted
 *   d_W         [V, d] bf16; NULL = not wanted (at least one of the two is)
 *   accumulate  0: d_W is written; 1: the gradient is added to what d_W holds,
 *               once and rounded once
 *   workspace   256-byte aligned
 * Outputs overlap no input and not each other.
 */
dllm_status dllm_loss_backward(const dllm_loss *p, const float *lse, const float *grad, uint16_t *d_hidden,
                               uint16_t *d_W, int32_t accumulate, int64_t piece, void *workspace,
                               size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* DLLM_LOSS_H */

/*
 * dllm_norm.h -- C ABI of the residual update between two blocks of a masked
 * diffusion LLM on AMD Instinct MI355X (gfx950): the norm behind a block, its
 * gate and residual scale, the sum into the residual stream and the norm
 * before the next block, with their gradients.
 *
 * For every token, with N(v, w) = w * v / sqrt(mean(v^2) + eps):
 *   u  = N(y, post), or y where there is no post
 *   x' = x + scale * gate * u      (gate: 1 where there is none)
 *   n  = N(x', pre)
 * y is the block's output, x the residual stream before it and x' behind it,
 * and n the input of the next block.  bf16 in and out; sums and everything
 * between input and output are fp32, and x' and n are rounded once each (n is
 * taken from x' before its rounding).  A row whose sum of squares passes fp32's
 * range (2^128) has a norm of 0.
 *
 * Memory: every pointer is a DEVICE pointer unless marked "host"; bf16 is
 * passed as uint16_t bit patterns; arrays are row-major, contiguous and
 * 16-byte aligned.  The caller owns everything; nothing is allocated.  Work is
 * queued on `stream` (a hipStream_t, NULL = the default stream), whose device
 * must be the current one, and the calls return without waiting.  Argument
 * errors return before anything is queued.  Calls queue kernels only and may
 * be captured in HIP graphs; two calls that may overlap in time need a
 * workspace each.  Results do not change from run to run.  The status codes
 * are those of dllm_readout.h.
 */
#ifndef DLLM_NORM_H
#define DLLM_NORM_H

#include <stddef.h>
#include <stdint.h>

#include "dllm_readout.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest hidden size. */
#define DLLM_NORM_DIM_MAX 8192

/*
 * What a program keeps for one place between two blocks (host struct).
 *   pre, post  [d] bf16 norm weights; NULL = there is no such norm
 *   d          hidden size, a multiple of 8, 8 <= d <= DLLM_NORM_DIM_MAX
 *   eps        finite, >= 0
 *   scale      finite; not read without y
 */
typedef struct {
  const uint16_t *pre;
  const uint16_t *post;
  int64_t d;
  float eps;
  float scale;
} dllm_norm;

/*
 * x_out = x', n = N(x', pre) for T tokens.
 *   x       [T, d] bf16
 *   y       [T, d] bf16; NULL = no update: n = N(x, pre), x_out must be NULL
 *   gate    [groups, d] bf16, or NULL with groups 0.  The tokens are taken as
 *           `groups` equal runs, one gate row each: T % groups == 0
 *           (1 = one gate, T = a gate for every token)
 *   x_out   [T, d] bf16; may be x (in place)
 *   n       [T, d] bf16; NULL exactly if there is no pre
 * Outputs overlap no input (but x_out = x) and not each other.  T = 0 queues
 * nothing.
 */
dllm_status dllm_residual_norm(const dllm_norm *norm, const uint16_t *x, const uint16_t *y, int64_t T,
                               const uint16_t *gate, int64_t groups, uint16_t *x_out, uint16_t *n, void *stream);

/*
 * Bytes of workspace dllm_residual_norm_backward needs (host-only
 * arithmetic).  0 if the norm, T or groups is invalid.
 */
size_t dllm_residual_norm_backward_workspace_bytes(const dllm_norm *norm, int64_t T, int64_t groups);

/*
 * Gradients of dllm_residual_norm from those of its outputs.
 *   x        [T, d] bf16: the stream behind the update (x_out; x without y)
 *   y, gate, groups   as in the forward call
 *            (y's values are read only where post or d_gate is there)
 *   d_n      [T, d] bf16 gradient of n; NULL exactly if there is no pre
 *   d_x_out  [T, d] bf16 gradient of x' from elsewhere; NULL = none
 *   d_x      [T, d] bf16: gradient of x (and of x'); may be d_x_out or d_n
 *   d_y      [T, d] bf16, NULL exactly if there is no y; may be y
 *   d_pre, d_post [d], d_gate [groups, d] float32: gradients summed over the
 *            tokens; NULL = not wanted, and NULL where there is no such input
 * At least one of d_n and d_x_out is given.  With an update x is taken as
 * stored, that is behind the rounding of x'.  Other overlaps of an output are
 * not allowed.  T = 0 queues nothing (and leaves the sums as they were).
 *   workspace  256-byte aligned
 */
dllm_status dllm_residual_norm_backward(const dllm_norm *norm, const uint16_t *x, const uint16_t *y, int64_t T,
                                        const uint16_t *gate, int64_t groups, const uint16_t *d_n,
                                        const uint16_t *d_x_out, uint16_t *d_x, uint16_t *d_y, float *d_pre,
                                        float *d_post, float *d_gate, void *workspace, size_t workspace_bytes,
                                        void *stream);

#ifdef __cplusplus
}
#endif
#endif /* DLLM_NORM_H */

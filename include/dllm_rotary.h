/*
 * dllm_rotary.h -- C ABI of rotary positions for the queries and keys of a
 * masked diffusion LLM on AMD Instinct MI355X (gfx950).
 *
 * A head's first rotary_dim dimensions are taken as rotary_dim / 2 pairs
 * (a, b); pair i of a token at position p is turned by the angle p * theta_i
 * and stretched by the plan's magnitude m:
 *   y_a = m (x_a cos - x_b sin),   y_b = m (x_b cos + x_a sin).
 * The other dimensions are copied.  bf16 in and out; the angle is reduced to
 * a fraction of a turn in fp64, so a far position is as exact as a near one,
 * and the rotation is computed in fp32 and rounded once.
 *
 * Memory: every pointer is a DEVICE pointer unless marked "host"; bf16 is
 * passed as uint16_t bit patterns.  Nothing is allocated.  Work is queued on
 * `stream` (a hipStream_t, NULL = the default stream), whose device must be
 * the current one, and the calls return without waiting.  Argument errors
 * return before anything is queued.  A call is one kernel launch and may be
 * captured in a HIP graph.  The status codes are those of dllm_readout.h.
 */
#ifndef DLLM_ROTARY_H
#define DLLM_ROTARY_H

#include <stddef.h>
#include <stdint.h>

#include "dllm_readout.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Which two dimensions make pair i (r = rotary_dim). */
typedef enum {
  DLLM_ROTARY_HALF = 0,       /* i and i + r / 2 */
  DLLM_ROTARY_INTERLEAVED = 1 /* 2 i and 2 i + 1 */
} dllm_rotary_layout;

/*
 * How the angles theta_i = base^(-2 i / r) are scaled for contexts longer
 * than the trained one, by a factor f >= 1:
 *   PLAIN    not at all
 *   LINEAR   theta_i / f (positions interpolated)
 *   BASE     base replaced by base * f^(r / (r - 2)): the slowest pair is
 *            interpolated by f, the fastest kept (r > 2)
 *   RAMP     by how often a pair turns over the trained length:
 *            n_i = original_len * theta_i / (2 pi),
 *            g_i = clamp((n_i - slow) / (fast - slow), 0, 1),
 *            theta_i (g_i + (1 - g_i) / f): pairs that turn more than `fast`
 *            times are kept, those that turn less than `slow` times are
 *            interpolated, the ones between are blended
 */
typedef enum {
  DLLM_ROTARY_PLAIN = 0,
  DLLM_ROTARY_LINEAR = 1,
  DLLM_ROTARY_BASE = 2,
  DLLM_ROTARY_RAMP = 3
} dllm_rotary_scaling;

/* Largest rotary_dim and head size a call takes. */
#define DLLM_ROTARY_DIM_MAX 512

/*
 * What a program keeps for its rotary positions (host struct).
 *   turns       device float64 [rotary_dim / 2]: turns per position,
 *               theta_i / (2 pi), from dllm_rotary_frequencies
 *   magnitude   m above, finite and > 0 (1 unless the scaling asks for more)
 *   rotary_dim  even, 2 <= rotary_dim <= DLLM_ROTARY_DIM_MAX
 *   layout      a dllm_rotary_layout
 */
typedef struct {
  const double *turns;
  float magnitude;
  int32_t rotary_dim;
  int32_t layout;
} dllm_rotary_plan;

/*
 * Fill turns (host, [rotary_dim / 2] float64) for a plan.  Host-only
 * arithmetic.  factor is read unless PLAIN; original_len, fast and slow for
 * RAMP only.  DLLM_ERR_INVALID_ARG for an odd or out-of-range rotary_dim, base
 * not > 1, factor not >= 1 or not finite, another scaling, BASE with
 * rotary_dim 2, or a RAMP without original_len >= 1 and fast > slow.
 */
dllm_status dllm_rotary_frequencies(int32_t rotary_dim, double base, int32_t scaling, double factor,
                                    int64_t original_len, double fast, double slow, double *turns);

/*
 * y = rotated x for T tokens of H heads of D dimensions.
 *   x, y        bf16; element (t, h, i) at t * token + h * head + i of its
 *               own strides (in elements).  y may be x with the same strides
 *               (in place); no other overlap.  x's strides may be 0
 *               (broadcast); y's elements must be distinct: head >= D and
 *               token >= (H - 1) head + D, or token >= D and
 *               head >= (T - 1) token + D
 *   positions   [T] int32, any values
 *   transpose   0: rotate.  1: rotate the other way (angle negated, same
 *               magnitude): the transposed map, which takes the gradient of
 *               y to the gradient of x
 * rotary_dim <= D <= DLLM_ROTARY_DIM_MAX.  T = 0 queues nothing.  Pointers
 * and strides need no alignment beyond the element's 2 bytes; the fast path
 * takes 16-byte aligned pointers, strides and D in multiples of 8, and in the
 * layout HALF a rotary_dim in multiples of 16.
 */
dllm_status dllm_rotary(const dllm_rotary_plan *plan, const uint16_t *x, int64_t T, int32_t H, int32_t D,
                        int64_t x_token, int64_t x_head, const int32_t *positions, int32_t transpose,
                        uint16_t *y, int64_t y_token, int64_t y_head, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* DLLM_ROTARY_H */

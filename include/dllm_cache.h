/*
 * dllm_cache.h -- C ABI of the 8-bit block cache of a masked diffusion LLM
 * on AMD Instinct MI355X (gfx950): write, attention, accumulation of
 * attention weights and eviction by them.
 *
 * Block-wise decoding keeps the keys and values of the prefix and suffix of
 * the current block in a cache and evicts those that receive little
 * attention (Sparse-dLLM: Accelerating Diffusion LLMs with Dynamic Cache
 * Eviction, Method and Pseudocode: average attention per key, max-pooled
 * with kernel 3, the best share kept; 32-token blocks in More Results).
 *
 * The cache.  Tokens are held in blocks of 32, each block of each key/value
 * head with its own power-of-two scale.  A pool has `pages` blocks; a
 * sequence's block table names the pages that hold its tokens in order, so
 * token j of a sequence is token j % 32 of page table[j / 32].
 *   k, v              [pages, kv_heads, 32 * head_dim] e4m3 bytes
 *   k_scale, v_scale  [pages, kv_heads] bytes: the scale's exponent + 127
 * A value is its e4m3 byte times 2^(scale byte - 127); scale bytes 0 and 255,
 * which no call writes, count as 1 and 254.  The bytes of a block stand in the
 * order in which the matrix instructions read them: with D = head_dim,
 *   k  [D / 32][2][32][16]: byte (c, h, t, j) is token t, dim h D/2 + 16 c + j
 *   v  [D / 32][2][32][16]: byte (c, h, r, b) is token 8 (b / 4) + 4 h + b % 4,
 *                           dim 32 c + r
 * so every 1 KiB of a block is one 16-byte load of each of a wave's lanes.
 *
 * A batch.  S sequences; sequence s brings the tokens cu[s] .. cu[s + 1] - 1
 * of the call's T new tokens (queries, or keys and values to write), and has
 * lens[s] tokens in the cache, the new ones counted.  Tokens at or behind
 * cu[S] belong to none: they are not read, and their rows of any output stay
 * as they were.
 *
 * Bounds.  The arrays of a batch are read on the device and clamped there:
 * cu to 0 .. T, lens to 0 .. max_len, sequences to their first max_new new
 * tokens.  A table entry outside 0 .. pages - 1 is no page: its tokens count
 * as absent (never attended, not written, weight unchanged).  No contents of
 * these arrays lead to an access outside the arrays given.
 *
 * Memory: every pointer is a DEVICE pointer unless marked "host"; bf16 is
 * passed as uint16_t bit patterns; arrays are row-major and contiguous where
 * no stride is given.  The caller owns everything; nothing is allocated.
 * Work is queued on `stream` (a hipStream_t, NULL = the default stream),
 * whose device must be the current one, and the calls return without
 * waiting.  Argument errors return before anything is queued.  Calls queue
 * kernels only and may be captured in HIP graphs; two calls that may overlap
 * in time (two streams, two graphs) need a workspace each.  Results do not
 * change from run to run.  The status codes are those of dllm_readout.h.
 */
#ifndef DLLM_CACHE_H
#define DLLM_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "dllm_readout.h"
#include "dllm_rotary.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DLLM_CACHE_BLOCK 32       /* tokens of a block */
#define DLLM_CACHE_SCALE_MIN 27   /* scale bytes a write chooses: 2^-100 ... */
#define DLLM_CACHE_SCALE_MAX 254  /* ... to 2^127 */

/*
 * A cache (host struct).  head_dim is 64, 128 or 256; kv_heads >= 1;
 * 1 <= pages < 2^31; k and v 16-byte aligned.
 */
typedef struct {
  uint8_t *k;
  uint8_t *v;
  uint8_t *k_scale;
  uint8_t *v_scale;
  int64_t pages;
  int32_t kv_heads;
  int32_t head_dim;
} dllm_cache;

/*
 * A batch (host struct).
 *   cu            [S + 1] int32, ascending from 0
 *   lens          [S] int32
 *   table         [S, table_blocks] int32
 *   S             1 <= S <= 65535
 *   table_blocks  >= 1; table_blocks * 32 < 2^31
 *   max_new       host bound on the new tokens of a sequence, >= 1
 *   max_len       host bound on lens, 1 <= max_len <= table_blocks * 32
 */
typedef struct {
  const int32_t *cu;
  const int32_t *lens;
  const int32_t *table;
  int32_t S;
  int32_t table_blocks;
  int32_t max_new;
  int32_t max_len;
} dllm_cache_batch;

/*
 * Write the new tokens' keys and values: token i of sequence s goes to slot
 * start[s] + i.  lens counts them (max of the old length and start + n).
 *   k, v        [T, kv_heads, D] bf16, element (t, h, i) at t * token +
 *               h * head + i (strides in elements, >= 0)
 *   start       [S] int32; a negative one writes nothing for its sequence
 *   positions   [T] int32 for the rotation of k; NULL only if plan is NULL
 *   plan        rotation of k before it is stored (rotary_dim <= head_dim);
 *               NULL: k is stored as it is
 * Every touched block gets the smallest scale 2^e with
 * g * max |x| <= 448 * 2^e over its new tokens' finite values, but at least
 * the scale it had if it holds other tokens of the sequence; those are
 * requantised when it grows.  g covers what a rotation can grow a value by:
 * 1.41421366 * magnitude for keys rotated in all dimensions, the larger of
 * that and 1 for keys rotated in some (the others stay as they are), else 1.
 * Values are rounded once, to nearest even, from an fp64 rotation.  What is
 * not finite, a key that its rotation takes beyond float32 among it, is
 * stored as NaN.  Slots of touched blocks at or behind lens[s] are cleared.
 * A page may be written through one table entry of a call only.
 */
dllm_status dllm_cache_write(const dllm_cache *cache, const dllm_cache_batch *batch, int64_t T, const uint16_t *k,
                             int64_t k_token, int64_t k_head, const uint16_t *v, int64_t v_token, int64_t v_head,
                             const int32_t *start, const int32_t *positions, const dllm_rotary_plan *plan,
                             void *stream);

/*
 * Bytes of workspace dllm_cache_attention needs for q_heads query heads
 * (host-only arithmetic).  0 if the cache or batch is invalid.
 */
size_t dllm_cache_attention_workspace_bytes(const dllm_cache *cache, const dllm_cache_batch *batch, int32_t q_heads);

/*
 * Attention of the new tokens' queries over the cache:
 *   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q . k_j),
 *   lse = ln sum_j p_j   (natural logarithm)
 * over the visible tokens j of the query's sequence: all j < lens[s], or
 * with causal, for query i of the n of its sequence, j <= lens[s] - n + i.
 * Query head h reads key/value head h / (q_heads / kv_heads).
 *   q        [T, q_heads, D] bf16 by strides (multiples of 8, 16-byte aligned)
 *   q_heads  a multiple of kv_heads
 *   scale    finite, > 0 (a normal float32)
 *   out      [T, q_heads, D] bf16, 16-byte aligned
 *   lse      [T, q_heads] float32, or NULL
 * out and lse overlap no input and not each other; T * q_heads < 2^31 - 1024
 * (else DLLM_ERR_UNSUPPORTED; the same for dllm_cache_weigh).
 * A query that sees no token gets out = 0 and lse = -inf.
 * Sums are fp32.  For its product with v a probability is rounded to fp16
 * once or twice (its own sum takes it unrounded), which below 2^-21 of the
 * largest one moves it by up to 2^-31 of that, and a value counts to within
 * 2^-33 of the head's largest.
 */
dllm_status dllm_cache_attention(const dllm_cache *cache, const dllm_cache_batch *batch, int64_t T, const uint16_t *q,
                                 int64_t q_token, int64_t q_head, int32_t q_heads, float scale, int32_t causal,
                                 uint16_t *out, float *lse, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Accumulate the attention each cached token received:
 *   weights[s, h, j] = decay * weights[s, h, j]
 *                      + sum exp(scale q . k_j - lse)
 * over the sequence's queries and the query heads of key/value head h that
 * see token j, for every j < lens[s]; the rest of weights stays as it was.
 *   lse      [T, q_heads] float32 as dllm_cache_attention wrote it for the
 *            same q, scale and causal
 *            (-inf: the query adds nothing; NaN: the tokens that it sees, and
 *            no others, become NaN)
 *   decay    0 <= decay <= 1; with 0 the old weights are not read
 *   weights  [S, kv_heads, table_blocks * 32] float32
 */
dllm_status dllm_cache_weigh(const dllm_cache *cache, const dllm_cache_batch *batch, int64_t T, const uint16_t *q,
                             int64_t q_token, int64_t q_head, int32_t q_heads, float scale, int32_t causal,
                             const float *lse, float decay, float *weights, void *stream);

/*
 * Evict: of each sequence and key/value head keep n = min(keep[s], lens[s])
 * tokens and move them, in order, to other pages of the pool.  Kept are
 *   - the first f = min(sink, n) tokens,
 *   - the last r = min(recent, n - f),
 *   - of the tokens between, the n - f - r with the largest pooled weight
 *     max(weights[j - pool / 2 .. j + pool / 2]) (within the sequence; NaN
 *     counts as the lowest), the lowest j first among equals.
 * Heads keep different tokens but equally many, so a sequence still has one
 * length.  Keys and values are moved as stored; a block's scale is the
 * largest of the blocks its tokens came from, and bytes are requantised only
 * where that differs from their own.  Slots of the last block behind the
 * kept tokens are cleared.
 *   weights      [S, kv_heads, table_blocks * 32] float32
 *   keep         [S] int32 (negative counts as 0)
 *   max_keep     host bound on keep, 1 <= max_keep <= out_blocks * 32; larger
 *                entries are clamped to it
 *   sink, recent >= 0;  pool odd, 1 <= pool <= 63
 *   table_out    [S, out_blocks] int32: the new pages; none of them may be in
 *                use by a table entry that this call reads, or appear twice
 *   lens_out     [S] int32: n
 *   kept         [S, kv_heads, max_keep] int32: the kept tokens' old places,
 *                ascending; first n written
 *   weights_out  [S, kv_heads, out_blocks * 32] float32: their weights; first
 *                n written.  NULL = not wanted; must not be weights
 *   workspace    dllm_cache_evict_workspace_bytes, 256-byte aligned
 * The old table and pages are untouched: the caller frees what it no longer
 * uses.  batch's cu and max_new are not read.
 */
size_t dllm_cache_evict_workspace_bytes(const dllm_cache *cache, const dllm_cache_batch *batch);

dllm_status dllm_cache_evict(const dllm_cache *cache, const dllm_cache_batch *batch, const float *weights,
                             const int32_t *keep, int32_t max_keep, int32_t sink, int32_t recent, int32_t pool,
                             const int32_t *table_out, int32_t out_blocks, int32_t *lens_out, int32_t *kept,
                             float *weights_out, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* DLLM_CACHE_H */

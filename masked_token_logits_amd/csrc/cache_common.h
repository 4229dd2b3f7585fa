// What the kernels of the 8-bit block cache share (include/dllm_cache.h): the
// clamped view of a batch, page look-up, block addresses and host checks.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "dllm_cache.h"

namespace dllm {

constexpr int kBlock = DLLM_CACHE_BLOCK;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short i16x2 __attribute__((ext_vector_type(2)));

// One sequence of a batch, clamped to the arrays' extents.
struct SeqView {
  int64_t q0;  // its first new token
  int n;       // its new tokens (causal masks count from here)
  int rows;    // those that this call computes: min(n, max_new)
  int len;     // its tokens in the cache
};

__device__ __forceinline__ SeqView seq_view(const dllm_cache_batch& b, int64_t T, int s) {
  SeqView v;
  const int t = (int)T;
  const int c0 = min(max(b.cu[s], 0), t), c1 = min(max(b.cu[s + 1], c0), t);
  v.q0 = c0;
  v.n = c1 - c0;
  v.rows = min(v.n, b.max_new);
  v.len = min(max(b.lens[s], 0), b.max_len);
  return v;
}

// The page of block `blk` (< table_blocks) of sequence s, -1 if it is none.
__device__ __forceinline__ int page_of(const int32_t* __restrict__ table, int table_blocks, int64_t pages, int s,
                                       int blk) {
  const int p = table[(int64_t)s * table_blocks + blk];
  return (p >= 0 && (int64_t)p < pages) ? p : -1;
}

__device__ __forceinline__ int64_t block_of(const dllm_cache& c, int page, int h) {
  return (int64_t)page * c.kv_heads + h;
}

// A stored scale byte: those that are not a normal float32's exponent count as the nearest
// that is, so that 0 is free to stand for no scale at all.
__device__ __forceinline__ int stored_scale(const uint8_t* scale, int64_t at) { return min(max((int)scale[at], 1), 254); }

// 2^(byte - 127) for a scale byte of 1 .. 254.
__device__ __forceinline__ float scale_value(int byte) { return __uint_as_float((uint32_t)byte << 23); }

inline bool cache_ok(const dllm_cache* c) {
  return c && c->k && c->v && c->k_scale && c->v_scale && c->pages >= 1 && c->kv_heads >= 1;
}
inline bool cache_supported(const dllm_cache* c) {
  return (c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256) && c->pages < ((int64_t)1 << 31) &&
         c->kv_heads <= 65535 && (((uintptr_t)c->k | (uintptr_t)c->v) & 15u) == 0;
}
inline bool batch_ok(const dllm_cache_batch* b) {
  return b && b->cu && b->lens && b->table && b->S >= 1 && b->S <= 65535 && b->table_blocks >= 1 &&
         b->table_blocks < (1 << 26) && b->max_new >= 1 && b->max_len >= 1 &&
         (int64_t)b->max_len <= (int64_t)b->table_blocks * kBlock;
}
inline bool tokens_ok(int64_t T) { return T >= 0 && T < ((int64_t)1 << 31); }
inline bool stride_ok(int64_t s) { return s >= 0 && s < ((int64_t)1 << 31); }

}  // namespace dllm

// The arithmetic of attention over e4m3 blocks, in matrix tiles of 32 queries.
//
// A wave holds 32 query rows as the columns of its tiles: lane l works for
// column l % 32, and the two lanes of a column share its softmax state.  A
// block's scores are S^T = K Q^T (v_mfma_f32_32x32x16_bf16, K the left
// operand), so lane l's 16 scores of a block belong to its own column, to
// the tokens 8 (i / 4) + 4 (l / 32) + i % 4.  The output is O^T = V^T P^T, in
// which the probabilities are the right operand and a block's stored order of
// V is the left one: nothing is transposed, and maxima, sums and rescalings
// are lane-local but for one exchange between the two halves.
//
// Keys are widened to bf16 on their way into the matrix pipe, with their
// block's power-of-two scale applied by the conversion; that is exact, and so
// are the products with bf16 queries.  Probabilities and values go in as
// fp16: 11 bits of a probability instead of bf16's 8 (with bf16 the output's
// error against fp64 was 1.4 times that of its own rounding, with fp16 it is
// that of the rounding), at the same rate.  fp16's range is met by keeping
// both relative: a probability to a running reference (below), a value to
// the largest scale of the blocks seen, from which a later block may differ
// by up to 2^7 before O is rescaled.  A value is then within 2^-33 of the
// largest one of the head, exact unless its block's scale is 2^15 smaller.
//
// The e4m3 matrix instructions would save the conversions (with queries and
// probabilities as sums of two e4m3 terms), but they align the 64 products
// of a sum to the largest and drop what lies more than 13 bits below it
// (measured: 2^16 + 2^2 comes out as 2^16), which put scores 1e-4 off.  The
// 16-bit instructions keep the full fp32 sum.
#pragma once

#include "cache_common.h"

namespace dllm {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Probabilities are held as 2^(s - ref), s the score in base 2 and ref a past
// running maximum less kOffset: O and the sum are rescaled only when the
// maximum has grown by more than kSlack over it, which after the first
// blocks is rare.  The largest probability of a column is so between 2^7 and
// 2^15 (fp16 ends at 2^16), and the smallest that counts 2^-25.
constexpr float kOffset = 7.0f, kSlack = 8.0f;
constexpr int kValueSlack = 7;  // 448 * 2^7 = 57344 is still an fp16 number

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// One 8-deep operand of a lane.
union Frag {
  bf16x8 b;
  bf16x2 b2[4];
  f16x8 h;
  f16x2 h2[4];
  i32x4 w;
};

// f(0), f(1), ... with constants, so that what they index is in registers from
// the first pass of the compiler on.
template <int I>
struct Const {
  static constexpr int value = I;
};
template <int I, int N, class F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(Const<I>{});
    each<I + 1, N>(f);
  }
}

// max and sum of the two lanes of a column, in both.
__device__ __forceinline__ float column_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float column_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// 16 e4m3 bytes, times the scale, as two operands of 8 bf16.
__device__ __forceinline__ void widen_keys(i32x4 raw, float scale, Frag& lo, Frag& hi) {
  lo.b2[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[0], scale, false);
  lo.b2[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[0], scale, true);
  lo.b2[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[1], scale, false);
  lo.b2[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[1], scale, true);
  hi.b2[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[2], scale, false);
  hi.b2[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[2], scale, true);
  hi.b2[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[3], scale, false);
  hi.b2[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[3], scale, true);
}

// 16 e4m3 bytes, times the scale, as two operands of 8 fp16.
__device__ __forceinline__ void widen_values(i32x4 raw, float scale, Frag& lo, Frag& hi) {
  lo.h2[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw[0], scale, false);
  lo.h2[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw[0], scale, true);
  lo.h2[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw[1], scale, false);
  lo.h2[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw[1], scale, true);
  hi.h2[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw[2], scale, false);
  hi.h2[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw[2], scale, true);
  hi.h2[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw[3], scale, false);
  hi.h2[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw[3], scale, true);
}

// This lane's half of a query row: dims half * D/2 .. of it, 8 to an operand.
template <int D>
__device__ __forceinline__ void load_query(Frag* q, const uint16_t* row, int half) {
  const i32x4* p = reinterpret_cast<const i32x4*>(row + half * (D / 2));
#pragma unroll
  for (int i = 0; i < D / 16; ++i) q[i].w = p[i];
}

// S^T of one block, 32 tokens x 32 queries, in units of q . k.  raw: the
// lane's D / 32 loads of 16 bytes of the key block.
template <int D>
__device__ __forceinline__ f32x16 scores(const Frag* q, const i32x4* raw, float k_scale) {
  f32x16 s = {};
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    Frag lo, hi;
    widen_keys(raw[i], k_scale, lo, hi);
    s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(lo.b, q[2 * i].b, s, 0, 0, 0);
    s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(hi.b, q[2 * i + 1].b, s, 0, 0, 0);
  }
  return s;
}

// Token of a lane's score i within its block.
__device__ __forceinline__ int token_of(int i, int half) { return 8 * (i >> 2) + 4 * half + (i & 3); }

// Softmax state of a column (both its lanes hold the same ref; sum is the
// lane's own share) and O^T.
template <int D>
struct Accumulator {
  f32x16 o[D / 32];
  float ref;  // base-2 reference; -inf before the first visible token
  float sum;
  int v_ref;  // scale byte that O is relative to; 0 before the first block
};

template <int D>
__device__ __forceinline__ void clear(Accumulator<D>& a) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) a.o[i][j] = 0.0f;
  a.ref = -INFINITY;
  a.sum = 0.0f;
  a.v_ref = 0;
}

template <int D>
__device__ __forceinline__ void rescale(Accumulator<D>& a, float alpha) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) a.o[i][j] *= alpha;
}

// 2^x for an integer x, 0 below fp32's normal range.
__device__ __forceinline__ float exact_power(int x) { return x < -126 ? 0.0f : __uint_as_float((uint32_t)(x + 127) << 23); }

// The factor that a block's values are widened with (its scale relative to
// O's), after O has been moved to a scale that covers it.  v_byte is uniform.
template <int D>
__device__ __forceinline__ float cover_values(Accumulator<D>& a, int v_byte) {
  if (a.v_ref == 0) a.v_ref = v_byte;
  if (v_byte > a.v_ref + kValueSlack) {
    rescale(a, exact_power(a.v_ref - v_byte));
    a.v_ref = v_byte;
  }
  return __uint_as_float((uint32_t)max(v_byte - a.v_ref + 127, 1) << 23);
}

// What a state with reference `own` counts for under reference `ref`.
__device__ __forceinline__ float part_of_ref(float own, float ref) {
  return own == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(own - ref);
}

// The negative of a reference, as the probabilities take it: a column that
// has seen no token (ref = -inf) gets probabilities of 0.
__device__ __forceinline__ float negative(float ref) { return ref == -INFINITY ? -INFINITY : -ref; }

// Move the reference to cover scores up to `top` (this lane's largest), if
// they have outgrown it.
template <int D>
__device__ __forceinline__ void cover(Accumulator<D>& a, float top, float scale2) {
  const float want = __builtin_fmaf(column_max(top), scale2, -kOffset);
  if (__any(want > a.ref + kSlack)) {
    const float ref = fmaxf(a.ref, want);
    const float alpha = part_of_ref(a.ref, ref);
    a.ref = ref;
    a.sum *= alpha;
    rescale(a, alpha);
  }
}

__device__ __forceinline__ float largest(const f32x16& s) {
  float top = s[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
  return top;
}

// Probabilities of one block's scores against the reference -neg, rounded to
// fp16 operands; returns their unrounded sum.
__device__ __forceinline__ float probabilities(const f32x16& s, float scale2, float neg, Frag* p) {
  float even = 0.0f, odd = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], scale2, neg));
    const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i + 1], scale2, neg));
    even += x;
    odd += y;
    p[i / 8].h2[(i % 8) / 2] = f16x2{(_Float16)x, (_Float16)y};
  }
  return even + odd;
}

template <int D>
__device__ __forceinline__ void probabilities(Accumulator<D>& a, const f32x16& s, float scale2, Frag* p) {
  a.sum += probabilities(s, scale2, negative(a.ref), p);
}

// O^T += V^T P^T of one block.  raw: the lane's D / 32 loads of its values.
template <int D>
__device__ __forceinline__ void add_values(Accumulator<D>& a, const Frag* p, const i32x4* raw, float v_scale) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    Frag lo, hi;
    widen_values(raw[i], v_scale, lo, hi);
    a.o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(lo.h, p[0].h, a.o[i], 0, 0, 0);
    a.o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(hi.h, p[1].h, a.o[i], 0, 0, 0);
  }
}

// NaN bytes of a chunk of values taken out of it: nan has a 1 in their place.
__device__ __forceinline__ void take_nan(i32x4& x, i32x4& nan) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    nan[j] = (((x[j] & 0x7f7f7f7f) + 0x01010101) >> 7) & 0x01010101;
    x[j] &= ~(nan[j] * 0xff);
  }
}

// O^T of a chunk made NaN where a NaN value (take_nan) is visible to the
// column: limit is its number of visible tokens of the block.
__device__ __forceinline__ void spread_nan(f32x16& o, i32x4 nan, int limit, int half) {
  Frag see[2], lo, hi;
#pragma unroll
  for (int j = 0; j < 16; j += 2)
    see[j / 8].h2[(j % 8) / 2] = f16x2{(_Float16)(token_of(j, half) < limit ? 1.0f : 0.0f),
                                       (_Float16)(token_of(j + 1, half) < limit ? 1.0f : 0.0f)};
  widen_values(nan * 0x38, 1.0f, lo, hi);  // 1.0
  f32x16 hit = {};
  hit = __builtin_amdgcn_mfma_f32_32x32x16_f16(lo.h, see[0].h, hit, 0, 0, 0);
  hit = __builtin_amdgcn_mfma_f32_32x32x16_f16(hi.h, see[1].h, hit, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < 16; ++j) o[j] = hit[j] > 0.0f ? NAN : o[j];
}

// add_values for a block that some of the tile's columns see only in part: a
// NaN value must not reach, as 0 * NaN, a column that masks its token.  NaN
// bytes are taken out of the product, and where one is visible the result is
// made NaN; that second product is made only if there is such a byte.
template <int D>
__device__ __forceinline__ void add_values_masked(Accumulator<D>& a, const Frag* p, const i32x4* raw, float v_scale,
                                                  int limit, int half) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    Frag lo, hi;
    i32x4 x = raw[i], nan;
    take_nan(x, nan);
    widen_values(x, v_scale, lo, hi);
    a.o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(lo.h, p[0].h, a.o[i], 0, 0, 0);
    a.o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(hi.h, p[1].h, a.o[i], 0, 0, 0);
    if (__any(nan[0] | nan[1] | nan[2] | nan[3])) spread_nan(a.o[i], nan, limit, half);
  }
}

// The lane's 16 bytes of values with those of tokens at or behind `limit`
// cleared: what lies there may be anything, NaN among it, and 0 * NaN is NaN.
__device__ __forceinline__ i32x4 clip_values(i32x4 v, int half, int limit) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = min(max(limit - (8 * i + 4 * half), 0), 4);
    v[i] &= n == 4 ? -1 : (1 << (8 * n)) - 1;
  }
  return v;
}

}  // namespace dllm

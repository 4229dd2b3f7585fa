// The rotation of one pair, shared by the rotary kernel and the cache write.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bf16.h"
#include "dllm_rotary.h"

namespace dllm {

// cos and sin of position * theta, given theta as turns per position, times
// the magnitude.  The product and its reduction to a fraction of a turn are
// fp64 (a position of 2^17 in fp32 turns would lose 17 bits of the fraction);
// the fraction is then small enough that fp32 holds it to 2^-25 of a turn.
__device__ __forceinline__ float2 rotary_angle(int pos, double turns, float magnitude) {
  double t = (double)pos * turns;
  t -= rint(t);
  float s, c;
  sincospif(2.0f * (float)t, &s, &c);
  return make_float2(c * magnitude, s * magnitude);
}

// (a, b) turned by (cos, sin).
__device__ __forceinline__ float rotated_a(float a, float b, float2 cs) { return a * cs.x - b * cs.y; }
__device__ __forceinline__ float rotated_b(float a, float b, float2 cs) { return b * cs.x + a * cs.y; }

// The same in fp64, for keys that are rounded to 4 significant bits: there an
// fp32 rotation falls on the other side of a rounding boundary about once in
// a million values, this one on none.  The fraction of a turn is taken to the
// nearest quarter, and the rest, at most an eighth of a turn, goes through
// the Taylor series of cosine and sine (the first term left out is below
// 2^-46); some 30 fp64 operations, at fp32's rate on this chip.
__device__ __forceinline__ double2 rotary_angle64(int pos, double turns, double magnitude) {
  double t = (double)pos * turns;
  t -= rint(t);
  const double quarter = rint(4.0 * t);
  const double x = (t - 0.25 * quarter) * 6.283185307179586476925286766559, z = x * x;
  double s = 1.0 / 6227020800.0;  // 1 / 13!
  s = fma(s, z, -1.0 / 39916800.0);
  s = fma(s, z, 1.0 / 362880.0);
  s = fma(s, z, -1.0 / 5040.0);
  s = fma(s, z, 1.0 / 120.0);
  s = fma(s, z, -1.0 / 6.0);
  s = fma(s * z, x, x);
  double c = -1.0 / 87178291200.0;  // -1 / 14!
  c = fma(c, z, 1.0 / 479001600.0);
  c = fma(c, z, -1.0 / 3628800.0);
  c = fma(c, z, 1.0 / 40320.0);
  c = fma(c, z, -1.0 / 720.0);
  c = fma(c, z, 1.0 / 24.0);
  c = fma(c, z, -0.5);
  c = fma(c, z, 1.0);
  const int q = (int)quarter & 3;  // a quarter of -2 .. 2
  const double cq = q & 1 ? s : c, sq = q & 1 ? c : s;
  return make_double2((q == 1 || q == 2 ? -cq : cq) * magnitude, (q >= 2 ? -sq : sq) * magnitude);
}

// x in fp32 with 20 bits behind the first and the last of them set if that is
// not exact (rounding to odd), so that a later rounding to far fewer bits is as if
// made from x itself.
__device__ __forceinline__ float odd_float(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  const uint32_t hi = (uint32_t)(u >> 32) | min((uint32_t)u, 1u);
  return (float)__longlong_as_double((int64_t)((uint64_t)hi << 32));
}

inline bool rotary_plan_ok(const dllm_rotary_plan* p, int64_t head_dim) {
  return p && p->turns && p->rotary_dim >= 2 && p->rotary_dim % 2 == 0 && p->rotary_dim <= head_dim &&
         p->rotary_dim <= DLLM_ROTARY_DIM_MAX && (p->layout == DLLM_ROTARY_HALF || p->layout == DLLM_ROTARY_INTERLEAVED) &&
         p->magnitude > 0.0f && p->magnitude <= 3.0e38f;
}

}  // namespace dllm

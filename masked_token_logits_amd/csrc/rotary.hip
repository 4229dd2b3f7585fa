// Rotary positions (include/dllm_rotary.h): the frequency table on the host
// and the kernel that rotates [T, H, D] bf16 heads.
#include "dllm_rotary.h"
#include "rotary_angle.h"

#include <math.h>

namespace dllm {
namespace {

constexpr int kThreads = 256;

// One workgroup takes `tokens` consecutive tokens: it computes their angles
// into LDS once and applies them to every head.
__global__ __launch_bounds__(kThreads) void k_rotary(dllm_rotary_plan plan, const uint16_t* x, int64_t T, int H, int D,
                                                     int64_t x_token, int64_t x_head,
                                                     const int32_t* __restrict__ positions, int transpose,
                                                     uint16_t* y, int64_t y_token, int64_t y_head) {
  __shared__ float2 cs[DLLM_ROTARY_DIM_MAX / 2];
  const int half = plan.rotary_dim / 2;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    const int pos = positions[t];
    for (int i = threadIdx.x; i < half; i += kThreads) {
      float2 a = rotary_angle(pos, plan.turns[i], plan.magnitude);
      if (transpose) a.y = -a.y;
      cs[i] = a;
    }
    __syncthreads();
    // a unit is a pair, or two of the dimensions behind the rotated ones
    const int units = (D + 1) / 2;
    for (int u = threadIdx.x; u < H * units; u += kThreads) {
      const int h = u / units, i = u - h * units;
      const uint16_t* px = x + t * x_token + h * x_head;
      uint16_t* py = y + t * y_token + h * y_head;
      if (i < half) {
        const int a = plan.layout == DLLM_ROTARY_HALF ? i : 2 * i;
        const int b = plan.layout == DLLM_ROTARY_HALF ? i + half : 2 * i + 1;
        const float xa = bf16_float(px[a]), xb = bf16_float(px[b]);
        py[a] = (uint16_t)float_bf16(rotated_a(xa, xb, cs[i]));
        py[b] = (uint16_t)float_bf16(rotated_b(xa, xb, cs[i]));
      } else {
        py[2 * i] = px[2 * i];
        if (2 * i + 1 < D) py[2 * i + 1] = px[2 * i + 1];
      }
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace dllm

extern "C" {

dllm_status dllm_rotary_frequencies(int32_t rotary_dim, double base, int32_t scaling, double factor,
                                    int64_t original_len, double fast, double slow, double* turns) {
  if (!turns || rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > DLLM_ROTARY_DIM_MAX) return DLLM_ERR_INVALID_ARG;
  if (!(base > 1.0) || !isfinite(base)) return DLLM_ERR_INVALID_ARG;
  if (scaling < DLLM_ROTARY_PLAIN || scaling > DLLM_ROTARY_RAMP) return DLLM_ERR_INVALID_ARG;
  if (scaling != DLLM_ROTARY_PLAIN && !(factor >= 1.0 && isfinite(factor))) return DLLM_ERR_INVALID_ARG;
  if (scaling == DLLM_ROTARY_BASE && rotary_dim == 2) return DLLM_ERR_INVALID_ARG;
  if (scaling == DLLM_ROTARY_RAMP && (original_len < 1 || !isfinite(fast) || !isfinite(slow) || !(fast > slow)))
    return DLLM_ERR_INVALID_ARG;
  const double r = rotary_dim, two_pi = 6.283185307179586476925286766559;
  if (scaling == DLLM_ROTARY_BASE) base *= pow(factor, r / (r - 2.0));
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double theta = pow(base, -2.0 * i / r);
    if (scaling == DLLM_ROTARY_LINEAR) theta /= factor;
    if (scaling == DLLM_ROTARY_RAMP) {
      double g = ((double)original_len * theta / two_pi - slow) / (fast - slow);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      theta *= g + (1.0 - g) / factor;
    }
    turns[i] = theta / two_pi;
  }
  return DLLM_OK;
}

dllm_status dllm_rotary(const dllm_rotary_plan* plan, const uint16_t* x, int64_t T, int32_t H, int32_t D,
                        int64_t x_token, int64_t x_head, const int32_t* positions, int32_t transpose, uint16_t* y,
                        int64_t y_token, int64_t y_head, void* stream) {
  if (T < 0 || T >= ((int64_t)1 << 31) || H < 1 || D < 1) return DLLM_ERR_INVALID_ARG;
  if (!dllm::rotary_plan_ok(plan, D) || (transpose != 0 && transpose != 1)) return DLLM_ERR_INVALID_ARG;
  if (x_token < 0 || x_head < 0 || y_token < 0 || y_head < 0) return DLLM_ERR_INVALID_ARG;
  if (D > DLLM_ROTARY_DIM_MAX || H > (1 << 20)) return DLLM_ERR_UNSUPPORTED;
  if (T == 0) return DLLM_OK;
  if (!x || !y || !positions) return DLLM_ERR_INVALID_ARG;
  if (x_token >= ((int64_t)1 << 31) || x_head >= ((int64_t)1 << 31) || y_token >= ((int64_t)1 << 31) ||
      y_head >= ((int64_t)1 << 31))
    return DLLM_ERR_UNSUPPORTED;  // keeps every offset below 2^62
  const bool by_token = y_head >= D && y_token >= (H - 1) * y_head + D;
  const bool by_head = y_token >= D && y_head >= (T - 1) * y_token + D;
  if ((T > 1 || H > 1) && !by_token && !by_head && !(T == 1 && y_head >= D) && !(H == 1 && y_token >= D))
    return DLLM_ERR_INVALID_ARG;
  if (x == y && (x_token != y_token || x_head != y_head)) return DLLM_ERR_INVALID_ARG;
  const unsigned grid = (unsigned)(T < 65536 ? T : 65536);
  hipLaunchKernelGGL(dllm::k_rotary, dim3(grid), dim3(dllm::kThreads), 0, reinterpret_cast<hipStream_t>(stream), *plan,
                     x, T, (int)H, (int)D, x_token, x_head, positions, (int)transpose, y, y_token, y_head);
  return hipGetLastError() == hipSuccess ? DLLM_OK : DLLM_ERR_HIP;
}

}  // extern "C"

// Rotary positions (include/dllm_rotary.h): the frequency table on the host
// and the kernel that rotates [T, H, D] bf16 heads.
#include "dllm_rotary.h"
#include "rotary_angle.h"

#include <math.h>

namespace dllm {
namespace {

constexpr int kThreads = 256, kTokens = 8;  // threads and, at most, tokens of a workgroup

// Any sizes, strides and alignment, element by element: a workgroup computes
// a token's angles into LDS once and applies them to every head.  70 of 128
// dimensions of 28 heads, 8192 tokens: 44 us, bound by the 2-byte accesses.
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

struct PieceArgs {
  dllm_rotary_plan plan;
  const uint16_t* x;
  int64_t T;
  int H, D;
  int64_t x_token, x_head;
  const int32_t* positions;
  int transpose;
  uint16_t* y;
  int64_t y_token, y_head;
  int pieces;          // of a head
  uint32_t per_piece;  // n / pieces = high word of n * per_piece: exact for n * pieces < 2^32; 0 where pieces is 1
  int tokens;          // of a workgroup
  uint32_t per_token;  // likewise n / (H * pieces), where there is more than one token
};

// n / d by d's reciprocal, which is 2^32 for d = 1 and does not fit: 0 stands for it.
__device__ __forceinline__ int divided(int n, uint32_t per) { return per ? (int)__umulhi((uint32_t)n, per) : n; }

// Heads in pieces of two units of 16 bytes: eight pairs, or what lies behind the
// rotated dimensions.  A workgroup takes as many tokens as give each thread a piece; its
// first loads are on their way while the angles go into LDS.
//
// Bound by memory: 8192 tokens of 32 heads of 128, all rotated, 21.8 us (6.2 TB/s read
// and written, the card's copy rate and some of its last-level cache); half of 28 heads
// out of a fused projection 23 us.  Four tokens to a workgroup however many pieces
// they have, their loads together, were no faster there and slower below 4096 tokens
// (512: 5.1 us against 3.8).  16384 tokens of 8 heads, at one token to a workgroup 18.7 us,
// take 14.0.
__global__ __launch_bounds__(kThreads) void k_rotary_pieces(PieceArgs a) {
  __shared__ float4 cs[kTokens][DLLM_ROTARY_DIM_MAX / 4];  // two pairs' (cos, sin)
  const int half = a.plan.rotary_dim / 2, rotated = (a.plan.rotary_dim + 15) / 16, of_token = a.H * a.pieces;
  const bool halves = a.plan.layout == DLLM_ROTARY_HALF;
  for (int64_t t0 = (int64_t)blockIdx.x * a.tokens; t0 < a.T; t0 += (int64_t)gridDim.x * a.tokens) {
    const int tokens = (int)min(a.T - t0, (int64_t)a.tokens), all = tokens * of_token;
    uint4 u[2];
    int t = 0, h = 0, piece = 0, first = 0, second = 0;  // the piece's token, head and number, its units' first dimensions
    auto load = [&](int n) {
      if (a.tokens > 1) {
        t = divided(n, a.per_token);
        n -= t * of_token;
      }
      h = divided(n, a.per_piece);
      piece = n - h * a.pieces;
      first = halves && piece < rotated ? 8 * piece : 16 * piece;
      second = halves && piece < rotated ? first + half : first + 8;
      const uint16_t* p = a.x + (t0 + t) * a.x_token + h * a.x_head;
      u[0] = *reinterpret_cast<const uint4*>(p + first);
      if (second < a.D) u[1] = *reinterpret_cast<const uint4*>(p + second);
    };
    int n = threadIdx.x;
    if (n < all) load(n);
    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
      const int j = a.tokens > 1 ? (uint32_t)i / (uint32_t)half : 0, pair = i - j * half;
      float2 c = rotary_angle(a.positions[t0 + j], a.plan.turns[pair], a.plan.magnitude);
      if (a.transpose) c.y = -c.y;
      reinterpret_cast<float2*>(cs[j])[pair] = c;
    }
    __syncthreads();
    while (n < all) {
      if (piece < rotated) {
        float4 c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = cs[t][piece * 4 + i];
        uint32_t* w0 = reinterpret_cast<uint32_t*>(&u[0]);
        uint32_t* w1 = reinterpret_cast<uint32_t*>(&u[1]);
        if (halves) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 c0 = make_float2(c[i].x, c[i].y), c1 = make_float2(c[i].z, c[i].w);
            const float a0 = bf16_float(w0[i] & 0xffff), a1 = bf16_float(w0[i] >> 16);
            const float b0 = bf16_float(w1[i] & 0xffff), b1 = bf16_float(w1[i] >> 16);
            w0[i] = float_bf16(rotated_a(a0, b0, c0)) | float_bf16(rotated_a(a1, b1, c1)) << 16;
            w1[i] = float_bf16(rotated_b(a0, b0, c0)) | float_bf16(rotated_b(a1, b1, c1)) << 16;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 ci = i % 2 ? make_float2(c[i / 2].z, c[i / 2].w) : make_float2(c[i / 2].x, c[i / 2].y);
            uint32_t& w = i < 4 ? w0[i] : w1[i - 4];
            const float xa = bf16_float(w & 0xffff), xb = bf16_float(w >> 16);
            const uint32_t y = float_bf16(rotated_a(xa, xb, ci)) | float_bf16(rotated_b(xa, xb, ci)) << 16;
            w = 8 * piece + i < half ? y : w;  // the last piece may hold dimensions behind the rotated ones
          }
        }
      }
      uint16_t* p = a.y + (t0 + t) * a.y_token + h * a.y_head;
      *reinterpret_cast<uint4*>(p + first) = u[0];
      if (second < a.D) *reinterpret_cast<uint4*>(p + second) = u[1];
      n += kThreads;
      if (n < all) load(n);
    }
    __syncthreads();  // cs is the next tokens'
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
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const bool aligned = (((uintptr_t)x | (uintptr_t)y) & 15u) == 0 && (x_token | x_head | y_token | y_head | D) % 8 == 0;
  if (aligned && (plan->rotary_dim % 16 == 0 || plan->layout == DLLM_ROTARY_INTERLEAVED)) {
    const int rotated = (plan->rotary_dim + 15) / 16, pieces = rotated + (D - 16 * rotated + 15) / 16, all = H * pieces;
    const int fit = dllm::kThreads / all, tokens = fit < 1 ? 1 : fit < dllm::kTokens ? fit : dllm::kTokens;
    const auto per = [](int d) { return d == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + d - 1) / d); };
    const dllm::PieceArgs a = {*plan, x, T, (int)H, (int)D, x_token, x_head, positions, (int)transpose, y, y_token, y_head,
                               pieces, per(pieces), tokens, per(all)};
    const int64_t groups = (T + tokens - 1) / tokens;
    const dim3 grid((unsigned)(groups < (1 << 22) ? groups : 1 << 22));
    hipLaunchKernelGGL(dllm::k_rotary_pieces, grid, dim3(dllm::kThreads), 0, st, a);
  } else {
    const dim3 grid((unsigned)(T < (1 << 16) ? T : 1 << 16));
    hipLaunchKernelGGL(dllm::k_rotary, grid, dim3(dllm::kThreads), 0, st, *plan, x, T, (int)H, (int)D, x_token, x_head,
                       positions, (int)transpose, y, y_token, y_head);
  }
  return hipGetLastError() == hipSuccess ? DLLM_OK : DLLM_ERR_HIP;
}

}  // extern "C"

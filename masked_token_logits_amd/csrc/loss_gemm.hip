// The three products of the loss's backward pass (include/dllm_loss.h), for
// one piece of the vocabulary:
//   dz[i, v]   = coef_i (exp(h_i . W_v - lse_i) - [v = t_i])
//   acc[i, c] += sum_v dz[i, v] W[v, c]
//   d_W[v, c]  = sum_i dz[i, v] h[i, c]
#include <math.h>

#include "bf16.h"
#include "loss_internal.h"
#include "online_state.h"

namespace dllm {
namespace {

typedef short bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

enum { kDz = 0, kDHidden = 1, kDW = 2 };

constexpr int kT = 64, kK = 32, kLd = kK + 8;

// 64 x 64 tiles of four waves, 32 x 32 each, K in steps of 32 through LDS.
template <int MODE>
__global__ __launch_bounds__(256) void k_loss_product(GradArgs a) {
  __shared__ __attribute__((aligned(16))) uint16_t As[kT * kLd], Bs[kT * kLd];
  const int M = min(a.ctr[0], a.L);
  const int rows = MODE == kDW ? a.n : M, cols = MODE == kDz ? a.n : a.d, K = MODE == kDz ? a.d : MODE == kDHidden ? a.n : M;
  const int tr = (rows + kT - 1) / kT, tc = (cols + kT - 1) / kT;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int64_t e = blockIdx.x; e < (int64_t)tr * tc; e += gridDim.x) {
    const int r0 = (int)(e / tc) * kT, c0 = (int)(e % tc) * kT;
    f32x4 acc[2][2] = {};
    for (int k0 = 0; k0 < K; k0 += kK) {
      uint4 ua = make_uint4(0, 0, 0, 0), ub = make_uint4(0, 0, 0, 0);
      // operands whose K is contiguous: row tid / 4, piece tid % 4; the others: k tid / 8, piece tid % 8
      const int rr = tid >> 2, kk = k0 + 8 * (tid & 3), kt = k0 + (tid >> 3), ct = 8 * (tid & 7);
      if constexpr (MODE == kDz) {
        if (r0 + rr < rows && kk < K) ua = *reinterpret_cast<const uint4*>(a.H + (int64_t)a.idx[r0 + rr] * a.d + kk);
        if (c0 + rr < cols && kk < K) ub = *reinterpret_cast<const uint4*>(a.W + (int64_t)(a.v0 + c0 + rr) * a.d + kk);
      } else if constexpr (MODE == kDHidden) {
        if (r0 + rr < rows && kk < K) ua = *reinterpret_cast<const uint4*>(a.dz + (int64_t)(r0 + rr) * a.ldz + kk);
        if (kt < K && c0 + ct < cols) ub = *reinterpret_cast<const uint4*>(a.W + (int64_t)(a.v0 + kt) * a.d + c0 + ct);
      } else {
        if (kt < K && r0 + ct < rows) ua = *reinterpret_cast<const uint4*>(a.dz + (int64_t)kt * a.ldz + r0 + ct);
        if (kt < K && c0 + ct < cols) ub = *reinterpret_cast<const uint4*>(a.H + (int64_t)a.idx[kt] * a.d + c0 + ct);
      }
      __syncthreads();
      if constexpr (MODE == kDW) {
        const uint32_t w[4] = {ua.x, ua.y, ua.z, ua.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) As[(ct + j) * kLd + (tid >> 3)] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
      } else {
        *reinterpret_cast<uint4*>(As + rr * kLd + 8 * (tid & 3)) = ua;
      }
      if constexpr (MODE == kDz) {
        *reinterpret_cast<uint4*>(Bs + rr * kLd + 8 * (tid & 3)) = ub;
      } else {
        const uint32_t w[4] = {ub.x, ub.y, ub.z, ub.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) Bs[(ct + j) * kLd + (tid >> 3)] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
      }
      __syncthreads();
      bf16x8 fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fa[i] = *reinterpret_cast<const bf16x8*>(As + ((wave >> 1) * 32 + i * 16 + (lane & 15)) * kLd + 8 * (lane >> 4));
        fb[i] = *reinterpret_cast<const bf16x8*>(Bs + ((wave & 1) * 32 + i * 16 + (lane & 15)) * kLd + 8 * (lane >> 4));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
    __syncthreads();
    // accumulator x of block (i, j): row 16 i + 4 (lane / 16) + x, column 16 j + lane % 16 of the wave's 32 x 32
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int r = r0 + (wave >> 1) * 32 + i * 16 + 4 * (lane >> 4) + x;
        if (r >= rows) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = c0 + (wave & 1) * 32 + j * 16 + (lane & 15);
          if constexpr (MODE == kDz) {
            if (c >= a.ldz) continue;
            float v = 0.f;  // entries behind the piece, up to a whole step of K
            if (c < cols)
              v = a.coef[r] * (__builtin_amdgcn_exp2f((acc[i][j][x] - a.lse[r]) * kLog2eF) - (a.v0 + c == a.tgt[r] ? 1.f : 0.f));
            a.dz[(int64_t)r * a.ldz + c] = (uint16_t)float_bf16(v);
          } else if constexpr (MODE == kDHidden) {
            if (c >= cols) continue;
            float* o = a.acc + (int64_t)r * a.d + c;
            const float v = a.first ? acc[i][j][x] : *o + acc[i][j][x];
            if (a.last)
              a.d_hidden[(int64_t)a.idx[r] * a.d + c] = (uint16_t)float_bf16(v);
            else
              *o = v;
          } else {
            if (c >= cols) continue;
            uint16_t* o = a.d_W + (int64_t)(a.v0 + r) * a.d + c;
            const float v = a.accumulate ? bf16_float(*o) + acc[i][j][x] : acc[i][j][x];
            *o = (uint16_t)float_bf16(v);
          }
        }
      }
  }
}

}  // namespace

hipError_t launch_loss_dz(const GradArgs& a, int grid, hipStream_t stream) {
  hipLaunchKernelGGL(k_loss_product<kDz>, dim3(grid), dim3(256), 0, stream, a);
  return hipGetLastError();
}
hipError_t launch_loss_d_hidden(const GradArgs& a, int grid, hipStream_t stream) {
  hipLaunchKernelGGL(k_loss_product<kDHidden>, dim3(grid), dim3(256), 0, stream, a);
  return hipGetLastError();
}
hipError_t launch_loss_d_W(const GradArgs& a, int grid, hipStream_t stream) {
  hipLaunchKernelGGL(k_loss_product<kDW>, dim3(grid), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace dllm

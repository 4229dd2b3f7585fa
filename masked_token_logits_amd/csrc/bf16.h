// bf16 words, and the host checks and workspaces shared by the rotary, norm,
// embedding and loss kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dllm {

__device__ __forceinline__ float bf16_float(uint32_t bits) { return __uint_as_float(bits << 16); }

// bf16 bits of x, nearest with ties to even; NaN stays NaN.
__device__ __forceinline__ uint32_t float_bf16(float x) {
  const __bf16 b = (__bf16)x;
  uint16_t u;
  __builtin_memcpy(&u, &b, 2);
  return u;
}

// Eight bf16 values of a 16-byte piece.
__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = float_bf16(f[2 * i]) | float_bf16(f[2 * i + 1]) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Whether n bytes at p and m bytes at q share any; a null pointer shares none.
inline bool overlaps(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return p && q && n && m && a < b + m && b < a + n;
}

// A workspace's parts, one behind another, each on 256 bytes; without a base only
// their size.
struct Parts {
  uint8_t* base;
  size_t size = 0;
  uint8_t* take(size_t bytes) {
    uint8_t* const p = base ? base + size : nullptr;
    size = (size + bytes + 255) / 256 * 256;
    return p;
  }
};

inline bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

}  // namespace dllm

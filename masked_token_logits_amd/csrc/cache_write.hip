// Write into the 8-bit block cache (include/dllm_cache.h): rotation of the
// keys, the blocks' scales, rounding to e4m3 and the cache's byte order.
#include "cache_common.h"
#include "rotary_angle.h"

namespace dllm {
namespace {

constexpr int kThreads = 256;

// Scale byte of a block whose largest magnitude is `big`: the smallest e with
// big <= 448 * 2^e, 448 = 1.75 * 2^8 being e4m3's largest value, read off
// big's exponent and mantissa.
__device__ __forceinline__ int scale_byte(float big) {
  const uint32_t u = __float_as_uint(fminf(big, 3.4028235e38f));
  if (u == 0) return 0;
  const int x = (int)(u >> 23) - 127;  // a subnormal counts as 2^-127: below every scale that is chosen
  return x - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0) + 127;
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.4028235e38f ? a : 0.0f;
}

// e4m3 value of byte b
__device__ __forceinline__ float e4m3_float(uint32_t b) {
  return __builtin_amdgcn_cvt_pk_f32_fp8((int)b, false)[0];
}

__device__ __forceinline__ uint32_t float_e4m3(float x) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, x, 0, false) & 0xffu;
}

// One workgroup: one touched block of one head.  Values pass through LDS as
// fp32 (rotated keys, values), because the cache's byte order of a block is
// not the order of the input rows.
template <int D>
__global__ __launch_bounds__(kThreads) void k_write(dllm_cache c, dllm_cache_batch b, int64_t T,
                                                    const uint16_t* __restrict__ k, int64_t k_token, int64_t k_head,
                                                    const uint16_t* __restrict__ v, int64_t v_token, int64_t v_head,
                                                    const int32_t* __restrict__ start,
                                                    const int32_t* __restrict__ positions, dllm_rotary_plan plan) {
  const int s = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  const SeqView q = seq_view(b, T, s);
  const int64_t st = start[s];
  if (st < 0 || q.rows == 0) return;
  const int64_t blk64 = st / kBlock + blockIdx.x;
  if (blk64 * kBlock >= st + q.rows || blk64 >= b.table_blocks) return;
  const int blk = (int)blk64;
  const int page = page_of(b.table, b.table_blocks, c.pages, s, blk);
  if (page < 0) return;
  const int64_t at = block_of(c, page, h);
  __shared__ float x[kBlock][D + 1];
  __shared__ float top[kThreads / 64];
  const int half = plan.turns ? plan.rotary_dim / 2 : 0;

  for (int side = 0; side < 2; ++side) {  // keys, then values
    const uint16_t* src = side ? v : k;
    const int64_t ts = side ? v_token : k_token, hs = side ? v_head : k_head;
    uint8_t* dst = (side ? c.v : c.k) + at * (kBlock * D);
    uint8_t* scale = (side ? c.v_scale : c.k_scale) + at;
    float big = 0.0f;
    bool held = false;
    __syncthreads();
    for (int u = tid; u < kBlock * D; u += kThreads) {
      const int t = u / D, d = u - t * D;
      const int64_t slot = (int64_t)blk * kBlock + t;
      float val = 0.0f;
      if (slot >= st && slot < st + q.rows) {
        val = bf16_float(src[(q.q0 + (slot - st)) * ts + (int64_t)h * hs + d]);
        big = fmaxf(big, finite_abs(val));
      } else if (slot < q.len) {
        held = true;
      }
      x[t][d] = val;
    }
    for (int o = 32; o; o >>= 1) big = fmaxf(big, __shfl_xor(big, o));
    if ((tid & 63) == 0) top[tid >> 6] = big;
    const int any_held = __syncthreads_or(held);
    big = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    if (side == 0 && half) big *= 1.41421366f * plan.magnitude;
    const int had = *scale;
    int byte = max(scale_byte(big), any_held ? had : 0);
    byte = min(max(byte, DLLM_CACHE_SCALE_MIN), DLLM_CACHE_SCALE_MAX);
    const float inv = __uint_as_float((uint32_t)(254 - byte) << 23);  // 2^(127 - byte); 2^-127 at the largest byte
    const float inv2 = byte == 254 ? __uint_as_float(0x00400000u) : inv;
    // 2^(had - byte): 0 where it underflows, as the requantised value then does
    const float old = had - byte < -126 ? 0.0f : __uint_as_float((uint32_t)(had - byte + 127) << 23);
    if (side == 0 && half) {
      // rotate the new rows in place, one pair at a time
      for (int u = tid; u < kBlock * half; u += kThreads) {
        const int t = u / half, i = u - t * half;
        const int64_t slot = (int64_t)blk * kBlock + t;
        if (slot < st || slot >= st + q.rows) continue;
        const double2 cs = rotary_angle64(positions[q.q0 + (slot - st)], plan.turns[i], plan.magnitude);
        const int a = plan.layout == DLLM_ROTARY_HALF ? i : 2 * i;
        const int e = plan.layout == DLLM_ROTARY_HALF ? i + half : 2 * i + 1;
        const double xa = x[t][a], xb = x[t][e];
        x[t][a] = odd_float(xa * cs.x - xb * cs.y);
        x[t][e] = odd_float(xb * cs.x + xa * cs.y);
      }
    }
    __syncthreads();
    // every byte of the block in the cache's order, 4 to a thread
    for (int u = tid * 4; u < kBlock * D; u += kThreads * 4) {
      const uint32_t prev = *reinterpret_cast<const uint32_t*>(dst + u);
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = u + j, cc = p >> 10, hh = (p >> 9) & 1, r = (p >> 4) & 31, e = p & 15;
        const int t = side ? 8 * (e >> 2) + 4 * hh + (e & 3) : r;
        const int d = side ? 32 * cc + r : hh * (D / 2) + 16 * cc + e;
        const int64_t slot = (int64_t)blk * kBlock + t;
        uint32_t byte8 = 0;
        if (slot >= st && slot < st + q.rows)
          byte8 = float_e4m3(x[t][d] * inv2);
        else if (slot < q.len)
          byte8 = float_e4m3(e4m3_float((prev >> (8 * j)) & 0xffu) * old);
        word |= byte8 << (8 * j);
      }
      *reinterpret_cast<uint32_t*>(dst + u) = word;
    }
    if (tid == 0) *scale = (uint8_t)byte;
  }
}

template <int D>
void launch_write(const dllm_cache& c, const dllm_cache_batch& b, int64_t T, const uint16_t* k, int64_t kt, int64_t kh,
                  const uint16_t* v, int64_t vt, int64_t vh, const int32_t* start, const int32_t* positions,
                  const dllm_rotary_plan& plan, hipStream_t st) {
  const int64_t most = b.max_new < T ? b.max_new : T;
  const int64_t blocks = (most + kBlock - 2) / kBlock + 1;  // a run of n tokens touches at most this many
  hipLaunchKernelGGL(k_write<D>, dim3((unsigned)blocks, c.kv_heads, b.S), dim3(kThreads), 0, st, c, b, T, k, kt, kh, v,
                     vt, vh, start, positions, plan);
}

}  // namespace
}  // namespace dllm

extern "C" dllm_status dllm_cache_write(const dllm_cache* cache, const dllm_cache_batch* batch, int64_t T,
                                        const uint16_t* k, int64_t k_token, int64_t k_head, const uint16_t* v,
                                        int64_t v_token, int64_t v_head, const int32_t* start,
                                        const int32_t* positions, const dllm_rotary_plan* plan, void* stream) {
  using namespace dllm;
  if (!cache_ok(cache) || !batch_ok(batch) || !tokens_ok(T)) return DLLM_ERR_INVALID_ARG;
  if (k_token < 0 || k_head < 0 || v_token < 0 || v_head < 0) return DLLM_ERR_INVALID_ARG;
  if (!cache_supported(cache)) return DLLM_ERR_UNSUPPORTED;
  if (plan && !rotary_plan_ok(plan, cache->head_dim)) return DLLM_ERR_INVALID_ARG;
  if (T == 0) return DLLM_OK;
  if (!k || !v || !start || (plan && !positions)) return DLLM_ERR_INVALID_ARG;
  if (!stride_ok(k_token) || !stride_ok(k_head) || !stride_ok(v_token) || !stride_ok(v_head)) return DLLM_ERR_UNSUPPORTED;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const dllm_rotary_plan none = {nullptr, 1.0f, 0, 0};
  const dllm_rotary_plan& p = plan ? *plan : none;
  const auto launch = cache->head_dim == 64 ? launch_write<64> : cache->head_dim == 128 ? launch_write<128> : launch_write<256>;
  launch(*cache, *batch, T, k, k_token, k_head, v, v_token, v_head, start, positions, p, st);
  return hipGetLastError() == hipSuccess ? DLLM_OK : DLLM_ERR_HIP;
}

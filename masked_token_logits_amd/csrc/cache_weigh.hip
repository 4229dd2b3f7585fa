// Accumulated attention weights of cached tokens (include/dllm_cache.h).
#include "cache_common.h"
#include "cache_tiles.h"

namespace dllm {
namespace {

struct WeighArgs {
  dllm_cache c;
  dllm_cache_batch b;
  int64_t T;
  const uint16_t* q;
  int64_t q_token, q_head;
  int q_heads, group;
  float scale2;
  int causal;
  const float* lse;
  float decay;
  float* weights;
};

// One wave: one block of one key/value head, against every query that may
// see it.  The block's keys are widened to bf16 (exact, scale included) once
// and stay in registers; queries come in as they are.
template <int D>
__global__ __launch_bounds__(64) void k_weigh(WeighArgs a) {
  const int s = blockIdx.z, h = blockIdx.y, blk = blockIdx.x, lane = threadIdx.x, col = lane & 31, half = lane >> 5;
  const SeqView q = seq_view(a.b, a.T, s);
  if ((int64_t)blk * kBlock >= q.len) return;
  const int page = page_of(a.b.table, a.b.table_blocks, a.c.pages, s, blk);
  if (page < 0) return;
  const int64_t at = block_of(a.c, page, h);
  const float ks = scale_value(a.c.k_scale[at]);
  Frag k[D / 16];
  const uint8_t* kp = a.c.k + at * (kBlock * D) + lane * 16;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    widen_keys(*reinterpret_cast<const i32x4*>(kp + i * 1024), ks, k[2 * i], k[2 * i + 1]);
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
  const int64_t rows = (int64_t)q.rows * a.group;
  for (int64_t row0 = 0; row0 < rows; row0 += 32) {
    const int64_t row = min(row0 + col, rows - 1);
    const int tok = (int)(row / a.group), head = h * a.group + (int)(row - (int64_t)tok * a.group);
    Frag qf[D / 16];
    load_query<D>(qf, a.q + (q.q0 + tok) * a.q_token + (int64_t)head * a.q_head, half);
    f32x16 sc = {};
#pragma unroll
    for (int i = 0; i < D / 16; ++i) sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[i].b, qf[i].b, sc, 0, 0, 0);
    float l = a.lse[(q.q0 + tok) * a.q_heads + head];
    if (row0 + col >= rows || l == -INFINITY) l = INFINITY;  // adds nothing
    const float ref = l * kLog2e;
    const int limit = (a.causal ? q.len - q.n + tok + 1 : q.len) - blk * kBlock;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i], a.scale2, -ref));
      acc[i] += token_of(i, half) < limit ? p : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    for (int o = 16; o; o >>= 1) acc[i] += __shfl_xor(acc[i], o);
  float* w = a.weights + ((int64_t)s * a.c.kv_heads + h) * ((int64_t)a.b.table_blocks * kBlock) + (int64_t)blk * kBlock;
  if (col == 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int t = token_of(i, half);
      if (blk * kBlock + t < q.len) w[t] = (a.decay == 0.0f ? 0.0f : a.decay * w[t]) + acc[i];
    }
  }
}

template <int D>
void launch(const WeighArgs& a, hipStream_t st) {
  const int blocks = (a.b.max_len + kBlock - 1) / kBlock;
  hipLaunchKernelGGL(k_weigh<D>, dim3(blocks, a.c.kv_heads, a.b.S), dim3(64), 0, st, a);
}

}  // namespace
}  // namespace dllm

extern "C" dllm_status dllm_cache_weigh(const dllm_cache* cache, const dllm_cache_batch* batch, int64_t T,
                                        const uint16_t* q, int64_t q_token, int64_t q_head, int32_t q_heads,
                                        float scale, int32_t causal, const float* lse, float decay, float* weights,
                                        void* stream) {
  using namespace dllm;
  if (!cache_ok(cache) || !batch_ok(batch) || !tokens_ok(T)) return DLLM_ERR_INVALID_ARG;
  if (q_heads < 1 || q_heads % cache->kv_heads != 0 || q_token < 0 || q_head < 0) return DLLM_ERR_INVALID_ARG;
  if (!(scale >= 1.17549435e-38f && scale <= 1.0e38f) || (causal != 0 && causal != 1)) return DLLM_ERR_INVALID_ARG;
  if (!(decay >= 0.0f && decay <= 1.0f) || !weights) return DLLM_ERR_INVALID_ARG;
  if (!cache_supported(cache) || q_heads > (1 << 16)) return DLLM_ERR_UNSUPPORTED;
  if (T > 0 && (!q || !lse)) return DLLM_ERR_INVALID_ARG;
  if (!stride_ok(q_token) || !stride_ok(q_head) || q_token % 8 != 0 || q_head % 8 != 0 || ((uintptr_t)q & 15u) != 0)
    return DLLM_ERR_UNSUPPORTED;
  const WeighArgs a = {*cache, *batch, T, q, q_token, q_head, q_heads, q_heads / cache->kv_heads, scale * kLog2e,
                       causal, lse, decay, weights};
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (cache->head_dim == 64) launch<64>(a, st);
  else if (cache->head_dim == 128) launch<128>(a, st);
  else launch<256>(a, st);
  return hipGetLastError() == hipSuccess ? DLLM_OK : DLLM_ERR_HIP;
}

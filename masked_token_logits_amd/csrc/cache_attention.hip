// Attention over the 8-bit block cache (include/dllm_cache.h).
#include "cache_common.h"
#include "cache_tiles.h"
#include "rotary_angle.h"

namespace dllm {
namespace {

struct AttendArgs {
  dllm_cache c;
  dllm_cache_batch b;
  int64_t T;
  const uint16_t* q;
  int64_t q_token, q_head;
  int q_heads, group;
  float scale2;
  int causal;
  uint16_t* out;
  float* lse;
};

// One wave: 32 query rows (row = token * group + head of the group) of one
// key/value head over the whole sequence.
template <int D>
__global__ __launch_bounds__(64) void k_attend(AttendArgs a) {
  const int s = blockIdx.z, h = blockIdx.y, lane = threadIdx.x, col = lane & 31, half = lane >> 5;
  const SeqView q = seq_view(a.b, a.T, s);
  const int64_t rows = (int64_t)q.rows * a.group;
  const int64_t row0 = (int64_t)blockIdx.x * 32;
  if (row0 >= rows) return;
  const int64_t row = min(row0 + col, rows - 1);
  const int tok = (int)(row / a.group), head = h * a.group + (int)(row - (int64_t)tok * a.group);
  Frag qf[D / 16];
  load_query<D>(qf, a.q + (q.q0 + tok) * a.q_token + (int64_t)head * a.q_head, half);
  // tokens that this column sees: [0, end); the whole tile: [0, most)
  const int end = a.causal ? min(max(q.len - q.n + tok + 1, 0), q.len) : q.len;
  const int last = (int)(min(row0 + 31, rows - 1) / a.group);
  const int most = a.causal ? min(max(q.len - q.n + last + 1, 0), q.len) : q.len;
  const int least = q.len - q.n + (int)(row0 / a.group) + 1;  // what the tile's first row sees
  const int blocks = (most + kBlock - 1) / kBlock;
  Accumulator<D> acc;
  clear(acc);
  for (int j = 0; j < blocks; ++j) {
    const int page = page_of(a.b.table, a.b.table_blocks, a.c.pages, s, j);
    if (page < 0) continue;
    const int64_t at = block_of(a.c, page, h);
    i32x4 raw[D / 32];
    const uint8_t* kp = a.c.k + at * (kBlock * D) + lane * 16;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) raw[i] = *reinterpret_cast<const i32x4*>(kp + i * 1024);
    f32x16 sc = scores<D>(qf, raw, scale_value(a.c.k_scale[at]));
#pragma unroll
    for (int i = 0; i < 16; ++i) sc[i] = token_of(i, half) < end - j * kBlock ? sc[i] : -INFINITY;
    cover<D>(acc, largest(sc), a.scale2);
    Frag p[2];
    probabilities<D>(acc, sc, a.scale2, p);
    const uint8_t* vp = a.c.v + at * (kBlock * D) + lane * 16;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      raw[i] = clip_values(*reinterpret_cast<const i32x4*>(vp + i * 1024), half, q.len - j * kBlock);
    const float vs = cover_values<D>(acc, a.c.v_scale[at]);
    if (a.causal && (j + 1) * kBlock > least)
      add_values_masked<D>(acc, p, raw, vs, end - j * kBlock, half);
    else
      add_values<D>(acc, p, raw, vs);
  }
  const float sum = acc.sum + other_half(acc.sum);
  if (row0 + col >= rows) return;
  const float inv = sum == 0.0f ? 0.0f : scale_value(acc.v_ref) / sum;
  const int64_t to = (q.q0 + tok) * a.q_heads + head;
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = float_bf16(acc.o[c][4 * i] * inv) | float_bf16(acc.o[c][4 * i + 1] * inv) << 16;
      const uint32_t hi = float_bf16(acc.o[c][4 * i + 2] * inv) | float_bf16(acc.o[c][4 * i + 3] * inv) << 16;
      *reinterpret_cast<uint2*>(a.out + to * D + 32 * c + 8 * i + 4 * half) = make_uint2(lo, hi);
    }
  if (a.lse && half == 0) a.lse[to] = sum == 0.0f ? -INFINITY : (acc.ref + __log2f(sum)) * kLn2;
}

template <int D>
void launch(const AttendArgs& a, hipStream_t st) {
  const int64_t most = (int64_t)(a.b.max_new < a.T ? a.b.max_new : a.T) * a.group;
  hipLaunchKernelGGL(k_attend<D>, dim3((unsigned)((most + 31) / 32), a.c.kv_heads, a.b.S), dim3(64), 0, st, a);
}

}  // namespace
}  // namespace dllm

extern "C" {

size_t dllm_cache_attention_workspace_bytes(const dllm_cache* cache, const dllm_cache_batch* batch, int32_t q_heads) {
  using namespace dllm;
  if (!cache_ok(cache) || !cache_supported(cache) || !batch_ok(batch) || q_heads < 1 || q_heads % cache->kv_heads != 0)
    return 0;
  return 256;
}

dllm_status dllm_cache_attention(const dllm_cache* cache, const dllm_cache_batch* batch, int64_t T, const uint16_t* q,
                                 int64_t q_token, int64_t q_head, int32_t q_heads, float scale, int32_t causal,
                                 uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace dllm;
  if (!cache_ok(cache) || !batch_ok(batch) || !tokens_ok(T)) return DLLM_ERR_INVALID_ARG;
  if (q_heads < 1 || q_heads % cache->kv_heads != 0 || q_token < 0 || q_head < 0) return DLLM_ERR_INVALID_ARG;
  if (!(scale >= 1.17549435e-38f && scale <= 1.0e38f) || (causal != 0 && causal != 1)) return DLLM_ERR_INVALID_ARG;
  if (!cache_supported(cache) || q_heads > (1 << 16)) return DLLM_ERR_UNSUPPORTED;
  if (T == 0) return DLLM_OK;
  if (!q || !out) return DLLM_ERR_INVALID_ARG;
  if (!stride_ok(q_token) || !stride_ok(q_head) || q_token % 8 != 0 || q_head % 8 != 0) return DLLM_ERR_UNSUPPORTED;
  if ((((uintptr_t)q | (uintptr_t)out) & 15u) != 0) return DLLM_ERR_UNSUPPORTED;
  const size_t need = dllm_cache_attention_workspace_bytes(cache, batch, q_heads);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u) != 0) return DLLM_ERR_WORKSPACE;
  const AttendArgs a = {*cache, *batch, T, q, q_token, q_head, q_heads, q_heads / cache->kv_heads, scale * kLog2e,
                        causal, out, lse};
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (cache->head_dim == 64) launch<64>(a, st);
  else if (cache->head_dim == 128) launch<128>(a, st);
  else launch<256>(a, st);
  return hipGetLastError() == hipSuccess ? DLLM_OK : DLLM_ERR_HIP;
}

}  // extern "C"

// Token embedding (include/dllm_embed.h): rows of a table looked up and
// scaled, and the table's gradient, the sum of the output's gradients over
// each token's places.
//
// The gradient goes by the tokens in sorted order (stable, so a token's places
// ascend): runs of equal tokens are cut into chunks of kChunk places, one wave
// to a chunk and 512 columns, which sums rows in fp32 in that order.  A run
// inside one chunk is written at once; the shares of one that spans chunks go
// to the workspace and a second kernel adds them, again in order.  So a token
// that is most of a batch, as the mask token is, is summed by as many waves as
// its places fill, and no result depends on timing.
#include "dllm_embed.h"

#include <math.h>

#include "bf16.h"

namespace dllm {
namespace {

constexpr int kChunk = 32;       // places of a chunk
constexpr int kCols = 512;       // columns of a wave: 64 lanes of 8
constexpr int kNoToken = 0x7FFFFFFF;  // sorts behind every token; its places have no row

__device__ __forceinline__ int known(int tok, int V) { return tok >= 0 && tok < V ? tok : kNoToken; }

__global__ __launch_bounds__(256) void k_embed(const uint16_t* __restrict__ table, int V, int d,
                                               const int32_t* __restrict__ tokens, int64_t T, float scale,
                                               uint16_t* __restrict__ out) {
  const int64_t pieces = d / 8, n = T * pieces;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / pieces, c = i - t * pieces;
    const int tok = known(tokens[t], V);
    uint4 u = make_uint4(0, 0, 0, 0);
    if (tok != kNoToken) {
      u = *reinterpret_cast<const uint4*>(table + (int64_t)tok * d + 8 * c);
      if (scale != 1.0f) {
        float f[8];
        unpack8(u, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= scale;
        u = pack8(f);
      }
    }
    *reinterpret_cast<uint4*>(out + t * d + 8 * c) = u;
  }
}

// A token's place in the sorted order is the number of tokens before it: the
// smaller ones, and the equal ones further up.  A wave counts for 64 tokens.
__global__ __launch_bounds__(64) void k_embed_rank(const int32_t* __restrict__ tokens, int T, int V,
                                                   int32_t* __restrict__ sorted, int32_t* __restrict__ place) {
  const int i = blockIdx.x * 64 + threadIdx.x;
  const int mine = i < T ? known(tokens[i], V) : kNoToken;
  int rank = 0;
  for (int base = 0; base < T; base += 64) {
    const int j0 = base + threadIdx.x;
    const int other = j0 < T ? known(tokens[j0], V) : kNoToken;
    const int n = min(64, T - base);
    for (int j = 0; j < n; ++j) {
      const int o = __builtin_amdgcn_readlane(other, j);
      rank += (o < mine || (o == mine && base + j < i)) ? 1 : 0;
    }
  }
  if (i < T) {
    sorted[rank] = mine;
    place[rank] = i;
  }
}

struct SumArgs {
  const int32_t *sorted, *place;
  int T, d;
  const uint16_t* d_out;
  float scale;
  int accumulate;
  uint16_t* d_table;
  float* part;  // [chunks][2][d]: a run that comes from the chunk before, and one that begins here and goes on
};

// The finished sum of 8 columns of a token's row.
__device__ __forceinline__ void finish(const SumArgs& a, int tok, int c, float* f) {
  uint16_t* o = a.d_table + (int64_t)tok * a.d + c;
  float old[8];
  if (a.accumulate) unpack8(*reinterpret_cast<const uint4*>(o), old);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = a.accumulate ? fmaf(f[j], a.scale, old[j]) : f[j] * a.scale;
  *reinterpret_cast<uint4*>(o) = pack8(f);
}

__global__ __launch_bounds__(64) void k_embed_sum(SumArgs a) {
  const int lane = threadIdx.x, begin = blockIdx.x * kChunk, n = min(kChunk, a.T - begin);
  const int c = blockIdx.y * kCols + lane * 8;
  const int at = begin + (lane < n ? lane : n - 1);
  const int tok = a.sorted[at], pl = a.place[at];
  const int before = begin > 0 ? a.sorted[begin - 1] : -1;
  const int behind = begin + n < a.T ? a.sorted[begin + n] : -1;
  const bool in = c < a.d;
  float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  int first = 0;  // where the run began
  for (int k = 0; k < n; ++k) {
    const int t = __builtin_amdgcn_readlane(tok, k), p = __builtin_amdgcn_readlane(pl, k);
    if (t == kNoToken) return;  // only those follow
    if (in) {
      float g[8];
      unpack8(*reinterpret_cast<const uint4*>(a.d_out + (int64_t)p * a.d + c), g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += g[j];
    }
    const int next = k + 1 < n ? __builtin_amdgcn_readlane(tok, k + 1) : behind;
    if (k + 1 < n && next == t) continue;
    const bool from = first == 0 && before == t, on = k + 1 == n && next == t;
    if (in) {
      if (!from && !on) {
        finish(a, t, c, f);
      } else {
        float* o = a.part + ((int64_t)blockIdx.x * 2 + (from ? 0 : 1)) * a.d + c;
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = f[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.f;
    first = k + 1;
  }
}

// The first place at or behind lo whose token is above tok.
__device__ __forceinline__ int upper(const int32_t* __restrict__ sorted, int lo, int T, int tok) {
  int hi = T;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (sorted[mid] <= tok)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

// Runs that span chunks, by the chunk in which they begin.  Sixteen waves take
// a sixteenth of the chunks each; a lane has 8 columns.
constexpr int kJoinWaves = 16, kJoinLanes = 64;

__global__ __launch_bounds__(kJoinWaves * kJoinLanes) void k_embed_join(SumArgs a) {
  __shared__ float lds[kJoinWaves][kJoinLanes][8];
  const int begin = blockIdx.x * kChunk, end = begin + kChunk;
  if (end >= a.T) return;  // nothing behind this chunk
  const int tok = a.sorted[end - 1];
  if (tok == kNoToken || a.sorted[end] != tok) return;
  if (a.sorted[begin] == tok && begin > 0 && a.sorted[begin - 1] == tok) return;  // it began further up
  const int last = (upper(a.sorted, end, a.T, tok) - 1) / kChunk;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.y * kCols + lane * 8;
  const int n = last - blockIdx.x + 1;
  const int lo = (int)((int64_t)n * wave / kJoinWaves), hi = (int)((int64_t)n * (wave + 1) / kJoinWaves);
  float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < a.d)
    for (int k = lo; k < hi; ++k) {
      const float* p = a.part + ((int64_t)(blockIdx.x + k) * 2 + (k == 0 ? 1 : 0)) * a.d + c;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += p[j];
    }
#pragma unroll
  for (int j = 0; j < 8; ++j) lds[wave][lane][j] = f[j];
  __syncthreads();
  if (wave == 0 && c < a.d) {
    for (int w = 1; w < kJoinWaves; ++w)
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += lds[w][lane][j];
    finish(a, tok, c, f);
  }
}

// Zeros for the rows of tokens that do not occur.
__global__ __launch_bounds__(256) void k_embed_clear(const int32_t* __restrict__ sorted, int T, int V, int d,
                                                     uint16_t* __restrict__ d_table) {
  for (int v = blockIdx.x; v < V; v += gridDim.x) {
    const int at = T > 0 ? upper(sorted, 0, T, v - 1) : 0;
    if (at < T && sorted[at] == v) continue;
    for (int c = threadIdx.x * 8; c < d; c += 256 * 8)
      *reinterpret_cast<uint4*>(d_table + (int64_t)v * d + c) = make_uint4(0, 0, 0, 0);
  }
}

bool sizes_ok(int64_t V, int64_t d, int64_t T) {
  return V >= 1 && V < ((int64_t)1 << 31) - 1 && d >= 1 && T >= 0 && T < ((int64_t)1 << 31) - 1024;
}
bool supported(int64_t d) { return d % 8 == 0 && d < ((int64_t)1 << 24); }

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

int64_t chunks_of(int64_t T) { return (T + kChunk - 1) / kChunk; }

}  // namespace
}  // namespace dllm

extern "C" {

dllm_status dllm_embed(const uint16_t* table, int64_t V, int64_t d, const int32_t* tokens, int64_t T, float scale,
                       uint16_t* out, void* stream) {
  if (!dllm::sizes_ok(V, d, T) || !isfinite(scale)) return DLLM_ERR_INVALID_ARG;
  if (!dllm::supported(d)) return DLLM_ERR_UNSUPPORTED;
  if (T == 0) return DLLM_OK;
  if (!table || !tokens || !out) return DLLM_ERR_INVALID_ARG;
  if (!dllm::aligned(table, 16) || !dllm::aligned(out, 16) || !dllm::aligned(tokens, 4)) return DLLM_ERR_UNSUPPORTED;
  const size_t n = (size_t)T * (size_t)d * 2;
  if (dllm::overlaps(out, n, table, (size_t)V * (size_t)d * 2) || dllm::overlaps(out, n, tokens, (size_t)T * 4))
    return DLLM_ERR_INVALID_ARG;
  const int64_t groups = (T * (d / 8) + 255) / 256;
  hipLaunchKernelGGL(dllm::k_embed, dim3((unsigned)(groups < (1 << 20) ? groups : 1 << 20)), dim3(256), 0,
                     reinterpret_cast<hipStream_t>(stream), table, (int)V, (int)d, tokens, T, scale, out);
  return hipGetLastError() == hipSuccess ? DLLM_OK : DLLM_ERR_HIP;
}

size_t dllm_embed_backward_workspace_bytes(int64_t V, int64_t d, int64_t T) {
  if (!dllm::sizes_ok(V, d, T) || !dllm::supported(d)) return 0;
  return 256 + 2 * dllm::up256((size_t)T * 4) + dllm::up256((size_t)dllm::chunks_of(T) * 2 * (size_t)d * 4);
}

dllm_status dllm_embed_backward(const int32_t* tokens, int64_t T, const uint16_t* d_out, int64_t V, int64_t d,
                                float scale, int32_t accumulate, uint16_t* d_table, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!dllm::sizes_ok(V, d, T) || !isfinite(scale) || (accumulate != 0 && accumulate != 1)) return DLLM_ERR_INVALID_ARG;
  if (!dllm::supported(d)) return DLLM_ERR_UNSUPPORTED;
  if (!d_table || (T > 0 && (!tokens || !d_out))) return DLLM_ERR_INVALID_ARG;
  if (!dllm::aligned(d_table, 16) || !dllm::aligned(d_out, 16) || !dllm::aligned(tokens, 4)) return DLLM_ERR_UNSUPPORTED;
  const size_t need = dllm_embed_backward_workspace_bytes(V, d, T), n = (size_t)V * (size_t)d * 2;
  if (!workspace || workspace_bytes < need || !dllm::aligned(workspace, 256)) return DLLM_ERR_WORKSPACE;
  if (dllm::overlaps(d_table, n, d_out, (size_t)T * (size_t)d * 2) || dllm::overlaps(d_table, n, tokens, (size_t)T * 4) ||
      dllm::overlaps(d_table, n, workspace, need))
    return DLLM_ERR_INVALID_ARG;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  uint8_t* w = reinterpret_cast<uint8_t*>(workspace);
  int32_t* sorted = reinterpret_cast<int32_t*>(w);
  int32_t* place = reinterpret_cast<int32_t*>(w + dllm::up256((size_t)T * 4));
  float* part = reinterpret_cast<float*>(w + 2 * dllm::up256((size_t)T * 4));
  if (T > 0)
    hipLaunchKernelGGL(dllm::k_embed_rank, dim3((unsigned)((T + 63) / 64)), dim3(64), 0, st, tokens, (int)T, (int)V,
                       sorted, place);
  if (!accumulate)
    hipLaunchKernelGGL(dllm::k_embed_clear, dim3((unsigned)(V < (1 << 18) ? V : 1 << 18)), dim3(256), 0, st, sorted,
                       (int)T, (int)V, (int)d, d_table);
  if (T > 0) {
    const dllm::SumArgs a = {sorted, place, (int)T, (int)d, d_out, scale, accumulate, d_table, part};
    const dim3 grid((unsigned)dllm::chunks_of(T), (unsigned)((d + dllm::kCols - 1) / dllm::kCols));
    hipLaunchKernelGGL(dllm::k_embed_sum, grid, dim3(64), 0, st, a);
    hipLaunchKernelGGL(dllm::k_embed_join, grid, dim3(dllm::kJoinWaves * dllm::kJoinLanes), 0, st, a);
  }
  return hipGetLastError() == hipSuccess ? DLLM_OK : DLLM_ERR_HIP;
}

}  // extern "C"

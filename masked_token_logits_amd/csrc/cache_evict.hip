// Eviction from the 8-bit block cache by accumulated attention weight
// (include/dllm_cache.h): selection of the kept tokens and their move.
#include "cache_common.h"

namespace dllm {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kMoveThreads = 256;

struct SelectArgs {
  const int32_t* lens;
  int max_len;
  int kv_heads;
  const float* weights;
  int64_t slots;  // of a row of weights
  const int32_t* keep;
  int max_keep, sink, recent, pool;
  int32_t* lens_out;
  int32_t* kept;
  float* weights_out;
  int64_t out_slots;
};

// Order-preserving bits of a weight: a > b as floats iff key(a) > key(b);
// -0 and 0 are equal, NaN is the lowest.
__device__ __forceinline__ uint32_t order_key(float w) {
  w = w != w ? -INFINITY : w + 0.0f;
  const uint32_t u = __float_as_uint(w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t pooled_key(const float* __restrict__ w, int j, int len, int reach) {
  uint32_t key = 0;
  for (int i = max(j - reach, 0); i <= min(j + reach, len - 1); ++i) key = max(key, order_key(w[i]));
  return key;
}

// One workgroup: the kept tokens of one sequence and head.  Four 8-bit radix
// passes find the m-th largest pooled key and how many equal to it are taken;
// a last pass writes the kept tokens in order.
__global__ __launch_bounds__(kSelectThreads) void k_select(SelectArgs a) {
  const int s = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int len = min(max(a.lens[s], 0), a.max_len);
  const int n = min(min(max(a.keep[s], 0), a.max_keep), len);
  const int first = min(a.sink, n), last = min(a.recent, n - first), m = n - first - last;
  const int lo = first, hi = len - last;  // the tokens between
  const float* w = a.weights + ((int64_t)s * a.kv_heads + h) * a.slots;
  const int reach = a.pool / 2;
  if (h == 0 && tid == 0) a.lens_out[s] = n;
  __shared__ uint32_t hist[256];
  __shared__ uint32_t prefix_s, want_s;
  __shared__ int gt[kSelectThreads / 64], eq[kSelectThreads / 64];
  uint32_t prefix = 0, mask = 0, want = (uint32_t)m;
  if (m > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
      for (int j = lo + tid; j < hi; j += kSelectThreads) {
        const uint32_t key = pooled_key(w, j, len, reach);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t left = want;
        int d = 255;
        for (; d > 0 && hist[d] < left; --d) left -= hist[d];
        prefix_s = prefix | (uint32_t)d << shift;
        want_s = left;
      }
      __syncthreads();
      prefix = prefix_s;
      want = want_s;
      mask |= 255u << shift;
    }
  }
  // wave w takes a contiguous run of the tokens between, so that its places
  // follow from the counts of the waves before it
  const int waves = kSelectThreads / 64;
  const int run = ((hi - lo + waves - 1) / waves + 63) / 64 * 64;
  const int b0 = lo + wave * run, b1 = min(b0 + run, hi);
  int n_gt = 0, n_eq = 0;
  if (m > 0)
    for (int j0 = b0; j0 < b1; j0 += 64) {
      const int j = j0 + lane;
      const uint32_t key = j < b1 ? pooled_key(w, j, len, reach) : 0;
      n_gt += __popcll(__ballot(j < b1 && key > prefix));
      n_eq += __popcll(__ballot(j < b1 && key == prefix));
    }
  if (lane == 0) gt[wave] = n_gt, eq[wave] = n_eq;
  __syncthreads();
  int32_t* kept = a.kept + ((int64_t)s * a.kv_heads + h) * a.max_keep;
  float* wo = a.weights_out ? a.weights_out + ((int64_t)s * a.kv_heads + h) * a.out_slots : nullptr;
  auto put = [&](int place, int j) {
    kept[place] = j;
    if (wo) wo[place] = w[j];
  };
  for (int j = tid; j < first; j += kSelectThreads) put(j, j);
  for (int j = tid; j < last; j += kSelectThreads) put(n - last + j, len - last + j);
  if (m > 0) {
    int eq_before = 0, place = first;
    for (int i = 0; i < wave; ++i) {
      place += gt[i] + min(eq[i], max((int)want - eq_before, 0));
      eq_before += eq[i];
    }
    for (int j0 = b0; j0 < b1; j0 += 64) {
      const int j = j0 + lane;
      const uint32_t key = j < b1 ? pooled_key(w, j, len, reach) : 0;
      const bool same = j < b1 && key == prefix;
      const uint64_t below = (1ull << lane) - 1, sames = __ballot(same);
      const bool take = (j < b1 && key > prefix) || (same && eq_before + __popcll(sames & below) < (int)want);
      const uint64_t takes = __ballot(take);
      if (take) put(place + __popcll(takes & below), j);
      place += __popcll(takes);
      eq_before += __popcll(sames);
    }
  }
}

struct MoveArgs {
  dllm_cache c;
  const int32_t* table;
  int table_blocks;
  const int32_t* table_out;
  int out_blocks;
  const int32_t* lens_out;
  const int32_t* kept;
  int max_keep;
};

// e4m3 byte b at a scale 2^(down) times larger
__device__ __forceinline__ uint32_t rescaled(uint32_t b, float down) {
  const float x = __builtin_amdgcn_cvt_pk_f32_fp8((int)b, false)[0] * down;
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, x, 0, false) & 0xffu;
}

// One workgroup: one new block of one head, gathered from its tokens' old
// places.
template <int D>
__global__ __launch_bounds__(kMoveThreads) void k_move(MoveArgs a) {
  const int s = blockIdx.z, h = blockIdx.y, blk = blockIdx.x, tid = threadIdx.x;
  const int n = a.lens_out[s];
  if (blk * kBlock >= n) return;
  const int to = page_of(a.table_out, a.out_blocks, a.c.pages, s, blk);
  if (to < 0) return;
  __shared__ int64_t src[kBlock];  // the token's old block, -1: none
  __shared__ int slot[kBlock];
  __shared__ int ke[kBlock], ve[kBlock];
  __shared__ int kmax, vmax;
  if (tid < kBlock) {
    const int t = blk * kBlock + tid;
    int64_t at = -1;
    if (t < n) {
      const int j = a.kept[((int64_t)s * a.c.kv_heads + h) * a.max_keep + t];
      const int page = page_of(a.table, a.table_blocks, a.c.pages, s, j / kBlock);
      if (page >= 0) at = block_of(a.c, page, h);
      slot[tid] = j % kBlock;
    } else {
      slot[tid] = 0;
    }
    src[tid] = at;
    int k = at >= 0 ? a.c.k_scale[at] : 0, v = at >= 0 ? a.c.v_scale[at] : 0;
    ke[tid] = k, ve[tid] = v;
    for (int o = 16; o; o >>= 1) {
      k = max(k, __shfl_xor(k, o));
      v = max(v, __shfl_xor(v, o));
    }
    if (tid == 0) kmax = max(k, DLLM_CACHE_SCALE_MIN), vmax = max(v, DLLM_CACHE_SCALE_MIN);
  }
  __syncthreads();
  const int64_t dst = block_of(a.c, to, h);
  for (int side = 0; side < 2; ++side) {
    const uint8_t* from = side ? a.c.v : a.c.k;
    uint8_t* out = (side ? a.c.v : a.c.k) + dst * (kBlock * D);
    const int top = side ? vmax : kmax;
    for (int u = tid * 4; u < kBlock * D; u += kMoveThreads * 4) {
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = u + j, hh = (p >> 9) & 1, r = (p >> 4) & 31, e = p & 15;
        const int t = side ? 8 * (e >> 2) + 4 * hh + (e & 3) : r;
        if (src[t] < 0) continue;
        const int o = slot[t];
        const int q = side ? (p & ~0x20f) | ((o >> 2) & 1) << 9 | (o >> 3) << 2 | (o & 3) : (p & ~0x1f0) | o << 4;
        uint32_t b = from[src[t] * (kBlock * D) + q];
        const int down = (side ? ve[t] : ke[t]) - top;
        if (down) b = rescaled(b, down < -126 ? 0.0f : __uint_as_float((uint32_t)(down + 127) << 23));
        word |= b << (8 * j);
      }
      *reinterpret_cast<uint32_t*>(out + u) = word;
    }
    if (tid == 0) (side ? a.c.v_scale : a.c.k_scale)[dst] = (uint8_t)top;
  }
}

}  // namespace
}  // namespace dllm

extern "C" {

size_t dllm_cache_evict_workspace_bytes(const dllm_cache* cache, const dllm_cache_batch* batch) {
  using namespace dllm;
  if (!cache_ok(cache) || !cache_supported(cache) || !batch_ok(batch)) return 0;
  return 256;
}

dllm_status dllm_cache_evict(const dllm_cache* cache, const dllm_cache_batch* batch, const float* weights,
                             const int32_t* keep, int32_t max_keep, int32_t sink, int32_t recent, int32_t pool,
                             const int32_t* table_out, int32_t out_blocks, int32_t* lens_out, int32_t* kept,
                             float* weights_out, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace dllm;
  if (!cache_ok(cache) || !batch_ok(batch)) return DLLM_ERR_INVALID_ARG;
  if (!weights || !keep || !table_out || !lens_out || !kept) return DLLM_ERR_INVALID_ARG;
  if (sink < 0 || recent < 0 || pool < 1 || pool > 63 || pool % 2 == 0) return DLLM_ERR_INVALID_ARG;
  if (out_blocks < 1 || out_blocks >= (1 << 26) || max_keep < 1 || (int64_t)max_keep > (int64_t)out_blocks * kBlock)
    return DLLM_ERR_INVALID_ARG;
  if (weights_out == weights || lens_out == batch->lens || lens_out == keep || table_out == batch->table)
    return DLLM_ERR_INVALID_ARG;
  if (!cache_supported(cache)) return DLLM_ERR_UNSUPPORTED;
  const size_t need = dllm_cache_evict_workspace_bytes(cache, batch);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u) != 0) return DLLM_ERR_WORKSPACE;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const SelectArgs sa = {batch->lens, batch->max_len, cache->kv_heads, weights, (int64_t)batch->table_blocks * kBlock,
                         keep, max_keep, sink, recent, pool, lens_out, kept, weights_out, (int64_t)out_blocks * kBlock};
  hipLaunchKernelGGL(k_select, dim3(cache->kv_heads, batch->S), dim3(kSelectThreads), 0, st, sa);
  if (hipGetLastError() != hipSuccess) return DLLM_ERR_HIP;
  const MoveArgs ma = {*cache, batch->table, batch->table_blocks, table_out, out_blocks, lens_out, kept, max_keep};
  const int most = max_keep < batch->max_len ? max_keep : batch->max_len;
  const dim3 grid((most + kBlock - 1) / kBlock, cache->kv_heads, batch->S);
  if (cache->head_dim == 64) hipLaunchKernelGGL(k_move<64>, grid, dim3(kMoveThreads), 0, st, ma);
  else if (cache->head_dim == 128) hipLaunchKernelGGL(k_move<128>, grid, dim3(kMoveThreads), 0, st, ma);
  else hipLaunchKernelGGL(k_move<256>, grid, dim3(kMoveThreads), 0, st, ma);
  return hipGetLastError() == hipSuccess ? DLLM_OK : DLLM_ERR_HIP;
}

}  // extern "C"

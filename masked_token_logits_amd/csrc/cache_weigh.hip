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

#define LDS_AS __attribute__((address_space(3)))

constexpr int kThreads = 256, kWaves = kThreads / 64;

// 16 values of every lane summed over the 32 lanes of its half: lane l of a
// half ends with the sum of value l / 2.  Each round halves the values and
// doubles the lanes that a sum covers.
__device__ __forceinline__ float sum_columns(float* x) {
  const int lane = threadIdx.x & 31;
  each<0, 4>([&](auto R) {
    constexpr int n = 8 >> decltype(R)::value, bit = 2 * n;
    const bool upper = lane & bit;
    each<0, n>([&](auto I) {
      constexpr int i = decltype(I)::value;
      const float keep = upper ? x[i + n] : x[i], give = upper ? x[i] : x[i + n];
      x[i] = keep + __shfl_xor(give, bit);
    });
  });
  return x[0] + __shfl_xor(x[0], 1);
}

// One workgroup: KW x NB blocks of 32 tokens of one key/value head, against
// every query that may see them.  A wave widens the keys of its NB blocks to
// bf16 once (exact, scale included) and keeps them in registers; query rows
// (token * group + head of the group) come in tiles of 32 through LDS, in the
// order in which the matrix instruction takes them, a step or two ahead.  KW waves
// share a tile for different blocks; with KW = 1 the four waves take different
// tiles of the same blocks and are summed at the end, which makes four times as
// many workgroups where there are few blocks.
template <int D, int NB, int KW>
__global__ __launch_bounds__(kThreads, 2) void k_weigh(WeighArgs a) {
  constexpr int RW = kWaves / KW, CH = D / 16;           // tiles of a step; 1 KiB chunks of a tile
  constexpr int kStep = RW * CH * 1024, kLoads = RW * CH / kWaves;  // bytes; loads of a wave
  constexpr int kRing = KW == 1 ? 2 : 3;                            // steps in LDS
  __shared__ __attribute__((aligned(1024))) uint8_t ring[kRing * kStep];
  const int s = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), kw = wave % KW, rw = wave / KW;
  const SeqView q = seq_view(a.b, a.T, s);
  // Early tokens are seen by more rows than late ones: every other 256
  // workgroups go through the blocks backwards, so that a compute unit's workgroups
  // come out alike.
  const bool backwards = a.causal && (((blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x) >> 8 & 1);
  const int first = (int)(backwards ? gridDim.x - 1 - blockIdx.x : blockIdx.x) * KW * NB;  // the workgroup's first block
  if ((int64_t)first * kBlock >= q.len) return;
  const int rows = q.rows * a.group;
  // a query sees tokens below len - n + its number + 1; rows before r0 see none of these
  const int before = q.len - q.n;
  const int64_t skip = a.causal ? (int64_t)max(first * kBlock - before, 0) * a.group : 0;
  const int tile0 = (int)min(skip, (int64_t)rows) / 32, steps = ((rows + 31) / 32 - tile0 + RW - 1) / RW;
  Frag k[NB][D / 16];
  int block[NB], limit[NB];  // number; its first token, counted from len - n
  bool ok[NB];
  each<0, NB>([&](auto N) {
    constexpr int b = decltype(N)::value;
    block[b] = first + kw * NB + b;
    const int page = (int64_t)block[b] * kBlock < q.len ? page_of(a.b.table, a.b.table_blocks, a.c.pages, s, block[b]) : -1;
    ok[b] = page >= 0;
    limit[b] = block[b] * kBlock - before;
    const int64_t at = block_of(a.c, max(page, 0), h);
    const float scale = scale_value(a.c.k_scale[at]);
    const uint8_t* p = a.c.k + at * (kBlock * D) + lane * 16;
    each<0, D / 32>([&](auto C) {
      constexpr int c = decltype(C)::value;
      widen_keys(*reinterpret_cast<const i32x4*>(p + c * 1024), scale, k[b][2 * c], k[b][2 * c + 1]);
    });
  });
  float acc[NB][16];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[b][i] = 0.0f;
  // Step t's row of this lane: the one whose queries it loads is also its column.
  static_assert(KW == 1 || KW == kWaves, "a wave loads queries of its own tile");
  struct Place {
    int row, tok, head;
  };
  auto place = [&](int t) {
    const int row = (tile0 + t * RW + rw) * 32 + col, real = min(row, rows - 1);
    const int tok = (int)((uint32_t)real / (uint32_t)a.group);
    return Place{row, tok, h * a.group + (real - tok * a.group)};
  };
  // The wave's share of a step's queries: kLoads chunks of its tile.
  auto load_step = [&](int t, const Place& p) {
    const uint16_t* src = a.q + (q.q0 + p.tok) * a.q_token + (int64_t)p.head * a.q_head + half * (D / 2);
    each<0, kLoads>([&](auto L) {
      const int x = wave * kLoads + decltype(L)::value;
      __builtin_amdgcn_global_load_lds((const void*)(src + x % CH * 8), (LDS_AS void*)(ring + (t % kRing) * kStep + x * 1024), 16,
                                       0, 0);
    });
  };
  // -lse of a row in base 2; -inf where it adds nothing
  auto negative_lse = [&](const Place& p) {
    const float l = a.lse[(q.q0 + p.tok) * a.q_heads + p.head];
    return p.row < rows && l != -INFINITY ? -l * kLog2e : -INFINITY;
  };
  if (steps > 0) {
    Place at[kRing];  // of steps t, t + 1, ...; behind the last step rows repeat, and add nothing
    each<0, kRing - 1>([&](auto t) {
      at[decltype(t)::value] = place(decltype(t)::value);
      load_step(decltype(t)::value, at[decltype(t)::value]);
    });
    float neg = negative_lse(at[0]);
    for (int t = 0; t < steps; ++t) {
      at[kRing - 1] = place(t + kRing - 1);
      const float neg_next = negative_lse(at[1]);
      asm volatile("" ::: "memory");
      // step t is in: only the loads of later ones and an lse may still be on their way
      __builtin_amdgcn_s_waitcnt((((kRing - 2) * kLoads + 1) & 15) | (7 << 4) | (0 << 8));
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      load_step(t + kRing - 1, at[kRing - 1]);  // where step t - 1 was
      const uint8_t* tile = ring + (t % kRing) * kStep + rw * CH * 1024 + lane * 16;
      f32x16 sc[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) sc[b] = f32x16{};
      each<0, CH>([&](auto C) {
        Frag f;
        f.w = *reinterpret_cast<const i32x4*>(tile + decltype(C)::value * 1024);
        each<0, NB>([&](auto N) {
          constexpr int b = decltype(N)::value;
          sc[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[b][decltype(C)::value].b, f.b, sc[b], 0, 0, 0);
        });
      });
      // columns of this tile that see a block only in part
      const int first_tok = (int)((uint32_t)min((tile0 + t * RW + rw) * 32, rows - 1) / (uint32_t)a.group);
      each<0, NB>([&](auto N) {
        constexpr int b = decltype(N)::value;
        if (a.causal && limit[b] + kBlock > first_tok + 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i) sc[b][i] = limit[b] + token_of(i, half) <= at[0].tok ? sc[b][i] : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[b][i] += __builtin_amdgcn_exp2f(__builtin_fmaf(sc[b][i], a.scale2, neg));
      });
      neg = neg_next;
      each<0, kRing - 1>([&](auto i) { at[decltype(i)::value] = at[decltype(i)::value + 1]; });
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
  float* w = a.weights + ((int64_t)s * a.c.kv_heads + h) * ((int64_t)a.b.table_blocks * kBlock);
  float* sums = reinterpret_cast<float*>(ring);
  each<0, NB>([&](auto N) {
    constexpr int b = decltype(N)::value;
    float sum = sum_columns(acc[b]);
    const int i = col >> 1, token = block[b] * kBlock + token_of(i, half);
    if constexpr (RW > 1) {
      if ((col & 1) == 0) sums[(rw * NB + b) * kBlock + token_of(i, half)] = sum;
      __syncthreads();
      if (rw == 0)
        for (int x = 1; x < RW; ++x) sum += sums[(x * NB + b) * kBlock + token_of(i, half)];
    }
    if (rw == 0 && (col & 1) == 0 && ok[b] && token < q.len)
      w[token] = (a.decay == 0.0f ? 0.0f : a.decay * w[token]) + sum;
  });
}

template <int D>
void launch(const WeighArgs& a, hipStream_t st) {
  constexpr int NB = D == 256 ? 1 : 2;
  const int blocks = (a.b.max_len + kBlock - 1) / kBlock;
  const int64_t wide = (int64_t)((blocks + kWaves * NB - 1) / (kWaves * NB)) * a.c.kv_heads * a.b.S;
  if (wide >= 512)
    hipLaunchKernelGGL((k_weigh<D, NB, kWaves>), dim3((blocks + kWaves * NB - 1) / (kWaves * NB), a.c.kv_heads, a.b.S),
                       dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL((k_weigh<D, NB, 1>), dim3((blocks + NB - 1) / NB, a.c.kv_heads, a.b.S), dim3(kThreads), 0, st, a);
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
  if (!cache_supported(cache) || T * (int64_t)q_heads >= ((int64_t)1 << 31) - 1024) return DLLM_ERR_UNSUPPORTED;
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

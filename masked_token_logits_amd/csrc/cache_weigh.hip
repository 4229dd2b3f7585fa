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
  uint32_t magic;  // row / group = high word of row * magic >> shift; 0: group is 1
  int shift;
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

// weights[token] = decay weights[token] + sum over queries of exp(scale q.k - lse): the
// scores of attention again, without their maximum, for lse is known.
//
// One workgroup: KW x 2 blocks of 32 tokens of one key/value head, against
// every query that may see them.  A wave widens the keys of its two blocks to
// bf16 once (exact, scale included) and keeps them in registers; query rows
// (token * group + head of the group) pass in tiles of 32 through LDS, a step or two
// ahead of their products.  With KW = 4 the waves share a tile for different blocks;
// with KW = 1 they take different tiles of the same blocks and are summed at the
// end, which makes four times as many workgroups where there are few blocks.
//
// Bound by the vector unit: 16 cycles for a score's fused multiply-add, exponential
// and sum, next to 32 x 32 of them in CH matrix instructions of 32 cycles.  4096
// causal queries of 32 heads of 128: 94 us (730 TFLOP/s), of which about 110 thousand
// of 195 thousand cycles are vector instructions and 68 thousand matrix ones.  Queries in
// 16-byte pieces straight from their rows kept the address unit as busy (104 us);
// exponentials of one tile woven between the products of the next gained nothing (99).
template <int D, int KW>
__global__ __launch_bounds__(kThreads, 2) void k_weigh(WeighArgs a) {
  constexpr int NB = 2;                             // blocks of a wave
  constexpr int RW = kWaves / KW, CH = D / 16;      // waves of different tiles; 1 KiB chunks of a tile
  constexpr int TW = KW > 1 && D <= 128 ? 2 : 1;    // tiles of a wave in a step
  constexpr int kRows = 32 * TW * RW;               // of a step
  constexpr int kChunks = TW * RW * CH / kWaves, kLoads = kChunks + 1;  // of a wave; its loads: these and an lse
  constexpr int kStep = kRows * (2 * D + 4);                            // bytes
  constexpr int kRing = KW == 1 || D == 256 ? 2 : 3;                    // steps in LDS
  __shared__ __attribute__((aligned(1024))) uint8_t ring[kRing * kStep];
  const int s = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), kw = wave % KW, rw = wave / KW;
  const SeqView q = seq_view(a.b, a.T, s);
  // Early tokens are seen by more rows than late ones under a causal mask: a wave
  // takes blocks from both ends, and all workgroups have the same work.
  const int blocks = (q.len + kBlock - 1) / kBlock, first = blockIdx.x * KW;  // the workgroup's first block
  if (first * NB >= blocks) return;
  const int rows = q.rows * a.group;
  // a query sees tokens below len - n + its number + 1; rows before see none of these
  const int before = q.len - q.n;
  auto tile_of = [&](int block) {
    const int64_t skip = a.causal ? (int64_t)max(block * kBlock - before, 0) * a.group : 0;
    return (int)min(skip, (int64_t)rows) / 32;
  };
  const int row0 = tile_of(first) * 32, steps = (rows - row0 + kRows - 1) / kRows;
  const int lone = (tile_of(max(blocks - first - KW, first)) * 32 - row0) / kRows;  // steps before the late blocks are seen
  Frag k[NB][D / 16];
  int block[NB], limit[NB];  // number; its first token, counted from len - n
  bool ok[NB];
  each<0, NB>([&](auto N) {
    constexpr int b = decltype(N)::value;
    block[b] = b == 0 ? first + kw : blocks - 1 - first - kw;
    const int page = (b == 0 ? block[b] * NB < blocks : block[b] > first + kw) ? page_of(a.b.table, a.b.table_blocks, a.c.pages, s, block[b]) : -1;
    ok[b] = page >= 0;
    limit[b] = block[b] * kBlock - before;
    const int64_t at = block_of(a.c, max(page, 0), h);
    const float scale = scale_value(stored_scale(a.c.k_scale, at));
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
  auto token_of_row = [&](int row) { return a.magic ? (int)(__umulhi((uint32_t)row, a.magic) >> a.shift) : row; };
  // The wave's share of a step's queries and of their lse.  A load takes 1 KiB of
  // whole rows, so that its lanes read whole lines; each lane finds one row's place and
  // hands it to the lanes that load it.  In a row's place in LDS its 16-byte units are
  // swapped by the row's number, so that lanes that read the same unit of 32 rows meet
  // in no bank.
  constexpr int kUnits = D / 8, kSwap = kUnits < 16 ? kUnits - 1 : 15, kPer = 64 / kUnits;  // kPer: rows of a load
  const int from = (KW == 1 ? 0 : wave * kChunks * kPer) + lane / kUnits;
  const int own = KW == 1 ? rw * 32 + col : lane % kRows;  // row of a step that this lane finds
  auto load_step = [&](int t) {
    uint8_t* to = ring + (t % kRing) * kStep;
    const int row = min(row0 + t * kRows + own, rows - 1);  // behind the last row it repeats, and adds nothing
    const int tok = token_of_row(row), head = h * a.group + (row - tok * a.group);
    const uint64_t src = (uint64_t)(a.q + (q.q0 + tok) * a.q_token + (int64_t)head * a.q_head);
    each<0, kChunks>([&](auto L) {
      constexpr int l = decltype(L)::value;
      const uint32_t lo = __shfl((uint32_t)src, from + l * kPer), hi = __shfl((uint32_t)(src >> 32), from + l * kPer);
      const uint32_t unit = (lane % kUnits) ^ ((from + l * kPer) & kSwap);
      __builtin_amdgcn_global_load_lds((const void*)((((uint64_t)hi << 32) | lo) + unit * 16),
                                       (LDS_AS void*)(to + (wave * kChunks + l) * 1024), 16, 0, 0);
    });
    if (lane * KW / (32 * TW) == kw)
      __builtin_amdgcn_global_load_lds((const void*)(a.lse + (q.q0 + tok) * a.q_heads + head),
                                       (LDS_AS void*)(to + kRows * 2 * D + rw * 128), 4, 0, 0);
  };
  if (steps > 0) {
    each<0, kRing - 1>([&](auto t) { load_step(decltype(t)::value); });
    // Tiles j to j + M of the wave's in step t, with its first N blocks
    auto scores = [&](int t, int j, auto m, auto n) {
      constexpr int M = decltype(m)::value, N = decltype(n)::value;
      const uint8_t* slot = ring + (t % kRing) * kStep;
      const int tile = rw * TW + j;
      f32x16 sc[M][N];
#pragma unroll
      for (int i = 0; i < M; ++i)
#pragma unroll
        for (int b = 0; b < N; ++b) sc[i][b] = f32x16{};
      each<0, CH>([&](auto C) {
        constexpr int c = decltype(C)::value;
        each<0, M>([&](auto I) {
          constexpr int i = decltype(I)::value;
          Frag f;
          f.w = *reinterpret_cast<const i32x4*>(slot + ((tile + i) * 32 + col) * (2 * D) +
                                                ((half * (kUnits / 2) + c) ^ (col & kSwap)) * 16);
          each<0, N>([&](auto B) {
            constexpr int b = decltype(B)::value;
            sc[i][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[b][c].b, f.b, sc[i][b], 0, 0, 0);
          });
        });
      });
      each<0, M>([&](auto I) {
        constexpr int i = decltype(I)::value;
        const int at = row0 + t * kRows + (tile + i) * 32, row = at + col;
        const float lse = reinterpret_cast<const float*>(slot + kRows * 2 * D)[(tile + i) * 32 + col];
        float neg = row < rows && lse != -INFINITY ? -lse * kLog2e : -INFINITY;  // -inf where it adds nothing
        const int first_tok = token_of_row(min(at, rows - 1));
        each<0, N>([&](auto B) {
          constexpr int b = decltype(B)::value;
          if (a.causal && limit[b] + kBlock > first_tok + 1) {  // columns of this tile that see a block only in part
            const int tok = token_of_row(min(row, rows - 1));
            if (__builtin_expect(__any(neg != neg), 0)) {
              // a NaN lse goes into its column's scores: added behind the mask, it would reach tokens that the
              // query does not see
              const float nan = neg != neg ? neg : 0.0f;
              each<b, N>([&](auto L) { sc[i][decltype(L)::value] += nan; });
              neg = neg != neg ? 0.0f : neg;
            }
#pragma unroll
            for (int x = 0; x < 16; ++x) sc[i][b][x] = limit[b] + token_of(x, half) <= tok ? sc[i][b][x] : -INFINITY;
          }
#pragma unroll
          for (int x = 0; x < 16; ++x) acc[b][x] += __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i][b][x], a.scale2, neg));
        });
      });
    };
    auto next = [&](int t) {
      asm volatile("" ::: "memory");
      // step t is in: only the loads of later ones may still be on their way
      __builtin_amdgcn_s_waitcnt(((kRing - 2) * kLoads & 15) | (7 << 4) | (0 << 8));
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      load_step(t + kRing - 1);  // where step t - 1 was
    };
    int t = 0;
    for (; t < lone; ++t) {
      next(t);
      scores(t, 0, Const<TW>{}, Const<1>{});
    }
    for (; t < steps; ++t) {
      next(t);
      for (int j = 0; j < TW; ++j)
        if (j == 0 || row0 + t * kRows + j * 32 < rows) scores(t, j, Const<1>{}, Const<NB>{});
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
  // With 256 workgroups of eight blocks every compute unit has one; below, four times
  // as many of two blocks fill it better, though each reads the queries again.  At 256
  // (2048 queries and tokens, 32 heads of 128) 45 us against 56, at 128 (1024 of
  // them) 24 against 21, at 64 with four queries to a key (2048) 136 against 69.
  const int blocks = (a.b.max_len + kBlock - 1) / kBlock, wide = (blocks + 2 * kWaves - 1) / (2 * kWaves);
  if ((int64_t)wide * a.c.kv_heads * a.b.S >= 256)
    hipLaunchKernelGGL((k_weigh<D, kWaves>), dim3(wide, a.c.kv_heads, a.b.S), dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL((k_weigh<D, 1>), dim3((blocks + 1) / 2, a.c.kv_heads, a.b.S), dim3(kThreads), 0, st, a);
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
  WeighArgs a = {*cache, *batch, T, q, q_token, q_head, q_heads, q_heads / cache->kv_heads, scale * kLog2e,
                 causal, lse, decay, weights, 0, 0};
  if (a.group > 1) {
    // magic = ceil(2^(31 + l) / group) < 2^32 with l = ceil(log2 group): exact below 2^31
    int l = 1;
    while ((1 << l) < a.group) ++l;
    a.magic = (uint32_t)((((uint64_t)1 << (31 + l)) + (uint64_t)a.group - 1) / (uint64_t)a.group);
    a.shift = l - 1;
  }
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (cache->head_dim == 64) launch<64>(a, st);
  else if (cache->head_dim == 128) launch<128>(a, st);
  else launch<256>(a, st);
  return hipGetLastError() == hipSuccess ? DLLM_OK : DLLM_ERR_HIP;
}

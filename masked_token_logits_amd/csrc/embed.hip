// Token embedding (include/dllm_embed.h): rows of a table looked up and
// scaled, and the table's gradient, the sum of the output's gradients over
// each token's places.
//
// The gradient goes by the tokens in sorted order (stable, so a token's places
// ascend): runs of equal tokens are cut into chunks of 32 (or 8) places, one wave
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

// Places of a chunk.  Short batches have chunks of 8, so that they fill more of
// the chip (the sums of 509 tokens of 256: 13.1 -> 5.6 us); long ones of 32, for
// the fewer shares of runs that span chunks.
constexpr int kChunkMost = 32, kChunkShort = 8, kShortMost = 8192;
constexpr int kCols = 512;       // columns of a wave: 64 lanes of 8
constexpr int kNoToken = 0x7FFFFFFF;  // sorts behind every token; its places have no row

// A thread to each 16 bytes of the output; neighbours have the same token, so its
// rows are read whole.  The time is the rows' bytes (131072 tokens of 4096: 364 us,
// 5.8 TB/s; 32 tokens: 2.6 us).
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

// Up to kRankMost tokens are sorted in one launch: a token's place in the
// order is the number of tokens before it, the smaller ones and the equal ones
// further up.  A workgroup places 64 tokens, its sixteen waves compare them
// with a sixteenth of the batch each, two instructions for 64 comparisons (509
// tokens: 5.8 us in one launch, where each of two passes by digits is three).
constexpr int kRankMost = 16384, kRankWaves = 16;

__global__ __launch_bounds__(64 * kRankWaves) void k_embed_rank(const int32_t* __restrict__ tokens, int T, int V,
                                                                int32_t* __restrict__ sorted,
                                                                int32_t* __restrict__ place,
                                                                int32_t* __restrict__ runs) {
  __shared__ int part[kRankWaves][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = blockIdx.x * 64, i = first + lane;
  if (blockIdx.x == 0 && threadIdx.x < 2) runs[threadIdx.x] = 0;
  const int mine = i < T ? known(tokens[i], V) : kNoToken;
  const int lo = (int)((int64_t)T * wave / kRankWaves), hi = (int)((int64_t)T * (wave + 1) / kRankWaves);
  int rank = 0;
  // those before the workgroup's own count where they are equal, those behind do not
  const int a = min(max(first, lo), hi), b = min(max(first + 64, lo), hi);
#pragma unroll 16
  for (int j = lo; j < a; ++j) rank += known(tokens[j], V) <= mine ? 1 : 0;
  for (int j = a; j < b; ++j) {
    const int o = known(tokens[j], V);
    rank += o < mine || (o == mine && j < i) ? 1 : 0;
  }
#pragma unroll 16
  for (int j = b; j < hi; ++j) rank += known(tokens[j], V) < mine ? 1 : 0;
  part[wave][lane] = rank;
  __syncthreads();
  if (wave == 0 && i < T) {
#pragma unroll
    for (int w = 1; w < kRankWaves; ++w) rank += part[w][lane];
    sorted[rank] = mine;
    place[rank] = i;
  }
}

// More are sorted by digits, the lowest first, each pass stable: how often each
// digit occurs in each tile of kTile tokens, where those of a tile begin, and
// the tokens to their places (65536 tokens, two passes of 9 bits: 5, 9 and 5 us each).
constexpr int kTile = 1024, kBinsMost = 1024;

struct PassArgs {
  const int32_t *tok, *at;  // at: the places so far; null = tokens in their own order
  int32_t *tok_out, *at_out;
  int32_t* counts;          // [bins][tiles]
  int32_t* runs;            // [2]: cleared for the sums
  int T, V, tiles, shift, bins;
};

// A token's digit; tokens without a row sort as V.
__device__ __forceinline__ int digit(const PassArgs& p, int tok) {
  return (min(tok, p.V) >> p.shift) & (p.bins - 1);
}

__global__ __launch_bounds__(256) void k_embed_count(PassArgs p) {
  __shared__ int hist[kBinsMost];
  if (blockIdx.x == 0 && threadIdx.x < 2) p.runs[threadIdx.x] = 0;
  for (int b = threadIdx.x; b < p.bins; b += 256) hist[b] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kTile / 256; ++k) {
    const int i = blockIdx.x * kTile + k * 256 + threadIdx.x;
    if (i < p.T) atomicAdd(&hist[digit(p, known(p.tok[i], p.V))], 1);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < p.bins; b += 256) p.counts[(int64_t)b * p.tiles + blockIdx.x] = hist[b];
}

// Where each digit's tokens of each tile begin: exclusive sums, in place, 16 to
// a thread.  One workgroup: 32768 counts are two rounds.
__global__ __launch_bounds__(1024) void k_embed_begin(int32_t* __restrict__ counts, int64_t n) {
  __shared__ int part[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int carry = 0;
  for (int64_t base = 0; base < n; base += 16 * 1024) {
    const int64_t i = base + threadIdx.x * 16;
    int v[16], mine = 0;
#pragma unroll
    for (int k = 0; k < 16; k += 4) {
      int4 u = make_int4(0, 0, 0, 0);
      if (i + k + 3 < n) {
        u = *reinterpret_cast<const int4*>(counts + i + k);
      } else {
        if (i + k < n) u.x = counts[i + k];
        if (i + k + 1 < n) u.y = counts[i + k + 1];
        if (i + k + 2 < n) u.z = counts[i + k + 2];
      }
      v[k] = u.x;
      v[k + 1] = u.y;
      v[k + 2] = u.z;
      v[k + 3] = u.w;
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) mine += v[k];
    int sum = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(sum, off);
      if (lane >= off) sum += o;
    }
    if (lane == 63) part[wave] = sum;
    __syncthreads();
    int before = carry, all = carry;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      before += w < wave ? part[w] : 0;
      all += part[w];
    }
    int run = before + sum - mine;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int c = v[k];
      v[k] = run;
      run += c;
    }
#pragma unroll
    for (int k = 0; k < 16; k += 4) {
      if (i + k + 3 < n) {
        *reinterpret_cast<int4*>(counts + i + k) = make_int4(v[k], v[k + 1], v[k + 2], v[k + 3]);
      } else {
        if (i + k < n) counts[i + k] = v[k];
        if (i + k + 1 < n) counts[i + k + 1] = v[k + 1];
        if (i + k + 2 < n) counts[i + k + 2] = v[k + 2];
      }
    }
    carry = all;
    __syncthreads();
  }
}

// Sixteen waves of 64 tokens: a token's place is its digit's beginning in the
// tile, the digit's tokens of the waves before, and those of the lanes before,
// which the digit's bits' ballots tell.
__global__ __launch_bounds__(kTile) void k_embed_place(PassArgs p) {
  __shared__ uint16_t count[kTile / 64][kBinsMost];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = blockIdx.x * kTile + threadIdx.x;
  for (int b = lane; b < p.bins; b += 64) count[wave][b] = 0;
  const int tok = i < p.T ? known(p.tok[i], p.V) : kNoToken, d = digit(p, tok);
  unsigned long long same = __ballot(i < p.T);
  for (int b = 1; b < p.bins; b <<= 1) {
    const unsigned long long set = __ballot((d & b) != 0);
    same &= d & b ? set : ~set;
  }
  const unsigned long long below = lane ? same & (~0ull >> (64 - lane)) : 0ull;
  if (i < p.T && below == 0) count[wave][d] = (uint16_t)__popcll(same);
  __syncthreads();
  if (i < p.T) {
    int to = p.counts[(int64_t)d * p.tiles + blockIdx.x] + __popcll(below);
    for (int w = 0; w < wave; ++w) to += count[w][d];
    p.tok_out[to] = tok;
    p.at_out[to] = p.at ? p.at[i] : i;
  }
}

// Runs that span chunks: where a run begins, its shares and its token.
struct Run {
  int first, shares, tok;
};
struct Runs {
  int32_t* count;   // [2]: runs of few shares, runs of many
  Run *few, *many;  // [chunks] each; their order changes no result
};
constexpr int kFewShares = 16;

struct SumArgs {
  const int32_t *sorted, *place;
  int T, d, chunk;
  const uint16_t* d_out;
  float scale;
  int accumulate;
  uint16_t* d_table;
  Runs runs;
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

// A chunk's runs, 512 columns.  Eight rows' loads are on their way together; the
// time is the rows of d_out and, with those that are cleared beside them, of the
// table (65536 tokens, 126464 rows of 4096: 350 us for 1.6 GB, 4.5 TB/s).
__device__ __forceinline__ void sum_chunk(const SumArgs& a, int chunk) {
  constexpr int kAtOnce = 8;  // rows whose loads are on their way together
  const int lane = threadIdx.x, begin = chunk * a.chunk, n = min(a.chunk, a.T - begin);
  const int c = blockIdx.y * kCols + lane * 8;
  const int at = begin + (lane < n ? lane : n - 1);
  const int tok = a.sorted[at], pl = a.place[at];
  const int before = begin > 0 ? a.sorted[begin - 1] : -1;
  const int behind = begin + n < a.T ? a.sorted[begin + n] : -1;
  const bool in = c < a.d;
  float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  bool from = before == __builtin_amdgcn_readlane(tok, 0);  // whether the run began in a chunk before
  for (int k0 = 0; k0 < n; k0 += kAtOnce) {
    if (__builtin_amdgcn_readlane(tok, k0) == kNoToken) return;  // only those follow
    uint4 u[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      u[k] = make_uint4(0, 0, 0, 0);
      const int p = __builtin_amdgcn_readlane(pl, min(k0 + k, n - 1));
      if (in && k0 + k < n) u[k] = *reinterpret_cast<const uint4*>(a.d_out + (int64_t)p * a.d + c);
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (k0 + k >= n) break;
      const int t = __builtin_amdgcn_readlane(tok, k0 + k);
      if (t == kNoToken) return;
      float g[8];
      unpack8(u[k], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += g[j];
      const bool last = k0 + k + 1 == n;
      const int next = last ? behind : __builtin_amdgcn_readlane(tok, min(k0 + k + 1, n - 1));
      if (!last && next == t) continue;
      const bool on = last && next == t;
      if (on && !from && blockIdx.y == 0 && lane == 0) {
        const int shares = (upper(a.sorted, begin + n, a.T, t) - 1) / a.chunk - chunk + 1;
        const bool few = shares <= kFewShares;
        (few ? a.runs.few : a.runs.many)[atomicAdd(a.runs.count + (few ? 0 : 1), 1)] = {chunk, shares, t};
      }
      if (in) {
        if (!from && !on) {
          finish(a, t, c, f);
        } else {
          float4* o = reinterpret_cast<float4*>(a.part + ((int64_t)chunk * 2 + (from ? 0 : 1)) * a.d + c);
          o[0] = make_float4(f[0], f[1], f[2], f[3]);
          o[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = 0.f;
      from = false;
    }
  }
}

// Zeros for the rows of 64 tokens that do not occur, 512 columns.
__device__ __forceinline__ void clear_rows(const SumArgs& a, int V, int first) {
  const int v = first + threadIdx.x, c = blockIdx.y * kCols + threadIdx.x * 8;
  const int at = v < V ? upper(a.sorted, 0, a.T, v - 1) : 0;
  unsigned long long none = __ballot(v < V && !(at < a.T && a.sorted[at] == v));
  while (none) {
    const int r = first + __ffsll((long long)none) - 1;
    none &= none - 1;
    if (c < a.d) *reinterpret_cast<uint4*>(a.d_table + (int64_t)r * a.d + c) = make_uint4(0, 0, 0, 0);
  }
}

// Workgroups of one wave: those of the chunks, and behind them those that clear.
__global__ __launch_bounds__(64) void k_embed_sum(SumArgs a, int V, int chunks) {
  if ((int)blockIdx.x < chunks)
    sum_chunk(a, blockIdx.x);
  else
    clear_rows(a, V, (blockIdx.x - chunks) * 64);
}

// The runs that span chunks.  Those of many shares take a workgroup for each 128
// columns, its sixteen waves a sixteenth of the shares each; those of few a
// wave for each 128 columns (half of 65536 tokens the mask token, 1024 shares of
// 4096: 25 us).
constexpr int kJoinWaves = 16, kJoinCols = 128;

// Shares lo .. hi - 1 of a run that begins in chunk `first`, two columns.
__device__ __forceinline__ float2 shares(const SumArgs& a, int first, int lo, int hi, int c) {
  float2 f = make_float2(0.f, 0.f);
#pragma unroll 8
  for (int s = lo; s < hi; ++s) {
    const float2 x = *reinterpret_cast<const float2*>(a.part + ((int64_t)(first + s) * 2 + (s == 0 ? 1 : 0)) * a.d + c);
    f = make_float2(f.x + x.x, f.y + x.y);
  }
  return f;
}
__device__ __forceinline__ void finish2(const SumArgs& a, int tok, int c, const float2& f) {
  uint32_t* o = reinterpret_cast<uint32_t*>(a.d_table + (int64_t)tok * a.d + c);
  const uint32_t old = a.accumulate ? *o : 0u;
  const float x = a.accumulate ? fmaf(f.x, a.scale, bf16_float(old & 0xFFFFu)) : f.x * a.scale;
  const float y = a.accumulate ? fmaf(f.y, a.scale, bf16_float(old >> 16)) : f.y * a.scale;
  *o = float_bf16(x) | float_bf16(y) << 16;
}

__global__ __launch_bounds__(64 * kJoinWaves) void k_embed_join(SumArgs a) {
  __shared__ float2 lds[kJoinWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, blocks = (a.d + kJoinCols - 1) / kJoinCols;
  const int64_t many = (int64_t)a.runs.count[1] * blocks, few = (int64_t)a.runs.count[0] * blocks;
  for (int64_t k = blockIdx.x; k < many; k += gridDim.x) {
    const Run r = a.runs.many[k / blocks];
    const int c = (int)(k % blocks) * kJoinCols + lane * 2;
    float2 f = make_float2(0.f, 0.f);
    if (c < a.d)
      f = shares(a, r.first, (int)((int64_t)r.shares * wave / kJoinWaves), (int)((int64_t)r.shares * (wave + 1) / kJoinWaves), c);
    lds[wave][lane] = f;
    __syncthreads();
    if (wave == 0 && c < a.d) {
#pragma unroll
      for (int w = 1; w < kJoinWaves; ++w) f = make_float2(f.x + lds[w][lane].x, f.y + lds[w][lane].y);
      finish2(a, r.tok, c, f);
    }
    __syncthreads();
  }
  for (int64_t k = (int64_t)blockIdx.x * kJoinWaves + wave; k < few; k += (int64_t)gridDim.x * kJoinWaves) {
    const Run r = a.runs.few[k / blocks];
    const int c = (int)(k % blocks) * kJoinCols + lane * 2;
    if (c < a.d) finish2(a, r.tok, c, shares(a, r.first, 0, r.shares, c));
  }
}

bool sizes_ok(int64_t V, int64_t d, int64_t T) {
  return V >= 1 && V < ((int64_t)1 << 31) - 1024 && d >= 1 && T >= 0 && T < ((int64_t)1 << 31) - 1024;
}
bool supported(int64_t d) { return d % 8 == 0 && d < ((int64_t)1 << 20); }

// Of the gradient: its sums' grid, a wave for each 32 places and one for each 64
// rows to clear, holds for fewer tokens than this.
constexpr int64_t kPlacesMost = (int64_t)1 << 30;
bool gradient_sizes_ok(int64_t V, int64_t d, int64_t T) { return sizes_ok(V, d, T) && T < kPlacesMost; }

int chunk_of(int64_t T) { return T <= kShortMost ? kChunkShort : kChunkMost; }
int64_t chunks_of(int64_t T) { return (T + chunk_of(T) - 1) / chunk_of(T); }
int64_t tiles_of(int64_t T) { return (T + kTile - 1) / kTile; }

// Digits of a token of 0 .. V: as few passes of at most 10 bits as there can be.
struct Digits {
  int passes, bits;
};
Digits digits_of(int64_t V) {
  int all = 1;
  while (V >> all) ++all;
  const int passes = (all + 9) / 10;
  return {passes, (all + passes - 1) / passes};
}

// Workspace of the gradient; returns its size.
struct Sorting {
  int32_t *sorted, *place, *sorted2, *place2, *counts;
  Runs runs;
  float* part;
};
size_t carve(int64_t V, int64_t d, int64_t T, uint8_t* base, Sorting* s) {
  Parts parts = {base};
  auto take = [&](size_t bytes) { return parts.take(bytes); };
  const size_t list = (size_t)T * 4, more = T > kRankMost ? list : 0;
  Sorting x;
  x.sorted = reinterpret_cast<int32_t*>(take(list));
  x.place = reinterpret_cast<int32_t*>(take(list));
  x.sorted2 = reinterpret_cast<int32_t*>(take(more));
  x.place2 = reinterpret_cast<int32_t*>(take(more));
  x.counts = reinterpret_cast<int32_t*>(take(more ? ((size_t)4 << digits_of(V).bits) * (size_t)tiles_of(T) : 0));
  x.runs.count = reinterpret_cast<int32_t*>(take(2 * 4));
  x.runs.few = reinterpret_cast<Run*>(take((size_t)chunks_of(T) * sizeof(Run)));
  x.runs.many = reinterpret_cast<Run*>(take((size_t)chunks_of(T) * sizeof(Run)));
  x.part = reinterpret_cast<float*>(take((size_t)chunks_of(T) * 2 * (size_t)d * 4));
  if (s) *s = x;
  return parts.size + 256;
}

void sort_tokens(const int32_t* tokens, int T, int V, const Sorting& s, hipStream_t st) {
  if (T <= kRankMost) {
    hipLaunchKernelGGL(k_embed_rank, dim3((unsigned)((T + 63) / 64)), dim3(64 * kRankWaves), 0, st, tokens, T, V, s.sorted,
                       s.place, s.runs.count);
    return;
  }
  const Digits g = digits_of(V);
  const int tiles = (int)tiles_of(T);
  PassArgs p = {tokens, nullptr, nullptr, nullptr, s.counts, s.runs.count, T, V, tiles, 0, 1 << g.bits};
  for (int k = 0; k < g.passes; ++k) {
    const bool to_first = (g.passes - 1 - k) % 2 == 0;  // the last pass ends in sorted, place
    p.tok_out = to_first ? s.sorted : s.sorted2;
    p.at_out = to_first ? s.place : s.place2;
    hipLaunchKernelGGL(k_embed_count, dim3((unsigned)tiles), dim3(256), 0, st, p);
    hipLaunchKernelGGL(k_embed_begin, dim3(1), dim3(1024), 0, st, s.counts, (int64_t)tiles << g.bits);
    hipLaunchKernelGGL(k_embed_place, dim3((unsigned)tiles), dim3(kTile), 0, st, p);
    p.tok = p.tok_out;
    p.at = p.at_out;
    p.shift += g.bits;
  }
}

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
  if (!dllm::gradient_sizes_ok(V, d, T) || !dllm::supported(d)) return 0;
  return dllm::carve(V, d, T, nullptr, nullptr);
}

dllm_status dllm_embed_backward(const int32_t* tokens, int64_t T, const uint16_t* d_out, int64_t V, int64_t d,
                                float scale, int32_t accumulate, uint16_t* d_table, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!dllm::gradient_sizes_ok(V, d, T) || !isfinite(scale) || (accumulate != 0 && accumulate != 1)) return DLLM_ERR_INVALID_ARG;
  if (!dllm::supported(d)) return DLLM_ERR_UNSUPPORTED;
  if (!d_table || (T > 0 && (!tokens || !d_out))) return DLLM_ERR_INVALID_ARG;
  if (!dllm::aligned(d_table, 16) || !dllm::aligned(d_out, 16) || !dllm::aligned(tokens, 4)) return DLLM_ERR_UNSUPPORTED;
  const size_t need = dllm_embed_backward_workspace_bytes(V, d, T), n = (size_t)V * (size_t)d * 2;
  if (!workspace || workspace_bytes < need || !dllm::aligned(workspace, 256)) return DLLM_ERR_WORKSPACE;
  if (dllm::overlaps(d_table, n, d_out, (size_t)T * (size_t)d * 2) || dllm::overlaps(d_table, n, tokens, (size_t)T * 4) ||
      dllm::overlaps(d_table, n, workspace, need) || dllm::overlaps(workspace, need, tokens, (size_t)T * 4) ||
      dllm::overlaps(workspace, need, d_out, (size_t)T * (size_t)d * 2))
    return DLLM_ERR_INVALID_ARG;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  dllm::Sorting w;
  dllm::carve(V, d, T, reinterpret_cast<uint8_t*>(workspace), &w);
  if (T > 0) dllm::sort_tokens(tokens, (int)T, (int)V, w, st);
  const int64_t chunks = dllm::chunks_of(T), clears = accumulate ? 0 : (V + 63) / 64;
  const dllm::SumArgs a = {w.sorted, w.place, (int)T, (int)d, dllm::chunk_of(T), d_out, scale, accumulate, d_table, w.runs, w.part};
  const unsigned cols = (unsigned)((d + dllm::kCols - 1) / dllm::kCols);
  if (chunks + clears > 0)
    hipLaunchKernelGGL(dllm::k_embed_sum, dim3((unsigned)(chunks + clears), cols), dim3(64), 0, st, a, (int)V, (int)chunks);
  if (chunks > 1)
    hipLaunchKernelGGL(dllm::k_embed_join, dim3((unsigned)(chunks < 512 ? chunks : 512)), dim3(64 * dllm::kJoinWaves), 0, st, a);
  return hipGetLastError() == hipSuccess ? DLLM_OK : DLLM_ERR_HIP;
}

}  // extern "C"

// Eviction from the 8-bit block cache by accumulated attention weight
// (include/dllm_cache.h): selection of the kept tokens and their move.
#include "cache_common.h"

#include <utility>

namespace dllm {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kEach = 8;                     // keys of a lane
constexpr int kChunk = kThreads * kEach;     // keys of a workgroup
constexpr int kMoveThreads = 256;
constexpr int kReach = 31;                   // pool / 2 at most
constexpr int kBins = 2048;                  // the first digit of a long selection: 11 bits

// What selection works on.  Long sequences are cut into chunks of kChunk
// tokens; a row is one sequence and head.
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
  // workspace of long selections
  int chunks;
  uint32_t* keys;        // [rows, chunks, kChunk]
  uint32_t* candidates;  // [rows, chunks, kChunk] keys whose first digit is the threshold's
  uint32_t* hist;        // [rows, chunks, kBins]
  int32_t* above;        // [rows, chunks] keys of a larger first digit
  int32_t* n_cand;       // [rows, chunks]
  int32_t* place;        // [rows, chunks] kept tokens before the chunk's
  int32_t* ties;         // [rows, chunks] tokens at the threshold before the chunk's
  uint32_t* threshold;   // [rows, 2] key, how many equal to it are kept
};

// One row's counts: n kept, `first` and `last` of them unconditionally, m by
// weight out of tokens [lo, hi).
struct Row {
  int len, n, first, last, m, lo, hi;
};

__device__ __forceinline__ Row row_of(const SelectArgs& a, int s) {
  Row r;
  r.len = min(max(a.lens[s], 0), a.max_len);
  r.n = min(min(max(a.keep[s], 0), a.max_keep), r.len);
  r.first = min(a.sink, r.n);
  r.last = min(a.recent, r.n - r.first);
  r.m = r.n - r.first - r.last;
  r.lo = r.first;
  r.hi = r.len - r.last;
  return r;
}

// Order-preserving bits of a weight: a > b as floats iff key(a) > key(b);
// -0 and 0 are equal, NaN is the lowest.
__device__ __forceinline__ uint32_t order_key(float w) {
  w = w != w ? -INFINITY : w + 0.0f;
  const uint32_t u = __float_as_uint(w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A lane's keys: token base + 64 i + lane of its wave's 64 kEach, so that a
// wave's tokens are in order and a workgroup's waves too.
__device__ __forceinline__ int token_at(int chunk, int i) {
  return chunk * kChunk + (threadIdx.x >> 6) * 64 * kEach + i * 64 + (threadIdx.x & 63);
}

// The pooled keys of a chunk, one load of each weight (and of its neighbours
// at the chunk's ends); 0, below every key, outside [lo, hi).
__device__ __forceinline__ void pooled_keys(const SelectArgs& a, const Row& r, const float* w, int chunk, uint32_t* lds,
                                            uint32_t* key) {
  const int reach = a.pool / 2, begin = chunk * kChunk - reach;
  float x[kEach + 1];
#pragma unroll
  for (int i = 0; i <= kEach; ++i) {
    const int at = i * kThreads + (int)threadIdx.x, j = begin + at;
    x[i] = at < kChunk + 2 * reach && j >= 0 && j < r.len ? w[j] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i <= kEach; ++i) {
    const int at = i * kThreads + (int)threadIdx.x, j = begin + at;
    if (at < kChunk + 2 * reach) lds[at] = j >= 0 && j < r.len ? order_key(x[i]) : 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int j = token_at(chunk, i), at = j - chunk * kChunk;
    uint32_t k = 0;
    if (j >= r.lo && j < r.hi)
      for (int d = 0; d <= 2 * reach; ++d) k = max(k, lds[at + d]);
    key[i] = k;
  }
}

__device__ __forceinline__ int wave_count(bool x) { return __popcll(__ballot(x)); }

// LDS of a search for a threshold: counts of a digit, and what the thread
// that finds the threshold's digit tells the others.
struct Search {
  uint32_t hist[kBins];
  int slots[kWaves];
  int digit, above;
};

// The digit of the want-th largest key, counted in hist (which ends cleared):
// the thread t looks after bins kBins - 1 - 2 t and the one below it, so that
// a scan over threads goes from large digits to small.  Returns the digit and the
// number of keys of larger ones, the same in all threads.
static_assert(kBins == 2 * kThreads, "two bins a thread");
__device__ __forceinline__ int find_digit(Search& l, int want, int n1, int n0, int* above) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, bin = kBins - 1 - 2 * (int)threadIdx.x;
  int upto = n0 + n1;
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 63) l.slots[wave] = upto;
  __syncthreads();
  for (int i = 0; i < wave; ++i) upto += l.slots[i];
  const int before = upto - n0 - n1;
  if (before < want && want <= upto) {
    const bool upper = want <= before + n1;
    l.digit = upper ? bin : bin - 1;
    l.above = upper ? before : before + n1;
  }
  __syncthreads();
  *above = l.above;
  return l.digit;
}

// The want-th largest (want >= 1) of some keys, all of them in lo .. hi, and
// the number of keys above it.  each(f) calls f(key, or 0 for none) for this
// thread's keys.  The bits in which lo and hi differ are found 11 at a time by
// counting digits in LDS; taking them from the first differing bit on spreads the
// counts over the bins however narrow the weights' range is.
template <class Each>
__device__ __forceinline__ uint32_t nth_largest(Search& l, uint32_t lo, uint32_t hi, int want, Each each, int* above) {
  *above = 0;
  if (lo == hi) return lo;
  int top = 31 - __clz(lo ^ hi);  // the bits above are known: t's
  uint32_t t = top == 31 ? 0 : lo >> (top + 1) << (top + 1);
  while (top >= 0) {
    const int shift = max(top - 10, 0);
    for (int i = threadIdx.x; i < kBins; i += kThreads) l.hist[i] = 0;
    __syncthreads();
    each([&](uint32_t key) {
      const bool in = key != 0 && (top == 31 || key >> (top + 1) == t >> (top + 1));
      if (in) atomicAdd(&l.hist[(key >> shift) & (kBins - 1)], 1u);
    });
    __syncthreads();
    const int bin = kBins - 1 - 2 * (int)threadIdx.x;
    int more;
    const int digit = find_digit(l, want, (int)l.hist[bin], (int)l.hist[bin - 1], &more);
    // with fewer than 11 bits left the digit holds known bits too
    t |= ((uint32_t)digit & ((2u << (top - shift)) - 1u)) << shift;
    want -= more;
    *above += more;
    top = shift - 1;
    __syncthreads();
  }
  return t;
}

__device__ __forceinline__ void put(const SelectArgs& a, int64_t row, float weight, int place, int j) {
  a.kept[row * a.max_keep + place] = j;
  if (a.weights_out) a.weights_out[row * a.out_slots + place] = weight;
}

// The tokens kept unconditionally.
__device__ __forceinline__ void put_ends(const SelectArgs& a, const Row& r, int64_t row, const float* w) {
  for (int j = threadIdx.x; j < r.first; j += kThreads) put(a, row, w[j], j, j);
  for (int j = threadIdx.x; j < r.last; j += kThreads) put(a, row, w[r.len - r.last + j], r.n - r.last + j, r.len - r.last + j);
}

// The chunk's kept tokens in order: those above the threshold, and of those at
// it the first `want` of the row; `place` and `ties` are the counts before the chunk.
__device__ __forceinline__ void put_chunk(const SelectArgs& a, int64_t row, const float* w, int chunk,
                                          const uint32_t* key, uint32_t threshold, int want, int place, int ties,
                                          int* slots) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t below = (1ull << lane) - 1;
  int n_gt = 0, n_eq = 0;
  float weight[kEach];  // all on their way at once, not one after another as they are put
#pragma unroll
  for (int i = 0; i < kEach; ++i) weight[i] = key[i] >= threshold ? w[token_at(chunk, i)] : 0.0f;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    n_gt += wave_count(key[i] > threshold);
    n_eq += wave_count(key[i] == threshold);
  }
  __syncthreads();
  if (lane == 0) slots[wave] = n_gt, slots[kWaves + wave] = n_eq;
  __syncthreads();
  for (int i = 0; i < wave; ++i) {
    place += slots[i] + min(slots[kWaves + i], max(want - ties, 0));
    ties += slots[kWaves + i];
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const bool same = key[i] == threshold;
    const uint64_t sames = __ballot(same);
    const bool take = key[i] > threshold || (same && ties + __popcll(sames & below) < want);
    const uint64_t takes = __ballot(take);
    if (take) put(a, row, weight[i], place + __popcll(takes & below), token_at(chunk, i));
    place += __popcll(takes);
    ties += __popcll(sames);
  }
}

__device__ __forceinline__ uint32_t wave_extreme(uint32_t x, bool largest) {
  for (int o = 32; o; o >>= 1) {
    const uint32_t y = __shfl_xor(x, o);
    x = largest ? max(x, y) : min(x, y);
  }
  return x;
}

// One workgroup: one row of at most kChunk tokens, whose keys stay in registers.
// Bound by the digits' counts and scans one after the other: 13 us for 32 heads of
// 4096 tokens.
__global__ __launch_bounds__(kThreads) void k_select_one(SelectArgs a) {
  __shared__ uint32_t lds[kChunk + 2 * kReach];
  __shared__ int slots[2][kWaves];
  __shared__ Search search;
  const int s = blockIdx.y, h = blockIdx.x;
  const Row r = row_of(a, s);
  const int64_t row = (int64_t)s * a.kv_heads + h;
  const float* w = a.weights + row * a.slots;
  if (h == 0 && threadIdx.x == 0) a.lens_out[s] = r.n;
  put_ends(a, r, row, w);
  if (r.m == 0) return;
  uint32_t key[kEach];
  pooled_keys(a, r, w, 0, lds, key);
  uint32_t lo = ~0u, hi = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (key[i] != 0) lo = min(lo, key[i]), hi = max(hi, key[i]);
  lo = wave_extreme(lo, false), hi = wave_extreme(hi, true);
  if ((threadIdx.x & 63) == 0) slots[0][threadIdx.x >> 6] = (int)lo, slots[1][threadIdx.x >> 6] = (int)hi;
  __syncthreads();
  for (int i = 0; i < kWaves; ++i) lo = min(lo, (uint32_t)slots[0][i]), hi = max(hi, (uint32_t)slots[1][i]);
  int above;
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) f(key[i]);
  };
  const uint32_t t = nth_largest(search, lo, hi, r.m, each, &above);
  put_chunk(a, row, w, 0, key, t, r.m - above, r.first, 0, &slots[0][0]);
}

// ---- long rows, in four kernels -------------------------------------------------------------------------------

// Keys of a chunk and the counts of their first 11 bits.
__global__ __launch_bounds__(kThreads) void k_keys(SelectArgs a) {
  __shared__ uint32_t lds[kChunk + 2 * kReach];
  __shared__ uint32_t hist[kBins];
  const int s = blockIdx.z, h = blockIdx.y, chunk = blockIdx.x;
  const Row r = row_of(a, s);
  const int64_t row = (int64_t)s * a.kv_heads + h, at = row * a.chunks + chunk;
  const float* w = a.weights + row * a.slots;
  if (chunk == 0) {
    put_ends(a, r, row, w);
    if (h == 0 && threadIdx.x == 0) a.lens_out[s] = r.n;
  }
  if (r.m == 0 || (int64_t)chunk * kChunk >= r.len) return;
  for (int i = threadIdx.x; i < kBins; i += kThreads) hist[i] = 0;
  uint32_t key[kEach];
  pooled_keys(a, r, w, chunk, lds, key);
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    a.keys[at * kChunk + token_at(0, i)] = key[i];
    if (key[i] != 0) atomicAdd(&hist[key[i] >> 21], 1u);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kThreads) a.hist[at * kBins + i] = hist[i];
}

// The threshold's first digit, and the chunk's keys of that digit.
__global__ __launch_bounds__(kThreads) void k_split(SelectArgs a) {
  __shared__ Search search;
  __shared__ int slots[kWaves], cands;
  const int s = blockIdx.z, h = blockIdx.y, chunk = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Row r = row_of(a, s);
  if (r.m == 0 || (int64_t)chunk * kChunk >= r.len) return;
  const int64_t row = (int64_t)s * a.kv_heads + h, at = row * a.chunks + chunk;
  const int chunks = (r.len + kChunk - 1) / kChunk;
  const int bin = kBins - 1 - 2 * (int)threadIdx.x;
  int n1 = 0, n0 = 0, larger;
  for (int c = 0; c < chunks; ++c) {
    const uint2 x = *reinterpret_cast<const uint2*>(a.hist + (row * a.chunks + c) * kBins + bin - 1);
    n0 += (int)x.x, n1 += (int)x.y;
  }
  if (threadIdx.x == 0) cands = 0;
  const uint32_t digit = (uint32_t)find_digit(search, r.m, n1, n0, &larger);
  int n_above = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint32_t key = a.keys[at * kChunk + token_at(0, i)];
    const bool is = key >> 21 == digit && key != 0;
    n_above += wave_count(key >> 21 > digit);
    const uint64_t all = __ballot(is);
    int to = 0;
    if (lane == 0 && all) to = atomicAdd(&cands, __popcll(all));  // their order does not matter
    to = __builtin_amdgcn_readfirstlane(to);
    if (is) a.candidates[at * kChunk + to + __popcll(all & ((1ull << lane) - 1))] = key;
  }
  __syncthreads();
  if (lane == 0) slots[wave] = n_above;
  __syncthreads();
  if (threadIdx.x == 0) {
    int n = 0;
    for (int i = 0; i < kWaves; ++i) n += slots[i];
    a.above[at] = n;
    a.n_cand[at] = cands;
  }
}

// The threshold among the candidates of a row, and what each chunk has before
// it.  One workgroup for a row; a wave takes a chunk at a time.  Up to kHeld
// candidates of up to kThreads chunks are brought into LDS once, more are read
// again for every digit.
constexpr int kHeld = 24 * 1024;

__global__ __launch_bounds__(kThreads) void k_threshold(SelectArgs a) {
  __shared__ uint32_t held[kHeld];
  __shared__ int offset[kThreads];
  __shared__ int slots[2][kWaves];
  __shared__ Search search;
  const int s = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Row r = row_of(a, s);
  if (r.m == 0) return;
  const int64_t row = (int64_t)s * a.kv_heads + h;
  const int chunks = (r.len + kChunk - 1) / kChunk;
  const uint32_t* cand = a.candidates + row * a.chunks * kChunk;
  const int32_t* n_cand = a.n_cand + row * a.chunks;
  // candidates and larger keys of all chunks; the candidates before each chunk
  int own = 0, larger = 0;
  for (int c = tid; c < chunks; c += kThreads) own += n_cand[c], larger += a.above[row * a.chunks + c];
  int upto = own;
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(upto, o);
    if (lane >= o) upto += y;
  }
  for (int o = 32; o; o >>= 1) larger += __shfl_xor(larger, o);
  if (lane == 63) slots[0][wave] = upto, slots[1][wave] = larger;
  __syncthreads();
  int total = 0;
  larger = 0;
  for (int i = 0; i < kWaves; ++i) {
    if (i < wave) upto += slots[0][i];
    total += slots[0][i], larger += slots[1][i];
  }
  offset[tid] = upto - own;
  const bool fits = total <= kHeld && chunks <= kThreads;
  __syncthreads();
  uint32_t lo = ~0u, hi = 0;
  // f(key, 0 where there is none) for this wave's chunks, eight loads at a time
  auto each_of = [&](int c, auto f) {
    const int n = n_cand[c];
    for (int i = 0; i < n; i += 512) {
      uint32_t x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = i + k * 64 + lane < n ? cand[(int64_t)c * kChunk + i + k * 64 + lane] : 0u;
#pragma unroll
      for (int k = 0; k < 8; ++k) f(x[k], i + k * 64 + lane);
    }
  };
  for (int c = wave; c < chunks; c += kWaves)
    each_of(c, [&](uint32_t key, int i) {
      if (key == 0) return;
      lo = min(lo, key), hi = max(hi, key);
      if (fits) held[offset[c] + i] = key;
    });
  lo = wave_extreme(lo, false), hi = wave_extreme(hi, true);
  __syncthreads();
  if (lane == 0) slots[0][wave] = (int)lo, slots[1][wave] = (int)hi;
  __syncthreads();
  for (int i = 0; i < kWaves; ++i) lo = min(lo, (uint32_t)slots[0][i]), hi = max(hi, (uint32_t)slots[1][i]);
  int above;
  auto each = [&](auto f) {
    if (fits)
      for (int i = tid; i < total; i += kThreads) f(held[i]);
    else
      for (int c = wave; c < chunks; c += kWaves) each_of(c, [&](uint32_t key, int) { f(key); });
  };
  const uint32_t t = nth_largest(search, lo, hi, r.m - larger, each, &above);
  const int want = r.m - larger - above;
  if (tid == 0) a.threshold[2 * row] = t, a.threshold[2 * row + 1] = (uint32_t)want;
  // per chunk: keys above and at the threshold, then their sums before it
  for (int c = wave; c < chunks; c += kWaves) {
    int gt = 0, eq = 0;
    const int n = n_cand[c];
    if (fits)
      for (int i = 0; i < n; i += 64) {
        const uint32_t key = i + lane < n ? held[offset[c] + i + lane] : 0u;
        gt += wave_count(key > t), eq += wave_count(key == t);
      }
    else
      each_of(c, [&](uint32_t key, int) { gt += wave_count(key > t), eq += wave_count(key == t); });
    if (lane == 0) a.place[row * a.chunks + c] = a.above[row * a.chunks + c] + gt, a.ties[row * a.chunks + c] = eq;
  }
  __syncthreads();
  if (wave == 0) {
    int place = r.first, ties = 0;
    for (int c0 = 0; c0 < chunks; c0 += 64) {
      const int c = c0 + lane;
      const int gt = c < chunks ? a.place[row * a.chunks + c] : 0, eq = c < chunks ? a.ties[row * a.chunks + c] : 0;
      int ties_to = eq;
      for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(ties_to, o);
        if (lane >= o) ties_to += y;
      }
      const int mine_ties = ties + ties_to - eq, taken = gt + min(eq, max(want - mine_ties, 0));
      int place_to = taken;
      for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(place_to, o);
        if (lane >= o) place_to += y;
      }
      if (c < chunks) a.place[row * a.chunks + c] = place + place_to - taken, a.ties[row * a.chunks + c] = mine_ties;
      ties += __shfl(ties_to, 63);
      place += __shfl(place_to, 63);
    }
  }
}

__global__ __launch_bounds__(kThreads) void k_keep(SelectArgs a) {
  __shared__ int slots[2 * kWaves];
  const int s = blockIdx.z, h = blockIdx.y, chunk = blockIdx.x;
  const Row r = row_of(a, s);
  if (r.m == 0 || (int64_t)chunk * kChunk >= r.len) return;
  const int64_t row = (int64_t)s * a.kv_heads + h, at = row * a.chunks + chunk;
  uint32_t key[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) key[i] = a.keys[at * kChunk + token_at(0, i)];
  put_chunk(a, row, a.weights + row * a.slots, chunk, key, a.threshold[2 * row], (int)a.threshold[2 * row + 1], a.place[at],
            a.ties[at], slots);
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

// 2^x, 0 below fp32's normal range (where e4m3 has long rounded to 0).
__device__ __forceinline__ float exact_scale(int x) { return x < -126 ? 0.0f : __uint_as_float((uint32_t)(x + 127) << 23); }

// One workgroup: one new block of one head, gathered from its tokens' old
// places.  Bound by memory: a kept token's keys are pieces of 16 bytes and its values
// single bytes of blocks that hold 32 tokens, so that the lines of a block are read
// whole or nearly.  16385 of up to 131072 tokens of 4 sequences and heads: 267 MB read for 71
// that are kept, 68 written, 70 us (4.8 TB/s); half of 4096 tokens, 32 heads, 16 us.
template <int D>
__global__ __launch_bounds__(kMoveThreads) void k_move(MoveArgs a) {
  const int s = blockIdx.z, h = blockIdx.y, blk = blockIdx.x, tid = threadIdx.x;
  const int t = blk * kBlock + (tid & (kBlock - 1));
  int n = a.lens_out[s], to = page_of(a.table_out, a.out_blocks, a.c.pages, s, blk);
  int j = t < a.max_keep ? a.kept[((int64_t)s * a.c.kv_heads + h) * a.max_keep + t] : 0;  // of use where t < n
  asm volatile("" : "+v"(n), "+v"(to), "+v"(j));  // the three on their way at once, not one behind the other's branch
  if (blk * kBlock >= n || to < 0) return;
  __shared__ int64_t src[kBlock];  // byte offset of the token's old block, -1: none
  __shared__ int slot[kBlock];
  __shared__ int ke[kBlock], ve[kBlock];
  __shared__ int kmax, vmax, kmixed, vmixed;  // largest scale bytes, and whether a token has another
  if (tid < kBlock) {
    int64_t at = -1;
    if (t < n) {
      const int page = page_of(a.table, a.table_blocks, a.c.pages, s, j / kBlock);
      if (page >= 0) at = block_of(a.c, page, h);
      slot[tid] = j % kBlock;
    } else {
      slot[tid] = 0;
    }
    src[tid] = at < 0 ? -1 : at * (kBlock * D);
    int k = at >= 0 ? stored_scale(a.c.k_scale, at) : 0, v = at >= 0 ? stored_scale(a.c.v_scale, at) : 0;
    const int k_own = k, v_own = v;
    ke[tid] = k, ve[tid] = v;
    for (int o = 16; o; o >>= 1) {
      k = max(k, __shfl_xor(k, o));
      v = max(v, __shfl_xor(v, o));
    }
    k = max(k, DLLM_CACHE_SCALE_MIN), v = max(v, DLLM_CACHE_SCALE_MIN);
    const bool km = __any(at >= 0 && k_own != k), vm = __any(at >= 0 && v_own != v);
    if (tid == 0) kmax = k, vmax = v, kmixed = km, vmixed = vm;
  }
  __syncthreads();
  const int64_t dst = block_of(a.c, to, h) * (kBlock * D);
  // Pieces of 16 bytes.  Of keys a piece is 16 dims of one token; of values it is
  // one dim of 16 tokens, 16 loads of a byte that are all in flight at once.
  for (int u = tid; u < kBlock * D / 16; u += kMoveThreads) {
    const int hh = (u >> 5) & 1, r = u & 31;
    i32x4 k = {0, 0, 0, 0};
    if (src[r] >= 0) k = *reinterpret_cast<const i32x4*>(a.c.k + src[r] + ((u & ~31) + slot[r]) * 16);
    uint32_t b[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int t = 8 * (e >> 2) + 4 * hh + (e & 3), o = slot[t];
      b[e] = src[t] < 0 ? 0 : a.c.v[src[t] + ((u & ~0x20) | ((o >> 2) & 1) << 5) * 16 + ((o >> 3) << 2 | (o & 3))];
    }
    if (kmixed && ke[r] != kmax) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t x = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) x |= rescaled((uint32_t)k[i] >> (8 * j) & 0xffu, exact_scale(ke[r] - kmax)) << (8 * j);
        k[i] = (int)x;
      }
    }
    if (vmixed) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int t = 8 * (e >> 2) + 4 * hh + (e & 3);
        if (ve[t] != vmax) b[e] = rescaled(b[e], exact_scale(ve[t] - vmax));
      }
    }
    i32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (int)(b[4 * i] | b[4 * i + 1] << 8 | b[4 * i + 2] << 16 | b[4 * i + 3] << 24);
    *reinterpret_cast<i32x4*>(a.c.k + dst + u * 16) = k;
    *reinterpret_cast<i32x4*>(a.c.v + dst + u * 16) = v;
  }
  if (tid == 0) {
    a.c.k_scale[block_of(a.c, to, h)] = (uint8_t)kmax;
    a.c.v_scale[block_of(a.c, to, h)] = (uint8_t)vmax;
  }
}

size_t chunks_of(int max_len) { return ((size_t)max_len + kChunk - 1) / kChunk; }

}  // namespace
}  // namespace dllm

extern "C" {

size_t dllm_cache_evict_workspace_bytes(const dllm_cache* cache, const dllm_cache_batch* batch) {
  using namespace dllm;
  if (!cache_ok(cache) || !cache_supported(cache) || !batch_ok(batch)) return 0;
  const size_t rows = (size_t)batch->S * cache->kv_heads, chunks = dllm::chunks_of(batch->max_len);
  if (chunks == 1) return 256;
  return rows * chunks * (2 * kChunk + kBins + 4) * sizeof(uint32_t) + rows * 2 * sizeof(uint32_t);
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
  SelectArgs sa = {batch->lens, batch->max_len, cache->kv_heads, weights, (int64_t)batch->table_blocks * kBlock, keep,
                   max_keep, sink, recent, pool, lens_out, kept, weights_out, (int64_t)out_blocks * kBlock};
  const size_t rows = (size_t)batch->S * cache->kv_heads, chunks = chunks_of(batch->max_len);
  // Rows that fit one workgroup's registers take one kernel: an eviction of half of 8192
  // tokens of 4 heads 18.5 us against 33.5 in four, of 64 heads 56 against 74.
  if (chunks == 1) {
    hipLaunchKernelGGL(k_select_one, dim3(cache->kv_heads, batch->S), dim3(kThreads), 0, st, sa);
  } else {
    uint32_t* p = static_cast<uint32_t*>(workspace);
    auto take = [&](size_t n) { return std::exchange(p, p + n); };
    sa.chunks = (int)chunks;
    sa.keys = take(rows * chunks * kChunk);
    sa.candidates = take(rows * chunks * kChunk);
    sa.hist = take(rows * chunks * kBins);
    sa.above = reinterpret_cast<int32_t*>(take(rows * chunks));
    sa.n_cand = reinterpret_cast<int32_t*>(take(rows * chunks));
    sa.place = reinterpret_cast<int32_t*>(take(rows * chunks));
    sa.ties = reinterpret_cast<int32_t*>(take(rows * chunks));
    sa.threshold = take(rows * 2);
    const dim3 grid((unsigned)chunks, cache->kv_heads, batch->S), per_row(cache->kv_heads, batch->S);
    hipLaunchKernelGGL(k_keys, grid, dim3(kThreads), 0, st, sa);
    hipLaunchKernelGGL(k_split, grid, dim3(kThreads), 0, st, sa);
    hipLaunchKernelGGL(k_threshold, per_row, dim3(kThreads), 0, st, sa);
    hipLaunchKernelGGL(k_keep, grid, dim3(kThreads), 0, st, sa);
  }
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

// Attention over the 8-bit block cache (include/dllm_cache.h).
#include "cache_common.h"
#include "cache_schedule.h"
#include "cache_tiles.h"
#include "persistent_sched.h"
#include "rotary_angle.h"

#include <algorithm>

namespace dllm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kNarrowParts = 256;  // a workgroup to a compute unit

// ---- parts of a tile, in the workspace -------------------------------------------------------------------------

// Each workgroup can leave two parts: slot 0 the one that begins inside a
// tile, slot 1 the one that ends inside one.  Per 32 rows of a part: ref and
// sum of its columns, the scale byte, and O^T as the lanes hold it.
template <int D>
struct PartRows {
  float ref[32], sum[32];
  int v_ref, pad[3];
  float o[D / 32][4][64][4];
};

__host__ __device__ constexpr size_t round256(size_t x) { return (x + 255) / 256 * 256; }

template <int D>
__device__ __forceinline__ PartRows<D>* part_of(const AttendArgs& a, int rows32, int w, int slot) {
  return reinterpret_cast<PartRows<D>*>(a.ws + round256(a.parts * sizeof(Stretch))) + ((int64_t)w * 2 + slot) * rows32;
}

size_t parts_bytes(int D, int parts, int rows32) {
  const size_t one = D == 64 ? sizeof(PartRows<64>) : D == 128 ? sizeof(PartRows<128>) : sizeof(PartRows<256>);
  return round256(parts * sizeof(Stretch)) + (size_t)parts * 2 * rows32 * one;
}

// ---- rows -------------------------------------------------------------------------------------------------------

// A lane's column of a tile of 32 rows.
struct Row {
  int64_t out;  // its row of out and lse
  int tok;      // its token, counted in the sequence's new ones
  int head;
  bool real;
};

__device__ __forceinline__ Row row_of(const AttendArgs& a, int64_t q0, int tokens, int h, int row) {
  const int rows = tokens * a.group;
  Row r;
  r.real = row < rows;
  row = min(row, rows - 1);
  r.tok = (int)((uint32_t)row / (uint32_t)a.group);
  r.head = h * a.group + (row - r.tok * a.group);
  r.out = (q0 + r.tok) * a.q_heads + r.head;
  return r;
}

// out and lse of one 32-dim chunk of 32 rows: o is the lane's share of O^T,
// not yet divided by sum, the column's whole sum.
template <int D>
__device__ __forceinline__ void write_rows(const AttendArgs& a, const Row& r, int chunk, const float* o, float ref,
                                           float sum, int v_ref) {
  const int half = (threadIdx.x & 63) >> 5;
  if (!r.real) return;
  const float inv = sum == 0.0f ? 0.0f : scale_value(v_ref) / sum;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = float_bf16(o[4 * i] * inv) | float_bf16(o[4 * i + 1] * inv) << 16;
    const uint32_t hi = float_bf16(o[4 * i + 2] * inv) | float_bf16(o[4 * i + 3] * inv) << 16;
    *reinterpret_cast<uint2*>(a.out + r.out * D + 32 * chunk + 8 * i + 4 * half) = make_uint2(lo, hi);
  }
  if (a.lse && chunk == 0 && half == 0) a.lse[r.out] = sum == 0.0f ? -INFINITY : (ref + __log2f(sum)) * kLn2;
}

// ---- few rows: the waves of a workgroup share the keys ----------------------------------------------------------

// One wave's run along the cache: blocks first, first + kWaves, ... below
// `last` of one sequence and head.  Pages and scales of 64 blocks at a time
// are looked up by the wave's lanes together.
template <int D>
struct Walk {
  const AttendArgs& a;
  int s, h, base, last;  // base: the block that lane 0's look-up stands for
  int page, k_byte, v_byte;

  __device__ Walk(const AttendArgs& a_, int s_, int h_, int first, int last_)
      : a(a_), s(s_), h(h_), base(first - 64), last(last_) {}

  // Pages of 64 blocks from j on, and their scales on their way.
  __device__ __forceinline__ void look(int j) {
    base = j;
    const int b = base + (threadIdx.x & 63);
    page = b < last ? page_of(a.b.table, a.b.table_blocks, a.c.pages, s, b) : -1;
    const int64_t at = block_of(a.c, max(page, 0), h);
    k_byte = stored_scale(a.c.k_scale, at);
    v_byte = stored_scale(a.c.v_scale, at);
  }

  // Wait for them here: behind a branch the wait would be for every load in
  // flight, at every use.
  __device__ __forceinline__ void looked() { asm volatile("" : "+v"(page), "+v"(k_byte), "+v"(v_byte)); }

  // Block j's keys and values on their way; false if it has no page.
  __device__ __forceinline__ bool load(int j, i32x4* k, i32x4* v) {
    const int p = __builtin_amdgcn_readlane(page, j - base);
    const int64_t at = block_of(a.c, max(p, 0), h) * (kBlock * D) + (threadIdx.x & 63) * 16;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) k[c] = *reinterpret_cast<const i32x4*>(a.c.k + at + c * 1024);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) v[c] = *reinterpret_cast<const i32x4*>(a.c.v + at + c * 1024);
    return p >= 0;
  }

  // The first look-up, with the block's loads behind it at once.
  __device__ __forceinline__ bool first(int j, i32x4* k, i32x4* v, int& kb, int& vb) {
    look(j);
    const bool ok = load(j, k, v);
    looked();
    kb = __builtin_amdgcn_readlane(k_byte, 0), vb = __builtin_amdgcn_readlane(v_byte, 0);
    return ok;
  }

  // Block j's scale bytes, and its keys and values on their way; false if it
  // has no page.
  __device__ __forceinline__ bool fetch(int j, i32x4* k, i32x4* v, int& kb, int& vb) {
    if (j >= base + 64 || j < base) {
      look(j);
      looked();
    }
    kb = __builtin_amdgcn_readlane(k_byte, j - base);
    vb = __builtin_amdgcn_readlane(v_byte, j - base);
    return load(j, k, v);
  }
};

// One workgroup: its stretch of the line, 32 rows at a time.  The four waves
// hold the same rows and take the blocks in turn, each straight from memory
// into registers with the next block in flight; at a tile's end their states
// are joined through LDS.
//
// Bound by memory, and where that takes little by what comes one after the other:
// schedule, pages, blocks, join.  One token of 16 sequences of up to 4096 tokens, 8 heads
// of 128: 20 us for 86 MB (4.3 TB/s), k_join 5.5; a 32-token block of 32 heads over
// 4096 tokens 12 us for 34 MB, k_join 4.5.  One workgroup to a compute unit: two, whose
// waves have half the registers and spill, took 26 and 17 us and made twice the
// parts; three blocks in a wave's registers instead of two 21 and 13.
template <int D>
__global__ __launch_bounds__(kThreads, 1) void k_attend_few(AttendArgs a) {
  __shared__ __attribute__((aligned(16))) float o_lds[kWaves][D / 32][4][64][4];
  __shared__ float ref_lds[kWaves][32], sum_lds[kWaves][32];
  __shared__ int v_lds[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 31, half = lane >> 5;
  int w;
  int64_t left;
  Stretch at = find_stretch<32, kBlock>(a, reinterpret_cast<int64_t*>(o_lds), &w, &left);
  __syncthreads();
  if (threadIdx.x == 0) reinterpret_cast<Stretch*>(a.ws)[w] = at;
  while (left > 0) {
    const SeqView q = seq_view(a.b, a.T, at.s);
    const int steps = tile_steps<32, kBlock>(a, q, at.rt);
    const int n = (int)min((int64_t)(steps - at.begin), left);
    const int row0 = at.rt * 32;
    const Row r = row_of(a, q.q0, q.rows, at.h, row0 + col);
    Frag qf[D / 16];
    load_query<D>(qf, a.q + (q.q0 + r.tok) * a.q_token + (int64_t)r.head * a.q_head, half);
    // this column sees tokens [0, end); blocks below `whole` are seen whole by every column
    const int end = a.causal ? min(max(q.len - q.n + r.tok + 1, 0), q.len) : q.len;
    const int whole = (a.causal ? min(max(q.len - q.n + (int)((uint32_t)row0 / (uint32_t)a.group) + 1, 0), q.len) : q.len) / kBlock;
    const int last = min(at.begin + n, (q.len + kBlock - 1) / kBlock);
    Accumulator<D> acc;
    clear(acc);
    Walk<D> walk(a, at.s, at.h, at.begin + wave, last);
    i32x4 k[D / 32], v[D / 32];
    int kb, vb;
    int j = at.begin + wave;
    const int clean = min(last, whole);  // blocks below need no mask
    auto add = [&](const i32x4* k, const i32x4* v, int kb, int vb) {
      const f32x16 sc = scores<D>(qf, k, scale_value(kb));
      cover<D>(acc, largest(sc), a.scale2);
      Frag p[2];
      probabilities<D>(acc, sc, a.scale2, p);
      add_values<D>(acc, p, v, cover_values<D>(acc, vb));
    };
    if (j < clean) {
      // two blocks in turn, each in registers of its own: copying the one in flight
      // to the other would wait for it
      i32x4 k2[D / 32], v2[D / 32];
      int kb2, vb2;
      bool ok = walk.first(j, k, v, kb, vb);
      for (;;) {
        const bool ok2 = walk.fetch(min(j + kWaves, clean - 1), k2, v2, kb2, vb2);
        if (ok) add(k, v, kb, vb);
        if ((j += kWaves) >= clean) break;
        ok = walk.fetch(min(j + kWaves, clean - 1), k, v, kb, vb);
        if (ok2) add(k2, v2, kb2, vb2);
        if ((j += kWaves) >= clean) break;
      }
    }
    for (; j < last; j += kWaves) {
      if (!walk.fetch(j, k, v, kb, vb)) continue;
      f32x16 sc = scores<D>(qf, k, scale_value(kb));
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[i] = token_of(i, half) < end - j * kBlock ? sc[i] : -INFINITY;
      cover<D>(acc, largest(sc), a.scale2);
      Frag p[2];
      probabilities<D>(acc, sc, a.scale2, p);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) v[c] = clip_values(v[c], half, q.len - j * kBlock);
      const float vs = cover_values<D>(acc, vb);
      if (a.causal)
        add_values_masked<D>(acc, p, v, vs, end - j * kBlock, half);
      else
        add_values<D>(acc, p, v, vs);
    }
    // join the waves: each takes some of the 32-dim chunks of all of them
    const float sum = column_sum(acc.sum);
    if (half == 0) ref_lds[wave][col] = acc.ref, sum_lds[wave][col] = sum;
    if (lane == 0) v_lds[wave] = acc.v_ref;
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(o_lds[wave][c][i][lane]) =
            make_float4(acc.o[c][4 * i], acc.o[c][4 * i + 1], acc.o[c][4 * i + 2], acc.o[c][4 * i + 3]);
    __syncthreads();
    float ref = -INFINITY, total = 0.0f, part[kWaves];
    int v_ref = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      ref = fmaxf(ref, ref_lds[i][col]);
      v_ref = max(v_ref, v_lds[i]);
    }
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      const float x = part_of_ref(ref_lds[i][col], ref);
      total += x * sum_lds[i][col];
      part[i] = x * exact_power(v_lds[i] - v_ref);
    }
    const bool complete = n == steps;
    PartRows<D>* out = part_of<D>(a, 1, w, at.begin > 0 ? 0 : 1);
    if (!complete && wave == 0) {
      if (half == 0) out->ref[col] = ref, out->sum[col] = total;
      if (lane == 0) out->v_ref = v_ref;
    }
#pragma unroll
    for (int c = wave; c < D / 32; c += kWaves) {
      float o[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = 0.0f;
#pragma unroll
      for (int x = 0; x < kWaves; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 y = *reinterpret_cast<const float4*>(o_lds[x][c][i][lane]);
          o[4 * i] += part[x] * y.x, o[4 * i + 1] += part[x] * y.y;
          o[4 * i + 2] += part[x] * y.z, o[4 * i + 3] += part[x] * y.w;
        }
      if (complete) {
        write_rows<D>(a, r, c, o, ref, total, v_ref);
      } else if (r.real) {  // the rest is never used
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(out->o[c][i][lane]) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      }
    }
    left -= n;
    if (left > 0) {
      next_tile<32>(a, at, steps);
      __syncthreads();
    }
  }
}

// ---- many rows: the keys pass through LDS -----------------------------------------------------------------------

#define LDS_AS __attribute__((address_space(3)))

// What a block without a page reads: its scores are finite and then left out.
__device__ __attribute__((aligned(16))) uint8_t no_page[kBlock * 256];

constexpr int kManyParts = 256;  // one workgroup to a compute unit
constexpr int kManyBlocks = 2;   // blocks of a step

// Pages and scales of a run of blocks, 64 at a time, one to a lane, so that
// in the loop they are a lane read instead of loads from two tables.
struct Lookup {
  int base;
  int64_t at;  // byte offset of the block's keys, and of its values
  int info;    // k byte | v byte << 8 | has a page << 16

  // Makes block j's (and 63 more) known.
  template <int D>
  __device__ __forceinline__ void cover(const AttendArgs& a, int s, int h, int j, int last) {
    if (__builtin_expect((uint32_t)(j - base) < 64u, 1)) return;
    base = __builtin_amdgcn_readfirstlane(j);
    const int b = j + (threadIdx.x & 63);
    const int page = b < last ? page_of(a.b.table, a.b.table_blocks, a.c.pages, s, b) : -1;
    const int64_t x = block_of(a.c, max(page, 0), h);
    at = page < 0 ? -1 : x * (kBlock * D);
    info = page < 0 ? 127 | 1 << 8 : stored_scale(a.c.k_scale, x) | stored_scale(a.c.v_scale, x) << 8 | 1 << 16;  // no page: moves no scale
    // wait for them here: behind the branch the wait would be for every load
    // in flight, at every use
    asm volatile("" : "+v"(at), "+v"(info));
  }
  __device__ __forceinline__ int info_of(int j) const { return __builtin_amdgcn_readlane(info, j - base); }
  __device__ __forceinline__ int64_t at_of(int j) const {
    const uint32_t lo = __builtin_amdgcn_readlane((int)at, j - base), hi = __builtin_amdgcn_readlane((int)(at >> 32), j - base);
    return (int64_t)((uint64_t)hi << 32 | lo);
  }
};
__device__ __forceinline__ int k_byte(int info) { return info & 0xff; }
__device__ __forceinline__ int v_byte(int info) { return info >> 8 & 0xff; }
__device__ __forceinline__ bool has_page(int info) { return info >> 16 != 0; }

// One workgroup: its stretch of the line, BM = 128 RG rows at a time, 32 RG
// to each of the 4 waves, one wave to a SIMD.  Blocks go from memory into a
// ring in LDS as stored, kAhead steps ahead, once for all rows; each wave
// widens them as it reads, once for its RG groups of 32 rows.  In the body of
// the loop the products of three blocks are in flight, independent of each other:
// the scores of block b + 1, the probabilities of block b and the output of
// block b - 1, so that the matrix pipe and the VALU work at the same time.
//
// Bound by instruction issue: of 8192 queries over 8192 tokens, 28 heads of 128 on 4 (962
// GFLOP, 830 to 895 us a call by the card's clock, 1075 to 1160 TFLOP/s where a bf16 product
// of 8192^3 reaches 1487), a SIMD's cycles are 56% matrix and 63% vector instructions,
// side by side: a score's exponential, scaling, sum, maximum and rounding and a widened key's and value's
// conversions.  Two groups of 32 rows to a wave halve the widening; a third has no registers.
template <int D, int RG>
__global__ __launch_bounds__(kThreads, 1) void k_attend_many(AttendArgs a) {
  constexpr int BM = kWaves * 32 * RG, KEYS = kBlock * kManyBlocks;
  constexpr int CH = D / 32;              // 1 KiB chunks of a block's keys or values
  constexpr int kStep = kManyBlocks * 2 * CH * 1024;  // bytes of a step: for each block its keys, then its values
  constexpr int kRing = D == 256 ? 4 : 5;             // steps in LDS
  constexpr int kAhead = kRing - 2;                   // steps that loads run ahead
  __shared__ __attribute__((aligned(1024))) uint8_t ring[kRing * kStep];
  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int w;
  int64_t left;
  Stretch at = find_stretch<BM, KEYS>(a, reinterpret_cast<int64_t*>(ring), &w, &left);
  __syncthreads();
  if (threadIdx.x == 0) reinterpret_cast<Stretch*>(a.ws)[w] = at;
  while (left > 0) {
    const SeqView q = seq_view(a.b, a.T, at.s);
    const int steps = tile_steps<BM, KEYS>(a, q, at.rt);
    const int n = (int)min((int64_t)(steps - at.begin), left);
    const int row0 = at.rt * BM + wave * 32 * RG;
    Row r[RG];
    int end[RG];
    Frag qf[RG][D / 16];
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      r[g] = row_of(a, q.q0, q.rows, at.h, row0 + g * 32 + col);
      load_query<D>(qf[g], a.q + (q.q0 + r[g].tok) * a.q_token + (int64_t)r[g].head * a.q_head, half);
      end[g] = a.causal ? min(max(q.len - q.n + r[g].tok + 1, 0), q.len) : q.len;
      // queries are only ever matrix operands: in the accumulation registers
      // they leave the others to the scores
      each<0, D / 16>([&](auto i) {
        i32x4 x = qf[g][decltype(i)::value].w;
        asm volatile("" : "+a"(x));
        qf[g][decltype(i)::value].w = x;
      });
    }
    // blocks below `whole` are seen whole by every row of the workgroup's tile
    const int least = a.causal ? min(max(q.len - q.n + (int)((uint32_t)(at.rt * BM) / (uint32_t)a.group) + 1, 0), q.len) : q.len;
    const int first = at.begin * kManyBlocks;
    const int last = min(first + n * kManyBlocks, (q.len + kBlock - 1) / kBlock);
    const int clean = max(min(last, least / kBlock), first);

    f32x16 o[RG][CH];
    float ref[RG], sum[RG];
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      ref[g] = -INFINITY, sum[g] = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[g][c][i] = 0.0f;
    }
    int v_ref = 0;

    Lookup ahead, here;
    ahead.base = here.base = -1000;
    // The wave's share of step t's loads: the keys or the values of one of its
    // blocks, CH loads, for every step alike (behind the last block they read
    // nothing of use), so that waits can count them.
    int put = 0;  // where in the ring the next step goes
    const uint8_t* mine = wave & 1 ? a.c.v : a.c.k;
    const uint8_t* nothing = no_page;
    asm volatile("" : "+s"(mine), "+s"(nothing));  // kept, not loaded again at every step
    const uint8_t* src;
    auto find_step = [&](int t) {
      const int j0 = first + t * kManyBlocks;
      ahead.cover<D>(a, at.s, at.h, j0, last);
      const int64_t from = ahead.at_of(j0 + (wave >> 1));
      src = from < 0 ? nothing : mine + from;
    };
    auto load_step = [&]() {
      uint8_t* dst = ring + put + wave * CH * 1024;
      each<0, CH>([&](auto c) {
        constexpr int x = decltype(c)::value * 1024;  // the instruction's offset counts on both sides
        __builtin_amdgcn_global_load_lds((const void*)(src + lane * 16 + (x & ~4095)), (LDS_AS void*)(dst + (x & ~4095)), 16,
                                         x & 4095, 0);
      });
      put = put + kStep == kRing * kStep ? 0 : put + kStep;
    };
    constexpr int kSlot = 2 * CH * 1024;  // a block's keys and values
    auto chunk_at = [&](int slot, int side, int c) {  // the lane's 16 bytes
      return *reinterpret_cast<const i32x4*>(ring + slot + (side * CH + c) * 1024);
    };
    auto chunk = [&](int j, int side, int c) {
      return chunk_at((j - first) % (kRing * kManyBlocks) * kSlot + lane * 16, side, c);
    };
    auto qk = [&](int j, int k_byte, f32x16* s) {
      const float ks = scale_value(k_byte);
#pragma unroll
      for (int g = 0; g < RG; ++g) s[g] = f32x16{};
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        Frag lo, hi;
        widen_keys(chunk(j, 0, c), ks, lo, hi);
#pragma unroll
        for (int g = 0; g < RG; ++g) s[g] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(lo.b, qf[g][2 * c].b, s[g], 0, 0, 0);
#pragma unroll
        for (int g = 0; g < RG; ++g) s[g] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(hi.b, qf[g][2 * c + 1].b, s[g], 0, 0, 0);
      }
    };
    auto pv = [&](int j, float vs, const Frag (*p)[2]) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        Frag lo, hi;
        widen_values(chunk(j, 1, c), vs, lo, hi);
#pragma unroll
        for (int g = 0; g < RG; ++g) o[g][c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(lo.h, p[g][0].h, o[g][c], 0, 0, 0);
#pragma unroll
        for (int g = 0; g < RG; ++g) o[g][c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(hi.h, p[g][1].h, o[g][c], 0, 0, 0);
      }
    };
    // The same where rows see the block in part: values at or behind the length
    // are cleared, and a NaN value reaches only the rows that see its token
    // (add_values_masked in cache_tiles.h says how).
    auto pv_masked = [&](int j, float vs, const Frag (*p)[2]) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        Frag lo, hi;
        i32x4 x = clip_values(chunk(j, 1, c), half, q.len - j * kBlock), nan;
        take_nan(x, nan);
        widen_values(x, vs, lo, hi);
#pragma unroll
        for (int g = 0; g < RG; ++g) {
          o[g][c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(lo.h, p[g][0].h, o[g][c], 0, 0, 0);
          o[g][c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(hi.h, p[g][1].h, o[g][c], 0, 0, 0);
        }
        if (__any(nan[0] | nan[1] | nan[2] | nan[3])) {
#pragma unroll
          for (int g = 0; g < RG; ++g) spread_nan(o[g][c], nan, end[g] - j * kBlock, half);
        }
      }
    };
    // (Constants and `each` here because loops in code marked as rare are not
    // unrolled, and what they index would live in memory.)
    auto rescale_all = [&](auto g, float alpha) {
      each<0, CH>([&](auto c) { o[decltype(g)::value][decltype(c)::value] *= alpha; });
    };
    auto value_scale = [&](int vb) {
      if (v_ref == 0) v_ref = vb;
      if (__builtin_expect(vb > v_ref + kValueSlack, 0)) {
        each<0, RG>([&](auto g) { rescale_all(g, exact_power(v_ref - vb)); });
        v_ref = vb;
      }
      return __uint_as_float((uint32_t)max(vb - v_ref + 127, 1) << 23);
    };

    f32x16 s[RG];   // scores
    Frag p[RG][2];  // probabilities
    float top[RG];
#pragma unroll
    for (int g = 0; g < RG; ++g) p[g][0].w = p[g][1].w = i32x4{0, 0, 0, 0};
    // Moves the references to cover s; O and the probabilities still to be used
    // follow (those are rounded to fp16 once more by that, in the few blocks where it
    // happens; the factor is not rounded, for below 2^-14 it would lose bits as an fp16
    // number.  That costs 8192 queries 0.3%, causal ones 1%; scaling O a block later instead,
    // when they are in it too, costs as much).
    float neg[RG];  // -ref, or -inf where no token has been seen
#pragma unroll
    for (int g = 0; g < RG; ++g) neg[g] = -INFINITY;
    auto cover_all = [&]() {
      bool grow = false;
#pragma unroll
      for (int g = 0; g < RG; ++g) grow |= __builtin_fmaf(top[g], a.scale2, -kOffset) > ref[g] + kSlack;
      if (__builtin_expect(__any(grow), 0)) {
        each<0, RG>([&](auto G) {
          constexpr int g = decltype(G)::value;
          const float to = fmaxf(ref[g], __builtin_fmaf(column_max(top[g]), a.scale2, -kOffset));
          const float alpha = part_of_ref(ref[g], to);
          ref[g] = to;
          neg[g] = negative(to);
          sum[g] *= alpha;
          rescale_all(G, alpha);
          each<0, 16>([&](auto I) {
            constexpr int i = decltype(I)::value;
            p[g][i / 8].h[i % 8] = (_Float16)((float)p[g][i / 8].h[i % 8] * alpha);
          });
        });
      }
    };

    // In step t: step t + 1 has landed for every wave, every wave is done with
    // step t - 2, and the loads of step t + kAhead begin in its place.
    auto begin_step = [&](int t) {
      find_step(t + kAhead);
      stage_sync<(kAhead - 2) * CH>();
      load_step();
    };
#pragma unroll
    for (int t = 0; t < kAhead; ++t) {
      find_step(t);
      load_step();
    }
    int j = first, t = 0;
    const int whole_steps = (clean - first) / kManyBlocks;
    if (whole_steps > 0) {
      stage_sync<(kAhead - 2) * CH>();
      here.cover<D>(a, at.s, at.h, first, last);
      int i0 = here.info_of(first), i1 = here.info_of(first + 1), i_before = i0;
      qk(first, k_byte(i0), s);
#pragma unroll
      for (int g = 0; g < RG; ++g) top[g] = largest(s[g]);
      const int lane16 = lane * 16;
      int cur = lane16, next = kStep + lane16, before = lane16;  // steps t, t + 1, t - 1 in the ring
      i32x4 raw[2 * CH];  // chunks of the keys of j + 1, then of the values of j - 1
      each<0, CH>([&](auto c) { raw[decltype(c)::value] = chunk_at(cur + kSlot, 0, decltype(c)::value); });
      Frag f[2];  // widened chunk halves: the one in use and the next
      {
        Frag hi;
        widen_keys(raw[0], scale_value(k_byte(i1)), f[0], hi);
      }
      // Scores of block j + 1 (keys in raw), probabilities of j, output of j - 1
      // (values at at_v; at first p is 0, and what is at at_v is block 1, which every
      // row sees whole); at_k2: keys of j + 2.
      auto body = [&](auto first_of_step, int at_v, int at_k2, int info_s, int info_k, int info_k2, int info_v) {
        if (__builtin_expect(!has_page(info_s), 0)) {
          each<0, RG>([&](auto G) {
            constexpr int g = decltype(G)::value;
            top[g] = -INFINITY;
            s[g] = s[g] * 0.0f - INFINITY;
          });
        }
        const float vs = value_scale(v_byte(info_v));
        cover_all();
        const float ks = scale_value(k_byte(info_k)), ks2 = scale_value(k_byte(info_k2));
        f32x16 s1[RG];
        Frag p1[RG][2];
        float x[16 * RG], add[RG];
#pragma unroll
        for (int g = 0; g < RG; ++g) add[g] = 0.0f;
        // 4 CH RG beats of one matrix instruction each, and between them an even
        // share of everything else: the next operand half widened, the next
        // chunk but one read from LDS, the probabilities of block j in three
        // stages a beat apart (argument, exponential, sum and rounding), and in
        // the second half the maxima of the new scores.  The barriers keep the
        // compiler from collecting like with like.
        constexpr int kBeats = 4 * CH * RG, kE = 16 * RG;
        each<0, kBeats + 2>([&](auto beat) {
          constexpr int h = decltype(beat)::value, F = h / RG, g = h % RG;  // operand half, row group
          if constexpr (h < kBeats) {
            if constexpr (F < 2 * CH) {
              const f32x16 zero = {};
              s1[g] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[F & 1].b, qf[g][F].b, F == 0 ? zero : s1[g], 0, 0, 0);
            } else {
              constexpr int c = (F - 2 * CH) / 2;
              o[g][c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[F & 1].h, p[g][F & 1].h, o[g][c], 0, 0, 0);
            }
            // In the first block of a step, while there is nothing yet to wait for:
            // the step's barrier, and the loads that it lets begin.
            if constexpr (decltype(first_of_step)::value && h == kBeats / 4) {
              asm volatile("" ::: "memory");
              __builtin_amdgcn_s_waitcnt(((kAhead - 2) * CH & 15) | (7 << 4) | (15 << 8));
              __builtin_amdgcn_s_barrier();
              asm volatile("" ::: "memory");
            }
            if constexpr (decltype(first_of_step)::value && h == kBeats / 4 + 1) load_step();
            // operand half F + 1: dwords 2 and 3 of its chunk if odd, else 0 and 1
            constexpr int N = (F + 1) % (4 * CH);
#pragma unroll
            for (int i = g * 2 / RG; i < (g + 1) * 2 / RG; ++i) {
              const int w = raw[N / 2][2 * (N & 1) + i];
              if constexpr (N < 2 * CH) {
                const float sc = N == 0 ? ks2 : ks;
                f[N & 1].b2[2 * i] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, sc, false);
                f[N & 1].b2[2 * i + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, sc, true);
              } else {
                f[N & 1].h2[2 * i] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, vs, false);
                f[N & 1].h2[2 * i + 1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, vs, true);
              }
            }
            __builtin_amdgcn_sched_barrier(0);  // widened early in the beat: the next instruction may need it
            // The values of j - 1 are read in the first half, the keys of j + 2 in the
            // second, and each half ends with one wait for all of them.
            if constexpr (h % (2 * RG) == 0) {
              constexpr int c = h / (2 * RG);
              if constexpr (c < CH)
                raw[CH + c] = chunk_at(at_v, 1, c);
              else
                raw[c - CH] = chunk_at(at_k2, 0, c - CH);
            }
            if constexpr (h + 1 == (2 * CH - 1) * RG || h + 1 == (4 * CH - 1) * RG) __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
            if constexpr (F >= 2 * CH + 1) {  // maxima of s1: 8 a row group, over the beats left
              constexpr int kFirst = (2 * CH + 1) * RG, kLeft = kBeats - kFirst;
              constexpr int m = h - kFirst;
#pragma unroll
              for (int i = m * 8 * RG / kLeft; i < (m + 1) * 8 * RG / kLeft; ++i) {
                const int gg = i / 8, e = i % 8 * 2;
                float most = __builtin_elementwise_maximum(s1[gg][e], s1[gg][e + 1]);
                if (e != 0) most = __builtin_elementwise_maximum(top[gg], most);
                asm volatile("" : "+v"(most));
                top[gg] = most;
              }
            }
          }
#pragma unroll
          for (int i = (h - 2) * kE / kBeats; i < (h - 1) * kE / kBeats; ++i)
            if (i >= 0) {
              float sum_to = add[i / 16] + x[i];
              asm volatile("" : "+v"(sum_to));  // here, not where it is used
              add[i / 16] = sum_to;
              if (i & 1) {
                int pair = __builtin_bit_cast(int, f16x2{(_Float16)x[i - 1], (_Float16)x[i]});
                asm volatile("" : "+v"(pair));
                p1[i / 16][i % 16 / 8].w[i % 8 / 2] = pair;
              }
            }
#pragma unroll
          for (int i = (h - 1) * kE / kBeats; i < h * kE / kBeats; ++i)
            if (i >= 0 && h <= kBeats) x[i] = __builtin_amdgcn_exp2f(x[i]);
          if (h < kBeats) {
#pragma unroll
            for (int i = h * kE / kBeats; i < (h + 1) * kE / kBeats; ++i)
              x[i] = __builtin_fmaf(s[i / 16][i % 16], a.scale2, neg[i / 16]);
            __builtin_amdgcn_sched_barrier(0);
          }
        });
#pragma unroll
        for (int g = 0; g < RG; ++g) {
          sum[g] += add[g];
          s[g] = s1[g];
          p[g][0] = p1[g][0], p[g][1] = p1[g][1];
        }
      };
      int i2, i3;
      for (;;) {
        here.cover<D>(a, at.s, at.h, j + 2, last);  // behind `last`: no page, zeros
        i2 = here.info_of(j + 2), i3 = here.info_of(j + 3);
        find_step(t + kAhead);
        body(Const<1>{}, before + kSlot, next, i0, i1, i2, i_before);
        body(Const<0>{}, cur, next + kSlot, i1, i2, i3, i0);
        i_before = i1, i0 = i2, i1 = i3;
        before = cur, cur = next;
        next = next + kStep >= kRing * kStep ? next + kStep - kRing * kStep : next + kStep;
        j += kManyBlocks;
        if (++t == whole_steps) break;
      }
      pv(j - 1, value_scale(v_byte(i_before)), p);
    }
    // blocks that some row sees in part, or not at all, one after the other
    for (; j < last; ++j) {
      if ((j - first) % kManyBlocks == 0) begin_step((j - first) / kManyBlocks);
      here.cover<D>(a, at.s, at.h, j, last);
      const int info = here.info_of(j);
      qk(j, k_byte(info), s);
#pragma unroll
      for (int g = 0; g < RG; ++g) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[g][i] = has_page(info) && token_of(i, half) < end[g] - j * kBlock ? s[g][i] : -INFINITY;
        top[g] = largest(s[g]);
      }
      cover_all();
#pragma unroll
      for (int g = 0; g < RG; ++g) sum[g] += probabilities(s[g], a.scale2, neg[g], p[g]);
      pv_masked(j, value_scale(v_byte(info)), p);
    }
    stage_sync<0>();  // loads that ran ahead have landed before the ring is used again
    // rows or parts
    const bool complete = n == steps;
    PartRows<D>* out = part_of<D>(a, kWaves * RG, w, at.begin > 0 ? 0 : 1) + wave * RG;
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      const float total = column_sum(sum[g]);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (complete) {
          float x[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = o[g][c][i];
          write_rows<D>(a, r[g], c, x, ref[g], total, v_ref);
        } else if (r[g].real) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(out[g].o[c][i][lane]) =
                make_float4(o[g][c][4 * i], o[g][c][4 * i + 1], o[g][c][4 * i + 2], o[g][c][4 * i + 3]);
        }
      }
      if (!complete) {
        if (half == 0) out[g].ref[col] = ref[g], out[g].sum[col] = total;
        if (lane == 0) out[g].v_ref = v_ref;
      }
    }
    left -= n;
    if (left > 0) {
      next_tile<BM>(a, at, steps);
      __syncthreads();
    }
  }
}

// ---- joining a tile's parts -------------------------------------------------------------------------------------

// One workgroup for each few stretches and 32-row, 32-dim piece of a tile: where
// stretch w is the first to begin inside its tile, the piece is joined here from
// w - 1's last part and the first parts of w, w + 1, ...  First the largest reference and
// value scale of all parts, then their sums under these: the waves take the parts
// in turn, a few in flight at a time, and what they have is added in order, so that the
// same call has the same result.  (Rescaling what was there for each part, a chain of
// dependent steps, was slower, and so was a workgroup for every stretch, most of them
// only to find no work.  The pieces of one tile are neighbours in the grid, for then
// they spread over the 8 chips: 4 tiles of 64 parts, 29 MB, take 11.5 us, all on
// one chip 31.)
constexpr int kJoinFlight = 4;

template <int D, int BM, int kTurns, int kStretches>
__global__ __launch_bounds__(kTurns * 64) void k_join(AttendArgs a) {
  __shared__ float o_lds[kTurns][4][64][4];
  __shared__ float ref_lds[kTurns][32], sum_lds[kTurns][32];
  __shared__ int v_lds[kTurns];
  const int chunk = blockIdx.x, sub = blockIdx.y, stretch0 = blockIdx.z * kStretches;
  const int lane = threadIdx.x & 63, turn = threadIdx.x >> 6, col = lane & 31, half = lane >> 5;
  const Stretch* all = reinterpret_cast<const Stretch*>(a.ws) + stretch0;
  uint64_t todo = __ballot(lane < kStretches && all[lane].parts > 0);
  for (; todo; todo &= todo - 1) {
    const int w0 = __ffsll((unsigned long long)todo) - 1, w = stretch0 + w0;
    const Stretch me = all[w0];
    const int row0 = me.rt * BM + sub * 32, parts = me.parts;
    if (row0 >= me.rows * a.group) continue;
    const Row r = row_of(a, me.q0, me.rows, me.h, row0 + col);
    auto part = [&](int i) { return part_of<D>(a, BM / 32, i == 0 ? w - 1 : w + i - 1, i == 0 ? 1 : 0) + sub; };
    float ref = -INFINITY, sum = 0.0f;
    int v = 0;
    for (int i = 2 * turn + half; i < parts; i += 2 * kTurns) {
      const PartRows<D>* p = part(i);
      ref = fmaxf(ref, p->ref[col]), v = max(v, p->v_ref);
    }
    ref = fmaxf(ref, __shfl_xor(ref, 32)), v = max(v, __shfl_xor(v, 32));
    if (half == 0) ref_lds[turn][col] = ref;
    if (lane == 0) v_lds[turn] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTurns; ++i) ref = fmaxf(ref, ref_lds[i][col]), v = max(v, v_lds[i]);
    float o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = 0.0f;
    if (r.real)
      for (int i0 = turn; i0 < parts; i0 += kTurns * kJoinFlight) {
        float4 x[kJoinFlight][4];
        float part_ref[kJoinFlight], part_sum[kJoinFlight];
        int part_v[kJoinFlight];
        each<0, kJoinFlight>([&](auto F) {
          constexpr int f = decltype(F)::value;
          const PartRows<D>* p = part(min(i0 + f * kTurns, parts - 1));  // the last one again adds nothing
          each<0, 4>([&](auto c) { x[f][decltype(c)::value] = *reinterpret_cast<const float4*>(p->o[chunk][decltype(c)::value][lane]); });
          part_ref[f] = p->ref[col], part_sum[f] = p->sum[col], part_v[f] = p->v_ref;
        });
        each<0, kJoinFlight>([&](auto F) {
          constexpr int f = decltype(F)::value;
          if (i0 + f * kTurns < parts) {
            const float m = part_of_ref(part_ref[f], ref), t = m * exact_power(part_v[f] - v);
            sum += m * part_sum[f];
            each<0, 4>([&](auto C) {
              constexpr int c = decltype(C)::value;
              o[4 * c] += x[f][c].x * t, o[4 * c + 1] += x[f][c].y * t;
              o[4 * c + 2] += x[f][c].z * t, o[4 * c + 3] += x[f][c].w * t;
            });
          }
        });
      }
    if (half == 0) sum_lds[turn][col] = sum;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<float4*>(o_lds[turn][c][lane]) = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
    __syncthreads();
    if (turn == 0) {
      for (int i = 1; i < min(parts, kTurns); ++i) {
        sum += sum_lds[i][col];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float4 x = *reinterpret_cast<const float4*>(o_lds[i][c][lane]);
          o[4 * c] += x.x, o[4 * c + 1] += x.y, o[4 * c + 2] += x.z, o[4 * c + 3] += x.w;
        }
      }
      write_rows<D>(a, r, chunk, o, ref, sum, v);
    }
    __syncthreads();  // before the next one's shares
  }
}

// The kernel for few rows takes calls of at most kFewRows rows of a head, and of more
// where they are small: its steps are 32 rows by 32 tokens, read from memory for each 32
// rows, where the other's start and parts cost about 25 us more.  Few / many, us, in
// steps times head_dim (a call is small up to kFewWork):
//   128 rows, 32 heads of 128, 4096 tokens: 21 / 38;  4 heads, 131072 tokens: 61 / 80
//   224 rows, 4 heads of 128: 4096 tokens (2^18.8) 19 / 27, 131072 tokens (2^23.8) 140 / 83
//   1024 rows, 1024 tokens, 32 heads of 128 (2^22): 44 / 53;  of 64 (2^21) 32 / 36
//   256 rows, 16384 tokens, 16 heads of 128 (2^23): 60 / 53
//   16 heads of 256: 1024 rows, 1024 tokens (2^22) 36 / 52;  4 heads, 448 rows, 16384 (2^22.8) 81 / 52
constexpr int kFewRows = 128;
constexpr double kFewWork = 4194304.0;

constexpr int many_groups(int D) { return D == 256 ? 1 : 2; }

// From the host's bounds on what the device holds.
bool few_rows(const AttendArgs& a) {
  const int64_t rows = (int64_t)std::min<int64_t>(a.b.max_new, a.T) * a.group;
  const double tiles = (double)((a.T * a.group + 31) / 32 + a.b.S - 1), blocks = (a.b.max_len + kBlock - 1) / kBlock;
  return rows <= kFewRows || tiles * a.c.kv_heads * blocks * a.c.head_dim <= kFewWork;
}

template <int D>
void launch(AttendArgs a, hipStream_t st) {
  constexpr int RG = many_groups(D), BM = kWaves * 32 * RG;
  if (!few_rows(a)) {
    a.parts = kManyParts;
    a.min_steps = 2;
    hipLaunchKernelGGL((k_attend_many<D, RG>), dim3(a.parts), dim3(kThreads), 0, st, a);
    hipLaunchKernelGGL((k_join<D, BM, 8, 8>), dim3(D / 32, BM / 32, a.parts / 8), dim3(8 * 64), 0, st, a);
  } else {
    a.parts = kNarrowParts;
    a.min_steps = std::min(kWaves, (a.b.max_len + kBlock - 1) / kBlock);  // a short tile's waves wait for nobody else's
    hipLaunchKernelGGL(k_attend_few<D>, dim3(a.parts), dim3(kThreads), 0, st, a);
    hipLaunchKernelGGL((k_join<D, 32, 4, 2>), dim3(D / 32, 1, a.parts / 2), dim3(4 * 64), 0, st, a);
  }
}

}  // namespace
}  // namespace dllm

extern "C" {

size_t dllm_cache_attention_workspace_bytes(const dllm_cache* cache, const dllm_cache_batch* batch, int32_t q_heads) {
  using namespace dllm;
  if (!cache_ok(cache) || !cache_supported(cache) || !batch_ok(batch) || q_heads < 1 || q_heads % cache->kv_heads != 0)
    return 0;
  const int D = cache->head_dim;
  const size_t few = parts_bytes(D, kNarrowParts, 1), many = parts_bytes(D, kManyParts, kWaves * many_groups(D));
  return batch->max_new * (int64_t)(q_heads / cache->kv_heads) > kFewRows ? (many > few ? many : few) : few;
}

dllm_status dllm_cache_attention(const dllm_cache* cache, const dllm_cache_batch* batch, int64_t T, const uint16_t* q,
                                 int64_t q_token, int64_t q_head, int32_t q_heads, float scale, int32_t causal,
                                 uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace dllm;
  if (!cache_ok(cache) || !batch_ok(batch) || !tokens_ok(T)) return DLLM_ERR_INVALID_ARG;
  if (q_heads < 1 || q_heads % cache->kv_heads != 0 || q_token < 0 || q_head < 0) return DLLM_ERR_INVALID_ARG;
  if (!(scale >= 1.17549435e-38f && scale <= 1.0e38f) || (causal != 0 && causal != 1)) return DLLM_ERR_INVALID_ARG;
  if (!cache_supported(cache) || T * (int64_t)q_heads >= ((int64_t)1 << 31) - 1024) return DLLM_ERR_UNSUPPORTED;
  if (T == 0) return DLLM_OK;
  if (!q || !out) return DLLM_ERR_INVALID_ARG;
  if (!stride_ok(q_token) || !stride_ok(q_head) || q_token % 8 != 0 || q_head % 8 != 0) return DLLM_ERR_UNSUPPORTED;
  if ((((uintptr_t)q | (uintptr_t)out) & 15u) != 0) return DLLM_ERR_UNSUPPORTED;
  const size_t need = dllm_cache_attention_workspace_bytes(cache, batch, q_heads);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u) != 0) return DLLM_ERR_WORKSPACE;
  const AttendArgs a = {*cache, *batch, T, q, q_token, q_head, q_heads, q_heads / cache->kv_heads, scale * kLog2e,
                        causal, out, lse, static_cast<char*>(workspace), 0, 0};
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (cache->head_dim == 64) launch<64>(a, st);
  else if (cache->head_dim == 128) launch<128>(a, st);
  else launch<256>(a, st);
  return hipGetLastError() == hipSuccess ? DLLM_OK : DLLM_ERR_HIP;
}

}  // extern "C"

// Attention over the 8-bit block cache (include/dllm_cache.h).
#include "cache_common.h"
#include "cache_schedule.h"
#include "cache_tiles.h"
#include "rotary_angle.h"

namespace dllm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kNarrowParts = 512;  // two workgroups to a compute unit

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

__device__ __forceinline__ Row row_of(const AttendArgs& a, const SeqView& q, int h, int row) {
  const int rows = q.rows * a.group;
  Row r;
  r.real = row < rows;
  row = min(row, rows - 1);
  r.tok = (int)((uint32_t)row / (uint32_t)a.group);
  r.head = h * a.group + (row - r.tok * a.group);
  r.out = (q.q0 + r.tok) * a.q_heads + r.head;
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

// What a state counts for when it is joined to others with reference `ref`
// and value scale `v_ref`.
__device__ __forceinline__ float share_of(float own_ref, float ref) {
  return own_ref == INFINITY ? 0.0f : __builtin_amdgcn_exp2f(own_ref - ref);
}

// ---- few rows: the waves of a workgroup share the keys ----------------------------------------------------------

// One wave's run along the cache: blocks first, first + kWaves, ... below
// `last` of one sequence and head.  Pages and scales of 64 blocks at a time
// are looked up by the wave's lanes together.
template <int D>
struct Walk {
  const AttendArgs& a;
  int s, h, base, last, have;  // base: the block that lane 0's look-up stands for
  int page, k_byte, v_byte;

  __device__ Walk(const AttendArgs& a_, int s_, int h_, int first, int last_, int len)
      : a(a_), s(s_), h(h_), base(first - 64), last(last_), have(len) {}

  // Block j's scale bytes, and its keys and values on their way; false if it
  // has no page.
  __device__ __forceinline__ bool fetch(int j, i32x4* k, i32x4* v, int& kb, int& vb) {
    const int lane = threadIdx.x & 63;
    if (j >= base + 64 || j < base) {
      base = j;
      const int b = base + lane;
      page = b < last ? page_of(a.b.table, a.b.table_blocks, a.c.pages, s, b) : -1;
      const int64_t at = block_of(a.c, max(page, 0), h);
      k_byte = a.c.k_scale[at];
      v_byte = a.c.v_scale[at];
    }
    const int i = j - base;
    const int p = __builtin_amdgcn_readlane(page, i);
    kb = __builtin_amdgcn_readlane(k_byte, i);
    vb = __builtin_amdgcn_readlane(v_byte, i);
    const int64_t at = block_of(a.c, max(p, 0), h) * (kBlock * D) + lane * 16;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) k[c] = *reinterpret_cast<const i32x4*>(a.c.k + at + c * 1024);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) v[c] = *reinterpret_cast<const i32x4*>(a.c.v + at + c * 1024);
    return p >= 0;
  }
};

// One workgroup: its stretch of the line, 32 rows at a time.  The four waves
// hold the same rows and take the blocks in turn, each straight from memory
// into registers with the next block in flight; at a tile's end their states
// are joined through LDS.
template <int D>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void k_attend_few(AttendArgs a) {
  __shared__ float o_lds[kWaves][D / 32][4][64][4];
  __shared__ float ref_lds[kWaves][32], sum_lds[kWaves][32];
  __shared__ int v_lds[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 31, half = lane >> 5;
  int w;
  int64_t left;
  Stretch at = find_stretch<32, kBlock>(a, &w, &left);
  if (threadIdx.x == 0) reinterpret_cast<Stretch*>(a.ws)[w] = at;
  while (left > 0) {
    const SeqView q = seq_view(a.b, a.T, at.s);
    const int steps = tile_steps<32, kBlock>(a, q, at.rt);
    const int n = (int)min((int64_t)(steps - at.begin), left);
    const int row0 = at.rt * 32;
    const Row r = row_of(a, q, at.h, row0 + col);
    Frag qf[D / 16];
    load_query<D>(qf, a.q + (q.q0 + r.tok) * a.q_token + (int64_t)r.head * a.q_head, half);
    // this column sees tokens [0, end); blocks below `whole` are seen whole by every column
    const int end = a.causal ? min(max(q.len - q.n + r.tok + 1, 0), q.len) : q.len;
    const int whole = (a.causal ? min(max(q.len - q.n + (int)((uint32_t)row0 / (uint32_t)a.group) + 1, 0), q.len) : q.len) / kBlock;
    const int last = min(at.begin + n, (q.len + kBlock - 1) / kBlock);
    Accumulator<D> acc;
    clear(acc);
    Walk<D> walk(a, at.s, at.h, at.begin + wave, last, q.len);
    i32x4 k[D / 32], v[D / 32];
    int kb, vb;
    int j = at.begin + wave;
    const int clean = min(last, whole);  // blocks below need no mask
    if (j < clean) {
      bool ok = walk.fetch(j, k, v, kb, vb);
      do {
        i32x4 k_next[D / 32], v_next[D / 32];
        int kb_next, vb_next;
        const bool ok_next = walk.fetch(min(j + kWaves, clean - 1), k_next, v_next, kb_next, vb_next);
        if (ok) {
          const f32x16 sc = scores<D>(qf, k, scale_value(kb));
          cover<D>(acc, largest(sc), a.scale2);
          Frag p[2];
          probabilities<D>(acc, sc, a.scale2, p);
          add_values<D>(acc, p, v, cover_values<D>(acc, vb));
        }
        ok = ok_next, kb = kb_next, vb = vb_next;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) k[c] = k_next[c], v[c] = v_next[c];
        j += kWaves;
      } while (j < clean);
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
    const float sum = acc.sum + other_half(acc.sum);
    if (half == 0) ref_lds[wave][col] = acc.ref, sum_lds[wave][col] = sum;
    if (lane == 0) v_lds[wave] = acc.v_ref;
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(o_lds[wave][c][i][lane]) =
            make_float4(acc.o[c][4 * i], acc.o[c][4 * i + 1], acc.o[c][4 * i + 2], acc.o[c][4 * i + 3]);
    __syncthreads();
    float ref = INFINITY, total = 0.0f, part[kWaves];
    int v_ref = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      const float x = ref_lds[i][col];
      ref = ref == INFINITY ? x : x == INFINITY ? ref : fmaxf(ref, x);
      v_ref = max(v_ref, v_lds[i]);
    }
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      const float x = share_of(ref_lds[i][col], ref);
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
      } else if (r.real) {
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

// ---- joining a tile's parts -------------------------------------------------------------------------------------

// One workgroup for each workgroup number w, 32-dim chunk and 32 rows of a tile: if w
// is the first to begin inside its tile, the tile is joined here from w - 1's
// last part and the first parts of w, w + 1, ...  The 16 waves take the parts in
// turn, and their shares are added in wave order.
constexpr int kJoinWaves = 16;

template <int D, int BM>
__global__ __launch_bounds__(kJoinWaves * 64) void k_join(AttendArgs a) {
  __shared__ float o_lds[kJoinWaves][4][64][4];
  __shared__ float ref_lds[kJoinWaves][32], sum_lds[kJoinWaves][32];
  __shared__ int v_lds[kJoinWaves];
  const int w = blockIdx.x, chunk = blockIdx.y, sub = blockIdx.z;
  const Stretch* all = reinterpret_cast<const Stretch*>(a.ws);
  const Stretch me = all[w];
  if (me.tile < 0 || me.begin == 0) return;
  if (w > 0 && all[w - 1].tile == me.tile && all[w - 1].begin > 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 31, half = lane >> 5;
  const SeqView q = seq_view(a.b, a.T, me.s);
  const int row0 = me.rt * BM + sub * 32;
  if (row0 >= q.rows * a.group) return;
  const Row r = row_of(a, q, me.h, row0 + col);
  // parts: w - 1's slot 1, then slot 0 of w .. w + more
  int more = 0;
  for (int i0 = w + 1;; i0 += 64) {
    const bool same = i0 + lane < a.parts && all[i0 + lane].tile == me.tile && all[i0 + lane].begin > 0;
    const uint64_t m = ~__ballot(same);
    more += m ? __ffsll((unsigned long long)m) - 1 : 64;
    if (m) break;
  }
  const int parts = more + 2;
  float ref = INFINITY, sum = 0.0f, o[16];
  int v_ref = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.0f;
  auto add = [&](float x_ref, float x_sum, int x_v, const float4* x) {
    const float to = ref == INFINITY ? x_ref : x_ref == INFINITY ? ref : fmaxf(ref, x_ref);
    const int v_to = max(v_ref, x_v);
    const float mine = share_of(ref, to), theirs = share_of(x_ref, to);
    sum = sum * mine + x_sum * theirs;
    const float m = mine * exact_power(v_ref - v_to), t = theirs * exact_power(x_v - v_to);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[4 * i] = o[4 * i] * m + x[i].x * t;
      o[4 * i + 1] = o[4 * i + 1] * m + x[i].y * t;
      o[4 * i + 2] = o[4 * i + 2] * m + x[i].z * t;
      o[4 * i + 3] = o[4 * i + 3] * m + x[i].w * t;
    }
    ref = to;
    v_ref = v_to;
  };
  for (int i = wave; i < parts; i += kJoinWaves) {
    const PartRows<D>* p = part_of<D>(a, BM / 32, i == 0 ? w - 1 : w + i - 1, i == 0 ? 1 : 0) + sub;
    float4 x[4];
    if (r.real) {
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = *reinterpret_cast<const float4*>(p->o[chunk][c][lane]);
      add(p->ref[col], p->sum[col], p->v_ref, x);
    }
  }
  if (half == 0) ref_lds[wave][col] = ref, sum_lds[wave][col] = sum;
  // v_ref may differ between the columns of a wave only where a column is not real
  const int v_wave = __builtin_amdgcn_readfirstlane(v_ref);
  if (lane == 0) v_lds[wave] = v_wave;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<float4*>(o_lds[wave][c][lane]) = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
  __syncthreads();
  if (wave != 0) return;
  for (int i = 1; i < min(parts, kJoinWaves); ++i) {
    float4 x[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = *reinterpret_cast<const float4*>(o_lds[i][c][lane]);
    add(ref_lds[i][col], sum_lds[i][col], v_lds[i], x);
  }
  write_rows<D>(a, r, chunk, o, ref, sum, v_ref);
}

template <int D>
void launch(AttendArgs a, hipStream_t st) {
  a.parts = kNarrowParts;
  a.min_steps = kWaves;
  hipLaunchKernelGGL(k_attend_few<D>, dim3(a.parts), dim3(kThreads), 0, st, a);
  hipLaunchKernelGGL((k_join<D, 32>), dim3(a.parts, D / 32, 1), dim3(kJoinWaves * 64), 0, st, a);
}

}  // namespace
}  // namespace dllm

extern "C" {

size_t dllm_cache_attention_workspace_bytes(const dllm_cache* cache, const dllm_cache_batch* batch, int32_t q_heads) {
  using namespace dllm;
  if (!cache_ok(cache) || !cache_supported(cache) || !batch_ok(batch) || q_heads < 1 || q_heads % cache->kv_heads != 0)
    return 0;
  return parts_bytes(cache->head_dim, kNarrowParts, 1);
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

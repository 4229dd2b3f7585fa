// Write into the 8-bit block cache (include/dllm_cache.h): rotation of the
// keys, the blocks' scales, rounding to e4m3 and the cache's byte order.
#include "cache_common.h"
#include "rotary_angle.h"

namespace dllm {
namespace {

constexpr int kThreads = 256;

// Scale byte of a block whose largest magnitude is `big`: the smallest e with
// big <= 448 * 2^e, 448 = 1.75 * 2^8 being e4m3's largest value, read off
// big's exponent and mantissa.
__device__ __forceinline__ int scale_byte(float big) {
  const uint32_t u = __float_as_uint(fminf(big, 3.4028235e38f));
  if (u == 0) return 0;
  const int x = (int)(u >> 23) - 127;  // a subnormal counts as 2^-127: below every scale that is chosen
  return x - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0) + 127;
}

// What a block's largest key may grow by: a rotated pair by sqrt 2 times the magnitude,
// the dimensions behind the rotated ones not at all.
__device__ __forceinline__ float key_gain(const dllm_rotary_plan& plan, int D) {
  const float g = 1.41421366f * plan.magnitude;
  return plan.rotary_dim < D ? fmaxf(g, 1.0f) : g;
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.4028235e38f ? a : 0.0f;
}

// e4m3 value of byte b
__device__ __forceinline__ float e4m3_float(uint32_t b) {
  return __builtin_amdgcn_cvt_pk_f32_fp8((int)b, false)[0];
}

__device__ __forceinline__ uint32_t float_e4m3(float x) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, x, 0, false) & 0xffu;
}

// The write for any strides, alignment and rotated dimensions.
// One workgroup: one touched block of one head.  Values pass through LDS as
// fp32 (rotated keys, values), because the cache's byte order of a block is
// not the order of the input rows.
//
// Bound by its 2-byte loads, and by angles that it computes for each head anew: 32768 tokens
// of 8 heads of 128 take 165 us where the kernel below takes 53.  It is the plain
// one that takes what the other does not: rotations in the layout HALF of other than a
// multiple of 32 dimensions (16 of 64, say), and rows that are not 16-byte aligned.
template <int D>
__global__ __launch_bounds__(kThreads) void k_write(dllm_cache c, dllm_cache_batch b, int64_t T,
                                                    const uint16_t* __restrict__ k, int64_t k_token, int64_t k_head,
                                                    const uint16_t* __restrict__ v, int64_t v_token, int64_t v_head,
                                                    const int32_t* __restrict__ start,
                                                    const int32_t* __restrict__ positions, dllm_rotary_plan plan) {
  const int s = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  const SeqView q = seq_view(b, T, s);
  const int64_t st = start[s];
  if (st < 0 || q.rows == 0) return;
  const int64_t blk64 = st / kBlock + blockIdx.x;
  if (blk64 * kBlock >= st + q.rows || blk64 >= b.table_blocks) return;
  const int blk = (int)blk64;
  const int page = page_of(b.table, b.table_blocks, c.pages, s, blk);
  if (page < 0) return;
  const int64_t at = block_of(c, page, h);
  __shared__ float x[kBlock][D + 1];
  __shared__ float top[kThreads / 64];
  const int half = plan.turns ? plan.rotary_dim / 2 : 0;

  for (int side = 0; side < 2; ++side) {  // keys, then values
    const uint16_t* src = side ? v : k;
    const int64_t ts = side ? v_token : k_token, hs = side ? v_head : k_head;
    uint8_t* dst = (side ? c.v : c.k) + at * (kBlock * D);
    uint8_t* scale = (side ? c.v_scale : c.k_scale) + at;
    float big = 0.0f;
    bool held = false;
    __syncthreads();
    for (int u = tid; u < kBlock * D; u += kThreads) {
      const int t = u / D, d = u - t * D;
      const int64_t slot = (int64_t)blk * kBlock + t;
      float val = 0.0f;
      if (slot >= st && slot < st + q.rows) {
        val = bf16_float(src[(q.q0 + (slot - st)) * ts + (int64_t)h * hs + d]);
        big = fmaxf(big, finite_abs(val));
      } else if (slot < q.len) {
        held = true;
      }
      x[t][d] = val;
    }
    for (int o = 32; o; o >>= 1) big = fmaxf(big, __shfl_xor(big, o));
    if ((tid & 63) == 0) top[tid >> 6] = big;
    const int any_held = __syncthreads_or(held);
    big = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    if (side == 0 && half) big *= key_gain(plan, D);
    const int had = stored_scale(scale, 0);
    int byte = max(scale_byte(big), any_held ? had : 0);
    byte = min(max(byte, DLLM_CACHE_SCALE_MIN), DLLM_CACHE_SCALE_MAX);
    const float inv = __uint_as_float((uint32_t)(254 - byte) << 23);  // 2^(127 - byte); 2^-127 at the largest byte
    const float inv2 = byte == 254 ? __uint_as_float(0x00400000u) : inv;
    // 2^(had - byte): 0 where it underflows, as the requantised value then does
    const float old = had - byte < -126 ? 0.0f : __uint_as_float((uint32_t)(had - byte + 127) << 23);
    if (side == 0 && half) {
      // rotate the new rows in place, one pair at a time
      for (int u = tid; u < kBlock * half; u += kThreads) {
        const int t = u / half, i = u - t * half;
        const int64_t slot = (int64_t)blk * kBlock + t;
        if (slot < st || slot >= st + q.rows) continue;
        const double2 cs = rotary_angle64(positions[q.q0 + (slot - st)], plan.turns[i], plan.magnitude);
        const int a = plan.layout == DLLM_ROTARY_HALF ? i : 2 * i;
        const int e = plan.layout == DLLM_ROTARY_HALF ? i + half : 2 * i + 1;
        const double xa = x[t][a], xb = x[t][e];
        x[t][a] = odd_float(xa * cs.x - xb * cs.y);
        x[t][e] = odd_float(xb * cs.x + xa * cs.y);
      }
    }
    __syncthreads();
    // every byte of the block in the cache's order, 4 to a thread
    for (int u = tid * 4; u < kBlock * D; u += kThreads * 4) {
      const uint32_t prev = *reinterpret_cast<const uint32_t*>(dst + u);
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = u + j, cc = p >> 10, hh = (p >> 9) & 1, r = (p >> 4) & 31, e = p & 15;
        const int t = side ? 8 * (e >> 2) + 4 * hh + (e & 3) : r;
        const int d = side ? 32 * cc + r : hh * (D / 2) + 16 * cc + e;
        const int64_t slot = (int64_t)blk * kBlock + t;
        uint32_t byte8 = 0;
        if (slot >= st && slot < st + q.rows)
          byte8 = float_e4m3(x[t][d] * inv2);
        else if (slot < q.len)
          byte8 = float_e4m3(e4m3_float((prev >> (8 * j)) & 0xffu) * old);
        word |= byte8 << (8 * j);
      }
      *reinterpret_cast<uint32_t*>(dst + u) = word;
    }
    if (tid == 0) *scale = (uint8_t)byte;
  }
}

struct WriteArgs {
  dllm_cache c;
  dllm_cache_batch b;
  int64_t T;
  const uint16_t *k, *v;
  int64_t k_token, k_head, v_token, v_head;
  const int32_t *start, *positions;
  dllm_rotary_plan plan;
  int heads;  // of a workgroup
};

__device__ __forceinline__ float largest_of(const i32x4& w) {  // of 8 bf16, what is not finite left out
  float big = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    big = fmaxf(big, finite_abs(__uint_as_float((uint32_t)w[i] << 16)));
    big = fmaxf(big, finite_abs(__uint_as_float((uint32_t)w[i] & 0xffff0000u)));
  }
  return big;
}

__device__ __forceinline__ int pack_e4m3(float a, float b, float c, float d, float scale) {
  i16x2 w = {0, 0};
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a, b, scale, false);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c, d, scale, true);
  return __builtin_bit_cast(int, w);
}

// 4 e4m3 bytes times `factor`, rounded again.
__device__ __forceinline__ int requantised(int w, float factor) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
  int x = __builtin_amdgcn_cvt_pk_fp8_f32(lo[0] * factor, lo[1] * factor, 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(hi[0] * factor, hi[1] * factor, x, true);
}

struct Scales {
  int byte;
  float scale, old;  // the new one's value; the old one's relative to it
};

__device__ __forceinline__ Scales scales_of(float big, int had, bool any_held) {
  Scales s;
  s.byte = min(max(max(scale_byte(big), any_held ? had : 0), DLLM_CACHE_SCALE_MIN), DLLM_CACHE_SCALE_MAX);
  s.scale = scale_value(s.byte);
  s.old = had - s.byte < -126 ? 0.0f : __uint_as_float((uint32_t)(had - s.byte + 127) << 23);
  return s;
}

// The write for 16-byte aligned rows and rotations whose pairs fall into pairs
// of 16-dim pieces: interleaved ones, and half layouts of a multiple of 32 dims.
// One workgroup of 2 D threads: one touched block, a.heads heads in turn.
// The first D threads have the keys: a token and two pieces of 16 dims that
// are each other's partners, whose 16 angles they keep in LDS for all heads
// (an angle costs some 40 fp64 operations, a rotated pair 4).  The others have
// the values: a token and 32 dims, turned into the cache's order through LDS.
//
// Bound by memory and the wait for it: 131072 tokens of 4 heads of 128, all rotated, 107 us
// for 404 MB (3.8 TB/s; a copy reaches 4.96), 4 workgroups to a compute unit; with one
// head's angles computed at a time 329 us, with 2 workgroups 164.
template <int D>
__global__ __launch_bounds__(2 * D, 4) void k_write_pieces(WriteArgs a) {
  constexpr int N = 2 * D, kPer = D / 32, kWaves = N / 64;  // kPer: threads of a token
  __shared__ __attribute__((aligned(16))) uint8_t rows[kBlock * D];
  uint8_t* const turned = rows;  // with arrays of their own, 40 KiB would hold three workgroups instead of four
  __shared__ float top[kWaves];
  __shared__ double2 cs[16][D];  // the key threads' angles: in registers they would halve the waves in flight
  const int s = blockIdx.z, tid = threadIdx.x;
  const SeqView q = seq_view(a.b, a.T, s);
  const int64_t st = a.start[s];
  if (st < 0 || q.rows == 0) return;
  const int64_t blk64 = st / kBlock + blockIdx.x;
  if (blk64 * kBlock >= st + q.rows || blk64 >= a.b.table_blocks) return;
  const int blk = (int)blk64;
  const int page = page_of(a.b.table, a.b.table_blocks, a.c.pages, s, blk);
  if (page < 0) return;
  const int h0 = blockIdx.y * a.heads, h1 = min(h0 + a.heads, a.c.kv_heads);
  // tokens of the block: [f0, f1) are written, others below `len` are held
  const int f0 = (int)max(st - (int64_t)blk * kBlock, (int64_t)0);
  const int f1 = (int)min(st + q.rows - (int64_t)blk * kBlock, (int64_t)kBlock);
  const int len = min(max(q.len - blk * kBlock, 0), kBlock);
  const bool any_held = min(f0, len) > 0 || len > f1;
  const bool key_side = tid < D;
  const int u = key_side ? tid : tid - D, t = u / kPer, part = u % kPer;
  const bool fresh = t >= f0 && t < f1, held = !fresh && t < len;
  const int64_t token = q.q0 + ((int64_t)blk * kBlock + t - st);  // only where fresh
  // key pieces: first dims p0, p1; pairs of this thread that are rotated (the first n_rot)
  const int r = a.plan.turns ? a.plan.rotary_dim : 0;
  const bool halves = a.plan.layout == DLLM_ROTARY_HALF;
  int p0 = 32 * part, p1 = p0 + 16, n_rot = min(max(r / 2 - 16 * part, 0), 16);
  if (halves) {
    n_rot = 32 * part < r ? 16 : 0;
    if (n_rot) p0 = 16 * part, p1 = r / 2 + 16 * part;
  }
  i32x4 x[4];  // 32 bf16
  auto load = [&](int h) {
    if (!fresh) return;
    if (key_side) {
      const i32x4* p = reinterpret_cast<const i32x4*>(a.k + token * a.k_token + h * a.k_head + p0);
      const i32x4* z = reinterpret_cast<const i32x4*>(a.k + token * a.k_token + h * a.k_head + p1);
      x[0] = p[0], x[1] = p[1], x[2] = z[0], x[3] = z[1];
    } else {
      const i32x4* p = reinterpret_cast<const i32x4*>(a.v + token * a.v_token + h * a.v_head + 32 * part);
      x[0] = p[0], x[1] = p[1], x[2] = p[2], x[3] = p[3];
    }
  };
  load(h0);
  if (fresh && n_rot) {  // half of them by the thread that has the same token's values
    const int pos = a.positions[token];
#pragma unroll 2
    for (int i = key_side ? 0 : 1; i < n_rot; i += 2) cs[i][u] = rotary_angle64(pos, a.plan.turns[16 * part + i], a.plan.magnitude);
  }
  // bytes of a value piece that are written and held: its tokens are 8 i + 4 half + 0 .. 3
  const int vhalf = (tid >> 5) & 1;
  i32x4 fresh_mask, held_mask;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t f = 0, o = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int y = 8 * i + 4 * vhalf + j;
      const bool is = y >= f0 && y < f1;
      f |= is ? 0xffu << (8 * j) : 0u;
      o |= !is && y < len ? 0xffu << (8 * j) : 0u;
    }
    fresh_mask[i] = (int)f, held_mask[i] = (int)o;
  }
  for (int h = h0; h < h1; ++h) {
    const int64_t at = block_of(a.c, page, h);
    float big = 0.0f;
    if (fresh) big = fmaxf(fmaxf(largest_of(x[0]), largest_of(x[1])), fmaxf(largest_of(x[2]), largest_of(x[3])));
    for (int o = 32; o; o >>= 1) big = fmaxf(big, __shfl_xor(big, o));
    if ((tid & 63) == 0) top[tid >> 6] = big;
    const int k_had = any_held ? stored_scale(a.c.k_scale, at) : 0, v_had = any_held ? stored_scale(a.c.v_scale, at) : 0;
    __syncthreads();
    float kbig = 0.0f, vbig = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves / 2; ++i) kbig = fmaxf(kbig, top[i]), vbig = fmaxf(vbig, top[kWaves / 2 + i]);
    if (r) kbig *= key_gain(a.plan, D);
    const Scales ks = scales_of(kbig, k_had, any_held), vs = scales_of(vbig, v_had, any_held);
    const i32x4 in[4] = {x[0], x[1], x[2], x[3]};
    if (h + 1 < h1) load(h + 1);
    auto value = [&](int e) { return __uint_as_float(e & 1 ? (uint32_t)in[e / 8][e % 8 / 2] & 0xffff0000u : (uint32_t)in[e / 8][e % 8 / 2] << 16); };
    if (key_side) {
      uint8_t* dst = a.c.k + at * (kBlock * D);
      i32x4* w0 = reinterpret_cast<i32x4*>(dst + ((p0 % (D / 2)) / 16 * 2 + p0 / (D / 2)) * 512 + t * 16);
      i32x4* w1 = reinterpret_cast<i32x4*>(dst + ((p1 % (D / 2)) / 16 * 2 + p1 / (D / 2)) * 512 + t * 16);
      i32x4 y0 = {0, 0, 0, 0}, y1 = {0, 0, 0, 0};
      if (fresh) {
        // four pairs at a time: dims 4 g + 0 .. 3 of both pieces, or dims 8 g + 0 .. 7 of the 32
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float ra[4], rb[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = 4 * g + i;
            ra[i] = halves ? value(e) : value(2 * e), rb[i] = halves ? value(16 + e) : value(2 * e + 1);
            if (e < n_rot) {
              const double da = ra[i], db = rb[i];
              const double2 c = cs[e][u];
              ra[i] = odd_float(da * c.x - db * c.y);
              rb[i] = odd_float(db * c.x + da * c.y);
            }
          }
          if (halves) {
            y0[g] = pack_e4m3(ra[0], ra[1], ra[2], ra[3], ks.scale);
            y1[g] = pack_e4m3(rb[0], rb[1], rb[2], rb[3], ks.scale);
          } else {
            const int lo = pack_e4m3(ra[0], rb[0], ra[1], rb[1], ks.scale), hi = pack_e4m3(ra[2], rb[2], ra[3], rb[3], ks.scale);
            (g < 2 ? y0 : y1)[g % 2 * 2] = lo;
            (g < 2 ? y0 : y1)[g % 2 * 2 + 1] = hi;
          }
          __builtin_amdgcn_sched_barrier(0);  // not all sixteen at once: their registers would spill
        }
      } else if (held) {
        y0 = *w0, y1 = *w1;
        if (ks.byte != k_had) {
#pragma unroll
          for (int i = 0; i < 4; ++i) y0[i] = requantised(y0[i], ks.old), y1[i] = requantised(y1[i], ks.old);
        }
      }
      *w0 = y0, *w1 = y1;
      if (tid == 0) a.c.k_scale[at] = (uint8_t)ks.byte;
    } else if (fresh) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        i32x4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          y[i] = pack_e4m3(value(16 * c + 4 * i), value(16 * c + 4 * i + 1), value(16 * c + 4 * i + 2),
                           value(16 * c + 4 * i + 3), vs.scale);
        *reinterpret_cast<i32x4*>(rows + t * D + 32 * part + 16 * c) = y;
      }
    }
    __syncthreads();
    {
      // 4 tokens by 4 dims: from a dword for each token to one for each dim
      const int quad = tid % (D / 4), g = tid / (D / 4);
      uint32_t y[4], z[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const uint32_t*>(rows + (4 * g + j) * D + 4 * quad);
      const uint32_t a01 = __builtin_amdgcn_perm(y[1], y[0], 0x05010400u), b01 = __builtin_amdgcn_perm(y[1], y[0], 0x07030602u);
      const uint32_t a23 = __builtin_amdgcn_perm(y[3], y[2], 0x05010400u), b23 = __builtin_amdgcn_perm(y[3], y[2], 0x07030602u);
      z[0] = __builtin_amdgcn_perm(a23, a01, 0x05040100u), z[1] = __builtin_amdgcn_perm(a23, a01, 0x07060302u);
      z[2] = __builtin_amdgcn_perm(b23, b01, 0x05040100u), z[3] = __builtin_amdgcn_perm(b23, b01, 0x07060302u);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = 4 * quad + j;
        *reinterpret_cast<uint32_t*>(turned + ((d / 32 * 2 + g % 2) * 32 + d % 32) * 16 + g / 2 * 4) = z[j];
      }
    }
    __syncthreads();
    {
      i32x4* w = reinterpret_cast<i32x4*>(a.c.v + at * (kBlock * D) + tid * 16);
      i32x4 y = *reinterpret_cast<const i32x4*>(turned + tid * 16) & fresh_mask;
      if (any_held) {
        i32x4 o = *w;
        if (vs.byte != v_had) {
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = requantised(o[i], vs.old);
        }
        y |= o & held_mask;
      }
      *w = y;
      if (tid == 0) a.c.v_scale[at] = (uint8_t)vs.byte;
    }
    // (the next head's first barrier stands between these reads of `turned` and its writes)
  }
}

template <int D>
void launch_write(const dllm_cache& c, const dllm_cache_batch& b, int64_t T, const uint16_t* k, int64_t kt, int64_t kh,
                  const uint16_t* v, int64_t vt, int64_t vh, const int32_t* start, const int32_t* positions,
                  const dllm_rotary_plan& plan, hipStream_t st) {
  const int64_t most = b.max_new < T ? b.max_new : T;
  const int64_t blocks = (most + kBlock - 2) / kBlock + 1;  // a run of n tokens touches at most this many
  const bool rows16 = ((kt | kh | vt | vh) & 7) == 0 && (((uintptr_t)k | (uintptr_t)v) & 15u) == 0;
  const bool pieces = !plan.turns || plan.layout == DLLM_ROTARY_INTERLEAVED || plan.rotary_dim % 32 == 0;
  // In pieces wherever they can be: one token of 64 sequences, 8 heads of 128, 9.3 us against
  // 12.6 in the general kernel, 2048 tokens of one 11.9 against 20.8, 32768 53 against 165.
  if (rows16 && pieces) {
    // heads of a workgroup: as many as leave some 4 workgroups for every compute unit
    int heads = c.kv_heads;
    while (heads > 1 && blocks * b.S * ((c.kv_heads + heads - 1) / heads) < 1024) heads = (heads + 1) / 2;
    const WriteArgs a = {c, b, T, k, v, kt, kh, vt, vh, start, positions, plan, heads};
    hipLaunchKernelGGL(k_write_pieces<D>, dim3((unsigned)blocks, (c.kv_heads + heads - 1) / heads, b.S), dim3(2 * D), 0,
                       st, a);
    return;
  }
  hipLaunchKernelGGL(k_write<D>, dim3((unsigned)blocks, c.kv_heads, b.S), dim3(kThreads), 0, st, c, b, T, k, kt, kh, v,
                     vt, vh, start, positions, plan);
}

}  // namespace
}  // namespace dllm

extern "C" dllm_status dllm_cache_write(const dllm_cache* cache, const dllm_cache_batch* batch, int64_t T,
                                        const uint16_t* k, int64_t k_token, int64_t k_head, const uint16_t* v,
                                        int64_t v_token, int64_t v_head, const int32_t* start,
                                        const int32_t* positions, const dllm_rotary_plan* plan, void* stream) {
  using namespace dllm;
  if (!cache_ok(cache) || !batch_ok(batch) || !tokens_ok(T)) return DLLM_ERR_INVALID_ARG;
  if (k_token < 0 || k_head < 0 || v_token < 0 || v_head < 0) return DLLM_ERR_INVALID_ARG;
  if (!cache_supported(cache)) return DLLM_ERR_UNSUPPORTED;
  if (plan && !rotary_plan_ok(plan, cache->head_dim)) return DLLM_ERR_INVALID_ARG;
  if (T == 0) return DLLM_OK;
  if (!k || !v || !start || (plan && !positions)) return DLLM_ERR_INVALID_ARG;
  if (!stride_ok(k_token) || !stride_ok(k_head) || !stride_ok(v_token) || !stride_ok(v_head)) return DLLM_ERR_UNSUPPORTED;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const dllm_rotary_plan none = {nullptr, 1.0f, 0, 0};
  const dllm_rotary_plan& p = plan ? *plan : none;
  const auto launch = cache->head_dim == 64 ? launch_write<64> : cache->head_dim == 128 ? launch_write<128> : launch_write<256>;
  launch(*cache, *batch, T, k, k_token, k_head, v, v_token, v_head, start, positions, p, st);
  return hipGetLastError() == hipSuccess ? DLLM_OK : DLLM_ERR_HIP;
}

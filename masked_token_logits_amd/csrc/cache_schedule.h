// How attention over the cache is dealt out to workgroups.
//
// The work is a line of steps: sequences in order, in each its key/value
// heads, in each its tiles of query rows, in each the steps along the cache
// that the tile's rows can see.  A fixed number of workgroups takes equal
// stretches of that line, so one long sequence among short ones, few rows
// with a long cache, and many rows with a short one all fill the chip, and
// the split follows the lengths on the device without the host knowing them.
// A tile that a stretch's end cuts is written in parts, which a second kernel
// joins in order: results do not depend on which workgroup ends first.
#pragma once

#include "cache_common.h"

namespace dllm {

struct AttendArgs {
  dllm_cache c;
  dllm_cache_batch b;
  int64_t T;
  const uint16_t* q;
  int64_t q_token, q_head;
  int q_heads, group;
  float scale2;  // scale * log2 e
  int causal;
  uint16_t* out;
  float* lse;
  char* ws;
  int parts;      // workgroups, a multiple of 8
  int min_steps;  // the shortest stretch worth a workgroup
};

// Where a workgroup's stretch begins: tile rt of head h of sequence s, whose
// first step is number `tile` on the line, at its step `begin`.  tile < 0: no
// work.  parts > 0: this is the first stretch to begin inside its tile, which
// is in that many parts, the first of them the end of the stretch before.
// Kept in the workspace for the kernel that joins the parts, with the
// sequence's first token and rows, so that it has one load to wait for.
struct Stretch {
  int64_t tile, q0;
  int s, h, rt, begin, rows, parts;
};

constexpr int kScheduleThreads = 256;

// floor(x / y) for 0 <= x < 2^53, y > 0: a quotient that is not whole is further
// below the next integer than fp64 rounds, and the division is a dozen
// instructions where the 64-bit integer one is a hundred.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) { return (int64_t)((double)x / (double)y); }

// Steps of KEYS tokens that row tile rt of BM rows (token * group + head of
// the group) needs; at least one, which writes what rows without a visible
// token get.
template <int BM, int KEYS>
__device__ __forceinline__ int tile_steps(const AttendArgs& a, const SeqView& q, int rt) {
  int seen = q.len;
  if (a.causal) {
    const uint32_t last = (uint32_t)(min((rt + 1) * BM, q.rows * a.group) - 1) / (uint32_t)a.group;
    seen = min(max(q.len - q.n + (int)last + 1, 0), q.len);
  }
  return max((seen + KEYS - 1) / KEYS, 1);
}

template <int BM>
__device__ __forceinline__ int row_tiles(const AttendArgs& a, const SeqView& q) {
  return (q.rows * a.group + BM - 1) / BM;
}

// sum over i in 0 .. n - 1 of floor((x i + y) / m), for x, y >= 0: the whole parts
// leave x, y < m, and then the points below a line are those beside it, with the
// axes exchanged (Euclid's steps).
__device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t x, int64_t y) {
  int64_t sum = 0;
  for (;;) {
    const int64_t whole_x = quotient(x, m), whole_y = quotient(y, m);
    sum += n * (n - 1) / 2 * whole_x + n * whole_y;
    x -= whole_x * m, y -= whole_y * m;
    const int64_t top = x * n + y;
    if (top < m) return sum;
    n = quotient(top, m);
    y = top - n * m;
    const int64_t was = m;
    m = x, x = was;
  }
}

// Steps of one head of a sequence.  Under a causal mask tile i < tiles - 1 whose last
// row sees c + l + 1 >= 1 tokens (c = len - n, l = floor(((i + 1) BM - 1) / group)) has
//   ceil((c + l + 1) / KEYS) = floor(((i + 1) BM - 1 + group (c + KEYS)) / (group KEYS)),
// the ones before it have 1.
template <int BM, int KEYS>
__device__ __forceinline__ int64_t head_steps(const AttendArgs& a, const SeqView& q) {
  const int tiles = row_tiles<BM>(a, q);
  if (tiles == 0) return 0;
  if (!a.causal) return (int64_t)tiles * tile_steps<BM, KEYS>(a, q, 0);
  const int64_t c = (int64_t)q.len - q.n, g = a.group;
  const int blind = c >= 0 ? 0 : (int)min((-c * g + BM) / BM - 1, (int64_t)tiles - 1), rest = tiles - 1 - blind;
  int64_t steps = blind + tile_steps<BM, KEYS>(a, q, tiles - 1);
  if (rest > 0) {
    const int64_t e = (c + KEYS) >> __builtin_ctz(KEYS), f = (c + KEYS) & (KEYS - 1);  // c + KEYS = e KEYS + f
    steps += e * rest + floor_sum(rest, g * KEYS, BM, (int64_t)BM * (blind + 1) - 1 + g * f);
  }
  return steps;
}

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ int64_t scan_wave(int64_t x) {
  const int lane = threadIdx.x & 63;
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Inclusive sum over the workgroup's 256 threads.
__device__ __forceinline__ int64_t scan(int64_t x, int64_t* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  x = scan_wave(x);
  __syncthreads();
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  for (int i = 0; i < wave; ++i) x += lds[i];
  return x;
}

// This workgroup's number w on the line, its stretch and the number of its
// steps, the same in every thread.  All 256 threads call it.  Workgroups go
// to the chip's 8 XCDs in turn, and neighbours on the line, which read the
// same keys, belong on one XCD's L2; where the line is too short for every
// workgroup they stay in turn, for else the first XCD would get it all.
// lds: 64 bytes of the kernel's LDS (handed in, for a kernel with loads that
// go straight to LDS must have one array of it: with more, the compiler waits for all
// such loads before every read).
template <int BM, int KEYS>
__device__ Stretch find_stretch(const AttendArgs& a, int64_t* lds, int* number, int64_t* steps) {
  int64_t& found_at = lds[kScheduleThreads / 64];
  int& found_s = *reinterpret_cast<int*>(lds + kScheduleThreads / 64 + 1);
  const int tid = threadIdx.x;
  int64_t total = 0, mine = 0, upto = 0;
  // Up to 64 sequences, where rows are few, every wave looks through by itself, one to
  // a lane: with no barrier, and no second look at the sequence that it finds (it saves 0.5
  // to 1 us; where rows are many the registers cost more).
  const bool by_wave = BM == 32 && a.b.S > 1 && a.b.S <= 64;
  SeqView lanes;
  if (by_wave) {
    const int lane = tid & 63;
    lanes = seq_view(a.b, a.T, min(lane, a.b.S - 1));
    mine = lane < a.b.S ? head_steps<BM, KEYS>(a, lanes) * a.c.kv_heads : 0;
    upto = scan_wave(mine);
    total = __shfl(upto, 63);
  } else if (a.b.S == 1) {
    total = head_steps<BM, KEYS>(a, seq_view(a.b, a.T, 0)) * a.c.kv_heads;
  } else {
    for (int s0 = 0; s0 < a.b.S; s0 += kScheduleThreads) {
      mine = s0 + tid < a.b.S ? head_steps<BM, KEYS>(a, seq_view(a.b, a.T, s0 + tid)) * a.c.kv_heads : 0;
      upto = scan(mine, lds);
      __syncthreads();
      if (tid == kScheduleThreads - 1) lds[0] = upto;
      __syncthreads();
      total += lds[0];
      __syncthreads();
    }
  }
  const int64_t parts = min((int64_t)a.parts, max(quotient(total + a.min_steps - 1, a.min_steps), (int64_t)1));
  const int w = parts == a.parts ? (int)(blockIdx.x % 8) * (a.parts / 8) + (int)blockIdx.x / 8 : (int)blockIdx.x;
  *number = w;
  Stretch r = {-1, 0, 0, 0, 0, 0, 0, 0};
  *steps = 0;
  if (w >= parts || total == 0) return r;
  const int64_t lo = quotient(total * w, parts), hi = quotient(total * (w + 1), parts);
  *steps = hi - lo;
  int64_t at = 0;  // the line up to sequence r.s
  SeqView q;
  if (by_wave) {
    const int found = __ffsll((unsigned long long)__ballot(upto - mine <= lo && lo < upto)) - 1;
    r.s = __builtin_amdgcn_readfirstlane(found);
    at = __shfl(upto - mine, found);
    q.q0 = __builtin_amdgcn_readlane((int)lanes.q0, r.s);
    q.n = __builtin_amdgcn_readlane(lanes.n, r.s);
    q.rows = __builtin_amdgcn_readlane(lanes.rows, r.s);
    q.len = __builtin_amdgcn_readlane(lanes.len, r.s);
  } else if (a.b.S > 1) {
    for (int s0 = 0; s0 < a.b.S; s0 += kScheduleThreads) {
      if (a.b.S > kScheduleThreads) {
        mine = s0 + tid < a.b.S ? head_steps<BM, KEYS>(a, seq_view(a.b, a.T, s0 + tid)) * a.c.kv_heads : 0;
        upto = scan(mine, lds);
      }
      __syncthreads();
      if (tid == 0) found_s = -1;
      if (tid == kScheduleThreads - 1) lds[0] = upto;
      __syncthreads();
      if (at + upto - mine <= lo && lo < at + upto) found_s = s0 + tid, found_at = at + upto - mine;
      __syncthreads();
      if (found_s >= 0) break;
      at += lds[0];
    }
    r.s = found_s;
    at = found_at;
  }
  if (!by_wave) q = seq_view(a.b, a.T, r.s);
  r.q0 = q.q0, r.rows = q.rows;
  const int64_t per_head = head_steps<BM, KEYS>(a, q);
  r.h = (int)quotient(lo - at, per_head);
  at += r.h * per_head;
  int n = tile_steps<BM, KEYS>(a, q, 0);
  if (!a.causal) {
    r.rt = (int)quotient(lo - at, n);
    at += (int64_t)r.rt * n;
  } else {
    while (lo >= at + n) {
      at += n;
      n = tile_steps<BM, KEYS>(a, q, ++r.rt);
    }
  }
  r.tile = at;
  r.begin = (int)(lo - at);
  // stretches w .. that begin before the tile's end, and the one before w
  if (r.begin > 0 && quotient(total * (w - 1), parts) <= at) r.parts = (int)quotient((at + n) * parts + total - 1, total) - w + 1;
  return r;
}

// The next tile on the line (whose last one ended before the work did).
template <int BM>
__device__ __forceinline__ void next_tile(const AttendArgs& a, Stretch& r, int steps_of_this) {
  r.tile += steps_of_this;
  r.begin = 0;
  if (++r.rt < row_tiles<BM>(a, seq_view(a.b, a.T, r.s))) return;
  r.rt = 0;
  if (++r.h < a.c.kv_heads) return;
  r.h = 0;
  do ++r.s;
  while (r.s < a.b.S - 1 && seq_view(a.b, a.T, r.s).rows == 0);
}

}  // namespace dllm

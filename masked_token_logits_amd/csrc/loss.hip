// Host side and row kernels of the masked cross entropy (include/dllm_loss.h).
//
// Forward is the readout's projection: the counted rows are compacted, the
// LM-head GEMM (for small products the loss's own) folds each row's logits into
// a running maximum and sum per vocabulary slice, and a wave for each row joins
// the slices and takes the target's logit.  Backward walks the vocabulary in
// pieces (loss_gemm.hip).
#include "dllm_loss.h"

#include <math.h>

#include <atomic>

#include "bf16.h"
#include "loss_internal.h"
#include "online_state.h"
#include "readout_internal.h"
#include "work_plan.h"

namespace dllm {
namespace {

__device__ __forceinline__ bool counts(uint8_t mask, int target, int V) { return mask != 0 && target >= 0 && target < V; }

// The positions that count, ascending, and zeros for the others' outputs.  One
// workgroup walks them in chunks, 16 positions to a thread; a thread's place in
// the list comes from the ballots of its count's bits and the waves before it.
// It also makes the persistent GEMM's plan, now that the number of rows is known.
// One launch, and a chunk's loads are all there is to wait for: 4 us for 512
// positions, 6 for 8192.
constexpr int kCompactThreads = 1024;

struct CompactArgs {
  const uint8_t* mask;
  const int32_t* targets;
  int L, V;
  PlanParams plan;
  float *losses, *lse;  // null: not wanted
  int32_t *idx, *ctr;
  uint16_t* zeros;      // 16 bytes of zeros for the products
};

__global__ __launch_bounds__(kCompactThreads) void k_loss_compact(CompactArgs a) {
  __shared__ unsigned long long best;
  __shared__ int wave_total[kCompactThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const unsigned long long below = lane ? ~0ull >> (64 - lane) : 0ull;
  const bool vector = (((uintptr_t)a.mask | (uintptr_t)a.targets) & 15u) == 0;
  int M = 0;
  for (int64_t base = 0; base < a.L; base += 16 * kCompactThreads) {
    const int64_t p0 = base + tid * 16;
    unsigned bits = 0;
    if (vector && p0 + 16 <= a.L) {
      const uint4 m = *reinterpret_cast<const uint4*>(a.mask + p0);
      const uint32_t w[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int4 t = *reinterpret_cast<const int4*>(a.targets + p0 + 4 * q);
        bits |= counts(w[q] & 0xFF, t.x, a.V) ? 1u << (4 * q) : 0u;
        bits |= counts(w[q] >> 8 & 0xFF, t.y, a.V) ? 2u << (4 * q) : 0u;
        bits |= counts(w[q] >> 16 & 0xFF, t.z, a.V) ? 4u << (4 * q) : 0u;
        bits |= counts(w[q] >> 24, t.w, a.V) ? 8u << (4 * q) : 0u;
      }
    } else {
      for (int j = 0; j < 16 && p0 + j < a.L; ++j) bits |= counts(a.mask[p0 + j], a.targets[p0 + j], a.V) ? 1u << j : 0u;
    }
    if (a.losses)
      for (int j = 0; j < 16 && p0 + j < a.L; ++j)
        if (!(bits >> j & 1)) a.losses[p0 + j] = a.lse[p0 + j] = 0.f;
    const int c = __popc(bits);
    int before = 0;
#pragma unroll
    for (int b = 0; b < 5; ++b) before += __popcll(__ballot((c >> b) & 1) & below) << b;
    if (lane == 63) wave_total[wave] = before + c;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kCompactThreads / 64; ++w) {
      before += w < wave ? wave_total[w] : 0;
      total += wave_total[w];
    }
    for (int o = M + before; bits; bits &= bits - 1) a.idx[o++] = (int)p0 + __ffs(bits) - 1;
    M += total;
    __syncthreads();
  }
  int S, n_rt;
  choose_plan(M, a.plan, &best, S, n_rt);
  if (tid == 0) {
    a.ctr[0] = M;
    a.ctr[3] = S;
    a.ctr[4] = n_rt;
    a.ctr[5] = 0;  // workgroups of k_loss_rows that have ended
    *reinterpret_cast<uint4*>(a.zeros) = make_uint4(0, 0, 0, 0);
  }
}

// The weighted sum of the rows' terms, in fp64 and a fixed order, by a workgroup.
template <int THREADS>
__device__ __forceinline__ void total_of(const float* terms, int M, float* loss) {
  __shared__ double part[THREADS / 64];
  double s = 0.0;
  for (int i0 = threadIdx.x; i0 < M; i0 += 8 * THREADS) {
    float t[8];  // loaded together; past the chip's own cache, since other chips' workgroups wrote them
#pragma unroll
    for (int k = 0; k < 8; ++k)
      t[k] = __hip_atomic_load(terms + min(i0 + k * THREADS, M - 1), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int k = 0; k < 8; ++k) s += i0 + k * THREADS < M ? (double)t[k] : 0.0;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int w = 0; w < THREADS / 64; ++w) t += part[w];
    *loss = (float)t;
  }
}

// The target's logit, summed as the forward product sums it: by its matrix
// instruction, in its order of K.  Where the target is almost sure, or logits are
// large, lse is this logit and little more, and the loss is their difference: from
// a sum in another order it had the roundings of both (a loss of 0.008 at a logit
// of 12, d 4096: 1e-3 of itself off, now 2e-5; at logits of 2^20 off by 2).
// Eight rows to a workgroup, one brought to LDS by each wave in pieces of 1024
// columns; one wave multiplies them, and the sums beside the diagonal are not
// used.  `first` is the stage that the wave's row begins with; `meanwhile` is done
// while the first piece is on its way.  The time is the chain of dependent
// instructions (d of 4096: 256 of them, 64 cycles each, 8 us) and, with many rows,
// how many workgroups a compute unit holds (k_loss_rows for 102 rows of 4096 17 us,
// with a sum in any order 10; 3900 of 3584 20 and 13; 7400 of 4096 38 and 20; by
// four rows to a workgroup 15, 28 and 44).
typedef short bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
constexpr int kDotRows = 8, kDotCols = 1024, kDotThreads = 64 * kDotRows;

struct DotLds {
  uint16_t w[kDotRows][kDotCols + 16], h[kDotRows][kDotCols + 16];  // rows 8 banks apart: 8 rows and 2 halves meet all 64
  float z[kDotRows];
};

template <class F>
__device__ __forceinline__ float target_logit(DotLds& lds, const uint16_t* w, const uint16_t* h, int d, int first, F meanwhile) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int stages = (d + kLossStep - 1) / kLossStep;
  uint4 x[2], y[2];
  auto load = [&](int q0) {  // stages q0 .. q0 + 15 in the row's order, zeros behind d and the last one
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int q = q0 + i * 8 + (lane >> 3), own = first + q < stages ? first + q : first + q - stages;
      const int k = own * kLossStep + (lane & 7) * 8;
      x[i] = y[i] = make_uint4(0, 0, 0, 0);
      if (q < stages && k < d) {
        x[i] = *reinterpret_cast<const uint4*>(w + k);
        y[i] = *reinterpret_cast<const uint4*>(h + k);
      }
    }
  };
  f32x16 acc = {};
  load(0);
  meanwhile();
  const int multiplier = (int)(blockIdx.x + blockIdx.x / 256) & 3;  // workgroups of a compute unit: each on another SIMD
  for (int q0 = 0; q0 < stages; q0 += kDotCols / kLossStep) {
    __syncthreads();  // the piece before has been read
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      *reinterpret_cast<uint4*>(&lds.w[wave][i * 512 + lane * 8]) = x[i];
      *reinterpret_cast<uint4*>(&lds.h[wave][i * 512 + lane * 8]) = y[i];
    }
    __syncthreads();
    load(q0 + kDotCols / kLossStep);
    if (wave == multiplier) {
      const uint16_t* fw = &lds.w[lane & (kDotRows - 1)][8 * (lane >> 5)];
      const uint16_t* fh = &lds.h[lane & (kDotRows - 1)][8 * (lane >> 5)];
      const int steps = min(stages - q0, kDotCols / kLossStep) * (kLossStep / 16);
      bf16x8 a[4], b[4];
      auto read = [&](int k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = *reinterpret_cast<const bf16x8*>(fw + 16 * (k + i));
          b[i] = *reinterpret_cast<const bf16x8*>(fh + 16 * (k + i));
        }
      };
      read(0);
      for (int k = 0; k < steps; k += 4) {  // the next four steps' operands are read behind these ones'
        bf16x8 c[4], e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          c[i] = a[i];
          e[i] = b[i];
        }
        read(min(k + 4, steps - 4));
        asm volatile("" ::: "memory");  // not moved to where they are used
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(c[i], e[i], acc, 0, 0, 0);
      }
    }
  }
  const int r = lane & 31;  // the lane's column; it has rows 0 .. 3, or 4 .. 7 behind lane 32, in its first results
  if (wave == multiplier && r < kDotRows && (lane >> 5) == (r >> 2)) {
    float z = acc[0];
#pragma unroll
    for (int i = 1; i < 4; ++i) z = (r & 3) == i ? acc[i] : z;
    lds.z[r] = z;
  }
  __syncthreads();
  return lds.z[wave];
}

// The stage of K that the forward product's tile with entry t begins with.
__device__ __forceinline__ int first_stage(bool small, int t, int d) {
  return small ? loss_few_start(t / kLossFewEntries, (d + kLossStep - 1) / kLossStep) : 0;
}

// lse - z for a logit z of the row, without lse's rounding: ln(s / 2^q) + m - z.
// The largest logit's own exponential in s is 2^q as the instruction rounds it, so
// what is left of their difference are the others'.
__device__ __forceinline__ float row_loss(const RowState& r, float lse, float z) {
  if (!(fabsf(r.m) < 0x1p29f)) return lse - z;
  const float top = __builtin_amdgcn_exp2f(fmaf(r.m, kLog2eF, -log2_ref(r.m)));
  return log1pf((r.s - top) / top) + (r.m - z);
}

// One wave for each row: the slices' partials joined, and the target's logit, which
// is a row of W for each.  With `loss` the last workgroup to end adds the terms, too.
__global__ __launch_bounds__(kDotThreads, 4) void k_loss_rows(const uint16_t* __restrict__ W,
                                                              const uint16_t* __restrict__ H, int d, int L,
                                                              const int32_t* __restrict__ targets,
                                                              const float* __restrict__ weights,
                                                              const int32_t* __restrict__ idx,
                                                              const int32_t* __restrict__ ctr, Partials p, bool records,
                                                              bool small, float* terms, float* __restrict__ losses,
                                                              float* __restrict__ lse, int32_t* __restrict__ ended,
                                                              float* __restrict__ loss) {
  __shared__ DotLds dot;
  const int M = min(ctr[0], L), slices = ctr[3];
  const int lane = threadIdx.x & 63;
  for (int row0 = blockIdx.x * kDotRows; row0 < M; row0 += gridDim.x * kDotRows) {
    const int row = row0 + (threadIdx.x >> 6), pos = idx[min(row, M - 1)], t = targets[pos];
    RowState r = row_state_empty();
    const float z = target_logit(dot, W + (int64_t)t * d, H + (int64_t)pos * d, d, first_stage(small, t, d), [&]() {
      const size_t base = (size_t)min(row, M - 1) * (size_t)slices;
      for (int j = lane; j < slices; j += 64) {
        RowState y = row_state_empty();
        if (records) {  // the few-row GEMM's (m, index, s, 0)
          const float4 rec = reinterpret_cast<const float4*>(p.m)[base + j];
          y.m = rec.x;
          y.s = rec.z;
        } else {
          y.m = p.m[base + j];
          y.s = p.s[base + j];
        }
        row_merge<false>(r, y);
      }
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) row_merge<false>(r, shfl_xor_state(r, off));
    });
    if (lane == 0 && row < M) {
      const float l = row_finish<false>(r).lse;
      // lse - z, before lse is rounded; the sum of exponentials may be a little below the target's own
      const float over = row_loss(r, l, z), x = over < 0.f ? 0.f : over;
      losses[pos] = x;
      lse[pos] = l;
      terms[row] = x * (weights ? weights[pos] : 1.f);
    }
  }
  if (!loss) return;
  __shared__ int last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();  // the workgroup's terms, before its arrival
    last = atomicAdd(ended, 1) == (int)gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (last) total_of<kDotThreads>(terms, M, loss);
}

__global__ __launch_bounds__(1024) void k_loss_total(const float* __restrict__ terms, const int32_t* __restrict__ ctr,
                                                     int L, float* __restrict__ loss) {
  total_of<1024>(terms, min(ctr[0], L), loss);
}

// What backward keeps of each counted row, in order: its hidden state and
// scalars, filled up with rows and columns of zeros; and zeros for the rows of
// d_hidden that do not count.  A wave takes a row (8192 positions of 3584, 3900
// counted: 27 us).
struct PrepareArgs {
  const uint16_t *W, *H;
  const uint8_t* mask;
  const int32_t* targets;
  const float *weights, *grad, *lse;
  const int32_t *idx, *ctr;
  int V, L, d, dp;
  bool small;  // the forward product's tiles
  uint16_t* rows;
  float *lse_of, *coef;
  int32_t* tgt;
  float *at_tgt, *left;
  uint16_t* d_hidden;
};

__global__ __launch_bounds__(kDotThreads, 4) void k_loss_prepare(PrepareArgs a) {
  const int M = min(a.ctr[0], a.L), Mp = (M + kLossStep - 1) / kLossStep * kLossStep, lane = threadIdx.x & 63;
  __shared__ DotLds dot;
  for (int i0 = blockIdx.x * kDotRows; i0 < max(a.L, Mp); i0 += gridDim.x * kDotRows) {
    const int i = i0 + (threadIdx.x >> 6), pos = M > 0 ? a.idx[min(i, M - 1)] : 0;
    auto rows = [&]() {
      if (i < Mp) {
        for (int c = 8 * lane; c < a.dp; c += 8 * 64) {
          uint4 u = make_uint4(0, 0, 0, 0);
          if (i < M && c < a.d) u = *reinterpret_cast<const uint4*>(a.H + (int64_t)pos * a.d + c);
          *reinterpret_cast<uint4*>(a.rows + (int64_t)i * a.dp + c) = u;
        }
      }
      if (a.d_hidden && i < a.L && !counts(a.mask[i], a.targets[i], a.V))
        for (int c = 8 * lane; c < a.d; c += 8 * 64)
          *reinterpret_cast<uint4*>(a.d_hidden + (int64_t)i * a.d + c) = make_uint4(0, 0, 0, 0);
    };
    float z = 0.f;
    int t = 0;
    if (i0 < M) {
      t = a.targets[pos];
      z = target_logit(dot, a.W + (int64_t)t * a.d, a.H + (int64_t)pos * a.d, a.d, first_stage(a.small, t, a.d), rows);
    } else {
      rows();
    }
    if (lane > 0 || i >= Mp) continue;
    const bool in = i < M;
    const float lse = in ? a.lse[pos] : 0.f, c = in ? (a.weights ? a.weights[pos] : 1.f) * (a.grad ? *a.grad : 1.f) : 0.f;
    // lse may be rounded to below a sure target's z
    const float over = z - lse, at = in ? c * expm1f(over > 0.f ? 0.f : over) : 0.f;
    a.lse_of[i] = lse * kLossPScale;
    a.coef[i] = fabsf(lse) < INFINITY ? c : NAN;
    a.tgt[i] = in ? t : -1;
    a.at_tgt[i] = at;
    a.left[i] = at - bf16_float(float_bf16(at));
  }
}

bool sizes_ok(int64_t V, int64_t d, int64_t L) {
  return V >= 1 && V < ((int64_t)1 << 31) - 1024 && d >= 1 && L >= 1 && L < ((int64_t)1 << 31) - 1024;
}
bool supported(int64_t d) { return d % 8 == 0 && d < ((int64_t)1 << 20); }

// The readout's few-row GEMM takes up to 32 rows: its slices, and four floats
// for each row's partial.
int64_t stream_slices(int64_t V) {
  const int64_t n = (V + kSmallBN - 1) / kSmallBN;
  return n < kMaxSmallSlices ? n : kMaxSmallSlices;
}

// Partials of the forward product: the persistent GEMM's plan, or a slice for
// each tile of few rows.
int64_t part_cap(int64_t V, int64_t L) {
  int64_t many = (L + kLargeBM - 1) / kLargeBM * kLargeBM * kMaxLargeSlices;
  // room for a plan that gives every compute unit an item, with one row tile, too
  // (102 rows, 126464 entries of 4096: 240 us; with 64 slices, for 256 rows, 540)
  if (many < kLargeBM * 1024) many = kLargeBM * 1024;
  if (L <= kSmallBM && many < 4 * kSmallBM * stream_slices(V)) many = 4 * kSmallBM * stream_slices(V);
  const int64_t few = loss_small(V, L) ? L * loss_few_slices(V) : 0;
  return many > few ? many : few;
}

struct Rows {
  int32_t *idx, *ctr;
  float* terms;
  Partials part;
  float *lse_of, *coef;
  int32_t* tgt;
  float *at_tgt, *left;
  uint16_t *zeros, *rows, *dz;
  float* acc;
  uint16_t* fix;
};

// Workspace of both directions; returns its size.
size_t carve(int64_t V, int64_t d, int64_t L, int64_t piece, uint8_t* base, Rows* r) {
  Parts parts = {base};
  auto take = [&](size_t bytes) { return parts.take(bytes); };
  Rows x = {};
  x.zeros = reinterpret_cast<uint16_t*>(take(16));
  x.idx = reinterpret_cast<int32_t*>(take((size_t)L * 4));
  x.ctr = reinterpret_cast<int32_t*>(take(16 * 4));
  if (piece == 0) {
    x.terms = reinterpret_cast<float*>(take((size_t)L * 4));
    x.part.m = reinterpret_cast<float*>(take((size_t)part_cap(V, L) * 4));
    x.part.a = reinterpret_cast<int32_t*>(take((size_t)part_cap(V, L) * 4));
    x.part.s = reinterpret_cast<float*>(take((size_t)part_cap(V, L) * 4));
  } else {
    const size_t rows = (size_t)loss_padded(L);
    x.lse_of = reinterpret_cast<float*>(take(rows * 4));
    x.coef = reinterpret_cast<float*>(take(rows * 4));
    x.tgt = reinterpret_cast<int32_t*>(take(rows * 4));
    x.at_tgt = reinterpret_cast<float*>(take(rows * 4));
    x.left = reinterpret_cast<float*>(take(rows * 4));
    x.rows = reinterpret_cast<uint16_t*>(take(rows * (size_t)loss_padded(d) * 2));
    x.dz = reinterpret_cast<uint16_t*>(take(rows * (size_t)piece * 2));
    x.fix = reinterpret_cast<uint16_t*>(take((size_t)(L < kLossFew ? L : kLossFew) * (size_t)d * 2));
    x.acc = reinterpret_cast<float*>(take((size_t)loss_shares(L, d, piece) * kLossTile * kLossTile * 4));
  }
  if (r) *r = x;
  return parts.size;
}

// A tile of dz is addressed by 32-bit byte offsets: 256 rows of a piece.
constexpr int64_t kMostPiece = (int64_t)1 << 22;

// The piece a call works with: as given, or about 1 GiB of dz, but at least
// 8192 entries, and never more than the vocabulary.
int64_t piece_of(int64_t V, int64_t L, int64_t piece) {
  if (piece == 0) {
    piece = ((int64_t)1 << 29) / L / 256 * 256;
    if (piece < 8192) piece = 8192;
  }
  const int64_t all = (V + 255) / 256 * 256;
  if (piece > kMostPiece) piece = kMostPiece;
  return piece < all ? piece : all;
}

dllm_status check(const dllm_loss* p) {
  if (!p || !sizes_ok(p->V, p->d, p->L)) return DLLM_ERR_INVALID_ARG;
  if (!supported(p->d)) return DLLM_ERR_UNSUPPORTED;
  if (!p->W_lm || !p->hidden || !p->mask || !p->targets) return DLLM_ERR_INVALID_ARG;
  if (!aligned(p->W_lm, 16) || !aligned(p->hidden, 16) || !aligned(p->targets, 4) || !aligned(p->weights, 4))
    return DLLM_ERR_UNSUPPORTED;
  return DLLM_OK;
}

// Whether an output shares memory with an input.
bool over_inputs(const dllm_loss* p, const void* out, size_t n) {
  const size_t L = (size_t)p->L, row = (size_t)p->d * 2;
  return overlaps(out, n, p->W_lm, (size_t)p->V * row) || overlaps(out, n, p->hidden, L * row) ||
         overlaps(out, n, p->mask, L) || overlaps(out, n, p->targets, L * 4) || overlaps(out, n, p->weights, L * 4);
}

// The current device's compute units, 0 where there is none; asked for once a device.
int device_cus() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 0;
  if (dev >= 0 && dev < kDevices && (cus = known[dev].load(std::memory_order_relaxed)) > 0) return cus;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
  if (dev >= 0 && dev < kDevices) known[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

unsigned grid_for(int64_t n, int64_t most) { return (unsigned)(n < most ? n : most); }

}  // namespace
}  // namespace dllm

extern "C" {

size_t dllm_loss_forward_workspace_bytes(int64_t V, int64_t d, int64_t L) {
  if (!dllm::sizes_ok(V, d, L) || !dllm::supported(d)) return 0;
  return dllm::carve(V, d, L, 0, nullptr, nullptr);
}

dllm_status dllm_loss_forward(const dllm_loss* p, float* loss, float* losses, float* lse, void* workspace,
                              size_t workspace_bytes, void* stream) {
  const dllm_status ok = dllm::check(p);
  if (ok != DLLM_OK) return ok;
  if (!loss || !losses || !lse) return DLLM_ERR_INVALID_ARG;
  if (!dllm::aligned(loss, 4) || !dllm::aligned(losses, 4) || !dllm::aligned(lse, 4)) return DLLM_ERR_UNSUPPORTED;
  const int64_t L = p->L;
  const size_t n = (size_t)L * 4, need = dllm::carve(p->V, p->d, L, 0, nullptr, nullptr);
  if (!workspace || workspace_bytes < need || !dllm::aligned(workspace, 256)) return DLLM_ERR_WORKSPACE;
  if (dllm::over_inputs(p, loss, 4) || dllm::over_inputs(p, losses, n) || dllm::over_inputs(p, lse, n) ||
      dllm::over_inputs(p, workspace, need) || dllm::overlaps(losses, n, lse, n) || dllm::overlaps(loss, 4, losses, n) ||
      dllm::overlaps(loss, 4, lse, n) || dllm::overlaps(workspace, need, loss, 4) ||
      dllm::overlaps(workspace, need, losses, n) || dllm::overlaps(workspace, need, lse, n))
    return DLLM_ERR_INVALID_ARG;
  const int cus = dllm::device_cus();
  if (cus <= 0) return DLLM_ERR_HIP;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  dllm::Rows r;
  dllm::carve(p->V, p->d, L, 0, reinterpret_cast<uint8_t*>(workspace), &r);
  // As the readout chooses it: up to 32 rows the few-row GEMM, more the persistent one where d is a multiple of 32
  // and its 32-bit offsets reach, else the streaming one; but small products have tiles of their own.
  // The streaming one is slower, more so with few rows, whose slices do not go by the count (50000 entries, us: 100
  // rows of 1000 149, of 1024 39; of 2040 270, of 2048 57; 4000 rows of 1000 586, of 1024 369; of 2040 1108, of 2048
  // 676).  All go by L, since the count stays on the device: 20 counted rows of 126464 x 4096 take 169 us as 20
  // positions, 197 among 1024 and 207 among 8192; of 4096 x 256 20, 20 and 26.
  const int64_t n_vt = (p->V + dllm::kLargeBN - 1) / dllm::kLargeBN, n_rt = (L + dllm::kLargeBM - 1) / dllm::kLargeBM;
  const bool persistent = p->d % dllm::kPersistBK == 0 && (int64_t)dllm::kPersistBN * p->d * 2 < ((int64_t)1 << 32) &&
                          (p->d % dllm::kPersistWideBK == 0 || L * p->d * 2 < ((int64_t)1 << 32));
  dllm::PlanParams plan = {};
  plan.tile_rows = dllm::kLargeBM;
  plan.n_vt = (int)n_vt;
  plan.grid = cus;
  plan.max_slices = 1024;
  plan.part_cap = dllm::part_cap(p->V, L);
  if (!persistent) {
    int64_t s = (4 * (int64_t)cus + n_rt - 1) / n_rt;
    if (s > dllm::kMaxLargeSlices) s = dllm::kMaxLargeSlices;
    plan.fixed_slices = (int)(s < n_vt ? s : n_vt);
  }
  const bool small = dllm::loss_small(p->V, L), stream_w = !small && L <= dllm::kSmallBM;
  if (small) plan.fixed_slices = (int)dllm::loss_few_slices(p->V);
  if (stream_w) plan.fixed_slices = (int)dllm::stream_slices(p->V);
  const dllm::CompactArgs ca = {p->mask, p->targets, (int)L, (int)p->V, plan, losses, lse, r.idx, r.ctr, r.zeros};
  hipLaunchKernelGGL(dllm::k_loss_compact, dim3(1), dim3(dllm::kCompactThreads), 0, st, ca);
  const dllm::LseArgs la = {p->W_lm, p->hidden, r.zeros, r.idx, r.ctr, r.part.m, r.part.s, (int)p->V, (int)p->d, (int)L};
  const int V = (int)p->V, d = (int)p->d;
  const hipError_t e = small      ? dllm::launch_loss_lse_small(la, st)
                       : stream_w ? dllm::launch_gemm_small(p->W_lm, p->hidden, d, V, r.idx, r.ctr, plan.fixed_slices, r.part, nullptr, st)
                       : persistent
                           ? dllm::launch_gemm_persistent(p->W_lm, p->hidden, d, V, r.idx, r.ctr, cus, r.part, st)
                           : dllm::launch_gemm_large(p->W_lm, p->hidden, d, V, r.idx, r.ctr, (int)n_rt, plan.fixed_slices, r.part, st);
  if (e != hipSuccess) return DLLM_ERR_HIP;
  // The last workgroup to end adds the terms of up to 1024 positions itself.  More are another kernel's: each
  // workgroup's arrival waits for its chip's cache to be written back.  Half of the positions counted, 4096 entries
  // of 256, us a call with the last workgroup and with a kernel: 64 positions 19 and 22, 512 20 and 23, 1024 22.0 and
  // 22.3, 1280 22.6 and 22.4, 1536 28 and 25, 4096 43 and 32.
  const bool ends = L <= 1024;
  hipLaunchKernelGGL(dllm::k_loss_rows, dim3(dllm::grid_for((L + dllm::kDotRows - 1) / dllm::kDotRows, 65536)),
                     dim3(dllm::kDotThreads), 0, st, p->W_lm, p->hidden, (int)p->d, (int)L, p->targets, p->weights, r.idx,
                     r.ctr, r.part, stream_w, small, r.terms, losses, lse, r.ctr + 5, ends ? loss : nullptr);
  if (!ends) hipLaunchKernelGGL(dllm::k_loss_total, dim3(1), dim3(1024), 0, st, r.terms, r.ctr, (int)L, loss);
  return hipGetLastError() == hipSuccess ? DLLM_OK : DLLM_ERR_HIP;
}

size_t dllm_loss_backward_workspace_bytes(int64_t V, int64_t d, int64_t L, int64_t piece) {
  if (!dllm::sizes_ok(V, d, L) || !dllm::supported(d) || piece < 0 || piece % 256 != 0) return 0;
  return dllm::carve(V, d, L, dllm::piece_of(V, L, piece), nullptr, nullptr);
}

dllm_status dllm_loss_backward(const dllm_loss* p, const float* lse, const float* grad, uint16_t* d_hidden,
                               uint16_t* d_W, int32_t accumulate, int64_t piece, void* workspace,
                               size_t workspace_bytes, void* stream) {
  const dllm_status ok = dllm::check(p);
  if (ok != DLLM_OK) return ok;
  if (!lse || (!d_hidden && !d_W) || (accumulate != 0 && accumulate != 1) || piece < 0 || piece % 256 != 0)
    return DLLM_ERR_INVALID_ARG;
  if (!dllm::aligned(lse, 4) || !dllm::aligned(grad, 4) || !dllm::aligned(d_hidden, 16) || !dllm::aligned(d_W, 16))
    return DLLM_ERR_UNSUPPORTED;
  const int64_t L = p->L, d = p->d, V = p->V;
  piece = dllm::piece_of(V, L, piece);
  const size_t need = dllm::carve(V, d, L, piece, nullptr, nullptr);
  if (!workspace || workspace_bytes < need || !dllm::aligned(workspace, 256)) return DLLM_ERR_WORKSPACE;
  const size_t nh = (size_t)L * (size_t)d * 2, nw = (size_t)V * (size_t)d * 2;
  const void* out[] = {d_hidden, d_W, workspace};
  const size_t size[] = {nh, nw, need};
  for (int i = 0; i < 3; ++i) {
    if (dllm::over_inputs(p, out[i], size[i]) || dllm::overlaps(out[i], size[i], lse, (size_t)L * 4) ||
        dllm::overlaps(out[i], size[i], grad, 4))
      return DLLM_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (dllm::overlaps(out[i], size[i], out[j], size[j])) return DLLM_ERR_INVALID_ARG;
  }
  const int cus = dllm::device_cus();
  if (cus <= 0) return DLLM_ERR_HIP;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  dllm::Rows r;
  dllm::carve(V, d, L, piece, reinterpret_cast<uint8_t*>(workspace), &r);
  dllm::PlanParams plan = {};
  plan.fixed_slices = 1;
  plan.tile_rows = dllm::kLargeBM;
  const dllm::CompactArgs ca = {p->mask, p->targets, (int)L, (int)V, plan, nullptr, nullptr, r.idx, r.ctr, r.zeros};
  hipLaunchKernelGGL(dllm::k_loss_compact, dim3(1), dim3(dllm::kCompactThreads), 0, st, ca);
  const int dp = (int)dllm::loss_padded(d), grid = cus < dllm::kLossGrid ? cus : dllm::kLossGrid;
  const dllm::PrepareArgs pa = {p->W_lm, p->hidden, p->mask,  p->targets, p->weights, grad,
                                lse,     r.idx,     r.ctr,    (int)V,     (int)L,     (int)d,
                                dp,      dllm::loss_small(V, L), r.rows,  r.lse_of,   r.coef,
                                r.tgt,   r.at_tgt,  r.left,   d_hidden};
  hipLaunchKernelGGL(dllm::k_loss_prepare, dim3(dllm::grid_for(dllm::loss_padded(L) / dllm::kDotRows, 65536)),
                     dim3(dllm::kDotThreads), 0, st, pa);
  dllm::GradArgs a = {};
  a.W = p->W_lm;
  a.zeros = r.zeros;
  a.rows = r.rows;
  a.idx = r.idx;
  a.ctr = r.ctr;
  a.lse = r.lse_of;
  a.coef = r.coef;
  a.tgt = r.tgt;
  a.at_tgt = r.at_tgt;
  a.left = r.left;
  a.dz = r.dz;
  a.acc = r.acc;
  a.fix = r.fix;
  a.d_hidden = d_hidden;
  a.d_W = d_W;
  a.ldz = piece;
  a.V = (int)V;
  a.d = (int)d;
  a.dp = dp;
  a.L = (int)L;
  a.accumulate = accumulate;
  for (int64_t v = 0; v < V; v += piece) {
    a.v0 = (int)v;
    a.n = (int)(V - v < piece ? V - v : piece);
    a.first = v == 0;
    if (dllm::launch_loss_dz(a, grid, st) != hipSuccess) return DLLM_ERR_HIP;
    if (d_hidden && dllm::launch_loss_d_hidden(a, grid, st) != hipSuccess) return DLLM_ERR_HIP;
    if (d_W && accumulate && dllm::launch_loss_targets(a, st) != hipSuccess) return DLLM_ERR_HIP;
    if (d_W && dllm::launch_loss_d_W(a, grid, st) != hipSuccess) return DLLM_ERR_HIP;
    if (d_W && !accumulate && dllm::launch_loss_targets(a, st) != hipSuccess) return DLLM_ERR_HIP;
  }
  if (d_W && accumulate && dllm::launch_loss_put(a, st) != hipSuccess) return DLLM_ERR_HIP;
  if (d_hidden && dllm::launch_loss_join(a, grid, st) != hipSuccess) return DLLM_ERR_HIP;
  return hipGetLastError() == hipSuccess ? DLLM_OK : DLLM_ERR_HIP;
}

}  // extern "C"

// The residual update between two blocks (include/dllm_norm.h):
//   u = N(y, post),  x' = x + scale gate u,  n = N(x', pre),
//   N(v, w) = w v r,  r = 1 / sqrt(mean(v^2) + eps),
// and its gradients.  With D = d_n pre and r, q the inverse roots of x' and y:
//   dx' = d_x_out + r (D - x' r^2 mean(D x'))       = d_x
//   du  = scale gate dx'
//   dy  = q (E - y q^2 mean(E y)),  E = du post     (du without post)
//   d_pre = sum d_n x' r,  d_post = sum du y q,  d_gate = sum scale dx' u
//
// A row stays in a workgroup's registers between its load and its store, so
// every operand passes once; the only exchange is the row's sums.
#include "dllm_norm.h"

#include <math.h>

#include <type_traits>

#include "bf16.h"

namespace dllm {
namespace {

// A workgroup's threads hold a row in pieces of 8 values, kPieces to a thread:
// THREADS is the smallest that fits, from 64 (up to 1024 values) to 512 (8192).
constexpr int kPieces = 2;

struct NormArgs {
  const uint16_t *x, *y, *pre, *post, *gate;
  int64_t T, group_rows;  // tokens, and tokens to a gate row
  int d;
  float eps, scale;
};

// Sums of N values over the workgroup, the same in every thread.  `slot`
// alternates between calls, so that one barrier serves each.
template <int THREADS, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*lds)[N], int slot) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v[i] += __shfl_xor(v[i], off);
  }
  if constexpr (THREADS > 64) {
    constexpr int W = THREADS / 64;
    float(*row)[N] = lds + slot * W;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) row[threadIdx.x >> 6][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v[i] += row[w][i];
    }
  }
}

// One workgroup to a row: the row is in registers when its first sum is known,
// so x, y, x' and n pass once and the time is their bytes (65536 tokens of 3584
// with both norms and a gate: 333 us, 5.6 TB/s; 32 tokens of 4096: 3.5 us, which
// is a row's loads and two rounds of sums).
__device__ __forceinline__ uint4 load8(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void store8(uint16_t* p, const uint4& u) { *reinterpret_cast<uint4*>(p) = u; }

template <int THREADS>
__global__ __launch_bounds__(THREADS) void k_residual_norm(NormArgs a, uint16_t* x_out, uint16_t* n_out) {
  __shared__ float lds[2 * (THREADS / 64)][1];
  const float per = 1.0f / (float)a.d;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const uint16_t* gate = a.gate ? a.gate + (t / a.group_rows) * a.d : nullptr;
    uint4 xu[kPieces], yu[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = 8 * (threadIdx.x + i * THREADS);
      xu[i] = yu[i] = make_uint4(0, 0, 0, 0);
      if (c < a.d) {
        xu[i] = load8(a.x + t * a.d + c);
        if (a.y) yu[i] = load8(a.y + t * a.d + c);
      }
    }
    float x[kPieces][8], u[kPieces][8];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      unpack8(xu[i], x[i]);
      unpack8(yu[i], u[i]);
    }
    if (a.y) {
      float q = a.scale;
      if (a.post) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) s[0] = fmaf(u[i][j], u[i][j], s[0]);
        group_sum<THREADS, 1>(s, lds, 0);
        q *= 1.0f / sqrtf(s[0] * per + a.eps);
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int c = 8 * (threadIdx.x + i * THREADS);
        if (c < a.d) {
          float w[8], g[8];
          if (a.post) unpack8(load8(a.post + c), w);
          if (gate) unpack8(load8(gate + c), g);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float z = u[i][j] * q;
            if (a.post) z *= w[j];
            if (gate) z *= g[j];
            x[i][j] += z;
          }
          store8(x_out + t * a.d + c, pack8(x[i]));
        }
      }
    }
    if (a.pre) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] = fmaf(x[i][j], x[i][j], s[0]);
      group_sum<THREADS, 1>(s, lds, 1);
      const float r = 1.0f / sqrtf(s[0] * per + a.eps);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int c = 8 * (threadIdx.x + i * THREADS);
        if (c < a.d) {
          float w[8];
          unpack8(load8(a.pre + c), w);
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] *= x[i][j] * r;
          store8(n_out + t * a.d + c, pack8(w));
        }
      }
    }
    if (THREADS > 64 && (!a.y || !a.post || !a.pre)) __syncthreads();  // one slot only: the next row's sums wait
  }
}

struct NormGrads {
  const uint16_t *d_n, *d_x_out;
  uint16_t *d_x, *d_y;
  float *d_gate;                  // written here where a run of tokens is one workgroup's
  float *part_pre, *part_post, *part_gate;  // [workgroups, d] else
  int64_t chunk;                  // tokens of a workgroup
  int chunks;                     // workgroups to a gate's run; 0: a workgroup has whole runs
  bool reads_y;                   // a gradient depends on y: through its norm or in the gate's sum
};

// A workgroup walks its tokens and keeps their share of the sums over tokens in
// registers; the next row's loads are on their way while one is worked on.  Six
// arrays pass once (32768 tokens of 3584 with both norms and a gate: 307 us with
// the sums, 4.6 TB/s, where a copy of as many bytes takes 5.0), and five where no
// gradient depends on y (32768 of 4096 with the norm before a block alone: 275 us,
// 4.9 TB/s; with y read 330).  POST, a norm behind the block, is the kernel's own
// constant: asked for within the loops it costs 1 percent at 3584 columns and
// 6 to 14 at 1024 and 256.
template <int THREADS, bool POST>
__global__ __launch_bounds__(THREADS) void k_residual_norm_backward(NormArgs a, NormGrads g) {
  __shared__ float lds[2 * (THREADS / 64)][3];
  // The weights and the gate of a thread's pieces, its own: loaded from memory
  // they would wait, in order, behind the next row's loads.
  __shared__ uint4 kept[3][kPieces][THREADS];
  auto keep = [&](int which, const uint16_t* p) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = 8 * (threadIdx.x + i * THREADS);
      if (c < a.d) kept[which][i][threadIdx.x] = load8(p + c);
    }
  };
  if (a.pre) keep(0, a.pre);
  if (POST) keep(1, a.post);
  const float per = 1.0f / (float)a.d;
  int64_t t0, t1;
  if (g.chunks > 0) {
    const int64_t run = blockIdx.x / g.chunks, k = blockIdx.x - run * g.chunks;
    t0 = run * a.group_rows + k * g.chunk;
    t1 = min(t0 + g.chunk, (run + 1) * a.group_rows);
  } else {
    t0 = blockIdx.x * g.chunk;
    t1 = min(t0 + g.chunk, a.T);
  }
  float s_pre[kPieces][8] = {}, s_post[kPieces][8] = {}, s_gate[kPieces][8] = {};
  int64_t run_end = g.chunks > 0 ? t1 : t0 + a.group_rows;
  uint4 xu[kPieces], yu[kPieces], nu[kPieces], du[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) xu[i] = yu[i] = nu[i] = du[i] = make_uint4(0, 0, 0, 0);
  auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = 8 * (threadIdx.x + i * THREADS);
      if (c < a.d) {
        const int64_t o = t * a.d + c;
        if (g.d_n) xu[i] = load8(a.x + o);
        if (g.reads_y) yu[i] = load8(a.y + o);
        if (g.d_n) nu[i] = load8(g.d_n + o);
        if (g.d_x_out) du[i] = load8(g.d_x_out + o);
      }
    }
  };
  if (t0 < t1) load(t0);
  int64_t run = t0 / a.group_rows;
  if (a.gate) keep(2, a.gate + run * a.d);
  const bool gate = a.gate != nullptr;
  for (int64_t t = t0; t < t1; ++t) {
    if (gate && g.chunks == 0 && t == run_end) {
      ++run;
      run_end += a.group_rows;
      keep(2, a.gate + run * a.d);
    }
    float x[kPieces][8], y[kPieces][8], dn[kPieces][8], dx[kPieces][8];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      unpack8(xu[i], x[i]);
      unpack8(yu[i], y[i]);
      unpack8(nu[i], dn[i]);
      unpack8(du[i], dx[i]);
    }
    if (t + 1 < t1) load(t + 1);  // on their way while this row is worked on
    // sums of x'^2, of D x' and of y^2
    float s[3] = {0.f, 0.f, 0.f};
    float w[kPieces][8];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = 8 * (threadIdx.x + i * THREADS);
      if (c < a.d && a.pre) {
        unpack8(kept[0][i][threadIdx.x], w[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[i][j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[0] = fmaf(x[i][j], x[i][j], s[0]);
        s[1] = fmaf(w[i][j] * dn[i][j], x[i][j], s[1]);
        s[2] = fmaf(y[i][j], y[i][j], s[2]);
      }
    }
    group_sum<THREADS, 3>(s, lds, 0);
    if (g.d_n) {
      const float r = 1.0f / sqrtf(s[0] * per + a.eps), m = s[1] * per * r * r;
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s_pre[i][j] = fmaf(dn[i][j], x[i][j] * r, s_pre[i][j]);
          dx[i][j] += r * (w[i][j] * dn[i][j] - x[i][j] * m);
        }
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = 8 * (threadIdx.x + i * THREADS);
      if (c < a.d) store8(g.d_x + t * a.d + c, pack8(dx[i]));
    }
    if (a.y) {
      const float q = POST ? 1.0f / sqrtf(s[2] * per + a.eps) : 1.0f;
      float e[3] = {0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int c = 8 * (threadIdx.x + i * THREADS);
        if (c < a.d) {
          float p[8], gt[8];
          if (POST) unpack8(kept[1][i][threadIdx.x], p);
          if (gate) unpack8(kept[2][i][threadIdx.x], gt);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float yq = y[i][j] * q;
            float z = a.scale * dx[i][j];
            if (gate) {
              s_gate[i][j] = fmaf(z, POST ? yq * p[j] : yq, s_gate[i][j]);
              z *= gt[j];
            }
            if (POST) {
              s_post[i][j] = fmaf(z, yq, s_post[i][j]);
              z *= p[j];
              e[0] = fmaf(z, y[i][j], e[0]);
            }
            dx[i][j] = z;
          }
        }
      }
      float m = 0.f;
      if (POST) {
        group_sum<THREADS, 3>(e, lds, 1);
        m = e[0] * per * q * q;
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int c = 8 * (threadIdx.x + i * THREADS);
        if (c < a.d) {
          if (POST) {
#pragma unroll
            for (int j = 0; j < 8; ++j) dx[i][j] = q * (dx[i][j] - y[i][j] * m);
          }
          store8(g.d_y + t * a.d + c, pack8(dx[i]));
        }
      }
      if (g.chunks == 0 && t + 1 == run_end) {
        if (g.d_gate) {
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            const int c = 8 * (threadIdx.x + i * THREADS);
            if (c < a.d) {
              float* o = g.d_gate + run * a.d + c;
#pragma unroll
              for (int j = 0; j < 8; ++j) o[j] = s_gate[i][j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) s_gate[i][j] = 0.f;
          }
        }
      }
    }
    if (THREADS > 64 && !(a.y && POST)) __syncthreads();  // one slot only: the next row's sums wait
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = 8 * (threadIdx.x + i * THREADS);
    if (c < a.d) {
      const int64_t o = (int64_t)blockIdx.x * a.d + c;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (g.part_pre) g.part_pre[o + j] = s_pre[i][j];
        if (g.part_post) g.part_post[o + j] = s_post[i][j];
        if (g.part_gate) g.part_gate[o + j] = s_gate[i][j];
      }
    }
  }
}

// out[run, c] = sum of part[run * count .. + count - 1, c]: sixteen waves take
// a sixteenth of the workgroups' shares each, in order (512 shares of 4096: 4 us).
constexpr int kSumWaves = 16;

struct Sums {
  const float* part[3];
  float* out[3];
  int count[3];
};

__global__ __launch_bounds__(64 * kSumWaves) void k_norm_sums(Sums s, int d) {
  __shared__ float lds[kSumWaves][64];
  const int which = blockIdx.z, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const int n = s.count[which], run = blockIdx.y;
  if (!s.part[which] || (which < 2 && run > 0)) return;
  const int lo = (int)((int64_t)n * wave / kSumWaves), hi = (int)((int64_t)n * (wave + 1) / kSumWaves);
  float v = 0.f;
  if (c < d) {
    const float* p = s.part[which] + (int64_t)run * n * d + c;
#pragma unroll 8
    for (int k = lo; k < hi; ++k) v += p[(int64_t)k * d];
  }
  lds[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && c < d) {
#pragma unroll
    for (int w = 1; w < kSumWaves; ++w) v += lds[w][lane];
    s.out[which][(int64_t)run * d + c] = v;
  }
}

// How the tokens of a backward call are dealt to workgroups.
struct Deal {
  int64_t groups;  // workgroups
  int64_t chunk;   // tokens of one
  int chunks;      // workgroups to a gate's run, 0 = a workgroup has whole runs
};

// Two workgroups to a compute unit, the best of 512, 1024 and 2048 workgroups for
// rows of 256 threads and more (32768 tokens of 3584: 307, 321 and 351 us).  Narrow
// rows, whose workgroups are one or two waves, would rather have more of them (of
// 2048: 213, 190 and 227; of 1024 164, 103 and 108; of 256 98, 56 and 41), short
// batches of them not always (4096 tokens of 512: 27, 25 and 29).  Two tokens to a
// workgroup where there are no more, as writing and adding the shares is then most
// of the time (509 tokens of 4096: 16.1 us; a token to each 18.8).
int64_t deal_to(int64_t T) { return T <= 512 ? (T + 1) / 2 : 512; }

Deal deal_tokens(int64_t T, int64_t runs) {  // T >= 1
  const int64_t n = runs > 0 ? runs : 1, rows = T / n;
  Deal x;
  const int64_t to = deal_to(T);
  if (n >= to) {
    const int64_t per = (n + to - 1) / to;
    x.chunk = per * rows;
    x.groups = (n + per - 1) / per;
    x.chunks = 0;
  } else {
    int64_t k = to / n;
    if (k > rows) k = rows;
    x.chunk = (rows + k - 1) / k;
    k = (rows + x.chunk - 1) / x.chunk;
    x.groups = n * k;
    x.chunks = (int)k;
  }
  return x;
}

dllm_status check_sizes(const dllm_norm* p, int64_t T, int64_t groups) {
  if (!p || T < 0 || groups < 0 || T >= ((int64_t)1 << 31)) return DLLM_ERR_INVALID_ARG;
  if (groups > 0 && (groups > (T > 1 ? T : 1) || T % groups != 0)) return DLLM_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || !isfinite(p->eps) || p->d < 1) return DLLM_ERR_INVALID_ARG;
  return p->d % 8 != 0 || p->d > DLLM_NORM_DIM_MAX ? DLLM_ERR_UNSUPPORTED : DLLM_OK;
}

dllm_status check_norm(const dllm_norm* p, int64_t T, const void* gate, int64_t groups) {
  const dllm_status st = check_sizes(p, T, groups);
  if (st != DLLM_OK) return st;
  if ((gate != nullptr) != (groups > 0)) return DLLM_ERR_INVALID_ARG;
  return aligned(p->pre, 16) && aligned(p->post, 16) && aligned(gate, 16) ? DLLM_OK : DLLM_ERR_UNSUPPORTED;
}

// Whether an output (n bytes) shares memory with one of the arrays; `same`
// may be exactly it.
struct Span {
  const void* p;
  size_t n;
};
template <int N>
bool clashes(const Span& out, const Span (&others)[N], const void* same = nullptr, const void* same2 = nullptr) {
  for (const Span& o : others) {
    if (o.p && (o.p == same || o.p == same2) && o.p == out.p && o.n == out.n) continue;
    if (overlaps(out.p, out.n, o.p, o.n)) return true;
  }
  return false;
}

static_assert(DLLM_NORM_DIM_MAX <= 512 * 8 * kPieces, "the widest workgroup holds a row");

template <class F>
void by_threads(int64_t d, F f) {
  if (d <= 64 * 8 * kPieces)
    f(std::integral_constant<int, 64>{});
  else if (d <= 128 * 8 * kPieces)
    f(std::integral_constant<int, 128>{});
  else if (d <= 256 * 8 * kPieces)
    f(std::integral_constant<int, 256>{});
  else
    f(std::integral_constant<int, 512>{});
}

}  // namespace
}  // namespace dllm

extern "C" {

dllm_status dllm_residual_norm(const dllm_norm* p, const uint16_t* x, const uint16_t* y, int64_t T,
                               const uint16_t* gate, int64_t groups, uint16_t* x_out, uint16_t* n, void* stream) {
  const dllm_status st = dllm::check_norm(p, T, gate, groups);
  if (st != DLLM_OK || T == 0) return st;  // empty arrays have no addresses to go by
  if ((p->pre != nullptr) != (n != nullptr) || (y != nullptr) != (x_out != nullptr)) return DLLM_ERR_INVALID_ARG;
  if ((!y && (p->post || gate)) || (!y && !p->pre) || (y && !isfinite(p->scale))) return DLLM_ERR_INVALID_ARG;
  if (!x) return DLLM_ERR_INVALID_ARG;
  if (!dllm::aligned(x, 16) || !dllm::aligned(y, 16) || !dllm::aligned(x_out, 16) || !dllm::aligned(n, 16))
    return DLLM_ERR_UNSUPPORTED;
  const size_t rows = (size_t)T * (size_t)p->d * 2, one = (size_t)p->d * 2;
  const dllm::Span in[] = {{x, rows}, {y, rows}, {gate, (size_t)groups * one}, {p->pre, one}, {p->post, one}};
  if (dllm::clashes({x_out, rows}, in, x) || dllm::clashes({n, rows}, in) || dllm::overlaps(n, rows, x_out, rows))
    return DLLM_ERR_INVALID_ARG;
  const dllm::NormArgs a = {x, y, p->pre, p->post, gate, T, groups > 0 ? T / groups : T, (int)p->d, p->eps, p->scale};
  const dim3 grid((unsigned)(T < (1 << 20) ? T : 1 << 20));
  dllm::by_threads(p->d, [&](auto threads) {
    constexpr int N = decltype(threads)::value;
    hipLaunchKernelGGL(dllm::k_residual_norm<N>, grid, dim3(N), 0, reinterpret_cast<hipStream_t>(stream), a, x_out, n);
  });
  return hipGetLastError() == hipSuccess ? DLLM_OK : DLLM_ERR_HIP;
}

size_t dllm_residual_norm_backward_workspace_bytes(const dllm_norm* p, int64_t T, int64_t groups) {
  if (dllm::check_sizes(p, T, groups) != DLLM_OK) return 0;
  const dllm::Deal deal = dllm::deal_tokens(T > 0 ? T : 1, groups);
  return (size_t)3 * (size_t)deal.groups * (size_t)p->d * sizeof(float) + 256;
}

dllm_status dllm_residual_norm_backward(const dllm_norm* p, const uint16_t* x, const uint16_t* y, int64_t T,
                                        const uint16_t* gate, int64_t groups, const uint16_t* d_n,
                                        const uint16_t* d_x_out, uint16_t* d_x, uint16_t* d_y, float* d_pre,
                                        float* d_post, float* d_gate, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  const dllm_status st = dllm::check_norm(p, T, gate, groups);
  if (st != DLLM_OK || T == 0) return st;  // empty arrays have no addresses to go by
  if ((p->pre != nullptr) != (d_n != nullptr) || (y != nullptr) != (d_y != nullptr)) return DLLM_ERR_INVALID_ARG;
  if ((!d_n && !d_x_out) || (!y && (p->post || gate)) || (y && !isfinite(p->scale))) return DLLM_ERR_INVALID_ARG;
  if ((d_pre && !p->pre) || (d_post && !p->post) || (d_gate && !gate)) return DLLM_ERR_INVALID_ARG;
  if (!x || !d_x) return DLLM_ERR_INVALID_ARG;
  const void* all[] = {x, y, d_n, d_x_out, d_x, d_y, d_pre, d_post, d_gate};
  for (const void* q : all)
    if (!dllm::aligned(q, 16)) return DLLM_ERR_UNSUPPORTED;
  const size_t rows = (size_t)T * (size_t)p->d * 2, one = (size_t)p->d * 2;
  const size_t need = dllm_residual_norm_backward_workspace_bytes(p, T, groups);
  if (!workspace || workspace_bytes < need || !dllm::aligned(workspace, 256)) return DLLM_ERR_WORKSPACE;
  const dllm::Span in[] = {{x, rows},   {y, rows},     {gate, (size_t)groups * one}, {p->pre, one},
                           {p->post, one}, {d_n, rows}, {d_x_out, rows}};
  const dllm::Span out[] = {{d_x, rows},       {d_y, rows}, {d_pre, 2 * one}, {d_post, 2 * one}, {d_gate, 2 * (size_t)groups * one},
                            {workspace, need}};
  for (int i = 0; i < 6; ++i) {
    const void* same = i == 0 ? (const void*)d_x_out : i == 1 ? (const void*)y : nullptr;
    if (dllm::clashes(out[i], in, same, i == 0 ? d_n : nullptr)) return DLLM_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (dllm::overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return DLLM_ERR_INVALID_ARG;
  }
  const dllm::NormArgs a = {x, y, p->pre, p->post, gate, T, groups > 0 ? T / groups : T, (int)p->d, p->eps, p->scale};
  const dllm::Deal deal = dllm::deal_tokens(T, groups);
  float* part = reinterpret_cast<float*>(workspace);
  const int64_t size = deal.groups * p->d;
  const bool whole = deal.chunks == 0;
  const dllm::NormGrads g = {d_n, d_x_out, d_x, d_y, whole ? d_gate : nullptr, d_pre ? part : nullptr,
                             d_post ? part + size : nullptr, !whole && d_gate ? part + 2 * size : nullptr, deal.chunk,
                             deal.chunks, p->post || d_gate};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  dllm::by_threads(p->d, [&](auto threads) {
    constexpr int N = decltype(threads)::value;
    if (p->post)
      hipLaunchKernelGGL((dllm::k_residual_norm_backward<N, true>), dim3((unsigned)deal.groups), dim3(N), 0, s, a, g);
    else
      hipLaunchKernelGGL((dllm::k_residual_norm_backward<N, false>), dim3((unsigned)deal.groups), dim3(N), 0, s, a, g);
  });
  if (hipGetLastError() != hipSuccess) return DLLM_ERR_HIP;
  if (g.part_pre || g.part_post || g.part_gate) {
    const dllm::Sums sums = {{g.part_pre, g.part_post, g.part_gate},
                             {d_pre, d_post, d_gate},
                             {(int)deal.groups, (int)deal.groups, deal.chunks}};
    const dim3 grid((unsigned)((p->d + 63) / 64), (unsigned)(g.part_gate ? groups : 1), g.part_gate ? 3 : 2);
    hipLaunchKernelGGL(dllm::k_norm_sums, grid, dim3(64 * dllm::kSumWaves), 0, s, sums, (int)p->d);
  }
  return hipGetLastError() == hipSuccess ? DLLM_OK : DLLM_ERR_HIP;
}

}  // extern "C"

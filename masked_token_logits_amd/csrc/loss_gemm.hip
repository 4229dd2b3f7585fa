// The three products of the loss's backward pass (include/dllm_loss.h), for
// one piece of the vocabulary:
//   dz[i, v]   = coef_i (exp(h_i . W_v - lse_i) - [v = t_i])
//   acc[i, c] += sum_v dz[i, v] W[v, c]
//   d_W[v, c]  = sum_i dz[i, v] h[i, c]
//
// MI355X mapping
//   * 256 x 256 tiles, one workgroup of four waves to a compute unit, 128 x 128
//     to a wave in 16 v_mfma_f32_32x32x16_bf16 a 16-deep K step.  The matrix
//     instruction's first operand is the side whose index runs along the
//     output's rows in memory (W's entries for dz, the hidden columns for the
//     gradients), so a lane stores runs of four neighbours.
//   * Both operands reach LDS by global->LDS DMA in 64-deep stages, 32 KiB each,
//     through a ring of five operand slots (all 160 KiB).  The stage's schedule is
//     the readout's persistent GEMM's: the second operand's tile of stage
//     q + 2 is queued in K steps 0 and 1, one barrier comes after K step 2, then
//     the first operand's tile of q + 2 while K step 3 runs.
//   * What K runs along in memory differs: the logits' product has K contiguous
//     on both sides, d_hidden's has W by rows of K, d_W's has both by rows of K.
//     Such operands are staged as they lie, [64 of K][256], and read by
//     ds_read_b64_tr_b16, which hands each lane four consecutive K of its
//     column: no transposed copy of W, dz or the hidden states exists.
#include <math.h>

#include <type_traits>

#include "bf16.h"
#include "loss_internal.h"
#include "online_state.h"
#include "persistent_sched.h"

namespace dllm {
namespace {

typedef short bf16x8 __attribute__((ext_vector_type(8)));
typedef short bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
#define LDS_AS __attribute__((address_space(3)))

constexpr int BT = kLossTile, BK = kLossStep, NT = 256;
constexpr int OPT = BT * BK;   // elements of an operand's tile
constexpr int SLOTS = 5;
constexpr int DMAS = 8;        // of a wave, for an operand's tile: 64 lanes x 16 bytes each
static_assert(SLOTS * OPT * 2 == 160 * 1024 && DMAS * 4 * 1024 == OPT * 2, "the ring fills LDS");

// Four K of a lane's column (see Side<true>).  The ring is only a parameter so
// that the restricted pointers tell the compiler that no DMA in flight writes
// what is read here: without that it drains them all before each of these
// reads.  The waits that make it true are stage_sync's.
__device__ __forceinline__ bf16x4 read_tr(LDS_AS const uint16_t* __restrict__ p, LDS_AS uint16_t* __restrict__ ring) {
  (void)ring;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS bf16x4*)p);
}

// An operand in memory, [256 rows][K] or, by rows of K, [K][256 columns].
// Sources outside it are drawn to its last row or piece: valid memory, whose
// products are not stored or meet zeros.
struct Operand {
  const uint16_t* p;  // the tile's first element at the first K
  int64_t ld;         // elements from row to row
  int64_t rows;       // rows that exist from there on (of K, for an operand by rows of K)
  int64_t cols;       // columns that exist from there on (of K, where K is contiguous)
  const uint16_t* zeros;
};

// One operand's way into LDS and from there into fragments.  TAIL: K is
// contiguous and its last stage reaches behind the row; zeros are read there.
template <bool BY_K, bool TAIL>
struct Side;

// K contiguous.  LDS [256][64]: row r holds its eight 16-byte pieces at piece ^
// ((r >> 1) & 7), so that the 16 lanes of a ds_read_b128 phase meet 64 banks.
template <bool TAIL>
struct Side<false, TAIL> {
  uint32_t off[DMAS];
  const char *base, *zeros;
  int lane_off, swz, col, cols;
  __device__ __forceinline__ void start(const Operand& o, int wave, int lane) {
    base = reinterpret_cast<const char*>(o.p);
    zeros = reinterpret_cast<const char*>(o.zeros);
    cols = (int)o.cols;
    const int r0 = wave * 8 + (lane >> 3), piece = (lane & 7) ^ ((r0 >> 1) & 7);
    col = piece * 8;
    const int last = (int)min(o.rows - 1, (int64_t)(BT - 1));
#pragma unroll
    for (int j = 0; j < DMAS; ++j) off[j] = ((uint32_t)min(r0 + 32 * j, last) * (uint32_t)o.ld + (uint32_t)col) * 2u;
    swz = ((lane & 31) >> 1) & 7;
    lane_off = (lane & 31) * BK;
  }
  __device__ __forceinline__ const char* source(int j, int k0) const {
    const char* p = base + (size_t)k0 * 2u + off[j];
    if constexpr (TAIL) p = k0 + col < cols ? p : zeros;
    return p;
  }
  __device__ __forceinline__ bf16x8 frag(const uint16_t* tile, int block, int kk, int lane) const {
    const int piece = ((kk * 2 + (lane >> 5)) ^ swz) * 8;
    return *reinterpret_cast<const bf16x8*>(tile + block * 32 * BK + lane_off + piece);
  }
};

// By rows of K.  LDS [64][256]: row k holds its eight 64-byte granules (32
// columns) at granule ^ (k & 3).  A 16-lane group of ds_read_b64_tr_b16 reads
// four rows of K, 16 columns of each, and gives lane i column i, four
// consecutive K; the swizzle puts the four rows of both groups of a phase into
// 64 different banks.
template <bool TAIL>
struct Side<true, TAIL> {
  static_assert(!TAIL, "rows of K are drawn to the last one");
  const char* base;
  int64_t ld2, rows;
  uint32_t k_off, col_off;
  int lane_off, sw;
  __device__ __forceinline__ void start(const Operand& o, int wave, int lane) {
    base = reinterpret_cast<const char*>(o.p);
    ld2 = o.ld * 2;
    rows = o.rows;
    const int k = wave * 2 + (lane >> 5), granule = ((lane & 31) >> 2) ^ (k & 3);
    k_off = (uint32_t)k * (uint32_t)ld2;
    col_off = (uint32_t)min((int64_t)(granule * 32 + (lane & 3) * 8), o.cols - 8) * 2u;
    sw = (lane & 15) >> 2;
    lane_off = (8 * (lane >> 5) + sw) * BT + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  }
  __device__ __forceinline__ const char* source(int j, int k0) const {
    const uint32_t last = (uint32_t)min(rows - 1 - k0, (int64_t)(BK - 1)) * (uint32_t)ld2;
    return base + (size_t)k0 * (size_t)ld2 + (min(k_off + (uint32_t)(8 * j) * (uint32_t)ld2, last) + col_off);
  }
  __device__ __forceinline__ bf16x8 frag(const uint16_t* tile, int block, int kk, int) const {
    LDS_AS uint16_t* ring = (LDS_AS uint16_t*)tile;
    LDS_AS const uint16_t* p = ring + lane_off + ((block ^ sw) * 32) + kk * 16 * BT;
    const bf16x4 lo = read_tr(p, ring), hi = read_tr(p + 4 * BT, ring);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// One tile: acc = sum over K stages of first (256) x second (256), and then
// epi(fr, fv, j, z): values z[0..3] of the second's index (wr + 2 fr) * 32 +
// lane % 32 and the first's index wv * 128 + fv * 32 + 8 j + 4 (lane / 32) + 0..3.
// nb: 32-blocks of the second operand that are wanted.
template <bool A_BY_K, bool A_TAIL, bool B_BY_K, class Epi>
__device__ __forceinline__ void tile_product(uint16_t* lds, const Operand& oa, const Operand& ob, int stages, int nb,
                                             Epi epi) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave >> 1, wv = wave & 1;
  Side<A_BY_K, A_TAIL> sa;
  Side<B_BY_K, false> sb;
  sa.start(oa, wave, lane);
  sb.start(ob, wave, lane);

  // Operand tiles alternate through the ring: the second's of stage q goes to
  // slot 2q % 5, the first's to (2q + 1) % 5.  Stages behind the last read the
  // first ones again and are never used.
  const int K = stages * BK;
  int a_k0 = 0, a_slot = 1, b_k0 = 0, b_slot = 0;
  auto next_slot = [](int s) { return s + 2 >= SLOTS ? s + 2 - SLOTS : s + 2; };
  auto dma = [&](const char* src, int slot, int j) {
    __builtin_amdgcn_global_load_lds((const void*)src, (LDS_AS void*)(lds + slot * OPT + (wave + 4 * j) * 512), 16, 0, 0);
  };
  auto issue_a = [&](int j) { dma(sa.source(j, a_k0), a_slot, j); };
  auto issue_b = [&](int j) { dma(sb.source(j, b_k0), b_slot, j); };
  auto advance_a = [&]() {
    a_slot = next_slot(a_slot);
    a_k0 = a_k0 + BK == K ? 0 : a_k0 + BK;
  };
  auto advance_b = [&]() {
    b_slot = next_slot(b_slot);
    b_k0 = b_k0 + BK == K ? 0 : b_k0 + BK;
  };

  auto run = [&](auto nfr_tag) {
    constexpr int NFR = decltype(nfr_tag)::value;
    auto frag = [&](int as, int bs, int kk, int i, bf16x8* fa, bf16x8* fb) {
      const int f = i >> 1;
      if ((i & 1) == 0) {
        if (NFR > 0) fa[f] = sa.frag(lds + as * OPT, wv * 4 + f, kk, lane);
      } else {
        if (f < NFR) fb[f] = sb.frag(lds + bs * OPT, wr + 2 * f, kk, lane);
      }
    };
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
      for (int j = 0; j < DMAS; ++j) issue_b(j);
      advance_b();
#pragma unroll
      for (int j = 0; j < DMAS; ++j) issue_a(j);
      advance_a();
    }
    stage_sync<2 * DMAS>();
    bf16x8 fxa[4], fxb[4], fya[4], fyb[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) frag(1, 0, 0, i, fxa, fxb);
    f32x16 acc[4][4];
    const f32x16 zero16 = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    int cas = 1, cbs = 0;
    auto kstep = [&](const bf16x8* a, const bf16x8* b, auto first_tag, auto between) {
      constexpr bool FIRST = decltype(first_tag)::value;
      constexpr int kOrder[16][2] = {{0, 0}, {1, 0}, {0, 1}, {1, 1}, {2, 0}, {2, 1}, {0, 2}, {1, 2},
                                     {2, 2}, {3, 0}, {3, 1}, {3, 2}, {0, 3}, {1, 3}, {2, 3}, {3, 3}};
#pragma unroll
      for (int m = 0; m < 8; ++m) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int fv = kOrder[2 * m + t][0], fr = kOrder[2 * m + t][1];
          if (fr < NFR)
            acc[fv][fr] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[fv], b[fr], FIRST ? zero16 : acc[fv][fr], 0, 0, 0);
        }
        between(m);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto stage = [&](auto first_tag) {
      const int nas = next_slot(cas), nbs = next_slot(cbs);
      kstep(fxa, fxb, first_tag, [&](int m) {
        if ((m & 1) == 0) issue_b(m >> 1);
        frag(cas, cbs, 1, m, fya, fyb);
      });
      kstep(fya, fyb, std::false_type{}, [&](int m) {
        if ((m & 1) == 0) issue_b(4 + (m >> 1));
        frag(cas, cbs, 2, m, fxa, fxb);
      });
      advance_b();
      kstep(fxa, fxb, std::false_type{}, [&](int m) { frag(cas, cbs, 3, m, fya, fyb); });
      stage_sync<DMAS>();  // the next stage has landed (the second's tile behind it may be in flight); this one is read
      kstep(fya, fyb, std::false_type{}, [&](int m) {
        issue_a(m);
        frag(nas, nbs, 0, m, fxa, fxb);
      });
      advance_a();
      cas = nas;
      cbs = nbs;
    };
    stage(std::true_type{});
    for (int q = 1; q < stages; ++q) stage(std::false_type{});
    if constexpr (NFR > 0) {
      // The accumulators are read one by one, by v_accvgpr_read: left to itself
      // the register allocator copies all of them at once and spills.  It does
      // not count these as readers of the matrix results, so the wait states
      // are written out, behind every matrix instruction by taking all live
      // accumulators as operands.
      if constexpr (NFR == 4)
        asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::"a"(acc[0][0]), "a"(acc[0][1]), "a"(acc[0][2]), "a"(acc[0][3]),
                     "a"(acc[1][0]), "a"(acc[1][1]), "a"(acc[1][2]), "a"(acc[1][3]), "a"(acc[2][0]), "a"(acc[2][1]),
                     "a"(acc[2][2]), "a"(acc[2][3]), "a"(acc[3][0]), "a"(acc[3][1]), "a"(acc[3][2]), "a"(acc[3][3]));
      else if constexpr (NFR == 3)
        asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::"a"(acc[0][0]), "a"(acc[0][1]), "a"(acc[0][2]), "a"(acc[1][0]),
                     "a"(acc[1][1]), "a"(acc[1][2]), "a"(acc[2][0]), "a"(acc[2][1]), "a"(acc[2][2]), "a"(acc[3][0]),
                     "a"(acc[3][1]), "a"(acc[3][2]));
      else if constexpr (NFR == 2)
        asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::"a"(acc[0][0]), "a"(acc[0][1]), "a"(acc[1][0]), "a"(acc[1][1]),
                     "a"(acc[2][0]), "a"(acc[2][1]), "a"(acc[3][0]), "a"(acc[3][1]));
      else
        asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::"a"(acc[0][0]), "a"(acc[1][0]), "a"(acc[2][0]), "a"(acc[3][0]));
#pragma unroll
      for (int fr = 0; fr < NFR; ++fr)
#pragma unroll
        for (int fv = 0; fv < 4; ++fv)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(z[i]) : "a"(acc[fv][fr][4 * j + i]));
            epi(fr, fv, j, z);
          }
    }
  };
  switch (min(4, max(0, (nb - wr + 1) / 2))) {
    case 4: run(std::integral_constant<int, 4>{}); break;
    case 3: run(std::integral_constant<int, 3>{}); break;
    case 2: run(std::integral_constant<int, 2>{}); break;
    case 1: run(std::integral_constant<int, 1>{}); break;
    default: run(std::integral_constant<int, 0>{}); break;
  }
  // the next tile's prologue counts its DMAs from zero and writes the ring
  stage_sync<0>();
}

__device__ __forceinline__ int blocks_of(int rows) { return min(8, max(0, (rows + 31) / 32)); }

// Where a lane's run of four stands in a tile: row of the second operand, and
// first of the four of the first.
struct Lane {
  int row0, col0, wr, wv;
  __device__ __forceinline__ Lane() {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wr = wave >> 1;
    wv = wave & 1;
    row0 = wr * 32 + (lane & 31);
    col0 = wv * 128 + 4 * (lane >> 5);
  }
  __device__ __forceinline__ int row(int fr) const { return row0 + 64 * fr; }
  __device__ __forceinline__ int col(int fv, int j) const { return col0 + 32 * fv + 8 * j; }
};

template <bool TAIL>
__global__ __launch_bounds__(NT, 1) void k_loss_dz(GradArgs a) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[SLOTS * OPT];
  const int M = min(a.ctr[0], a.L), Mp = (M + BK - 1) / BK * BK, np = (a.n + BK - 1) / BK * BK;
  const int n_rt = (M + BT - 1) / BT, n_vt = (a.n + BT - 1) / BT;
  const Lane at;
  for (int e = xcd_remap(blockIdx.x, gridDim.x); e < n_rt * n_vt; e += gridDim.x) {
    int rt, vt;
    item_coords(e, n_rt, n_vt, rt, vt);
    const int r0 = rt * BT, c0 = vt * BT;
    const Operand w = {a.W + (int64_t)(a.v0 + c0) * a.d, a.d, a.n - c0, a.d, a.zeros};
    const Operand h = {a.rows + (int64_t)r0 * a.dp, a.dp, Mp - r0, a.dp, nullptr};
    float lse[4], coef[4];
    int hit[4];  // the target's place in the tile
#pragma unroll
    for (int fr = 0; fr < 4; ++fr) {
      const int r = min(r0 + at.row(fr), Mp - 1);
      lse[fr] = a.lse[r];
      coef[fr] = a.coef[r];
      hit[fr] = a.tgt[r] - a.v0 - c0;
    }
    const bool whole = c0 + BT <= a.n;
    tile_product<false, TAIL, false>(lds, w, h, a.dp / BK, blocks_of(Mp - r0), [&](int fr, int fv, int j, float* z) {
      const int r = r0 + at.row(fr), c = at.col(fv, j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = __builtin_amdgcn_exp2f((z[i] - lse[fr]) * kLog2eF);
        z[i] = coef[fr] * (p - (c + i == hit[fr] ? 1.f : 0.f));
      }
      if (!whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = c0 + c + i < a.n ? z[i] : 0.f;
      }
      if (r < Mp && c0 + c < np)
        *reinterpret_cast<uint2*>(a.dz + (int64_t)r * a.ldz + c0 + c) =
            make_uint2(float_bf16(z[0]) | float_bf16(z[1]) << 16, float_bf16(z[2]) | float_bf16(z[3]) << 16);
    });
  }
}

// d_hidden has rows / 256 x d / 256 tiles, often fewer than compute units or a
// little more: their K stages are one line, cut into equal lengths, so every
// workgroup has the same work.  A workgroup's part of a tile is a share of its
// own, kept in fp32 in the accumulators' order over all pieces, and the shares
// are added at the end, in order.
__global__ __launch_bounds__(NT, 1) void k_loss_d_hidden(GradArgs a) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[SLOTS * OPT];
  const int M = min(a.ctr[0], a.L), Mp = (M + BK - 1) / BK * BK;
  const int n_rt = (M + BT - 1) / BT, n_ct = (a.d + BT - 1) / BT;
  const int64_t tiles = (int64_t)n_rt * n_ct, stages = (a.n + BK - 1) / BK, line = tiles * stages;
  const int64_t cuts = loss_cuts(tiles, a.ldz);
  for (int64_t g = xcd_remap(blockIdx.x, gridDim.x); g < cuts; g += gridDim.x) {
    const int64_t lo = line * g / cuts, hi = line * (g + 1) / cuts;
    const int64_t t0 = tiles * g / cuts, t1 = (tiles * (g + 1) + cuts - 1) / cuts;
    for (int64_t t = t0; t < t1; ++t) {
      const int64_t s0 = max(lo, t * stages) - t * stages, s1 = min(hi, (t + 1) * stages) - t * stages;
      float4* share = reinterpret_cast<float4*>(a.acc) + (g + t) * (BT * BT / 4) + threadIdx.x;
      if (s1 <= s0) {  // a piece too short to give this workgroup a stage of the tile
        if (a.first)
          for (int i = 0; i < BT * BT / 4 / NT; ++i) share[i * NT] = make_float4(0.f, 0.f, 0.f, 0.f);
        continue;
      }
      int rt, ct;
      item_coords((int)t, n_rt, n_ct, rt, ct);
      const int r0 = rt * BT, c0 = ct * BT, k0 = (int)s0 * BK;
      const Operand w = {a.W + (int64_t)(a.v0 + k0) * a.d + c0, a.d, a.n - k0, a.d - c0, nullptr};
      const Operand z = {a.dz + (int64_t)r0 * a.ldz + k0, a.ldz, Mp - r0, 0, nullptr};
      tile_product<true, false, false>(lds, w, z, (int)(s1 - s0), blocks_of(M - r0), [&](int fr, int fv, int j, float* v) {
        float4* o = share + ((fr * 4 + fv) * 4 + j) * NT;
        float4 x = a.first ? make_float4(0.f, 0.f, 0.f, 0.f) : *o;
        x.x += v[0];
        x.y += v[1];
        x.z += v[2];
        x.w += v[3];
        *o = x;
      });
    }
  }
}

// d_hidden of a tile: its shares added, in the order of the cuts.
__global__ __launch_bounds__(NT) void k_loss_join(GradArgs a) {
  const int M = min(a.ctr[0], a.L);
  const int n_rt = (M + BT - 1) / BT, n_ct = (a.d + BT - 1) / BT;
  const int64_t tiles = (int64_t)n_rt * n_ct, cuts = loss_cuts(tiles, a.ldz);
  const Lane at;
  constexpr int kParts = 16;  // of a tile: one (fr, fv)
  for (int64_t e = blockIdx.x; e < tiles * kParts; e += gridDim.x) {
    const int64_t t = e / kParts;
    const int part = (int)(e - t * kParts), fr = part >> 2, fv = part & 3;
    int rt, ct;
    item_coords((int)t, n_rt, n_ct, rt, ct);
    const int r = rt * BT + at.row(fr);
    const int64_t g0 = t * cuts / tiles, g1 = ((t + 1) * cuts + tiles - 1) / tiles;
    if (r >= M) continue;
    const int64_t o = (int64_t)a.idx[r] * a.d;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4* p = reinterpret_cast<const float4*>(a.acc) + (g0 + t) * (BT * BT / 4) + (part * 4 + j) * NT + threadIdx.x;
      float4 s = *p;
      for (int64_t g = g0 + 1; g < g1; ++g) {
        p += BT * BT / 4;
        s.x += p->x;
        s.y += p->y;
        s.z += p->z;
        s.w += p->w;
      }
      const int c = ct * BT + at.col(fv, j);
      if (c < a.d)
        *reinterpret_cast<uint2*>(a.d_hidden + o + c) =
            make_uint2(float_bf16(s.x) | float_bf16(s.y) << 16, float_bf16(s.z) | float_bf16(s.w) << 16);
    }
  }
}

__global__ __launch_bounds__(NT, 1) void k_loss_d_W(GradArgs a) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[SLOTS * OPT];
  const int M = min(a.ctr[0], a.L), Mp = (M + BK - 1) / BK * BK;
  if (M == 0) {
    if (a.accumulate) return;
    const int64_t n = (int64_t)a.n * a.d / 8;
    uint4* o = reinterpret_cast<uint4*>(a.d_W + (int64_t)a.v0 * a.d);
    for (int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x; i < n; i += (int64_t)gridDim.x * NT) o[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int n_vt = (a.n + BT - 1) / BT, n_ct = (a.d + BT - 1) / BT;
  const Lane at;
  for (int64_t e = xcd_remap(blockIdx.x, gridDim.x); e < (int64_t)n_vt * n_ct; e += gridDim.x) {
    int vt, ct;
    item_coords((int)e, n_vt, n_ct, vt, ct);
    const int r0 = vt * BT, c0 = ct * BT;
    const Operand h = {a.rows + c0, a.dp, Mp, a.dp - c0, nullptr};
    const Operand z = {a.dz + r0, a.ldz, Mp, a.ldz - r0, nullptr};
    tile_product<true, false, true>(lds, h, z, Mp / BK, blocks_of(a.n - r0), [&](int fr, int fv, int j, float* v) {
      const int r = r0 + at.row(fr), c = c0 + at.col(fv, j);
      if (r >= a.n || c >= a.d) return;
      uint2* o = reinterpret_cast<uint2*>(a.d_W + (int64_t)(a.v0 + r) * a.d + c);
      if (a.accumulate) {
        const uint2 u = *o;
        v[0] += bf16_float(u.x & 0xFFFF);
        v[1] += bf16_float(u.x >> 16);
        v[2] += bf16_float(u.y & 0xFFFF);
        v[3] += bf16_float(u.y >> 16);
      }
      *o = make_uint2(float_bf16(v[0]) | float_bf16(v[1]) << 16, float_bf16(v[2]) | float_bf16(v[3]) << 16);
    });
  }
}

}  // namespace

hipError_t launch_loss_dz(const GradArgs& a, int grid, hipStream_t stream) {
  if (a.d % BK == 0)
    hipLaunchKernelGGL(k_loss_dz<false>, dim3(grid), dim3(NT), 0, stream, a);
  else
    hipLaunchKernelGGL(k_loss_dz<true>, dim3(grid), dim3(NT), 0, stream, a);
  return hipGetLastError();
}
hipError_t launch_loss_d_hidden(const GradArgs& a, int grid, hipStream_t stream) {
  hipLaunchKernelGGL(k_loss_d_hidden, dim3(grid), dim3(NT), 0, stream, a);
  return hipGetLastError();
}
hipError_t launch_loss_d_W(const GradArgs& a, int grid, hipStream_t stream) {
  hipLaunchKernelGGL(k_loss_d_W, dim3(grid), dim3(NT), 0, stream, a);
  return hipGetLastError();
}
hipError_t launch_loss_join(const GradArgs& a, int grid, hipStream_t stream) {
  hipLaunchKernelGGL(k_loss_join, dim3(grid), dim3(NT), 0, stream, a);
  return hipGetLastError();
}

}  // namespace dllm

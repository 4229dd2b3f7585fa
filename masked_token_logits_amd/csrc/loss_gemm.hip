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
//   * With many rows the matrix instructions are the time.  3900 rows (16 row
//     tiles), 152064 entries of 3584, 4.2 Tflop a product: dz 3.9 ms (1.08
//     Pflop/s), d_hidden 3.3 (1.27), d_W 3.7 (1.16); a library's plain products
//     of 8192^3 reach 1.39, 1.22 and 1.07 with operands laid out like that.  dz
//     has the exponentials and 1.2 GB of stores at each tile's end on top.
//   * With few rows W's bytes are (see k_loss_dz, k_loss_d_W_few).
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
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
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

// An operand in memory, [256 rows][K] or, by rows of K, [K][256 columns], from
// its first element of a tile on: the rows that exist there (of K, for one by
// rows of K) and the columns (of K, where K is contiguous).  Sources outside it
// are drawn to its last row or piece: valid memory, whose products are not
// stored or meet zeros.
struct Operand {
  const uint16_t* p;
  int rows, cols;
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
  uint32_t ld2;  // bytes from row to row
  int lane_off, swz, row, col, cols;
  __device__ __forceinline__ void init(int64_t ld, const uint16_t* no_values, int wave, int lane) {
    zeros = reinterpret_cast<const char*>(no_values);
    ld2 = (uint32_t)ld * 2u;
    row = wave * 8 + (lane >> 3);
    col = ((lane & 7) ^ ((row >> 1) & 7)) * 8;
    swz = ((lane & 31) >> 1) & 7;
    lane_off = (lane & 31) * BK;
  }
  __device__ __forceinline__ void start(const Operand& o) {
    base = reinterpret_cast<const char*>(o.p);
    cols = o.cols;
    const int last = min(o.rows - 1, BT - 1);
#pragma unroll
    for (int j = 0; j < DMAS; ++j) off[j] = (uint32_t)min(row + 32 * j, last) * ld2 + (uint32_t)col * 2u;
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
  uint32_t ld2, k_off, col_off;
  int rows, lane_off, col, sw;
  __device__ __forceinline__ void init(int64_t ld, const uint16_t*, int wave, int lane) {
    ld2 = (uint32_t)ld * 2u;
    const int k = wave * 2 + (lane >> 5);
    k_off = (uint32_t)k * ld2;
    col = (((lane & 31) >> 2) ^ (k & 3)) * 32 + (lane & 3) * 8;
    sw = (lane & 15) >> 2;
    lane_off = (8 * (lane >> 5) + sw) * BT + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  }
  __device__ __forceinline__ void start(const Operand& o) {
    base = reinterpret_cast<const char*>(o.p);
    rows = o.rows;
    col_off = (uint32_t)min(col, o.cols - 8) * 2u;
  }
  __device__ __forceinline__ const char* source(int j, int k0) const {
    const uint32_t last = (uint32_t)min(rows - 1 - k0, BK - 1) * ld2;
    return base + (size_t)k0 * (size_t)ld2 + (min(k_off + (uint32_t)(8 * j) * ld2, last) + col_off);
  }
  __device__ __forceinline__ bf16x8 frag(const uint16_t* tile, int block, int kk, int) const {
    LDS_AS uint16_t* ring = (LDS_AS uint16_t*)tile;
    LDS_AS const uint16_t* p = ring + lane_off + ((block ^ sw) * 32) + kk * 16 * BT;
    const bf16x4 lo = read_tr(p, ring), hi = read_tr(p + 4 * BT, ring);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// By rows of K, half as wide: rows of K of 256 bytes, four to a DMA, swizzled like
// the wide ones.  LDS [64][128].
constexpr int kNarrow = 128;
struct NarrowSide {
  int k, col, sw, lane_off;
  __device__ __forceinline__ NarrowSide(int wave, int lane) {
    k = wave * 4 + (lane >> 4);
    col = (((lane & 15) >> 2) ^ (k & 3)) * 32 + (lane & 3) * 8;
    sw = (lane & 15) >> 2;
    lane_off = (8 * (lane >> 5) + sw) * kNarrow + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  }
  // where the lane's first DMA of [K][ld] reads the tile from column c0 on, drawn to the last of `cols`
  __device__ __forceinline__ const uint16_t* source(const uint16_t* p, int64_t ld, int c0, int cols) const {
    return p + (int64_t)k * ld + min(c0 + col, cols - 8);
  }
  __device__ __forceinline__ bf16x8 frag(const uint16_t* tile, int block, int kk) const {
    LDS_AS uint16_t* ring = (LDS_AS uint16_t*)tile;
    LDS_AS const uint16_t* p = ring + lane_off + ((block ^ sw) * 32) + kk * 16 * kNarrow;
    const bf16x4 lo = read_tr(p, ring), hi = read_tr(p + 4 * kNarrow, ring);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// One tile of a workgroup's work: the operands at its first K, the K it has,
// the stage it starts with (later ones follow, then those before it) and the
// 32-blocks of the second operand that are wanted.
struct Item {
  Operand a, b;
  int stages, start, nb;
};

// Where a lane's values stand in a tile: z[i] of (fr, fv, j) is row(fr) of the
// second operand, and col(fv, j) + i of the first.
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

// A workgroup's tiles, one after another.  Their stages are one stream: the
// DMAs run two stages ahead, across the end of a tile into the next one (with
// tiles of one stage the one behind that), so that its first stages land while
// this one's results are stored.
//
// work.first(cursor) and work.next(cursor) walk the tiles (false behind the
// last, the cursor then stays), work.describe(cursor) gives an Item,
// work.begin(cursor) is called before a tile's first stage, and
// work.end(cursor, spare, fr, read) behind the last one for each of the lane's
// rows: read(fv, j, z) gives four accumulators, spare is 8 KiB of LDS of the wave's.
// STREAM_A: the first operand's tiles are read by this workgroup only.
template <bool A_BY_K, bool A_TAIL, bool B_BY_K, bool STREAM_A, class Work>
__device__ __forceinline__ void run_tiles(uint16_t* lds, Work& work) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave >> 1, wv = wave & 1;
  typename Work::Cursor cur, ahead;
  if (!work.first(cur)) return;
  // this tile, the next and the one behind it; at the end the last one again,
  // whose stages are then read and not used
  Item it = work.describe(cur), it1, it2;
  ahead = cur;
  bool more = work.next(ahead), more2;
  it1 = work.describe(ahead);
  typename Work::Cursor nxt = ahead;
  more2 = work.next(ahead);
  it2 = work.describe(ahead);

  Side<A_BY_K, A_TAIL> sa;
  Side<B_BY_K, false> sb;
  sa.init(work.lda(), work.zeros(), wave, lane);
  sb.init(work.ldb(), nullptr, wave, lane);
  // Operand tiles alternate through the ring: the second's of stage q goes to
  // slot 2q % 5, the first's to (2q + 1) % 5.
  int a_k0 = it.start * BK, a_K = it.stages * BK, a_left = it.stages, a_rel = 0, a_slot = 1;
  int b_k0 = a_k0, b_K = a_K, b_left = a_left, b_rel = 0, b_slot = 0;
  sa.start(it.a);
  sb.start(it.b);
  auto next_slot = [](int s) { return s + 2 >= SLOTS ? s + 2 - SLOTS : s + 2; };
  constexpr int kPolicy = STREAM_A ? 2 : 0;  // 2: non-temporal
  // before a stage's first DMA of a side: the next tile's, where this one's are all queued
  auto turn_a = [&]() {
    if (a_left > 0) return;
    const Item& n = a_rel == 0 ? it1 : it2;
    ++a_rel;
    sa.start(n.a);
    a_k0 = n.start * BK;
    a_K = n.stages * BK;
    a_left = n.stages;
  };
  auto turn_b = [&]() {
    if (b_left > 0) return;
    const Item& n = b_rel == 0 ? it1 : it2;
    ++b_rel;
    sb.start(n.b);
    b_k0 = n.start * BK;
    b_K = n.stages * BK;
    b_left = n.stages;
  };
  auto issue_a = [&](int j) {
    __builtin_amdgcn_global_load_lds((const void*)sa.source(j, a_k0), (LDS_AS void*)(lds + a_slot * OPT + (wave + 4 * j) * 512), 16,
                                     0, kPolicy);
  };
  auto issue_b = [&](int j) {
    __builtin_amdgcn_global_load_lds((const void*)sb.source(j, b_k0), (LDS_AS void*)(lds + b_slot * OPT + (wave + 4 * j) * 512), 16,
                                     0, 0);
  };
  auto advance_a = [&]() {
    a_slot = next_slot(a_slot);
    a_k0 = a_k0 + BK == a_K ? 0 : a_k0 + BK;
    --a_left;
  };
  auto advance_b = [&]() {
    b_slot = next_slot(b_slot);
    b_k0 = b_k0 + BK == b_K ? 0 : b_k0 + BK;
    --b_left;
  };

  bf16x8 fxa[4], fxb[4], fya[4], fyb[4];
  auto frag = [&](int as, int bs, int kk, int i, bf16x8* fa, bf16x8* fb) {
    const int f = i >> 1;
    if ((i & 1) == 0)
      fa[f] = sa.frag(lds + as * OPT, wv * 4 + f, kk, lane);
    else
      fb[f] = sb.frag(lds + bs * OPT, wr + 2 * f, kk, lane);
  };
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    turn_b();
#pragma unroll
    for (int j = 0; j < DMAS; ++j) issue_b(j);
    advance_b();
    turn_a();
#pragma unroll
    for (int j = 0; j < DMAS; ++j) issue_a(j);
    advance_a();
  }
  stage_sync<2 * DMAS>();
  int cas = 1, cbs = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) frag(1, 0, 0, i, fxa, fxb);

  for (;;) {
    work.begin(cur);
    auto run = [&](auto nfr_tag) {
      constexpr int NFR = decltype(nfr_tag)::value;
      f32x16 acc[4][4];
      const f32x16 zero16 = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
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
        turn_b();
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
        turn_a();
        kstep(fya, fyb, std::false_type{}, [&](int m) {
          issue_a(m);
          frag(nas, nbs, 0, m, fxa, fxb);
        });
        advance_a();
        cas = nas;
        cbs = nbs;
      };
      const int stages = it.stages;
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
        // this stage's slot of the first operand is free until the next stage's DMAs
        uint16_t* spare = lds + (cas + SLOTS - 2) % SLOTS * OPT + wave * (OPT / 4);
#pragma unroll
        for (int fr = 0; fr < NFR; ++fr)
          work.end(cur, spare, fr, [&](int fv, int j, float* z) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(z[i]) : "a"(acc[fv][fr][4 * j + i]));
          });
      }
    };
    switch (min(4, max(0, (it.nb - wr + 1) / 2))) {
      case 4: run(std::integral_constant<int, 4>{}); break;
      case 3: run(std::integral_constant<int, 3>{}); break;
      case 2: run(std::integral_constant<int, 2>{}); break;
      case 1: run(std::integral_constant<int, 1>{}); break;
      default: run(std::integral_constant<int, 0>{}); break;
    }
    stage_sync<63>();  // no wave's DMAs reach the spare slot before every wave has left it
    if (!more) break;
    cur = nxt;
    it = it1;
    --a_rel;
    --b_rel;
    nxt = ahead;
    it1 = it2;
    more = more2;
    more2 = work.next(ahead);
    it2 = work.describe(ahead);
  }
  stage_sync<0>();  // the DMAs behind the last stage
}

__device__ __forceinline__ int blocks_of(int rows) { return min(8, max(0, (rows + 31) / 32)); }

// A lane's results of one row, as bf16, through the wave's 8 KiB of spare LDS
// [32 rows][128 columns], so that they leave in 256-byte runs: store(row,
// column, 16 bytes).  Row r holds its 16-byte pieces at piece ^ (r & 15): the 16
// pieces of a read meet all banks, the rows of a write half of them twice.
// patch(p, r, h) may change a row of the lane's in LDS before.
template <class Make, class Patch, class Store>
__device__ __forceinline__ void store_rows(uint16_t* spare, const Lane& at, int fr, Make make, Patch patch, Store store) {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));  // the addresses are made here, not kept through the tile's stages
  const int r = lane & 31, h = lane >> 5;
  LDS_AS uint8_t* p = (LDS_AS uint8_t*)spare;
  asm volatile("" ::: "memory");  // a wave's LDS accesses are done in order: the last call's reads, these writes
#pragma unroll
  for (int fv = 0; fv < 4; ++fv)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x2 u = make(fv, j);
      *(LDS_AS u32x2*)(p + r * 256 + ((fv * 4 + j) ^ (r & 15)) * 16 + h * 8) = u;
      __builtin_amdgcn_sched_barrier(0);  // one run at a time: all of them at once do not fit the registers
    }
  asm volatile("" ::: "memory");
  patch(p, r, h);
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int rr = i * 4 + (lane >> 4), piece = lane & 15;
    u32x4 u = *(LDS_AS const u32x4*)(p + rr * 256 + ((piece ^ (rr & 15)) * 16));
    asm volatile("" : "+v"(u));  // read by all lanes together, not inside the store's bounds
    store(at.wr * 32 + 64 * fr + rr, at.wv * 128 + piece * 8, make_uint4(u.x, u.y, u.z, u.w));
  }
}

template <bool TAIL>
struct DzWork {
  const GradArgs& a;
  int Mp, np, n_rt, n_vt;
  Lane at;
  float lse[4], coef[4], at_tgt[4];
  int tgt[4];
  struct Cursor {
    int e, r0, c0;
  };
  __device__ __forceinline__ int64_t lda() const { return a.d; }
  __device__ __forceinline__ int64_t ldb() const { return a.dp; }
  __device__ __forceinline__ const uint16_t* zeros() const { return a.zeros; }
  __device__ __forceinline__ bool place(Cursor& c) const {
    if (c.e >= n_rt * n_vt) return false;
    int rt, vt;
    item_coords(c.e, n_rt, n_vt, rt, vt);
    c.r0 = rt * BT;
    c.c0 = vt * BT;
    return true;
  }
  __device__ __forceinline__ bool first(Cursor& c) const {
    c.e = xcd_remap(blockIdx.x, gridDim.x);
    return place(c);
  }
  __device__ __forceinline__ bool next(Cursor& c) const {
    Cursor n = c;
    n.e += gridDim.x;
    if (!place(n)) return false;
    c = n;
    return true;
  }
  __device__ __forceinline__ Item describe(const Cursor& c) const {
    return {{a.W + (int64_t)(a.v0 + c.c0) * a.d, a.n - c.c0, a.d},
            {a.rows + (int64_t)c.r0 * a.dp, Mp - c.r0, a.dp},
            a.dp / BK,
            // One row tile: the time is W's bytes.  Its rows are a power of two apart, and tiles that all
            // stand at the same place of them ask a few channels for everything (102 rows, 126464 entries
            // of 4096: 260 us; 206 where each stands at another).  More row tiles share W's tiles in step.
            n_rt == 1 ? (int)((int64_t)c.e * 7 % (a.dp / BK)) : 0,
            blocks_of(Mp - c.r0)};
  }
  __device__ __forceinline__ void begin(const Cursor& c) {
#pragma unroll
    for (int fr = 0; fr < 4; ++fr) {
      const int r = min(c.r0 + at.row(fr), Mp - 1);
      lse[fr] = a.lse[r];
      coef[fr] = a.coef[r];
      tgt[fr] = a.tgt[r];
      at_tgt[fr] = a.at_tgt[r];
    }
  }
  template <class Z>
  __device__ __forceinline__ void end(const Cursor& c, uint16_t* spare, int fr, Z read) const {
    // the end of the piece counted from the lane's first column, and the target's place in the wave's
    int end = a.n - c.c0 - at.col0, hit = tgt[fr] - a.v0 - c.c0 - at.wv * 128;
    asm volatile("" : "+v"(hit), "+v"(end));  // made here, not kept through the tile's stages
    const bool whole = c.c0 + BT <= a.n;
    store_rows(
        spare, at, fr,
        [&](int fv, int j) {
          float z[4];
          read(fv, j, z);
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = loss_p(z[i], lse[fr]) * coef[fr];
          if (!whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = 32 * fv + 8 * j + i < end ? z[i] : 0.f;
          }
          return u32x2{float_bf16(z[0]) | float_bf16(z[1]) << 16, float_bf16(z[2]) | float_bf16(z[3]) << 16};
        },
        [&](LDS_AS uint8_t* p, int r, int h) {
          if (h == 0 && hit >= 0 && hit < 128)
            *(LDS_AS uint16_t*)(p + r * 256 + ((hit >> 3) ^ (r & 15)) * 16 + (hit & 7) * 2) = (uint16_t)float_bf16(at_tgt[fr]);
        },
        [&](int row, int col, const uint4& u) {
          if (c.r0 + row < Mp && c.c0 + col < np)
            *reinterpret_cast<uint4*>(a.dz + (int64_t)(c.r0 + row) * a.ldz + c.c0 + col) = u;
        });
  }
};

template <bool TAIL>
__global__ __launch_bounds__(NT, 1) void k_loss_dz(GradArgs a) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[SLOTS * OPT];
  const int M = min(a.ctr[0], a.L);
  DzWork<TAIL> work = {a, (M + BK - 1) / BK * BK, (a.n + BK - 1) / BK * BK, (M + BT - 1) / BT, (a.n + BT - 1) / BT, Lane()};
  // With one row tile W is streamed (102 rows, 126464 entries of 4096: 217 -> 198 us); more share its tiles.
  if (work.n_rt <= 1)
    run_tiles<false, TAIL, false, true>(lds, work);
  else
    run_tiles<false, TAIL, false, false>(lds, work);
}

// d_hidden has rows / 256 x d / 256 tiles, often fewer than compute units or a
// little more: their K stages are one line, cut into equal lengths, so every
// workgroup has the same work.  A workgroup's part of a tile is a share of its
// own, kept in fp32 in the accumulators' order over all pieces, and the shares
// are added at the end, in order.
//
// A workgroup takes its tiles from the last to the first.  With less than a
// tile each (cuts just above tiles) it has the first stages of one tile and the
// last ones of the tile before, and in that order it works, like all the
// others, near the stage that as much time has passed: one region of W and dz
// is in the caches, not one for each workgroup.  Whole tiles start where the
// time stands, too, and wrap around.
struct DHiddenWork {
  const GradArgs& a;
  int M, Mp, n_rt, n_ct, stages;
  int64_t g, lo, hi, low, high;  // the workgroup's cut, its stages of the line, and the tiles that it may have some of
  Lane at;
  struct Cursor {
    int64_t t;
    int s0, s1, r0, c0, passed;
  };
  __device__ __forceinline__ DHiddenWork(const GradArgs& args, int m, int64_t cut, int64_t tiles, int64_t cuts) : a(args), M(m), g(cut) {
    Mp = (M + BK - 1) / BK * BK;
    n_rt = (M + BT - 1) / BT;
    n_ct = (a.d + BT - 1) / BT;
    stages = (a.n + BK - 1) / BK;
    lo = tiles * stages * g / cuts;
    hi = tiles * stages * (g + 1) / cuts;
    low = tiles * g / cuts;
    high = (tiles * (g + 1) + cuts - 1) / cuts;
  }
  // the cut's stages of tile t; none where a piece is too short to have one
  __device__ __forceinline__ void part(int64_t t, int& s0, int& s1) const {
    s0 = (int)max(lo - t * stages, (int64_t)0);
    s1 = (int)min(hi - t * stages, (int64_t)stages);
  }
  __device__ __forceinline__ int64_t lda() const { return a.d; }
  __device__ __forceinline__ int64_t ldb() const { return a.ldz; }
  __device__ __forceinline__ const uint16_t* zeros() const { return nullptr; }
  // from tile t on, downwards, to a part that has stages
  __device__ __forceinline__ bool place(Cursor& c) const {
    for (; c.t >= low; --c.t) {
      part(c.t, c.s0, c.s1);
      if (c.s1 <= c.s0) continue;
      int rt, ct;
      item_coords((int)c.t, n_rt, n_ct, rt, ct);
      c.r0 = rt * BT;
      c.c0 = ct * BT;
      return true;
    }
    return false;
  }
  __device__ __forceinline__ bool first(Cursor& c) const {
    c.passed = 0;
    c.t = high - 1;
    return place(c);
  }
  __device__ __forceinline__ bool next(Cursor& c) const {
    Cursor n = c;
    n.passed += n.s1 - n.s0;
    if (n.passed >= stages) n.passed -= stages;
    --n.t;
    if (!place(n)) return false;
    c = n;
    return true;
  }
  __device__ __forceinline__ Item describe(const Cursor& c) const {
    const int k0 = c.s0 * BK;
    return {{a.W + (int64_t)(a.v0 + k0) * a.d + c.c0, a.n - k0, a.d - c.c0},
            {a.dz + (int64_t)c.r0 * a.ldz + k0, Mp - c.r0, 0},
            c.s1 - c.s0,
            c.s1 - c.s0 == stages ? c.passed : 0,
            blocks_of(M - c.r0)};
  }
  __device__ __forceinline__ void begin(const Cursor&) const {}
  template <class Z>
  __device__ __forceinline__ void end(const Cursor& c, uint16_t*, int fr, Z read) const {
    float4* share = reinterpret_cast<float4*>(a.acc) + (g + c.t) * (BT * BT / 4) + threadIdx.x;
#pragma unroll
    for (int fv = 0; fv < 4; ++fv) {
      float4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = a.first ? make_float4(0.f, 0.f, 0.f, 0.f) : share[((fr * 4 + fv) * 4 + j) * NT];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[4];
        read(fv, j, v);
        x[j].x += v[0];
        x[j].y += v[1];
        x[j].z += v[2];
        x[j].w += v[3];
        share[((fr * 4 + fv) * 4 + j) * NT] = x[j];
      }
    }
  }
};

// With one row tile: the j-th of the cuts in the order of the stages, within a
// tile, at which they begin, a multiple of cuts / gcd(tiles, cuts) each.
// Neighbours in an XCD then have the same stages of different columns and share
// dz's tiles; W is then streamed (102 rows, 126464 entries of 4096: 234 us in the
// cuts' own order, 211 in this one, 207 with W past the caches).
__device__ __forceinline__ int cut_by_stage(int j, int tiles, int cuts) {
  int r0 = cuts, r1 = tiles, x0 = 0, x1 = 1;  // x1 * tiles = r1 modulo cuts
  while (r1 != 0) {
    const int k = r0 / r1, r = r0 - k * r1, x = x0 - k * x1;
    r0 = r1;
    r1 = r;
    x0 = x1;
    x1 = x;
  }
  const int n = cuts / r0, inverse = (x0 % n + n) % n;
  return (int)((int64_t)(j / r0) * inverse % n) + j % r0 * n;
}

__global__ __launch_bounds__(NT, 1) void k_loss_d_hidden(GradArgs a) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[SLOTS * OPT];
  const int M = min(a.ctr[0], a.L), n_rt = (M + BT - 1) / BT, n_ct = (a.d + BT - 1) / BT;
  const int64_t tiles = (int64_t)n_rt * n_ct, cuts = min(loss_cuts(tiles, a.ldz), (int64_t)gridDim.x);
  int g = xcd_remap(blockIdx.x, gridDim.x);
  if (g >= cuts) return;
  if (n_rt == 1) g = cut_by_stage(g, (int)tiles, (int)cuts);
  DHiddenWork work(a, M, g, tiles, cuts);
  if (a.first)
    for (int64_t t = work.low; t < work.high; ++t) {
      int s0, s1;
      work.part(t, s0, s1);
      float4* share = reinterpret_cast<float4*>(a.acc) + (g + t) * (BT * BT / 4) + threadIdx.x;
      if (s1 <= s0)  // a part that this piece does not reach, and a later one may
        for (int i = 0; i < BT * BT / 4 / NT; ++i) share[i * NT] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  if (n_rt == 1)
    run_tiles<true, false, false, true>(lds, work);
  else
    run_tiles<true, false, false, false>(lds, work);
}

// d_hidden of a tile: its shares added, in the order of the cuts (3900 rows of
// 3584, 480 shares of 256 KiB: 75 us; 102 rows: 10).
__global__ __launch_bounds__(NT) void k_loss_join(GradArgs a, int grid) {
  const int M = min(a.ctr[0], a.L);
  const int n_rt = (M + BT - 1) / BT, n_ct = (a.d + BT - 1) / BT;
  const int64_t tiles = (int64_t)n_rt * n_ct, cuts = min(loss_cuts(tiles, a.ldz), (int64_t)grid);
  const Lane at;
  constexpr int kParts = 64;  // of a tile: one (fr, fv, j)
  for (int64_t e = blockIdx.x; e < tiles * kParts; e += gridDim.x) {
    const int64_t t = e / kParts;
    const int part = (int)(e - t * kParts), fr = part >> 4, fv = (part >> 2) & 3, j = part & 3;
    int rt, ct;
    item_coords((int)t, n_rt, n_ct, rt, ct);
    const int r = rt * BT + at.row(fr), c = ct * BT + at.col(fv, j);
    const int64_t g0 = t * cuts / tiles, g1 = ((t + 1) * cuts + tiles - 1) / tiles;
    if (r >= M || c >= a.d) continue;
    // what dz's rounding left of the target's entry, times its row of W
    const float left = a.left[r];
    const uint2 w = *reinterpret_cast<const uint2*>(a.W + (int64_t)a.tgt[r] * a.d + c);
    float4 s = make_float4(left * bf16_float(w.x & 0xFFFF), left * bf16_float(w.x >> 16), left * bf16_float(w.y & 0xFFFF),
                           left * bf16_float(w.y >> 16));
    const float4* p = reinterpret_cast<const float4*>(a.acc) + (g0 + t) * (BT * BT / 4) + part * NT + threadIdx.x;
#pragma unroll 4
    for (int64_t g = g0; g < g1; ++g, p += BT * BT / 4) s = make_float4(s.x + p->x, s.y + p->y, s.z + p->z, s.w + p->w);
    *reinterpret_cast<uint2*>(a.d_hidden + (int64_t)a.idx[r] * a.d + c) =
        make_uint2(float_bf16(s.x) | float_bf16(s.y) << 16, float_bf16(s.z) | float_bf16(s.w) << 16);
  }
}

struct DWWork {
  const GradArgs& a;
  int Mp, n_vt, n_ct;
  Lane at;
  struct Cursor {
    int e, r0, c0;
  };
  __device__ __forceinline__ int64_t lda() const { return a.dp; }
  __device__ __forceinline__ int64_t ldb() const { return a.ldz; }
  __device__ __forceinline__ const uint16_t* zeros() const { return nullptr; }
  __device__ __forceinline__ bool place(Cursor& c) const {
    if (c.e >= n_vt * n_ct) return false;
    int vt, ct;
    item_coords(c.e, n_vt, n_ct, vt, ct);
    c.r0 = vt * BT;
    c.c0 = ct * BT;
    return true;
  }
  __device__ __forceinline__ bool first(Cursor& c) const {
    c.e = xcd_remap(blockIdx.x, gridDim.x);
    return place(c);
  }
  __device__ __forceinline__ bool next(Cursor& c) const {
    Cursor n = c;
    n.e += gridDim.x;
    if (!place(n)) return false;
    c = n;
    return true;
  }
  __device__ __forceinline__ Item describe(const Cursor& c) const {
    return {{a.rows + c.c0, Mp, a.dp - c.c0}, {a.dz + c.r0, Mp, (int)a.ldz - c.r0}, Mp / BK, 0, blocks_of(a.n - c.r0)};
  }
  __device__ __forceinline__ void begin(const Cursor&) const {}
  template <class Z>
  __device__ __forceinline__ void end(const Cursor& c, uint16_t* spare, int fr, Z read) const {
    if (!a.accumulate) {
      store_rows(
          spare, at, fr,
          [&](int fv, int j) {
            float z[4];
            read(fv, j, z);
            return u32x2{float_bf16(z[0]) | float_bf16(z[1]) << 16, float_bf16(z[2]) | float_bf16(z[3]) << 16};
          },
          [](LDS_AS uint8_t*, int, int) {},
          [&](int row, int col, const uint4& u) {
            if (c.r0 + row < a.n && c.c0 + col < a.d)
              *reinterpret_cast<uint4*>(a.d_W + (int64_t)(a.v0 + c.r0 + row) * a.d + c.c0 + col) = u;
          });
      return;
    }
    // added in fp32 and rounded once, so not through the bf16 rows above
    const int r = c.r0 + at.row(fr);
#pragma unroll
    for (int fv = 0; fv < 4; ++fv)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[4];
        read(fv, j, v);
        const int col = c.c0 + at.col(fv, j);
        if (r >= a.n || col >= a.d) continue;
        uint2* o = reinterpret_cast<uint2*>(a.d_W + (int64_t)(a.v0 + r) * a.d + col);
        const uint2 u = *o;
        v[0] += bf16_float(u.x & 0xFFFF);
        v[1] += bf16_float(u.x >> 16);
        v[2] += bf16_float(u.y & 0xFFFF);
        v[3] += bf16_float(u.y >> 16);
        *o = make_uint2(float_bf16(v[0]) | float_bf16(v[1]) << 16, float_bf16(v[2]) | float_bf16(v[3]) << 16);
      }
  }
};

__global__ __launch_bounds__(NT, 1) void k_loss_d_W(GradArgs a) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[SLOTS * OPT];
  const int M = min(a.ctr[0], a.L);
  if (M <= kLossFew) return;  // k_loss_d_W_few's
  DWWork work = {a, (M + BK - 1) / BK * BK, (a.n + BT - 1) / BT, (a.d + BT - 1) / BT, Lane()};
  run_tiles<true, false, true, false>(lds, work);
}

// d_W of few rows: K is a few stages and the time is d_W's own bytes, so what
// counts is that stores never stop.  128 entries x 256 columns to a workgroup, one
// stage of both operands in 48 KiB of LDS, three workgroups to a compute unit:
// while one stores, the others load and multiply (126464 entries of 4096: 205 us
// for 60 rows, 253 for 102, 370 for 250, where the 256 x 256 tiles take 345 for 102
// and 450 for 250; d_W's bytes alone, 150).
constexpr int FV = kNarrow;  // entries of a tile

__global__ __launch_bounds__(NT, 3) void k_loss_d_W_few(GradArgs a, int n_vt, int n_ct) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[BK * (BT + FV)];
  const int M = min(a.ctr[0], a.L), Mp = (M + BK - 1) / BK * BK;
  if (M > kLossFew || (M == 0 && a.accumulate)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wr = wave >> 1, wv = wave & 1;
  const int vt = blockIdx.x / n_ct, ct = blockIdx.x - vt * n_ct, r0 = vt * FV, c0 = ct * BT;
  uint16_t *la = lds, *lb = lds + BK * BT;
  Side<true, false> sa;
  sa.init(a.dp, nullptr, wave, lane);
  sa.start({a.rows + c0, Mp, a.dp - c0});
  const NarrowSide sb(wave, lane);
  const char* bsrc = reinterpret_cast<const char*>(sb.source(a.dz, a.ldz, r0, (int)a.ldz));
  f32x16 acc[4][2] = {};
  for (int k0 = 0; k0 < Mp; k0 += BK) {
#pragma unroll
    for (int j = 0; j < DMAS; ++j)
      __builtin_amdgcn_global_load_lds((const void*)sa.source(j, k0), (LDS_AS void*)(la + (wave + 4 * j) * 512), 16, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      __builtin_amdgcn_global_load_lds((const void*)(bsrc + (size_t)(k0 + 16 * j) * (size_t)a.ldz * 2),
                                       (LDS_AS void*)(lb + (wave + 4 * j) * 512), 16, 0, 0);
    stage_sync<0>();
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      bf16x8 fa[4], fb[2];
#pragma unroll
      for (int f = 0; f < 4; ++f) fa[f] = sa.frag(la, wv * 4 + f, kk, lane);
#pragma unroll
      for (int f = 0; f < 2; ++f) fb[f] = sb.frag(lb, wr * 2 + f, kk);
#pragma unroll
      for (int fv = 0; fv < 4; ++fv)
#pragma unroll
        for (int fr = 0; fr < 2; ++fr) acc[fv][fr] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[fv], fb[fr], acc[fv][fr], 0, 0, 0);
    }
    stage_sync<0>();  // everyone has read the stage
  }
  Lane at;
#pragma unroll
  for (int fr = 0; fr < 2; ++fr) {
    const int first = r0 + wr * 64 + fr * 32;  // of the wave's 32 entries
    if (!a.accumulate) {
      store_rows(
          lds + wave * (OPT / 4), at, 0,
          [&](int fv, int j) {
            return u32x2{float_bf16(acc[fv][fr][4 * j]) | float_bf16(acc[fv][fr][4 * j + 1]) << 16,
                         float_bf16(acc[fv][fr][4 * j + 2]) | float_bf16(acc[fv][fr][4 * j + 3]) << 16};
          },
          [](LDS_AS uint8_t*, int, int) {},
          [&](int row, int col, const uint4& u) {
            const int r = first + row - wr * 32;
            // written once and not read here: kept out of the caches that W's next pass wants (102 rows: 248 us, cached 274)
            if (r < a.n && c0 + col < a.d)
              __builtin_nontemporal_store(u32x4{u.x, u.y, u.z, u.w},
                                          reinterpret_cast<u32x4*>(a.d_W + (int64_t)(a.v0 + r) * a.d + c0 + col));
          });
      continue;
    }
    const int r = first + (lane & 31);
#pragma unroll
    for (int fv = 0; fv < 4; ++fv)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = c0 + at.col(fv, j);
        if (r >= a.n || col >= a.d) continue;
        uint2* o = reinterpret_cast<uint2*>(a.d_W + (int64_t)(a.v0 + r) * a.d + col);
        const uint2 u = *o;
        const f32x16& z = acc[fv][fr];
        *o = make_uint2(float_bf16(z[4 * j] + bf16_float(u.x & 0xFFFF)) | float_bf16(z[4 * j + 1] + bf16_float(u.x >> 16)) << 16,
                        float_bf16(z[4 * j + 2] + bf16_float(u.y & 0xFFFF)) | float_bf16(z[4 * j + 3] + bf16_float(u.y >> 16)) << 16);
      }
  }
}

// Small products, whose 256 x 256 tiles would leave most of the chip idle: 128
// rows x 128 entries to a workgroup, 64 x 64 to a wave, and a ring of four 32 KiB
// stages with one barrier each, three stages ahead: with few tiles nothing else
// hides the memory's latency (3700 rows, 1000 entries of 1024: 16 us, where the persistent GEMM takes 38; 16 rows, 500 entries of 2048: 21).
constexpr int FR = 128, FV2 = kLossFewEntries, FRING = 4;
constexpr int FSTAGE = BK * (FR + FV2);  // elements of a stage

// pw, ph: where this lane's DMAs read W and the rows (row (wave + 4 j) * 8 + lane / 8 of each side, 16-byte
// piece ^ ((row >> 1) & 7) of it); K's stages from k0 on, then those before; zeros behind d.
template <bool TAIL>
__device__ __forceinline__ void small_product(uint16_t* lds, const uint16_t* const (&pw)[4], const uint16_t* const (&ph)[4],
                                              int stages, int k0, int d, const uint16_t* zeros, f32x16 (&acc)[2][2]) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wr = wave >> 1, wv = wave & 1;
  const int row = wave * 8 + (lane >> 3), col = ((lane & 7) ^ ((row >> 1) & 7)) * 8;
  auto issue = [&](int slot) {
    const bool in = !TAIL || k0 + col < d;
    uint16_t* to = lds + slot * FSTAGE + wave * 512;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      __builtin_amdgcn_global_load_lds((const void*)(in ? pw[j] + k0 : zeros), (LDS_AS void*)(to + 4 * j * 512), 16, 0, 0);
      __builtin_amdgcn_global_load_lds((const void*)(in ? ph[j] + k0 : zeros), (LDS_AS void*)(to + BK * FV2 + 4 * j * 512), 16, 0, 0);
    }
    k0 = k0 + BK >= stages * BK ? 0 : k0 + BK;
  };
  // stages behind the last are the first ones again, and never used
  issue(0);
  issue(1);
  issue(2);
  const int swz = ((lane & 31) >> 1) & 7;
  for (int q = 0; q < stages; ++q) {
    stage_sync<16>();  // stage q has landed, the two behind it may be in flight; and every wave has read stage q - 1
    issue((q + 3) & (FRING - 1));
    const uint16_t* w = lds + (q & (FRING - 1)) * FSTAGE + (wv * 64 + (lane & 31)) * BK;
    const uint16_t* h = lds + (q & (FRING - 1)) * FSTAGE + BK * FV2 + (wr * 64 + (lane & 31)) * BK;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const int piece = ((kk * 2 + (lane >> 5)) ^ swz) * 8;
      bf16x8 fw[2], fh[2];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        fw[f] = *reinterpret_cast<const bf16x8*>(w + f * 32 * BK + piece);
        fh[f] = *reinterpret_cast<const bf16x8*>(h + f * 32 * BK + piece);
      }
#pragma unroll
      for (int fv = 0; fv < 2; ++fv)
#pragma unroll
        for (int fr = 0; fr < 2; ++fr) acc[fv][fr] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fw[fv], fh[fr], acc[fv][fr], 0, 0, 0);
    }
  }
  stage_sync<0>();  // the DMAs behind the last stage
}

template <bool TAIL>
__global__ __launch_bounds__(NT, 1) void k_loss_lse_small(LseArgs a, int n_rt, int slices) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[FRING * FSTAGE];
  const int M = min(a.ctr[0], a.L);
  const int vt = blockIdx.x / n_rt, rt = blockIdx.x - vt * n_rt, r0 = rt * FR, c0 = vt * FV2;
  if (r0 >= M) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wr = wave >> 1, wv = wave & 1;
  const int row = wave * 8 + (lane >> 3), col = ((lane & 7) ^ ((row >> 1) & 7)) * 8, stages = (a.d + BK - 1) / BK;
  const uint16_t *pw[4], *ph[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    pw[j] = a.W + (int64_t)min(c0 + row + 32 * j, a.V - 1) * a.d + col;
    ph[j] = a.H + (int64_t)a.idx[min(r0 + row + 32 * j, M - 1)] * a.d + col;
  }
  f32x16 acc[2][2] = {};
  small_product<TAIL>(lds, pw, ph, stages, loss_few_start(vt, stages) * BK, a.d, a.zeros, acc);
  float* wave_m = reinterpret_cast<float*>(lds);  // [2][FR] of the two waves with the same rows
  float* wave_s = wave_m + 2 * FR;
  auto off = [](int x) { return 8 * (x >> 2) + (x & 3); };
#pragma unroll
  for (int fr = 0; fr < 2; ++fr) {
    RowState r = row_state_empty();
#pragma unroll
    for (int fv = 0; fv < 2; ++fv) {
      const int v = c0 + wv * 64 + fv * 32 + 4 * (lane >> 5);
      float z[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) z[x] = v + off(x) < a.V ? acc[fv][fr][x] : -INFINITY;
      row_fold<false, 16>(r, z, 0, off);
    }
    row_merge<false>(r, shfl_xor_state(r, 32));
    if (lane < 32) {
      wave_m[wv * FR + wr * 64 + fr * 32 + lane] = r.m;
      wave_s[wv * FR + wr * 64 + fr * 32 + lane] = r.s;
    }
  }
  __syncthreads();
  if (tid < FR && r0 + tid < M) {
    RowState x = row_state_empty(), y = row_state_empty();
    x.m = wave_m[tid];
    x.s = wave_s[tid];
    y.m = wave_m[FR + tid];
    y.s = wave_s[FR + tid];
    row_merge<false>(x, y);
    a.m[(int64_t)(r0 + tid) * slices + vt] = x.m;
    a.s[(int64_t)(r0 + tid) * slices + vt] = x.s;
  }
}

template <bool TAIL>
__global__ __launch_bounds__(NT, 1) void k_loss_dz_small(GradArgs a, int n_rt) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[FRING * FSTAGE];
  const int M = min(a.ctr[0], a.L), Mp = (M + BK - 1) / BK * BK, np = (a.n + BK - 1) / BK * BK;
  const int vt = blockIdx.x / n_rt, rt = blockIdx.x - vt * n_rt, r0 = rt * FR, c0 = vt * FV2;
  if (r0 >= Mp) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wr = wave >> 1, wv = wave & 1;
  const int row = wave * 8 + (lane >> 3), col = ((lane & 7) ^ ((row >> 1) & 7)) * 8, stages = a.dp / BK;
  const uint16_t *pw[4], *ph[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    pw[j] = a.W + (int64_t)(a.v0 + min(c0 + row + 32 * j, a.n - 1)) * a.d + col;
    ph[j] = a.rows + (int64_t)min(r0 + row + 32 * j, Mp - 1) * a.dp + col;
  }
  f32x16 acc[2][2] = {};
  small_product<TAIL>(lds, pw, ph, stages, vt * 7 % stages * BK, a.d, a.zeros, acc);
#pragma unroll
  for (int fr = 0; fr < 2; ++fr) {
    const int r = r0 + wr * 64 + fr * 32 + (lane & 31);
    if (r >= Mp) continue;
    const float lse = a.lse[r], coef = a.coef[r];
    const uint32_t target = float_bf16(a.at_tgt[r]);
    const int hit = a.tgt[r] - a.v0;
#pragma unroll
    for (int fv = 0; fv < 2; ++fv)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + wv * 64 + fv * 32 + 8 * j + 4 * (lane >> 5);
        if (c >= np) continue;
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          b[i] = float_bf16(loss_p(acc[fv][fr][4 * j + i], lse) * coef);
          b[i] = c + i == hit ? target : b[i];
          b[i] = c + i < a.n ? b[i] : 0u;
        }
        *reinterpret_cast<uint2*>(a.dz + (int64_t)r * a.ldz + c) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
      }
  }
}

// d_W of few tiles: both sides by rows of K, 128 x 128 to a workgroup, the same
// ring (460 rows, 4096 entries of 256: 9.8 us, by 256 x 256 tiles 21.5; the step of
// 3700 rows, 1000 entries of 1024: 140 and 177; of 1000, 8000 of 1024, 128 large
// tiles: 170 either way).
__global__ __launch_bounds__(NT, 1) void k_loss_d_W_small(GradArgs a, int n_ct) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[FRING * FSTAGE];
  const int M = min(a.ctr[0], a.L), stages = (M + BK - 1) / BK;
  if (M == 0 && a.accumulate) return;
  const int vt = blockIdx.x / n_ct, ct = blockIdx.x - vt * n_ct, r0 = vt * FV2, c0 = ct * FR;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wr = wave >> 1, wv = wave & 1;
  static_assert(FR == kNarrow && FV2 == kNarrow, "both sides are narrow ones");
  const NarrowSide side(wave, lane);
  const uint16_t *pa = side.source(a.rows, a.dp, c0, a.dp), *pb = side.source(a.dz, a.ldz, r0, (int)a.ldz);
  f32x16 acc[2][2] = {};
  if (stages > 0) {
    int k0 = 0;
    auto issue = [&](int slot) {
      uint16_t* to = lds + slot * FSTAGE + wave * 512;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        __builtin_amdgcn_global_load_lds((const void*)(pa + (int64_t)(k0 + 16 * j) * a.dp), (LDS_AS void*)(to + 4 * j * 512), 16, 0, 0);
        __builtin_amdgcn_global_load_lds((const void*)(pb + (int64_t)(k0 + 16 * j) * a.ldz),
                                         (LDS_AS void*)(to + BK * FR + 4 * j * 512), 16, 0, 0);
      }
      k0 = k0 + BK >= stages * BK ? 0 : k0 + BK;
    };
    // as in small_product
    issue(0);
    issue(1);
    issue(2);
    for (int q = 0; q < stages; ++q) {
      stage_sync<16>();
      issue((q + 3) & (FRING - 1));
      const uint16_t* t = lds + (q & (FRING - 1)) * FSTAGE;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        bf16x8 fa[2], fb[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          fa[f] = side.frag(t, wv * 2 + f, kk);
          fb[f] = side.frag(t + BK * FR, wr * 2 + f, kk);
        }
#pragma unroll
        for (int fv = 0; fv < 2; ++fv)
#pragma unroll
          for (int fr = 0; fr < 2; ++fr) acc[fv][fr] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[fv], fb[fr], acc[fv][fr], 0, 0, 0);
      }
    }
    stage_sync<0>();  // the DMAs behind the last stage
  }
#pragma unroll
  for (int fr = 0; fr < 2; ++fr) {
    const int row = r0 + wr * 64 + fr * 32 + (lane & 31);
    if (row >= a.n) continue;
#pragma unroll
    for (int fv = 0; fv < 2; ++fv)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = c0 + wv * 64 + fv * 32 + 8 * j + 4 * (lane >> 5);
        if (col >= a.d) continue;
        uint2* o = reinterpret_cast<uint2*>(a.d_W + (int64_t)(a.v0 + row) * a.d + col);
        float z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = acc[fv][fr][4 * j + i];
        if (a.accumulate) {
          const uint2 u = *o;
          z[0] += bf16_float(u.x & 0xFFFF);
          z[1] += bf16_float(u.x >> 16);
          z[2] += bf16_float(u.y & 0xFFFF);
          z[3] += bf16_float(u.y >> 16);
        }
        *o = make_uint2(float_bf16(z[0]) | float_bf16(z[1]) << 16, float_bf16(z[2]) | float_bf16(z[3]) << 16);
      }
  }
}

// Few rows: the rows of d_W that are targets, with what dz's rounding left of
// their entries.  They are summed anew, in fp32 and the order of the rows, and take
// their places behind the piece's product; where it is accumulated, whose old
// values are gone then, they go to `fix` before it and to their places at the end
// (k_loss_put).  A workgroup has
// 512 columns of one target, which the first row with it answers for; its waves
// take a quarter of the rows each.  Every target reads all rows, from the caches
// (102 rows of 4096: 17 us; 250: 43).
__device__ __forceinline__ bool first_with(const GradArgs& a, int M, int i, int v) {
  bool before = false;
  for (int k = threadIdx.x & 63; k < M; k += 64) before |= k < i && a.tgt[k] == v;
  return __ballot(before) == 0;
}

__global__ __launch_bounds__(256) void k_loss_targets(GradArgs a) {
  __shared__ float z[kLossFew], part[4][512];
  const int M = min(a.ctr[0], a.L), i = blockIdx.x;
  if (M > kLossFew || i >= M) return;
  const int v = a.tgt[i] - a.v0;
  if (v < 0 || v >= a.n || !first_with(a, M, i, a.tgt[i])) return;
  for (int m = threadIdx.x; m < M; m += 256)
    z[m] = bf16_float(a.dz[(int64_t)m * a.ldz + v]) + (a.tgt[m] - a.v0 == v ? a.left[m] : 0.f);
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.y * 512 + lane * 8;
  const int lo = M * wave / 4, hi = M * (wave + 1) / 4;
  float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < a.d)
    for (int m0 = lo; m0 < hi; m0 += 8) {
      uint4 u[8];  // loads of eight rows together; those behind the last one are the last one's
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = *reinterpret_cast<const uint4*>(a.rows + (int64_t)min(m0 + k, hi - 1) * a.dp + c);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (m0 + k >= hi) break;
        float h[8];
        unpack8(u[k], h);
        const float w = z[m0 + k];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = fmaf(w, h[j], f[j]);
      }
    }
#pragma unroll
  for (int j = 0; j < 8; ++j) part[wave][lane * 8 + j] = f[j];
  __syncthreads();
  if (wave > 0 || c >= a.d) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = (part[0][lane * 8 + j] + part[1][lane * 8 + j]) + (part[2][lane * 8 + j] + part[3][lane * 8 + j]);
  if (a.accumulate) {
    float old[8];
    unpack8(*reinterpret_cast<const uint4*>(a.d_W + (int64_t)(a.v0 + v) * a.d + c), old);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] += old[j];
  }
  uint16_t* row = a.accumulate ? a.fix + (int64_t)i * a.d : a.d_W + (int64_t)(a.v0 + v) * a.d;
  *reinterpret_cast<uint4*>(row + c) = pack8(f);
}

__global__ __launch_bounds__(64) void k_loss_put(GradArgs a) {
  const int M = min(a.ctr[0], a.L), i = blockIdx.x, c = blockIdx.y * 512 + threadIdx.x * 8;
  if (M > kLossFew || i >= M || !first_with(a, M, i, a.tgt[i]) || c >= a.d) return;
  *reinterpret_cast<uint4*>(a.d_W + (int64_t)a.tgt[i] * a.d + c) = *reinterpret_cast<const uint4*>(a.fix + (int64_t)i * a.d + c);
}

}  // namespace

hipError_t launch_loss_lse_small(const LseArgs& a, hipStream_t stream) {
  const int n_rt = (a.L + FR - 1) / FR, slices = (int)loss_few_slices(a.V);
  const dim3 grid((unsigned)slices * (unsigned)n_rt);
  if (a.d % BK == 0)
    hipLaunchKernelGGL(k_loss_lse_small<false>, grid, dim3(NT), 0, stream, a, n_rt, slices);
  else
    hipLaunchKernelGGL(k_loss_lse_small<true>, grid, dim3(NT), 0, stream, a, n_rt, slices);
  return hipGetLastError();
}
hipError_t launch_loss_dz(const GradArgs& a, int grid, hipStream_t stream) {
  if (loss_small(a.n, a.L)) {
    const int n_rt = (a.L + FR - 1) / FR;
    const dim3 small((unsigned)((a.n + FV2 - 1) / FV2) * (unsigned)n_rt);
    if (a.d % BK == 0)
      hipLaunchKernelGGL(k_loss_dz_small<false>, small, dim3(NT), 0, stream, a, n_rt);
    else
      hipLaunchKernelGGL(k_loss_dz_small<true>, small, dim3(NT), 0, stream, a, n_rt);
  } else if (a.d % BK == 0) {
    hipLaunchKernelGGL(k_loss_dz<false>, dim3(grid), dim3(NT), 0, stream, a);
  } else {
    hipLaunchKernelGGL(k_loss_dz<true>, dim3(grid), dim3(NT), 0, stream, a);
  }
  return hipGetLastError();
}
hipError_t launch_loss_d_hidden(const GradArgs& a, int grid, hipStream_t stream) {
  hipLaunchKernelGGL(k_loss_d_hidden, dim3(grid), dim3(NT), 0, stream, a);
  return hipGetLastError();
}
hipError_t launch_loss_d_W(const GradArgs& a, int grid, hipStream_t stream) {
  if (loss_small(a.n, a.d)) {
    const int cols = (a.d + FR - 1) / FR;
    hipLaunchKernelGGL(k_loss_d_W_small, dim3((unsigned)((a.n + FV2 - 1) / FV2) * (unsigned)cols), dim3(NT), 0, stream, a, cols);
    return hipGetLastError();
  }
  // how many rows there are is known on the device: one of the two returns at once
  if (a.L > kLossFew) hipLaunchKernelGGL(k_loss_d_W, dim3(grid), dim3(NT), 0, stream, a);
  const int n_vt = (a.n + FV - 1) / FV, n_ct = (a.d + BT - 1) / BT;
  hipLaunchKernelGGL(k_loss_d_W_few, dim3((unsigned)n_vt * (unsigned)n_ct), dim3(NT), 0, stream, a, n_vt, n_ct);
  return hipGetLastError();
}
hipError_t launch_loss_targets(const GradArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(k_loss_targets, dim3(a.L < kLossFew ? a.L : kLossFew, (a.d + 511) / 512), dim3(256), 0, stream, a);
  return hipGetLastError();
}
hipError_t launch_loss_put(const GradArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(k_loss_put, dim3(a.L < kLossFew ? a.L : kLossFew, (a.d + 511) / 512), dim3(64), 0, stream, a);
  return hipGetLastError();
}
hipError_t launch_loss_join(const GradArgs& a, int grid, hipStream_t stream) {
  hipLaunchKernelGGL(k_loss_join, dim3(16 * grid), dim3(NT), 0, stream, a, grid);
  return hipGetLastError();
}

}  // namespace dllm

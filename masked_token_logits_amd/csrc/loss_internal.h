// What the loss's host side (loss.hip) and its products (loss_gemm.hip) share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dllm_loss.h"

namespace dllm {

constexpr int kLossStep = 64;   // K of a stage: rows, entries and columns are filled up to this
constexpr int kLossTile = 256;  // rows and columns of a product's tile
constexpr int kLossGrid = 256;  // most workgroups of a product

inline int64_t loss_padded(int64_t n) { return (n + kLossStep - 1) / kLossStep * kLossStep; }

// dz is rounded to bf16, and what that leaves of a row's largest entry, the
// target's, is given back to the fp32 sums: to d_hidden always (one more row of W
// each), to d_W with up to so many rows.  With more, d_W's errors average out to
// 1.41 times the output's own rounding; with few, single rows decide them (102
// rows: up to 1.6 times).  Up to as many, d_W has a kernel whose time is its own bytes.
constexpr int kLossFew = 256;

// dz's probability, exp(z - lse): the difference is taken before anything rounds
// it, as (lse - z) / 256 between 0 and 1 (the clamp is the multiply-add's own),
// so logits of any size give no more than 1, and what lies 256 below gives 0.  A
// NaN logit gives a number, too: its row's lse is NaN, and so is its coefficient.
constexpr float kLossPScale = 1.0f / 256.0f;
__device__ __forceinline__ float loss_p(float z, float scaled_lse) {
  const float x = __builtin_amdgcn_fmed3f(fmaf(z, -kLossPScale, scaled_lse), 0.0f, 1.0f);
  return __builtin_amdgcn_exp2f(x * (-1.44269504088896340736f / kLossPScale));
}

// The backward pass of one vocabulary piece.  Rows are the counted positions
// in ascending order, M = ctr[0] of them, filled up to Mp with rows that have
// no gradient.
struct GradArgs {
  const uint16_t* W;        // [V, d]
  const uint16_t* zeros;    // 16 bytes of them
  const uint16_t* rows;     // [Mp, dp] the counted rows of hidden, zeros behind d and M
  const int32_t *idx, *ctr;
  const float* lse;         // [Mp] lse * kLossPScale; 0 behind M
  const float* coef;        // [Mp] grad * weight; NaN where lse is not finite, 0 behind M
  const int32_t* tgt;       // [Mp] the target, -1 behind M
  const float* at_tgt;      // [Mp] dz there
  const float* left;        // [Mp] what its rounding to bf16 leaves of it
  uint16_t* dz;             // [Mp, ldz]: the piece's gradient of the logits
  float* acc;               // the rows' gradient over the pieces so far, in shares of a tile each
  uint16_t* fix;            // [kLossFew, d] few rows, accumulated: d_W's rows of the targets
  uint16_t *d_hidden, *d_W;
  int64_t ldz;              // entries of a whole piece
  int V, d, dp, L;
  int v0, n;                // the piece: entries v0 .. v0 + n - 1
  int first, accumulate;
};

// A product of L rows (at most) and n entries, or of n entries and d columns, is small if its 256 x 256 tiles are
// too few for half the chip; it then has tiles of 128 x 128 (the whole loss of 128
// rows, 16384 entries of 4096, 64 large tiles: 51 us, by large ones 69; 8 rows,
// 32000 of 4096: 53 and 75; 256 rows, 32000 of 2048, 125 tiles: 58 and 53, but
// with the gradients 254 and 265).
inline bool loss_small(int64_t n, int64_t L) {
  return (n + kLossTile - 1) / kLossTile * ((L + kLossTile - 1) / kLossTile) <= kLossGrid / 2;
}

// The small forward product: the running maximum and sum of each row and tile.
constexpr int kLossFewEntries = 128;  // of a tile
// The stage of K that a tile begins with: neighbours ask different channels.
__host__ __device__ inline int loss_few_start(int tile, int stages) { return tile * 7 % stages; }
inline int64_t loss_few_slices(int64_t V) { return (V + kLossFewEntries - 1) / kLossFewEntries; }
struct LseArgs {
  const uint16_t *W, *H, *zeros;
  const int32_t *idx, *ctr;
  float *m, *s;  // [rows][slices]
  int V, d, L;
};
hipError_t launch_loss_lse_small(const LseArgs& a, hipStream_t stream);

// grid: workgroups of the products, the same for all of a call
hipError_t launch_loss_dz(const GradArgs& a, int grid, hipStream_t stream);        // dz
hipError_t launch_loss_d_hidden(const GradArgs& a, int grid, hipStream_t stream);  // acc += dz . W
hipError_t launch_loss_d_W(const GradArgs& a, int grid, hipStream_t stream);       // d_W = dz^T . rows
hipError_t launch_loss_targets(const GradArgs& a, hipStream_t stream);             // few rows: behind d_W, or before it where that accumulates
hipError_t launch_loss_put(const GradArgs& a, hipStream_t stream);                 // and that behind all pieces
hipError_t launch_loss_join(const GradArgs& a, int grid, hipStream_t stream);      // d_hidden = sum of acc's shares

// How d_hidden's product is cut: its tiles' stages as one line, dealt to so
// many workgroups, at least four stages of a whole piece to each.
__host__ __device__ inline int64_t loss_cuts(int64_t tiles, int64_t piece) {
  int64_t n = tiles * (piece / kLossStep) / 4;
  if (n < tiles) n = tiles;
  return n < kLossGrid ? n : kLossGrid;
}

// Shares of acc, a tile's floats each: workgroup g's of tile t is share g + t.
inline int64_t loss_shares(int64_t L, int64_t d, int64_t piece) {
  const int64_t t = (L + kLossTile - 1) / kLossTile * ((d + kLossTile - 1) / kLossTile);
  return t + loss_cuts(t, piece);
}

}  // namespace dllm

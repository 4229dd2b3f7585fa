// What the loss's host side (loss.hip) and its products (loss_gemm.hip) share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dllm_loss.h"

namespace dllm {

constexpr int kLossPad = 64;  // rows and entries of dz are filled up to this

// The backward pass of one vocabulary piece.  Rows are the counted positions
// in ascending order, ctr[0] of them.
struct GradArgs {
  const uint16_t *W, *H;  // [V, d], [L, d]
  const int32_t *idx, *ctr;
  const float *lse, *coef;  // per row: log-sum-exp, and grad * weight
  const int32_t* tgt;       // per row: the target
  uint16_t* dz;             // [rows, ldz]: the piece's gradient of the logits
  float* acc;               // [rows, d]: the rows' gradient over the pieces so far
  uint16_t *d_hidden, *d_W;
  int64_t ldz;
  int V, d, L;
  int v0, n;                // the piece: entries v0 .. v0 + n - 1
  int first, last, accumulate;
};

hipError_t launch_loss_dz(const GradArgs& a, int grid, hipStream_t stream);        // dz
hipError_t launch_loss_d_hidden(const GradArgs& a, int grid, hipStream_t stream);  // acc += dz . W, d_hidden at the last
hipError_t launch_loss_d_W(const GradArgs& a, int grid, hipStream_t stream);       // d_W = dz^T . H

}  // namespace dllm

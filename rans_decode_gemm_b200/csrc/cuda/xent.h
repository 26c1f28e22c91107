// xent.h -- softmax cross entropy over a compressed vocabulary head: plan and
// launch entry point (xent.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "kernels.h"

namespace ansdev {

struct XentPlan {
  uint32_t M, N, K;
  uint32_t grad, f16;
  uint32_t piece;    // W rows of one piece of the vocabulary (the last may hold fewer)
  uint32_t chunk;    // tokens whose probabilities of one piece exist at a time
  int sms;
  // workspace, byte offsets
  size_t off_images, off_probs, off_blocks, off_moved, off_x16, off_factor, off_state, off_acc, off_target, off_gemm, bytes;
};

struct XentArgs {
  const uint16_t* X;
  uint32_t scale_kind;
  const void* scales;
  uint32_t group_k;
  uint32_t vocab;
  const int32_t* targets;
  float* loss;
  float* lse;
  const float* weight;  // null: 1
  uint16_t* dX;         // null: no gradient
  uint32_t* status;
};

// Running state of M rows: reference r (units of log 2), sum l of the others, target
// logit, and this piece's factors of the gradient's sum.  lift: one value.
struct XentState {
  float *ref, *sum, *zt, *alpha, *beta, *lift;
};

// A piece's blocks joined into the state of tokens m0 .. m0 + m - 1.
struct XentJoin {
  XentState st;
  const float2* blocks;    // (reference, sum): [n_blocks][stride], tokens m0 .. m0 + m - 1 from column 0
  uint32_t stride, n_blocks, m0, m, rows, f16;
  uint32_t beside;         // runs beside the next piece's decoding
  uint32_t* moved;         // one bit a token, in order: has blocks under another reference
  uint16_t* probs;         // m x rows, or null
  // the targets' rows of W
  const int32_t* targets;
  const uint8_t* images;
  uint16_t* target_rows;   // M x K in operand form
  uint32_t n0, vocab, K;
};
cudaError_t launch_xent_join(const XentJoin& j, cudaStream_t stream);

// Zeros in the images of rows [first, rows): padding behind the vocabulary, whose
// probabilities are 0, and 0 times an infinity or a NaN is not.
cudaError_t launch_xent_blank(uint8_t* images, uint32_t first, uint32_t rows, uint32_t K, cudaStream_t stream);

void make_xent_plan(const LayerDev& L, uint32_t M, bool grad, int sms, XentPlan* plan);
cudaError_t launch_xent(const XentPlan& plan, const LayerDev& L, const XentArgs& a, void* ws, cudaStream_t stream);

}  // namespace ansdev

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

void make_xent_plan(const LayerDev& L, uint32_t M, bool grad, int sms, XentPlan* plan);
cudaError_t launch_xent(const XentPlan& plan, const LayerDev& L, const XentArgs& a, void* ws, cudaStream_t stream);

}  // namespace ansdev

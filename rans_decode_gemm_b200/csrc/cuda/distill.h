// distill.h -- distillation from a teacher's top logits over a compressed
// vocabulary head: plan and launch entry point (distill.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "kernels.h"
#include "operand.h"

namespace ansdev {

constexpr uint32_t kDistillMaxTop = 256;

struct DistillPlan {
  uint32_t M, N, K, top, vocab_words;
  uint32_t grad, f16;
  uint32_t piece;    // loss only: W rows of a piece.  Gradient: of all but the first
  uint32_t first;    // of the first
  uint32_t chunk;    // tokens at a time
  uint32_t stride;   // of the blocks' references
  int sms;
  size_t off_images, off_probs, off_blocks, off_x16, off_factor, off_state, off_words, off_ids, off_z, off_t, off_coef,
      off_gemm, bytes;
};

struct DistillArgs {
  const uint16_t* X;
  uint32_t scale_kind;
  const void* scales;
  uint32_t group_k;
  uint32_t vocab;
  float per_t;
  const int32_t* ids;        // [M][top]
  const float* logits;       // [M][top]
  const float* teacher_lse;  // [M], or null: the listed logits hold all of the teacher's mass
  float *loss, *lse;
  const float* weight;       // null: 1
  uint16_t* dX;              // null: no gradient
  uint32_t* status;
};

// (the vocabulary may be any up to N: the plan is for N)
void make_distill_plan(const LayerDev& L, uint32_t M, uint32_t top, bool grad, int sms, DistillPlan* plan);
cudaError_t launch_distill(const DistillPlan& plan, const LayerDev& L, const DistillArgs& a, void* ws, cudaStream_t stream);

}  // namespace ansdev

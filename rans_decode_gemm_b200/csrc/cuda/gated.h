// gated.h -- the gated feed-forward block on two compressed layers, and its
// gradient: plans and launch entry points (gated.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "kernels.h"
#include "operand.h"

namespace ansdev {

enum : uint32_t { kActSilu = 0, kActGelu = 1, kActGeluTanh = 2, kActRelu = 3 };

// Workspace of a call (byte offsets): the decoded weights of both layers, gate and
// up images side by side (image j of the gate at 8192 j, of the up at 8192 j +
// 4096), X in f16 where the weights are, and for the gradient the rows that meet
// them in the transposed product.
struct GatedPlan {
  uint32_t M, N, K, f16, grad;
  bool prep;  // gradient: dG and dU need a form of their own (f16, or row scales applied)
  int sms;
  OperandGemmPlan back;
  size_t off_images, off_x16, off_factor, off_rows, off_rows_factor, off_gemm, bytes;
};

struct GatedArgs {
  const uint16_t* X;
  uint32_t scale_kind;
  const void *gate_scales, *up_scales;
  uint32_t group_k, act;
  uint16_t* H;               // forward
  const uint16_t* dH;        // gradient
  uint16_t *dX, *dG, *dU;    // (dX null: not computed)
  uint32_t* status;
};

// (the workspace's first `head` bytes are not used)
void make_gated_plan(const LayerDev& L, uint32_t M, uint32_t scale_kind, bool grad, int sms, size_t head, GatedPlan* plan);
// Through operand images, any M.
cudaError_t launch_gated(const GatedPlan& plan, const LayerDev& gate, const LayerDev& up, const GatedArgs& a, void* ws,
                         cudaStream_t stream);
// X (bf16, M x K) under a power of two of its row, and what its products are times then.
cudaError_t launch_gated_x(const uint16_t* X, uint32_t M, uint32_t K, uint16_t* out, float* factor, cudaStream_t stream);
// H = act(G) * U of products that are there (fp32, M x N), times factor[m] first (or null).  M up to 65535.
cudaError_t launch_gated_join(const float* G, const float* U, const float* factor, uint32_t M, uint32_t N, uint32_t act,
                              uint16_t* H, cudaStream_t stream);

cudaError_t set_live_wait_budget_gated(long long cycles);

}  // namespace ansdev

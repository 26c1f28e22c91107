// verify.h -- verification of drafted tokens from logits: plan and launch entry
// point (verify.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace ansdev {

struct VerifyArgs {
  const float* target;       // logits, row r at r * target_stride
  uint64_t target_stride;
  const float* draft;        // the draft model's logits, or null
  uint64_t draft_stride;
  uint32_t n_seqs, n_drafted, vocab;
  const int32_t* starts;     // [n_seqs + 1]
  const int32_t* tokens;     // [n_drafted]
  const float* u;            // [n_drafted]
  const float* v;            // [n_seqs]
  const float* temperature;  // [n_seqs], or null: 1
  int32_t* accepted;         // [n_seqs]
  int32_t* out;              // [n_drafted + n_seqs]
  uint32_t* status;
};

constexpr uint32_t kVerifyMaxRows = 1u << 20;
constexpr uint32_t kVerifyMaxVocab = 1u << 24;

// The parts that a row's sum comes in, and the workspace that holds them.
struct VerifyPlan {
  uint32_t chunk;  // logits of a part (a multiple of 1024; the last may hold fewer)
  uint32_t n_chunks;
  size_t bytes;
};
void make_verify_plan(uint32_t n_seqs, uint32_t n_drafted, uint32_t vocab, VerifyPlan* plan);
cudaError_t launch_verify(const VerifyPlan& plan, const VerifyArgs& a, void* ws, cudaStream_t stream);

}  // namespace ansdev

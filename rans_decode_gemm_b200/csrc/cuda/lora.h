// lora.h -- low-rank adapters of many requests beside a projection: plans and
// launch entry points (lora.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace ansdev {

constexpr uint32_t kLoraMaxRank = 128;
constexpr uint32_t kLoraMaxAdapters = 256;

struct LoraDev {
  const uint16_t* A;   // bf16 n x rank x K
  const uint16_t* B;   // bf16 n x N x rank
  const float* scale;  // n, or null: 1
  uint32_t n, rank, N, K;
};

// Tokens grouped by adapter, in device memory: positions hold the tokens sorted
// by adapter (those without one left out), adapter a's at [off[a], off[a + 1]),
// both multiples of 16; perm gives each position's token (all ones: none); tiles
// of at most tm positions of one adapter each.
struct LoraGroups {
  uint32_t* n_tiles;
  uint32_t* off;
  uint32_t* perm;
  uint32_t* tile_adapter;
  uint32_t* tile_start;
  uint32_t* tile_count;
};

struct LoraPlan {
  uint32_t M, tm, max_tiles, positions, likely;
  uint32_t few;   // forward pass of few tokens: tiles found where they are used
  int sms;
  uint32_t splits_k, len_k;  // ranges of a sum over K, and their length
  uint32_t splits_n, len_n;  // of a sum over N
  size_t off_groups, off_part, off_h, off_dh, bytes;
};
void make_lora_plan(uint32_t M, const LoraDev& L, bool grad, int sms, LoraPlan* plan);

// Y[m][n] += s_a sum_j (sum_k X[m][k] A_a[j][k]) B_a[n][j], in two parts: what
// needs X only, and what needs Y (launched in this order on one stream, anything
// that leaves the workspace alone between them).
cudaError_t launch_lora_shrink(const LoraPlan& plan, const LoraDev& L, const uint16_t* X, const int32_t* ids,
                               void* ws, uint32_t* status, cudaStream_t stream);
cudaError_t launch_lora_expand(const LoraPlan& plan, const LoraDev& L, const int32_t* ids, float* Y, void* ws,
                               cudaStream_t stream);
// dH[m][j] = s_a sum_n dY[m][n] B_a[n][j];  dA_a = sum_m dH[m]^T X[m];
// dB_a = s_a sum_m dY[m]^T (X[m] A_a^T);  delta[m] = dH[m] A_a where delta is
// given (fp32 M x K, rows of tokens with an adapter only).
// In two parts: dH and X A_a^T, and what is made of them.  With delta, the second
// part runs beside one kernel launched between the two, which has to wait for
// the first as every kernel does, and to leave workspace and operands alone.
cudaError_t launch_lora_grad_shrink(const LoraPlan& plan, const LoraDev& L, const uint16_t* X,
                                    const uint16_t* dY, const int32_t* ids, void* ws, uint32_t* status,
                                    cudaStream_t stream);
cudaError_t launch_lora_grad_outer(const LoraPlan& plan, const LoraDev& L, const uint16_t* X,
                                   const uint16_t* dY, const int32_t* ids, float* dA, float* dB,
                                   float* delta, void* ws, cudaStream_t stream);

}  // namespace ansdev

// operand.h -- decoding a range of a compressed layer into 16-bit tensor-core
// operands, and GEMMs that read those operands either way round.  Host-side
// plans and launch entry points shared by the gradient, adapter and loss
// operators.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "kernels.h"

namespace ansdev {

// Operand images: the weights of a range of W rows as 16-bit values, 4 KB per
// 128 rows x 16 columns (row r at byte 32 r, its two 16-byte halves swapped
// where bit 2 of r is set: the 32-byte shared-memory swizzle), the image of
// the range's rows 128 b .. + 127 and columns 16 j .. + 15 at byte
// (b * K / 16 + j) * 4096.  bf16 weights stay bf16.  Every other format's
// values are exact in f16 (int4 with group scales: q * s, exact for scales in
// [2^-14, 2^12]; row scales are not part of the image).
inline bool operand_is_f16(uint32_t dtype) { return dtype != 1; }
inline size_t operand_bytes(uint64_t rows, uint32_t K) { return static_cast<size_t>(rows) * K * 2; }

// Decodes row blocks [row0, row0 + rows) (multiples of tile_n) into images, one
// every `step` bytes (two layers' images may lie side by side).  beside: starts as the
// decoding before it leaves SMs free and does not wait for it (griddep_beside() in
// ptx.cuh), whose images it does not touch.
constexpr uint32_t kOperandImage = 4096;
cudaError_t launch_operand_decode(const LayerDev& L, uint32_t row0, uint32_t rows,
                                  uint32_t scale_kind, const void* scales, uint32_t group_k,
                                  uint8_t* images, uint32_t* status, int sms, cudaStream_t stream,
                                  uint32_t step = kOperandImage, bool beside = false);

// Rounds of tiles that decoding them takes on that many SMs.
uint32_t operand_decode_rounds(uint32_t tiles, uint32_t ctas);

// Rows of a bf16 matrix as f16 under a power of two of their own: out[m][c] =
// f16(in[m][c] * s[c] * 2^e), factor[m] = 2^-e, with e such that the row's
// largest finite magnitude lands in [2^14, 2^15).  scale_kind: s[c] as bf16 (1)
// or fp32 (2), else 1.  f16 false: out[m][c] = bf16(in[m][c] * s[c]), factor 1
// (for bf16 weights that carry row scales).
cudaError_t launch_row_prep(const uint16_t* in, uint32_t M, uint32_t C, uint32_t scale_kind,
                            const void* scales, bool f16, uint16_t* out, float* factor, cudaStream_t stream);

// A GEMM on operand images of `rows` W rows and K columns, 16-bit row-major
// operands, fp32 sums:
//   transposed:  out[m][k] = sum_n G[m][n] W[n][k]        (k < K)
//   logits:      z[m][n] = f[m] s_n sum_k X[m][k] W[n][k]  (n < rows)
// The transposed sum may be cut into `splits` ranges of n.
struct OperandGemmPlan {
  uint32_t trans, f16;
  uint32_t M, rows, K;
  uint32_t bn;       // tokens of one tile
  uint32_t splits;   // ranges of the sum (transposed only)
  uint32_t sms;
};
OperandGemmPlan plan_operand_gemm(bool trans, bool f16, uint32_t M, uint32_t rows, uint32_t K, int sms);
// Workspace of a sum that is cut (256-byte aligned).
size_t operand_gemm_workspace(const OperandGemmPlan& plan);

// What happens to the transposed sums v[m][k].
struct OperandGemmOut {
  // out16: out16[m * ld + k] = bf16(beta[m] * v + add[m * ld + k]), the addend
  //   taken for rows with 0 <= ids[m] < n_ids only (add may be null).
  // out32: out32[m * ld + k] = alpha[m] * (its old value) + beta[m] * v;
  //   alpha null: the old value is not read.  beta null: 1.
  // drops: where beta[m] is 0 the row is, whatever v is (NaN beside infinite weights).
  float* out32;
  uint16_t* out16;
  uint32_t ld;
  const float* alpha;
  const float* beta;
  const float* add;
  const int32_t* ids;
  uint32_t n_ids;
  uint32_t drops;
};

// What happens to the logits: they are folded into softmax sums, 32 rows of W
// (a block) at a time.  With r a reference in units of log 2 (a whole number),
//   e[m][n] = 2^(z[m][n] log2(e) - r),  blocks[block][m] = (r, sum of the block's e),
//   probs[m * rows + n] = e * s_n * lift (16-bit; null: not stored),
// except that rows n0 + n >= vocab count for nothing, and neither does the token's
// target, whose logit is stored in zt[m]: it has no part in r either, or the others
// of a token that is all but certain would be stored far below 1.  r is ref_in[m],
// unless the block's largest logit lies more than kXentSlack above it: then r is
// that logit, rounded up.
constexpr float kXentSlack = 5.75f;    // e^4: what probabilities may exceed 1 by
constexpr float kXentNone = -3.0e38f;  // the reference before any logit
struct XentEpilogue {
  const float* factor;     // f[m], or null: 1
  uint32_t scale_kind;     // s_n: bf16 (1), fp32 (2) at scales[n], else 1
  const void* scales;
  const float* lift;       // one value
  const float* ref_in;
  const int32_t* targets;
  float* zt;
  float2* blocks;          // [rows / 32][stride]
  uint32_t stride;
  uint16_t* probs;
  uint32_t n0, vocab;
  // Lists in place of targets (listed given, targets and zt not): per token up to
  // `top` rows of W, ascending (-1: none), whose logits go to z_listed, in the same
  // places.  listed: bit b % 32 of word [(b / 32) * listed_stride + m] is set where
  // block b of 32 rows (of the whole vocabulary) holds rows of token m's list.  Logits
  // are times per_t (probs are not).
  // probs then have probs_ld columns.
  const uint32_t* listed;
  uint32_t listed_stride, top, probs_ld;
  const int32_t* ids;
  float* z_listed;
  float per_t;
};

// A second layer of the same shape in a transposed product, whose sum runs over
// both: out[m][k] = sum_n G[m][n] W[n][k] + G2[m][n] W2[n][k].  (The plan is made
// for twice a layer's rows.)  step: bytes from an image to a layer's next.
struct OperandPair {
  const uint8_t* images;
  const void* rows16;
  uint32_t step;
};

// Exactly one of out (transposed) and xent (logits) is given.
cudaError_t launch_operand_gemm(const OperandGemmPlan& plan, const uint8_t* images, const void* rows16,
                                const OperandGemmOut* out, const XentEpilogue* xent, void* ws, uint32_t* status,
                                cudaStream_t stream, const OperandPair* pair = nullptr);

// Internal test hook: sums in parts only where their kernel was built with that many
// registers a thread (what it needs, or more).
void set_part_registers(uint32_t least);

cudaError_t set_live_wait_budget_operand(long long cycles);
cudaError_t set_live_wait_budget_operand_gemm(long long cycles);

// 2-D tiled tensor map (gemm.cu).
cudaError_t encode_tmap(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t inner,
                        uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                        CUtensorMapSwizzle swizzle);

}  // namespace ansdev

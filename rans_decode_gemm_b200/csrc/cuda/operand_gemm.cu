// operand_gemm.cu -- tcgen05 GEMMs on operand images (operand.h), either way
// round, and the row kernels beside them.
//
//   logits       D[n][m] = sum_k W[n][k] X[m][k]
//   transposed   D[k][m] = sum_n W[n][k] G[m][n]    (a gradient that leaves the layer)
//
// One layout of W serves both.  An image is 128 rows of 32 bytes under the
// 32-byte swizzle.  Read as rows n with 16 consecutive k it is a K-major
// operand; read as 16 consecutive output features k by 8-row groups of n it is
// the canonical MN-major one (atoms of 16 k x 8 n, 256 bytes apart along n),
// so the transposed product needs neither a second copy of W nor a
// transposing load.  Tokens are the MMA's N dimension in both: 128 rows of W
// (or of W^T) by up to 256 tokens, fp32 accumulators in two TMEM sets so that
// the epilogue of a tile overlaps the MMAs of the next.
//
// A stage holds 64 steps of the sum: 16 KB of W by one copy (logits: four
// consecutive images; transposed: one box of half of each of eight images)
// and a 64 x bn box of the tokens by TMA under the 128-byte swizzle.  Four K = 16
// MMAs and one commit a stage.  (Eight 2 KB copies instead of the box held the
// transposed product at 158 ns an MMA against 115.)
//
// The logits never reach memory: the epilogue turns them into exponentials
// under a reference that is known before the tile (the row's reference after
// the earlier pieces), and only a block of 32 logits that rises far above it
// takes a reference of its own.  A warp holds 32 rows n by 32 tokens at a time, one n
// a lane; maxima and sums over n for the 32 tokens take 31 exchanges each
// (halving the tokens and the lanes together) and end with token j in lane j.
// What bounds it: loads against 4 stages of 48 KB (192 KB, about 1.8 us of them).
// 115 ns an MMA, 70 % of the tensor pipe's cycles, 1.25-1.33 PFLOP/s on 2048 x 9472
// x 4096 either way (117 and 125 us); with 3 stages 135 and 161 us.  A pair of
// CTAs on one tile (32 KB a stage and SM) measured the same, and L2 prefetches
// of the boxes 10-25 % more.  A last round of tiles dealt out evenly to all SMs
// (the CTA with a tile's end adding the others' parts), 1.73 rounds in place of 2,
// gained 1 %: the SMs that run share the chip's power.
// Warps: 0 loads, 1 MMA issue (and TMEM owner), 2-9 epilogue: two for each
// quarter of TMEM's lanes, on alternating 32 tokens.  (With one each, the
// epilogue of the logits took longer than the MMAs of a K = 2048 tile.)
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "gemm_common.cuh"
#include "launch.h"
#include "operand.h"
#include "rans_core.cuh"

namespace ansdev {

constexpr uint32_t kOgBM = 128, kOgBK = 64;
constexpr uint32_t kOgABytes = kOgBM * kOgBK * 2;  // 16 KB
constexpr uint32_t kOgEpiWarps = 8;
constexpr uint32_t kOgThreads = (2 + kOgEpiWarps) * 32;
constexpr uint32_t kOgMaxStages = 8;
constexpr uint32_t kOgSmemTiles = 200 * 1024;  // stages
constexpr uint32_t kOgSmem = kOgSmemTiles + 1024;

struct OperandGemmDev {
  const uint8_t* images;
  CUtensorMap tmap_b;  // tokens: 64 x b_box_rows boxes, 128-byte swizzle
  CUtensorMap tmap_a;  // transposed: images as rows of 512 eight-byte words, boxes of 256 x 8
  OperandGemmOut out;
  XentEpilogue xent;
  uint32_t f16;
  uint32_t* status;
  uint32_t M, bn, m_blocks, n_tiles, splits;
  float* parts;            // where splits > 1: [tile without its split][split][bn][128]
  uint32_t k_slabs;      // images per 128-row block (K / 16)
  uint32_t out_cols;     // rows of D that exist: rows of W, or K (transposed)
  uint32_t n_kb;         // stages of the whole sum
  uint32_t b_box_rows, stages, stage_bytes;
  uint32_t idesc, idesc_tail;
};

// Over the warp's lanes for each of 32 values at once: lane j ends with value
// j's result.
template <typename Op>
__device__ __forceinline__ float across_lanes(float (&x)[32], uint32_t lane, Op op) {
#pragma unroll
  for (uint32_t w = 16; w > 0; w >>= 1) {
    const bool up = (lane & w) != 0;
#pragma unroll
    for (uint32_t i = 0; i < w; ++i) {
      const float give = up ? x[i] : x[i + w], keep = up ? x[i + w] : x[i];
      x[i] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, give, w));
    }
  }
  return x[0];
}

// 32 logits of 32 tokens (v[j]: this lane's row n against token m + j), folded
// as XentEpilogue says.  c: this lane's row in the piece; m: first token; token
// m + lane's reference, target and factor come in tok.
struct XentToken {
  float ref, factor;
  int32_t target;
};
__device__ __forceinline__ XentToken xent_token(const XentEpilogue& E, uint32_t m, bool in) {
  XentToken t;
  t.ref = in ? __ldcg(E.ref_in + m) : 0.0f;
  t.target = in ? __ldg(E.targets + m) : -1;
  t.factor = E.factor != nullptr && in ? __ldcg(E.factor + m) : 1.0f;
  return t;
}
__device__ __forceinline__ void xent_fold(const XentEpilogue& E, uint32_t f16, uint32_t rows, const uint32_t (&v)[32],
                                          float scale, float lift, uint32_t c, uint32_t m, uint32_t n_tok,
                                          uint32_t lane, const XentToken& tok) {
  constexpr float kLog2E = 1.4426950408889634f;
  const bool m_in = lane < n_tok;
  const float ref_in = tok.ref, factor = tok.factor;
  const int32_t target = tok.target;
  const bool n_in = E.n0 + c < E.vocab;
  float z[32], x[32];
#pragma unroll
  for (uint32_t j = 0; j < 32; ++j) {
    z[j] = __uint_as_float(v[j]) * scale;
    if (E.factor != nullptr) z[j] *= __shfl_sync(0xFFFFFFFFu, factor, j);
    if (!n_in) z[j] = -INFINITY;
  }
  // targets among this warp's rows (one that is past the vocabulary is none): few
  // and far between, so that the loops above and below carry no test for them
  const uint32_t first = E.n0 + c - lane;
  const bool hit = target >= 0 && static_cast<uint32_t>(target) < E.vocab && static_cast<uint32_t>(target) - first < 32u;
  for (uint32_t hits = __ballot_sync(0xFFFFFFFFu, hit); hits != 0; hits &= hits - 1) {
    const uint32_t k = __ffs(hits) - 1;
    if (lane == static_cast<uint32_t>(__shfl_sync(0xFFFFFFFFu, target, k)) - first) {
#pragma unroll
      for (uint32_t j = 0; j < 32; ++j) {
        if (j == k) {
          E.zt[m + j] = z[j];
          z[j] = -INFINITY;
        }
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (uint32_t j = 0; j < 32; ++j) x[j] = z[j];
  const float top = across_lanes(x, lane, [](float a, float b) { return fmaxf(a, b); }) * kLog2E;
  float ref = ref_in;
  if (top > ref_in + kXentSlack && top <= 3.0e38f) ref = ceilf(top);
#pragma unroll
  for (uint32_t j = 0; j < 32; ++j) {
    const float r = __shfl_sync(0xFFFFFFFFu, ref, j);
    // (the approximate instruction: 2^-22, the same in every use)
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x[j]) : "f"(fmaf(z[j], kLog2E, -r)));
  }
  const float ps = n_in ? scale * lift : 0.0f;  // (a padding row's scale may be anything)
  if (E.probs != nullptr) {
    uint16_t* p = E.probs + static_cast<uint64_t>(m) * rows + c;
    auto store = [&](uint32_t j) {
      const float q = x[j] * ps;
      *p = f16 ? __half_as_ushort(__float2half_rn(q)) : __bfloat16_as_ushort(__float2bfloat16_rn(q));
      p += rows;
    };
    if (n_tok == 32) {
#pragma unroll
      for (uint32_t j = 0; j < 32; ++j) store(j);
    } else {
#pragma unroll
      for (uint32_t j = 0; j < 32; ++j)
        if (j < n_tok) store(j);
    }
  }
  const float sum = across_lanes(x, lane, [](float a, float b) { return a + b; });
  if (m_in) E.blocks[static_cast<uint64_t>(c / 32) * E.stride + m + lane] = make_float2(ref, sum);
}

template <bool kTrans>
__global__ void __launch_bounds__(kOgThreads, 1) operand_gemm_kernel(const __grid_constant__ OperandGemmDev P) {
  extern __shared__ __align__(1024) uint8_t dsmem_raw[];
  __shared__ __align__(8) uint64_t full[kOgMaxStages], empty[kOgMaxStages];
  __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2], mma_done;
  __shared__ uint32_t tmem_slot;
  __shared__ uint32_t abort_flag;

  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // stages on a 1024-byte boundary (the 128-byte swizzle atom)
  const uint32_t smem_s = (smem_u32(dsmem_raw) + 1023u) & ~1023u;
  const uint32_t n_st = P.stages;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (uint32_t i = 0; i < kOgMaxStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kOgEpiWarps);  // one arrival per epilogue warp
    }
    mbar_init(&mma_done, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  } else if (warp == 0 && lane == 0) {
    prefetch_tmap(&P.tmap_b);
    if (kTrans) prefetch_tmap(&P.tmap_a);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  volatile uint32_t* abort = &abort_flag;
  griddep_wait();
  griddep_launch_dependents();

  // tile t: row block ab, token block mb, range sp of the sum.  Row block
  // major, so that the CTAs running at one time share W through L2.
  const uint32_t per_ab = P.m_blocks * P.splits;
  auto tile_of = [&](uint32_t t, uint32_t& ab, uint32_t& mb, uint32_t& sp, uint32_t& kb0, uint32_t& kb1) {
    ab = t / per_ab;
    const uint32_t r = t - ab * per_ab;
    sp = r / P.m_blocks;
    mb = r - sp * P.m_blocks;
    kb0 = cta_begin(P.n_kb, P.splits, sp);
    kb1 = cta_begin(P.n_kb, P.splits, sp + 1);
  };

  if (warp == 0) {
    // ======================= loads =======================
    if (lane == 0) {
      uint32_t it = 0, s = 0, ph = 1;  // the first pass over the ring finds it free
      bool live = true;
      for (uint32_t t = blockIdx.x; t < P.n_tiles && live; t += gridDim.x) {
        uint32_t ab, mb, sp, kb0, kb1;
        tile_of(t, ab, mb, sp, kb0, kb1);
        for (uint32_t kb = kb0; kb < kb1; ++kb, ++it) {
          if (it >= n_st && !wait_live(&empty[s], ph, abort, P.status, 20)) {
            live = false;
            break;
          }
          const uint32_t bar = smem_u32(&full[s]);
          const uint32_t a_s = smem_s + s * P.stage_bytes, b_s = a_s + kOgABytes;
          if (kTrans) {
            // half of each of eight images in one box.  Where the last block
            // of k holds fewer, the box runs into the next row block's (or, at
            // the end, is filled with zeros): rows of D that are never stored.
            mbar_arrive_expect_tx_s(bar, kOgABytes + P.b_box_rows * kOgBK * 2);
            tma_load_2d_s(a_s, &P.tmap_a, static_cast<int32_t>((kb & 1u) * 256u),
                          static_cast<int32_t>((kb >> 1) * P.k_slabs + 8 * ab), bar);
          } else {
            const uint32_t cnt = min(4u, P.k_slabs - 4 * kb);
            mbar_arrive_expect_tx_s(bar, cnt * kSlabBytes + P.b_box_rows * kOgBK * 2);
            bulk_g2s_s(a_s, P.images + (static_cast<uint64_t>(ab) * P.k_slabs + 4 * kb) * kSlabBytes,
                       cnt * kSlabBytes, bar);
          }
          tma_load_2d_s(b_s, &P.tmap_b, static_cast<int32_t>(kb * kOgBK), static_cast<int32_t>(mb * P.bn), bar);
          if (++s == n_st) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // loads still in flight (only after an abort) land before exit
      const uint32_t first = it > n_st ? it - n_st : 0;
      for (uint32_t q = first; q < it; ++q) wait_drain(&full[q % n_st], (q / n_st) & 1u, P.status);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ======================= MMA issue =======================
    if (lane == 0) {
      // logits A: K-major, 8-row groups 256 B apart (SBO), image j of a stage
      // is its K = 16 slice j.  Transposed A: MN-major, atoms of 16 k 2 KB
      // apart (LBO), 8-row groups of n 256 B apart (SBO); the K = 16 slice j
      // starts 16 rows (512 B) further.  B: 128-byte swizzle, 8-row groups
      // 1024 B apart, slice j 32 j bytes into each row.
      const uint64_t da = (kTrans ? (128ull << 16) : (1ull << 16)) | (16ull << 32) | (1ull << 46) | (6ull << 61);
      const uint64_t db = (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
      uint32_t s = 0, ph = 0, acc = 0;
      bool live = true;
      for (uint32_t t = blockIdx.x; t < P.n_tiles && live; t += gridDim.x, ++acc) {
        uint32_t ab, mb, sp, kb0, kb1;
        tile_of(t, ab, mb, sp, kb0, kb1);
        const uint32_t b = acc & 1u;
        if (acc >= 2 && !wait_live(&acc_empty[b], ((acc >> 1) + 1) & 1u, abort, P.status, 21)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + b * 256;
        // the last token block is narrower when M is not a multiple of bn
        const uint32_t idesc = mb == P.m_blocks - 1 ? P.idesc_tail : P.idesc;
        for (uint32_t kb = kb0; kb < kb1; ++kb) {
          if (!wait_live(&full[s], ph, abort, P.status, 22)) {
            live = false;
            break;
          }
          tc_fence_after();
          const uint32_t a16 = (smem_s + s * P.stage_bytes) >> 4, b16 = a16 + (kOgABytes >> 4);
          const uint32_t cnt = kTrans ? 4u : min(4u, P.k_slabs - 4 * kb);
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j)
            if (j < cnt)
              umma_f16(d_tmem, da | (a16 + j * ((kTrans ? 512u : kSlabBytes) >> 4)), db | (b16 + 2 * j), idesc,
                       (kb != kb0 || j != 0) ? 1u : 0u);
          umma_commit(&empty[s]);
          if (++s == n_st) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (live) umma_commit(&acc_full[b]);
      }
      umma_commit(&mma_done);
      wait_drain(&mma_done, 0, P.status);
    }
    __syncwarp();
  } else {
    // ======================= epilogue (warps 2-9) =======================
    // 32 tokens at a time.  Transposed: what is read of global memory for them
    // (the old values or the addend, 32 independent loads; the tokens' factors,
    // one a lane) is asked for before the previous 32 are stored, and for a
    // tile's first 32 before its sums are ready.  Logits: likewise the tokens'
    // references, targets and factors.
    const uint32_t quad = warp & 3u, turn = 32u * ((warp - 2) >> 2);
    const OperandGemmOut& O = P.out;
    // (a part of a sum that is cut goes to memory as it is)
    const bool cut = kTrans && P.splits > 1;
    const bool rmw = kTrans && !cut && O.out32 != nullptr && O.alpha != nullptr;
    const bool adds = kTrans && !cut && O.out32 == nullptr && O.add != nullptr;
    const float lift = kTrans ? 1.0f : __ldcg(P.xent.lift);
    uint32_t acc = 0;
    for (uint32_t t = blockIdx.x; t < P.n_tiles; t += gridDim.x, ++acc) {
      uint32_t ab, mb, sp, kb0, kb1;
      tile_of(t, ab, mb, sp, kb0, kb1);
      const uint32_t b = acc & 1u;
      const uint32_t c = ab * kOgBM + 32 * quad + lane;  // this thread's row of D
      const bool c_in = c < P.out_cols;
      const uint32_t m0 = mb * P.bn;
      const uint32_t cols = min(P.bn, P.M - m0);
      const uint64_t tile_at = static_cast<uint64_t>(m0) * O.ld + c;
      float* out32 = O.out32;
      float scale = 1.0f;
      if (!kTrans) {
        if (P.xent.scale_kind == 1) scale = bf16_to_f32(__ldg(static_cast<const uint16_t*>(P.xent.scales) + c));
        else if (P.xent.scale_kind == 2) scale = __ldg(static_cast<const float*>(P.xent.scales) + c);
      }
      float old[32], my_alpha = 1.0f, my_beta = 1.0f;
      XentToken tok;
      auto ask = [&](uint32_t c0) {
        const uint32_t m = m0 + c0 + lane;
        const bool m_in = c0 + lane < cols;
        if constexpr (!kTrans) {
          tok = xent_token(P.xent, m, m_in);
          return;
        }
        if (rmw) my_alpha = m_in ? __ldcg(O.alpha + m) : 0.0f;
        if (!cut && O.beta != nullptr) my_beta = m_in ? __ldcg(O.beta + m) : 0.0f;
        if (rmw || adds) {
          uint32_t want = cols - c0 < 32 ? (1u << (cols - c0)) - 1u : 0xFFFFFFFFu;
          if (adds) {
            // tokens that take the addend
            const int32_t id = m_in ? __ldg(O.ids + m) : -1;
            want = __ballot_sync(0xFFFFFFFFu, id >= 0 && static_cast<uint32_t>(id) < O.n_ids);
          }
          if (!c_in) want = 0;
          const float* src = (rmw ? out32 : O.add) + tile_at + static_cast<uint64_t>(c0) * O.ld;
#pragma unroll
          for (uint32_t j = 0; j < 32; ++j)
            old[j] = (want >> j) & 1u ? __ldcg(src + static_cast<uint64_t>(j) * O.ld) : 0.0f;
        }
      };
      if (turn < cols) ask(turn);
      const bool ok = wait_live(&acc_full[b], (acc >> 1) & 1u, abort, P.status, 23, 64);
      tc_fence_after();
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      if (turn >= cols && lane == 0) mbar_arrive(&acc_empty[b]);
      for (uint32_t c0 = turn; c0 < cols; c0 += 64) {
        uint32_t v[32];
        tmem_ld32(tmem_base + ((32 * quad) << 16) + b * 256 + c0, v);
        tmem_ld_wait();
        if (c0 + 64 >= cols) {
          // this warp has read its last of the tile's sums
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[b]);
        }
        if constexpr (!kTrans) {
          const XentToken now = tok;
          if (c0 + 64 < cols) ask(c0 + 64);
          xent_fold(P.xent, P.f16, P.out_cols, v, scale, lift, c, m0 + c0, min(32u, cols - c0), lane, now);
        } else if (cut) {
          const uint64_t at = static_cast<uint64_t>(ab * P.m_blocks + mb) * P.splits + sp;
          float* part = P.parts + (at * P.bn + c0) * kOgBM + 32 * quad + lane;
#pragma unroll
          for (uint32_t j = 0; j < 32; ++j)
            if (c0 + j < cols) __stcg(part + j * kOgBM, __uint_as_float(v[j]));
        } else {
          float x[32];
#pragma unroll
          for (uint32_t j = 0; j < 32; ++j) {
            x[j] = __uint_as_float(v[j]);
            if (O.beta != nullptr) x[j] *= __shfl_sync(0xFFFFFFFFu, my_beta, j);
            if (rmw) x[j] = fmaf(__shfl_sync(0xFFFFFFFFu, my_alpha, j), old[j], x[j]);
            else if (adds) x[j] += old[j];
          }
          if (c0 + 64 < cols) ask(c0 + 64);
          const uint64_t at = tile_at + static_cast<uint64_t>(c0) * O.ld;
          if (c_in) {
#pragma unroll
            for (uint32_t j = 0; j < 32; ++j) {
              if (c0 + j >= cols) break;
              const uint64_t i = at + static_cast<uint64_t>(j) * O.ld;
              if (O.out32 != nullptr) out32[i] = x[j];
              else O.out16[i] = __bfloat16_as_ushort(__float2bfloat16_rn(x[j]));
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, 512);
}

// The parts of sums that are cut, added in order and stored: a warp a token of a
// tile, four rows of D a lane.  (Parts in planes of M x K, added by a kernel over the
// whole of them, held a bf16 4096 x 4096 gradient of 200 tokens at 45.6 us against 42.7;
// added by the CTA with a tile's last part, behind flags, at 51.3.)
struct JoinParts {
  OperandGemmOut out;
  const float* parts;
  uint32_t M, bn, m_blocks, splits, out_cols;
};
__global__ void __launch_bounds__(256) join_parts_kernel(const __grid_constant__ JoinParts P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tile = blockIdx.x, ab = tile / P.m_blocks, j = blockIdx.y * 8 + threadIdx.x / 32;
  const uint32_t m = (tile - ab * P.m_blocks) * P.bn + j, c = 4 * (threadIdx.x % 32), k = ab * kOgBM + c;
  if (m >= P.M || j >= P.bn || k >= P.out_cols) return;  // (out_cols is a multiple of 16)
  const OperandGemmOut& O = P.out;
  const float* part = P.parts + (static_cast<uint64_t>(tile) * P.splits * P.bn + j) * kOgBM + c;
  const uint64_t at = static_cast<uint64_t>(m) * O.ld + k, step = static_cast<uint64_t>(P.bn) * kOgBM;
  float4 old = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float alpha = 0.0f;
  bool adds = false;
  if (O.out32 != nullptr && O.alpha != nullptr) {
    alpha = __ldcg(O.alpha + m);
    old = __ldcg(reinterpret_cast<const float4*>(O.out32 + at));
    adds = true;
  } else if (O.out32 == nullptr && O.add != nullptr) {
    const int32_t id = __ldg(O.ids + m);
    adds = id >= 0 && static_cast<uint32_t>(id) < O.n_ids;
    alpha = 1.0f;
    if (adds) old = __ldcg(reinterpret_cast<const float4*>(O.add + at));
  }
  float4 v = __ldcg(reinterpret_cast<const float4*>(part));
#pragma unroll 4
  for (uint32_t s = 1; s < P.splits; ++s) {
    const float4 u = __ldcg(reinterpret_cast<const float4*>(part + s * step));
    v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
  }
  if (O.beta != nullptr) {
    const float f = __ldcg(O.beta + m);
    v.x *= f; v.y *= f; v.z *= f; v.w *= f;
  }
  if (adds) {
    v.x = fmaf(alpha, old.x, v.x); v.y = fmaf(alpha, old.y, v.y); v.z = fmaf(alpha, old.z, v.z); v.w = fmaf(alpha, old.w, v.w);
  }
  if (O.out32 != nullptr) {
    *reinterpret_cast<float4*>(O.out32 + at) = v;
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(O.out16 + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

OperandGemmPlan plan_operand_gemm(bool trans, bool f16, uint32_t M, uint32_t rows, uint32_t K, int sms) {
  OperandGemmPlan p;
  p.trans = trans;
  p.f16 = f16;
  p.M = M;
  p.rows = rows;
  p.K = K;
  p.sms = static_cast<uint32_t>(sms);
  const uint64_t blocks = ((trans ? K : rows) + 127) / 128;
  const uint32_t n_kb = ((trans ? rows : K) + kOgBK - 1) / kOgBK;
  // Rounds of tiles over the SMs, at about 300 ns a stage and 0.65 ns for each of
  // its tokens (one round of 32 stages measured 19.3, 19.4, 22.2 and 28.7 us at
  // 32, 64, 128 and 256 tokens, some 9 of it the launch and its ends).  A narrow
  // tile hardly runs faster, so it only serves to fill the SMs.  A sum over n may
  // be cut instead (8 stages a part at least): its parts are written and read at
  // about 4 TB/s by a second kernel.
  uint64_t least = ~0ull;
  for (uint32_t bn = 256; bn >= 32; bn /= 2) {
    if (bn > 32 && M <= bn / 2) continue;
    const uint64_t tiles = blocks * ((M + bn - 1) / bn);
    const uint32_t most = trans ? std::min(16u, std::max(1u, n_kb / 8)) : 1u;
    for (uint32_t s = 1; s <= most; ++s) {
      const uint64_t rounds = (tiles * s + p.sms - 1) / p.sms;
      uint64_t cost = rounds * ((n_kb + s - 1) / s) * (300 + bn * 13 / 20);
      if (s > 1) cost += 3000 + static_cast<uint64_t>(M) * K * s / 500;
      if (cost < least) {
        least = cost;
        p.bn = bn;
        p.splits = s;
      }
    }
  }
  return p;
}

size_t operand_gemm_workspace(const OperandGemmPlan& p) {
  if (p.splits <= 1) return 0;
  const size_t tiles = static_cast<size_t>((p.K + kOgBM - 1) / kOgBM) * ((p.M + p.bn - 1) / p.bn);
  return tiles * p.splits * p.bn * kOgBM * 4;
}

cudaError_t launch_operand_gemm(const OperandGemmPlan& plan, const uint8_t* images, const void* rows16,
                                const OperandGemmOut* out, const XentEpilogue* xent, void* ws, uint32_t* status,
                                cudaStream_t stream) {
  if (plan.M == 0) return cudaSuccess;
  OperandGemmDev P;
  std::memset(&P, 0, sizeof(P));
  P.images = images;
  if (out) P.out = *out;
  if (xent) P.xent = *xent;
  P.f16 = plan.f16;
  P.status = status;
  P.M = plan.M;
  P.bn = plan.bn;
  P.m_blocks = (plan.M + plan.bn - 1) / plan.bn;
  P.splits = plan.splits;
  P.parts = static_cast<float*>(ws);
  P.k_slabs = plan.K / 16;
  P.out_cols = plan.trans ? plan.K : plan.rows;
  const uint32_t red = plan.trans ? plan.rows : plan.K;
  P.n_kb = (red + kOgBK - 1) / kOgBK;
  P.n_tiles = (P.out_cols + kOgBM - 1) / kOgBM * P.m_blocks * P.splits;
  P.b_box_rows = std::min(plan.M, plan.bn);
  P.stage_bytes = kOgABytes + plan.bn * kOgBK * 2;
  P.stages = std::min(kOgMaxStages, kOgSmemTiles / P.stage_bytes);
  const uint32_t tail = plan.M - (P.m_blocks - 1) * plan.bn;
  // bit 15: A is MN-major
  P.idesc = idesc_f16(plan.f16 ? 0u : 1u, 128, plan.bn) | (plan.trans ? 1u << 15 : 0u);
  P.idesc_tail = idesc_f16(plan.f16 ? 0u : 1u, 128, (tail + 15) / 16 * 16) | (plan.trans ? 1u << 15 : 0u);
  cudaError_t e = encode_tmap(&P.tmap_b, CU_TENSOR_MAP_DATA_TYPE_UINT16, rows16, red, plan.M,
                              static_cast<uint64_t>(red) * 2, kOgBK, P.b_box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  if (plan.trans) {
    const uint64_t images_n = static_cast<uint64_t>(plan.rows / 128) * P.k_slabs;
    e = encode_tmap(&P.tmap_a, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, images, kSlabBytes / 8, images_n, kSlabBytes, 256, 8,
                    CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e != cudaSuccess) return e;
  }
  auto kern = plan.trans ? operand_gemm_kernel<true> : operand_gemm_kernel<false>;
  static std::atomic<uint64_t> attr_set{0};
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(attr_set.load() & (1ull << dev))) {
    e = cudaFuncSetAttribute(operand_gemm_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kOgSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(operand_gemm_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kOgSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set.fetch_or(1ull << dev);
  }
  const uint32_t grid = std::min(P.n_tiles, plan.sms);
  e = launch_pdl(kern, dim3(grid), dim3(kOgThreads), kOgSmem, stream, P);
  if (e != cudaSuccess || plan.splits == 1) return e;
  // a CTA 8 tokens of a tile
  const JoinParts J{P.out, P.parts, plan.M, plan.bn, P.m_blocks, plan.splits, P.out_cols};
  return launch_pdl(join_parts_kernel, dim3(P.n_tiles / plan.splits, (P.b_box_rows + 7) / 8), dim3(256), 0, stream, J);
}

// ---- rows of bf16 as scaled f16 ----------------------------------------------
// One CTA a row: the largest finite magnitude first, then the conversion (the
// row comes from L2 the second time).  f16 under a power of two of the row's
// own (its largest value then lies in [2^14, 2^15)) keeps 11 bits of every value
// down to 2^-28 of the row's largest, and what is smaller is off by at most 2^-39
// of it; bf16 would keep 8 bits of every v * s.  Infinities and NaN pass through.  Runs beside the decoding
// of the weights.
constexpr uint32_t kPrepThreads = 256;
__global__ void __launch_bounds__(kPrepThreads) row_prep_kernel(const uint16_t* __restrict__ in, uint32_t C,
                                                                uint32_t kind, const void* scales, bool f16,
                                                                uint16_t* __restrict__ out,
                                                                float* __restrict__ factor) {
  __shared__ float part[kPrepThreads / 32];
  griddep_beside();
  const uint64_t row = static_cast<uint64_t>(blockIdx.x) * C;
  auto values = [&](uint32_t c, float (&v)[8]) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(in + row + c));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
    if (kind == 1) {
      const uint4 s = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(scales) + c));
      const uint32_t u[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] *= __uint_as_float(u[k] << 16);
        v[2 * k + 1] *= __uint_as_float(u[k] & 0xFFFF0000u);
      }
    } else if (kind == 2) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(scales) + c);
      const float4 s = __ldg(p), r = __ldg(p + 1);
      v[0] *= s.x; v[1] *= s.y; v[2] *= s.z; v[3] *= s.w;
      v[4] *= r.x; v[5] *= r.y; v[6] *= r.z; v[7] *= r.w;
    }
  };
  float top = 0.0f;
  for (uint32_t c = threadIdx.x * 8; c < C; c += kPrepThreads * 8) {
    float v[8];
    values(c, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float a = fabsf(v[k]);
      if (a <= 3.402823466e38f) top = fmaxf(top, a);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
  __syncthreads();
#pragma unroll
  for (uint32_t k = 0; k < kPrepThreads / 32; ++k) top = fmaxf(top, part[k]);
  // 2^e with top * 2^e in [2^14, 2^15); both powers stay normal numbers
  const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
  const int e = top == 0.0f || !f16 ? 0 : min(126, max(-113, 14 - ex));
  const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
  if (threadIdx.x == 0) factor[blockIdx.x] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  for (uint32_t c = threadIdx.x * 8; c < C; c += kPrepThreads * 8) {
    float v[8];
    values(c, v);
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (f16) {
        const __half2 h = __floats2half2_rn(v[2 * k] * up, v[2 * k + 1] * up);
        o[k] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        o[k] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(out + row + c) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  griddep_beside_end();
}

cudaError_t launch_row_prep(const uint16_t* in, uint32_t M, uint32_t C, uint32_t scale_kind,
                            const void* scales, bool f16, uint16_t* out, float* factor, cudaStream_t stream) {
  if (M == 0) return cudaSuccess;
  return launch_pdl(row_prep_kernel, dim3(M), dim3(kPrepThreads), 0, stream, in, C, scale_kind, scales, f16,
                    out, factor);
}

cudaError_t set_live_wait_budget_operand_gemm(long long cycles) {
  return cudaMemcpyToSymbol(g_live_wait_budget, &cycles, sizeof(cycles));
}

}  // namespace ansdev

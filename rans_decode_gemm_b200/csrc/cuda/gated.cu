// gated.cu -- the gated feed-forward block on two compressed layers:
//
//   G = X Wg^T,  U = X Wu^T,  H = act(G) * U
//   dG = dH * U * act'(G),  dU = dH * act(G),  dX = dG Wg + dU Wu
//
// Both layers are decoded into operand images (operand.h), gate and up side by
// side, and one tcgen05 product meets both: 128 tokens are the MMA's M, 128 rows of
// Wg and the same 128 of Wu its N = 256, so that a token's g_n and u_n end in one
// TMEM lane, 128 columns apart, and the thread that reads them has all that H_n, or
// dG_n and dU_n, take.  G and U never reach memory; the gradient computes them
// again.  dX is one transposed product over both layers' rows (operand_gemm.cu).
//
// A stage of a wide tile holds 64 steps of the sum: 16 KB of tokens by TMA (128-byte
// swizzle) and 32 KB of images by one copy.  An image's rows are K-major under the 32-byte
// swizzle, so 8 KB of a gate and an up image are one 256-row operand.  Where the tiles
// would leave SMs idle they are of 64 or 32 rows: a box of that part of each of eight
// images.
//
// Measured alone (fp8 14336 x 4096, 2048 tokens): the decoding 67 us a layer, the product
// 362 (481 GFLOP, 1.33 PFLOP/s).  int8 with the gradient: 67 a layer, the product 447, of
// which its epilogue (58 MB of dH read, 235 MB written) adds some 80, dX 373.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "gated.h"
#include "gemm_common.cuh"
#include "launch.h"
#include "rans_core.cuh"

namespace ansdev {

constexpr uint32_t kGaBM = 128, kGaBK = 64;
constexpr uint32_t kGaABytes = kGaBM * kGaBK * 2;           // 16 KB of tokens
// kBN rows of both layers; narrow tiles take two blocks of 64 a stage, whose MMAs are as
// short as a stage's barriers are long (int4 14336 x 4096, 2048 tokens in tiles of 64 rows:
// 539 us, with a block a stage 699)
__host__ __device__ constexpr uint32_t ga_block_bytes(uint32_t bn) { return kGaABytes + 2 * bn * kGaBK * 2; }
__host__ __device__ constexpr uint32_t ga_blocks(uint32_t bn) { return bn == 128 ? 1u : 2u; }
__host__ __device__ constexpr uint32_t ga_stage_bytes(uint32_t bn) { return ga_blocks(bn) * ga_block_bytes(bn); }
__host__ __device__ constexpr uint32_t ga_stages(uint32_t bn) { return 192 * 1024 / ga_stage_bytes(bn); }
constexpr uint32_t kGaSmem = 192 * 1024 + 1024;
constexpr uint32_t kGaEpiWarps = 16;
constexpr uint32_t kGaThreads = (2 + kGaEpiWarps) * 32;

// act(g) and, where asked, its derivative.  Sigmoids for tanh and erfc for 1 + erf:
// the small values at negative g keep their digits.
template <bool kSlope>
__device__ __forceinline__ void activation(uint32_t act, float g, float& value, float& slope) {
  if (act == kActRelu) {
    value = g < 0.0f ? 0.0f : g;  // (NaN stays)
    if (kSlope) slope = g > 0.0f ? 1.0f : 0.0f;
  } else if (act == kActGelu) {
    const float p = 0.5f * erfcf(-0.70710678118654752f * g);
    value = g * p;
    if (kSlope) slope = fmaf(g * 0.39894228040143268f, __expf(-0.5f * g * g), p);
  } else {
    float y = g, dy = 1.0f;  // value = g * sigmoid(y)
    if (act == kActGeluTanh) {
      constexpr float kA = 1.5957691216057308f;  // 2 sqrt(2 / pi)
      const float q = 0.044715f * g * g;
      y = kA * fmaf(g, q, g);
      if (kSlope) dy = kA * fmaf(3.0f, q, 1.0f);
    }
    const float e = __expf(-y);
    const float p = __fdividef(1.0f, 1.0f + e);  // (0 from 2^126 on)
    value = g * p;
    // p' = p (1 - p) y', and 1 - p = e p (far out there is nothing of it, and g y' may be infinite)
    if (kSlope) slope = e > 1e30f || e < 1e-30f ? p : fmaf(g * dy, p * (e * p), p);
  }
}

// Rows of the transposed product: dG and dU times the row scales, before they are
// rounded to bf16.  In f16 they come under a power of two of the token's that no value
// of its can pass 2^15 with: |dG s| <= max |dH| * 1.14 |x| sqrt(K) * (the largest weight,
// scale and all) * (the largest scale), and |dU s| likewise (|act'| < 1.13, |act(g)| <=
// |g|).  A bound need not be met: it is some 2^7 above what a trained layer's values
// come to, and f16 holds 11 bits of them down to 2^-28 of it, so 2^-21 of the largest.
// Where a row of far larger scales has no part in a token's gradient the bound can be
// 2^20 and more too large; gated_rows_kernel sees to such tokens.
struct GatedRows {
  uint16_t *gate, *up;      // null: dG and dU themselves are the rows
  const float* bound;       // [M]: max |dH| * 1.14 |x| sqrt(K) * (the largest code); null: no power of two
  const float* scale_parts; // kScaleParts largest scales
  float* factor;            // [M]: 2^-e, for the product's sums
  float* top;               // [M]: the largest magnitude that a token's rows hold
};
constexpr uint32_t kScaleParts = 64;

struct GatedDev {
  const uint8_t* images;
  CUtensorMap tmap_x;       // tokens: 64 x b_rows boxes, 128-byte swizzle
  CUtensorMap tmap_w;       // narrow tiles: images as rows of 512 eight-byte words, boxes of 4 bn x 8
  const float* factor;      // a token's factor, or null: 1
  const void *gate_scales, *up_scales;
  uint32_t scale_kind, act;
  uint16_t* H;
  const uint16_t* dH;
  uint16_t *dG, *dU;
  GatedRows rows;
  uint32_t* status;
  uint32_t M, N, m_blocks, n_tiles, k_slabs, n_kb, box_rows, f16;
};

// Eight row scales from n on.
__device__ __forceinline__ void row_scales8(uint32_t kind, const void* scales, uint32_t n, float (&s)[8]) {
  if (kind == 1) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(scales) + n));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s[2 * k] = __uint_as_float(w[k] << 16);
      s[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(scales) + n);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    s[0] = a.x; s[1] = a.y; s[2] = a.z; s[3] = a.w;
    s[4] = b.x; s[5] = b.y; s[6] = b.z; s[7] = b.w;
  }
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t f16x2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool kGrad, uint32_t kBN>
__global__ void __launch_bounds__(kGaThreads, 1) gated_gemm_kernel(const __grid_constant__ GatedDev P) {
  constexpr uint32_t kGaStages = ga_stages(kBN), kGaStageBytes = ga_stage_bytes(kBN);
  constexpr uint32_t kBlocks = ga_blocks(kBN), kBlockBytes = ga_block_bytes(kBN);
  extern __shared__ __align__(1024) uint8_t dsmem_raw[];
  __shared__ __align__(8) uint64_t full[kGaStages], empty[kGaStages];
  __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2], mma_done;
  __shared__ uint32_t tmem_slot;
  __shared__ uint32_t abort_flag;

  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t smem_s = (smem_u32(dsmem_raw) + 1023u) & ~1023u;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (uint32_t i = 0; i < kGaStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kGaEpiWarps);  // one arrival per epilogue warp
    }
    mbar_init(&mma_done, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  } else if (warp == 0 && lane == 0) {
    prefetch_tmap(&P.tmap_x);
    if (kBN < 128) prefetch_tmap(&P.tmap_w);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  volatile uint32_t* abort = &abort_flag;
  griddep_wait();
  griddep_launch_dependents();

  // tile t: rows kBN ab of both layers, tokens 128 mb; row block major, so that the
  // CTAs running at one time share the weights through L2
  if (warp == 0) {
    // ======================= loads =======================
    if (lane == 0) {
      uint32_t it = 0, s = 0, ph = 1;  // the first pass over the ring finds it free
      bool live = true;
      for (uint32_t t = blockIdx.x; t < P.n_tiles && live; t += gridDim.x) {
        const uint32_t ab = t / P.m_blocks, mb = t - ab * P.m_blocks;
        for (uint32_t kb0 = 0; kb0 < P.n_kb; kb0 += kBlocks, ++it) {
          if (it >= kGaStages && !wait_live(&empty[s], ph, abort, P.status, 20)) {
            live = false;
            break;
          }
          const uint32_t bar = smem_u32(&full[s]);
          const uint32_t here = min(kBlocks, P.n_kb - kb0);
          if constexpr (kBN == 128) {
            const uint32_t bytes = min(4u, P.k_slabs - 4 * kb0) * 2 * kSlabBytes;
            mbar_arrive_expect_tx_s(bar, bytes + P.box_rows * kGaBK * 2);
            bulk_g2s_s(smem_s + s * kGaStageBytes + kGaABytes,
                       P.images + (static_cast<uint64_t>(ab) * P.k_slabs + 4 * kb0) * 2 * kSlabBytes, bytes, bar);
          } else {
            mbar_arrive_expect_tx_s(bar, here * (kBlockBytes - kGaABytes + P.box_rows * kGaBK * 2));
          }
#pragma unroll
          for (uint32_t q = 0; q < kBlocks; ++q) {
            if (q >= here) break;
            const uint32_t kb = kb0 + q, a_s = smem_s + s * kGaStageBytes + q * kBlockBytes;
            if constexpr (kBN < 128) {
              // (where the last block of k holds fewer images, the box runs into the next
              // row block's, or is filled with zeros: operands that no MMA takes)
              constexpr uint32_t kParts = 128 / kBN;
              const uint32_t block = ab / kParts, part = ab - block * kParts;
              tma_load_2d_s(a_s + kGaABytes, &P.tmap_w, static_cast<int32_t>(part * kBN * 4),
                            static_cast<int32_t>(2 * (block * P.k_slabs + 4 * kb)), bar);
            }
            tma_load_2d_s(a_s, &P.tmap_x, static_cast<int32_t>(kb * kGaBK), static_cast<int32_t>(mb * kGaBM), bar);
          }
          if (++s == kGaStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // loads still in flight (only after an abort) land before exit
      const uint32_t first = it > kGaStages ? it - kGaStages : 0;
      for (uint32_t q = first; q < it; ++q) wait_drain(&full[q % kGaStages], (q / kGaStages) & 1u, P.status);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ======================= MMA issue =======================
    if (lane == 0) {
      // tokens: 128-byte swizzle, 8-row groups 1024 B apart, K = 16 slice j 32 j bytes
      // into each row.  Weights: 32-byte swizzle, 8-row groups 256 B apart, slice j the
      // j-th pair of images.
      const uint64_t da = (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
      const uint64_t db = (1ull << 16) | (16ull << 32) | (1ull << 46) | (6ull << 61);
      uint32_t s = 0, ph = 0, acc = 0;
      bool live = true;
      for (uint32_t t = blockIdx.x; t < P.n_tiles && live; t += gridDim.x, ++acc) {
        const uint32_t b = acc & 1u;
        if (acc >= 2 && !wait_live(&acc_empty[b], ((acc >> 1) + 1) & 1u, abort, P.status, 21)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + b * 2 * kBN;
        const uint32_t idesc = idesc_f16(P.f16 ? 0u : 1u, 128, 2 * kBN);
        for (uint32_t kb0 = 0; kb0 < P.n_kb; kb0 += kBlocks) {
          if (!wait_live(&full[s], ph, abort, P.status, 22)) {
            live = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (uint32_t q = 0; q < kBlocks; ++q) {
            if (kb0 + q >= P.n_kb) break;
            const uint32_t a16 = (smem_s + s * kGaStageBytes + q * kBlockBytes) >> 4, b16 = a16 + (kGaABytes >> 4);
            const uint32_t cnt = min(4u, P.k_slabs - 4 * (kb0 + q));
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
              if (j < cnt)
                umma_f16(d_tmem, da | (a16 + 2 * j), db | (b16 + j * (kBN * 64 >> 4)), idesc,
                         (kb0 + q != 0 || j != 0) ? 1u : 0u);
          }
          umma_commit(&empty[s]);
          if (++s == kGaStages) {
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
    // ======================= epilogue (warps 2-17) =======================
    // a token a lane; four warps for each quarter of TMEM's lanes, which take the tile's
    // rows in turn, 16 at a time
    const uint32_t quad = warp & 3u, turn = (warp - 2) >> 2;
    float top_scale = 1.0f;
    if (kGrad && P.rows.bound != nullptr && P.scale_kind != 0) {
      top_scale = fmaxf(__ldcg(P.rows.scale_parts + lane), __ldcg(P.rows.scale_parts + 32 + lane));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top_scale = fmaxf(top_scale, __shfl_xor_sync(0xFFFFFFFFu, top_scale, d));
      // (row scales come in G or U and in the row itself)
      if (P.scale_kind != 3) top_scale *= top_scale;
    }
    uint32_t acc = 0;
    for (uint32_t t = blockIdx.x; t < P.n_tiles; t += gridDim.x, ++acc) {
      const uint32_t ab = t / P.m_blocks, mb = t - ab * P.m_blocks;
      const uint32_t b = acc & 1u;
      const uint32_t m = mb * kGaBM + 32 * quad + lane;
      const bool m_in = m < P.M;
      const float f = P.factor != nullptr && m_in ? __ldcg(P.factor + m) : 1.0f;
      float up = 1.0f, up2 = 1.0f;
      if (kGrad && P.rows.bound != nullptr && m_in) {
        // 2^e with the bound times 2^e in [2^14, 2^15), in two steps: up to 2^141, which no
        // fp32 holds, and a row scale times the first alone stays finite (|e| / 2 <= 71; the
        // scale's square is in the bound)
        const float bound = __ldcg(P.rows.bound + m) * top_scale;
        const int ex = static_cast<int>(__float_as_uint(bound) >> 23) - 127;  // (-127: 2^-126 and less)
        const int e = max(-113, 14 - ex);
        up = __uint_as_float(static_cast<uint32_t>(e / 2 + 127) << 23);
        up2 = __uint_as_float(static_cast<uint32_t>(e - e / 2 + 127) << 23);
        // (2^-e is below the normal numbers from e = 127 on, and exact)
        if (ab == 0 && turn == 0)
          P.rows.factor[m] = __uint_as_float(e <= 126 ? static_cast<uint32_t>(127 - e) << 23 : 1u << (149 - e));
      }
      const uint64_t row = static_cast<uint64_t>(m) * P.N;
      const bool ok = wait_live(&acc_full[b], (acc >> 1) & 1u, abort, P.status, 23, 64);
      tc_fence_after();
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      if (16 * turn >= kBN && lane == 0) mbar_arrive(&acc_empty[b]);
      [[maybe_unused]] float top = 0.0f;
#pragma unroll
      for (uint32_t c0 = 16 * turn; c0 < kBN; c0 += 64) {
        const uint32_t n0 = ab * kBN + c0;
        uint32_t g[16], u[16];
        const uint32_t at = tmem_base + ((32 * quad) << 16) + b * 2 * kBN + c0;
        tmem_ld16(at, g);
        tmem_ld16(at + kBN, u);
        uint4 d[2];
        if (kGrad) {
#pragma unroll
          for (uint32_t k = 0; k < 2; ++k)
            d[k] = m_in ? __ldg(reinterpret_cast<const uint4*>(P.dH + row + n0) + k) : make_uint4(0, 0, 0, 0);
        }
        tmem_ld_wait();
        if (c0 + 64 >= kBN) {
          // this warp has read its last of the tile's sums
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[b]);
        }
#pragma unroll
        for (uint32_t k = 0; k < 2; ++k) {
          float sg[8], su[8];
          if (P.scale_kind == 1 || P.scale_kind == 2) {
            row_scales8(P.scale_kind, P.gate_scales, n0 + 8 * k, sg);
            row_scales8(P.scale_kind, P.up_scales, n0 + 8 * k, su);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) sg[i] = su[i] = 1.0f;
          }
          uint32_t o[4], o2[4], q[4], q2[4];
          const uint32_t dw[4] = {d[k].x, d[k].y, d[k].z, d[k].w};
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i) {
            float r[2], r2[2];
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) {
              const uint32_t j = 8 * k + 2 * i + h;
              const float gv = __uint_as_float(g[j]) * sg[2 * i + h] * f;
              const float uv = __uint_as_float(u[j]) * su[2 * i + h] * f;
              float value, slope;
              activation<kGrad>(P.act, gv, value, slope);
              if (kGrad) {
                const float dh = __uint_as_float(h ? dw[i] & 0xFFFF0000u : dw[i] << 16);
                r[h] = dh * (uv * slope);
                r2[h] = dh * value;
              } else {
                r[h] = value * uv;
              }
            }
            o[i] = bf16x2(r[0], r[1]);
            if (kGrad) {
              o2[i] = bf16x2(r2[0], r2[1]);
              if (P.rows.gate != nullptr) {
                const float s0 = sg[2 * i] * up, s1 = sg[2 * i + 1] * up, t0 = su[2 * i] * up, t1 = su[2 * i + 1] * up;
                const float v[4] = {r[0] * s0 * up2, r[1] * s1 * up2, r2[0] * t0 * up2, r2[1] * t1 * up2};
                q[i] = P.f16 ? f16x2(v[0], v[1]) : bf16x2(v[0], v[1]);
                q2[i] = P.f16 ? f16x2(v[2], v[3]) : bf16x2(v[2], v[3]);
#pragma unroll
                for (const float a : v) top = fmaxf(top, fabsf(a));
              }
            }
          }
          if (m_in) {
            const uint64_t to = row + n0 + 8 * k;
            *reinterpret_cast<uint4*>((kGrad ? P.dG : P.H) + to) = make_uint4(o[0], o[1], o[2], o[3]);
            if (kGrad) {
              *reinterpret_cast<uint4*>(P.dU + to) = make_uint4(o2[0], o2[1], o2[2], o2[3]);
              if (P.rows.gate != nullptr) {
                *reinterpret_cast<uint4*>(P.rows.gate + to) = make_uint4(q[0], q[1], q[2], q[3]);
                *reinterpret_cast<uint4*>(P.rows.up + to) = make_uint4(q2[0], q2[1], q2[2], q2[3]);
              }
            }
          }
        }
      }
      // (the order of maxima changes nothing)
      if (kGrad && P.rows.bound != nullptr && m_in && top > 0.0f)
        atomicMax(reinterpret_cast<int*>(P.rows.top + m), __float_as_int(top));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, 512);
}

// ---- products that are there ---------------------------------------------------
// X under a power of two of its row, for products that take it as f16: the row's largest
// finite value lies in [2^14, 2^15), and f16 then holds all 8 bits of the others down to
// 2^-31 of it and is off by 2^-39 of it below.  A CTA a token; with it a call of few
// tokens takes 2 to 4 us more (int8 14336 x 4096, 1 token: 181.8 to 184.7).
__global__ void __launch_bounds__(256) gated_x_kernel(const uint16_t* __restrict__ X, uint32_t K, uint16_t* __restrict__ out,
                                                      float* __restrict__ factor) {
  __shared__ float part[8];
  griddep_wait();
  griddep_launch_dependents();
  const uint64_t row = static_cast<uint64_t>(blockIdx.x) * K;
  auto load = [&](uint32_t c) { return __ldg(reinterpret_cast<const uint4*>(X + row + c)); };
  float top = 0.0f;
  for (uint32_t c = threadIdx.x * 8; c < K; c += 2048) {
    const uint4 q = load(c);
    for (const uint32_t w : {q.x, q.y, q.z, q.w})
      for (const uint32_t h : {w << 16, w & 0xFFFF0000u}) {
        const float a = fabsf(__uint_as_float(h));
        if (a <= 3.402823466e38f) top = fmaxf(top, a);
      }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
  __syncthreads();
#pragma unroll
  for (uint32_t k = 0; k < 8; ++k) top = fmaxf(top, part[k]);
  // (both powers stay normal numbers)
  const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
  const int e = top == 0.0f ? 0 : min(126, max(-113, 14 - ex));
  const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
  if (threadIdx.x == 0) factor[blockIdx.x] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  for (uint32_t c = threadIdx.x * 8; c < K; c += 2048) {
    const uint4 q = load(c);
    auto times = [&](uint32_t w) {
      return bf16x2(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
    };
    *reinterpret_cast<uint4*>(out + row + c) = make_uint4(times(q.x), times(q.y), times(q.z), times(q.w));
  }
}

cudaError_t launch_gated_x(const uint16_t* X, uint32_t M, uint32_t K, uint16_t* out, float* factor, cudaStream_t stream) {
  return launch_pdl(gated_x_kernel, dim3(M), dim3(256), 0, stream, X, K, out, factor);
}

// factor: of a token's G and U, or null.  Eight of a token's values a thread.
__global__ void __launch_bounds__(256) gated_join_kernel(const float* __restrict__ G, const float* __restrict__ U,
                                                         const float* factor, uint32_t n8, uint32_t act,
                                                         uint16_t* __restrict__ H) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t n = blockIdx.x * 256 + threadIdx.x;
  if (n >= n8) return;
  const uint64_t i = static_cast<uint64_t>(blockIdx.y) * n8 + n;
  const float f = factor != nullptr ? __ldcg(factor + blockIdx.y) : 1.0f;
  uint32_t o[4];
#pragma unroll
  for (uint32_t k = 0; k < 2; ++k) {
    const float4 g = __ldcg(reinterpret_cast<const float4*>(G) + 2 * i + k);
    const float4 u = __ldcg(reinterpret_cast<const float4*>(U) + 2 * i + k);
    const float gv[4] = {g.x, g.y, g.z, g.w}, uv[4] = {u.x, u.y, u.z, u.w};
    float r[4], slope;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      activation<false>(act, gv[j] * f, r[j], slope);
      r[j] *= uv[j] * f;
    }
    o[2 * k] = bf16x2(r[0], r[1]);
    o[2 * k + 1] = bf16x2(r[2], r[3]);
  }
  reinterpret_cast<uint4*>(H)[i] = make_uint4(o[0], o[1], o[2], o[3]);
}

cudaError_t launch_gated_join(const float* G, const float* U, const float* factor, uint32_t M, uint32_t N, uint32_t act,
                              uint16_t* H, cudaStream_t stream) {
  const uint32_t n8 = N / 8;
  return launch_pdl(gated_join_kernel, dim3((n8 + 255) / 256, M), dim3(256), 0, stream, G, U, factor, n8, act, H);
}

// ---- bounds of the gradient's rows ----------------------------------------------
// The largest scales of both layers, in kScaleParts parts.  (Group scales are part of
// the images' values and bound those; row scales are met once more by the rows.)
__global__ void __launch_bounds__(256) gated_scales_kernel(const void* gate, const void* up, uint32_t kind, uint64_t count,
                                                           float* parts) {
  __shared__ float part[8];
  griddep_wait();
  griddep_launch_dependents();
  float top = 0.0f;
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x; i < 2 * count; i += kScaleParts * 256) {
    const void* from = i < count ? gate : up;
    const uint64_t n = i < count ? i : i - count;
    const float s = fabsf(kind == 2 ? __ldg(static_cast<const float*>(from) + n)
                                    : bf16_to_f32(__ldg(static_cast<const uint16_t*>(from) + n)));
    if (s <= 3.402823466e38f) top = fmaxf(top, s);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int k = 1; k < 8; ++k) top = fmaxf(top, part[k]);
  parts[blockIdx.x] = top;
}

// Beside the decoding: 1.14 max |dH| |x| sqrt(K) times the largest code, of finite
// values.  A CTA a token.
__global__ void __launch_bounds__(256) gated_bound_kernel(const uint16_t* __restrict__ X, const uint16_t* __restrict__ dH,
                                                          uint32_t N, uint32_t K, float per, float* __restrict__ bound,
                                                          float* __restrict__ rows_top) {
  __shared__ float part[8][2];
  griddep_beside();
  auto values = [&](const uint16_t* p, float (&v)[8]) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = fabsf(__uint_as_float(w[k] << 16));
      v[2 * k + 1] = fabsf(__uint_as_float(w[k] & 0xFFFF0000u));
    }
  };
  // (the norm under the row's largest, so that no square passes fp32)
  const uint64_t m = blockIdx.x;
  float top_h = 0.0f, top_x = 0.0f, v[8];
  for (uint32_t c = threadIdx.x * 8; c < N; c += 2048) {
    values(dH + m * N + c, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) top_h = v[k] <= 3.402823466e38f ? fmaxf(top_h, v[k]) : top_h;
  }
  for (uint32_t c = threadIdx.x * 8; c < K; c += 2048) {
    values(X + m * K + c, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) top_x = v[k] <= 3.402823466e38f ? fmaxf(top_x, v[k]) : top_x;
  }
  auto across = [&](float x, uint32_t slot, bool sum) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const float o = __shfl_xor_sync(0xFFFFFFFFu, x, d);
      x = sum ? x + o : fmaxf(x, o);
    }
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32][slot] = x;
    return x;
  };
  across(top_h, 0, false);
  across(top_x, 1, false);
  __syncthreads();
  for (int k = 0; k < 8; ++k) {
    top_h = fmaxf(top_h, part[k][0]);
    top_x = fmaxf(top_x, part[k][1]);
  }
  const float down = top_x > 0.0f ? 1.0f / top_x : 0.0f;
  float sum = 0.0f;
  for (uint32_t c = threadIdx.x * 8; c < K; c += 2048) {
    values(X + m * K + c, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float y = v[k] <= 3.402823466e38f ? v[k] * down : 0.0f;
      sum = fmaf(y, y, sum);
    }
  }
  __syncthreads();
  across(sum, 0, true);
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0f;
    for (int k = 0; k < 8; ++k) sum += part[k][0];
    // (the largest fp32 in place of what is past it)
    bound[m] = fminf(top_h * sqrtf(sum * static_cast<float>(K)) * top_x * per, 3.0e38f);
    rows_top[m] = 0.0f;
  }
  griddep_beside_end();
}

// Tokens whose largest row value lies below 2^-12, 2^26 and more below their bound: f16's
// steps of 2^-24 there are 2^-12 of it, more than what bf16 leaves of a value.  Their rows
// come of dG and dU as they are rounded, under a power of two of their own largest.  Where
// no token is one the call takes 2 us more (int8 4096 x 4096, 200 tokens: 111.6 to 113.7; the
// kernel alone 5.5 us for 2048 tokens).
constexpr float kRowsLow = 1.0f / 4096;
constexpr uint32_t kRowsTokens = 8;  // a CTA
struct GatedLowRows {
  const uint16_t *dG, *dU;
  const void *gate_scales, *up_scales;
  GatedRows rows;
  uint32_t scale_kind, M, N;
};
__global__ void __launch_bounds__(512) gated_rows_kernel(const __grid_constant__ GatedLowRows P) {
  __shared__ float part[16][2];
  griddep_wait();
  griddep_launch_dependents();
  // (each thread the same: eight tokens' maxima at once)
  const uint32_t m0 = blockIdx.x * kRowsTokens;
  uint32_t low = 0;
#pragma unroll
  for (uint32_t k = 0; k < kRowsTokens; ++k) {
    const float held = m0 + k < P.M ? __ldcg(P.rows.top + m0 + k) : 0.0f;
    low |= (held < kRowsLow && held > 0.0f ? 1u : 0u) << k;
  }
  for (; low != 0; low &= low - 1) {
    const uint32_t m = m0 + __ffs(low) - 1;
    const uint64_t row = static_cast<uint64_t>(m) * P.N;
    // eight values of dG (half 0) or dU (half 1), and those times their scales
    auto values = [&](uint32_t half, uint32_t n, float (&v)[8], float (&vs)[8]) {
      const uint4 u = __ldcg(reinterpret_cast<const uint4*>((half ? P.dU : P.dG) + row + n));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      float s[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
      if (P.scale_kind == 1 || P.scale_kind == 2) row_scales8(P.scale_kind, half ? P.up_scales : P.gate_scales, n, s);
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) {
        v[k] = __uint_as_float(k & 1 ? w[k / 2] & 0xFFFF0000u : w[k / 2] << 16);
        vs[k] = v[k] * s[k];
      }
    };
    float top = 0.0f, top_v = 0.0f, v[8], vs[8];
    for (uint32_t half = 0; half < 2; ++half)
      for (uint32_t n = 8 * threadIdx.x; n < P.N; n += 4096) {
        values(half, n, v, vs);
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
          top = fmaxf(top, fabsf(vs[k]));
          top_v = fmaxf(top_v, fabsf(v[k]));
        }
      }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      top_v = fmaxf(top_v, __shfl_xor_sync(0xFFFFFFFFu, top_v, d));
    }
    __syncthreads();  // (the token before has been read)
    if (threadIdx.x % 32 == 0) {
      part[threadIdx.x / 32][0] = top;
      part[threadIdx.x / 32][1] = top_v;
    }
    __syncthreads();
    for (uint32_t k = 0; k < 16; ++k) {
      top = fmaxf(top, part[k][0]);
      top_v = fmaxf(top_v, part[k][1]);
    }
    // (near the end of bf16's own range dG and dU have fewer bits than the rows)
    const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    if (!(top_v >= 0x1p-100f) || ex < -110 || ex > 126) continue;
    const float up = __uint_as_float(static_cast<uint32_t>(14 - ex + 127) << 23);
    if (threadIdx.x == 0) P.rows.factor[m] = __uint_as_float(static_cast<uint32_t>(127 - 14 + ex) << 23);
    for (uint32_t half = 0; half < 2; ++half)
      for (uint32_t n = 8 * threadIdx.x; n < P.N; n += 4096) {
        values(half, n, v, vs);
        *reinterpret_cast<uint4*>((half ? P.rows.up : P.rows.gate) + row + n) =
            make_uint4(f16x2(vs[0] * up, vs[1] * up), f16x2(vs[2] * up, vs[3] * up), f16x2(vs[4] * up, vs[5] * up),
                       f16x2(vs[6] * up, vs[7] * up));
      }
  }
}

static size_t aligned(size_t n) { return (n + 1023) / 1024 * 1024; }

// The tile's rows: rounds of tiles over the SMs, at 395, 277 and 259 ns for 64 steps of
// the sum (a narrow tile's take more a row, so that it only serves to fill the SMs), and
// the last epilogue, which nothing hides: 16, 8 and 5 us with the gradient.  (int4 with
// the gradient, by tiles of 128, 64 and 32 rows: 4096 x 4096, 200 tokens 120, 101 and
// 111 us, 301 tokens 130, 126 and 139; 14336 x 4096, 2048 tokens 921, 997 and 1,321;
// 1024 x 1024, 40 tokens 70, 57 and 57.)
static uint32_t gated_rows_of_tile(uint32_t M, uint32_t N, uint32_t K, bool grad, uint32_t sms) {
  const uint64_t m_blocks = (M + kGaBM - 1) / kGaBM, n_kb = (K + kGaBK - 1) / kGaBK;
  uint64_t least = ~0ull;
  uint32_t best = 128;
  for (const uint32_t bn : {128u, 64u, 32u}) {
    const uint64_t rounds = (N / bn * m_blocks + sms - 1) / sms;
    const uint64_t last = bn == 128 ? 16000 : bn == 64 ? 8000 : 5000;
    const uint64_t cost = rounds * n_kb * (bn == 128 ? 395 : bn == 64 ? 277 : 259) + (grad ? last : last / 4);
    if (cost < least) {
      least = cost;
      best = bn;
    }
  }
  return best;
}

void make_gated_plan(const LayerDev& L, uint32_t M, uint32_t scale_kind, bool grad, int sms, size_t head, GatedPlan* p) {
  p->M = M;
  p->N = L.N;
  p->K = L.K;
  p->f16 = operand_is_f16(L.dtype);
  p->grad = grad;
  p->sms = sms;
  p->prep = p->f16 || scale_kind == 1 || scale_kind == 2;
  p->back = plan_operand_gemm(true, p->f16, M, 2 * L.N, L.K, sms);
  size_t at = head;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += aligned(n);
    return o;
  };
  p->off_images = take(2 * operand_bytes(L.N, L.K));
  p->off_x16 = take(p->f16 ? static_cast<size_t>(M) * L.K * 2 : 0);
  p->off_factor = take(p->f16 ? static_cast<size_t>(M) * 4 : 0);
  p->off_rows = take(grad && p->prep ? static_cast<size_t>(M) * L.N * 4 : 0);
  p->off_rows_factor = take(grad && p->f16 ? (static_cast<size_t>(M) * 3 + kScaleParts) * 4 : 0);
  p->off_gemm = take(grad ? operand_gemm_workspace(p->back) : 0);
  p->bytes = at;
}

template <bool kGrad, uint32_t kBN>
static cudaError_t launch_gated_tiles(GatedDev& P, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(attr_set.load() & (1ull << dev))) {
    e = cudaFuncSetAttribute(gated_gemm_kernel<kGrad, kBN>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGaSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set.fetch_or(1ull << dev);
  }
  P.n_tiles = P.N / kBN * P.m_blocks;
  if (kBN < 128) {
    e = encode_tmap(&P.tmap_w, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, P.images, kSlabBytes / 8,
                    static_cast<uint64_t>(P.N / 128) * P.k_slabs * 2, kSlabBytes, kBN * 4, 8, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(gated_gemm_kernel<kGrad, kBN>, dim3(std::min(P.n_tiles, static_cast<uint32_t>(sms))), dim3(kGaThreads),
                    kGaSmem, stream, P);
}
template <bool kGrad>
static cudaError_t launch_gated_gemm(GatedDev& P, uint32_t K, int sms, cudaStream_t stream) {
  switch (gated_rows_of_tile(P.M, P.N, K, kGrad, static_cast<uint32_t>(sms))) {
    case 128: return launch_gated_tiles<kGrad, 128>(P, sms, stream);
    case 64: return launch_gated_tiles<kGrad, 64>(P, sms, stream);
    default: return launch_gated_tiles<kGrad, 32>(P, sms, stream);
  }
}

cudaError_t launch_gated(const GatedPlan& p, const LayerDev& gate, const LayerDev& up, const GatedArgs& a, void* ws,
                         cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint8_t* images = w + p.off_images;
  uint16_t* x16 = reinterpret_cast<uint16_t*>(w + p.off_x16);
  float* factor = reinterpret_cast<float*>(w + p.off_factor);
  float* rows_factor = reinterpret_cast<float*>(w + p.off_rows_factor);
  float* bound = rows_factor + p.M;
  float* rows_top = bound + p.M;
  float* scale_parts = rows_top + p.M;
  const bool bounds = p.grad && p.f16 && a.dX != nullptr;
  cudaError_t e = cudaSuccess;
  if (bounds && a.scale_kind != 0)
    e = launch_pdl(gated_scales_kernel, dim3(kScaleParts), dim3(256), 0, stream, a.gate_scales, a.up_scales, a.scale_kind,
                   a.scale_kind == 3 ? static_cast<uint64_t>(p.N) * (p.K / a.group_k) : static_cast<uint64_t>(p.N),
                   scale_parts);
  if (e != cudaSuccess) return e;
  e = launch_operand_decode(gate, 0, p.N, a.scale_kind, a.gate_scales, a.group_k, images, a.status, p.sms, stream,
                            2 * kOperandImage);
  if (e == cudaSuccess)
    e = launch_operand_decode(up, 0, p.N, a.scale_kind, a.up_scales, a.group_k, images + kOperandImage, a.status, p.sms,
                              stream, 2 * kOperandImage, true);
  if (e == cudaSuccess && p.f16) e = launch_row_prep(a.X, p.M, p.K, 0, nullptr, true, x16, factor, stream);
  if (e == cudaSuccess && bounds) {
    const uint32_t dt = gate.dtype;
    const float code = dt == kDtInt8 ? 128.0f : dt == kDtFp8 ? 448.0f : dt == kDtInt4 || dt == kDtInt4Pairs ? 8.0f : 6.0f;
    e = launch_pdl(gated_bound_kernel, dim3(p.M), dim3(256), 0, stream, a.X, a.dH, p.N, p.K, 1.14f * code, bound, rows_top);
  }
  if (e != cudaSuccess) return e;
  GatedDev P;
  std::memset(&P, 0, sizeof(P));
  P.images = images;
  P.factor = p.f16 ? factor : nullptr;
  P.gate_scales = a.gate_scales;
  P.up_scales = a.up_scales;
  P.scale_kind = a.scale_kind;
  P.act = a.act;
  P.H = a.H;
  P.dH = a.dH;
  P.dG = a.dG;
  P.dU = a.dU;
  P.status = a.status;
  P.M = p.M;
  P.N = p.N;
  P.m_blocks = (p.M + kGaBM - 1) / kGaBM;
  P.k_slabs = p.K / 16;
  P.n_kb = (p.K + kGaBK - 1) / kGaBK;
  P.box_rows = std::min(p.M, kGaBM);
  P.f16 = p.f16;
  e = encode_tmap(&P.tmap_x, CU_TENSOR_MAP_DATA_TYPE_UINT16, p.f16 ? x16 : a.X, p.K, p.M, static_cast<uint64_t>(p.K) * 2,
                  kGaBK, P.box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  if (!p.grad) return launch_gated_gemm<false>(P, p.K, p.sms, stream);
  const uint16_t *rows = a.dG, *rows2 = a.dU;
  if (p.prep && a.dX != nullptr) {
    P.rows.gate = reinterpret_cast<uint16_t*>(w + p.off_rows);
    P.rows.up = P.rows.gate + static_cast<uint64_t>(p.M) * p.N;
    if (bounds) {
      P.rows.bound = bound;
      P.rows.scale_parts = scale_parts;
      P.rows.factor = rows_factor;
      P.rows.top = rows_top;
    }
    rows = P.rows.gate;
    rows2 = P.rows.up;
  }
  e = launch_gated_gemm<true>(P, p.K, p.sms, stream);
  if (e != cudaSuccess || a.dX == nullptr) return e;
  if (bounds) {
    const GatedLowRows low{a.dG, a.dU, a.gate_scales, a.up_scales, P.rows, a.scale_kind, p.M, p.N};
    e = launch_pdl(gated_rows_kernel, dim3((p.M + kRowsTokens - 1) / kRowsTokens), dim3(512), 0, stream, low);
    if (e != cudaSuccess) return e;
  }
  OperandGemmOut out;
  std::memset(&out, 0, sizeof(out));
  out.out16 = a.dX;
  out.ld = p.K;
  out.beta = bounds ? rows_factor : nullptr;
  const OperandPair pair{images + kOperandImage, rows2, 2 * kOperandImage};
  return launch_operand_gemm(p.back, images, rows, &out, nullptr, w + p.off_gemm, a.status, stream, &pair);
}

cudaError_t set_live_wait_budget_gated(long long cycles) {
  return cudaMemcpyToSymbol(g_live_wait_budget, &cycles, sizeof(cycles));
}

}  // namespace ansdev

// xent.cu -- softmax cross entropy over a compressed vocabulary head, a piece
// of the vocabulary at a time, with the gradient of the hidden states.
//
//   z_n = x . w_n (n < vocab),  lse = log sum_n exp z_n,  loss = lse - z_t,
//   dx = g (sum_n p_n w_n - w_t),  p_n = exp(z_n - lse).
//
// One pass over the vocabulary serves loss and gradient.  Per piece: its
// weights are decoded once into operand images; one GEMM computes the logits
// and folds them, in its epilogue, into blocks of exponentials and their sums
// (operand.h); a row kernel joins the blocks into the running reference and
// sum; and a transposed GEMM on the same images adds the exponentials times W
// to the row's running sum of the gradient, rescaled as it is stored where the
// reference moved.  Two products of 2 M V K operations in all, against three for
// a pass that has the sums first.
//
// The reference is a whole number r in units of log 2 that lies at most
// kXentSlack below the largest logit so far (the target's aside), so that moving
// it rescales by powers of two, exactly, and after the first piece it hardly moves.
//
// The target's own term stays out of the running sums and their reference, so that
// the others' exponentials keep their bits (f16 has 22 powers of two below the
// reference for all 11 of them) however certain the target is.  With l the others'
// sum and e_t the target's, dx = g / (l + e_t) (sum_{n != t} e_n w_n - l w_t):
// the coefficient 1 - p_t is l / (l + e_t) and keeps its relative precision
// where p_t is near 1, and so does the loss, log(1 + l / e_t).  Where e_t passes the
// others' reference, all of it is divided by e_t.
//
// Measured on a 32000 x 4096 bf16 head with 2048 tokens: 1.10 ms a call in runs of
// ten, 1.26 over seconds, under the power cap.  Its kernels one by one, with a cold
// cache, take 1.19: the two products 0.43 and 0.47 (see operand_gemm.cu), decoding
// 0.18, joining the blocks 0.035, rescaling and the targets' rows 0.053, the rest
// 0.02; they read 1.28 GB and write 0.15.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gemm_common.cuh"
#include "launch.h"
#include "operand.h"
#include "rans_core.cuh"
#include "xent.h"

namespace ansdev {

constexpr uint32_t kXentThreads = 256;
constexpr float kLn2 = 0.69314718055994531f, kLog2E = 1.4426950408889634f;

// 2^e for a whole e; 0 below the normal range.
__device__ __forceinline__ float pow2(float e) {
  return e < -126.0f ? 0.0f : __uint_as_float(static_cast<uint32_t>(static_cast<int>(fminf(e, 127.0f)) + 127) << 23);
}

// Beside the first piece's decoding.  Clears the state, checks the targets and sets lift: f16 probabilities carry
// the row scale of W, so they are stored under a power of two that puts the
// largest scale in [2^8, 2^9): a probability of e^4 (kXentSlack) stays below the
// largest f16, and 11 bits are kept where probability times scale is down to 2^-22 of
// the reference's times the largest scale.
__global__ void __launch_bounds__(1024) xent_begin_kernel(XentState st, uint32_t M, const int32_t* __restrict__ targets,
                                                          uint32_t vocab, uint32_t f16, uint32_t kind,
                                                          const void* scales, uint32_t* status) {
  __shared__ float part[32];
  griddep_beside();
  bool bad = false;
  for (uint32_t m = blockIdx.x * 1024 + threadIdx.x; m < M; m += gridDim.x * 1024) {
    st.ref[m] = kXentNone;
    st.sum[m] = 0.0f;
    const int32_t t = __ldg(targets + m);
    bad = bad || (t >= 0 && static_cast<uint32_t>(t) >= vocab);
  }
  if (bad) atomicOr(status, kStatusBadIndex);
  if (blockIdx.x != 0) return;  // (the first CTA is the one that ends last)
  float top = 0.0f;
  if (f16 && (kind == 1 || kind == 2)) {
    // (there are scales up to the next multiple of 128)
    for (uint32_t n = 4 * threadIdx.x; n < vocab; n += 4096) {
      float4 v;
      if (kind == 1) {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(scales) + n));
        v = make_float4(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xFFFF0000u), __uint_as_float(q.y << 16),
                        __uint_as_float(q.y & 0xFFFF0000u));
      } else {
        v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(scales) + n));
      }
      uint32_t at = n;
      for (const float s : {fabsf(v.x), fabsf(v.y), fabsf(v.z), fabsf(v.w)})
        if (at++ < vocab && s <= 3.402823466e38f) top = fmaxf(top, s);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < 32; ++k) top = fmaxf(top, part[k]);
    const int ex = top == 0.0f ? 0 : static_cast<int>(__float_as_uint(top) >> 23) - 127;
    *st.lift = f16 ? pow2(static_cast<float>(min(126, max(-118, 8 - ex)))) : 1.0f;
  }
  griddep_beside_end();
}

// kTok tokens a CTA (32, or 8 where there are few), one a lane of each of a warp's
// 32 / kTok shares; the shares of all warps take the blocks in turn, 8 loads in
// flight each, and are joined in order.  The largest of a token's block
// references is the piece's.
constexpr uint32_t kJoinWarps = 16, kJoinBatch = 8;
template <uint32_t kTok>
__global__ void __launch_bounds__(32 * kJoinWarps) xent_join_kernel(const __grid_constant__ XentJoin P) {
  constexpr uint32_t kShares = kJoinWarps * 32 / kTok;
  __shared__ float part_ref[kShares][kTok + 1], part_low[kShares][kTok + 1], part_sum[kShares][kTok + 1];
  if (P.beside == 0) griddep_wait();
  griddep_launch_dependents();
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t tok = threadIdx.x % kTok, share = threadIdx.x / kTok, col = blockIdx.x * kTok + tok;
  const bool in = col < P.m;
  const uint32_t m = P.m0 + col;
  // (ref, s): sums under the largest reference so far; low: the smallest that a
  // sum other than 0 came under
  float ref = kXentNone, low = INFINITY, s = 0.0f;
  for (uint32_t b0 = share; b0 < P.n_blocks; b0 += kJoinBatch * kShares) {
    float2 u[kJoinBatch];
#pragma unroll
    for (uint32_t k = 0; k < kJoinBatch; ++k) {
      const uint32_t b = b0 + k * kShares;
      u[k] = in && b < P.n_blocks ? __ldcg(P.blocks + static_cast<uint64_t>(b) * P.stride + col)
                                  : make_float2(kXentNone, 0.0f);
    }
    float top = ref;
#pragma unroll
    for (uint32_t k = 0; k < kJoinBatch; ++k) top = fmaxf(top, u[k].x);
    s = s == 0.0f ? 0.0f : s * pow2(ref - top);
    ref = top;
#pragma unroll
    for (uint32_t k = 0; k < kJoinBatch; ++k) {
      if (u[k].y == 0.0f) continue;
      s += u[k].y * pow2(u[k].x - ref);
      low = fminf(low, u[k].x);
    }
  }
  part_ref[share][tok] = ref;
  part_low[share][tok] = low;
  part_sum[share][tok] = s;
  __syncthreads();
  if (warp == 0) {
    // (with 8 tokens, all four shares of the warp do the same)
    const float ref_old = in ? __ldcg(P.st.ref + m) : kXentNone;
    const float l = in ? __ldcg(P.st.sum + m) : 0.0f;
    ref = ref_old;
#pragma unroll 16
    for (uint32_t k = 0; k < kShares; ++k) {
      ref = fmaxf(ref, part_ref[k][tok]);
      low = fminf(low, part_low[k][tok]);
    }
    s = 0.0f;
#pragma unroll 16
    for (uint32_t k = 0; k < kShares; ++k) {
      const float v = part_sum[k][tok];
      s += v == 0.0f ? 0.0f : v * pow2(part_ref[k][tok] - ref);
    }
    const uint32_t moved = __ballot_sync(0xFFFFFFFFu, in && low < ref);
    if (in && lane < kTok) {
      const float keep = ref_old == kXentNone ? 0.0f : pow2(ref_old - ref);
      P.st.ref[m] = ref;
      P.st.sum[m] = fmaf(l, keep, s);  // (NaN stays NaN)
      if (P.probs != nullptr) {
        P.st.alpha[m] = keep;
        P.st.beta[m] = 1.0f / __ldcg(P.st.lift);  // a power of two
      }
    }
    if (P.probs != nullptr && lane == 0) {
      if constexpr (kTok == 32) P.moved[blockIdx.x] = moved;
      else reinterpret_cast<uint8_t*>(P.moved)[blockIdx.x] = static_cast<uint8_t>(moved);
    }
  }
  if (P.beside != 0) griddep_beside_end();
}

// What the transposed product and the end need of a piece.  Probabilities of
// blocks under another reference than their token's are rescaled: in the first
// piece nearly all of them, later hardly any.  And targets in the piece have
// their rows of W copied while it is here.  A CTA takes 32 tokens, 32 blocks and a
// share of the columns, a warp 4 of the tokens; 4 lanes a block, 16 bytes a lane.
__global__ void __launch_bounds__(256) xent_piece_kernel(const __grid_constant__ XentJoin P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t moved = __ldcg(P.moved + blockIdx.x);
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, b = 32 * blockIdx.y + lane;
  const uint32_t row0 = blockIdx.x * 32 + 4 * warp;
  const int32_t mine = lane < 4 && row0 + lane < P.m ? __ldg(P.targets + P.m0 + row0 + lane) : -1;
  const bool here = mine >= 0 && static_cast<uint32_t>(mine) < P.vocab && static_cast<uint32_t>(mine) - P.n0 < P.rows;
  for (uint32_t todo = __ballot_sync(0xFFFFFFFFu, here); todo != 0; todo &= todo - 1) {
    const uint32_t k = __ffs(todo) - 1;
    const uint32_t tc = static_cast<uint32_t>(__shfl_sync(0xFFFFFFFFu, mine, k)) - P.n0;
    const uint32_t k_slabs = P.K / 16, rr = tc & 127u;
    const uint8_t* src = P.images + static_cast<uint64_t>(tc >> 7) * k_slabs * kSlabBytes + rr * 32u;
    uint16_t* dst = P.target_rows + static_cast<uint64_t>(P.m0 + row0 + k) * P.K;
    for (uint32_t q = 32 * blockIdx.y + lane; q < P.K / 8; q += 32 * gridDim.y)
      *reinterpret_cast<uint4*>(dst + 8 * q) = __ldcg(reinterpret_cast<const uint4*>(
          src + static_cast<uint64_t>(q >> 1) * kSlabBytes + (((q & 1u) ^ ((rr >> 2) & 1u)) << 4)));
  }
  if (moved == 0 || 32 * blockIdx.y >= P.n_blocks) return;
#pragma unroll
  for (uint32_t k = 0; k < 4; ++k) {
    const uint32_t col = row0 + k;
    if (col >= P.m || ((moved >> (4 * warp + k)) & 1u) == 0) continue;
    const float ref = __ldcg(P.st.ref + P.m0 + col);
    const float r = b < P.n_blocks ? __ldcg(P.blocks + static_cast<uint64_t>(b) * P.stride + col).x : ref;
    const float f = pow2(r - ref);
    uint4* row = reinterpret_cast<uint4*>(P.probs + static_cast<uint64_t>(col) * P.rows + 1024 * blockIdx.y);
    uint4 w[4];
    float g[4];
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) {
      g[q] = __shfl_sync(0xFFFFFFFFu, f, 8 * q + lane / 4);
      if (g[q] != 1.0f) w[q] = __ldcg(row + 32 * q + lane);
    }
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) {
      if (g[q] == 1.0f) continue;
      uint32_t* u = reinterpret_cast<uint32_t*>(&w[q]);
      if (P.f16) {
        // (in fp32: a factor of 2^-25 is none of f16's values, but a stored value is up to
        // 2^14, and its product with the factor may be one)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(u + i));
          const __half2 h = __floats2half2_rn(x.x * g[q], x.y * g[q]);
          u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
      } else {
        const __nv_bfloat162 h = __float2bfloat162_rn(g[q]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(u + i), h);
          u[i] = *reinterpret_cast<const uint32_t*>(&x);
        }
      }
      row[32 * q + lane] = w[q];
    }
  }
}

cudaError_t launch_xent_join(const XentJoin& j, cudaStream_t stream) {
  return j.m <= 128 ? launch_pdl(xent_join_kernel<8>, dim3((j.m + 7) / 8), dim3(32 * kJoinWarps), 0, stream, j)
                    : launch_pdl(xent_join_kernel<32>, dim3((j.m + 31) / 32), dim3(32 * kJoinWarps), 0, stream, j);
}

__global__ void __launch_bounds__(256) xent_blank_kernel(uint8_t* images, uint32_t first, uint32_t rows, uint32_t k_slabs) {
  griddep_wait();
  griddep_launch_dependents();
  const uint64_t n = static_cast<uint64_t>(rows - first) * k_slabs * 2;
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<uint64_t>(gridDim.x) * 256) {
    const uint64_t slab = (i / 2) % k_slabs;
    const uint32_t row = first + static_cast<uint32_t>(i / 2 / k_slabs);
    *reinterpret_cast<uint4*>(images + ((row >> 7) * static_cast<uint64_t>(k_slabs) + slab) * kSlabBytes + (row & 127u) * 32u +
                              16 * (i & 1)) = make_uint4(0, 0, 0, 0);
  }
}

cudaError_t launch_xent_blank(uint8_t* images, uint32_t first, uint32_t rows, uint32_t K, cudaStream_t stream) {
  const uint64_t items = static_cast<uint64_t>(rows - first) * (K / 8);
  return launch_pdl(xent_blank_kernel, dim3(static_cast<uint32_t>(std::min<uint64_t>((items + 255) / 256, 1024))), dim3(256), 0,
                    stream, images, first, rows, K / 16);
}

struct XentFinish {
  const int32_t* targets;
  const void* scales;
  XentState st;
  const float* acc;        // M x K
  const uint16_t* target_rows;
  const float* weight;
  float *loss, *lse;
  uint16_t* dX;
  uint32_t vocab, K, scale_kind, f16;
};

__global__ void __launch_bounds__(kXentThreads) xent_finish_kernel(const __grid_constant__ XentFinish P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t m = blockIdx.x;
  const int32_t target = __ldg(P.targets + m);
  const bool valid = target >= 0 && static_cast<uint32_t>(target) < P.vocab;
  // (others without a finite logit have no reference: their sum, 0 or not finite, stands for itself)
  const float ref_raw = __ldcg(P.st.ref + m), ref = ref_raw == kXentNone ? 0.0f : ref_raw;
  const float l = __ldcg(P.st.sum + m);
  const float zt = valid ? __ldcg(P.st.zt + m) : -INFINITY;
  // the target's distance from the others' reference, units of log 2 (a target alone is its own reference)
  const float dt = valid && l == 0.0f ? 0.0f : fmaf(zt, kLog2E, -ref);
  const float g = !valid ? 0.0f : (P.weight != nullptr ? __ldg(P.weight + m) : 1.0f);
  float lse, loss, ca;  // ca: g / (l + e_t)
  if (valid && dt >= 0.0f && dt <= 3.0e38f) {
    // a target above the others: all of it under the target's own exponential
    const float down = exp2f(-dt), q = l * down;
    loss = log1pf(q);
    lse = zt + loss;
    ca = g * down / (1.0f + q);
  } else {
    const float total = l + (valid ? exp2f(dt) : 0.0f);
    lse = fmaf(ref, kLn2, logf(total));
    // near the reference: log(1 + l / e_t), exact where the loss is small
    loss = !valid ? 0.0f : dt > -30.0f ? log1pf(l * exp2f(-dt)) : fmaf(-dt, kLn2, logf(total));
    ca = g / total;
  }
  if (valid && !isfinite(lse)) {
    loss = lse - zt;
    ca = NAN;
  }
  if (threadIdx.x == 0) {
    P.lse[m] = lse;
    P.loss[m] = loss;
  }
  if (P.dX == nullptr) return;
  float s = 1.0f;
  if (valid && P.scale_kind == 1) s = bf16_to_f32(__ldg(static_cast<const uint16_t*>(P.scales) + target));
  else if (valid && P.scale_kind == 2) s = __ldg(static_cast<const float*>(P.scales) + target);
  const float ct = ca * l * s;
  for (uint32_t k = 4 * threadIdx.x; k < P.K; k += 4 * kXentThreads) {
    const uint64_t at = static_cast<uint64_t>(m) * P.K + k;
    uint32_t lo = 0, hi = 0;
    if (valid) {
      const float4 a = __ldcg(reinterpret_cast<const float4*>(P.acc + at));
      const uint2 w = __ldcg(reinterpret_cast<const uint2*>(P.target_rows + at));
      float t[4];
      if (P.f16) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
        const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
        t[0] = p.x; t[1] = p.y; t[2] = q.x; t[3] = q.y;
      } else {
        t[0] = __uint_as_float(w.x << 16);
        t[1] = __uint_as_float(w.x & 0xFFFF0000u);
        t[2] = __uint_as_float(w.y << 16);
        t[3] = __uint_as_float(w.y & 0xFFFF0000u);
      }
      const __nv_bfloat162 p = __floats2bfloat162_rn(ca * a.x - ct * t[0], ca * a.y - ct * t[1]);
      const __nv_bfloat162 q = __floats2bfloat162_rn(ca * a.z - ct * t[2], ca * a.w - ct * t[3]);
      lo = *reinterpret_cast<const uint32_t*>(&p);
      hi = *reinterpret_cast<const uint32_t*>(&q);
    }
    *reinterpret_cast<uint2*>(P.dX + at) = make_uint2(lo, hi);
  }
}

static size_t aligned(size_t n) { return (n + 1023) / 1024 * 1024; }

// W rows of a piece, most, in blocks of 128: its images (2 K bytes a row) and a
// chunk's probabilities are what has to stay in L2.  Without probabilities the
// images may fill 80 MB.  With few tokens a piece is a row of tiles, and may be
// as long as there are SMs.
constexpr uint32_t kXentMostBlocks = 80, kXentLeastBlocks = 24;
constexpr uint32_t kXentImageBytes = 80u << 20;

static uint32_t waves(uint64_t tiles, uint32_t sms) { return static_cast<uint32_t>((tiles + sms - 1) / sms); }

void make_xent_plan(const LayerDev& L, uint32_t M, bool grad, int sms_in, XentPlan* p) {
  const uint32_t sms = static_cast<uint32_t>(sms_in);
  p->M = M;
  p->N = L.N;
  p->K = L.K;
  p->grad = grad;
  p->f16 = operand_is_f16(L.dtype);
  p->sms = sms_in;
  // chunks of equal size, at most 4096 tokens with probabilities to store
  const uint32_t fit = grad ? 4096u : 16384u;
  const uint32_t chunks = (M + fit - 1) / fit;
  p->chunk = chunks <= 1 ? M : std::min(M, ((M + chunks - 1) / chunks + 255) / 256 * 256);
  // The piece that costs least over the vocabulary: its logits' tiles come in
  // rounds of the SMs (about 460 ns a stage of 64 columns), its decoding in rounds
  // of tiles (11.8 us beyond what the work itself takes, for 8,192 symbols), and
  // its launches and the kernels' ends take some 8 us, with a gradient 35.
  const uint32_t m_blocks = (p->chunk + 255) / 256, blocks = L.N / 128, unit = L.tile_n / 128;
  const uint32_t fill = grad ? 0u : kXentImageBytes / (256u * L.K);
  const uint32_t most = std::min(blocks, std::max({kXentMostBlocks, sms / m_blocks, fill})) / unit * unit;
  const uint32_t symbols = L.tile_n * L.tile_k / (L.dtype == kDtInt4Pairs || L.dtype == kDtFp4Pairs ? 2u : 1u);
  const uint64_t round_ns = 11800ull * symbols / 8192, wave_ns = 460ull * ((L.K + 63) / 64);
  auto cost_of = [&](uint32_t b) {
    if (b == 0) return uint64_t(0);
    return wave_ns * waves(static_cast<uint64_t>(b) * m_blocks, sms) +
           round_ns * operand_decode_rounds(b / unit * L.n_kt, sms) + (grad ? 35000 : 8000);
  };
  uint32_t best = most;
  uint64_t best_cost = ~0ull;
  for (uint32_t b = most; b >= std::min(most, kXentLeastBlocks); b -= unit) {
    const uint64_t cost = (blocks / b) * cost_of(b) + cost_of(blocks % b);
    if (cost < best_cost) {
      best_cost = cost;
      best = b;
    }
    if (b <= unit) break;
  }
  p->piece = best * 128;
  // the gradient's product, for the usual and the last of pieces and chunks
  size_t gemm = 0;
  if (grad)
    for (const uint32_t rows : {p->piece, L.N - (L.N - 1) / p->piece * p->piece})
      for (const uint32_t m : {p->chunk, M - (M - 1) / p->chunk * p->chunk})
        gemm = std::max(gemm, operand_gemm_workspace(plan_operand_gemm(true, p->f16, m, rows, L.K, sms_in)));
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += aligned(n);
    return o;
  };
  const size_t MK = static_cast<size_t>(M) * L.K;
  p->off_images = take(operand_bytes(p->piece, L.K));
  p->off_probs = take(grad ? static_cast<size_t>(p->chunk) * p->piece * 2 : 0);
  p->off_blocks = take(static_cast<size_t>(p->chunk) * (p->piece / 32) * 8);
  p->off_moved = take((static_cast<size_t>(p->chunk) + 31) / 32 * 4);
  p->off_x16 = take(p->f16 ? MK * 2 : 0);
  p->off_factor = take(p->f16 ? static_cast<size_t>(M) * 4 : 0);
  p->off_state = take((static_cast<size_t>(M) * 5 + 1) * 4);
  p->off_acc = take(grad ? MK * 4 : 0);
  p->off_target = take(grad ? MK * 2 : 0);
  p->off_gemm = take(gemm);
  p->bytes = at;
}

cudaError_t launch_xent(const XentPlan& p, const LayerDev& L, const XentArgs& a, void* ws, cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint8_t* images = w + p.off_images;
  uint16_t* probs = p.grad ? reinterpret_cast<uint16_t*>(w + p.off_probs) : nullptr;
  float2* blocks = reinterpret_cast<float2*>(w + p.off_blocks);
  float* acc = reinterpret_cast<float*>(w + p.off_acc);
  uint16_t* target_rows = reinterpret_cast<uint16_t*>(w + p.off_target);
  float* state = reinterpret_cast<float*>(w + p.off_state);
  const XentState st{state, state + p.M, state + 2ull * p.M, state + 3ull * p.M, state + 4ull * p.M,
                     state + 5ull * p.M};
  uint16_t* x16 = reinterpret_cast<uint16_t*>(w + p.off_x16);
  float* x_factor = reinterpret_cast<float*>(w + p.off_factor);
  const uint16_t* x = p.f16 ? x16 : a.X;
  const float* factor = p.f16 ? x_factor : nullptr;
  XentJoin j;
  bool pending = false;  // j is still to be joined
  cudaError_t e;
  for (uint32_t n0 = 0; n0 < a.vocab; n0 += p.piece) {
    const uint32_t rows = std::min(p.piece, p.N - n0);
    e = launch_operand_decode(L, n0, rows, a.scale_kind, a.scales, a.group_k, images, a.status, p.sms, stream);
    if (e != cudaSuccess) return e;
    if (p.grad && n0 + rows > a.vocab) {
      e = launch_xent_blank(images, a.vocab - n0, rows, p.K, stream);
      if (e != cudaSuccess) return e;
    }
    if (n0 == 0) {
      e = launch_pdl(xent_begin_kernel, dim3(std::min(64u, (p.M + 1023) / 1024)), dim3(1024), 0, stream, st, p.M, a.targets,
                     a.vocab, p.f16, a.scale_kind, a.scales, a.status);
      if (e == cudaSuccess && p.f16) e = launch_row_prep(a.X, p.M, p.K, 0, nullptr, true, x16, x_factor, stream);
      if (e != cudaSuccess) return e;
    }
    if (pending) {
      j.beside = 1;
      e = launch_xent_join(j, stream);
      if (e != cudaSuccess) return e;
      pending = false;
    }
    for (uint32_t m0 = 0; m0 < p.M; m0 += p.chunk) {
      const uint32_t m = std::min(p.chunk, p.M - m0);
      XentEpilogue f = {};
      f.factor = factor ? factor + m0 : nullptr;
      f.scale_kind = a.scale_kind;
      f.scales = a.scale_kind == 1 ? static_cast<const void*>(static_cast<const uint16_t*>(a.scales) + n0)
                 : a.scale_kind == 2 ? static_cast<const void*>(static_cast<const float*>(a.scales) + n0) : nullptr;
      f.lift = st.lift;
      f.ref_in = st.ref + m0;
      f.targets = a.targets + m0;
      f.zt = st.zt + m0;
      f.blocks = blocks;
      f.stride = p.chunk;
      f.probs = probs;
      f.n0 = n0;
      f.vocab = a.vocab;
      e = launch_operand_gemm(plan_operand_gemm(false, p.f16, m, rows, p.K, p.sms), images,
                              x + static_cast<uint64_t>(m0) * p.K, nullptr, &f, w + p.off_gemm, a.status, stream);
      if (e != cudaSuccess) return e;
      j.st = st;
      j.blocks = blocks;
      j.stride = p.chunk;
      j.n_blocks = rows / 32;
      j.m0 = m0;
      j.m = m;
      j.rows = rows;
      j.f16 = p.f16;
      j.moved = reinterpret_cast<uint32_t*>(w + p.off_moved);
      j.probs = probs;
      j.targets = a.targets;
      j.images = images;
      j.target_rows = target_rows;
      j.n0 = n0;
      j.vocab = a.vocab;
      j.K = p.K;
      j.beside = 0;
      const uint32_t groups = (m + 31) / 32;
      // without a gradient, the last tokens' blocks are joined beside the next
      // piece's decoding
      pending = !p.grad && m0 + m == p.M && n0 + p.piece < a.vocab;
      if (pending) break;
      e = launch_xent_join(j, stream);
      if (e != cudaSuccess) return e;
      if (!p.grad) continue;
      // as many CTAs a group as its blocks take, or as the copies of rows can use
      const uint32_t copies = std::min((p.K / 8 + 31) / 32, std::max(1u, 4u * static_cast<uint32_t>(p.sms) / groups));
      e = launch_pdl(xent_piece_kernel, dim3(groups, std::max((j.n_blocks + 31) / 32, copies)), dim3(256), 0, stream, j);
      if (e != cudaSuccess) return e;
      OperandGemmOut back = {};
      back.out32 = acc + static_cast<uint64_t>(m0) * p.K;
      back.ld = p.K;
      back.alpha = n0 == 0 ? nullptr : st.alpha + m0;
      back.beta = st.beta + m0;
      e = launch_operand_gemm(plan_operand_gemm(true, p.f16, m, rows, p.K, p.sms), images, probs, &back, nullptr,
                              w + p.off_gemm, a.status, stream);
      if (e != cudaSuccess) return e;
    }
  }
  XentFinish f;
  f.targets = a.targets;
  f.scales = a.scales;
  f.st = st;
  f.acc = acc;
  f.target_rows = target_rows;
  f.weight = a.weight;
  f.loss = a.loss;
  f.lse = a.lse;
  f.dX = a.dX;
  f.vocab = a.vocab;
  f.K = p.K;
  f.scale_kind = a.scale_kind;
  f.f16 = p.f16;
  return launch_pdl(xent_finish_kernel, dim3(p.M), dim3(kXentThreads), 0, stream, f);
}

}  // namespace ansdev

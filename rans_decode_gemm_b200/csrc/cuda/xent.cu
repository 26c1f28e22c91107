// xent.cu -- softmax cross entropy over a compressed vocabulary head, a piece
// of the vocabulary at a time, with the gradient of the hidden states.
//
//   z_n = x . w_n (n < vocab),  lse = log sum_n exp z_n,  loss = lse - z_t,
//   dx = g (sum_n p_n w_n - w_t),  p_n = exp(z_n - lse).
//
// One pass over the vocabulary serves loss and gradient.  Per piece: its
// weights are decoded once into operand images, one GEMM gives the piece's
// logits, a row kernel folds them into the running reference r (the largest
// logit so far) and sum l and turns them into exp(z - r), and a transposed GEMM
// on the same images adds exp(z - r) W to the row's running sum of the
// gradient, rescaled by exp(r_old - r_new) as it is stored.  Two products of
// 2 M V K operations in all, against three for a pass that has the sums first.
// Logits exist for one piece and one chunk of tokens.
//
// The target's own term stays out of the running sums.  With l the others'
// sum and e_t the target's, dx = g / (l + e_t) (sum_{n != t} e_n w_n - l w_t):
// the coefficient 1 - p_t is l / (l + e_t) and keeps its relative precision
// where p_t is near 1, and so does the loss, log(1 + l / e_t).
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
constexpr uint32_t kXentPieceMax = 8192;  // logits of a row in registers: 32 a thread
constexpr uint32_t kXentPer = kXentPieceMax / kXentThreads / 4;  // float4s a thread

// Running state of M rows: reference r, sum l of the others, target logit,
// and this piece's factors of the gradient's sum.
struct XentState {
  float *ref, *sum, *zt, *alpha, *beta;
};

struct XentStep {
  const float* logits;    // chunk x rows
  const float* factor;    // power of two of each row's f16 form, or null
  const int32_t* targets;
  const void* scales;     // row scales of the layer (scale_kind 1, 2), for P
  const uint8_t* images;
  uint16_t* probs;        // chunk x rows, or null (no gradient)
  uint16_t* target_rows;  // M x K: the target's weights in operand form
  uint32_t* status;
  XentState st;
  uint32_t m0;            // first token of the chunk
  uint32_t n0, rows;      // the piece
  uint32_t vocab, K, scale_kind, f16, first;
};

// Sum and maximum over the CTA, in a fixed order.
__device__ __forceinline__ float2 block_sum_max(float s, float t, float2* part) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, d));
  }
  __syncthreads();
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = make_float2(s, t);
  __syncthreads();
  float2 r = part[0];
#pragma unroll
  for (uint32_t k = 1; k < kXentThreads / 32; ++k) {
    r.x += part[k].x;
    r.y = fmaxf(r.y, part[k].y);
  }
  return r;
}

// One CTA a row of the chunk: the row's logits of this piece stay in
// registers between the maximum, the sum and the probabilities.
__global__ void __launch_bounds__(kXentThreads) xent_step_kernel(const __grid_constant__ XentStep P) {
  __shared__ float2 part[kXentThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t m = P.m0 + blockIdx.x;
  const int32_t target = __ldg(P.targets + m);
  const bool valid = target >= 0 && static_cast<uint32_t>(target) < P.vocab;
  if (P.first && threadIdx.x == 0 && target >= 0 && !valid) atomicOr(P.status, kStatusBadIndex);
  const float up = P.factor != nullptr ? __ldcg(P.factor + m) : 1.0f;
  const float* row = P.logits + static_cast<uint64_t>(blockIdx.x) * P.rows;
  const uint32_t lim = P.vocab > P.n0 ? min(P.rows, P.vocab - P.n0) : 0u;  // columns that count
  // -inf past the vocabulary
  float z[kXentPer][4];
  float top = -INFINITY;
#pragma unroll
  for (uint32_t i = 0; i < kXentPer; ++i) {
    const uint32_t c = 4 * (threadIdx.x + i * kXentThreads);
    float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (c < P.rows) q = __ldcg(reinterpret_cast<const float4*>(row + c));
    const float w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
      z[i][k] = c + k < lim ? w[k] * up : -INFINITY;
      top = fmaxf(top, z[i][k]);
    }
  }
  top = block_sum_max(0.0f, top, part).y;
  // An infinite reference is replaced by 0, so that +inf gives an infinite sum
  // and a row of -inf a sum of 0.  NaN stays NaN through the sum.
  const float ref_old = P.first ? -INFINITY : __ldcg(P.st.ref + m);
  const float ref = fmaxf(ref_old, top);
  const float base = isinf(ref) ? 0.0f : ref;
  // nothing but -inf so far: sums of 0 (or NaN, which 0 keeps)
  const float keep = ref_old == -INFINITY ? 0.0f : __expf((isinf(ref_old) ? 0.0f : ref_old) - base);
  const bool here = valid && static_cast<uint32_t>(target) >= P.n0 && static_cast<uint32_t>(target) < P.n0 + P.rows;
  const uint32_t tc = here ? static_cast<uint32_t>(target) - P.n0 : 0xFFFFFFFFu;
  float s = 0.0f, big = 0.0f;
#pragma unroll
  for (uint32_t i = 0; i < kXentPer; ++i) {
    const uint32_t c = 4 * (threadIdx.x + i * kXentThreads);
    float sc[4] = {1.0f, 1.0f, 1.0f, 1.0f};
    if (P.probs != nullptr && c < P.rows) {
      if (P.scale_kind == 1) {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(P.scales) + P.n0 + c));
        sc[0] = __uint_as_float(q.x << 16);
        sc[1] = __uint_as_float(q.x & 0xFFFF0000u);
        sc[2] = __uint_as_float(q.y << 16);
        sc[3] = __uint_as_float(q.y & 0xFFFF0000u);
      } else if (P.scale_kind == 2) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(P.scales) + P.n0 + c));
        sc[0] = q.x; sc[1] = q.y; sc[2] = q.z; sc[3] = q.w;
      }
    }
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
      float e = c + k < lim ? __expf(z[i][k] - base) : 0.0f;
      if (c + k == tc) {
        P.st.zt[m] = z[i][k];
        e = 0.0f;
      }
      s += e;
      z[i][k] = e * sc[k];
      big = fmaxf(big, fabsf(z[i][k]));
    }
  }
  const float2 r = block_sum_max(s, big, part);
  if (threadIdx.x == 0) {
    P.st.ref[m] = ref;
    P.st.sum[m] = P.first ? r.x : fmaf(__ldcg(P.st.sum + m), keep, r.x);
  }
  if (P.probs == nullptr) return;
  // f16: under a power of two that puts the row's largest value in
  // [2^14, 2^15), undone by beta.  11 bits of every value down to 2^-29 of it.
  int e2 = 0;
  if (P.f16 && r.y > 0.0f && r.y <= 3.402823466e38f)
    e2 = min(126, max(-113, 14 - (static_cast<int>(__float_as_uint(r.y) >> 23) - 127)));
  const float lift = __uint_as_float(static_cast<uint32_t>(e2 + 127) << 23);
  if (threadIdx.x == 0) {
    P.st.alpha[m] = keep;
    P.st.beta[m] = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
  }
  uint16_t* out = P.probs + static_cast<uint64_t>(blockIdx.x) * P.rows;
#pragma unroll
  for (uint32_t i = 0; i < kXentPer; ++i) {
    const uint32_t c = 4 * (threadIdx.x + i * kXentThreads);
    if (c >= P.rows) continue;
    uint32_t lo, hi;
    if (!valid) {
      lo = hi = 0;
    } else if (P.f16) {
      const __half2 a = __floats2half2_rn(z[i][0] * lift, z[i][1] * lift);
      const __half2 b = __floats2half2_rn(z[i][2] * lift, z[i][3] * lift);
      lo = *reinterpret_cast<const uint32_t*>(&a);
      hi = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(z[i][0], z[i][1]);
      const __nv_bfloat162 b = __floats2bfloat162_rn(z[i][2], z[i][3]);
      lo = *reinterpret_cast<const uint32_t*>(&a);
      hi = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint2*>(out + c) = make_uint2(lo, hi);
  }
  if (here) {
    // the target's row of W, while its piece is here
    const uint32_t k_slabs = P.K / 16, rr = tc & 127u;
    const uint8_t* src = P.images + static_cast<uint64_t>(tc >> 7) * k_slabs * kSlabBytes + rr * 32u;
    for (uint32_t q = threadIdx.x; q < P.K / 8; q += kXentThreads) {
      const uint4 v = __ldcg(reinterpret_cast<const uint4*>(src + static_cast<uint64_t>(q >> 1) * kSlabBytes +
                                                           (((q & 1u) ^ ((rr >> 2) & 1u)) << 4)));
      *reinterpret_cast<uint4*>(P.target_rows + static_cast<uint64_t>(m) * P.K + 8 * q) = v;
    }
  }
}

struct XentFinish {
  const int32_t* targets;
  const void* scales;
  XentState st;
  const float* acc;        // splits x M x K
  uint64_t split_stride;
  const uint16_t* target_rows;
  const float* weight;
  float *loss, *lse;
  uint16_t* dX;
  uint32_t vocab, K, scale_kind, f16, splits;
};

__global__ void __launch_bounds__(kXentThreads) xent_finish_kernel(const __grid_constant__ XentFinish P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t m = blockIdx.x;
  const int32_t target = __ldg(P.targets + m);
  const bool valid = target >= 0 && static_cast<uint32_t>(target) < P.vocab;
  const float ref = __ldcg(P.st.ref + m), l = __ldcg(P.st.sum + m);
  const float base = isinf(ref) ? 0.0f : ref;
  const float zt = valid ? __ldcg(P.st.zt + m) : -INFINITY;
  const float et = valid ? expf(zt - base) : 0.0f;
  const float total = l + et;
  if (threadIdx.x == 0) {
    P.lse[m] = base + logf(total);
    float loss = 0.0f;
    // near the reference: log(1 + l / e_t), exact where the loss is small
    if (valid)
      loss = isinf(ref) ? P.lse[m] - zt
                        : zt > base - 20.0f ? log1pf(l * expf(base - zt)) : (base - zt) + logf(total);
    P.loss[m] = loss;
  }
  if (P.dX == nullptr) return;
  const float g = !valid ? 0.0f : (P.weight != nullptr ? __ldg(P.weight + m) : 1.0f);
  float s = 1.0f;
  if (valid && P.scale_kind == 1) s = bf16_to_f32(__ldg(static_cast<const uint16_t*>(P.scales) + target));
  else if (valid && P.scale_kind == 2) s = __ldg(static_cast<const float*>(P.scales) + target);
  const float ca = g / total, ct = ca * l * s;
  for (uint32_t k = 4 * threadIdx.x; k < P.K; k += 4 * kXentThreads) {
    const uint64_t at = static_cast<uint64_t>(m) * P.K + k;
    uint32_t lo = 0, hi = 0;
    if (valid) {
      float4 a = __ldcg(reinterpret_cast<const float4*>(P.acc + at));
      for (uint32_t q = 1; q < P.splits; ++q) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(P.acc + q * P.split_stride + at));
        a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
      }
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

void make_xent_plan(const LayerDev& L, uint32_t M, bool grad, int sms, XentPlan* p) {
  p->M = M;
  p->N = L.N;
  p->K = L.K;
  p->grad = grad;
  p->f16 = operand_is_f16(L.dtype);
  p->sms = sms;
  // pieces of equal size, at most what a row kernel holds in registers
  const uint32_t blocks = L.N / L.tile_n, most = kXentPieceMax / L.tile_n;
  const uint32_t pieces = (blocks + most - 1) / most;
  p->piece = (blocks + pieces - 1) / pieces * L.tile_n;
  // a chunk's logits and probabilities within 96 MB, so that they stay in L2
  const uint32_t fit = std::max(256u, static_cast<uint32_t>((96ull << 20) / (6ull * p->piece)) / 256 * 256);
  const uint32_t chunks = (M + fit - 1) / fit;
  p->chunk = chunks <= 1 ? M : std::min(M, ((M + chunks - 1) / chunks + 255) / 256 * 256);
  // one plan for every chunk and piece: partial sums only where one chunk
  // holds all tokens
  // (the last piece's sum has to have that many ranges too)
  const uint32_t last = L.N - (L.N - 1) / p->piece * p->piece;
  p->splits = grad && chunks <= 1 ? plan_operand_gemm(true, p->f16, M, last, L.K, 8, sms).splits : 1;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += aligned(n);
    return o;
  };
  const size_t MK = static_cast<size_t>(M) * L.K;
  p->off_images = take(operand_bytes(p->piece, L.K));
  p->off_logits = take(static_cast<size_t>(p->chunk) * p->piece * 4);
  p->off_probs = take(grad ? static_cast<size_t>(p->chunk) * p->piece * 2 : 0);
  p->off_x16 = take(p->f16 ? MK * 2 : 0);
  p->off_factor = take(p->f16 ? static_cast<size_t>(M) * 4 : 0);
  p->off_state = take(static_cast<size_t>(M) * 4 * 5);
  p->off_acc = take(grad ? MK * 4 * p->splits : 0);
  p->off_target = take(grad ? MK * 2 : 0);
  p->bytes = at;
}

cudaError_t launch_xent(const XentPlan& p, const LayerDev& L, const XentArgs& a, void* ws, cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint8_t* images = w + p.off_images;
  float* logits = reinterpret_cast<float*>(w + p.off_logits);
  uint16_t* probs = p.grad ? reinterpret_cast<uint16_t*>(w + p.off_probs) : nullptr;
  float* acc = reinterpret_cast<float*>(w + p.off_acc);
  uint16_t* target_rows = reinterpret_cast<uint16_t*>(w + p.off_target);
  float* state = reinterpret_cast<float*>(w + p.off_state);
  XentState st{state, state + p.M, state + 2ull * p.M, state + 3ull * p.M, state + 4ull * p.M};
  const uint16_t* x = a.X;
  const float* factor = nullptr;
  cudaError_t e;
  if (p.f16) {
    uint16_t* x16 = reinterpret_cast<uint16_t*>(w + p.off_x16);
    float* f = reinterpret_cast<float*>(w + p.off_factor);
    e = launch_row_prep(a.X, p.M, p.K, 0, nullptr, true, x16, f, stream);
    if (e != cudaSuccess) return e;
    x = x16;
    factor = f;
  }
  const uint64_t MK = static_cast<uint64_t>(p.M) * p.K;
  for (uint32_t n0 = 0; n0 < p.N; n0 += p.piece) {
    const uint32_t rows = std::min(p.piece, p.N - n0);
    e = launch_operand_decode(L, n0, rows, a.scale_kind, a.scales, a.group_k, images, a.status, p.sms, stream);
    if (e != cudaSuccess) return e;
    for (uint32_t m0 = 0; m0 < p.M; m0 += p.chunk) {
      const uint32_t m = std::min(p.chunk, p.M - m0);
      OperandGemmOut fwd;
      fwd.out32 = logits;
      fwd.ld = rows;
      fwd.scale_kind = a.scale_kind;
      fwd.scales = a.scale_kind == 1 ? static_cast<const void*>(static_cast<const uint16_t*>(a.scales) + n0)
                   : a.scale_kind == 2 ? static_cast<const void*>(static_cast<const float*>(a.scales) + n0) : nullptr;
      e = launch_operand_gemm(plan_operand_gemm(false, p.f16, m, rows, p.K, 1, p.sms), images,
                              x + static_cast<uint64_t>(m0) * p.K, fwd, a.status, stream);
      if (e != cudaSuccess) return e;
      XentStep s;
      s.logits = logits;
      s.factor = factor;
      s.targets = a.targets;
      s.scales = a.scales;
      s.images = images;
      s.probs = probs;
      s.target_rows = target_rows;
      s.status = a.status;
      s.st = st;
      s.m0 = m0;
      s.n0 = n0;
      s.rows = rows;
      s.vocab = a.vocab;
      s.K = p.K;
      s.scale_kind = a.scale_kind;
      s.f16 = p.f16;
      s.first = n0 == 0;
      e = launch_pdl(xent_step_kernel, dim3(m), dim3(kXentThreads), 0, stream, s);
      if (e != cudaSuccess) return e;
      if (!p.grad) continue;
      OperandGemmPlan tp = plan_operand_gemm(true, p.f16, m, rows, p.K, 1, p.sms);
      tp.splits = p.splits;
      OperandGemmOut back;
      back.out32 = acc + static_cast<uint64_t>(m0) * p.K;
      back.split_stride = MK;
      back.ld = p.K;
      back.alpha = n0 == 0 ? nullptr : st.alpha + m0;
      back.beta = st.beta + m0;
      e = launch_operand_gemm(tp, images, probs, back, a.status, stream);
      if (e != cudaSuccess) return e;
    }
  }
  XentFinish f;
  f.targets = a.targets;
  f.scales = a.scales;
  f.st = st;
  f.acc = acc;
  f.split_stride = MK;
  f.target_rows = target_rows;
  f.weight = a.weight;
  f.loss = a.loss;
  f.lse = a.lse;
  f.dX = a.dX;
  f.vocab = a.vocab;
  f.K = p.K;
  f.scale_kind = a.scale_kind;
  f.f16 = p.f16;
  f.splits = p.splits;
  return launch_pdl(xent_finish_kernel, dim3(p.M), dim3(kXentThreads), 0, stream, f);
}

}  // namespace ansdev

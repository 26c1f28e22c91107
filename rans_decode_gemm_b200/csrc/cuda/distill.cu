// distill.cu -- distillation from a teacher's top logits over a compressed
// vocabulary head, forward and backward.
//
//   z_n = x . w_n / T (n < vocab),  lse = log sum_n exp z_n,  p_n = exp(z_n - lse)
//   t_j = exp(v_j / T - teacher's lse) of the listed n_j,  S = sum_j t_j
//   loss = sum_j t_j (log t_j - log p_{n_j}),  dx = g / T sum_n (S p_n - t_n) w_n
//
// As in xent.cu the logits never reach memory: the first product folds them into
// blocks of exponentials under a reference that is known before, and their sums.
// The listed rows' logits leave that epilogue as they are, and have no part in the
// exponentials: a student that has learnt its teacher is all but certain of what the
// teacher lists, and S p - t is then the difference of numbers that agree.  Where it
// is stored once more, in the place of its exponential, it is already taken, in 64
// bits, and is rounded once, relative to itself.
//
// That needs lse first, so with a gradient the whole vocabulary is decoded once and
// its images and all the exponentials of a chunk of tokens are kept (2 bytes each);
// the second product then is one launch over all of it, and writes dX.  Two products
// of 2 M V K operations in all.  Blocks under another reference than their token's
// are rescaled before it: nearly all of the first rows of the vocabulary, which are
// a piece of their own, and hardly any of the others.
//
// Measured alone (32000 x 4096 bf16, 2048 tokens of 64 listed, with the gradient): the
// decoding 150 us, logits 50 + 401 (537 GFLOP, 1.19 PFLOP/s), joins 7 + 15, coefficients
// 9, rows rescaled 24, the product back 399 (1.35 PFLOP/s); the lists (23 us) run beside the
// decoding.  The products bound it.  Without a gradient and at 16 tokens the decoding does:
// 91 + 63 of 217 us, the products, which read 262 MB of images, 32 + 30.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "distill.h"
#include "gemm_common.cuh"
#include "launch.h"
#include "rans_core.cuh"
#include "xent.h"

namespace ansdev {

constexpr uint32_t kDiThreads = 128;
constexpr uint32_t kDiWords = 1024;  // words of a list's bits at a time: 2^20 rows of W
constexpr double kLn2d = 0.69314718055994531, kLog2Ed = 1.4426950408889634;

__device__ __forceinline__ float pow2f_whole(float e) {
  return e < -126.0f ? 0.0f : __uint_as_float(static_cast<uint32_t>(static_cast<int>(fminf(e, 127.0f)) + 127) << 23);
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
  return x;
}
__device__ __forceinline__ double warp_max(double x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x = fmax(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
  return x;
}

struct DistillBegin {
  const int32_t* ids;
  const float *logits, *teacher_lse;
  XentState st;
  uint32_t* words;     // [vocab_words][M]
  int32_t* sorted;     // [M][top]: the list in order, every row once, then -1
  double* t;           // [M][top]: what the teacher has on them
  double2* held;       // [M]: (S, sum_j t_j log t_j)
  uint32_t* status;
  uint32_t M, top, vocab, vocab_words;
  float per_t;
};

// Beside the decoding: sets lift.  f16 exponentials carry the row scale of W and are stored under a power of two that
// puts the largest scale in [1, 2), so that those of e^4 (kXentSlack) times it lie at
// 2^7, and what is listed may be 2^14 above 1 before the token's row is moved.
__global__ void __launch_bounds__(1024) distill_lift_kernel(float* lift, uint32_t vocab, uint32_t f16, uint32_t kind,
                                                            const void* scales) {
  __shared__ float part[32];
  griddep_beside();
  float top = 0.0f;
  if (f16 && (kind == 1 || kind == 2)) {
    // (there are scales up to the next multiple of 128)
#pragma unroll 4
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
    *lift = f16 ? pow2f_whole(static_cast<float>(min(126, max(-118, -ex)))) : 1.0f;
  }
  griddep_beside_end();
}

// Beside the decoding.  A CTA a token puts its list in order.
__global__ void __launch_bounds__(kDiThreads) distill_begin_kernel(const __grid_constant__ DistillBegin P) {
  __shared__ int32_t id[kDistillMaxTop];
  __shared__ double a[kDistillMaxTop], t[kDistillMaxTop];
  __shared__ bool head[kDistillMaxTop];
  __shared__ uint32_t bits[kDiWords];
  __shared__ double part[kDiThreads / 32][2];
  griddep_beside();
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, m = blockIdx.x;
  bool bad = false;
  double top = -INFINITY;
  const uint64_t at = static_cast<uint64_t>(m) * P.top;
  for (uint32_t j = threadIdx.x; j < P.top; j += kDiThreads) {
    int32_t n = __ldg(P.ids + at + j);
    if (n >= 0 && static_cast<uint32_t>(n) >= P.vocab) {
      bad = true;
      n = -1;
    }
    id[j] = n < 0 ? -1 : n;
    a[j] = static_cast<double>(__ldg(P.logits + at + j)) * P.per_t;
    if (n >= 0) top = fmax(top, a[j]);  // (a NaN comes back with the exponentials)
  }
  if (bad) atomicOr(P.status, kStatusBadIndex);
  top = warp_max(top);
  if (lane == 0) part[warp][0] = top;
  __syncthreads();
  for (uint32_t k = 0; k < kDiThreads / 32; ++k) top = fmax(top, part[k][0]);
  double norm;
  if (P.teacher_lse != nullptr) {
    norm = __ldg(P.teacher_lse + m);
  } else {
    const double from = top == -INFINITY ? 0.0 : top;
    double s = 0.0;
    for (uint32_t j = threadIdx.x; j < P.top; j += kDiThreads)
      if (id[j] >= 0) s += exp(a[j] - from);
    s = warp_sum(s);
    if (lane == 0) part[warp][1] = s;
    __syncthreads();
    s = 0.0;
    for (uint32_t k = 0; k < kDiThreads / 32; ++k) s += part[k][1];
    norm = top == -INFINITY ? 0.0 : from + log(s);  // (nothing above -infinity: all shares are 0)
  }
  // every entry's share, and its part of sum t log t
  double sum = 0.0, self = 0.0;
  for (uint32_t j = threadIdx.x; j < P.top; j += kDiThreads) {
    double v = 0.0;
    if (id[j] >= 0 && a[j] != -INFINITY) {  // (of -infinity there is nothing, whatever the teacher's lse)
      const double log_t = a[j] - norm;
      v = exp(log_t);
      sum += v;
      if (v != 0.0) self += v * log_t;
    }
    t[j] = v;
  }
  sum = warp_sum(sum);
  self = warp_sum(self);
  __syncthreads();  // (part has been read, t is written)
  if (lane == 0) {
    part[warp][0] = sum;
    part[warp][1] = self;
  }
  // a row that is listed more than once counts as one with the sum
  for (uint32_t j = threadIdx.x; j < P.top; j += kDiThreads) {
    bool first = id[j] >= 0;
    for (uint32_t i = 0; first && i < j; ++i) first = id[i] != id[j];
    head[j] = first;
  }
  __syncthreads();
  uint32_t heads = 0;
  for (uint32_t j = 0; j < P.top; ++j) heads += head[j] ? 1u : 0u;
  for (uint32_t j = threadIdx.x; j < P.top; j += kDiThreads) {
    if (head[j]) {
      uint32_t rank = 0;
      double all = 0.0;
      for (uint32_t i = 0; i < P.top; ++i) {
        if (id[i] == id[j]) all += t[i];
        else if (head[i] && id[i] < id[j]) ++rank;
      }
      P.sorted[at + rank] = id[j];
      P.t[at + rank] = all;
    }
    if (j >= heads) {
      P.sorted[at + j] = -1;
      P.t[at + j] = 0.0;
    }
  }
  for (uint32_t w0 = 0; w0 < P.vocab_words; w0 += kDiWords) {
    const uint32_t n = min(kDiWords, P.vocab_words - w0);
    for (uint32_t w = threadIdx.x; w < n; w += kDiThreads) bits[w] = 0;
    __syncthreads();
    for (uint32_t j = threadIdx.x; j < P.top; j += kDiThreads) {
      const uint32_t w = static_cast<uint32_t>(id[j]) / 1024u - w0;
      if (id[j] >= 0 && w < n) atomicOr(&bits[w], 1u << (static_cast<uint32_t>(id[j]) / 32u % 32u));
    }
    __syncthreads();
    for (uint32_t w = threadIdx.x; w < n; w += kDiThreads) P.words[static_cast<uint64_t>(w0 + w) * P.M + m] = bits[w];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    for (uint32_t k = 1; k < kDiThreads / 32; ++k) {
      sum += part[k][0];
      self += part[k][1];
    }
    P.held[m] = make_double2(sum, self);
    P.st.ref[m] = kXentNone;
    P.st.sum[m] = 0.0f;
  }
  griddep_beside_end();
}

// A token's final numbers, by a warp: loss and lse, and for the gradient its listed
// coefficients as they are stored, beta (what the second product's sums are times)
// and the shift that its exponentials take.
//
// With R the larger of the others' reference r and the listed logits' own (units of
// log 2), e_j = 2^(z_j - R) and total = l 2^(r - R) + sum_j e_j, the gradient is
//   g S / (T total) (sum_{n not listed} e_n 2^(r - R) w_n + sum_j (p_j - t_j / S) total w_j).
// All of it is stored in units of 2^r, in which the others already are, unless the
// largest of the listed then passes 2^14 (f16; 2^100 in bf16): the row is shifted down by
// as much as it does, whatever the others lose by that being below 2^-38 of the row's largest.
// Where all are listed there is no r, and f16 would lose what is small of a student that has
// learnt its teacher: the listed then are in units of their own largest.
struct DistillCoef {
  XentState st;
  const double* t;
  const double2* held;
  const int32_t* sorted;
  float* z;              // listed logits; coefficients come in their place
  const void* scales;
  const float* weight;
  float *loss, *lse;
  int32_t* shift;        // kDropRow: the row is all zeros
  float* beta;
  uint32_t M, top, scale_kind, f16, grad;
  float per_t;
};
constexpr int32_t kDropRow = 0x7FFFFFFF;
constexpr uint32_t kCoefWarps = 4;

__device__ __forceinline__ void distill_coefs(const DistillCoef& P, uint32_t m, float ref_raw, double l, uint32_t lane) {
  constexpr uint32_t kEach = kDistillMaxTop / 32;
  const uint64_t at = static_cast<uint64_t>(m) * P.top;
  const double2 held = __ldcg(P.held + m);
  double z[kEach], t[kEach];
  bool in[kEach];
  double top = -INFINITY;
#pragma unroll
  for (uint32_t k = 0; k < kEach; ++k) {
    const uint32_t j = 32 * k + lane;
    in[k] = j < P.top && __ldcg(P.sorted + at + j) >= 0;
    z[k] = in[k] ? static_cast<double>(__ldcg(P.z + at + j)) : 0.0;
    t[k] = in[k] ? __ldcg(P.t + at + j) : 0.0;
    if (in[k]) top = fmax(top, z[k] * kLog2Ed);
  }
  top = warp_max(top);
  // R and r (a row without others, or without a finite logit among them, has no r of its own)
  const bool has_ref = ref_raw != kXentNone;
  double R = has_ref ? fmax(static_cast<double>(ref_raw), ceil(top)) : ceil(top);
  if (!(fabs(R) <= 1e300)) R = 0.0;
  const double r = has_ref ? static_cast<double>(ref_raw) : R;
  const double D = R - r;
  double total = 0.0;
#pragma unroll
  for (uint32_t k = 0; k < kEach; ++k)
    if (in[k]) total += exp2(z[k] * kLog2Ed - R);
  total = warp_sum(total);
  total += l == 0.0 ? 0.0 : l * exp2(-D);
  const double lse = R * kLn2d + log(total);
  double cross = 0.0;
#pragma unroll
  for (uint32_t k = 0; k < kEach; ++k)
    if (in[k] && t[k] != 0.0) cross += t[k] * (z[k] - lse);
  cross = warp_sum(cross);
  const double S = held.x;
  if (lane == 0) {
    P.lse[m] = static_cast<float>(lse);
    P.loss[m] = S == 0.0 ? 0.0f : static_cast<float>(held.y - cross);
  }
  if (P.grad == 0) return;
  if (S == 0.0) {
    if (lane == 0) {
      P.shift[m] = kDropRow;
      P.beta[m] = 0.0f;
    }
    return;
  }
  const double lift = __ldcg(P.st.lift);
  double c[kEach];
  double most = 0.0;
#pragma unroll
  for (uint32_t k = 0; k < kEach; ++k) {
    c[k] = 0.0;
    if (!in[k]) continue;
    const int32_t n = __ldcg(P.sorted + at + 32 * k + lane);
    double s = lift;
    if (P.scale_kind == 1) s *= bf16_to_f32(__ldg(static_cast<const uint16_t*>(P.scales) + n));
    else if (P.scale_kind == 2) s *= __ldg(static_cast<const float*>(P.scales) + n);
    c[k] = (exp2(z[k] * kLog2Ed - R) - t[k] / S * total) * s;
    const double big = fabs(c[k]);
    if (big <= 1e300) most = fmax(most, big);
  }
  most = warp_max(most);
  const int E = most == 0.0 ? -2000 : ilogb(most), limit = P.f16 ? 14 : 100;
  const bool over = E + D > limit;
  // the listed are times 2^up, and beta 2^-up.  Beside others without mass (l = 0: all their
  // exponentials are 0) f16 holds the listed alone, the largest of them in [2^14, 2^15)
  const bool alone = P.f16 && l == 0.0f;
  const int up = alone ? min(limit - E, 100) : over ? limit - E : static_cast<int>(D);
  const int back = -up;
  if (lane == 0) {
    P.shift[m] = over && !alone ? static_cast<int32_t>(fmin(E + D - limit, 1e6)) : 0;
    const double g = P.weight != nullptr ? static_cast<double>(__ldg(P.weight + m)) : 1.0;
    double beta = ldexp(g * P.per_t * S / total / lift, back);
    if (!isfinite(lse)) beta = __longlong_as_double(0x7FF8000000000000ll);
    P.beta[m] = static_cast<float>(beta);
  }
#pragma unroll
  for (uint32_t k = 0; k < kEach; ++k)
    if (in[k]) P.z[at + 32 * k + lane] = static_cast<float>(ldexp(c[k], up));
}

__global__ void __launch_bounds__(32 * kCoefWarps) distill_coef_kernel(const __grid_constant__ DistillCoef P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t m = blockIdx.x * kCoefWarps + threadIdx.x / 32;
  if (m < P.M) distill_coefs(P, m, __ldcg(P.st.ref + m), __ldcg(P.st.sum + m), threadIdx.x % 32);
}

// Few tokens' blocks joined into their state, a CTA a token (xent.cu's kernel takes 8
// or 32 of them, and is two CTAs for 16: 8.7 us for 592 blocks where this takes 4), and,
// behind the last piece, their final numbers in the same launch.
struct DistillJoin {
  DistillCoef coef;        // (M: the tokens)
  const float2* blocks;    // [n_blocks][stride]
  uint32_t stride, n_blocks, beside, last;
};
constexpr uint32_t kFewTokens = 128;
__global__ void __launch_bounds__(256) distill_join_kernel(const __grid_constant__ DistillJoin P) {
  __shared__ float part_ref[8], part_sum[8];
  if (P.beside == 0) griddep_wait();
  griddep_launch_dependents();
  const uint32_t m = blockIdx.x, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const float ref_old = __ldcg(P.coef.st.ref + m), l = __ldcg(P.coef.st.sum + m);
  float ref = kXentNone, s = 0.0f;
  for (uint32_t b0 = threadIdx.x; b0 < P.n_blocks; b0 += 4 * 256) {
    float2 u[4];
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k)
      u[k] = b0 + 256 * k < P.n_blocks ? __ldcg(P.blocks + static_cast<uint64_t>(b0 + 256 * k) * P.stride + m)
                                       : make_float2(kXentNone, 0.0f);
    const float top = fmaxf(fmaxf(fmaxf(u[0].x, u[1].x), fmaxf(u[2].x, u[3].x)), ref);
    s = s == 0.0f ? 0.0f : s * pow2f_whole(ref - top);
    ref = top;
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k)
      if (u[k].y != 0.0f) s += u[k].y * pow2f_whole(u[k].x - ref);
  }
  float top = ref;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  s = s == 0.0f ? 0.0f : s * pow2f_whole(ref - top);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  if (lane == 0) {
    part_ref[warp] = top;
    part_sum[warp] = s;
  }
  __syncthreads();
  if (warp == 0) {
    // (every lane does the same)
    ref = ref_old;
    for (uint32_t k = 0; k < 8; ++k) ref = fmaxf(ref, part_ref[k]);
    s = 0.0f;
    for (uint32_t k = 0; k < 8; ++k) s += part_sum[k] == 0.0f ? 0.0f : part_sum[k] * pow2f_whole(part_ref[k] - ref);
    const float keep = ref_old == kXentNone ? 0.0f : pow2f_whole(ref_old - ref);
    s = fmaf(l, keep, s);  // (NaN stays NaN)
    if (lane == 0) {
      P.coef.st.ref[m] = ref;
      P.coef.st.sum[m] = s;
    }
    if (P.last != 0) distill_coefs(P.coef, m, ref, s, lane);
  }
  if (P.beside != 0) griddep_beside_end();
}

// The exponentials of a chunk as the second product takes them: blocks under another
// reference than their token's are rescaled, rows that were shifted likewise, rows
// without a teacher are zeros, and the listed coefficients go to their places.  A CTA
// takes 32 tokens and 32 blocks (1,024 columns), a warp 4 of the tokens; 4 lanes a block.
struct DistillRows {
  const float* ref;          // from the chunk's first token on, as the rest
  const int32_t* shift;
  const int32_t* sorted;
  const float* coef;
  const float2* blocks;
  uint16_t* probs;
  uint32_t m, top, rows, n_blocks, stride, f16;
};
__device__ __forceinline__ uint16_t to_operand(float x, uint32_t f16) {
  return f16 ? __half_as_ushort(__float2half_rn(x)) : __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
__global__ void __launch_bounds__(256) distill_rows_kernel(const __grid_constant__ DistillRows P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t row0 = blockIdx.x * 32 + 4 * warp, b = 32 * blockIdx.y + lane;
  if (row0 >= P.m) return;
  float r[4] = {kXentNone, kXentNone, kXentNone, kXentNone};
  const bool b_in = b < P.n_blocks;
  if (b_in) {
    // (columns up to the stride, a multiple of 4, are there)
    const float4* q = reinterpret_cast<const float4*>(P.blocks + static_cast<uint64_t>(b) * P.stride + row0);
    const float4 u = __ldcg(q), v = __ldcg(q + 1);
    r[0] = u.x; r[1] = u.z; r[2] = v.x; r[3] = v.z;
  }
  // what the four tokens need is asked for together: their references and shifts, a lane
  // each, and their lists' first 32 entries
  const bool mine = lane < 4 && row0 + lane < P.m;
  const float my_ref = mine ? __ldcg(P.ref + row0 + lane) : 0.0f;
  const int32_t my_shift = mine ? __ldcg(P.shift + row0 + lane) : 0;
  int32_t list[4];
#pragma unroll
  for (uint32_t k = 0; k < 4; ++k)
    list[k] = lane < P.top && row0 + k < P.m ? __ldcg(P.sorted + static_cast<uint64_t>(row0 + k) * P.top + lane) : -1;
#pragma unroll
  for (uint32_t k = 0; k < 4; ++k) {
    const uint32_t col = row0 + k;
    if (col >= P.m) break;
    const float ref = __shfl_sync(0xFFFFFFFFu, my_ref, k);
    const int32_t shift = __shfl_sync(0xFFFFFFFFu, my_shift, k);
    const bool drop = shift == kDropRow;
    const float f = !b_in ? 1.0f : drop ? 0.0f : pow2f_whole(r[k] - ref - static_cast<float>(shift));
    const uint64_t at = static_cast<uint64_t>(col) * P.rows + 1024ull * blockIdx.y;
    if (__any_sync(0xFFFFFFFFu, f != 1.0f)) {
      uint4* row = reinterpret_cast<uint4*>(P.probs + at);
      uint4 w[4];
      float g[4];
#pragma unroll
      for (uint32_t q = 0; q < 4; ++q) {
        g[q] = __shfl_sync(0xFFFFFFFFu, f, 8 * q + lane / 4);
        if (g[q] != 1.0f && g[q] != 0.0f) w[q] = __ldcg(row + 32 * q + lane);
      }
#pragma unroll
      for (uint32_t q = 0; q < 4; ++q) {
        if (g[q] == 1.0f) continue;
        if (g[q] == 0.0f) {
          // (a NaN among them is in the token's lse, and so in beta)
          w[q] = make_uint4(0, 0, 0, 0);
        } else {
          uint32_t* u = reinterpret_cast<uint32_t*>(&w[q]);
          if (P.f16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 x = __half22float2(*reinterpret_cast<const __half2*>(u + i));
              const __half2 h = __floats2half2_rn(x.x * g[q], x.y * g[q]);
              u[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
          } else {
            const float s = g[q];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(u[i] << 16) * s,
                                                             __uint_as_float(u[i] & 0xFFFF0000u) * s);
              u[i] = *reinterpret_cast<const uint32_t*>(&x);
            }
          }
        }
        row[32 * q + lane] = w[q];
      }
    }
    if (drop) continue;
    __syncwarp();
    for (uint32_t q = 0; q < P.top; q += 32) {
      const uint32_t j = q + lane;
      int32_t n = list[k];
      if (q != 0) n = j < P.top ? __ldcg(P.sorted + static_cast<uint64_t>(col) * P.top + j) : -1;
      const uint32_t c = static_cast<uint32_t>(n) - 1024u * blockIdx.y;
      if (n >= 0 && c < 1024u) P.probs[at + c] = to_operand(__ldcg(P.coef + static_cast<uint64_t>(col) * P.top + j), P.f16);
      // (in order: the rest lie behind these columns)
      if (__any_sync(0xFFFFFFFFu, n < 0 || (n >= 0 && static_cast<uint32_t>(n) >= 1024u * (blockIdx.y + 1)))) break;
    }
  }
}

static size_t aligned(size_t n) { return (n + 1023) / 1024 * 1024; }

void make_distill_plan(const LayerDev& L, uint32_t M, uint32_t top, bool grad, int sms_in, DistillPlan* p) {
  const uint32_t sms = static_cast<uint32_t>(sms_in), unit = L.tile_n / 128;
  p->M = M;
  p->N = L.N;
  p->K = L.K;
  p->top = top;
  p->vocab_words = (L.N + 1023) / 1024;
  p->grad = grad;
  p->f16 = operand_is_f16(L.dtype);
  p->sms = sms_in;
  if (!grad) {
    XentPlan x;
    make_xent_plan(L, M, false, sms_in, &x);
    p->chunk = x.chunk;
    p->piece = p->first = x.piece;
  } else {
    // chunks of equal size, at most 4096 tokens
    const uint32_t chunks = (M + 4095) / 4096;
    p->chunk = chunks <= 1 ? M : std::min(M, ((M + chunks - 1) / chunks + 255) / 256 * 256);
    // Rescaling a chunk's exponentials reads and writes them at some 5 TB/s; a first
    // piece, whose references serve the others, costs two launches and the end of a
    // round, some 15 us.  A sixteenth of the vocabulary at least, in whole rounds.
    const uint32_t m_blocks = (p->chunk + 255) / 256, blocks = L.N / 128;
    p->piece = p->first = L.N;
    if (4ull * p->chunk * L.N / 5000000 > 15) {
      uint32_t b = sms / m_blocks;
      while (b < blocks / 16) b += std::max(1u, sms / m_blocks);
      b = std::max(unit, b / unit * unit);
      if (b < blocks) {
        p->first = b * 128;
        p->piece = L.N - p->first;
      }
    }
  }
  p->stride = (p->chunk + 3) / 4 * 4;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += aligned(n);
    return o;
  };
  const uint32_t kept = grad ? L.N : p->piece;
  size_t gemm = 0;
  if (grad)
    for (const uint32_t m : {p->chunk, M - (M - 1) / p->chunk * p->chunk})
      gemm = std::max(gemm, operand_gemm_workspace(plan_operand_gemm(true, p->f16, m, L.N, L.K, sms_in)));
  const size_t MT = static_cast<size_t>(M) * top;
  p->off_images = take(operand_bytes(kept, L.K));
  p->off_probs = take(grad ? static_cast<size_t>(p->chunk) * L.N * 2 : 0);
  p->off_blocks = take(static_cast<size_t>(p->stride) * (kept / 32) * 8);
  p->off_x16 = take(p->f16 ? static_cast<size_t>(M) * L.K * 2 : 0);
  p->off_factor = take(p->f16 ? static_cast<size_t>(M) * 4 : 0);
  p->off_state = take((static_cast<size_t>(M) * 4 + 1) * 4);
  p->off_words = take(static_cast<size_t>(p->vocab_words) * M * 4);
  p->off_ids = take(MT * 4);
  p->off_z = take(MT * 4);
  p->off_t = take(MT * 8);
  p->off_coef = take(static_cast<size_t>(M) * 16);
  p->off_gemm = take(gemm);
  p->bytes = at;
}

cudaError_t launch_distill(const DistillPlan& p, const LayerDev& L, const DistillArgs& a, void* ws, cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint8_t* images = w + p.off_images;
  uint16_t* probs = p.grad ? reinterpret_cast<uint16_t*>(w + p.off_probs) : nullptr;
  float2* blocks = reinterpret_cast<float2*>(w + p.off_blocks);
  float* state = reinterpret_cast<float*>(w + p.off_state);
  // (shift and beta in what xent.cu has as the target's logit and alpha)
  int32_t* shift = reinterpret_cast<int32_t*>(state + 2ull * p.M);
  float* beta = state + 3ull * p.M;
  const XentState st{state, state + p.M, nullptr, nullptr, nullptr, state + 4ull * p.M};
  uint16_t* x16 = reinterpret_cast<uint16_t*>(w + p.off_x16);
  float* x_factor = reinterpret_cast<float*>(w + p.off_factor);
  uint32_t* words = reinterpret_cast<uint32_t*>(w + p.off_words);
  int32_t* ids = reinterpret_cast<int32_t*>(w + p.off_ids);
  float* z = reinterpret_cast<float*>(w + p.off_z);
  double* t = reinterpret_cast<double*>(w + p.off_t);
  double2* held = reinterpret_cast<double2*>(w + p.off_coef);
  const uint16_t* x = p.f16 ? x16 : a.X;
  const float* factor = p.f16 ? x_factor : nullptr;
  // the vocabulary in whole tiles
  const uint32_t all = (a.vocab + L.tile_n - 1) / L.tile_n * L.tile_n;
  cudaError_t e;
  auto begin = [&]() {
    const DistillBegin q{a.ids, a.logits, a.teacher_lse, st, words, ids, t, held, a.status, p.M, p.top, a.vocab,
                         p.vocab_words, a.per_t};
    cudaError_t r = launch_pdl(distill_lift_kernel, dim3(1), dim3(1024), 0, stream, st.lift, a.vocab, p.f16, a.scale_kind,
                               a.scales);
    if (r == cudaSuccess) r = launch_pdl(distill_begin_kernel, dim3(p.M), dim3(kDiThreads), 0, stream, q);
    if (r == cudaSuccess && p.f16) r = launch_row_prep(a.X, p.M, p.K, 0, nullptr, true, x16, x_factor, stream);
    return r;
  };
  // the logits of rows n0 .. n0 + rows - 1 (images from `from` on) for tokens m0 ..,
  // folded into blocks from block b0 on
  auto logits = [&](uint32_t n0, uint32_t rows, const uint8_t* from, uint32_t b0, uint32_t m0, uint32_t m) {
    XentEpilogue f = {};
    f.factor = factor ? factor + m0 : nullptr;
    f.scale_kind = a.scale_kind;
    f.scales = a.scale_kind == 1 ? static_cast<const void*>(static_cast<const uint16_t*>(a.scales) + n0)
               : a.scale_kind == 2 ? static_cast<const void*>(static_cast<const float*>(a.scales) + n0) : nullptr;
    f.lift = st.lift;
    f.ref_in = st.ref + m0;
    f.blocks = blocks + static_cast<uint64_t>(b0) * p.stride;
    f.stride = p.stride;
    f.probs = p.grad ? probs + n0 : nullptr;
    f.probs_ld = all;
    f.n0 = n0;
    f.vocab = a.vocab;
    f.listed = words + m0;
    f.listed_stride = p.M;
    f.top = p.top;
    f.ids = ids + static_cast<uint64_t>(m0) * p.top;
    f.z_listed = z + static_cast<uint64_t>(m0) * p.top;
    f.per_t = a.per_t;
    return launch_operand_gemm(plan_operand_gemm(false, p.f16, m, rows, p.K, p.sms), from,
                               x + static_cast<uint64_t>(m0) * p.K, nullptr, &f, w + p.off_gemm, a.status, stream);
  };
  auto coefs_of = [&](uint32_t m0, uint32_t m) {
    const uint64_t at = static_cast<uint64_t>(m0) * p.top;
    return DistillCoef{XentState{st.ref + m0, st.sum + m0, nullptr, nullptr, nullptr, st.lift}, t + at, held + m0, ids + at,
                       z + at, a.scales, a.weight ? a.weight + m0 : nullptr, a.loss + m0, a.lse + m0, shift + m0, beta + m0,
                       m, p.top, a.scale_kind, p.f16, p.grad, a.per_t};
  };
  // their blocks joined into the tokens' state, and, behind the last rows, the tokens'
  // final numbers
  auto join = [&](uint32_t rows, uint32_t b0, uint32_t m0, uint32_t m, bool beside, bool last) {
    const float2* from = blocks + static_cast<uint64_t>(b0) * p.stride;
    if (m <= kFewTokens) {
      const DistillJoin j{coefs_of(m0, m), from, p.stride, rows / 32, beside, last};
      return launch_pdl(distill_join_kernel, dim3(m), dim3(256), 0, stream, j);
    }
    XentJoin j = {};
    j.st = st;
    j.blocks = from;
    j.stride = p.stride;
    j.n_blocks = rows / 32;
    j.m0 = m0;
    j.m = m;
    j.beside = beside;
    cudaError_t r = launch_xent_join(j, stream);
    if (r != cudaSuccess || !last) return r;
    return launch_pdl(distill_coef_kernel, dim3((m + kCoefWarps - 1) / kCoefWarps), dim3(32 * kCoefWarps), 0, stream,
                      coefs_of(m0, m));
  };
  if (!p.grad) {
    // the last tokens' blocks of a piece are joined beside the decoding of the next
    const uint32_t m_last = (p.M - 1) / p.chunk * p.chunk;
    uint32_t before = 0;  // rows of the piece before
    for (uint32_t n0 = 0; n0 < a.vocab; n0 += p.piece) {
      const uint32_t rows = std::min(p.piece, all - n0);
      const bool last = n0 + p.piece >= a.vocab;
      e = launch_operand_decode(L, n0, rows, a.scale_kind, a.scales, a.group_k, images, a.status, p.sms, stream);
      if (e == cudaSuccess && n0 == 0) e = begin();
      if (e == cudaSuccess && n0 != 0) e = join(before, 0, m_last, p.M - m_last, true, false);
      for (uint32_t m0 = 0; e == cudaSuccess && m0 < p.M; m0 += p.chunk) {
        const uint32_t m = std::min(p.chunk, p.M - m0);
        e = logits(n0, rows, images, 0, m0, m);
        if (e == cudaSuccess && (last || m0 != m_last)) e = join(rows, 0, m0, m, false, last);
      }
      if (e != cudaSuccess) return e;
      before = rows;
    }
    return cudaSuccess;
  }
  e = launch_operand_decode(L, 0, all, a.scale_kind, a.scales, a.group_k, images, a.status, p.sms, stream);
  if (e == cudaSuccess) e = begin();
  if (e == cudaSuccess && all > a.vocab) e = launch_xent_blank(images, a.vocab, all, p.K, stream);
  if (e != cudaSuccess) return e;
  for (uint32_t m0 = 0; m0 < p.M; m0 += p.chunk) {
    const uint32_t m = std::min(p.chunk, p.M - m0);
    for (uint32_t n0 = 0; n0 < all;) {
      const uint32_t rows = std::min(n0 == 0 ? p.first : p.piece, all - n0);
      e = logits(n0, rows, images + static_cast<uint64_t>(n0 / 128) * (p.K / 16) * kSlabBytes, n0 / 32, m0, m);
      if (e == cudaSuccess) e = join(rows, n0 / 32, m0, m, false, n0 + rows == all);
      if (e != cudaSuccess) return e;
      n0 += rows;
    }
    const uint64_t at = static_cast<uint64_t>(m0) * p.top;
    const DistillRows d{st.ref + m0, shift + m0, ids + at, z + at, blocks, probs, m, p.top, all, all / 32, p.stride, p.f16};
    e = launch_pdl(distill_rows_kernel, dim3((m + 31) / 32, (all / 32 + 31) / 32), dim3(256), 0, stream, d);
    if (e != cudaSuccess) return e;
    OperandGemmOut back = {};
    back.out16 = a.dX + static_cast<uint64_t>(m0) * p.K;
    back.ld = p.K;
    back.beta = beta + m0;
    back.drops = 1;
    // (the plan that the workspace was made for; fewer rows are cut into no more parts)
    OperandGemmPlan g = plan_operand_gemm(true, p.f16, m, p.N, p.K, p.sms);
    g.rows = all;
    g.splits = std::min(g.splits, std::max(1u, all / 512));
    e = launch_operand_gemm(g, images, probs, &back, nullptr, w + p.off_gemm, a.status, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace ansdev

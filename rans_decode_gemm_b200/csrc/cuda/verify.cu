// verify.cu -- which drafted tokens a target's logits accept, and the token that
// follows them.
//
//   p = softmax(z / T) of a target row, q = softmax(y / T) of a draft row;
//   draft i of a sequence is accepted while u_i q_i(x_i) < p_i(x_i);
//   the next token is the first n with  sum_{j <= n} w_j > v sum_j w_j,
//   w = max(0, p - q) of the row that refused, or p of the row behind the last draft.
//
// A decision compares numbers that may lie next to one another, so everything is
// held in 64 bits: a running sum over a vocabulary has a border every 1 / vocab,
// which sums in 32 bits would move.  And p - q of models that agree is a difference of
// like numbers: what an exponential is off by must be small against kNoMass, from which
// on a difference counts.  2^d is a table of 64ths times the polynomial of degree 4 that
// agrees with 2^f at the five Chebyshev points of |f| <= 1 / 128 (2.4e-15 of the value), or,
// far from a row's reference, a table of sixteenths times that of degree 6 on |f| <= 1 / 32.
//
// Two kernels.  The first reads every row once and leaves a reference and a sum for
// each part of it; the second, a cluster of eight CTAs a sequence, joins the parts
// of the rows that it decides by, and reads the one or two rows that the next token
// is drawn from once more.
//
// Measured, 64 sequences of 8 drafts with the draft's logits, vocabulary 130001 (500 MB):
// the first kernel 118 us alone (4.0 TB/s; the bytes alone would take 76): 18 instructions a
// logit, 7.5 of them of 64 bits, at 61 % of the issue slots and 48 % of the 64-bit pipe.  The
// second 36 (50 MB in two passes, and five rounds of joins one behind another).  16 logits a
// thread at a time and four CTAs an SM: with a polynomial of degree 3, 144 us for both; with 8
// logits 154, three CTAs 157, five 155; with the next 16 asked for before these are summed 142,
// for 16 registers more, not taken for 1 %.  One sequence of 5 drafts of 32000 logits: 8.2 and
// 14 us alone, each latency from end to end.
#include <cuda_runtime.h>

#include <algorithm>

#include "gemm_common.cuh"
#include "launch.h"
#include "rans_core.cuh"
#include "verify.h"

namespace ansdev {

constexpr uint32_t kVerifyThreads = 256, kVerifyWarps = kVerifyThreads / 32;
constexpr uint32_t kVerifyCluster = 8;
constexpr uint32_t kVerifyMaxChunks = 64;
constexpr double kLog2E64 = 1.4426950408889634, kLn2_64 = 0.69314718055994531;
constexpr double kNoRef = -1.0e300;              // the reference of a part without a finite logit
// p - q is rounding from here down: 9.1e-13.  (Of p = q some 1e-14 is left: both polynomials'
// 2.4e-15, and a sum of 2^17 exponentials, 128 of them one after another, another 1e-14 at most.)
constexpr double kNoMass = 1.0 / (1ull << 40);

// 2^(i / 64)
__constant__ double g_powers[64] = {
    1.0, 1.0108892860517005, 1.0218971486541166, 1.0330248790212284,
    1.0442737824274138, 1.0556451783605572, 1.0671404006768237, 1.0787607977571199,
    1.0905077326652577, 1.102382583307841, 1.1143867425958924, 1.1265216186082418,
    1.1387886347566916, 1.1511892299529827, 1.1637248587775775, 1.1763969916502812,
    1.189207115002721, 1.202156731452703, 1.215247359980469, 1.22848053610687,
    1.241857812073484, 1.255380757024691, 1.2690509571917332, 1.2828700160787783,
    1.2968395546510096, 1.3109612115247644, 1.3252366431597413, 1.339667524053303,
    1.3542555469368927, 1.3690024229745905, 1.383909881963832, 1.3989796725383112,
    1.4142135623730951, 1.42961333839197, 1.4451808069770467, 1.460917794180647,
    1.4768261459394993, 1.4929077282912648, 1.5091644275934228, 1.5255981507445384,
    1.5422108254079407, 1.559004400237837, 1.5759808451078865, 1.593142151342267,
    1.6104903319492543, 1.6280274218573478, 1.645755478153965, 1.6636765803267364,
    1.681792830507429, 1.7001063537185235, 1.718619298122478, 1.7373338352737062,
    1.7562521603732995, 1.7753764925265212, 1.7947090750031072, 1.8142521755003989,
    1.8340080864093424, 1.8539791250833855, 1.8741676341103, 1.8945759815869656,
    1.9152065613971474, 1.9360617934922943, 1.9571441241754002, 1.978456026387951};

// 2^d as value * scale (scale a power of two times a sixteenth power of two; 0 for
// d below -1020 and for -infinity).  d at most 1000.
__device__ __forceinline__ void exp2_parts(double d, const double* sixteenths, double& value, double& scale) {
  constexpr double kRound = 422212465065984.0;  // 1.5 * 2^48: adding it rounds to sixteenths
  const bool none = static_cast<uint32_t>(__double2hiint(d)) > 0xC08FE000u;  // below -1020
  d = __hiloint2double(none ? 0 : __double2hiint(d), __double2loint(d));     // (a finite polynomial)
  const double a = d + kRound;
  const int q = __double2loint(a);
  const double f = d - (a - kRound);
  value = fma(f, 0.0001540375624545771, 0.001333381881538924);
  value = fma(value, f, 0.009618129106525682);
  value = fma(value, f, 0.05550410865209357);
  value = fma(value, f, 0.24022650695910086);
  value = fma(value, f, 0.6931471805599468);
  value = fma(value, f, 1.0);
  const double s = sixteenths[q & 15];
  scale = __hiloint2double(none ? 0 : __double2hiint(s) + ((q >> 4) << 20), none ? 0 : __double2loint(s));
}
__device__ __forceinline__ double exp2_of(double d, const double* sixteenths) {
  double value, scale;
  exp2_parts(d, sixteenths, value, scale);
  return value * scale;
}
// 2^k for a whole k <= 0; 0 below -1020
__device__ __forceinline__ double pow2_whole(double k) {
  return k < -1020.0 ? 0.0 : __hiloint2double((static_cast<int>(k) + 1023) << 20, 0);
}

// A logit's distance from a reference, in units of log 2.  The product is rounded by
// itself, as the reference was that came of it: equal logits are then at distance 0
// however large they are, which a fused product would miss by half a step of 2^-53.
__device__ __forceinline__ double distance(double z, double c, double ref) {
  return __dsub_rn(__dmul_rn(z, c), ref);
}

// The same for logits up to 500 above a reference of no more than 2^30 and no more than
// 900 below it, in fewer instructions: one fused product rounds z c - ref to 64ths, a
// second has what is left of it, the polynomial is of degree 4 for 6, and the table holds
// its high words less the index that comes with the exponent.
constexpr double k64th = 105553116266496.0;  // 1.5 * 2^46
struct Near {
  double c, from;      // log2(e) / T;  k64th - ref
  float low, within;   // the logit of distance -900; and up to which magnitude all are near
};
__device__ __forceinline__ bool is_near(double ref) { return fabs(ref) <= 1073741824.0; }
// per: 1 / c
__device__ __forceinline__ Near near_of(double c, double per, double ref) {
  Near r;
  r.c = c;
  r.from = k64th - ref;
  r.low = static_cast<float>((ref - 900.0) * per);
  r.within = static_cast<float>(fmin(ref + 500.0, 900.0 - ref) * per);
  return r;
}
__device__ __forceinline__ void near_parts(float z, const Near& r, const double* table, double& value, double& scale) {
  const double x = z;
  const double a = fma(x, r.c, r.from);
  const int q = __double2loint(a);
  const double f = fma(x, r.c, r.from - a);
  value = fma(f, 0.009618140859595685, 0.05550421039186821);
  value = fma(value, f, 0.2402265069589214);
  value = fma(value, f, 0.6931471805583931);
  value = fma(value, f, 1.0);
  const double s = table[q & 63];
  scale = __hiloint2double(__double2hiint(s) + (q << 14), __double2loint(s));
}

__device__ __forceinline__ void fill_tables(uint32_t i, double* sixteenths, double* near_table) {
  const double s = g_powers[i];
  if (i % 4 == 0) sixteenths[i / 4] = s;
  near_table[i] = __hiloint2double(__double2hiint(s) - static_cast<int>(i << 14), __double2loint(s));
}

// log2(e) / T; 0 for a greedy sequence.  (T from 1e30 on leaves all finite logits alike already.)
struct Heat {
  double c, per;  // log2(e) / T and its inverse
};
__device__ __forceinline__ Heat heat_of(const float* temperature, uint32_t b) {
  const float t = temperature == nullptr ? 1.0f : __ldg(temperature + b);
  const double t64 = fminf(t, 1e30f);
  return t > 0.0f ? Heat{kLog2E64 / t64, kLn2_64 * t64} : Heat{0.0, 0.0};
}

// The last sequence whose first row (its drafts' rows and, for a target, one more
// for every sequence before) is at most `row`; by whole warps.
__device__ __forceinline__ uint32_t sequence_of(const int32_t* starts, uint32_t n_seqs, uint32_t row, uint32_t extra,
                                                uint32_t lane) {
  uint32_t lo = 0, hi = n_seqs;
  while (hi - lo > 1) {
    const uint32_t step = (hi - lo + 31) / 32, at = lo + lane * step;
    const bool in = lane == 0 || (at < hi && static_cast<int64_t>(__ldg(starts + at)) + extra * at <= row);
    const uint32_t bits = __ballot_sync(0xFFFFFFFFu, in);
    const uint32_t k = 31 - __clz(bits);
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

struct VerifyDev {
  VerifyArgs a;
  double2* parts;  // [target rows, then draft rows][n_chunks]: (reference, sum), or (value, index) of the largest
  uint32_t chunk, n_chunks;
};

// One part of one row.
__global__ void __launch_bounds__(kVerifyThreads, 4) verify_sums_kernel(const __grid_constant__ VerifyDev P) {
  __shared__ double sixteenths[16], near_table[64];
  __shared__ double part_ref[kVerifyWarps], part_sum[kVerifyWarps];
  const VerifyArgs& A = P.a;
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  if (threadIdx.x < 64) fill_tables(threadIdx.x, sixteenths, near_table);
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t row = blockIdx.x / P.n_chunks, part = blockIdx.x - row * P.n_chunks;
  const uint32_t n_target = A.n_drafted + A.n_seqs;
  const bool is_target = row < n_target;
  const uint32_t r = is_target ? row : row - n_target;
  const float* z = is_target ? A.target + static_cast<uint64_t>(r) * A.target_stride
                             : A.draft + static_cast<uint64_t>(r) * A.draft_stride;
  // groups of four logits on 16-byte boundaries: group g holds logits 4 g - off .. + 3
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(z) >> 2) & 3u;
  const uint32_t groups = (A.vocab + off + 3) / 4;
  const uint32_t g0 = part * (P.chunk / 4), g1 = part + 1 == P.n_chunks ? groups : min(groups, g0 + P.chunk / 4);
  const float* base = z - off;
  // groups that lie within the row; the first and the last may not
  constexpr uint32_t kDeep = 4, kStep = kDeep * kVerifyThreads;
  const uint32_t in0 = off == 0 ? 0u : 1u, in1 = min(g1, (A.vocab + off) / 4);
  auto load = [&](uint32_t g, float (&x)[4 * kDeep]) {
    if (g >= in0 && g + (kDeep - 1) * kVerifyThreads < in1) {
#pragma unroll
      for (uint32_t k = 0; k < kDeep; ++k) {
        const float4 q = __ldcs(reinterpret_cast<const float4*>(base + 4ull * g) + k * kVerifyThreads);
        x[4 * k] = q.x;
        x[4 * k + 1] = q.y;
        x[4 * k + 2] = q.z;
        x[4 * k + 3] = q.w;
      }
    } else {
#pragma unroll
      for (uint32_t k = 0; k < 4 * kDeep; ++k) {
        // (places in 32 bits: the first group's wrap below 0, and are none)
        const uint32_t at = g + (k / 4) * kVerifyThreads, n = 4 * at - off + k % 4;
        x[k] = at < g1 && n < A.vocab ? __ldg(z + n) : -INFINITY;
      }
    }
  };
  // (the first are on their way while the row's sequence is looked up)
  float x[4 * kDeep];
  load(g0 + threadIdx.x, x);
  const uint32_t b = sequence_of(A.starts, A.n_seqs, r, is_target ? 1u : 0u, lane);
  const Heat heat = heat_of(A.temperature, b);
  const double c = heat.c;
  const bool greedy = c == 0.0;
  if (greedy && !is_target) return;  // (all that a greedy sequence asks is the target's largest)
  __syncthreads();
  bool bad = false, near = false;
  double ref = kNoRef, sum = 0.0;
  Near at_ref = {};
  at_ref.within = -1.0f;  // (none is)
  float best = -INFINITY;
  uint32_t best_at = 0xFFFFFFFFu;
  for (uint32_t g = g0 + threadIdx.x; g < g1; g += kStep) {
    if (g >= g0 + kStep) load(g, x);
    if (greedy) {
      float top = x[0];
#pragma unroll
      for (uint32_t k = 0; k < 4 * kDeep; ++k) {
        bad = bad || !(x[k] <= 3.402823466e38f);
        top = fmaxf(top, x[k]);
      }
      if (top > best) {
        best = top;
#pragma unroll
        for (int k = 4 * kDeep - 1; k >= 0; --k)
          if (x[k] == top) best_at = 4 * (g + (k / 4) * kVerifyThreads) + k % 4 - off;
      }
      continue;
    }
    // one comparison a logit finds NaN, infinities, and what lies far from the reference
    bool all_near = true;
#pragma unroll
    for (uint32_t k = 0; k < 4 * kDeep; ++k) all_near = all_near && fabsf(x[k]) <= at_ref.within;
    if (!all_near) {
      float top = x[0];
#pragma unroll
      for (uint32_t k = 0; k < 4 * kDeep; ++k) {
        bad = bad || !(x[k] <= 3.402823466e38f);
        top = fmaxf(top, x[k]);
      }
      // (64 bits reach 2^500 above a reference and more, so that it hardly ever moves)
      const double d = __dmul_rn(top, c);
      if (d > ref + 500.0 && fabsf(top) <= 3.402823466e38f) {
        const double next = rint(d);
        sum *= pow2_whole(fmax(ref - next, -2000.0));
        ref = next;
        at_ref = near_of(c, heat.per, ref);
        near = is_near(ref);
        if (!near) at_ref.within = -1.0f;
      }
      if (!near && ref != kNoRef) {
#pragma unroll 1
        for (uint32_t k = 0; k < 4 * kDeep; ++k) {
          double value, scale;
          float xk = x[0];
#pragma unroll
          for (uint32_t j = 1; j < 4 * kDeep; ++j) xk = j == k ? x[j] : xk;
          exp2_parts(distance(xk, c, ref), sixteenths, value, scale);
          sum = fma(value, scale, sum);
        }
      }
      if (!near) continue;
#pragma unroll
      for (uint32_t k = 0; k < 4 * kDeep; ++k) x[k] = fmaxf(x[k], at_ref.low);  // (2^-900 is as good as nothing)
    }
#pragma unroll
    for (uint32_t k = 0; k < 4 * kDeep; ++k) {
      double value, scale;
      near_parts(x[k], at_ref, near_table, value, scale);
      sum = fma(value, scale, sum);
    }
  }
  double2* out = P.parts + static_cast<uint64_t>(row) * P.n_chunks + part;
  bad = __syncthreads_or(bad) != 0;
  if (bad) {
    if (threadIdx.x == 0) *out = make_double2(kNoRef, __longlong_as_double(0x7FF8000000000000ll));
    return;
  }
  if (greedy) {
    ref = best;
    sum = best_at;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const double v = __shfl_xor_sync(0xFFFFFFFFu, ref, d), at = __shfl_xor_sync(0xFFFFFFFFu, sum, d);
      if (v > ref || (v == ref && at < sum)) {
        ref = v;
        sum = at;
      }
    }
  } else {
    double top = ref;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmax(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    sum *= pow2_whole(fmax(ref - top, -2000.0));
    ref = top;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  }
  if (lane == 0) {
    part_ref[warp] = ref;
    part_sum[warp] = sum;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (uint32_t w = 1; w < kVerifyWarps; ++w) {
    const double r2 = part_ref[w], s2 = part_sum[w];
    if (greedy) {
      if (r2 > ref || (r2 == ref && s2 < sum)) {
        ref = r2;
        sum = s2;
      }
    } else {
      const double top = fmax(ref, r2);
      sum = sum * pow2_whole(fmax(ref - top, -2000.0)) + s2 * pow2_whole(fmax(r2 - top, -2000.0));
      ref = top;
    }
  }
  *out = make_double2(ref, sum);
}

// A row's parts, two a lane, and those joined: (reference, sum), or (value, index) of
// the largest; sum NaN (index -1) where the row has no distribution.  By whole warps.
struct RowParts {
  double2 u[kVerifyMaxChunks / 32];
};
__device__ __forceinline__ RowParts row_parts(const VerifyDev& P, uint64_t row, bool greedy, uint32_t lane) {
  RowParts r;
#pragma unroll
  for (uint32_t k = 0; k < kVerifyMaxChunks / 32; ++k) {
    const uint32_t at = lane + 32 * k;
    r.u[k] = at < P.n_chunks ? __ldcg(P.parts + row * P.n_chunks + at)
                             : (greedy ? make_double2(-INFINITY, 4294967295.0) : make_double2(kNoRef, 0.0));
  }
  return r;
}
__device__ __forceinline__ double2 join_parts(const RowParts& r, bool greedy) {
  bool bad = false;
#pragma unroll
  for (uint32_t k = 0; k < kVerifyMaxChunks / 32; ++k) bad = bad || isnan(r.u[k].y);
  bad = __any_sync(0xFFFFFFFFu, bad);
  if (greedy) {
    double top = -INFINITY, at = 4294967295.0;
#pragma unroll
    for (uint32_t k = 0; k < kVerifyMaxChunks / 32; ++k)
      if (r.u[k].x > top || (r.u[k].x == top && r.u[k].y < at)) {
        top = r.u[k].x;
        at = r.u[k].y;
      }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const double v = __shfl_xor_sync(0xFFFFFFFFu, top, d), w = __shfl_xor_sync(0xFFFFFFFFu, at, d);
      if (v > top || (v == top && w < at)) {
        top = v;
        at = w;
      }
    }
    if (bad || top == -INFINITY) at = -1.0;
    return make_double2(top, at);
  }
  double top = kNoRef, sum = 0.0;
#pragma unroll
  for (uint32_t k = 0; k < kVerifyMaxChunks / 32; ++k) top = fmax(top, r.u[k].x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmax(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
#pragma unroll
  for (uint32_t k = 0; k < kVerifyMaxChunks / 32; ++k) sum += r.u[k].y * pow2_whole(fmax(r.u[k].x - top, -2000.0));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  if (bad || sum == 0.0) sum = __longlong_as_double(0x7FF8000000000000ll);
  return make_double2(top, sum);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ double cluster_read(const double* p, uint32_t rank) {
  uint32_t at;
  double v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(at) : "memory");
  return v;
}

// Of eight sums in order, the first whose running total passes `aim`, or else the
// last above 0 (8: none is); `before` ends as the total before it.
template <typename F>
__device__ __forceinline__ uint32_t first_past(double aim, double& before, F sum_of) {
  double run = before;
  uint32_t last = 8;
  double last_before = before;
#pragma unroll
  for (uint32_t k = 0; k < 8; ++k) {
    const double s = sum_of(k);
    if (s > 0.0) {
      last = k;
      last_before = run;
      if (run + s > aim) break;
    }
    run += s;
  }
  before = last_before;
  return last;
}

// w of the row that the next token is drawn from, times what the exponentials of p sum to.
struct VerifyRows {
  const float *p, *q;      // the last row, and the draft's (null: none)
  double c, p_ref, q_ref;
  double ratio;            // the sum of p's exponentials over that of q's
  Near p_near, q_near;
  bool near;
  uint32_t without;        // a token that counts for nothing (a draft without logits), or -1
};
// kMany rows of 32 logits from n on (a lane's: n, n + 32, ...; 0 from `end` on).
template <uint32_t kMany>
__device__ __forceinline__ void verify_weights(const VerifyRows& R, uint32_t n, uint32_t end, const double* sixteenths,
                                               const double* near_table, double (&w)[kMany]) {
  float zp[kMany], zq[kMany];
#pragma unroll
  for (uint32_t k = 0; k < kMany; ++k) {
    zp[k] = n + 32 * k < end ? __ldg(R.p + n + 32 * k) : -INFINITY;
    zq[k] = R.q != nullptr && n + 32 * k < end ? __ldg(R.q + n + 32 * k) : -INFINITY;
  }
  if (R.near) {
    // (what is masked came out between 2^-970 and 2^-830; less than that, and less than 0, is none)
    constexpr int kSome = (1023 - 830) << 20;
#pragma unroll
    for (uint32_t k = 0; k < kMany; ++k) {
      double value, scale;
      near_parts(fmaxf(zp[k], R.p_near.low), R.p_near, near_table, value, scale);
      w[k] = __dmul_rn(value, scale);
    }
    if (R.q != nullptr) {
#pragma unroll
      for (uint32_t k = 0; k < kMany; ++k) {
        double value, scale;
        near_parts(fmaxf(zq[k], R.q_near.low), R.q_near, near_table, value, scale);
        // (both products rounded alike, so that equal probabilities leave 0)
        w[k] = fma(-R.ratio, __dmul_rn(value, scale), w[k]);
      }
    }
#pragma unroll
    for (uint32_t k = 0; k < kMany; ++k)
      if (__double2hiint(w[k]) < kSome) w[k] = 0.0;
  } else {
#pragma unroll 1
    for (uint32_t k = 0; k < kMany; ++k) {
      float xp = zp[0], xq = zq[0];
#pragma unroll
      for (uint32_t j = 1; j < kMany; ++j) {
        xp = j == k ? zp[j] : xp;
        xq = j == k ? zq[j] : xq;
      }
      double v = exp2_of(distance(xp, R.c, R.p_ref), sixteenths);
      if (R.q != nullptr) v = fmax(fma(-R.ratio, exp2_of(distance(xq, R.c, R.q_ref), sixteenths), v), 0.0);
#pragma unroll
      for (uint32_t j = 0; j < kMany; ++j)
        if (j == k) w[j] = v;
    }
  }
  if (R.without != 0xFFFFFFFFu) {
#pragma unroll
    for (uint32_t k = 0; k < kMany; ++k)
      if (n + 32 * k == R.without) w[k] = 0.0;
  }
}

// Drafts of a sequence whose rows' sums are kept until it is known which one is drawn from.
constexpr uint32_t kKnown = 32;

// A cluster a sequence.  Every CTA decides where the sequence stops; for the next
// token the vocabulary is cut into 64 runs, one a warp.
__global__ void __cluster_dims__(kVerifyCluster, 1, 1) __launch_bounds__(kVerifyThreads, 4)
    verify_decide_kernel(const __grid_constant__ VerifyDev P) {
  __shared__ double sixteenths[16], near_table[64];
  __shared__ double run_sum[kVerifyWarps], cta_sum[2], piece_sum[kVerifyWarps];
  __shared__ double2 row_join[2], known[kKnown][2];
  __shared__ uint32_t first;
  __shared__ int32_t last_some;
  const VerifyArgs& A = P.a;
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint32_t b = blockIdx.x / kVerifyCluster, rank = blockIdx.x % kVerifyCluster;
  if (threadIdx.x < 64) fill_tables(threadIdx.x, sixteenths, near_table);
  griddep_wait();
  griddep_launch_dependents();
  // (whatever starts hold, rows stay within the logits)
  const int32_t raw0 = __ldg(A.starts + b), raw1 = __ldg(A.starts + b + 1);
  const int32_t drafted = static_cast<int32_t>(A.n_drafted);
  const int32_t s0 = max(0, min(raw0, drafted)), s1 = max(s0, min(raw1, drafted));
  bool wrong = s0 != raw0 || s1 != raw1 || (b == 0 && raw0 != 0) || (b + 1 == A.n_seqs && raw1 != drafted);
  const uint32_t count = static_cast<uint32_t>(s1 - s0), t0 = static_cast<uint32_t>(s0) + b;
  const uint64_t n_target = static_cast<uint64_t>(A.n_drafted) + A.n_seqs;
  const Heat heat = heat_of(A.temperature, b);
  const double c = heat.c, v = __ldg(A.v + b);
  const bool greedy = c == 0.0;
  if (threadIdx.x == 0) {
    first = count;
    last_some = -1;
  }
  __syncthreads();
  // a warp a draft, in turn, and one the row behind the last
  for (uint32_t i = warp; i <= count; i += kVerifyWarps) {
    // (another warp may write it meanwhile: all lanes go by what one of them read)
    if (i > __shfl_sync(0xFFFFFFFFu, *static_cast<volatile uint32_t*>(&first), 0)) break;
    const bool has_q = A.draft != nullptr && !greedy && i < count;
    const RowParts pt = row_parts(P, t0 + i, greedy, lane);
    RowParts pd = pt;
    if (has_q) pd = row_parts(P, n_target + s0 + i, false, lane);
    int32_t x = -1;
    float u = 0.0f, zx = 0.0f, yx = 0.0f;
    if (i < count) {
      x = __ldg(A.tokens + s0 + i);
      u = __ldg(A.u + s0 + i);
    }
    const bool in = x >= 0 && static_cast<uint32_t>(x) < A.vocab;
    if (in && !greedy) {
      zx = __ldg(A.target + (t0 + i) * A.target_stride + x);
      if (A.draft != nullptr) yx = __ldg(A.draft + static_cast<uint64_t>(s0 + i) * A.draft_stride + x);
    }
    const double2 t = join_parts(pt, greedy);
    double2 d = make_double2(0.0, 1.0);
    if (has_q) d = join_parts(pd, false);
    if (i < kKnown && lane == 0) {
      known[i][0] = t;
      known[i][1] = d;
    }
    if (i == count) break;
    bool keep = false;
    if (greedy) {
      keep = in && t.y == static_cast<double>(x);
    } else if (in) {
      // u q < p, both times both sums (false where a row has no distribution)
      const double ep = exp2_of(distance(zx, c, t.x), sixteenths);
      const double eq = has_q ? exp2_of(distance(yx, c, d.x), sixteenths) : 1.0;
      keep = u * eq * t.y < ep * d.y;
    }
    if (!keep && lane == 0) atomicMin(&first, i);
    __syncwarp();
  }
  __syncthreads();
  const uint32_t stop = first;
  const bool refused = stop < count;
  const uint32_t row = t0 + stop;
  if (rank == 0) {
    if (threadIdx.x == 0) A.accepted[b] = static_cast<int32_t>(stop);
    for (uint32_t i = threadIdx.x; i <= count; i += kVerifyThreads) {
      const int32_t x = i < count ? __ldg(A.tokens + s0 + i) : 0;
      wrong = wrong || x < 0 || static_cast<uint32_t>(x) >= A.vocab;
      if (i != stop) A.out[t0 + i] = i < stop ? x : -1;
    }
    if (wrong) atomicOr(A.status, kStatusBadIndex);
  }
  const bool has_draft = refused && A.draft != nullptr && !greedy;
  if (warp < 2) {
    double2 t = make_double2(0.0, 1.0);
    if (stop < kKnown) t = known[stop][warp];
    else if (warp == 0) t = join_parts(row_parts(P, row, greedy, lane), greedy);
    else if (has_draft) t = join_parts(row_parts(P, n_target + s0 + stop, false, lane), false);
    if (lane == 0) row_join[warp] = t;
  }
  if (greedy) {
    // (rows that wrong starts give to sequences of other temperatures may hold sums)
    const double at = row_join[0].y;
    if (rank == 0 && threadIdx.x == 0) A.out[row] = at >= 0.0 && at < A.vocab ? static_cast<int32_t>(at) : -1;
    return;
  }
  __syncthreads();
  if (isnan(row_join[0].y) || isnan(row_join[1].y)) {
    if (rank == 0 && threadIdx.x == 0) A.out[row] = -1;
    return;
  }
  VerifyRows R;
  R.c = c;
  R.p = A.target + static_cast<uint64_t>(row) * A.target_stride;
  R.p_ref = row_join[0].x;
  R.q = has_draft ? A.draft + static_cast<uint64_t>(s0 + stop) * A.draft_stride : nullptr;
  R.q_ref = row_join[1].x;
  R.ratio = row_join[0].y / row_join[1].y;
  R.near = is_near(R.p_ref) && is_near(R.q_ref);
  R.p_near = near_of(c, heat.per, R.p_ref);
  R.q_near = near_of(c, heat.per, R.q_ref);
  R.without = 0xFFFFFFFFu;
  if (refused && A.draft == nullptr) {
    const int32_t x = __ldg(A.tokens + s0 + stop);
    if (x >= 0 && static_cast<uint32_t>(x) < A.vocab) R.without = static_cast<uint32_t>(x);
  }
  // runs are whole numbers of 256 logits
  const uint32_t run = (A.vocab + 64 * 256 - 1) / (64 * 256) * 256;
  for (uint32_t turn = 0;; ++turn) {
    const uint64_t n0 = static_cast<uint64_t>(rank * kVerifyWarps + warp) * run;
    const uint32_t end = static_cast<uint32_t>(min(static_cast<uint64_t>(A.vocab), n0 + run));
    double s = 0.0;
    for (uint64_t n = n0; n < end; n += 256) {
      double w[8];
      verify_weights(R, static_cast<uint32_t>(n) + lane, end, sixteenths, near_table, w);
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) s += w[k];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    if (lane == 0) run_sum[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      double all = 0.0;
      for (uint32_t k = 0; k < kVerifyWarps; ++k) all += run_sum[k];
      cta_sum[turn] = all;
    }
    cluster_arrive();
    cluster_wait();
    double all = 0.0;
#pragma unroll
    for (uint32_t k = 0; k < kVerifyCluster; ++k) all += cluster_read(&cta_sum[turn], k);
    if (turn == 0 && refused && all <= kNoMass * row_join[0].y) {
      // nothing that p has more of than q: p itself
      R.q = nullptr;
      R.without = 0xFFFFFFFFu;
      continue;
    }
    const double aim = v * all;
    double before = 0.0;
    const uint32_t at = first_past(aim, before, [&](uint32_t k) { return cluster_read(&cta_sum[turn], k); });
    // (a row has some mass, but for one that wrong starts left without sums)
    if (at == 8 && rank == 0 && threadIdx.x == 0) A.out[row] = -1;
    // (every CTA's sums have been read: it may end when all have come here)
    cluster_arrive();
    if (at != rank) {
      cluster_wait();
      return;
    }
    const uint32_t w_at = first_past(aim, before, [&](uint32_t k) { return run_sum[k]; });
    // that run once more, 256 logits a warp at a time, kept until it is known which hold
    // the token
    const uint32_t r0 = (rank * kVerifyWarps + w_at) * run, r1 = min(A.vocab, r0 + run);
    int32_t behind = -1;
    for (uint32_t n8 = r0;; n8 += 256 * kVerifyWarps) {
      const bool last = n8 + 256 * kVerifyWarps >= r1;
      const uint32_t p0 = n8 + 256 * warp;
      double w[8];
      verify_weights(R, p0 + lane, r1, sixteenths, near_table, w);
      s = 0.0;
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) s += w[k];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
      __syncthreads();  // (the sums of the round before have been read)
      if (lane == 0) piece_sum[warp] = s;
      __syncthreads();
      double all8 = 0.0;
#pragma unroll
      for (uint32_t k = 0; k < kVerifyWarps; ++k) all8 += piece_sum[k];
      double after = before;
      const uint32_t p_at = first_past(aim, after, [&](uint32_t k) { return piece_sum[k]; });
      // (behind the last round there is nothing: what the rounding of sums has left over
      // goes to the last token that has some)
      if (!(before + all8 > aim) && !last) {
        before += all8;
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
          const uint32_t some = __ballot_sync(0xFFFFFFFFu, w[k] > 0.0);
          if (some != 0) behind = p0 + 32 * k + 31 - __clz(some);
        }
        continue;
      }
      if (p_at == 8) {
        // (nothing in the last round)
        if (lane == 0) atomicMax(&last_some, behind);
        __syncthreads();
        if (threadIdx.x == 0) A.out[row] = last_some;
        cluster_wait();
        return;
      }
      if (p_at != warp) {
        cluster_wait();
        return;
      }
      uint32_t token = 0xFFFFFFFFu;
      bool done = false;
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) {
        double upto = w[k];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const double o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
          if (lane >= static_cast<uint32_t>(d)) upto += o;
        }
        const uint32_t some = __ballot_sync(0xFFFFFFFFu, w[k] > 0.0);
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, w[k] > 0.0 && after + upto > aim);
        if (!done && past != 0) {
          token = p0 + 32 * k + __ffs(past) - 1;
          done = true;
        } else if (!done && some != 0) {
          token = p0 + 32 * k + 31 - __clz(some);
        }
        after += __shfl_sync(0xFFFFFFFFu, upto, 31);
      }
      if (lane == 0) A.out[row] = static_cast<int32_t>(token);
      cluster_wait();
      return;
    }
  }
}

void make_verify_plan(uint32_t n_seqs, uint32_t n_drafted, uint32_t vocab, VerifyPlan* p) {
  // parts of 1,024 to 32,768 logits: one round of 148 SMs, at four CTAs each, or many
  // of long parts; 64 of a row at most.  (The size can be asked for without a device, so that
  // the count of SMs is not one's; any other works the same.)
  const uint64_t rows = 2ull * n_drafted + n_seqs, all = rows * vocab;
  uint64_t chunk = (all / (148 * 4) + 1023) / 1024 * 1024;
  chunk = std::max<uint64_t>(1024, std::min<uint64_t>(chunk, 32768));
  // (a row that starts off a 16-byte boundary has up to three places more)
  const uint64_t places = static_cast<uint64_t>(vocab) + 3;
  chunk = std::max(chunk, ((places + kVerifyMaxChunks - 1) / kVerifyMaxChunks + 1023) / 1024 * 1024);
  p->chunk = static_cast<uint32_t>(chunk);
  p->n_chunks = static_cast<uint32_t>((places + chunk - 1) / chunk);
  p->bytes = static_cast<size_t>(rows) * p->n_chunks * sizeof(double2);
}

cudaError_t launch_verify(const VerifyPlan& plan, const VerifyArgs& a, void* ws, cudaStream_t stream) {
  const VerifyDev P{a, static_cast<double2*>(ws), plan.chunk, plan.n_chunks};
  const uint32_t rows = a.n_drafted + a.n_seqs + (a.draft != nullptr ? a.n_drafted : 0u);
  const cudaError_t e =
      launch_pdl(verify_sums_kernel, dim3(rows * plan.n_chunks), dim3(kVerifyThreads), 0, stream, P);
  if (e != cudaSuccess) return e;
  return launch_pdl(verify_decide_kernel, dim3(a.n_seqs * kVerifyCluster), dim3(kVerifyThreads), 0, stream, P);
}

}  // namespace ansdev

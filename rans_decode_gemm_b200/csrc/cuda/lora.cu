// lora.cu -- low-rank adapters of many requests beside a projection:
//   h = x A_a^T (rank values),  y += s_a h B_a^T,
// and their gradients dh = s_a dy B_a, dx = dh A_a, dA_a = sum dh^T x,
// dB_a = s_a sum dy^T h, a the adapter of each token.
//
// Tokens are grouped by adapter first (a stable counting sort), so that every
// product has one adapter's weights as an operand.  All of them are bound by
// memory: at rank r a token's x of K values meets r dot products, and a tile of
// y of 64 columns takes r steps of a sum.  So the matrix instructions here are
// the warp-wide m16n8k16 ones, whose operands come straight from registers:
// there is no tile to stage, and the order of a sum's steps, and of output
// columns inside a warp's block, is chosen so that every lane's share of an
// operand is one contiguous vector load (each kernel says how).
//
// h and dh are kept in 32 bits and enter the second product as the sum of two
// bf16 values (16 bits of them; off by 2^-17 at most), so that the product is as
// exact as the fp32 outputs it is added to.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "launch.h"
#include "lora.h"
#include "rans_core.cuh"

namespace ansdev {

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// v as hi + lo, both bf16.  An infinite v has lo 0, not inf - inf.
__device__ __forceinline__ void split_bf16(float v, uint16_t& hi, uint16_t& lo) {
  const __nv_bfloat16 h = __float2bfloat16_rn(v);
  hi = __bfloat16_as_ushort(h);
  const float r = v - __bfloat162float(h);
  lo = isfinite(v) ? __bfloat16_as_ushort(__float2bfloat16_rn(r)) : uint16_t(0);
}

__device__ __forceinline__ uint4 ldg16(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ uint2 ldg8(const uint16_t* p) { return __ldg(reinterpret_cast<const uint2*>(p)); }

// ---- grouping -----------------------------------------------------------------
// One CTA; warp w takes a contiguous range of tokens, so the order inside an
// adapter is the tokens' own.
__global__ void __launch_bounds__(1024) lora_group_kernel(const int32_t* __restrict__ ids, uint32_t M, uint32_t n,
                                                          uint32_t tm, LoraGroups G, uint32_t* status) {
  __shared__ uint32_t cnt[32][kLoraMaxAdapters];
  __shared__ uint32_t total[kLoraMaxAdapters], start[kLoraMaxAdapters];
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (uint32_t i = threadIdx.x; i < 32 * n; i += 1024) cnt[i / n][i % n] = 0;
  __syncthreads();
  const uint32_t per = (M + 1023) / 1024 * 32;
  const uint32_t b = min(M, warp * per), e = min(M, b + per);
  bool bad = false;
  auto id_of = [&](uint32_t m) -> uint32_t {
    const int32_t id = m < e ? __ldg(ids + m) : -1;
    if (id >= static_cast<int32_t>(n)) bad = true;
    return id < 0 || id >= static_cast<int32_t>(n) ? 0xFFFFFFFFu : static_cast<uint32_t>(id);
  };
  for (uint32_t m = b; m < e; m += 32) {
    const uint32_t id = id_of(m + lane);
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
    if (id != 0xFFFFFFFFu && lane == __ffs(same) - 1) cnt[warp][id] += __popc(same);
    __syncwarp();
  }
  if (bad) atomicOr(status, kStatusBadIndex);
  __syncthreads();
  if (threadIdx.x < n) {
    uint32_t run = 0;
    for (uint32_t w = 0; w < 32; ++w) {
      const uint32_t v = cnt[w][threadIdx.x];
      cnt[w][threadIdx.x] = run;
      run += v;
    }
    total[threadIdx.x] = run;
  }
  __syncthreads();
  if (threadIdx.x < n) {
    uint32_t at = 0, tile = 0;
    for (uint32_t a = 0; a < threadIdx.x; ++a) {
      at += total[a];
      tile += (total[a] + tm - 1) / tm;
    }
    const uint32_t mine = total[threadIdx.x];
    start[threadIdx.x] = at;
    G.off[threadIdx.x] = at;
    for (uint32_t i = 0; i < mine; i += tm, ++tile) {
      G.tile_adapter[tile] = threadIdx.x;
      G.tile_start[tile] = at + i;
      G.tile_count[tile] = min(tm, mine - i);
    }
    if (threadIdx.x == n - 1) {
      G.off[n] = at + mine;
      *G.n_tiles = tile;
    }
  }
  __syncthreads();
  for (uint32_t m = b; m < e; m += 32) {
    const uint32_t id = id_of(m + lane);
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
    if (id != 0xFFFFFFFFu) {
      const uint32_t first = cnt[warp][id];
      G.perm[start[id] + first + __popc(same & lanemask_lt())] = m + lane;
    }
    __syncwarp();
    if (id != 0xFFFFFFFFu && lane == __ffs(same) - 1) cnt[warp][id] += __popc(same);
    __syncwarp();
  }
}

// ---- shrink: a token's C values against rank rows or columns -------------------
// part[split][p][j] = sum over the split's range of c of in[perm[p]][c] * w,
// w = A[j][c] (kCols false) or B[c][j] (kCols true).  A CTA takes one tile of
// tokens (16 or 64) and one range; its 8 warps share the token groups of 16 and
// interleave the range's steps of 32, and are summed in warp order.
constexpr uint32_t kShrinkThreads = 256;

struct ShrinkDev {
  LoraGroups G;
  const uint16_t* in;       // M x C
  const uint16_t* weights;  // adapter a at a * C * rank
  float* part;              // split x M x rank
  uint32_t C, rank, M, groups;  // groups: token groups of 16 in a tile (1 or 4)
  uint32_t len;
};

// Both operands are contiguous along the sum, so lane (g, t) takes values
// 8t .. 8t + 7 of every 32 from its rows; the same 8 serve two instructions, and
// both operands agree on which step of the sum each value is.
template <int NJ>
__device__ __forceinline__ void shrink_rows(const ShrinkDev& P, const uint16_t* x0, const uint16_t* x1,
                                            const uint16_t* w, uint32_t c_begin, uint32_t c_end, uint32_t step,
                                            uint32_t g, uint32_t t, float* red) {
  float acc[NJ][4] = {};
  const uint32_t nj = P.rank / 8;
  for (uint32_t c0 = c_begin; c0 < c_end; c0 += step) {
    const uint32_t c = c0 + 8 * t;
    const bool in = c < c_end;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint4 a = in && x0 ? ldg16(x0 + c) : zero, b = in && x1 ? ldg16(x1 + c) : zero;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (j < nj) {
        const uint4 v = in ? ldg16(w + static_cast<uint64_t>(8 * j + g) * P.C + c) : zero;
        mma_bf16(acc[j], a.x, b.x, a.y, b.y, v.x, v.y);
        mma_bf16(acc[j], a.z, b.z, a.w, b.w, v.z, v.w);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    if (j < nj) {
      float* r = red + g * P.rank + 8 * j + 2 * t;
      r[0] = acc[j][0];
      r[1] = acc[j][1];
      r[8 * P.rank] = acc[j][2];
      r[8 * P.rank + 1] = acc[j][3];
    }
  }
}

// W consecutive bf16 of a row, as W / 2 (at least one) registers.
template <int W>
struct RowVec { uint32_t v[W / 2]; };
template <>
struct RowVec<1> { uint32_t v[1]; };
template <int W>
__device__ __forceinline__ RowVec<W> load_row(const uint16_t* p) {
  RowVec<W> r;
  if constexpr (W == 1) {
    r.v[0] = __ldg(p);
  } else if constexpr (W == 2) {
    r.v[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  } else if constexpr (W == 4) {
    const uint2 q = ldg8(p);
    r.v[0] = q.x; r.v[1] = q.y;
  } else {
    const uint4 q = ldg16(p);
    r.v[0] = q.x; r.v[1] = q.y; r.v[2] = q.z; r.v[3] = q.w;
  }
  return r;
}
// Element j of two rows as one register (row a low).
template <int W>
__device__ __forceinline__ uint32_t pair_of(const RowVec<W>& a, const RowVec<W>& b, int j) {
  return __byte_perm(a.v[j / 2], b.v[j / 2], (j & 1) ? 0x7632u : 0x5410u);
}

// The weights' rows run along the rank, so lane (g, t) takes W consecutive
// columns g W .. of each of the 8 rows 8t .. 8t + 7 of every 32, and pairs of rows
// are put together in registers: column j of instruction i is g W + i.
// One block of 8 W columns from `col` on.  (N and the ranges are multiples of
// 32.)
template <int W>
__device__ __forceinline__ void shrink_cols(const ShrinkDev& P, const uint16_t* x0, const uint16_t* x1,
                                            const uint16_t* w, uint32_t col, uint32_t c_begin, uint32_t c_end,
                                            uint32_t step, uint32_t g, uint32_t t, float* red) {
  float acc[W][4] = {};
  for (uint32_t c0 = c_begin; c0 < c_end; c0 += step) {
    const uint32_t c = c0 + 8 * t;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint4 a = x0 ? ldg16(x0 + c) : zero, b = x1 ? ldg16(x1 + c) : zero;
    RowVec<W> r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = load_row<W>(w + static_cast<uint64_t>(c + i) * P.rank + col + g * W);
#pragma unroll
    for (int j = 0; j < W; ++j) {
      mma_bf16(acc[j], a.x, b.x, a.y, b.y, pair_of<W>(r[0], r[1], j), pair_of<W>(r[2], r[3], j));
      mma_bf16(acc[j], a.z, b.z, a.w, b.w, pair_of<W>(r[4], r[5], j), pair_of<W>(r[6], r[7], j));
    }
  }
#pragma unroll
  for (int j = 0; j < W; ++j) {
    float* q = red + g * P.rank + col + 2 * t * W + j;
    q[0] = acc[j][0];
    q[W] = acc[j][1];
    q[8 * P.rank] = acc[j][2];
    q[8 * P.rank + W] = acc[j][3];
  }
}

template <bool kCols, int NJ>
__global__ void __launch_bounds__(kShrinkThreads) lora_shrink_kernel(const __grid_constant__ ShrinkDev P) {
  extern __shared__ float red[];  // 8 warps x 16 tokens x rank
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tile = blockIdx.x;
  if (tile >= __ldcg(P.G.n_tiles)) return;
  const uint32_t a = __ldcg(P.G.tile_adapter + tile), start = __ldcg(P.G.tile_start + tile),
                 count = __ldcg(P.G.tile_count + tile);
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const uint32_t grp = warp % P.groups, kw = warp / P.groups, n_kw = 8 / P.groups;
  const uint32_t c_begin = blockIdx.y * P.len, c_end = min(P.C, c_begin + P.len);
  const uint32_t r0 = grp * 16 + g, r1 = r0 + 8;
  const uint16_t* x0 = r0 < count ? P.in + static_cast<uint64_t>(__ldcg(P.G.perm + start + r0)) * P.C : nullptr;
  const uint16_t* x1 = r1 < count ? P.in + static_cast<uint64_t>(__ldcg(P.G.perm + start + r1)) * P.C : nullptr;
  const uint16_t* w = P.weights + static_cast<uint64_t>(a) * P.C * P.rank;
  float* mine = red + warp * 16 * P.rank;
  const uint32_t first = c_begin + kw * 32, step = n_kw * 32;
  if constexpr (kCols) {
    // the rank in blocks of 64, 32, 16 and 8 columns
    for (uint32_t col = 0; col < P.rank;) {
      const uint32_t rest = P.rank - col;
      if (rest >= 64) { shrink_cols<8>(P, x0, x1, w, col, first, c_end, step, g, t, mine); col += 64; }
      else if (rest >= 32) { shrink_cols<4>(P, x0, x1, w, col, first, c_end, step, g, t, mine); col += 32; }
      else if (rest >= 16) { shrink_cols<2>(P, x0, x1, w, col, first, c_end, step, g, t, mine); col += 16; }
      else { shrink_cols<1>(P, x0, x1, w, col, first, c_end, step, g, t, mine); col += 8; }
    }
  } else {
    shrink_rows<NJ>(P, x0, x1, w, first, c_end, step, g, t, mine);
  }
  __syncthreads();
  const uint32_t per = 16 * P.rank;
  for (uint32_t i = threadIdx.x; i < P.groups * per; i += kShrinkThreads) {
    const uint32_t row = i / P.rank;
    if (row >= count) break;
    const uint32_t gi = i / per, at = i - gi * per;
    float s = 0.0f;
    for (uint32_t q = 0; q < n_kw; ++q) s += red[(q * P.groups + gi) * per + at];
    P.part[(static_cast<uint64_t>(blockIdx.y) * P.M + start + row) * P.rank + (i - row * P.rank)] = s;
  }
}

// h[p][j] = s_a * sum over the splits, in order.
__global__ void __launch_bounds__(256) lora_sum_kernel(LoraGroups G, const float* __restrict__ part, uint32_t splits,
                                                       uint32_t M, uint32_t rank, const float* scale,
                                                       float* __restrict__ h) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tile = blockIdx.x;
  if (tile >= __ldcg(G.n_tiles)) return;
  const uint32_t a = __ldcg(G.tile_adapter + tile), start = __ldcg(G.tile_start + tile),
                 count = __ldcg(G.tile_count + tile);
  const float s = scale != nullptr ? __ldg(scale + a) : 1.0f;
  const uint64_t base = static_cast<uint64_t>(start) * rank;
  for (uint32_t i = threadIdx.x; i < count * rank; i += 256) {
    float v = 0.0f;
    for (uint32_t q = 0; q < splits; ++q) v += __ldcg(part + static_cast<uint64_t>(q) * M * rank + base + i);
    h[base + i] = v * s;
  }
}

// ---- expand: rank values of a token against C outputs --------------------------
// kCols false: out[m][c] += sum_j h[p][j] * B[c][j];  kCols true: out[m][c] =
// sum_j h[p][j] * A[j][c].  A warp takes 64 columns of a tile's tokens; lane
// (g, t) holds columns g 8 + i of instruction i, so that the sums it ends with
// are columns 16 t .. 16 t + 15 of its rows: four 16-byte accesses a row.
struct ExpandDev {
  LoraGroups G;
  const float* h;           // splits x M x rank
  const float* scale;       // per adapter, or null: 1
  const uint16_t* weights;  // adapter a at a * C * rank
  float* out;               // M x C
  uint32_t C, rank, M, splits, tm;
};

template <bool kCols>
__global__ void __launch_bounds__(256) lora_expand_kernel(const __grid_constant__ ExpandDev P) {
  extern __shared__ __align__(16) uint16_t hs[];  // hi then lo: tm x pitch
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tile = blockIdx.x;
  if (tile >= __ldcg(P.G.n_tiles)) return;
  const uint32_t a = __ldcg(P.G.tile_adapter + tile), start = __ldcg(P.G.tile_start + tile),
                 count = __ldcg(P.G.tile_count + tile);
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const uint32_t r16 = (P.rank + 15) / 16 * 16, pitch = r16 + 8;
  uint16_t* lo_s = hs + P.tm * pitch;
  const float s = P.scale != nullptr ? __ldg(P.scale + a) : 1.0f;
  const uint32_t rows = (count + 15) / 16 * 16;
  for (uint32_t i = threadIdx.x; i < rows * r16; i += blockDim.x) {
    const uint32_t row = i / r16, j = i - row * r16;
    float v = 0.0f;
    if (row < count && j < P.rank)
      for (uint32_t q = 0; q < P.splits; ++q)
        v += __ldcg(P.h + (static_cast<uint64_t>(q) * P.M + start + row) * P.rank + j);
    split_bf16(v * s, hs[row * pitch + j], lo_s[row * pitch + j]);
  }
  __syncthreads();
  const uint32_t c0 = (blockIdx.y * (blockDim.x / 32) + warp) * 64;
  if (c0 >= P.C) return;
  const uint16_t* w = P.weights + static_cast<uint64_t>(a) * P.C * P.rank;
  const uint32_t cl = c0 + 16 * t;  // this lane's output columns
  const bool col_in = cl < P.C;
  for (uint32_t r = 0; r < rows; r += 16) {
    const bool v0 = r + g < count && col_in, v1 = r + g + 8 < count && col_in;
    float* y0 = v0 ? P.out + static_cast<uint64_t>(__ldcg(P.G.perm + start + r + g)) * P.C + cl : nullptr;
    float* y1 = v1 ? P.out + static_cast<uint64_t>(__ldcg(P.G.perm + start + r + g + 8)) * P.C + cl : nullptr;
    float4 o0[4], o1[4];
    if constexpr (!kCols) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (v0) o0[q] = *reinterpret_cast<const float4*>(y0 + 4 * q);
        if (v1) o1[q] = *reinterpret_cast<const float4*>(y1 + 4 * q);
      }
    }
    float acc[8][4] = {};
    const uint32_t h0 = (r + g) * pitch + 4 * t, h1 = h0 + 8 * pitch;
    for (uint32_t k = 0; k < r16; k += 16) {
      const uint2 a0 = *reinterpret_cast<const uint2*>(hs + h0 + k), a1 = *reinterpret_cast<const uint2*>(hs + h1 + k);
      const uint2 l0 = *reinterpret_cast<const uint2*>(lo_s + h0 + k),
                  l1 = *reinterpret_cast<const uint2*>(lo_s + h1 + k);
      const uint32_t j = k + 4 * t;  // this lane's steps of the sum
      if constexpr (!kCols) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint2 b = j < P.rank ? ldg8(w + static_cast<uint64_t>(c0 + g * 8 + i) * P.rank + j) : make_uint2(0, 0);
          mma_bf16(acc[i], a0.x, a1.x, a0.y, a1.y, b.x, b.y);
          mma_bf16(acc[i], l0.x, l1.x, l0.y, l1.y, b.x, b.y);
        }
      } else {
        RowVec<8> v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[q] = RowVec<8>{};
          if (j + q < P.rank && c0 + g * 8 < P.C) v[q] = load_row<8>(w + static_cast<uint64_t>(j + q) * P.C + c0 + g * 8);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t b0 = pair_of<8>(v[0], v[1], i), b1 = pair_of<8>(v[2], v[3], i);
          mma_bf16(acc[i], a0.x, a1.x, a0.y, a1.y, b0, b1);
          mma_bf16(acc[i], l0.x, l1.x, l0.y, l1.y, b0, b1);
        }
      }
    }
    // columns 16 t + i (c0 of instruction i) and 16 t + 8 + i (c1)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = 4 * (q & 1), k = q >> 1;
      float4 u = make_float4(acc[i][k], acc[i + 1][k], acc[i + 2][k], acc[i + 3][k]);
      float4 v = make_float4(acc[i][k + 2], acc[i + 1][k + 2], acc[i + 2][k + 2], acc[i + 3][k + 2]);
      if constexpr (!kCols) {
        if (v0) { u.x += o0[q].x; u.y += o0[q].y; u.z += o0[q].z; u.w += o0[q].w; }
        if (v1) { v.x += o1[q].x; v.y += o1[q].y; v.z += o1[q].z; v.w += o1[q].w; }
      }
      if (v0) *reinterpret_cast<float4*>(y0 + 4 * q) = u;
      if (v1) *reinterpret_cast<float4*>(y1 + 4 * q) = v;
    }
  }
}

// ---- outer: the sum over an adapter's tokens of z^T t ---------------------------
// out[c][j] = sum_p z[perm[p]][c] * h[p][j] for one adapter, in dB's layout (C x
// rank) or dA's (rank x C, kRankMajor).  A CTA takes 64 columns c; its 8 warps
// share the blocks of 32 ranks and split the tokens, 16 a step.  Lane (g, t)
// loads columns 8 g .. 8 g + 7 of tokens 4 t .. 4 t + 3 (16 bytes each) and
// puts pairs of tokens together in registers; h comes from shared memory,
// transposed, as hi + lo.
constexpr uint32_t kOuterThreads = 256, kOuterTokens = 128;
constexpr uint32_t kOuterPitch = kOuterTokens + 8;

struct OuterDev {
  LoraGroups G;
  const uint16_t* z;  // M x C
  const float* h;     // M x rank
  float* out;
  uint32_t C, rank, jblocks;  // blocks of 32 ranks, rounded up to a power of two
};

template <bool kRankMajor>
__global__ void __launch_bounds__(kOuterThreads) lora_outer_kernel(const __grid_constant__ OuterDev P) {
  extern __shared__ __align__(16) uint8_t outer_smem[];
  uint16_t* hi_s = reinterpret_cast<uint16_t*>(outer_smem);  // rank x pitch
  uint16_t* lo_s = hi_s + P.rank * kOuterPitch;
  float* red = reinterpret_cast<float*>(outer_smem);         // 8 warps x 64 x 32, after the last step
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t a = blockIdx.y, c0 = blockIdx.x * 64;
  const uint32_t p_begin = __ldcg(P.G.off + a), p_end = __ldcg(P.G.off + a + 1);
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const uint32_t jb = warp % P.jblocks, tw = warp / P.jblocks, n_tw = 8 / P.jblocks;
  const uint32_t nj = min(4u, P.rank > 32 * jb ? (P.rank - 32 * jb) / 8 : 0u);
  const bool col_in = c0 + 8 * g < P.C;
  float acc[4][4][4] = {};  // pairs of columns, rank blocks of 8
  for (uint32_t p0 = p_begin; p0 < p_end; p0 += kOuterTokens) {
    const uint32_t n_tok = min(kOuterTokens, p_end - p0);
    const uint32_t n16 = (n_tok + 15) / 16 * 16;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < n16 * P.rank; i += kOuterThreads) {
      const uint32_t p = i / P.rank, j = i - p * P.rank;
      const float v = p < n_tok ? __ldcg(P.h + static_cast<uint64_t>(p0 + p) * P.rank + j) : 0.0f;
      split_bf16(v, hi_s[j * kOuterPitch + p], lo_s[j * kOuterPitch + p]);
    }
    __syncthreads();
    for (uint32_t s = 16 * tw; s < n16; s += 16 * n_tw) {
      RowVec<8> z[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        z[q] = RowVec<8>{};
        const uint32_t p = s + 4 * t + q;
        if (p < n_tok && col_in)
          z[q] = load_row<8>(P.z + static_cast<uint64_t>(__ldcg(P.G.perm + p0 + p)) * P.C + c0 + 8 * g);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < nj) {
          const uint32_t at = (32 * jb + 8 * j + g) * kOuterPitch + s + 4 * t;
          const uint2 bh = *reinterpret_cast<const uint2*>(hi_s + at), bl = *reinterpret_cast<const uint2*>(lo_s + at);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t a0 = pair_of<8>(z[0], z[1], 2 * u), a1 = pair_of<8>(z[0], z[1], 2 * u + 1);
            const uint32_t a2 = pair_of<8>(z[2], z[3], 2 * u), a3 = pair_of<8>(z[2], z[3], 2 * u + 1);
            mma_bf16(acc[u][j], a0, a1, a2, a3, bh.x, bh.y);
            mma_bf16(acc[u][j], a0, a1, a2, a3, bl.x, bl.y);
          }
        }
      }
    }
  }
  __syncthreads();
  // column 8 g + 2 u (rows g of instruction u) and 8 g + 2 u + 1 (rows g + 8)
  float* mine = red + warp * 64 * 32;
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float* r = mine + (8 * g + 2 * u) * 32 + 8 * j + 2 * t;
      r[0] = acc[u][j][0];
      r[1] = acc[u][j][1];
      r[32] = acc[u][j][2];
      r[33] = acc[u][j][3];
    }
  __syncthreads();
  const uint32_t cols = min(64u, P.C - c0);
  for (uint32_t i = threadIdx.x; i < cols * P.rank; i += kOuterThreads) {
    const uint32_t c = kRankMajor ? i % cols : i / P.rank;
    const uint32_t j = kRankMajor ? i / cols : i - c * P.rank;
    float v = 0.0f;
    for (uint32_t q = 0; q < n_tw; ++q) v += red[((q * P.jblocks + j / 32) * 64 + c) * 32 + j % 32];
    const uint64_t base = static_cast<uint64_t>(a) * P.C * P.rank;
    if (kRankMajor) P.out[base + static_cast<uint64_t>(j) * P.C + c0 + c] = v;
    else P.out[base + static_cast<uint64_t>(c0 + c) * P.rank + j] = v;
  }
}

// ---- host ----------------------------------------------------------------------
static size_t aligned(size_t n) { return (n + 255) / 256 * 256; }

static LoraGroups groups_at(uint8_t* p, uint32_t M, uint32_t n, uint32_t max_tiles) {
  LoraGroups G;
  uint32_t* w = reinterpret_cast<uint32_t*>(p);
  G.n_tiles = w;
  G.off = w + 1;
  G.perm = G.off + n + 1;
  G.tile_adapter = G.perm + M;
  G.tile_start = G.tile_adapter + max_tiles;
  G.tile_count = G.tile_start + max_tiles;
  return G;
}

// Ranges of a sum over C: enough CTAs for the SMs, at least 256 values each.
static void split_range(uint32_t C, uint32_t tiles, uint32_t most, int sms, uint32_t* splits, uint32_t* len) {
  uint32_t want = std::max(1u, 2u * static_cast<uint32_t>(sms) / std::max(1u, tiles));
  want = std::min({want, most, std::max(1u, C / 256)});
  *len = ((C + want - 1) / want + 255) / 256 * 256;
  *splits = (C + *len - 1) / *len;
}

void make_lora_plan(uint32_t M, const LoraDev& L, bool grad, int sms, LoraPlan* p) {
  p->M = M;
  // tiles of 16 tokens where few share an adapter, of 64 where a tile's weights
  // are read for more of them
  p->tm = M <= 256 ? 16 : 64;
  p->max_tiles = static_cast<uint32_t>(
      std::min<uint64_t>(M, static_cast<uint64_t>(M) / p->tm + std::min(L.n, M)));
  const uint32_t likely = (M + p->tm - 1) / p->tm;
  split_range(L.K, likely, 16, sms, &p->splits_k, &p->len_k);
  split_range(L.N, likely, 16, sms, &p->splits_n, &p->len_n);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += aligned(n);
    return o;
  };
  const size_t row = static_cast<size_t>(M) * L.rank * 4;
  p->off_groups = take((2ull + L.n + M + 3ull * p->max_tiles) * 4);
  p->off_part = take(row * (grad ? std::max(p->splits_k, p->splits_n) : p->splits_k));
  p->off_h = take(grad ? row : 0);
  p->off_dh = take(grad ? row : 0);
  p->bytes = at;
}

// The opt-in shared memory of a kernel, once per device.
template <typename K>
static cudaError_t allow_smem(K kern, uint32_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load() & (1ull << dev))) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev);
  return e;
}

template <bool kCols, int NJ>
static cudaError_t shrink_variant(const ShrinkDev& P, dim3 grid, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(lora_shrink_kernel<kCols, NJ>, 8 * 16 * kLoraMaxRank * 4, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(lora_shrink_kernel<kCols, NJ>, grid, dim3(kShrinkThreads), 8 * 16 * P.rank * 4, stream, P);
}

static cudaError_t shrink(const LoraPlan& p, const LoraDev& L, const LoraGroups& G, bool cols, const uint16_t* in,
                          float* part, cudaStream_t stream) {
  ShrinkDev P;
  P.G = G;
  P.in = in;
  P.weights = cols ? L.B : L.A;
  P.part = part;
  P.C = cols ? L.N : L.K;
  P.rank = L.rank;
  P.M = p.M;
  P.groups = p.tm / 16;
  P.len = cols ? p.len_n : p.len_k;
  const dim3 grid(p.max_tiles, cols ? p.splits_n : p.splits_k);
  if (cols) return shrink_variant<true, 8>(P, grid, stream);
  if (L.rank <= 16) return shrink_variant<false, 2>(P, grid, stream);
  if (L.rank <= 32) return shrink_variant<false, 4>(P, grid, stream);
  if (L.rank <= 64) return shrink_variant<false, 8>(P, grid, stream);
  return shrink_variant<false, 16>(P, grid, stream);
}

template <bool kCols>
static cudaError_t expand(const LoraPlan& p, const LoraDev& L, const LoraGroups& G, const float* h, uint32_t splits,
                          const float* scale, float* out, int sms, cudaStream_t stream) {
  ExpandDev P;
  P.G = G;
  P.h = h;
  P.scale = scale;
  P.weights = kCols ? L.A : L.B;
  P.out = out;
  P.C = kCols ? L.K : L.N;
  P.rank = L.rank;
  P.M = p.M;
  P.splits = splits;
  P.tm = p.tm;
  // as many warps a CTA as still leave every SM a CTA
  const uint32_t blocks = (P.C + 63) / 64, likely = (p.M + p.tm - 1) / p.tm;
  uint32_t warps = 8;
  while (warps > 1 && (blocks + warps - 1) / warps * likely < static_cast<uint32_t>(sms)) warps /= 2;
  const uint32_t smem = 2 * p.tm * ((L.rank + 15) / 16 * 16 + 8) * 2;  // 34 KB at most
  return launch_pdl(lora_expand_kernel<kCols>, dim3(p.max_tiles, (blocks + warps - 1) / warps), dim3(32 * warps), smem,
                    stream, P);
}

template <bool kRankMajor>
static cudaError_t outer(const LoraDev& L, const LoraGroups& G, const uint16_t* z, const float* h, float* out,
                         cudaStream_t stream) {
  constexpr uint32_t kMost = 2 * kLoraMaxRank * kOuterPitch * 2;  // above the 64 KB of the sums
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(lora_outer_kernel<kRankMajor>, kMost, done);
  if (e != cudaSuccess) return e;
  OuterDev P;
  P.G = G;
  P.z = z;
  P.h = h;
  P.out = out;
  P.C = kRankMajor ? L.K : L.N;
  P.rank = L.rank;
  P.jblocks = L.rank <= 32 ? 1 : L.rank <= 64 ? 2 : 4;
  const uint32_t smem = std::max(2 * L.rank * kOuterPitch * 2, 8u * 64 * 32 * 4);
  return launch_pdl(lora_outer_kernel<kRankMajor>, dim3((P.C + 63) / 64, L.n), dim3(kOuterThreads), smem, stream, P);
}

static int current_sms() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

cudaError_t launch_lora_forward(const LoraPlan& p, const LoraDev& L, const uint16_t* X, const int32_t* ids, float* Y,
                                void* ws, uint32_t* status, cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  const LoraGroups G = groups_at(w + p.off_groups, p.M, L.n, p.max_tiles);
  float* part = reinterpret_cast<float*>(w + p.off_part);
  cudaError_t e = launch_pdl(lora_group_kernel, dim3(1), dim3(1024), 0, stream, ids, p.M, L.n, p.tm, G, status);
  if (e == cudaSuccess) e = shrink(p, L, G, false, X, part, stream);
  if (e == cudaSuccess) e = expand<false>(p, L, G, part, p.splits_k, L.scale, Y, current_sms(), stream);
  return e;
}

cudaError_t launch_lora_grad(const LoraPlan& p, const LoraDev& L, const uint16_t* X, const uint16_t* dY,
                             const int32_t* ids, float* dA, float* dB, float* delta, void* ws, uint32_t* status,
                             cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  const LoraGroups G = groups_at(w + p.off_groups, p.M, L.n, p.max_tiles);
  float* part = reinterpret_cast<float*>(w + p.off_part);
  float* h = reinterpret_cast<float*>(w + p.off_h);
  float* dh = reinterpret_cast<float*>(w + p.off_dh);
  cudaError_t e = launch_pdl(lora_group_kernel, dim3(1), dim3(1024), 0, stream, ids, p.M, L.n, p.tm, G, status);
  auto sum = [&](uint32_t splits, float* to) {
    return launch_pdl(lora_sum_kernel, dim3(p.max_tiles), dim3(256), 0, stream, G, part, splits, p.M, L.rank, L.scale,
                      to);
  };
  if (e == cudaSuccess) e = shrink(p, L, G, false, X, part, stream);
  if (e == cudaSuccess) e = sum(p.splits_k, h);
  if (e == cudaSuccess) e = shrink(p, L, G, true, dY, part, stream);
  if (e == cudaSuccess) e = sum(p.splits_n, dh);
  if (e == cudaSuccess) e = outer<false>(L, G, dY, h, dB, stream);
  if (e == cudaSuccess) e = outer<true>(L, G, X, dh, dA, stream);
  if (e == cudaSuccess && delta != nullptr) e = expand<true>(p, L, G, dh, 1, nullptr, delta, current_sms(), stream);
  return e;
}

}  // namespace ansdev

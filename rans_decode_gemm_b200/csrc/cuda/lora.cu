// lora.cu -- low-rank adapters of many requests beside a projection:
//   h = x A_a^T (rank values),  y += s_a h B_a^T,
// and their gradients dh = s_a dy B_a, dx = dh A_a, dA_a = sum dh^T x,
// dB_a = s_a sum dy^T h, a the adapter of each token.
//
// Tokens are grouped by adapter first (a stable counting sort into positions,
// each adapter's starting on a multiple of 16), so that every product has one
// adapter's weights as an operand.  All of them are bound by memory: at rank r
// a token's x of K values meets r dot products, and a tile of y of 64 columns
// takes r steps of a sum.  A tile of r columns is too narrow to feed tcgen05, and
// its tokens lie anywhere, so these are the warp-wide m16n8k16 instructions on
// tiles that cp.async gathers, several stages ahead.
//
// h and dh are kept in 32 bits and enter the products with fp32 results (y, dA,
// dB) as the sum of two bf16 values (17 bits with the second one's sign; off by 2^-17
// at most, 2.2e-6 in the root mean square, which is what dA and dB are off by).  A
// third part brought 500 tokens' dA from 2.5e-6 to 6e-7 and the outer products from 70
// us to 97.
// dx is bf16, and there dh is rounded to bf16 once: the second part would move
// dx by less than its own rounding does, and costs as many matrix instructions
// again, which are what bounds that product (a rank of 64 into 4096 x 14336: 84
// us with both parts).
//
// Measured at rank 64, 4096 tokens of 2 adapters, 4096 x 14336, each alone: both
// shrinks 52 us (150 MB of x and dy; 3 TB/s), both outer products 99 us (19 GFLOP in
// two parts, 40 % of the 520 TFLOP/s these instructions reach; see kOuterStages),
// the expansion into dx 53 us (235 MB written; 4.4 TB/s); one token at rank 16,
// 4096 x 4096: 7 us beside a base product of 35.  Times of whole calls in this file
// are from runs of ten; over seconds, under the power cap, large ones take some
// 10 % longer.  The outer products and the
// expansion are launched beside the decoding of the weights (griddep_beside).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "launch.h"
#include "lora.h"
#include "rans_core.cuh"

namespace ansdev {

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
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

// Is one of two bf16 values infinite or NaN (an exponent of all ones carries into the
// bit above)?  An infinite factor meets the first part of a split value alone: times a
// second part of 0, or of the other sign, it would leave NaN where the product is an
// infinity.
__device__ __forceinline__ uint32_t not_finite2(uint32_t v) { return ((v & 0x7FFF7FFFu) + 0x00800080u) & 0x80008000u; }

__device__ __forceinline__ uint4 ldg16(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ uint2 ldg8(const uint16_t* p) { return __ldg(reinterpret_cast<const uint2*>(p)); }

// 16 bytes from global to shared memory, zeros where !in (src is then not read).
__device__ __forceinline__ void cp16(uint32_t dst_s, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst_s), "l"(src), "r"(in ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// Rows of a staged tile are an odd number of 16-byte chunks apart, so that the 8
// rows a matrix load touches lie in different banks.
constexpr uint32_t kChunkRow = 9 * 16;  // 64 values and one chunk
__host__ __device__ constexpr uint32_t odd_row(uint32_t cols) { return ((cols / 8) | 1u) * 16u; }
constexpr uint32_t kNoToken = 0xFFFFFFFFu;
// Ranks are held in rows of 16, 32, 64 or 128 (zeros from the rank on): a row's
// length is then a constant of the instance, and so are all offsets inside tiles.
__host__ __device__ constexpr uint32_t rank_row(uint32_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

// ---- grouping -----------------------------------------------------------------
// One CTA; warp w takes a contiguous range of tokens, so the order inside an
// adapter is the tokens' own.  Positions up to the adapter's next multiple of 16
// hold no token.
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
      at += (total[a] + 15) / 16 * 16;
      tile += (total[a] + tm - 1) / tm;
    }
    const uint32_t mine = total[threadIdx.x], padded = (mine + 15) / 16 * 16;
    start[threadIdx.x] = at;
    G.off[threadIdx.x] = at;
    for (uint32_t i = 0; i < mine; i += tm, ++tile) {
      G.tile_adapter[tile] = threadIdx.x;
      G.tile_start[tile] = at + i;
      G.tile_count[tile] = min(tm, padded - i);
    }
    for (uint32_t i = mine; i < padded; ++i) G.perm[at + i] = kNoToken;
    if (threadIdx.x == n - 1) {
      G.off[n] = at + padded;
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

// Few tokens: a tile is found without the grouping kernel.  Token m leads a tile
// when a multiple of 16 tokens of its adapter precede it; the tile is m and the
// next 15 of them.  One warp counts and collects them 32 tokens at a time (the
// others wait); false where m leads none.  `bad` is set for an index past the
// adapters.
struct FewTile {
  uint32_t adapter, count;
};
__device__ __forceinline__ bool few_tile(const int32_t* __restrict__ ids, uint32_t M, uint32_t n, uint32_t m,
                                         uint32_t (&tok)[16], uint32_t& found_s, FewTile& tile, bool& bad) {
  const int32_t id = __ldg(ids + m);
  bad = id >= static_cast<int32_t>(n);
  if (id < 0 || bad) return false;
  if (threadIdx.x < 32) {
    const uint32_t lane = threadIdx.x;
    uint32_t before = 0, found = 0;
    for (uint32_t b = 0; b < M && found < 16; b += 32) {
      const bool mine = b + lane < M && __ldg(ids + b + lane) == id;
      const uint32_t same = __ballot_sync(0xFFFFFFFFu, mine);
      const uint32_t from = m <= b ? 0xFFFFFFFFu : m >= b + 32 ? 0u : 0xFFFFFFFFu << (m - b);  // tokens from m on
      before += __popc(same & ~from);
      const uint32_t at = found + __popc(same & from & lanemask_lt());
      if (mine && (from >> lane) & 1u && at < 16) tok[at] = b + lane;
      found += __popc(same & from);
    }
    if (lane == 0) found_s = before % 16 == 0 ? min(16u, found) : 0u;
  }
  __syncthreads();
  tile.adapter = static_cast<uint32_t>(id);
  tile.count = found_s;
  return tile.count != 0;
}

// ---- shrink: a token's C values against rank rows or columns -------------------
// part[split][p][j] = sum over the split's range of c of in[perm[p]][c] * w,
// w = A[j][c] (kCols false) or B[c][j] (kCols true).  A CTA takes one tile of 16
// or 64 positions and one range; a stage is 64 values of c for all of them and
// their weights.  With 64 positions each of the 4 warps has 16 of them; with 16,
// each has a quarter of the stage's sum, and the warps are added in order.
// Three stages: 626.5 us for the same call against 638 with four (fewer CTAs an SM).
constexpr uint32_t kShrinkThreads = 128, kShrinkStages = 3;

struct ShrinkDev {
  LoraGroups G;
  const uint16_t* in;       // M x C
  const uint16_t* weights;  // adapter a at a * C * rank
  float* part;              // split x positions x rank
  uint64_t part_stride;     // positions x rank
  uint32_t C, rank, groups; // groups: 16-position groups of a tile (1 or 4)
  uint32_t len, splits;
  // few tokens: tile m is the one that token m leads, and rows of part are tokens
  const int32_t* ids;
  uint32_t* status;
  uint32_t M, n;
};

__host__ __device__ constexpr uint32_t shrink_w_bytes(bool cols, uint32_t rank) {
  return cols ? 64 * odd_row(rank_row(rank)) : rank * kChunkRow;
}

template <bool kCols, bool kFew, int NJ>
__device__ __forceinline__ void shrink_cta(const ShrinkDev& P, uint8_t* stages_smem, uint32_t (&tok)[16], uint32_t& found) {
  const uint32_t tile = blockIdx.x;
  uint32_t a, start = 0, count;
  if constexpr (kFew) {
    FewTile ft;
    bool bad;
    const bool leads = few_tile(P.ids, P.M, P.n, tile, tok, found, ft, bad);
    if (bad && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(P.status, kStatusBadIndex);
    if (!leads) return;
    a = ft.adapter;
    count = ft.count;
  } else {
    if (tile >= __ldcg(P.G.n_tiles)) return;
    a = __ldcg(P.G.tile_adapter + tile);
    start = __ldcg(P.G.tile_start + tile);
    count = __ldcg(P.G.tile_count + tile);
  }
  const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  const uint32_t c_begin = blockIdx.y * P.len, c_end = min(P.C, c_begin + P.len);
  const uint32_t x_bytes = 16 * P.groups * kChunkRow, stage = x_bytes + shrink_w_bytes(kCols, P.rank);
  const uint32_t base = smem_u32(stages_smem);
  const uint32_t nj = P.rank / 8;
  const uint16_t* w = P.weights + static_cast<uint64_t>(a) * P.C * P.rank;
  // this thread's rows of x: tid / 8 of each group, chunk tid % 8
  const uint16_t* x[4];
  bool x_in[4];
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) {
    const uint32_t row = tid / 8 + 16 * i;
    uint32_t m = kNoToken;
    if (i < P.groups && row < count) m = kFew ? tok[row] : __ldcg(P.G.perm + start + row);
    x_in[i] = m != kNoToken;
    x[i] = P.in + (x_in[i] ? static_cast<uint64_t>(m) * P.C : 0ull);
  }
  auto load = [&](uint32_t xs, uint32_t c0) {
    const uint32_t wsm = xs + x_bytes;
    const uint32_t c = c0 + 8 * (tid % 8);
    const bool in = c < c_end;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
      if (i < P.groups)
        cp16(xs + (tid / 8 + 16 * i) * kChunkRow + (tid % 8) * 16, x[i] + (in ? c : 0u), in && x_in[i]);
    if constexpr (!kCols) {
      const uint16_t* src = w + (in ? static_cast<uint64_t>(tid / 8) * P.C + c : 0ull);
#pragma unroll
      for (uint32_t i = 0; i < (NJ + 1) / 2; ++i) {
        const uint32_t j = tid / 8 + 16 * i;
        if (j < P.rank) cp16(wsm + j * kChunkRow + (tid % 8) * 16, src, in);
        if (in) src += 16ull * P.C;
      }
    } else {
      // NJ chunks a row (those past the rank are not used)
      const uint32_t q = tid % NJ;
      if (q < nj) {
        const uint16_t* src = w + static_cast<uint64_t>(c0 + tid / NJ) * P.rank + 8 * q;
#pragma unroll
        for (uint32_t i = 0; i < 64 * NJ / kShrinkThreads; ++i) {
          const uint32_t row = tid / NJ + i * (kShrinkThreads / NJ);
          const bool r_in = c0 + row < c_end;
          cp16(wsm + row * odd_row(8 * NJ) + q * 16, r_in ? src : w, r_in);
          src += kShrinkThreads / NJ * P.rank;
        }
      }
    }
  };
  const uint32_t n_steps = c_end > c_begin ? (c_end - c_begin + 63) / 64 : 0u;
#pragma unroll
  for (uint32_t i = 0; i + 1 < kShrinkStages; ++i) {
    if (i < n_steps) load(base + i * stage, c_begin + 64 * i);
    cp_commit();
  }
  float acc[NJ][4] = {};
  const uint32_t row0 = P.groups == 4 ? 16 * warp : 0u;
  const uint32_t ks0 = P.groups == 4 ? 0u : warp, ks1 = P.groups == 4 ? 4u : warp + 1;
  uint32_t xs_next = base, load_next = base + (kShrinkStages - 1) * stage;
  const uint32_t ring_end = base + kShrinkStages * stage;
  for (uint32_t it = 0; it < n_steps; ++it) {
    cp_wait<kShrinkStages - 2>();
    __syncthreads();
    if (it + kShrinkStages - 1 < n_steps) load(load_next, c_begin + 64 * (it + kShrinkStages - 1));
    cp_commit();
    if ((load_next += stage) == ring_end) load_next = base;
    const uint32_t xs = xs_next, wsm = xs + x_bytes;
    if ((xs_next += stage) == ring_end) xs_next = base;
    if (row0 >= count) continue;  // this warp's group is empty
#pragma unroll 4
    for (uint32_t ks = ks0; ks < ks1; ++ks) {
      uint32_t f[4];
      ldsm4(f, xs + (row0 + (lane & 15u)) * kChunkRow + (2 * ks + (lane >> 4)) * 16);
      // two blocks of 8 ranks a load (lanes 16-31 address the second; where there
      // is none, the first again, unused)
#pragma unroll
      for (int j = 0; j < NJ; j += 2) {
        if (j < nj) {
          const uint32_t jl = j + 1 < nj ? j + (lane >> 4) : j;
          uint32_t q[4];
          if constexpr (!kCols) ldsm4(q, wsm + (8 * jl + (lane & 7u)) * kChunkRow + (2 * ks + ((lane >> 3) & 1u)) * 16);
          else ldsm4_t(q, wsm + (16 * ks + (lane & 15u)) * odd_row(8 * NJ) + jl * 16);
          mma_bf16(acc[j], f[0], f[1], f[2], f[3], q[0], q[1]);
          if (j + 1 < nj) mma_bf16(acc[j + 1], f[0], f[1], f[2], f[3], q[2], q[3]);
        }
      }
    }
  }
  float* out = P.part + blockIdx.y * P.part_stride + static_cast<uint64_t>(start) * P.rank;
  if (P.groups == 4) {
    if (row0 >= count) return;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (j < nj) {
        float* r = out + static_cast<uint64_t>(row0 + g) * P.rank + 8 * j + 2 * t;
        *reinterpret_cast<float2*>(r) = make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2*>(r + 8 * P.rank) = make_float2(acc[j][2], acc[j][3]);
      }
    }
    return;
  }
  cp_wait<0>();
  __syncthreads();
  float* red = reinterpret_cast<float*>(stages_smem);  // 4 warps x 16 x rank
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    if (j < nj) {
      float* r = red + (16 * warp + g) * P.rank + 8 * j + 2 * t;
      r[0] = acc[j][0];
      r[1] = acc[j][1];
      r[8 * P.rank] = acc[j][2];
      r[8 * P.rank + 1] = acc[j][3];
    }
  }
  __syncthreads();
  const uint32_t per = 16 * P.rank;
  for (uint32_t i = tid; i < count * P.rank; i += kShrinkThreads) {
    const float v = ((red[i] + red[per + i]) + red[2 * per + i]) + red[3 * per + i];
    if constexpr (kFew) out[static_cast<uint64_t>(tok[i / P.rank]) * P.rank + i % P.rank] = v;
    else out[i] = v;
  }
}

// Both products in one launch (z 0: rows of A, z 1: columns of B; the forward pass
// has the first alone).
struct ShrinkBoth {
  ShrinkDev d[2];
};
template <bool kFew, int NJ>
__global__ void __launch_bounds__(kShrinkThreads) lora_shrink_kernel(const __grid_constant__ ShrinkBoth P) {
  extern __shared__ __align__(128) uint8_t stages_smem[];
  __shared__ uint32_t tok[16], found;
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.y >= P.d[blockIdx.z].splits) return;
  if (blockIdx.z == 0) shrink_cta<false, kFew, NJ>(P.d[0], stages_smem, tok, found);
  else if constexpr (!kFew) shrink_cta<true, false, NJ>(P.d[1], stages_smem, tok, found);
}

// Four neighbouring sums over the splits, in order, 8 loads in flight.
__device__ __forceinline__ float4 sum_parts(const float* p, uint32_t splits, uint64_t stride) {
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (uint32_t q0 = 0; q0 < splits; q0 += 8) {
    float4 u[8];
#pragma unroll
    for (uint32_t q = 0; q < 8; ++q)
      u[q] = q0 + q < splits ? __ldcg(reinterpret_cast<const float4*>(p + (q0 + q) * stride))
                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (uint32_t q = 0; q < 8; ++q) {
      v.x += u[q].x; v.y += u[q].y; v.z += u[q].z; v.w += u[q].w;
    }
  }
  return v;
}
// Four values times s as their two bf16 parts (hi and lo 8-byte aligned).
__device__ __forceinline__ void split4(const float4& v, float s, uint16_t* hi, uint16_t* lo) {
  uint16_t h[4], l[4];
  split_bf16(v.x * s, h[0], l[0]);
  split_bf16(v.y * s, h[1], l[1]);
  split_bf16(v.z * s, h[2], l[2]);
  split_bf16(v.w * s, h[3], l[3]);
  *reinterpret_cast<uint2*>(hi) = make_uint2(h[0] | (uint32_t(h[1]) << 16), h[2] | (uint32_t(h[3]) << 16));
  *reinterpret_cast<uint2*>(lo) = make_uint2(l[0] | (uint32_t(l[1]) << 16), l[2] | (uint32_t(l[3]) << 16));
}

// The splits' sums, in order, times s_a, as two bf16 parts: hp[part][p][j], rows
// of rank_row values (zeros from the rank on).
// z: which of the two products.
struct JoinDev {
  const float* part[2];
  uint32_t splits[2];
  uint16_t* hp[2];
};
__global__ void __launch_bounds__(256) lora_join_kernel(LoraGroups G, const __grid_constant__ JoinDev D,
                                                        uint64_t part_stride, uint32_t rank, const float* scale,
                                                        uint64_t hp_stride) {
  const float* __restrict__ part = D.part[blockIdx.z];
  uint16_t* __restrict__ hp = D.hp[blockIdx.z];
  const uint32_t splits = D.splits[blockIdx.z];
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tile = blockIdx.x;
  if (tile >= __ldcg(G.n_tiles)) return;
  const uint32_t a = __ldcg(G.tile_adapter + tile), start = __ldcg(G.tile_start + tile),
                 count = __ldcg(G.tile_count + tile);
  const float s = scale != nullptr ? __ldg(scale + a) : 1.0f;
  const uint32_t rr = rank_row(rank), per = rr / 4;
  for (uint32_t i = blockIdx.y * 256 + threadIdx.x; i < count * per; i += 256 * gridDim.y) {
    const uint32_t row = i / per, j = 4 * (i - row * per);
    // (a position without a token stays 0 even beside an infinite weight)
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (j < rank && __ldcg(G.perm + start + row) != kNoToken)
      v = sum_parts(part + static_cast<uint64_t>(start + row) * rank + j, splits, part_stride);
    const uint64_t at = static_cast<uint64_t>(start + row) * rr + j;
    split4(v, s, hp + at, hp + hp_stride + at);
  }
}

// ---- expand: rank values of a token against C outputs --------------------------
// kCols false: out[m][c] += sum_j h[p][j] * B[c][j];  kCols true: out[m][c] =
// sum_j h[p][j] * A[j][c].  A warp takes 64 columns of a tile's tokens.  Which of
// them is column n of instruction i (expand_col) is chosen so that lane (g, t)
// ends with columns 16 q + 4 t .. + 3 of its rows, q = 0 .. 3: a row's four lanes
// write 64 neighbouring bytes at a time.
// Along the sum lane t has steps 4 t .. 4 t + 3 of every 16, in both operands.
// kCols takes the first part of h alone.
// The warp's weights stay in registers for all of the tile's tokens: kSteps (1, 2, 4
// or 8) blocks of 16 ranks.
struct ExpandDev {
  LoraGroups G;
  const float* part;        // few tokens: sums of the shrink (splits x M x rank)
  const uint16_t* hp;       // else: their two bf16 parts, joined and scaled
  uint64_t part_stride, hp_stride;
  const float* scale;       // of the sums: per adapter, or null: 1
  const uint16_t* weights;  // adapter a at a * C * rank
  float* out;               // M x C
  uint32_t C, rank, splits, tm;
  const int32_t* ids;       // few tokens (see ShrinkDev)
  uint32_t M, n;
};

// Column of the warp's 64 that is column n of instruction i.
__device__ __forceinline__ constexpr uint32_t expand_col(uint32_t n, uint32_t i) {
  return 32 * (n & 1u) + 16 * (i >> 2) + 4 * (n >> 1) + (i & 3u);
}

template <bool kCols>
__device__ __forceinline__ void expand_weights(const ExpandDev& P, const uint16_t* w, uint32_t c0, uint32_t k, uint32_t g,
                                               uint32_t t, uint32_t (&b)[8][2]) {
  const uint32_t j = k + 4 * t;  // this lane's steps of the sum
  if constexpr (!kCols) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint2 v = j < P.rank ? ldg8(w + static_cast<uint64_t>(c0 + expand_col(g, i)) * P.rank + j) : make_uint2(0, 0);
      b[i][0] = v.x;
      b[i][1] = v.y;
    }
  } else {
    // columns of instructions 0-3 and of 4-7 are four neighbours each
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t col = c0 + expand_col(g, 4 * h);
      const bool in = j < P.rank && col < P.C;  // (the rank is a multiple of 8, C of 16)
      const uint16_t* p = w + (in ? static_cast<uint64_t>(j) * P.C + col : 0ull);
      uint2 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = in ? ldg8(p + static_cast<uint64_t>(q) * P.C) : make_uint2(0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t sel = (e & 1) ? 0x7632u : 0x5410u;
        b[4 * h + e][0] = e < 2 ? __byte_perm(v[0].x, v[1].x, sel) : __byte_perm(v[0].y, v[1].y, sel);
        b[4 * h + e][1] = e < 2 ? __byte_perm(v[2].x, v[3].x, sel) : __byte_perm(v[2].y, v[3].y, sel);
      }
    }
  }
}

// sum + the eight products of x and y; not those whose y is not finite, where finite_only.
__device__ __forceinline__ float dot8(const uint4& x, const uint4& y, float sum, bool finite_only) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = __uint_as_float(i & 1 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
    const float b = __uint_as_float(i & 1 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16);
    if (!finite_only || isfinite(b)) sum = fmaf(a, b, sum);
  }
  return sum;
}
// What expand_cta does for the warp's columns c0 .. + 63 into y, with infinite and NaN
// weights kept from h's second part.  Out of line, in plain fp32: rare.
__device__ __noinline__ void expand_apart(const ExpandDev& P, const uint16_t* w, const uint16_t* hi, const uint16_t* lo,
                                          uint32_t pitch, const uint32_t* tok, uint32_t count, uint32_t c0) {
  for (uint32_t r = 0; r < count; ++r) {
    const uint32_t m = tok[r];
    if (m == kNoToken) continue;
    for (uint32_t c = c0 + threadIdx.x % 32; c < c0 + 64; c += 32) {
      float sum = 0.0f;
      for (uint32_t j = 0; j < P.rank; j += 8) {
        const uint4 b = ldg16(w + static_cast<uint64_t>(c) * P.rank + j);
        sum = dot8(*reinterpret_cast<const uint4*>(hi + r * pitch + j), b, sum, false);
        sum = dot8(*reinterpret_cast<const uint4*>(lo + r * pitch + j), b, sum, true);
      }
      P.out[static_cast<uint64_t>(m) * P.C + c] += sum;
    }
  }
}

template <bool kCols, bool kFew, int kSteps>
__device__ __forceinline__ void expand_cta(const ExpandDev& P, uint16_t* hs, uint32_t (&tok)[16], uint32_t& found) {
  const uint32_t tile = blockIdx.x;
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const uint32_t r16 = (P.rank + 15) / 16 * 16;
  constexpr uint32_t kRow = 16 * kSteps, pitch = kRow + 8;
  uint16_t* lo_s = hs + P.tm * pitch;
  const uint32_t c0 = (blockIdx.y * (blockDim.x / 32) + warp) * 64;
  uint32_t b[kSteps][8][2];
  uint32_t a, start = 0, count;
  if constexpr (kFew) {
    FewTile ft;
    bool bad;
    if (!few_tile(P.ids, P.M, P.n, tile, tok, found, ft, bad)) return;
    a = ft.adapter;
    count = 16;
  } else {
    if (tile >= __ldcg(P.G.n_tiles)) return;
    a = __ldcg(P.G.tile_adapter + tile);
    start = __ldcg(P.G.tile_start + tile);
    count = __ldcg(P.G.tile_count + tile);
  }
  const uint16_t* w = P.weights + static_cast<uint64_t>(a) * P.C * P.rank;
  bool apart = false;  // the warp has weights that are not finite
  if (c0 < P.C) {
#pragma unroll
    for (int q = 0; q < kSteps; ++q) expand_weights<kCols>(P, w, c0, 16 * q, g, t, b[q]);
  }
  if constexpr (!kFew) {
    constexpr uint32_t per = kRow / 8;
    for (uint32_t i = threadIdx.x; i < (kCols ? 1 : 2) * count * per; i += blockDim.x) {
      const uint32_t part = i >= count * per ? 1u : 0u, k = i - part * count * per;
      const uint32_t row = k / per, q = k - row * per;
      *reinterpret_cast<uint4*>((part ? lo_s : hs) + row * pitch + 8 * q) = __ldcg(reinterpret_cast<const uint4*>(
          P.hp + part * P.hp_stride + static_cast<uint64_t>(start + row) * kRow + 8 * q));
    }
  } else {
    const float s = P.scale != nullptr ? __ldg(P.scale + a) : 1.0f;
    constexpr uint32_t per = kRow / 4;
    for (uint32_t i = threadIdx.x; i < 16 * per; i += blockDim.x) {
      const uint32_t row = i / per, j = 4 * (i - row * per);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (j < P.rank && row < found)
        v = sum_parts(P.part + static_cast<uint64_t>(tok[row]) * P.rank + j, P.splits, P.part_stride);
      split4(v, s, hs + row * pitch + j, lo_s + row * pitch + j);
    }
  }
  if constexpr (!kCols) {
    uint32_t odd = 0;
    if (c0 < P.C) {
#pragma unroll
      for (int q = 0; q < kSteps; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) odd |= not_finite2(b[q][i][0]) | not_finite2(b[q][i][1]);
    }
    apart = __any_sync(0xFFFFFFFFu, odd != 0);
  }
  __syncthreads();
  if (c0 >= P.C) return;
  if (apart) {
    expand_apart(P, w, hs, lo_s, pitch, kFew ? tok : P.G.perm + start, kFew ? found : count, c0);
    return;
  }
  const uint32_t cl = c0 + 4 * t;  // this lane's output columns: cl + 16 q .. + 3
  for (uint32_t r = 0; r < count; r += 16) {
    uint32_t m0, m1;
    if constexpr (kFew) {
      m0 = g < found ? tok[g] : kNoToken;
      m1 = g + 8 < found ? tok[g + 8] : kNoToken;
    } else {
      m0 = __ldcg(P.G.perm + start + r + g);
      m1 = __ldcg(P.G.perm + start + r + g + 8);
    }
    const bool v0 = m0 != kNoToken, v1 = m1 != kNoToken;
    float* y0 = P.out + (v0 ? static_cast<uint64_t>(m0) * P.C + cl : 0ull);
    float* y1 = P.out + (v1 ? static_cast<uint64_t>(m1) * P.C + cl : 0ull);
    float4 o0[4], o1[4];
    if constexpr (!kCols) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (v0) o0[q] = *reinterpret_cast<const float4*>(y0 + 16 * q);
        if (v1) o1[q] = *reinterpret_cast<const float4*>(y1 + 16 * q);
      }
    }
    float acc[8][4] = {};
    const uint32_t h0 = (r + g) * pitch + 4 * t, h1 = h0 + 8 * pitch;
    auto step = [&](const uint16_t* part, uint32_t k, const uint32_t (&bk)[8][2]) {
      const uint2 a0 = *reinterpret_cast<const uint2*>(part + h0 + k), a1 = *reinterpret_cast<const uint2*>(part + h1 + k);
#pragma unroll
      for (int i = 0; i < 8; ++i) mma_bf16(acc[i], a0.x, a1.x, a0.y, a1.y, bk[i][0], bk[i][1]);
    };
#pragma unroll
    for (int q = 0; q < kSteps; ++q) {
      if (16u * q >= r16) continue;
      step(hs, 16 * q, b[q]);
      if constexpr (!kCols) step(lo_s, 16 * q, b[q]);
    }
    // columns 16 q + 4 t + e: instruction 4 (q & 1) + e, its even (q < 2) or odd column
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = 4 * (q & 1), k = q >> 1;
      float4 u = make_float4(acc[i][k], acc[i + 1][k], acc[i + 2][k], acc[i + 3][k]);
      float4 v = make_float4(acc[i][k + 2], acc[i + 1][k + 2], acc[i + 2][k + 2], acc[i + 3][k + 2]);
      if constexpr (!kCols) {
        if (v0) { u.x += o0[q].x; u.y += o0[q].y; u.z += o0[q].z; u.w += o0[q].w; }
        if (v1) { v.x += o1[q].x; v.y += o1[q].y; v.z += o1[q].z; v.w += o1[q].w; }
      }
      const bool in = c0 + 16 * q < P.C;  // (C is a multiple of 16)
      if (v0 && in) *reinterpret_cast<float4*>(y0 + 16 * q) = u;
      if (v1 && in) *reinterpret_cast<float4*>(y1 + 16 * q) = v;
    }
  }
}
// (kCols, into dx: beside the outer products, which run beside the decoding)
template <bool kCols, bool kFew, int kSteps>
__global__ void __launch_bounds__(128) lora_expand_kernel(const __grid_constant__ ExpandDev P) {
  extern __shared__ __align__(16) uint16_t hs[];  // hi then lo: tm x pitch
  __shared__ uint32_t tok[16], found;
  if constexpr (!kCols) griddep_wait();
  griddep_launch_dependents();
  expand_cta<kCols, kFew, kSteps>(P, hs, tok, found);
  if constexpr (kCols) griddep_beside_end();
}

// ---- outer: the sum over an adapter's tokens of z^T t ---------------------------
// out[c][j] = sum_p z[perm[p]][c] * h[p][j] for one adapter, in dB's layout (C x
// rank) or dA's (rank x C, kRankMajor).  A CTA takes 64 columns c and up to 64 ranks
// (kHalf: half of those in rows of 128.  All 128 left room for one CTA an SM: 181
// us for 3,332 tokens of 12 adapters at rank 104, 6400 x 11008; halves, 167);
// a stage is 64 positions of z and of h's two parts, both read by transposing
// matrix loads.  Warps 0-3 have 16 columns each and the stage's first 32
// positions, warps 4-7 the same columns and the other 32; the halves are added
// at the end.  The tokens of a stage are looked up a stage before its loads.
// Two stages leave room for three CTAs an SM at rank 64.  With three stages the
// outer products of the call above took 70 us alone, but beside the decoding the
// call was slower: 639 against 628.5 us; with 500 tokens at rank 16, 78 against 74.
constexpr uint32_t kOuterThreads = 256, kOuterStages = 2;

struct OuterDev {
  LoraGroups G;
  const uint16_t* z;   // M x C
  const uint16_t* hp;  // 2 x positions x rank_row
  uint64_t hp_stride;
  float* out;
  uint32_t C, rank;
};
__host__ __device__ constexpr uint32_t outer_stage_bytes(uint32_t row) { return 64 * kChunkRow + 2 * 64 * odd_row(row); }

// What outer_cta does, with z's infinities and NaN kept from h's second part (row: of
// hp; the ranks r0 .. + ranks - 1).  Out of line, in plain fp32, four columns by four
// ranks a thread: rare.
template <bool kRankMajor>
__device__ __noinline__ void outer_apart(const OuterDev& P, uint32_t c0, uint32_t row, uint32_t r0, uint32_t ranks) {
  const uint32_t a = blockIdx.y, c = c0 + 4 * (threadIdx.x % 16), j = 4 * (threadIdx.x / 16);
  if (c >= P.C || j >= ranks) return;  // (C is a multiple of 16, the ranks of 8)
  const uint32_t p_begin = __ldcg(P.G.off + a), p_end = __ldcg(P.G.off + a + 1);
  auto values = [](uint2 v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xFFFF0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xFFFF0000u);
  };
  float sum[4][4] = {};
  const uint16_t* h = P.hp + static_cast<uint64_t>(p_begin) * row + r0 + j;
#pragma unroll 2
  for (uint32_t p = p_begin; p < p_end; ++p, h += row) {
    const uint32_t m = __ldcg(P.G.perm + p);
    const uint2 zv = m == kNoToken ? make_uint2(0, 0) : ldg8(P.z + static_cast<uint64_t>(m) * P.C + c);
    float z[4], hi[4], lo[4];
    values(zv, z);
    values(__ldcg(reinterpret_cast<const uint2*>(h)), hi);
    values(__ldcg(reinterpret_cast<const uint2*>(h + P.hp_stride)), lo);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float z2 = isfinite(z[i]) ? z[i] : 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[i][k] = fmaf(z2, lo[k], fmaf(z[i], hi[k], sum[i][k]));
    }
  }
  float* out = P.out + static_cast<uint64_t>(a) * P.C * P.rank;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      out[kRankMajor ? static_cast<uint64_t>(r0 + j + k) * P.C + c + i : static_cast<uint64_t>(c + i) * P.rank + r0 + j + k] = sum[i][k];
}

template <bool kRankMajor, int NJ, bool kHalf>
__device__ __forceinline__ void outer_cta(const OuterDev& P, uint32_t c0, uint8_t* stages_smem) {
  constexpr uint32_t kRow = kHalf ? 128 : 8 * NJ;  // of hp
  const uint32_t r0 = kHalf ? 64 * blockIdx.z : 0u, ranks = kHalf ? min(64u, P.rank - r0) : P.rank;
  const uint32_t a = blockIdx.y;
  const uint32_t p_begin = __ldcg(P.G.off + a), p_end = __ldcg(P.G.off + a + 1);
  const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  const uint32_t cw = 16 * (warp & 3u), half = warp >> 2;
  const uint32_t nj2 = (ranks + 15) / 16;
  constexpr uint32_t h_row = odd_row(8 * NJ), h_bytes = 64 * h_row, stage = outer_stage_bytes(8 * NJ);
  const uint32_t base = smem_u32(stages_smem);
  const bool col_in = c0 + 8 * (tid % 8) < P.C;
  const uint32_t n_steps = (p_end - p_begin + 63) / 64;
  // this thread's two rows of z: positions tid / 8 and tid / 8 + 32 of a stage
  uint32_t ahead[2];
  auto look = [&](uint32_t it) {
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i) {
      const uint32_t p = p_begin + 64 * it + tid / 8 + 32 * i;
      ahead[i] = p < p_end ? __ldcg(P.G.perm + p) : kNoToken;
    }
  };
  // and its chunks of h: NJ a row, of positions tid / NJ and every 256 / NJ further,
  // of the one part and the other
  const uint16_t* h_src = P.hp + static_cast<uint64_t>(p_begin + tid / NJ) * kRow + r0 + 8 * (tid % NJ);
  auto load = [&](uint32_t zs, uint32_t it) {
    const uint32_t hsm = zs + 64 * kChunkRow + (tid / NJ) * h_row + (tid % NJ) * 16;
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i) {
      const bool in = ahead[i] != kNoToken && col_in;
      cp16(zs + (tid / 8 + 32 * i) * kChunkRow + (tid % 8) * 16,
           P.z + (in ? static_cast<uint64_t>(ahead[i]) * P.C + c0 + 8 * (tid % 8) : 0ull), in);
    }
    constexpr uint32_t kRows = kOuterThreads / NJ;  // positions in one go
    const uint32_t left = p_end - p_begin - 64 * it;
#pragma unroll
    for (uint32_t part = 0; part < 2; ++part)
#pragma unroll
      for (uint32_t i = 0; i < (kRows >= 64 ? 1 : 64 / kRows); ++i) {
        const uint32_t row = tid / NJ + i * kRows;
        if (kRows > 64 && row >= 64) break;
        const bool in = row < left;
        cp16(hsm + part * h_bytes + i * kRows * h_row,
             in ? h_src + part * P.hp_stride + static_cast<uint64_t>(64 * it + i * kRows) * kRow : P.hp, in);
      }
  };
  float acc[NJ][4] = {};
  look(0);
#pragma unroll
  for (uint32_t i = 0; i + 1 < kOuterStages; ++i) {
    if (i < n_steps) {
      load(base + i * stage, i);
      look(i + 1);
    }
    cp_commit();
  }
  uint32_t zs_next = base, load_next = base + (kOuterStages - 1) * stage;
  const uint32_t ring_end = base + kOuterStages * stage;
  for (uint32_t it = 0; it < n_steps; ++it) {
    cp_wait<kOuterStages - 2>();
    __syncthreads();
    if (it + kOuterStages - 1 < n_steps) {
      load(load_next, it + kOuterStages - 1);
      look(it + kOuterStages);
    }
    cp_commit();
    if ((load_next += stage) == ring_end) load_next = base;
    const uint32_t zs = zs_next, hsm = zs + 64 * kChunkRow;
    if ((zs_next += stage) == ring_end) zs_next = base;
    const uint32_t n16 = min(4u, (p_end - p_begin - 64 * it) / 16);
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) {
      const uint32_t ks = 2 * half + k;
      if (ks >= n16) break;
      uint32_t f[4];
      ldsm4_t(f, zs + (16 * ks + (lane & 7u) + ((lane >> 4) << 3)) * kChunkRow + (cw / 8 + ((lane >> 3) & 1u)) * 16);
      // two blocks of 8 ranks a load: lanes 16-31 address the second
      const uint32_t hr = hsm + (16 * ks + (lane & 15u)) * h_row + (lane >> 4) * 16;
#pragma unroll
      for (int j = 0; j < NJ / 2; ++j) {
        if (j < nj2) {
          uint32_t hi[4], lo[4];
          ldsm4_t(hi, hr + j * 32);
          ldsm4_t(lo, hr + h_bytes + j * 32);
          mma_bf16(acc[2 * j], f[0], f[1], f[2], f[3], hi[0], hi[1]);
          mma_bf16(acc[2 * j + 1], f[0], f[1], f[2], f[3], hi[2], hi[3]);
          mma_bf16(acc[2 * j], f[0], f[1], f[2], f[3], lo[0], lo[1]);
          mma_bf16(acc[2 * j + 1], f[0], f[1], f[2], f[3], lo[2], lo[3]);
        }
      }
    }
  }
  cp_wait<0>();
  // the sums were formed without a look at z: where one is not finite, again
  bool odd = false;
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    odd = odd || !isfinite(acc[j][0]) || !isfinite(acc[j][1]) || !isfinite(acc[j][2]) || !isfinite(acc[j][3]);
  if (__syncthreads_or(odd)) {
    outer_apart<kRankMajor>(P, c0, kRow, r0, ranks);
    return;
  }
  float4* other = reinterpret_cast<float4*>(stages_smem);  // the second half's sums: [rank blocks][4 warps][32 lanes]
  const uint32_t nj = ranks / 8;
  if (half == 1) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (j < nj) other[(j * 4 + (warp & 3u)) * 32 + lane] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
  }
  __syncthreads();
  if (half == 1 || c0 + cw >= P.C) return;  // (C is a multiple of 16)
  const uint32_t c = c0 + cw + g;
  float* out = P.out + static_cast<uint64_t>(a) * P.C * P.rank;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    if (j < nj) {
      const float4 v = other[(j * 4 + warp) * 32 + lane];
      const float s0 = acc[j][0] + v.x, s1 = acc[j][1] + v.y, s2 = acc[j][2] + v.z, s3 = acc[j][3] + v.w;
      const uint32_t r = r0 + 8 * j + 2 * t;
      if constexpr (kRankMajor) {
        out[static_cast<uint64_t>(r) * P.C + c] = s0;
        out[static_cast<uint64_t>(r + 1) * P.C + c] = s1;
        out[static_cast<uint64_t>(r) * P.C + c + 8] = s2;
        out[static_cast<uint64_t>(r + 1) * P.C + c + 8] = s3;
      } else {
        *reinterpret_cast<float2*>(out + static_cast<uint64_t>(c) * P.rank + r) = make_float2(s0, s1);
        *reinterpret_cast<float2*>(out + static_cast<uint64_t>(c + 8) * P.rank + r) = make_float2(s2, s3);
      }
    }
  }
}

// Both gradients in one launch: dB's blocks of columns first, then dA's.
struct OuterBoth {
  OuterDev b, a;
  uint32_t b_blocks;
  uint32_t beside;  // runs beside the decoding of the weights
};
template <int NJ, bool kHalf>
__global__ void __launch_bounds__(kOuterThreads) lora_outer_kernel(const __grid_constant__ OuterBoth P) {
  extern __shared__ __align__(128) uint8_t stages_smem[];
  if (P.beside == 0) griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x < P.b_blocks) outer_cta<false, NJ, kHalf>(P.b, blockIdx.x * 64, stages_smem);
  else outer_cta<true, NJ, kHalf>(P.a, (blockIdx.x - P.b_blocks) * 64, stages_smem);
  if (P.beside != 0) griddep_beside_end();
}

// ---- host ----------------------------------------------------------------------
static size_t aligned(size_t n) { return (n + 255) / 256 * 256; }

static LoraGroups groups_at(uint8_t* p, uint32_t positions, uint32_t n, uint32_t max_tiles) {
  LoraGroups G;
  uint32_t* w = reinterpret_cast<uint32_t*>(p);
  G.n_tiles = w;
  G.off = w + 1;
  G.perm = G.off + n + 1;
  G.tile_adapter = G.perm + positions;
  G.tile_start = G.tile_adapter + max_tiles;
  G.tile_count = G.tile_start + max_tiles;
  return G;
}

// Tiles to expect: of few tokens, every one may name its own adapter.
static uint32_t likely_tiles(uint32_t M, uint32_t tm, uint32_t n) {
  const uint32_t full = (M + tm - 1) / tm;
  return M <= 64 ? std::max(full, std::min(M, n)) : full;
}

// Ranges of a sum over C: enough CTAs for the SMs, at least 256 values each.
static void split_range(uint32_t C, uint32_t tiles, uint32_t most, int sms, uint32_t* splits, uint32_t* len) {
  uint32_t want = std::max(1u, 4u * static_cast<uint32_t>(sms) / std::max(1u, tiles));
  want = std::min({want, most, std::max(1u, C / 256)});
  *len = ((C + want - 1) / want + 63) / 64 * 64;
  *splits = (C + *len - 1) / *len;
}

// Up to this many tokens a tile holds 16 (few tokens share an adapter).
constexpr uint32_t kLoraSmallTiles = 256;
// Up to this many, in the forward pass, tiles are found and the splits added
// where they are used, which saves two launches (a call of 32 tokens 127 us
// against 131 with them) but repeats the search in every CTA: at 122 tokens 74.6
// against 74.0 us, at 210 tokens of 22 adapters 147 against 126.
constexpr uint32_t kLoraFewTokens = 64;

void make_lora_plan(uint32_t M, const LoraDev& L, bool grad, int sms, LoraPlan* p) {
  p->M = M;
  p->sms = sms;
  p->tm = M <= kLoraSmallTiles ? 16 : 64;
  const uint32_t used = std::min(L.n, M);  // adapters that can have tokens
  p->few = !grad && M <= kLoraFewTokens;
  p->max_tiles = p->few ? M : static_cast<uint32_t>(std::min<uint64_t>(M, static_cast<uint64_t>(M) / p->tm + used));
  p->positions = p->few ? M : static_cast<uint32_t>((static_cast<uint64_t>(M) + 15ull * used + 15) / 16 * 16);
  p->likely = likely_tiles(M, p->tm, L.n);
  const uint32_t likely = p->likely;
  split_range(L.K, likely, 16, sms, &p->splits_k, &p->len_k);
  split_range(L.N, likely, 16, sms, &p->splits_n, &p->len_n);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += aligned(n);
    return o;
  };
  const size_t sums = static_cast<size_t>(p->positions) * L.rank * 4;
  const size_t parts = static_cast<size_t>(p->positions) * rank_row(L.rank) * 4;
  p->off_groups = take((2ull + L.n + p->positions + 3ull * p->max_tiles) * 4);
  p->off_part = take(sums * (grad ? p->splits_k + p->splits_n : p->splits_k));
  p->off_h = take(p->few ? 0 : parts);
  p->off_dh = take(grad ? parts : 0);
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

// Instances by the rank's 8-column blocks, rounded up to 2, 4, 8 or 16.
template <typename F>
static cudaError_t by_rank(uint32_t rank, F f) {
  if (rank <= 16) return f(std::integral_constant<int, 2>{});
  if (rank <= 32) return f(std::integral_constant<int, 4>{});
  if (rank <= 64) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

// x against A's rows into part_x, and (gradients) dy against B's columns into part_y.
template <bool kFew>
static cudaError_t shrink(const LoraPlan& p, const LoraDev& L, const LoraGroups& G, const uint16_t* x, float* part_x,
                          const uint16_t* dy, float* part_y, const int32_t* ids, uint32_t* status, cudaStream_t stream) {
  ShrinkBoth P;
  for (uint32_t q = 0; q < 2; ++q) {
    ShrinkDev& d = P.d[q];
    d.G = G;
    d.in = q ? dy : x;
    d.weights = q ? L.B : L.A;
    d.part = q ? part_y : part_x;
    d.part_stride = static_cast<uint64_t>(p.positions) * L.rank;
    d.C = q ? L.N : L.K;
    d.rank = L.rank;
    d.groups = p.tm / 16;
    d.len = q ? p.len_n : p.len_k;
    d.splits = q ? p.splits_n : p.splits_k;
    d.ids = ids;
    d.status = status;
    d.M = p.M;
    d.n = L.n;
  }
  const bool both = dy != nullptr;
  const dim3 grid(p.max_tiles, both ? std::max(p.splits_k, p.splits_n) : p.splits_k, both ? 2 : 1);
  const uint32_t w_bytes = std::max(shrink_w_bytes(false, L.rank), both ? shrink_w_bytes(true, L.rank) : 0u);
  const uint32_t smem = kShrinkStages * (16 * (p.tm / 16) * kChunkRow + w_bytes);
  return by_rank(L.rank, [&](auto nj) {
    constexpr int NJ = decltype(nj)::value;
    constexpr uint32_t kMost = kShrinkStages * (64 * kChunkRow + (shrink_w_bytes(false, 8 * NJ) > shrink_w_bytes(true, 8 * NJ)
                                                                      ? shrink_w_bytes(false, 8 * NJ)
                                                                      : shrink_w_bytes(true, 8 * NJ)));
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(lora_shrink_kernel<kFew, NJ>, kMost, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(lora_shrink_kernel<kFew, NJ>, grid, dim3(kShrinkThreads), smem, stream, P);
  });
}

static cudaError_t join(const LoraPlan& p, const LoraDev& L, const LoraGroups& G, const JoinDev& D, cudaStream_t stream) {
  const uint32_t row = rank_row(L.rank);
  return launch_pdl(lora_join_kernel, dim3(p.max_tiles, std::max(1u, p.tm * row / 1024), D.hp[1] ? 2 : 1), dim3(256), 0,
                    stream, G, D, static_cast<uint64_t>(p.positions) * L.rank, L.rank, L.scale,
                    static_cast<uint64_t>(p.positions) * row);
}

// h: the shrink's sums (part) or their joined parts (hp), one of them null.
template <bool kCols, bool kFew>
static cudaError_t expand(const LoraPlan& p, const LoraDev& L, const LoraGroups& G, const int32_t* ids, const float* part,
                          const uint16_t* hp, float* out, cudaStream_t stream) {
  const uint32_t row = rank_row(L.rank);
  ExpandDev P;
  P.G = G;
  P.part = part;
  P.hp = hp;
  P.part_stride = static_cast<uint64_t>(p.positions) * L.rank;
  P.hp_stride = static_cast<uint64_t>(p.positions) * row;
  P.scale = L.scale;
  P.weights = kCols ? L.A : L.B;
  P.out = out;
  P.C = kCols ? L.K : L.N;
  P.rank = L.rank;
  P.splits = p.splits_k;
  P.tm = p.tm;
  P.ids = ids;
  P.M = p.M;
  P.n = L.n;
  // as many warps a CTA as still leave every SM two CTAs
  const uint32_t blocks = (P.C + 63) / 64;
  uint32_t warps = 4;
  while (warps > 1 && (blocks + warps - 1) / warps * p.likely < 2u * static_cast<uint32_t>(p.sms)) warps /= 2;
  const uint32_t smem = (kCols ? 1 : 2) * p.tm * (row + 8) * 2;  // 34 KB at most
  const dim3 grid(p.max_tiles, (blocks + warps - 1) / warps), block(32 * warps);
  if (L.rank <= 16) return launch_pdl(lora_expand_kernel<kCols, kFew, 1>, grid, block, smem, stream, P);
  if (L.rank <= 32) return launch_pdl(lora_expand_kernel<kCols, kFew, 2>, grid, block, smem, stream, P);
  if (L.rank <= 64) return launch_pdl(lora_expand_kernel<kCols, kFew, 4>, grid, block, smem, stream, P);
  return launch_pdl(lora_expand_kernel<kCols, kFew, 8>, grid, block, smem, stream, P);
}

static cudaError_t outer(const LoraPlan& p, const LoraDev& L, const LoraGroups& G, const uint16_t* dY, const uint16_t* h,
                         float* dB, const uint16_t* X, const uint16_t* dh, float* dA, bool beside, cudaStream_t stream) {
  const uint64_t hp_stride = static_cast<uint64_t>(p.positions) * rank_row(L.rank);
  OuterBoth P;
  P.b = OuterDev{G, dY, h, hp_stride, dB, L.N, L.rank};
  P.a = OuterDev{G, X, dh, hp_stride, dA, L.K, L.rank};
  P.b_blocks = (L.N + 63) / 64;
  P.beside = beside;
  return by_rank(L.rank, [&](auto nj) {
    constexpr bool kHalf = decltype(nj)::value == 16;
    constexpr int NJ = kHalf ? 8 : decltype(nj)::value;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(lora_outer_kernel<NJ, kHalf>, kOuterStages * outer_stage_bytes(8 * NJ), done);
    if (e != cudaSuccess) return e;
    return launch_pdl(lora_outer_kernel<NJ, kHalf>, dim3(P.b_blocks + (L.K + 63) / 64, L.n, kHalf ? 2 : 1),
                      dim3(kOuterThreads), kOuterStages * outer_stage_bytes(8 * NJ), stream, P);
  });
}

cudaError_t launch_lora_shrink(const LoraPlan& p, const LoraDev& L, const uint16_t* X, const int32_t* ids, void* ws,
                               uint32_t* status, cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  const LoraGroups G = groups_at(w + p.off_groups, p.positions, L.n, p.max_tiles);
  float* part = reinterpret_cast<float*>(w + p.off_part);
  if (p.few) return shrink<true>(p, L, G, X, part, nullptr, nullptr, ids, status, stream);
  cudaError_t e = launch_pdl(lora_group_kernel, dim3(1), dim3(1024), 0, stream, ids, p.M, L.n, p.tm, G, status);
  if (e == cudaSuccess) e = shrink<false>(p, L, G, X, part, nullptr, nullptr, ids, status, stream);
  if (e == cudaSuccess)
    e = join(p, L, G, JoinDev{{part, nullptr}, {p.splits_k, 0}, {reinterpret_cast<uint16_t*>(w + p.off_h), nullptr}}, stream);
  return e;
}

cudaError_t launch_lora_expand(const LoraPlan& p, const LoraDev& L, const int32_t* ids, float* Y, void* ws,
                               cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  const LoraGroups G = groups_at(w + p.off_groups, p.positions, L.n, p.max_tiles);
  if (p.few) return expand<false, true>(p, L, G, ids, reinterpret_cast<float*>(w + p.off_part), nullptr, Y, stream);
  return expand<false, false>(p, L, G, ids, nullptr, reinterpret_cast<uint16_t*>(w + p.off_h), Y, stream);
}

cudaError_t launch_lora_grad_shrink(const LoraPlan& p, const LoraDev& L, const uint16_t* X, const uint16_t* dY,
                                    const int32_t* ids, void* ws, uint32_t* status, cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  const LoraGroups G = groups_at(w + p.off_groups, p.positions, L.n, p.max_tiles);
  float* part = reinterpret_cast<float*>(w + p.off_part);
  uint16_t* h = reinterpret_cast<uint16_t*>(w + p.off_h);
  uint16_t* dh = reinterpret_cast<uint16_t*>(w + p.off_dh);
  cudaError_t e = launch_pdl(lora_group_kernel, dim3(1), dim3(1024), 0, stream, ids, p.M, L.n, p.tm, G, status);
  float* part_y = part + static_cast<uint64_t>(p.splits_k) * p.positions * L.rank;
  if (e == cudaSuccess) e = shrink<false>(p, L, G, X, part, dY, part_y, ids, status, stream);
  if (e == cudaSuccess) e = join(p, L, G, JoinDev{{part, part_y}, {p.splits_k, p.splits_n}, {h, dh}}, stream);
  return e;
}

cudaError_t launch_lora_grad_outer(const LoraPlan& p, const LoraDev& L, const uint16_t* X, const uint16_t* dY,
                                   const int32_t* ids, float* dA, float* dB, float* delta, void* ws,
                                   cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  const LoraGroups G = groups_at(w + p.off_groups, p.positions, L.n, p.max_tiles);
  uint16_t* h = reinterpret_cast<uint16_t*>(w + p.off_h);
  uint16_t* dh = reinterpret_cast<uint16_t*>(w + p.off_dh);
  cudaError_t e = outer(p, L, G, dY, h, dB, X, dh, dA, delta != nullptr, stream);
  if (e == cudaSuccess && delta != nullptr) e = expand<true, false>(p, L, G, ids, nullptr, dh, delta, stream);
  return e;
}

}  // namespace ansdev

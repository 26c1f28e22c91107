// operand.cu -- decodes a range of a compressed layer into 16-bit operand
// images in global memory (the layout of operand.h).
//
// The fused GEMM hands each decoded slab to the tensor core and forgets it.
// An operator that meets the same weights more than once (the logits of a
// piece of the vocabulary and then their gradient; every token block of a
// transposed product) decodes them here once and reads the images.
//
// One warp streams one contiguous run of tiles (RunPipe) and writes each
// 128 x 16 slab into its 4 KB slot, which leaves by one contiguous 4 KB bulk copy
// (a second slot a warp changed nothing: 114.2 against 113.6 us for a call on a
// bf16 14336 x 4096 layer).  One CTA an SM.  What bounds it is how far the
// decoders' instructions fill the issue slots (57 % with 17 warps) and how evenly
// tiles go into warps, a tile being one warp's.  A round of tiles takes about
// 11.8 us and 1.05 us for each warp of the SM (8,192-symbol tiles), so few rounds
// of many warps are best: a CTA has as many, up to the 25 that shared memory
// holds, as bring the tiles out in whole rounds.  That layer's 7,168 tiles: 16
// warps, four rounds for 3.03 of work, 114 us; 17 in three rounds 100 us; 25 in
// two 90 us.  Kernels that do not need the weights are launched beside this one and
// run where its CTAs leave room or have ended (13 warps, to leave them more,
// cost more than it gave: a gradient of adapters on 14336 x 4096 int4 329.5 us
// against 321.7).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <type_traits>

#include "gemm_common.cuh"
#include "launch.h"
#include "operand.h"
#include "rans_core.cuh"

namespace ansdev {

constexpr uint32_t kOpWarps = 25;  // at most
constexpr uint32_t kOpThreads = kOpWarps * 32;
constexpr uint32_t kOpRawAhead = 3;  // raw-byte groups loaded ahead of their use
// [slots 4 KB a warp][rings 4,224 B a warp][slot table 16 KB][barriers 4 x 8 B a warp]
__host__ __device__ constexpr uint32_t op_off_ring(uint32_t warps) { return warps * kSlabBytes; }
__host__ __device__ constexpr uint32_t op_off_lut(uint32_t warps) { return op_off_ring(warps) + warps * kRingStride; }
__host__ __device__ constexpr uint32_t op_off_bars(uint32_t warps) { return op_off_lut(warps) + kSlots * 4; }
__host__ __device__ constexpr uint32_t op_smem(uint32_t warps) { return op_off_bars(warps) + warps * 4 * 8; }

struct OperandDev {
  LayerDev L;
  const uint16_t* group_scales;  // bf16 N x n_groups, or null: 1
  uint32_t group_k, n_groups;
  uint32_t tile0, n_tiles;       // the range's tiles
  uint32_t block0;               // its first 128-row block
  uint8_t* images;
  uint32_t step;                 // bytes from an image to the next
  uint32_t beside;               // does not wait for the kernel before it
  uint32_t* status;
};

// e2m1 codes as exact f16: the magnitudes' low bytes are all zero, so one
// byte permute looks both high bytes up; bit 3 of a code is the sign.
__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t c0, uint32_t c1) {
  const uint32_t sel = (c0 & 7u) | ((c1 & 7u) << 4);
  const uint32_t hi = __byte_perm(0x3E3C3800u, 0x46444240u, sel);
  return __byte_perm(hi, 0u, 0x1404u) | ((c0 & 8u) << 12) | ((c1 & 8u) << 28);
}

template <uint32_t DT>
constexpr bool is_pair_symbols = DT == kDtInt4Pairs || DT == kDtFp4Pairs;

// One group's symbols as 16-bit operand values: 8 columns of a row, or 16 for
// pair symbols.
template <uint32_t DT, uint32_t kOut>
__device__ __forceinline__ void operand_values(const uint32_t (&e)[8], uint64_t raw8, __half2 scale,
                                               uint32_t (&o)[kOut]) {
  if constexpr (DT == kDtBf16Split) fmt_bf16_split(e, raw8, o);
  else if constexpr (DT == kDtInt4) fmt_int4_f16_scaled(e, scale, o);
  else if constexpr (DT == kDtInt4Pairs) fmt_int4pair_f16_scaled(e, scale, o);
  else if constexpr (DT == kDtInt8) fmt_int8_f16(e, o);
  else if constexpr (DT == kDtFp8) fmt_fp8_f16(e, o);
  else if constexpr (DT == kDtFp4) {
#pragma unroll
    for (int p = 0; p < 4; ++p) o[p] = e2m1x2_f16x2((e[2 * p] >> 12) & 0xFu, (e[2 * p + 1] >> 12) & 0xFu);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = e2m1x2_f16x2((e[k] >> 12) & 0xFu, (e[k] >> 16) & 0xFu);
  }
}

__device__ __forceinline__ void sts_quad(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

template <uint32_t DT, bool kWide>
__global__ void __launch_bounds__(kOpThreads, 1) operand_decode_kernel(const __grid_constant__ OperandDev P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint32_t abort_flag;
  constexpr bool kPair = is_pair_symbols<DT>;
  constexpr bool kInt4 = DT == kDtInt4 || DT == kDtInt4Pairs;
  constexpr uint32_t kGroups = kPair ? 4 : 8, kOut = kPair ? 8 : 4;
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const LayerDev& L = P.L;
  const uint32_t cta_warps = blockDim.x / 32;
  uint32_t* lut = reinterpret_cast<uint32_t*>(smem + op_off_lut(cta_warps));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + op_off_bars(cta_warps));
  const bool single = L.single_symbol != kNoSymbol;

  if (threadIdx.x == 0) abort_flag = 0;
  for (uint32_t i = threadIdx.x; i < cta_warps * 4; i += blockDim.x) {
    mbar_init(&bars[i], 1);
    fence_mbar_init();
  }
  if (!single) build_lut(lut, L, warp, cta_warps, lane);
  __syncthreads();
  // the prologue above read only kernel parameters
  if (P.beside == 0) griddep_wait();
  griddep_launch_dependents();

  volatile uint32_t* abort = &abort_flag;
  // warp-major over the CTAs, so that few tiles spread over all of them
  const uint32_t n_warps = gridDim.x * cta_warps, me = warp * gridDim.x + blockIdx.x;
  const uint32_t t_begin = P.tile0 + cta_begin(P.n_tiles, n_warps, me);
  const uint32_t t_end = P.tile0 + cta_begin(P.n_tiles, n_warps, me + 1);
  const uint32_t n_kt = L.n_kt, H = L.tile_n / 128, C = L.tile_k / 16, S = L.tile_n * L.tile_k;
  const uint32_t k_slabs = L.K / 16;
  const uint32_t lt = lanemask_lt(), lut_s = smem_u32(lut);
  const uint32_t swz = ((lane >> 2) & 1u) << 4;
  const uint32_t w_s = smem_u32(smem + warp * kSlabBytes);
  RunPipe pipe;
  rp_init(pipe, smem + op_off_ring(cta_warps) + warp * kRingStride, bars + 4 * warp);
  TileCursor tc;
  tc.x = tc.pos = tc.cb = tc.bytes = 0;
  tc.xw = 0;

  bool run_ok = false;
  uint64_t run_start = 0, a_next = 0;
  uint32_t run_bytes = 0, base = 0;
  if (t_begin < t_end) {
    run_ok = run_extent(L, t_begin, t_end - 1, &run_start, &run_bytes);
    if (run_ok) {
      base = rp_run_begin(pipe, L.stream + run_start, run_bytes);
      rp_prefetch(pipe, base, lane, abort, P.status);
    }
    a_next = run_start;
  }
  // raw sign/mantissa bytes (bf16): the next groups' in flight; a run's tiles
  // are consecutive, so the loads run on into the next tile
  const uint32_t groups = S / 256;
  uint64_t rq[kOpRawAhead];
#pragma unroll
  for (uint32_t k = 0; k < kOpRawAhead; ++k) rq[k] = 0;
  bool rq_ready = false;

  for (uint32_t t = t_begin; t < t_end; ++t) {
    const uint32_t rb = t / n_kt, kt = t - rb * n_kt;
    bool zero_tile = !run_ok;
    if (run_ok) {
      const uint64_t a = a_next, b = __ldg(reinterpret_cast<const unsigned long long*>(L.offsets) + t + 1);
      a_next = b;
      if (!run_tile_begin(pipe, L, a, b, run_start, base, tc, lane, abort, P.status)) {
        run_ok = false;
        zero_tile = true;
      }
    }
    if (zero_tile && lane == 0) atomicOr(P.status, kStatusBadOffsets);
    __half2 gscale[8];
    if constexpr (kInt4) {
#pragma unroll
      for (uint32_t q = 0; q < 8; ++q) {
        float sv = 1.0f;
        if (P.group_scales != nullptr && q / 4 < H) {
          const uint32_t row = rb * L.tile_n + lane + 32 * q;
          sv = bf16_to_f32(__ldg(P.group_scales + static_cast<uint64_t>(row) * P.n_groups +
                                 kt * L.tile_k / P.group_k));
        }
        gscale[q] = __float2half2_rn(sv);
      }
    }
    const unsigned long long* raw_tile = nullptr;
    const uint32_t raw_lim = (t + 1 < t_end) ? groups + kOpRawAhead : groups;
    if constexpr (DT == kDtBf16Split) {
      if (!zero_tile) {
        raw_tile = reinterpret_cast<const unsigned long long*>(L.raw + static_cast<uint64_t>(t) * S) + lane;
        if (!rq_ready) {
#pragma unroll
          for (uint32_t k = 0; k < kOpRawAhead; ++k) rq[k] = __ldcs(raw_tile + 32 * k);
        }
      }
    }
    const uint32_t const_e = zero_tile ? 0u : (single ? L.single_symbol << 12 : 0u);
    // a tile of constant symbols (a single-symbol codebook, or zeros for a
    // tile with bad offsets) takes its own instantiation, so that the decoding
    // path carries no branch for it
    auto slabs = [&](auto const_sym) {
      constexpr bool kConst = decltype(const_sym)::value;
      for (uint32_t us = 0; us < H * C; ++us) {
        const uint32_t h = us % H, s = us / H;
        uint32_t o_prev[kOut];
#pragma unroll
        for (uint32_t k = 0; k < kOut; ++k) o_prev[k] = 0;
        // the store of a group is deferred into the next group's decode chain
        auto store_prev = [&](uint32_t gg) {
          if (gg == 1) {
            // the previous slab's copy has read the slot
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
          }
          const uint32_t row_s = w_s + (32 * ((gg - 1) & 3) + lane) * 32;
          if constexpr (kPair) {
            sts_quad(row_s + swz, o_prev[0], o_prev[1], o_prev[2], o_prev[3]);
            sts_quad(row_s + (16u ^ swz), o_prev[4], o_prev[5], o_prev[6], o_prev[7]);
          } else {
            sts_quad(row_s + ((((gg - 1) >> 2) << 4) ^ swz), o_prev[0], o_prev[1], o_prev[2], o_prev[3]);
          }
        };
#pragma unroll
        for (uint32_t gg = 0; gg < kGroups; ++gg) {
          [[maybe_unused]] const uint32_t g = us * 8 + gg;
          [[maybe_unused]] const uint64_t raw8 = rq[0];
          if constexpr (DT == kDtBf16Split) {
            if (!kConst || !zero_tile) {
#pragma unroll
              for (uint32_t k = 0; k + 1 < kOpRawAhead; ++k) rq[k] = rq[k + 1];
              if (g + kOpRawAhead < raw_lim) rq[kOpRawAhead - 1] = __ldcs(raw_tile + 32 * (g + kOpRawAhead));
            }
          }
          uint32_t e[8], o[kOut];
          if constexpr (kConst) {
#pragma unroll
            for (int k = 0; k < 8; ++k) e[k] = const_e;
            if (gg > 0) store_prev(gg);
          } else {
            rp_group(pipe, tc.pos, lane, abort, P.status);
            if constexpr (kWide) {
              decode_pair(tc.xw, tc.pos, lut_s, pipe.ring_s, lt, e[0], e[1]);
              if (gg > 0) store_prev(gg);
#pragma unroll
              for (int k = 2; k < 8; k += 2) decode_pair(tc.xw, tc.pos, lut_s, pipe.ring_s, lt, e[k], e[k + 1]);
            } else {
              e[0] = decode_step(tc.x, tc.pos, lut_s, pipe.ring_s, lt);
              if (gg > 0) store_prev(gg);
#pragma unroll
              for (int k = 1; k < 8; ++k) e[k] = decode_step(tc.x, tc.pos, lut_s, pipe.ring_s, lt);
            }
          }
          __half2 gs = __float2half2_rn(1.0f);
          if constexpr (kInt4) gs = h ? gscale[4 + (gg & 3)] : gscale[gg & 3];
          operand_values<DT>(e, raw8, gs, o);
#pragma unroll
          for (uint32_t k = 0; k < kOut; ++k) o_prev[k] = (kConst && zero_tile) ? 0u : o[k];
        }
        store_prev(kGroups);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
          bulk_s2g_s(P.images + (static_cast<uint64_t>(rb * H + h - P.block0) * k_slabs + kt * C + s) * P.step,
                     w_s, kSlabBytes);
      }
    };
    if (zero_tile || single) slabs(std::true_type{});
    else slabs(std::false_type{});
    rq_ready = DT == kDtBf16Split && !zero_tile && t + 1 < t_end;
    if (!zero_tile && !run_tile_end(L, tc, single) && lane == 0) atomicOr(P.status, kStatusCorrupt);
  }
  rp_drain(pipe, P.status);
  if (lane == 0) bulk_wait_all();
  if (P.beside != 0) griddep_beside_end();
}

template <uint32_t DT, bool kWide>
static cudaError_t launch_variant(const OperandDev& P, uint32_t grid, uint32_t warps, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(attr_set.load() & (1ull << dev))) {
    e = cudaFuncSetAttribute(operand_decode_kernel<DT, kWide>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             op_smem(kOpWarps));
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set.fetch_or(1ull << dev);
  }
  return launch_pdl(operand_decode_kernel<DT, kWide>, dim3(grid), dim3(warps * 32), op_smem(warps), stream, P);
}

uint32_t operand_decode_rounds(uint32_t tiles, uint32_t ctas) {
  return (tiles + ctas * kOpWarps - 1) / (ctas * kOpWarps);
}

cudaError_t launch_operand_decode(const LayerDev& L, uint32_t row0, uint32_t rows, uint32_t scale_kind,
                                  const void* scales, uint32_t group_k, uint8_t* images,
                                  uint32_t* status, int sms, cudaStream_t stream, uint32_t step,
                                  bool beside) {
  if (rows == 0) return cudaSuccess;
  OperandDev P;
  std::memset(&P, 0, sizeof(P));
  P.L = L;
  if (scale_kind == 3) {
    P.group_scales = static_cast<const uint16_t*>(scales);
    P.group_k = group_k;
    P.n_groups = L.K / group_k;
  }
  P.tile0 = row0 / L.tile_n * L.n_kt;
  P.n_tiles = rows / L.tile_n * L.n_kt;
  P.block0 = row0 / 128;
  P.images = images;
  P.step = step;
  P.beside = beside ? 1u : 0u;
  P.status = status;
  // one CTA an SM (with fewer tiles than that, one tile a CTA), and the fewest
  // warps that need no more rounds of tiles than the most warps would
  const uint32_t cap = static_cast<uint32_t>(sms), grid = P.n_tiles < cap ? P.n_tiles : cap;
  const uint32_t rounds = operand_decode_rounds(P.n_tiles, grid);
  // (8 at least: they build the slot table together, which takes one warp 20 us)
  const uint32_t warps = std::max(8u, (P.n_tiles + grid * rounds - 1) / (grid * rounds));
  switch (L.dtype) {
#define ANS_OPERAND_CASE(DT) \
  case DT: return L.wide ? launch_variant<DT, true>(P, grid, warps, stream) : launch_variant<DT, false>(P, grid, warps, stream);
    ANS_OPERAND_CASE(kDtInt4)
    ANS_OPERAND_CASE(kDtBf16Split)
    ANS_OPERAND_CASE(kDtFp8)
    ANS_OPERAND_CASE(kDtInt4Pairs)
    ANS_OPERAND_CASE(kDtInt8)
    ANS_OPERAND_CASE(kDtFp4)
    ANS_OPERAND_CASE(kDtFp4Pairs)
#undef ANS_OPERAND_CASE
  }
  return cudaErrorInvalidValue;
}

cudaError_t set_live_wait_budget_operand(long long cycles) {
  return cudaMemcpyToSymbol(g_live_wait_budget, &cycles, sizeof(cycles));
}

}  // namespace ansdev

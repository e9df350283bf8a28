// Gradient of an LLM.int8() projection's input, through the frozen int8
// weight, on the tensor cores:
//
//   dX[i][k] = fp16(base[i][k] + sum_j dY[i][j] * WR[k][j])
//   WR[k][j] = fp16(wq[j][k] * (aw[j] / 127))
//
// M = rows of dY, N = h, reduction over o. dY [s][o] is K-major as it lies.
// wq [o][h] has the reduction index outside: its tiles are an MN-major
// operand, so nothing is transposed; each int8 tile is turned into fp16 on
// its way into shared memory.
//
// The weight is rounded to fp16, as in the layer's outlier rows, because one
// fp16 operand holds no more of a code times its factor: results are 2.9e-4 off
// (rms, relative) instead of the 2.1e-4 of their own rounding to fp16. Splitting
// it, or dY times the factor, into two numbers would double the MMAs, which are
// the bound. The fp32 sums stay in their accumulators over a part's whole
// reduction; the tensor cores round them toward zero at every MMA of 16
// products: they end 1.5e-6 of their size too small after 4096 products of
// either sign, 3.0e-6 after 20480, 5.7e-6 after 49152, 1.5e-5 after 262144
// (products of one sign: 5.6e-6, 1.8e-5, 3.4e-5, 9.3e-5), which a rounding to
// fp16 outweighs; k_shrink and k_outer, whose results are fp32, change
// accumulators for that reason.
//
// Bound: the fp16 tensor cores (2 s h o operations) and, back to back, the
// power cap at prefill sizes (4096 x 5120 x 20480: 670 us in a burst, 800 us
// under the cap; 596 us in a burst with the conversion switched off). A pair of
// CTAs computes a tile of MT x 256 rows by 256 columns (tcgen05
// cta_group::2), so that per stage of 64 reduction indices a CTA stores and
// reads only half of each operand: the converted weight costs shared memory no
// more than a plain fp16 one would, and its global traffic is half. With MT = 2
// (more than 256 rows) a converted tile serves two MMAs: half the conversions,
// 772 -> 679 us. Two groups of eight warps convert alternate stages: TMA brings
// the codes and their column scales into a ring of their own, a lane takes 16
// codes of it and writes 16 fp16 values through the 128-byte swizzle, 11
// instructions for four codes. Their signal to the issuing CTA releases, at
// cluster scope, what they wrote to shared memory and nothing else
// (mbar_arrive_smem): a release of all memory waits for a round trip to L2 in
// every stage (1238 us instead of 777 with MT = 1), and even if single threads
// pass the stages on for the others, the way is longer by it (131 x 4096 x 4096
// 24.4 us instead of 22.5, 250 x 5120 x 20480 74 to 108 instead of 72).
//
//   warp 0      TMA producer of dY
//   warp 1      one thread of rank 0 issues the MMAs
//   warp 2      allocates TMEM (two 256-column accumulators); TMA producer of
//               the codes
//   warps 4-7   epilogue: TMEM -> + base -> fp16
//   warps 8-23  converters
//
// Tiles that do not fill a round of all pairs (the last ones, or all of a
// small problem) are cut along o into equal parts, each of which leaves an
// fp32 tile in the workspace; k_input_grad_sum adds them in order.
//
// Every wait is bounded; a role that gives up records a status bit, and the
// CTA drains what it started and returns.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_fp16.h>

#include "ptx_finetune_sm100.cuh"
#include "rows_common.cuh"

namespace llmint8 {
namespace igrad {

constexpr int BM = 128;   // rows per CTA and MMA (256 per pair)
constexpr int BN = 256;   // columns of h per pair
constexpr int BNH = 128;  // columns whose weight this CTA converts
constexpr int BK = 64;    // reduction indices per stage
constexpr int UMMA_K = 16;
constexpr uint32_t TMEM_COLS = 512;  // two accumulators
constexpr uint32_t A_TILE_BYTES = BM * BK * 2;
constexpr uint32_t B_STAGE_BYTES = BNH * BK * 2;
constexpr uint32_t B_BLOCK_BYTES = 64 * BK * 2;  // 64 columns x 64 reduction rows
constexpr int EPI_WARP0 = 4, EPI_THREADS = 128;
constexpr int CVT_WARP0 = 8, CVT_WARPS = 8, CVT_THREADS = 32 * CVT_WARPS;
constexpr int CVT_GROUPS = 2;
constexpr int NUM_THREADS = 32 * (CVT_WARP0 + CVT_GROUPS * CVT_WARPS);
constexpr uint32_t FULL_ARRIVALS = 1 + 2 * CVT_WARPS;
constexpr uint32_t RAW_BYTES = BNH * BK;                    // codes of a stage
constexpr uint32_t RAW_STAGE_BYTES = RAW_BYTES + 4 * BK;    // + its column scales
constexpr int MAX_PAIRS = 74;
constexpr int MAX_PARTS = 2 * MAX_PAIRS;  // units that leave fp32 tiles
constexpr size_t PART_ELEMS = 2 * BM * BN;  // of each 256 rows of such a unit

// Shared memory by rows per unit (MT times 256): the stages of dY and of the
// converted weight, the codes, barriers.
template <int MT>
struct Smem {
  static constexpr int STAGES = MT == 1 ? 5 : 4;
  static constexpr int RAW_STAGES = STAGES;  // stages of int8 codes in flight
  static constexpr uint32_t A_STAGE = MT * A_TILE_BYTES;
  static constexpr uint32_t B_OFF = STAGES * A_STAGE;
  static constexpr uint32_t RAW_OFF = B_OFF + STAGES * B_STAGE_BYTES;
  static constexpr uint32_t BAR_OFF = RAW_OFF + RAW_STAGES * RAW_STAGE_BYTES;
  static constexpr size_t BYTES = 1024 + BAR_OFF + 256;
};

static_assert(Smem<1>::BYTES <= 232448 && Smem<2>::BYTES <= 232448, "shared memory per CTA");
static_assert(Smem<1>::RAW_STAGES >= Smem<1>::STAGES && Smem<2>::RAW_STAGES >= Smem<2>::STAGES,
              "see the converters' waits");
static_assert((4 * Smem<1>::STAGES + 5) * 8 + 8 <= 256, "barrier block size");

// How the tiles are shared out: the first `whole` ones are computed whole,
// each of the other `rest` in `parts` parts along the reduction.
struct Plan {
  int32_t mt;                   // 256-row blocks of a tile: 1 or 2
  int32_t num_m, num_n, num_k;  // tiles of mt * 256 rows, of 256 columns, stages
  int32_t whole, rest, parts;
};

struct Params {
  int32_t s, h, o;
  Plan plan;
  const int8_t *wq;   // [o][h]
  const float *aw;    // [o]
  const __half *base; // [s][h] or null
  __half *out;        // [s][h]
  float *part;        // [rest * parts][mt * 256][256], in part_quad's order
  int32_t *status;
  uint64_t timeout_ns;
};

// Where four columns (4 q ...) of a row of the fp32 tiles lie, in float4s: the
// 32 rows of an epilogue warp next to each other, so that its stores, and the
// loads of k_input_grad_sum, are whole lines (row after row of 1 KB, a warp's
// store touched 32 of them: 22.3 us instead of 20.5 for 131 x 4096 x 4096).
__device__ __forceinline__ size_t part_quad(size_t row, int q) {
  return (row / 32 * (BN / 4) + q) * 32 + row % 32;
}

// One piece of work: a tile and a range of its stages.
struct Unit {
  int32_t m, n, k0, k1;
  int32_t slot;  // fp32 tile it leaves, or -1 for a whole tile
  int32_t blocks;  // its 256-row blocks that have rows
};

__device__ __forceinline__ bool unit_at(const Params &p, int32_t idx, Unit &u) {
  const Plan &pl = p.plan;
  int32_t tile;
  if (idx < pl.whole) {
    tile = idx;
    u.k0 = 0;
    u.k1 = pl.num_k;
    u.slot = -1;
  } else {
    const int32_t t = idx - pl.whole;
    if (t >= pl.rest * pl.parts) return false;
    const int32_t part = t / pl.rest;
    tile = pl.whole + t % pl.rest;
    u.k0 = (int32_t)((int64_t)pl.num_k * part / pl.parts);
    u.k1 = (int32_t)((int64_t)pl.num_k * (part + 1) / pl.parts);
    u.slot = pl.parts > 1 ? t : -1;
  }
  u.m = tile % pl.num_m;
  u.n = tile / pl.num_m;
  u.blocks = min(pl.mt, (p.s - u.m * pl.mt * 2 * BM + 2 * BM - 1) / (2 * BM));
  return true;
}

// A row's factor f = aw / 127 in the form the conversion uses, all exact but
// for lo's last bit: f = (hi + lo) * p2 with p2 a power of two, as fp16 pairs.
// hi + lo lies in [2^-6, 2^-5) (lower only for the two smallest binary16
// values of aw), so a code times it and, for every binary16 aw, p2 stay in
// range; lo's error is below 2^-18 of f.
struct Factor {
  __half2 hi, lo, p2;
};

__device__ __forceinline__ Factor factor_of(float aw) {
  const float f = aw * (1.0f / 127.0f);
  const int e = max((int)((__float_as_uint(f) >> 23) & 0xff) - 127 + 6, -24);
  const float m = f * __uint_as_float((uint32_t)(127 - e) << 23);
  Factor r;
  const __half hi = __float2half_rn(m);
  r.hi = __half2half2(hi);
  r.lo = __float2half2_rn(m - __half2float(hi));
  r.p2 = __float2half2_rn(__uint_as_float((uint32_t)(127 + e) << 23));
  return r;
}

// Two int8 codes q (given as q + 128 in the low bytes of fp16 numbers
// 1024 + (q + 128)) times the factor. The subtraction is exact; q * (hi + lo)
// is rounded once to fp16 (its q * lo term to 2^-22 of it before), and the
// power of two only where the result is subnormal.
__device__ __forceinline__ uint32_t scale_pair(uint32_t h, const Factor &f) {
  const __half2 q = __hadd2(*reinterpret_cast<const __half2 *>(&h), __float2half2_rn(-1152.0f));
  const __half2 v = __hmul2(__hfma2(q, f.hi, __hmul2(q, f.lo)), f.p2);
  return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint2 codes_to_half(uint32_t w, const Factor &f) {
  const uint32_t x = w ^ 0x80808080u;
  return make_uint2(scale_pair(prmt(x, 0x64646464u, 0x4140), f),
                    scale_pair(prmt(x, 0x64646464u, 0x4342), f));
}

// Item i of lane j of every four lanes becomes item j of lane i.
__device__ __forceinline__ void quad_transpose(uint4 (&t)[4], int lane) {
#pragma unroll
  for (int bit = 1; bit < 4; bit *= 2) {
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int lo = 0; lo < 4; ++lo) {
      if (lo & bit) continue;
      uint4 &a = t[lo], &b = t[lo + bit];
      uint4 m = up ? a : b;
      m.x = __shfl_xor_sync(0xffffffffu, m.x, bit);
      m.y = __shfl_xor_sync(0xffffffffu, m.y, bit);
      m.z = __shfl_xor_sync(0xffffffffu, m.z, bit);
      m.w = __shfl_xor_sync(0xffffffffu, m.w, bit);
      a = up ? m : a;
      b = up ? b : m;
    }
  }
}

// BASE: whether another gradient is added (p.base; its registers would cost the
// kernel without one spills).
template <int MT, bool BASE>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    k_input_grad(const __grid_constant__ CUtensorMap tmA,
                 const __grid_constant__ CUtensorMap tmW, const Params p) {
  using L = Smem<MT>;
  constexpr int STAGES = L::STAGES, RAW_STAGES = L::RAW_STAGES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  uint8_t *base = smem_raw + pad;
  const uint32_t sA = smem_u32(base);
  const uint32_t sB = sA + L::B_OFF;
  uint64_t *bars = reinterpret_cast<uint64_t *>(base + L::BAR_OFF);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int st) { return bar0 + 8u * st; };
  auto empty_bar = [&](int st) { return bar0 + 8u * (STAGES + st); };
  auto raw_full_bar = [&](int st) { return bar0 + 8u * (2 * STAGES + st); };
  auto raw_empty_bar = [&](int st) { return bar0 + 8u * (2 * STAGES + RAW_STAGES + st); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 * RAW_STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 * RAW_STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 2 * RAW_STAGES + 4);
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 2 * STAGES + 2 * RAW_STAGES + 5);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(full_bar(i), FULL_ARRIVALS);
      mbar_init(empty_bar(i), 1);
    }
    for (int i = 0; i < RAW_STAGES; ++i) {
      mbar_init(raw_full_bar(i), 1);
      mbar_init(raw_empty_bar(i), CVT_WARPS);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 2 * EPI_THREADS);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 2) {
    tmem_alloc_pair(smem_u32(tmem_holder), TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before either signals the other's
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  grid_dependency_wait();

  // accumulator of block b of the pair's it-th unit: with one block per unit
  // the two alternate between units, with two each block has its own
  auto acc_of = [](int32_t it, int b) { return MT == 1 ? (it & 1) : b; };
  auto acc_use = [](int32_t it) { return (uint32_t)(MT == 1 ? it >> 1 : it) & 1u; };
  const int32_t pair = (int32_t)blockIdx.x >> 1, npairs = (int32_t)gridDim.x >> 1;
  Unit u;
  if (warp == 0 && lane == 0) {
    // ------------------------------------------------- TMA producer (dY)
    uint32_t stage = 0, phase = 0;
    bool ok = true, issued = false;
    for (int32_t idx = pair; ok && unit_at(p, idx, u); idx += npairs) {
      const int32_t row = u.m * (MT * 2 * BM) + (int32_t)rank * BM;
      for (int32_t kb = u.k0; kb < u.k1; ++kb) {
        if (!mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.status,
                               LLMINT8_DEV_TIMEOUT_PRODUCER, p.timeout_ns)) {
          ok = false;
          break;
        }
        if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), u.blocks * 2 * A_TILE_BYTES);
        for (int b = 0; b < u.blocks; ++b)
          tma_load_2d_pair(sA + stage * L::A_STAGE + b * A_TILE_BYTES, &tmA,
                           mapa_shared(full_bar(stage), 0), kb * BK, row + b * 2 * BM);
        issued = true;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {
      // let every copy this CTA started land before shared memory goes: a
      // phase whose copies came in may still miss converters, so wait a
      // while instead of for the barriers
      const uint64_t t0 = global_timer_ns();
      while (issued && global_timer_ns() - t0 < 200000u) __nanosleep(1000);
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc = idesc_f16_f32_mn(2 * BM, BN, false, true);
    uint32_t stage = 0, phase = 0;
    bool ok = true, any = false;
    int32_t it = 0;
    for (int32_t idx = pair; ok && unit_at(p, idx, u); idx += npairs, ++it) {
      for (int32_t kb = u.k0; ok && kb < u.k1; ++kb) {
        if (!mbar_wait_bounded_cluster(full_bar(stage), phase, abort_flag, p.status,
                                       LLMINT8_DEV_TIMEOUT_MMA, p.timeout_ns)) {
          ok = false;
          break;
        }
        const uint64_t b_desc = smem_desc_mn_sw128(sB + stage * B_STAGE_BYTES, B_BLOCK_BYTES);
        for (int b = 0; b < u.blocks; ++b) {
          const int acc = acc_of(it, b);
          if (kb == u.k0 &&
              !mbar_wait_bounded_cluster(tempty_bar(acc), acc_use(it) ^ 1u, abort_flag, p.status,
                                         LLMINT8_DEV_TIMEOUT_MMA, p.timeout_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t a_desc =
              smem_desc_kmajor_sw128(sA + stage * L::A_STAGE + b * A_TILE_BYTES);
#pragma unroll
          for (int k = 0; k < BK / UMMA_K; ++k)
            mma_f16_pair(tmem_base + acc * BN, a_desc + (uint64_t)((k * UMMA_K * 2) >> 4),
                         b_desc + (uint64_t)((k * UMMA_K * 128) >> 4), idesc,
                         (kb > u.k0 || k > 0) ? 1u : 0u);
          any = true;
        }
        if (!ok) break;
        mma_commit_pair(mapa_shared(empty_bar(stage), 0));
        mma_commit_pair(mapa_shared(empty_bar(stage), 1));
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      // (a block without rows passes its accumulator on unused)
      for (int b = 0; b < MT; ++b) {
        if (b >= u.blocks &&
            !mbar_wait_bounded_cluster(tempty_bar(acc_of(it, b)), acc_use(it) ^ 1u, abort_flag,
                                       p.status, LLMINT8_DEV_TIMEOUT_MMA, p.timeout_ns)) {
          ok = false;
          break;
        }
        mma_commit_pair(mapa_shared(tfull_bar(acc_of(it, b)), 0));
        mma_commit_pair(mapa_shared(tfull_bar(acc_of(it, b)), 1));
      }
    }
    if (!ok && any) {
      volatile int never = 0;
      mma_commit_pair(mapa_shared(drain_bar, 0));
      mbar_wait_bounded(drain_bar, 0, &never, p.status, LLMINT8_DEV_TIMEOUT_DRAIN, p.timeout_ns);
    }
  } else if (warp == 2 && lane == 0) {
    // ------------------------- TMA producer of the codes and their scales
    uint32_t stage = 0, phase = 0, issued = 0, last_par = 0;
    bool ok = true;
    for (int32_t idx = pair; ok && unit_at(p, idx, u); idx += npairs) {
      const int32_t col = u.n * BN + (int32_t)rank * BNH;
      for (int32_t kb = u.k0; kb < u.k1; ++kb) {
        if (!mbar_wait_bounded(raw_empty_bar(stage), phase ^ 1u, abort_flag, p.status,
                               LLMINT8_DEV_TIMEOUT_PRODUCER, p.timeout_ns)) {
          ok = false;
          break;
        }
        const uint32_t dst = smem_u32(base) + L::RAW_OFF + stage * RAW_STAGE_BYTES;
        const uint32_t scale_bytes = 4u * (uint32_t)min(BK, p.o - kb * BK);  // o % 16 == 0
        mbar_arrive_expect_tx(raw_full_bar(stage), RAW_BYTES + scale_bytes);
        tma_load_2d(dst, &tmW, raw_full_bar(stage), col, kb * BK);
        bulk_load_1d(dst + RAW_BYTES, p.aw + kb * BK, scale_bytes, raw_full_bar(stage));
        issued |= 1u << stage;
        last_par = (last_par & ~(1u << stage)) | (phase << stage);
        if (++stage == RAW_STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {  // let every copy land before shared memory goes
      volatile int never = 0;
      for (int st = 0; st < RAW_STAGES; ++st)
        if ((issued >> st) & 1u)
          mbar_wait_bounded(raw_full_bar(st), (last_par >> st) & 1u, &never, p.status,
                            LLMINT8_DEV_TIMEOUT_DRAIN, p.timeout_ns);
    }
  } else if (warp >= EPI_WARP0 && warp < CVT_WARP0) {
    // --------------------------------------------------------- epilogue
    const int ew = warp & 3;
    int32_t it = 0;
    bool ok = true;
    for (int32_t idx = pair; ok && unit_at(p, idx, u); idx += npairs, ++it) {
      for (int b = 0; b < MT; ++b) {
        const int acc = acc_of(it, b);
        ok = mbar_wait_bounded(tfull_bar(acc), acc_use(it), abort_flag, p.status,
                               LLMINT8_DEV_TIMEOUT_EPILOGUE, p.timeout_ns);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        const uint32_t t_row = tmem_base + ((uint32_t)(ew * 32) << 16) + acc * BN;
        const int in_block = (int)rank * BM + ew * 32 + lane;
        const int32_t row = (u.m * MT + b) * (2 * BM) + in_block;
        if (b < u.blocks) {
          for (int c = 0; c < BN / 32; ++c) {
            const int32_t j0 = u.n * BN + c * 32;
            uint32_t v[32];
            __syncwarp();
            tmem_ld_32x32b_x32(t_row + c * 32, v);
            tmem_ld_wait();
            if (row - lane >= p.s || j0 >= p.h) continue;  // (the whole warp)
            if (u.slot >= 0) {
              if (row >= p.s) continue;
              float4 *dst =
                  reinterpret_cast<float4 *>(p.part) +
                  part_quad(((size_t)u.slot * MT + b) * (2 * BM) + in_block, c * 8);
#pragma unroll
              for (int q = 0; q < 8; ++q)
                dst[q * 32] =
                    make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]),
                                __uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3]));
              continue;
            }
            // h is a multiple of 16: 8 columns are all inside or all outside
            if constexpr (!BASE) {
#pragma unroll
              for (int q8 = 0; q8 < 4; ++q8) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[8 * q8 + e]);
                if (row < p.s && j0 + 8 * q8 < p.h)
                  store8(p.out + (int64_t)row * p.h + j0 + 8 * q8, f);
              }
              continue;
            }
            // with a base to read, four lanes' rows change places with their
            // octets, so that four lanes load and store 64 bytes of one row
            // (4096 rows, 4096 x 1024: 78 us instead of 98; stores alone gain
            // nothing from it)
            const int32_t quad = row - (lane & 3), col = j0 + 8 * (lane & 3);
            uint4 t[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              t[q] = make_uint4(0u, 0u, 0u, 0u);
              if (quad + q < p.s && col < p.h)
                t[q] = *reinterpret_cast<const uint4 *>(p.base + (int64_t)(quad + q) * p.h + col);
            }
            quad_transpose(t, lane);
#pragma unroll
            for (int q8 = 0; q8 < 4; ++q8) {
              Vec8<__half> bv;
              bv.q = t[q8];
              float f[8];
              bv.get(f);
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] += __uint_as_float(v[8 * q8 + e]);
              t[q8] = pack8(f);
            }
            quad_transpose(t, lane);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (quad + q < p.s && col < p.h)
                *reinterpret_cast<uint4 *>(p.out + (int64_t)(quad + q) * p.h + col) = t[q];
          }
        }
        __syncwarp();
        tc_fence_before();
        mbar_arrive_cluster(mapa_shared(tempty_bar(acc), 0));
      }
    }
  } else if (warp >= CVT_WARP0) {
    // ------------------------------------------------------- converters
    // group g takes the pair's stages g, g + CVT_GROUPS, ... in order
    const int group = (warp - CVT_WARP0) / CVT_WARPS;
    const int ct = (threadIdx.x - CVT_WARP0 * 32) % CVT_THREADS;
    // lane: 16 codes (16 of the CTA's columns) of reduction rows r0, r0 + 32
    const int r0 = ct >> 3, c = ct & 7, blk = c >> 2;
    uint32_t stage = group, phase = 0, rstage = group % RAW_STAGES, rphase = 0;
    bool ok = true;
    int32_t skip = group;  // stages of the sequence before this group's next one
    for (int32_t idx = pair; ok && unit_at(p, idx, u); idx += npairs) {
      int32_t kb = u.k0 + skip;
      for (; kb < u.k1; kb += CVT_GROUPS) {
        // the slot's turn first, then its codes: once the stage STAGES before
        // this one has been multiplied, the other group is done with its codes
        // too, so the parity of the codes' barrier is not mistaken for that of
        // their slot's previous use
        ok = mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.status,
                               LLMINT8_DEV_TIMEOUT_PRODUCER, p.timeout_ns) &&
             mbar_wait_bounded(raw_full_bar(rstage), rphase, abort_flag, p.status,
                               LLMINT8_DEV_TIMEOUT_PRODUCER, p.timeout_ns);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const uint8_t *src = base + L::RAW_OFF + rstage * RAW_STAGE_BYTES;
        uint4 raw[2];
        float sc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int kr = r0 + 32 * i;
          raw[i] = *reinterpret_cast<const uint4 *>(src + kr * 128 + c * 16);
          const float aw = *reinterpret_cast<const float *>(src + RAW_BYTES + 4 * kr);
          sc[i] = kb * BK + kr < p.o ? aw : 0.0f;
        }
        uint8_t *dst = base + L::B_OFF + stage * B_STAGE_BYTES + blk * B_BLOCK_BYTES;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int kr = r0 + 32 * i;
          const Factor f = factor_of(sc[i]);
          // 16-byte chunks 2m and 2m + 1 of the row's 128 bytes; the lanes of
          // the second block write them in the other order, so that a quarter
          // of a warp covers all eight bank groups
          const uint4 w = raw[i];
          const uint2 a = codes_to_half(blk ? w.z : w.x, f), b = codes_to_half(blk ? w.w : w.y, f);
          const uint2 d = codes_to_half(blk ? w.x : w.z, f), e = codes_to_half(blk ? w.y : w.w, f);
          const int m0 = 2 * (c & 3) + blk;
          *reinterpret_cast<uint4 *>(dst + kr * 128 + ((m0 ^ (kr & 7)) << 4)) =
              make_uint4(a.x, a.y, b.x, b.y);
          *reinterpret_cast<uint4 *>(dst + kr * 128 + (((m0 ^ 1) ^ (kr & 7)) << 4)) =
              make_uint4(d.x, d.y, e.x, e.y);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_smem(mapa_shared(full_bar(stage), 0));
          mbar_arrive(raw_empty_bar(rstage));
        }
        stage += CVT_GROUPS;
        if (stage >= STAGES) {
          stage -= STAGES;
          phase ^= 1u;
        }
        rstage += CVT_GROUPS;
        if (rstage >= RAW_STAGES) {
          rstage -= RAW_STAGES;
          rphase ^= 1u;
        }
      }
      skip = kb - u.k1;
    }
  }

  tc_fence_before();
  __syncthreads();
  // neither CTA frees the pair's TMEM, or leaves, while the other may still
  // use its barriers or its accumulator
  cluster_sync();
  tc_fence_after();
  if (warp == 2) tmem_dealloc_pair(tmem_base, TMEM_COLS);
}

// The tiles computed in parts: out = fp16(base + the parts in order). A
// thread holds 8 columns of one row of a tile, a warp those of 32 rows.
constexpr int SUM_THREADS = 256;
__global__ void __launch_bounds__(SUM_THREADS) k_input_grad_sum(const Params p) {
  grid_dependency_wait();
  const int32_t idx = blockIdx.x * SUM_THREADS + threadIdx.x;
  const int32_t per_tile = p.plan.mt * 2 * BM * (BN / 8);
  const int32_t t = idx / per_tile, e = idx % per_tile;
  if (t >= p.plan.rest) return;
  const int32_t tile = p.plan.whole + t;
  const int32_t in_tile = e / (32 * (BN / 8)) * 32 + e % 32;
  const int32_t oct = e / 32 % (BN / 8);
  const int32_t row = (tile % p.plan.num_m) * (p.plan.mt * 2 * BM) + in_tile;
  const int32_t col = (tile / p.plan.num_m) * BN + oct * 8;
  if (row >= p.s || col >= p.h) return;
  float f[8] = {};
  if (p.base) {
    Vec8<__half> b;
    b.load(p.base + (int64_t)row * p.h + col);
    b.get(f);
  }
  float acc[8] = {};
#pragma unroll 4
  for (int32_t part = 0; part < p.plan.parts; ++part) {
    const float4 *src =
        reinterpret_cast<const float4 *>(p.part) +
        part_quad((size_t)(part * p.plan.rest + t) * p.plan.mt * (2 * BM) + in_tile, oct * 2);
    const float4 a = src[0], b = src[32];
    acc[0] += a.x;
    acc[1] += a.y;
    acc[2] += a.z;
    acc[3] += a.w;
    acc[4] += b.x;
    acc[5] += b.y;
    acc[6] += b.z;
    acc[7] += b.w;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] += acc[k];
  store8(p.out + (int64_t)row * p.h + col, f);
}

}  // namespace igrad
}  // namespace llmint8

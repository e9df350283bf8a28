// The adapters' products on the tensor cores, for batches of more than a few
// rows (formulas: adapters.cuh):
//
//   k_shrink   v = X . F^T over the features: 128 rows per cluster, the
//              features cut over the cluster's CTAs, their partial sums added
//              through distributed shared memory in rank order
//   k_expand   out = base + scale * v . F: 128 rows x 64 features per step; in
//              the backward pass further blocks do k_pack's work
//   k_pack     g or v as the operand of k_outer
//   k_outer    dF = scale * P^T . Q over the rows of one adapter: 256 features
//              per cluster, the blocks of 64 rows cut over its CTAs
//
// All are bound by bytes: at rank r an fp16 feature takes part in 2 r to 4 r
// operations. What they read once (X, dY, base) streams through TMA rings;
// the factors and the s x r arrays stay in L2.
//
// A tile of rows may mix adapters. tile_slots() numbers the distinct ones;
// k_shrink and k_expand multiply the whole tile with each adapter's factor
// into columns (or a step) of its own and keep, per row, its own adapter's,
// so nothing of another adapter or row can reach a row. k_outer sums over
// rows: in a block of rows that is not all one adapter's, the others' rows of
// both operands are zeroed in shared memory.
//
// v, g and the sums are fp32. As tensor-core operands they are split into two
// fp16 numbers (hi + lo, 22 bits) after an exact scaling by a power of two
// that brings the largest of a row (k_expand) or of an adapter's rows
// (k_outer) to [2^14, 2^15), so neither large nor small gradients leave the
// fp16 range. The tensor cores round each accumulation toward zero, a bias
// that grows with the number of MMAs into one accumulator (1.3e-6 of the
// result, rms, after 52 of them; 0.4e-6 after 16); so k_shrink and k_outer
// move on to a fresh one every 16 and add them up in fp32.
//
// Every wait is bounded, as in the GEMMs: a role that gives up sets a status
// bit, the others follow, copies in flight land, TMEM is freed.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_fp16.h>

#include "adapters.cuh"
#include "ptx_finetune_sm100.cuh"
#include "rows_common.cuh"

namespace llmint8 {
namespace lora {

constexpr int TM = 128;                      // rows of a tile
constexpr uint32_t SMEM_LIMIT = 232448;

// ------------------------------------------------------------ shared parts

struct TileSlots {
  int32_t id[TM];       // adapter of each row, -1 for none
  int32_t slot[TM];     // number of that adapter within the tile, or -1
  int32_t adapter[TM];  // adapter of each slot, by first row
  int32_t rank[TM];     // terms that adapter uses
  int32_t first[TM];    // slot of the rows that lead one
  int32_t per_warp[4];
  int32_t count;
};

// Whole block (at least TM threads, whole warps).
__device__ __forceinline__ void tile_slots(const int32_t *ids, int64_t row0, int64_t s, int32_t n,
                                           const int32_t *rank, int32_t r, TileSlots &ts) {
  const int t = threadIdx.x, w = t >> 5, lane = t & 31;
  int a = -1, lead = t;
  unsigned leaders = 0;
  if (t < TM) {
    if (row0 + t < s) a = adapter_of(ids, row0 + t, n);
    ts.id[t] = a;
  }
  // one adapter's rows, perhaps with rows without one
  const int32_t one = row0 < s ? adapter_of(ids, row0, n) : -1;
  if (__syncthreads_and(t >= TM || a == one || a < 0)) {
    if (t < TM) ts.slot[t] = a >= 0 ? 0 : -1;
    if (t == 0) {
      ts.adapter[0] = one;
      ts.rank[0] = one >= 0 ? rank_of(rank, one, r) : 0;
      ts.count = one >= 0 ? 1 : 0;
    }
    __syncthreads();
    return;
  }
  if (t < TM) {
    const unsigned same = __match_any_sync(0xffffffffu, a);
    const int head = __ffs(same) - 1;
    lead = (w << 5) + head;
    if (lane == head && a >= 0) {
      for (int j = 0; j < (w << 5); j += 4) {
        const int4 q = *reinterpret_cast<const int4 *>(&ts.id[j]);
        const int hit = q.x == a ? 0 : q.y == a ? 1 : q.z == a ? 2 : q.w == a ? 3 : -1;
        if (hit >= 0) {
          lead = j + hit;
          break;
        }
      }
    }
    __syncwarp();
    lead = __shfl_sync(0xffffffffu, lead, head);
    leaders = __ballot_sync(0xffffffffu, a >= 0 && lead == t);
    if (lane == 0) ts.per_warp[w] = __popc(leaders);
  }
  __syncthreads();
  if (t < TM && a >= 0 && lead == t) {
    int slot = __popc(leaders & ((1u << lane) - 1u));
    for (int i = 0; i < w; ++i) slot += ts.per_warp[i];
    ts.first[t] = slot;
    ts.adapter[slot] = a;
    ts.rank[slot] = rank_of(rank, a, r);
  }
  if (t == 0) ts.count = ts.per_warp[0] + ts.per_warp[1] + ts.per_warp[2] + ts.per_warp[3];
  __syncthreads();
  if (t < TM) ts.slot[t] = a >= 0 ? ts.first[lead] : -1;
  __syncthreads();
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.0f;  // NaN and infinities count as 0
}

// The power of two 2^e that brings `largest` to [2^14, 2^15) as
// largest * 2^-e; 1 for 0. e stays within what fp32 holds.
__device__ __forceinline__ int scale_exponent(float largest) {
  if (!(largest > 0.0f)) return 0;
  const int e = (int)((__float_as_uint(largest) >> 23) & 0xff) - 127 - 14;
  return max(-112, min(112, e));
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Eight fp32 values times `f` as hi + lo fp16 octets.
__device__ __forceinline__ void split8(const float (&x)[8], float f, uint4 &hi, uint4 &lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = x[2 * i] * f, b = x[2 * i + 1] * f;
    const __half2 hh = __floats2half2_rn(a, b);
    const float2 back = __half22float2(hh);
    // an infinity keeps its sign in hi; its lo is not inf - inf
    const __half2 ll = __floats2half2_rn(isinf(back.x) ? 0.0f : a - back.x,
                                         isinf(back.y) ? 0.0f : b - back.y);
    h[i] = *reinterpret_cast<const uint32_t *>(&hh);
    l[i] = *reinterpret_cast<const uint32_t *>(&ll);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Shared by the roles of a CTA.
struct Ctl {
  uint32_t tmem;
  int abort;
};

// ------------------------------------------------------------------ k_shrink

constexpr int SH_THREADS = 256;
constexpr int SH_KB = 64;       // features per stage
constexpr int SH_DRAIN = 4;     // stages (of 4 MMAs) that one accumulator sums
constexpr int SH_MAX_STAGES = 8;
constexpr int SH_MAX_SPLIT = 16;  // clusters past 8 CTAs need the device's leave
constexpr int SH_MAX_ACC = 8;
constexpr uint32_t SH_X_BYTES = TM * SH_KB * 2;

struct ShrinkParams {
  int32_t s, k, n, r;
  int32_t split;        // CTAs of a cluster
  int32_t slots;        // adapters of a pass over the features
  int32_t stages, accs; // accumulators of `cols` TMEM columns
  int32_t cols, tmem_cols;
  uint32_t stage_bytes;
  const int32_t *ids, *rank;
  float *v;             // [s][r]
  float *vmax;          // [s] largest finite |v| of each row
  uint32_t *amax;       // [n] of each adapter's rows (bits; zero before), or null
  const float *w;       // another [s][r] whose adapters' maxima go to w_amax, or null
  uint32_t *w_amax;
  int32_t *status;
  uint64_t timeout_ns;
};

struct ShrinkJob {
  CUtensorMap x, f;  // X [s][k] in 64 x 128 boxes, F [n * r][k] in 64 x r boxes
  ShrinkParams p;
};

// Adapters of a pass: 64 columns' worth, one at least.
__host__ __device__ inline int32_t shrink_slots(int32_t r) { return r < 64 ? 64 / r : 1; }
__host__ __device__ inline int32_t shrink_cols(int32_t r) {
  return (shrink_slots(r) * r + 15) / 16 * 16;
}
__host__ __device__ inline uint32_t shrink_stage_bytes(int32_t r) {
  return SH_X_BYTES + (uint32_t)shrink_cols(r) * 128;
}
// slots, barriers, alignment (the partial sums [TM][r + 1] take the ring's place)
constexpr uint32_t SH_FIXED_BYTES = (uint32_t)sizeof(TileSlots) + 16 + 384 + 1024;
static_assert(SH_X_BYTES * 4 >= TM * (64 + 1) * 4 && SH_X_BYTES * 5 >= TM * (MAX_R + 1) * 4,
              "partial sums in a ring of four or more stages");

// Largest finite |x[t]|, t < r, over a warp.
__device__ __forceinline__ float warp_row_max(const float *x, int r) {
  float m = 0.0f;
  for (int t = threadIdx.x & 31; t < r; t += 32) m = fmaxf(m, finite_abs(x[t]));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}

// Grid: (m tiles * split, y, jobs), clusters of `split` along x. Where the row
// tiles leave SMs free, y clusters share the passes over the adapters of a tile
// of mixed rows (150 rows of 16 adapters, rank 128, 12288 -> 512, the whole
// forward call: 148 us with one cluster per tile, 51 with 9).
// NC: octets of terms that a thread sums in registers (r <= 8 NC).
template <int NC>
__global__ void __launch_bounds__(SH_THREADS, NC <= 8 ? 2 : 1)
    k_shrink(const __grid_constant__ ShrinkJob j0, const __grid_constant__ ShrinkJob j1) {
  const ShrinkJob &job = blockIdx.z == 0 ? j0 : j1;
  const ShrinkParams &p = job.p;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t *base = smem_raw + pad;
  const uint32_t ring = smem_u32(base);
  const int ldp = p.r + 1;
  uint8_t *after = base + p.stages * p.stage_bytes;
  TileSlots &ts = *reinterpret_cast<TileSlots *>(after);
  uint64_t *bars = reinterpret_cast<uint64_t *>(after + (sizeof(TileSlots) + 15) / 16 * 16);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int st) { return bar0 + 8u * st; };
  auto empty_bar = [&](int st) { return bar0 + 8u * (SH_MAX_STAGES + st); };
  auto tfull = [&](int a) { return bar0 + 8u * (2 * SH_MAX_STAGES + a); };
  auto tempty = [&](int a) { return bar0 + 8u * (2 * SH_MAX_STAGES + SH_MAX_ACC + a); };
  const uint32_t drain = bar0 + 8u * (2 * SH_MAX_STAGES + 2 * SH_MAX_ACC);
  Ctl *ctl = reinterpret_cast<Ctl *>(bars + 2 * SH_MAX_STAGES + 2 * SH_MAX_ACC + 1);
  volatile int *abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t cta = p.split > 1 ? cluster_ctarank() : 0;
  const int64_t row0 = (int64_t)(blockIdx.x / p.split) * TM;
  const int32_t nk = (p.k + SH_KB - 1) / SH_KB;
  // this CTA's blocks of features are cta, cta + split, ...: the cluster reads
  // neighbouring parts of a row at a time
  const int32_t blocks = (nk - (int32_t)cta + p.split - 1) / p.split;
  // this cluster's passes over the adapters are blockIdx.y, + gridDim.y, ...
  const int32_t first = (int32_t)blockIdx.y * p.slots, step = (int32_t)gridDim.y * p.slots;
  const int early = first == 0 ? min(p.stages, blocks) : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(full_bar(i), 2);  // X, F
      mbar_init(empty_bar(i), 1);
    }
    for (int a = 0; a < p.accs; ++a) {
      mbar_init(tfull(a), 1);
      mbar_init(tempty(a), TM);
    }
    mbar_init(drain, 1);
    ctl->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&job.x);
    tma_prefetch_desc(&job.f);
    // the first X tiles come in while the rows' adapters are sorted out
    for (int i = 0; i < early; ++i) {
      mbar_arrive_expect_tx(full_bar(i), SH_X_BYTES);
      tma_load_2d(ring + i * p.stage_bytes, &job.x, full_bar(i),
                  ((int32_t)cta + i * p.split) * SH_KB, (int32_t)row0);
    }
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(&ctl->tmem), p.tmem_cols);
    tmem_relinquish();
  }
  grid_dependency_trigger();
  tc_fence_before();
  tile_slots(p.ids, row0, p.s, p.n, p.rank, p.r, ts);  // ends with a barrier
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  float sums[NC * 8];  // epilogue warps: their row's v over this CTA's features
#pragma unroll
  for (int t = 0; t < NC * 8; ++t) sums[t] = 0.0f;

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------ TMA producer
    uint32_t stage = 0, phase = 0, issued = (1u << early) - 1u, last_par = 0;
    bool ok = true;
    int32_t ahead = early;  // stages whose X is under way
    for (int32_t s0 = first; ok && s0 < ts.count; s0 += step) {
      const int32_t ns = min(p.slots, ts.count - s0);
      for (int32_t i = 0; i < blocks; ++i, --ahead) {
        const int32_t kb = (int32_t)cta + i * p.split;
        if (!mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.status,
                               LLMINT8_DEV_TIMEOUT_PRODUCER, p.timeout_ns)) {
          ok = false;
          break;
        }
        const uint32_t dst = ring + stage * p.stage_bytes;
        if (ahead <= 0) {
          mbar_arrive_expect_tx(full_bar(stage), SH_X_BYTES);
          tma_load_2d(dst, &job.x, full_bar(stage), kb * SH_KB, (int32_t)row0);
        }
        mbar_arrive_expect_tx(full_bar(stage), (uint32_t)(ns * p.r) * 128);
        for (int32_t q = 0; q < ns; ++q)
          tma_load_2d(dst + SH_X_BYTES + (uint32_t)(q * p.r) * 128, &job.f, full_bar(stage),
                      kb * SH_KB, ts.adapter[s0 + q] * p.r);
        issued |= 1u << stage;
        last_par = (last_par & ~(1u << stage)) | (phase << stage);
        if ((int)++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok || ts.count == 0) {  // let every copy land before shared memory goes
      volatile int never = 0;
      for (int st = 0; st < p.stages; ++st) {
        if (!((issued >> st) & 1u)) continue;
        // an early X tile that never got its F
        if (ahead > 0 && st >= early - ahead) mbar_arrive(full_bar(st));
        mbar_wait_bounded(full_bar(st), (last_par >> st) & 1u, &never, p.status,
                          LLMINT8_DEV_TIMEOUT_DRAIN, p.timeout_ns);
      }
    }
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------------- MMA issuer
    uint32_t stage = 0, phase = 0, aphase = 0;
    int acc = 0;
    bool ok = true, any = false;
    for (int32_t s0 = first; ok && s0 < ts.count; s0 += step) {
      const uint32_t idesc =
          idesc_f16_f32(TM, (min(p.slots, ts.count - s0) * p.r + 15) / 16 * 16);
      for (int32_t kb = 0; kb < blocks; ++kb) {
        const int32_t i = kb % SH_DRAIN;
        ok = (i > 0 || mbar_wait_bounded(tempty(acc), aphase ^ 1u, abort_flag, p.status,
                                         LLMINT8_DEV_TIMEOUT_MMA, p.timeout_ns)) &&
             mbar_wait_bounded(full_bar(stage), phase, abort_flag, p.status,
                               LLMINT8_DEV_TIMEOUT_MMA, p.timeout_ns);
        if (!ok) break;
        tc_fence_after();
        const uint32_t src = ring + stage * p.stage_bytes;
        const uint64_t a = smem_desc_kmajor_sw128(src);
        const uint64_t b = smem_desc_kmajor_sw128(src + SH_X_BYTES);
#pragma unroll
        for (int k = 0; k < SH_KB / 16; ++k)
          mma_f16(tmem + acc * p.cols, a + (uint64_t)(2 * k), b + (uint64_t)(2 * k), idesc,
                  (i > 0 || k > 0) ? 1u : 0u);
        any = true;
        mma_commit(empty_bar(stage));
        if ((int)++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
        if (i == SH_DRAIN - 1 || kb + 1 == blocks) {
          mma_commit(tfull(acc));
          if (++acc == p.accs) {
            acc = 0;
            aphase ^= 1u;
          }
        }
      }
    }
    if (!ok && any) {
      volatile int never = 0;
      mma_commit(drain);
      mbar_wait_bounded(drain, 0, &never, p.status, LLMINT8_DEV_TIMEOUT_DRAIN, p.timeout_ns);
    }
  } else if (warp >= 4) {
    // ----------------------------------- epilogue: this CTA's partial sums
    const int row = threadIdx.x - 128;
    const int slot = ts.slot[row];
    int acc = 0;
    uint32_t aphase = 0;
    bool ok = true;
    for (int32_t s0 = first; ok && s0 < ts.count; s0 += step) {
      const int32_t s1 = min(s0 + p.slots, ts.count);
      for (int32_t kb = 0; kb < blocks; kb += SH_DRAIN) {
        ok = mbar_wait_bounded(tfull(acc), aphase, abort_flag, p.status,
                               LLMINT8_DEV_TIMEOUT_EPILOGUE, p.timeout_ns);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        const uint32_t src = tmem + ((uint32_t)((warp & 3) * 32) << 16) + acc * p.cols;
        for (int32_t sl = s0; sl < s1; ++sl) {
          if (!__any_sync(0xffffffffu, slot == sl)) continue;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            if (c * 8 >= p.r) break;
            uint32_t v[8];
            tmem_ld_32x32b_x8(src + (uint32_t)((sl - s0) * p.r + c * 8), v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 8; ++e)
              sums[c * 8 + e] += slot == sl ? __uint_as_float(v[e]) : 0.0f;
          }
        }
        tc_fence_before();
        mbar_arrive(tempty(acc));
        if (++acc == p.accs) {
          acc = 0;
          aphase ^= 1u;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, p.tmem_cols);
  // the partial sums over the ring's memory (its copies have landed, its
  // products are done)
  float *part = reinterpret_cast<float *>(base);
  if (warp >= 4) {
    const int row = threadIdx.x - 128, slot = ts.slot[row];
    const int rk = slot >= 0 ? ts.rank[slot] : 0;
#pragma unroll
    for (int t = 0; t < NC * 8; ++t)
      if (t < p.r) part[row * ldp + t] = t < rk ? sums[t] : 0.0f;
  }
  __syncthreads();
  // the cluster's partial sums, in rank order; this CTA finishes TM / split rows
  if (p.split > 1) cluster_sync();
  const int rows = TM / p.split;
  for (int i = warp; i < rows; i += SH_THREADS / 32) {
    const int row = (int)cta * rows + i;
    if (row0 + row >= p.s) continue;
    const int a = ts.id[row];
    if (p.w != nullptr && a >= 0 && first == 0) {
      const float wm = warp_row_max(p.w + (row0 + row) * p.r, p.r);
      if (lane == 0) atomicMax(p.w_amax + a, __float_as_uint(wm));
    }
    // (rows without an adapter are the first cluster's)
    if (gridDim.y > 1 && max(ts.slot[row], 0) / p.slots % gridDim.y != blockIdx.y) continue;
    float largest = 0.0f;
#pragma unroll 2
    for (int t = lane; t < p.r; t += 32) {
      float sum = 0.0f;
      if (p.split > 1) {
        // eight CTAs' loads under way before the first is added
        const uint32_t at = smem_u32(part + row * ldp + t);
        for (int q0 = 0; q0 < p.split; q0 += 8) {
          float x[8];
#pragma unroll
          for (int q = 0; q < 8; ++q)
            x[q] = q0 + q < p.split ? ld_cluster_f32(mapa_shared(at, (uint32_t)(q0 + q))) : 0.0f;
#pragma unroll
          for (int q = 0; q < 8; ++q) sum += x[q];
        }
      } else {
        sum = part[row * ldp + t];
      }
      p.v[(row0 + row) * p.r + t] = sum;
      largest = fmaxf(largest, finite_abs(sum));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, d));
    if (lane == 0) {
      p.vmax[row0 + row] = largest;
      if (p.amax != nullptr && a >= 0) atomicMax(p.amax + a, __float_as_uint(largest));
    }
  }
  if (p.split > 1) cluster_sync();  // no CTA leaves while its sums are read
}

// amax[a] = largest finite |w| of adapter a's rows of an [s][r] array (zero
// before): one warp per row.
__global__ void __launch_bounds__(256)
    k_adapter_max(const float *__restrict__ w, int64_t s, int32_t n, int32_t r,
                  const int32_t *__restrict__ ids, uint32_t *__restrict__ amax) {
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= s) return;
  const int a = adapter_of(ids, row, n);
  if (a < 0) return;
  const float m = warp_row_max(w + row * r, r);
  if ((threadIdx.x & 31) == 0) atomicMax(amax + a, __float_as_uint(m));
}

// -------------------------------------------------------------------- k_pack

constexpr int OU_KB = 64;                 // rows of a block; 32: 121 us instead of 116 for the
                                          // backward pass of 4096 x 20480 at rank 64
constexpr uint32_t OU_CORE = OU_KB * 16;  // 8 terms of 64 rows

// r rounded up to 16: columns of a product
__host__ __device__ inline int32_t outer_r16(int32_t r) { return (r + 15) / 16 * 16; }
// P of a block of 64 rows: hi octets, then lo octets, each as 8 core matrices
// of 8 rows x 8 terms
__host__ __device__ inline uint32_t outer_p_bytes(int32_t r) {
  return 2 * (uint32_t)(outer_r16(r) / 8) * OU_CORE;
}

// What is noted about a block of rows: their adapter when all 64 have the same
// one, or
constexpr int32_t OU_NONE = -1, OU_MIXED = -2;

struct PackJob {
  const float *p;        // [s][r]
  const uint32_t *amax;  // [n]
  uint8_t *out;          // [blocks of 64 rows][outer_p_bytes]
};

struct PackParams {
  PackJob job[2];
  int32_t jobs, blocks;  // jobs * blocks blocks of threads
  int32_t s, n, r;
  const int32_t *ids;
  int32_t *info;         // [blocks]
};

// One block of rows of one job (index i of jobs * blocks), by a whole block of
// threads: each row scaled for its own adapter; zeros for rows without one,
// rows past s and terms past r.
__device__ __forceinline__ void pack_block(const PackParams &p, int32_t i) {
  const PackJob &job = p.job[i / p.blocks];
  const int32_t b = i % p.blocks;
  const int64_t row0 = (int64_t)b * OU_KB;
  if (i < p.blocks) {  // the note, once
    const int64_t row = row0 + threadIdx.x;
    const bool mine = threadIdx.x < OU_KB;
    const int a = mine && row < p.s ? adapter_of(p.ids, row, p.n) : -1;
    const int lead = adapter_of(p.ids, row0, p.n);
    const bool same = __syncthreads_and(!mine || a == lead);
    const bool none = __syncthreads_and(a < 0);
    if (threadIdx.x == 0) p.info[b] = none ? OU_NONE : same ? lead : OU_MIXED;
  }
  uint8_t *dst = job.out + (size_t)b * outer_p_bytes(p.r);
  const int octs = outer_r16(p.r) / 8;
  for (int e = threadIdx.x; e < octs * OU_KB; e += blockDim.x) {
    const int oct = e / OU_KB, k = e % OU_KB;
    const int64_t row = row0 + k;
    const int a = row < p.s ? adapter_of(p.ids, row, p.n) : -1;
    float x[8] = {}, f = 0.0f;
    if (a >= 0 && oct < p.r / 8) {
      f = pow2(-scale_exponent(__uint_as_float(job.amax[a])));
      Vec8<float> v;
      v.load(job.p + row * p.r + oct * 8);
      v.get(x);
    }
    uint4 hi, lo;
    split8(x, f, hi, lo);
    *reinterpret_cast<uint4 *>(dst + oct * OU_CORE + k * 16) = hi;
    *reinterpret_cast<uint4 *>(dst + (octs + oct) * OU_CORE + k * 16) = lo;
  }
}

// On its own where no k_expand runs (dX not wanted). Grid: jobs * blocks.
constexpr int PK_THREADS = 256;
__global__ void __launch_bounds__(PK_THREADS) k_pack(const __grid_constant__ PackParams p) {
  grid_dependency_trigger();
  grid_dependency_wait();
  pack_block(p, (int32_t)blockIdx.x);
}

// ------------------------------------------------------------------ k_expand

constexpr int EX_N = 64;           // features per step
constexpr int EX_WARPS = 13, EX_THREADS = 32 * EX_WARPS;
constexpr int EX_EPI_THREADS = 256;
constexpr int EX_ACC = 4;          // accumulators of EX_N columns
constexpr int EX_MAX_RING = 8, EX_MAX_F = 4;
constexpr int EX_LOADERS = 2;      // warps 2 and 3
constexpr uint32_t EX_TILE_BYTES = TM * EX_N * 2;

struct ExpandParams {
  int32_t s, o, n, r;
  int32_t steps, chunks;   // feature steps, cut into chunks (one per CTA and row tile)
  int32_t ring, fbufs;     // base / output tiles, factor tiles in shared memory
  const float *v, *vmax, *scale;
  const __half *f;         // [n][r][o]
  const int32_t *ids, *rank;
  int32_t has_base;
  int32_t *status;
  uint64_t timeout_ns;
};

// rows of a factor tile: r, and the first 8 again when r is an odd multiple of 8
__host__ __device__ inline int32_t expand_f_rows(int32_t r) { return r % 16 ? r + 8 : r; }
__host__ __device__ inline uint32_t expand_bytes(int32_t r, int32_t ring, int32_t fbufs) {
  return (uint32_t)ring * EX_TILE_BYTES + (uint32_t)fbufs * expand_f_rows(r) * 128 +
         (uint32_t)r * 2 * TM * 2 + (uint32_t)sizeof(TileSlots) + TM * 4 + 512 + 1024;
}

// Grid: row tiles * chunks, then the blocks that k_pack would have.
__global__ void __launch_bounds__(EX_THREADS)
    k_expand(const __grid_constant__ CUtensorMap tm_base,
             const __grid_constant__ CUtensorMap tm_out, const ExpandParams p,
             const __grid_constant__ PackParams pack) {
  const int32_t tiles = (p.s + TM - 1) / TM;
  if ((int32_t)(blockIdx.x / p.chunks) >= tiles) {
    grid_dependency_trigger();
    grid_dependency_wait();
    pack_block(pack, (int32_t)blockIdx.x - tiles * p.chunks);
    return;
  }
  grid_dependency_trigger();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t *base = smem_raw + pad;
  const uint32_t ring = smem_u32(base);
  const int32_t frows = expand_f_rows(p.r);
  const uint32_t fbuf = ring + (uint32_t)p.ring * EX_TILE_BYTES;
  uint8_t *vop = base + p.ring * EX_TILE_BYTES + p.fbufs * frows * 128;  // hi, lo octets of v
  uint8_t *after = vop + p.r * 2 * TM * 2;
  TileSlots &ts = *reinterpret_cast<TileSlots *>(after);
  float *factor = reinterpret_cast<float *>(after + (sizeof(TileSlots) + 15) / 16 * 16);  // [TM]
  uint64_t *bars = reinterpret_cast<uint64_t *>(factor + TM);
  const uint32_t bar0 = smem_u32(bars);
  auto bfull = [&](int i) { return bar0 + 8u * i; };                    // base tile in
  auto bempty = [&](int i) { return bar0 + 8u * (EX_MAX_RING + i); };   // output tile out
  auto ready = [&](int i) { return bar0 + 8u * (2 * EX_MAX_RING + i); };  // output tile done
  auto ffull = [&](int i) { return bar0 + 8u * (3 * EX_MAX_RING + i); };
  auto fempty = [&](int i) { return bar0 + 8u * (3 * EX_MAX_RING + EX_MAX_F + i); };
  auto tfull = [&](int i) { return bar0 + 8u * (3 * EX_MAX_RING + 2 * EX_MAX_F + i); };
  auto tempty = [&](int i) { return bar0 + 8u * (3 * EX_MAX_RING + 2 * EX_MAX_F + EX_ACC + i); };
  const uint32_t drain = bar0 + 8u * (3 * EX_MAX_RING + 2 * EX_MAX_F + 2 * EX_ACC);
  Ctl *ctl = reinterpret_cast<Ctl *>(bars + 3 * EX_MAX_RING + 2 * EX_MAX_F + 2 * EX_ACC + 1);
  volatile int *abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row0 = (int64_t)(blockIdx.x / p.chunks) * TM;
  const int32_t chunk = (int32_t)(blockIdx.x % p.chunks);
  // this CTA's i-th step is chunk + i * chunks: the CTAs of a row tile read
  // and write neighbouring parts of a row at a time
  const int32_t mine = (p.steps - chunk + p.chunks - 1) / p.chunks;
  auto col_of = [&](int32_t i) { return (chunk + i * p.chunks) * EX_N; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.ring; ++i) {
      mbar_init(bfull(i), 1);
      mbar_init(bempty(i), 1);
      mbar_init(ready(i), EX_EPI_THREADS);
    }
    for (int i = 0; i < p.fbufs; ++i) {
      mbar_init(ffull(i), 1);
      mbar_init(fempty(i), 1);
    }
    for (int i = 0; i < EX_ACC; ++i) {
      mbar_init(tfull(i), 1);
      mbar_init(tempty(i), EX_EPI_THREADS);
    }
    mbar_init(drain, 1);
    ctl->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_out);
    // the first base tiles (no product of the preceding kernel) come in while
    // the rows' slots and v are set up
    if (p.has_base)
      for (int i = 0; i < min(p.ring, mine); ++i) {
        mbar_arrive_expect_tx(bfull(i), EX_TILE_BYTES);
        tma_load_2d(ring + i * EX_TILE_BYTES, &tm_base, bfull(i), col_of(i), (int32_t)row0);
      }
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(&ctl->tmem), EX_N * EX_ACC);
    tmem_relinquish();
  }
  tc_fence_before();
  tile_slots(p.ids, row0, p.s, p.n, p.rank, p.r, ts);
  grid_dependency_wait();  // v and vmax are the preceding kernel's
  // v of the tile as the MMA's A operand: core matrices of 8 rows x 8 terms,
  // all of the rows' for an octet of terms one after another; r hi columns,
  // then r lo columns
  for (int i = threadIdx.x; i < TM * (p.r / 8); i += EX_THREADS) {
    const int row = i % TM, oct = i / TM;
    float x[8] = {};
    float f = 0.0f;
    if (ts.id[row] >= 0) {
      const int e = scale_exponent(p.vmax[row0 + row]);
      f = pow2(-e);
      Vec8<float> v;
      v.load(p.v + (row0 + row) * p.r + oct * 8);
      v.get(x);
      if (oct == 0) factor[row] = p.scale[ts.id[row]] * pow2(e);
    }
    uint4 hi, lo;
    split8(x, f, hi, lo);
    const int at = (row / 8) * 128 + (row % 8) * 16;
    *reinterpret_cast<uint4 *>(vop + oct * (TM * 16) + at) = hi;
    *reinterpret_cast<uint4 *>(vop + (p.r / 8 + oct) * (TM * 16) + at) = lo;
  }
  fence_proxy_async_smem();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  const int32_t count = ts.count;

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------ base tiles by TMA
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    const int32_t early = p.has_base ? min(p.ring, mine) : 0;
    uint32_t issued = (1u << early) - 1u, last_par = 0;
    if (early == p.ring) phase = 1;
    else slot = early;
    for (int32_t n = early; n < mine; ++n) {
      if (!mbar_wait_bounded(bempty(slot), phase ^ 1u, abort_flag, p.status,
                             LLMINT8_DEV_TIMEOUT_PRODUCER, p.timeout_ns)) {
        ok = false;
        break;
      }
      if (p.has_base) {
        mbar_arrive_expect_tx(bfull(slot), EX_TILE_BYTES);
        tma_load_2d(ring + slot * EX_TILE_BYTES, &tm_base, bfull(slot), col_of(n), (int32_t)row0);
        issued |= 1u << slot;
        last_par = (last_par & ~(1u << slot)) | (phase << slot);
      } else {
        mbar_arrive(bfull(slot));
      }
      if (++slot == p.ring) {
        slot = 0;
        phase ^= 1u;
      }
    }
    if (!ok) {
      volatile int never = 0;
      for (int st = 0; st < p.ring; ++st)
        if ((issued >> st) & 1u)
          mbar_wait_bounded(bfull(st), (last_par >> st) & 1u, &never, p.status,
                            LLMINT8_DEV_TIMEOUT_DRAIN, p.timeout_ns);
    }
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------------- MMA issuer
    const uint32_t idesc = idesc_f16_f32_mn(TM, EX_N, false, true);
    const uint32_t va = smem_u32(vop);
    int fb = 0, acc = 0;
    uint32_t fphase = 0, tphase = 0;
    bool ok = true, any = false;
    for (int32_t i = 0; ok && i < mine * count; ++i) {
      ok = mbar_wait_bounded(tempty(acc), tphase ^ 1u, abort_flag, p.status,
                             LLMINT8_DEV_TIMEOUT_MMA, p.timeout_ns) &&
           mbar_wait_bounded(ffull(fb), fphase, abort_flag, p.status, LLMINT8_DEV_TIMEOUT_MMA,
                             p.timeout_ns);
      if (!ok) break;
      tc_fence_after();
      // 16 of the 2 r columns of v at a time; column c meets factor row
      // c mod r (a chunk that crosses from hi to lo runs on into the copy of
      // the first 8 rows)
      for (int c = 0; c < 2 * p.r; c += 16)
        mma_f16(tmem + acc * EX_N, smem_desc_core(va + (c / 8) * (TM * 16), TM * 16, 128),
                smem_desc_mn_sw128(fbuf + fb * frows * 128 + (c < p.r ? c : c - p.r) * 128, 0),
                idesc, c > 0 ? 1u : 0u);
      any = true;
      mma_commit(fempty(fb));
      mma_commit(tfull(acc));
      if (++fb == p.fbufs) {
        fb = 0;
        fphase ^= 1u;
      }
      if (++acc == EX_ACC) {
        acc = 0;
        tphase ^= 1u;
      }
    }
    if (!ok && any) {
      volatile int never = 0;
      mma_commit(drain);
      mbar_wait_bounded(drain, 0, &never, p.status, LLMINT8_DEV_TIMEOUT_DRAIN, p.timeout_ns);
    }
  } else if (warp == 2 || warp == 3) {
    // ---------------- factor tiles [rows][64], zeros past the adapter's rank;
    // a tile's copies are under way while the warp's previous one completes.
    // fbufs is even, so each buffer is one warp's.
    const int32_t jobs = mine * count;
    int32_t pending = -1;  // buffer whose copies were issued last
    auto publish = [&](int fb) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(ffull(fb));
    };
    bool ok = true;
    for (int32_t i = warp - 2; i < jobs; i += EX_LOADERS) {
      const int fb = i % p.fbufs;
      const uint32_t par = (uint32_t)((i / p.fbufs) & 1) ^ 1u;
      if (pending >= 0 && !__all_sync(0xffffffffu, mbar_test(fempty(fb), par))) {
        // no buffer free yet: the previous tile need not wait for one
        cp_async_wait<0>();
        publish(pending);
        pending = -1;
      }
      ok = mbar_wait_bounded(fempty(fb), par, abort_flag, p.status, LLMINT8_DEV_TIMEOUT_PRODUCER,
                             p.timeout_ns);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const int sl = i % count;
      const int a = ts.adapter[sl], rk = ts.rank[sl];
      const int32_t col = col_of(i / count) + (lane & 7) * 8;
      const __half *src = p.f + (int64_t)a * p.r * p.o + col;
      const uint32_t dst = fbuf + fb * frows * 128;
      for (int row = lane >> 3; row < frows; row += 4) {
        const int t = row < p.r ? row : row - p.r;
        const bool in = t < rk && col < p.o;
        cp_async_16(dst + row * 128 + (((lane & 7) ^ (row & 7)) << 4),
                    in ? src + (int64_t)t * p.o : p.f, in);
      }
      cp_async_commit();
      if (pending >= 0) {
        cp_async_wait<1>();
        publish(pending);
      }
      pending = fb;
    }
    cp_async_wait<0>();
    if (ok && pending >= 0) publish(pending);
  } else if (warp == EX_WARPS - 1 && lane == 0) {
    // ---------------------------------------------- output tiles by TMA
    int prev = -1;  // tile whose store may still read shared memory
    for (int32_t n = 0; n < mine; ++n) {
      const int slot = n % p.ring;
      if (!mbar_wait_bounded(ready(slot), (uint32_t)((n / p.ring) & 1), abort_flag, p.status,
                             LLMINT8_DEV_TIMEOUT_EPILOGUE, p.timeout_ns))
        break;
      tma_store_2d(&tm_out, ring + slot * EX_TILE_BYTES, col_of(n), (int32_t)row0);
      bulk_commit_group();
      if (prev >= 0) {
        bulk_wait_group_read1();
        mbar_arrive(bempty(prev));
      }
      prev = slot;
    }
    bulk_wait_group0();
  } else if (warp >= 4 && warp < EX_WARPS - 1) {
    // --------------------------------------------------------- epilogue
    // row = TMEM lane; 32 of the step's 64 columns per warp. All eight warps
    // take every step: a parity wait tells only neighbouring phases apart, so
    // no barrier of these rings may have waiters that skip phases.
    const int row = (warp & 3) * 32 + lane, half = (warp - 4) >> 2;
    const int my = ts.slot[row];
    const float f = my >= 0 ? factor[row] : 0.0f;
    int slot = 0, acc = 0;
    uint32_t bphase = 0, tphase = 0;
    bool ok = true;
    for (int32_t n = 0; ok && n < mine; ++n) {
      ok = mbar_wait_bounded(bfull(slot), bphase, abort_flag, p.status,
                             LLMINT8_DEV_TIMEOUT_EPILOGUE, p.timeout_ns);
      ok = __all_sync(0xffffffffu, ok);
      uint8_t *tile = base + slot * EX_TILE_BYTES + row * 128;
      if (ok && !p.has_base && my < 0) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4 *>(tile + (((half * 4 + c) ^ (row & 7)) << 4)) =
              make_uint4(0u, 0u, 0u, 0u);
      }
      for (int32_t sl = 0; ok && sl < count; ++sl) {
        ok = mbar_wait_bounded(tfull(acc), tphase, abort_flag, p.status,
                               LLMINT8_DEV_TIMEOUT_EPILOGUE, p.timeout_ns);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        if (__any_sync(0xffffffffu, my == sl)) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + acc * EX_N + half * 32,
                             v);
          tmem_ld_wait();
          if (my == sl) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint8_t *at = tile + (((half * 4 + c) ^ (row & 7)) << 4);
              float x[8] = {};
              if (p.has_base) {
                Vec8<__half> b;
                b.load(reinterpret_cast<const __half *>(at));
                b.get(x);
              }
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = fmaf(f, __uint_as_float(v[8 * c + e]), x[e]);
              store8(reinterpret_cast<__half *>(at), x);
            }
          }
          __syncwarp();
        }
        tc_fence_before();
        mbar_arrive(tempty(acc));
        if (++acc == EX_ACC) {
          acc = 0;
          tphase ^= 1u;
        }
      }
      if (!ok) break;
      fence_proxy_async_smem();
      mbar_arrive(ready(slot));
      if (++slot == p.ring) {
        slot = 0;
        bphase ^= 1u;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, EX_N * EX_ACC);
}

// ------------------------------------------------------------------- k_outer

constexpr int OU_COLS = 256;       // features per cluster: two M = 128 products
constexpr int OU_SUM_WARPS = 8;
constexpr int OU_THREADS = 32 * (2 + OU_SUM_WARPS);
constexpr int OU_DRAIN = 2;        // blocks (of 8 MMAs per product) that one accumulator sums
constexpr int OU_MAX_STAGES = 6;
constexpr int OU_MAX_SPLIT = 8;
constexpr int OU_WINDOW = 512;     // blocks of rows looked through at a time
constexpr uint32_t OU_Q_BYTES = OU_KB * OU_COLS * 2;
constexpr uint32_t OU_BLOCK_BYTES = OU_KB * 128;  // 64 features x 64 rows

struct OuterParams {
  int32_t s, w, n, r;      // rows, features
  int32_t split, stages, tmem_cols;
  int32_t col_tiles;
  uint32_t stage_bytes;
  const uint8_t *p;        // k_pack's output
  const int32_t *info;
  const uint32_t *amax;    // [n]
  const int32_t *ids, *rank;
  const float *scale;
  float *out;              // [n][r][w]
  int32_t *status;
  uint64_t timeout_ns;
};

struct OuterJob {
  CUtensorMap q;           // Q [s][w] in 64 x 64 boxes
  OuterParams p;
};

// block list, masks, barriers, alignment
constexpr uint32_t OU_FIXED_BYTES = OU_WINDOW * (8 + 4) + 512 + 1024;

// NC: octets of terms that a thread sums in registers (r <= 8 NC). Grid: (col
// tiles of both jobs * split, 1, n), clusters of `split` along x.
//   warp 0     TMA producer: 64 rows x 256 features of Q, and their P
//   warp 1     TMEM, MMA issuer
//   warps 2-9  zero the rows of other adapters in mixed blocks (both
//              operands, whatever they hold) before the MMAs; add each
//              accumulator to the sums in their registers (one product and a
//              quarter of its features each); add up the cluster's and store
template <int NC>
__global__ void __launch_bounds__(OU_THREADS, NC <= 8 ? 2 : 1)
    k_outer(const __grid_constant__ OuterJob j0, const __grid_constant__ OuterJob j1) {
  const int32_t group = (int32_t)(blockIdx.x / j0.p.split);
  const bool second = group >= j0.p.col_tiles;
  const OuterJob &job = second ? j1 : j0;
  const OuterParams &p = job.p;
  const int32_t col0 = (second ? group - j0.p.col_tiles : group) * OU_COLS;
  const int32_t a = (int32_t)blockIdx.z;
  const uint32_t cta = p.split > 1 ? cluster_ctarank() : 0;
  const int32_t r16 = outer_r16(p.r);
  const uint32_t p_bytes = outer_p_bytes(p.r);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t *base = smem_raw + pad;
  const uint32_t ring = smem_u32(base);
  uint8_t *after = base + p.stages * p.stage_bytes;
  uint64_t *masks = reinterpret_cast<uint64_t *>(after);            // [OU_WINDOW]
  int32_t *list = reinterpret_cast<int32_t *>(masks + OU_WINDOW);   // [OU_WINDOW]
  uint64_t *bars = reinterpret_cast<uint64_t *>(list + OU_WINDOW);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int i) { return bar0 + 8u * i; };
  auto clean = [&](int i) { return bar0 + 8u * (OU_MAX_STAGES + i); };
  auto empty = [&](int i) { return bar0 + 8u * (2 * OU_MAX_STAGES + i); };
  auto tfull = [&](uint32_t i) { return bar0 + 8u * (3 * OU_MAX_STAGES + i); };
  auto tempty = [&](uint32_t i) { return bar0 + 8u * (3 * OU_MAX_STAGES + 2 + i); };
  const uint32_t drain = bar0 + 8u * (3 * OU_MAX_STAGES + 4);
  Ctl *ctl = reinterpret_cast<Ctl *>(bars + 3 * OU_MAX_STAGES + 5);
  volatile int *abort_flag = &ctl->abort;
  int32_t *listed = reinterpret_cast<int32_t *>(ctl + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(clean(i), OU_SUM_WARPS);
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull(i), 1);
      mbar_init(tempty(i), 32 * OU_SUM_WARPS);
    }
    mbar_init(drain, 1);
    ctl->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&job.q);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl->tmem), p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  grid_dependency_wait();  // P, info and amax are the preceding kernels'

  // sums of a thread's feature: product `prod`, TMEM lane quarter (warp & 3)
  const int prod = (warp - 2) >> 2;
  float acc[NC * 8];
#pragma unroll
  for (int t = 0; t < NC * 8; ++t) acc[t] = 0.0f;

  const int64_t blocks = ((int64_t)p.s + OU_KB - 1) / OU_KB;
  // blocks and accumulators that this CTA has used before the window, counted
  // apart: a window's last accumulator may sum fewer than OU_DRAIN blocks, but
  // the ring passes over no slot
  uint32_t it0 = 0, use0 = 0;
  uint32_t cleaned = 0;  // phase of each slot's clean barrier, which only
                         // mixed blocks use
  bool failed = false, used = false;
  for (int64_t w0 = 0; w0 < blocks; w0 += OU_WINDOW) {
    const int nb = (int)min((int64_t)OU_WINDOW, blocks - w0);
    // which rows of each block are the adapter's
    for (int b = 32 * warp; b < nb; b += OU_THREADS) {
      const int32_t what = b + lane < nb ? p.info[w0 + b + lane] : OU_NONE;
      if (b + lane < nb && what != OU_MIXED) masks[b + lane] = what == a ? ~0ull : 0ull;
      unsigned mixed = __ballot_sync(0xffffffffu, what == OU_MIXED);
      while (mixed) {
        const int e = __ffs(mixed) - 1;
        mixed &= mixed - 1;
        const int64_t r0 = (w0 + b + e) * OU_KB + lane;
        const unsigned lo = __ballot_sync(0xffffffffu, r0 < p.s && p.ids[r0] == a);
        const unsigned hi = __ballot_sync(0xffffffffu, r0 + 32 < p.s && p.ids[r0 + 32] == a);
        if (lane == 0) masks[b + e] = (uint64_t)hi << 32 | lo;
      }
    }
    __syncthreads();
    if (warp == 0) {  // the non-empty blocks, in order
      int cnt = 0;
      for (int b = 0; b < nb; b += 32) {
        const bool any = b + lane < nb && masks[b + lane] != 0;
        const unsigned v = __ballot_sync(0xffffffffu, any);
        if (any) list[cnt + __popc(v & ((1u << lane) - 1u))] = b + lane;
        cnt += __popc(v);
      }
      if (lane == 0) *listed = cnt;
    }
    __syncthreads();
    const int32_t total = *listed;
    used |= total > 0;
    // this CTA's i-th block of the window is list[cta + i * split]
    const int32_t mine = total > (int32_t)cta ? (total - (int32_t)cta + p.split - 1) / p.split : 0;
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------- TMA producer
      for (int32_t i = 0; i < mine; ++i) {
        const uint32_t it = it0 + i;
        const int st = (int)(it % p.stages);
        if (!mbar_wait_bounded(empty(st), ((it / p.stages) & 1u) ^ 1u, abort_flag, p.status,
                               LLMINT8_DEV_TIMEOUT_PRODUCER, p.timeout_ns))
          break;
        const uint32_t dst = ring + st * p.stage_bytes;
        const int64_t b = w0 + list[cta + i * p.split];
        mbar_arrive_expect_tx(full(st), OU_Q_BYTES + p_bytes);
#pragma unroll
        for (int c = 0; c < OU_COLS / 64; ++c)
          tma_load_2d(dst + c * OU_BLOCK_BYTES, &job.q, full(st), col0 + c * 64,
                      (int32_t)(b * OU_KB));
        bulk_load_1d(dst + OU_Q_BYTES, p.p + (size_t)b * p_bytes, p_bytes, full(st));
      }
    } else if (warp == 1 && lane == 0) {
      // ----------------------------------------------------- MMA issuer
      const uint32_t idesc = idesc_f16_f32_mn(128, r16, true, true);
      for (int32_t i = 0; i < mine; ++i) {
        const uint32_t it = it0 + i, use = use0 + i / OU_DRAIN, buf = use & 1u;
        const int st = (int)(it % p.stages);
        const uint32_t par = (it / p.stages) & 1u;
        const bool fresh = i % OU_DRAIN == 0;
        if ((fresh && !mbar_wait_bounded(tempty(buf), ((use >> 1) & 1u) ^ 1u, abort_flag, p.status,
                                         LLMINT8_DEV_TIMEOUT_MMA, p.timeout_ns)) ||
            !mbar_wait_bounded(full(st), par, abort_flag, p.status, LLMINT8_DEV_TIMEOUT_MMA,
                               p.timeout_ns) ||
            (masks[list[cta + i * p.split]] != ~0ull &&
             !mbar_wait_bounded(clean(st), (cleaned >> st) & 1u, abort_flag, p.status,
                                LLMINT8_DEV_TIMEOUT_MMA, p.timeout_ns)))
          break;
        if (masks[list[cta + i * p.split]] != ~0ull) cleaned ^= 1u << st;
        tc_fence_after();
        const uint32_t src = ring + st * p.stage_bytes;
#pragma unroll
        for (int c = 0; c < 2; ++c)
          for (int hl = 0; hl < 2; ++hl)
#pragma unroll
            for (int k = 0; k < OU_KB / 16; ++k)
              mma_f16(tmem + (buf * 2 + c) * r16,
                      smem_desc_mn_sw128(src + c * 2 * OU_BLOCK_BYTES + k * 2048, OU_BLOCK_BYTES),
                      smem_desc_core(src + OU_Q_BYTES + hl * (p_bytes / 2) + k * 256, 128,
                                     OU_CORE),
                      idesc, (!fresh || hl > 0 || k > 0) ? 1u : 0u);
        mma_commit(empty(st));
        if (i % OU_DRAIN == OU_DRAIN - 1 || i + 1 == mine) mma_commit(tfull(buf));
      }
    } else if (warp >= 2) {
      const int ct = threadIdx.x - 64;
      const int k = ct & 63, o0 = ct >> 6;
      bool ok = true;
      // group j of OU_DRAIN blocks is cleaned while group j - 1 is multiplied
      for (int32_t j = 0; ok && j <= (mine + OU_DRAIN - 1) / OU_DRAIN; ++j) {
        for (int32_t i = j * OU_DRAIN; ok && i < min(mine, (j + 1) * OU_DRAIN); ++i) {
          const uint32_t it = it0 + i;
          const int st = (int)(it % p.stages);
          const uint64_t mask = masks[list[cta + i * p.split]];
          if (mask == ~0ull) continue;
          // the slot's previous block multiplied, then this one's copy landed
          // (its full barrier alone would not do: these warps skip the blocks
          // that need no cleaning, and a parity wait tells only neighbouring
          // phases apart. The empty barrier is safe: the group before last is
          // summed, so at most one of its phases is open.)
          const uint32_t par = (it / p.stages) & 1u;
          ok = mbar_wait_bounded(empty(st), par ^ 1u, abort_flag, p.status,
                                 LLMINT8_DEV_TIMEOUT_MMA, p.timeout_ns) &&
               mbar_wait_bounded(full(st), par, abort_flag, p.status, LLMINT8_DEV_TIMEOUT_MMA,
                                 p.timeout_ns);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          if (!((mask >> k) & 1u)) {
            uint8_t *q = base + st * p.stage_bytes;
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            for (int c = o0; c < 8 * (OU_COLS / 64); c += 4)
              *reinterpret_cast<uint4 *>(q + (c >> 3) * OU_BLOCK_BYTES + k * 128 + (c & 7) * 16) =
                  zero;
            for (int oct = o0; oct < 2 * (r16 / 8); oct += 4)
              *reinterpret_cast<uint4 *>(q + OU_Q_BYTES + oct * OU_CORE + k * 16) = zero;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(clean(st));
        }
        if (!ok || j == 0) continue;
        const uint32_t use = use0 + j - 1, buf = use & 1u;
        ok = mbar_wait_bounded(tfull(buf), (use >> 1) & 1u, abort_flag, p.status,
                               LLMINT8_DEV_TIMEOUT_EPILOGUE, p.timeout_ns);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        const uint32_t src =
            tmem + ((uint32_t)((warp & 3) * 32) << 16) + (buf * 2 + prod) * r16;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if (c * 8 >= p.r) break;
          uint32_t v[8];
          tmem_ld_32x32b_x8(src + c * 8, v);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[c * 8 + e] += __uint_as_float(v[e]);
        }
        tc_fence_before();
        mbar_arrive(tempty(buf));
      }
    }
    __syncthreads();
    it0 += (uint32_t)mine;
    use0 += (uint32_t)((mine + OU_DRAIN - 1) / OU_DRAIN);
    if (*abort_flag) {
      failed = true;
      break;
    }
  }
  if (failed) {  // MMAs and copies in flight end before shared memory goes
    if (warp == 1 && lane == 0) {
      volatile int never = 0;
      mma_commit(drain);
      mbar_wait_bounded(drain, 0, &never, p.status, LLMINT8_DEV_TIMEOUT_DRAIN, p.timeout_ns);
    }
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 200000u) __nanosleep(1000);
    __syncthreads();
  }
  // partial sums [r][OU_COLS] over the ring's memory (every product has been
  // read, so every copy has landed)
  float *part = reinterpret_cast<float *>(base);
  if (warp >= 2) {
    const int feature = prod * 128 + (warp & 3) * 32 + lane;
#pragma unroll
    for (int t = 0; t < NC * 8; ++t)
      if (t < p.r) part[t * OU_COLS + feature] = acc[t];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, p.tmem_cols);
  if (p.split > 1) cluster_sync();
  const float f = p.scale[a] * pow2(scale_exponent(__uint_as_float(p.amax[a])));
  // (an adapter without rows has zeros, whatever its scale)
  const int rk = used ? rank_of(p.rank, a, p.r) : 0;
  // this CTA's terms are cta, cta + split, ...; four features per thread, and
  // every CTA's load under way before the first is added
  const int quads = OU_COLS / 4, terms = (p.r - (int)cta + p.split - 1) / p.split;
#pragma unroll 2
  for (int i = threadIdx.x; i < terms * quads; i += OU_THREADS) {
    const int t = (int)cta + (i / quads) * p.split, c = (i % quads) * 4;
    const uint32_t at = smem_u32(part + t * OU_COLS + c);
    float4 x[OU_MAX_SPLIT];
#pragma unroll
    for (int q = 0; q < OU_MAX_SPLIT; ++q)
      x[q] = q >= p.split    ? make_float4(0.f, 0.f, 0.f, 0.f)
             : p.split > 1   ? ld_cluster_f32x4(mapa_shared(at, (uint32_t)q))
                             : *reinterpret_cast<const float4 *>(part + t * OU_COLS + c);
    float4 sum = x[0];
#pragma unroll
    for (int q = 1; q < OU_MAX_SPLIT; ++q) {
      sum.x += x[q].x;
      sum.y += x[q].y;
      sum.z += x[q].z;
      sum.w += x[q].w;
    }
    if (col0 + c < p.w)  // w is a multiple of 16; an unused term is 0 whatever its sum
      *reinterpret_cast<float4 *>(p.out + ((int64_t)a * p.r + t) * p.w + col0 + c) =
          t < rk ? make_float4(f * sum.x, f * sum.y, f * sum.z, f * sum.w)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (p.split > 1) cluster_sync();
}

}  // namespace lora
}  // namespace llmint8

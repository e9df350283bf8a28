// Low-rank adapters of many requests beside one projection. Row i of a batch
// uses adapter a = ids[i] (none when the id is outside [0, n)), which holds
// rank[a] <= r rank-one terms, A[a][t][0..h) and B[a][t][0..o):
//
//   v[i][t] = X[i] . A[a][t]
//   out[i]  = fp16(base[i] + scale[a] * sum_t v[i][t] * B[a][t])
//
// Both factors are rank-major, so the backward pass is the same two products
// with A and B exchanged (g = dY . B, dX = base + scale * g . A), plus one
// sum over the rows of each adapter:
//
//   dA[a][t] = scale[a] * sum_{i: ids[i] = a} g[i][t] * X[i]
//   dB[a][t] = scale[a] * sum_{i: ids[i] = a} v[i][t] * dY[i]
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "ptx_finetune_sm100.cuh"
#include "rows_common.cuh"

namespace llmint8 {
namespace lora {

constexpr int MAX_R = 128;

__device__ __forceinline__ int adapter_of(const int32_t *ids, int64_t i, int32_t n) {
  const int a = ids[i];
  return a >= 0 && a < n ? a : -1;
}

__device__ __forceinline__ int rank_of(const int32_t *rank, int a, int r) {
  return rank ? max(0, min(rank[a], r)) : r;
}

// ----------------------------- up to a tile of rows (decode steps, short prompts)
//
// Each row reads its own adapter's factors, so the work is spread over (row,
// slice of the features) blocks on CUDA cores, with fp32 products and sums.
// k_rows_shrink leaves one partial sum of v per slice; k_rows_expand, launched
// as its programmatic dependent, has its first factor rows in registers before
// it waits for them. Against the tensor-core kernels, which multiply a whole
// tile of rows with every adapter in it (forward, 12288 -> 20480, rank 64): 64
// rows of 64 adapters 48 us instead of 178, 128 of 64 68 instead of 184; rows
// of one adapter, which those kernels suit best, 25 instead of 19 at 64 rows
// and 45 instead of 21 at 128.

constexpr int RS_SLICE = 512;       // features of a k_rows_shrink block
constexpr int RS_THREADS = 256;
constexpr int RE_THREADS = 128;
constexpr int RE_SLICE = 8 * RE_THREADS;  // features of a k_rows_expand block
constexpr int RE_AHEAD = 16;        // factor rows held in registers

// part[slice][i][t] = X[i] . F[a][t] over the slice. Grid (slices, s).
__global__ void __launch_bounds__(RS_THREADS)
    k_rows_shrink(const __half *__restrict__ X, int32_t s, int32_t h, const __half *__restrict__ F,
                  const int32_t *__restrict__ ids, const int32_t *__restrict__ rank, int32_t n,
                  int32_t r, float *__restrict__ part) {
  grid_dependency_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.y;
  const int a = adapter_of(ids, row, n);
  const int rk = a >= 0 ? rank_of(rank, a, r) : 0;
  const int c0 = blockIdx.x * RS_SLICE + lane * 8;  // and 256 features further
  float x[2][8];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    Vec8<__half> v;
    v.zero();
    if (c0 + 256 * u < h) v.load(X + row * h + c0 + 256 * u);
    v.get(x[u]);
  }
  float *dst = part + ((int64_t)blockIdx.x * s + row) * r;
  const __half *f = F + (int64_t)max(a, 0) * r * h;
#pragma unroll 4
  for (int t = warp; t < r; t += RS_THREADS / 32) {
    float acc = 0.0f;
    if (t < rk) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (c0 + 256 * u >= h) continue;
        Vec8<__half> v;
        v.load(f + (int64_t)t * h + c0 + 256 * u);
        float y[8];
        v.get(y);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc = fmaf(x[u][e], y[e], acc);
      }
    }
    acc = warp_sum(acc);
    if (lane == 0) dst[t] = acc;
  }
}

// out[i][8c..] = base + scale * sum_t v[i][t] * F[a][t][8c..]; v itself to
// v_out (or null). out may be null: v alone. Grid (slices of out, s).
// (part is k_rows_shrink's, which may still run when this kernel starts: not
// __restrict__, so that no read of it can move before the wait.)
__global__ void __launch_bounds__(RE_THREADS)
    k_rows_expand(const float *part, int32_t slices, int32_t s, int32_t o,
                  const __half *__restrict__ F, const int32_t *__restrict__ ids,
                  const float *__restrict__ scale, const int32_t *__restrict__ rank, int32_t n,
                  int32_t r, const __half *base, __half *out, float *__restrict__ v_out) {
  __shared__ float seg_sum[RE_THREADS];
  __shared__ float v[MAX_R];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.y;
  const int col = blockIdx.x * RE_SLICE + tid * 8;
  const int a = adapter_of(ids, row, n);
  const int rk = a >= 0 ? rank_of(rank, a, r) : 0;
  const __half *f = F + (int64_t)max(a, 0) * r * o + col;
  const bool in = out != nullptr && col < o;
  Vec8<__half> ahead[RE_AHEAD], b;
#pragma unroll
  for (int t = 0; t < RE_AHEAD; ++t) {
    ahead[t].zero();
    if (in && t < rk) ahead[t].load(f + (int64_t)t * o);
  }
  b.zero();
  if (in && base) b.load(base + row * o + col);
  grid_dependency_wait();
  // v: the slices' sums, by RE_THREADS / r threads per term in turn
  const int segs = RE_THREADS / r, t0 = tid % r, seg = tid / r;
  float sum = 0.0f;
  if (seg < segs)
    for (int q = seg; q < slices; q += segs) sum += part[((int64_t)q * s + row) * r + t0];
  seg_sum[tid] = sum;
  __syncthreads();
  if (tid < r) {
    float t = 0.0f;
    for (int q = 0; q < segs; ++q) t += seg_sum[q * r + tid];
    v[tid] = t;
    if (v_out && blockIdx.x == 0) v_out[row * r + tid] = t;
  }
  __syncthreads();
  if (!in) return;
  if (a < 0) {
    *reinterpret_cast<uint4 *>(out + row * o + col) = b.q;
    return;
  }
  float acc[8] = {}, y[8];
#pragma unroll
  for (int t = 0; t < RE_AHEAD; ++t) {
    if (t < rk) {
      ahead[t].get(y);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(v[t], y[e], acc[e]);
    }
  }
#pragma unroll 8
  for (int t = RE_AHEAD; t < rk; ++t) {
    Vec8<__half> w;
    w.load(f + (int64_t)t * o);
    w.get(y);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = fmaf(v[t], y[e], acc[e]);
  }
  b.get(y);
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = fmaf(scale[a], acc[e], y[e]);
  store8(out + row * o + col, y);
}

// d[a][t][8c..] = scale[a] * sum of p[i][t] * Q[i][8c..] over the adapter's
// rows, in order: RO_TERMS terms and eight features per thread. Grid (slices
// of both jobs, n, ceil(r / RO_TERMS)); only the adapter's rows are read.
constexpr int RO_THREADS = 128;
constexpr int RO_SLICE = 8 * RO_THREADS;
constexpr int RO_TERMS = 8;
constexpr int RO_MAX_ROWS = 128;

struct RowsOuterJob {
  const float *p;   // [s][r]
  const __half *q;  // [s][w]
  float *d;         // [n][r][w]
  int32_t w;
};

__global__ void __launch_bounds__(RO_THREADS)
    k_rows_outer(const RowsOuterJob j0, const RowsOuterJob j1, int32_t slices0, int32_t s,
                 const int32_t *__restrict__ ids, const float *__restrict__ scale,
                 const int32_t *__restrict__ rank, int32_t n, int32_t r) {
  __shared__ int32_t rows[RO_MAX_ROWS];
  __shared__ float p[RO_MAX_ROWS][RO_TERMS];
  __shared__ int32_t per_warp[RO_THREADS / 32];
  const bool second = (int32_t)blockIdx.x >= slices0;
  const RowsOuterJob &job = second ? j1 : j0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int a = blockIdx.y, t0 = blockIdx.z * RO_TERMS;
  const int col = ((int)blockIdx.x - (second ? slices0 : 0)) * RO_SLICE + tid * 8;
  // the adapter's rows, in order
  const bool mine = tid < s && ids[tid] == a;
  const unsigned v = __ballot_sync(0xffffffffu, mine);
  if (lane == 0) per_warp[warp] = __popc(v);
  __syncthreads();
  int at = __popc(v & ((1u << lane) - 1u)), count = 0;
  for (int i = 0; i < RO_THREADS / 32; ++i) {
    if (i < warp) at += per_warp[i];
    count += per_warp[i];
  }
  if (mine) rows[at] = tid;
  // (an adapter without rows has zeros, whatever its scale)
  const int rk = count > 0 ? rank_of(rank, a, r) : 0;
  grid_dependency_wait();  // p is the preceding kernels'
  __syncthreads();
  for (int i = tid; i < count * RO_TERMS; i += RO_THREADS) {
    const int t = t0 + i % RO_TERMS;
    p[i / RO_TERMS][i % RO_TERMS] = t < rk ? job.p[(int64_t)rows[i / RO_TERMS] * r + t] : 0.0f;
  }
  __syncthreads();
  if (col >= job.w) return;
  float acc[RO_TERMS][8] = {};
  if (t0 < rk) {
#pragma unroll 4
    for (int i = 0; i < count; ++i) {
      Vec8<__half> q;
      q.load(job.q + (int64_t)rows[i] * job.w + col);
      float x[8];
      q.get(x);
#pragma unroll
      for (int t = 0; t < RO_TERMS; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[t][e] = fmaf(p[i][t], x[e], acc[t][e]);
    }
  }
  const float f = scale[a];
#pragma unroll
  for (int t = 0; t < RO_TERMS; ++t) {
    if (t0 + t >= r) break;
    float y[8];
    // (an unused term is 0 whatever its sum)
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = t0 + t < rk ? f * acc[t][e] : 0.0f;
    store8(job.d + ((int64_t)a * r + t0 + t) * job.w + col, y);
  }
}

}  // namespace lora
}  // namespace llmint8

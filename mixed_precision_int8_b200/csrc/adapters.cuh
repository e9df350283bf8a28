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

#include "ptx_sm100.cuh"
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

// v[i][t] = X[i] . F[a][t] (0 where the row has no adapter or t >= rank):
// one warp per (row, t).
__global__ void k_shrink_simple(const __half *X, int64_t s, int32_t h, const __half *F,
                                const int32_t *ids, const int32_t *rank, int32_t n, int32_t r,
                                float *v) {
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w >= s * r) return;
  const int64_t i = w / r;
  const int t = (int)(w % r);
  const int a = adapter_of(ids, i, n);
  float acc = 0.0f;
  if (a >= 0 && t < rank_of(rank, a, r)) {
    const __half *x = X + i * h, *f = F + ((int64_t)a * r + t) * h;
    for (int c = lane; c < h / 8; c += 32) {
      Vec8<__half> xv, fv;
      xv.load(x + 8 * c);
      fv.load(f + 8 * c);
      float xf[8], ff[8];
      xv.get(xf);
      fv.get(ff);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc = fmaf(xf[e], ff[e], acc);
    }
    acc = warp_sum(acc);
  }
  if (lane == 0) v[w] = acc;
}

// out[i][8c..] = fp16(base + scale * sum_t v[i][t] * F[a][t][8c..])
__global__ void k_expand_simple(const float *v, int64_t s, int32_t o, const __half *F,
                                const int32_t *ids, const float *scale, const int32_t *rank,
                                int32_t n, int32_t r, const __half *base, __half *out) {
  const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int nv = o / 8;
  if (idx >= s * nv) return;
  const int64_t i = idx / nv;
  const int c = (int)(idx % nv);
  const int a = adapter_of(ids, i, n);
  Vec8<__half> b;
  b.zero();
  if (base) b.load(base + i * o + 8 * c);
  if (a >= 0) {
    float acc[8] = {}, f[8];
    const int rk = rank_of(rank, a, r);
    for (int t = 0; t < rk; ++t) {
      Vec8<__half> fv;
      fv.load(F + ((int64_t)a * r + t) * o + 8 * c);
      fv.get(f);
      const float x = v[i * r + t];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(x, f[e], acc[e]);
    }
    b.get(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = fmaf(scale[a], acc[e], f[e]);
    store8(out + i * o + 8 * c, f);
  } else {
    *reinterpret_cast<uint4 *>(out + i * o + 8 * c) = b.q;
  }
}

// d[a][t][8c..] = scale[a] * sum over the adapter's rows of p[i][t] * Q[i][8c..]
__global__ void k_outer_simple(const float *p, const __half *Q, int64_t s, int32_t w,
                               const int32_t *ids, const float *scale, const int32_t *rank,
                               int32_t n, int32_t r, float *d) {
  const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int nv = w / 8;
  if (idx >= (int64_t)n * r * nv) return;
  const int c = (int)(idx % nv);
  const int t = (int)(idx / nv % r);
  const int a = (int)(idx / nv / r);
  float acc[8] = {}, f[8];
  if (t < rank_of(rank, a, r)) {
    for (int64_t i = 0; i < s; ++i) {
      if (ids[i] != a) continue;
      Vec8<__half> qv;
      qv.load(Q + i * w + 8 * c);
      qv.get(f);
      const float x = p[i * r + t];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(x, f[e], acc[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] *= scale[a];
  store8(d + idx * 8, acc);
}

}  // namespace lora
}  // namespace llmint8

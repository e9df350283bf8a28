// Layer norm over the rows that feed an LLM.int8() projection, and its
// backward pass.
//
//   mean = sum_j x_j / h        var = sum_j (x_j - mean)^2 / h
//   rstd = 1 / sqrt(var + eps)  xh_j = (x_j - mean) * rstd
//   y_j  = xh_j * gamma_j + beta_j
//   g_j  = dy_j * gamma_j
//   dx_j = rstd * (g_j - sum(g)/h - xh_j * sum(g * xh)/h)
//   dgamma_j = sum_rows dy_j * xh_j      dbeta_j = sum_rows dy_j
//
// Every sum is fp32; the variance is summed from the centred values, which
// keeps rows whose mean is large against their spread. The only roundings
// below fp32 are the stores of y and (for an fp16 x) dx.
//
// Bound: bytes. A row is read once and kept in registers (kVec8 vectors of
// eight elements per thread) between the sums and the store; rows too long
// for that are re-read from L2 by the *_long kernels.
#pragma once

#include <cstdint>

#include "ptx_sm100.cuh"
#include "rows_common.cuh"

namespace llmint8 {
namespace ln {

constexpr int MAX_THREADS = 512;
constexpr int MAX_VEC = 4;                            // vectors of 8 per thread
constexpr int64_t MAX_ROW = 8LL * MAX_VEC * MAX_THREADS;  // longest row held in registers

template <typename TX, typename TP, int NV>
__global__ void __launch_bounds__(MAX_THREADS)
    k_ln_forward(const TX *__restrict__ x, int32_t h, const TP *__restrict__ gamma,
                 const TP *__restrict__ beta, float eps, __half *__restrict__ y,
                 float *__restrict__ mean_out, float *__restrict__ rstd_out) {
  __shared__ float red[2][32];
  const int64_t row = blockIdx.x;
  const int nvec = h >> 3;
  const TX *xr = x + row * h;
  Vec8<TX> v[NV];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    v[i].zero();
    if (c < nvec) v[i].load(xr + 8 * c);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float f[8];
    v[i].get(f);
    sum += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
  }
  const float mean = block_sum(sum, red[0]) / (float)h;
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    float f[8];
    v[i].get(f);
    if (c < nvec) {
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(f[e] - mean, f[e] - mean, sq);
    }
  }
  const float rstd = 1.0f / sqrtf(block_sum(sq, red[1]) / (float)h + eps);
  __half *yr = y + row * h;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c >= nvec) continue;
    Vec8<TP> gv, bv;
    gv.load(gamma + 8 * c);
    bv.zero();
    if (beta) bv.load(beta + 8 * c);
    float f[8], g[8], b[8];
    v[i].get(f);
    gv.get(g);
    bv.get(b);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = fmaf((f[e] - mean) * rstd, g[e], b[e]);
    store8(yr + 8 * c, f);
  }
  if (threadIdx.x == 0) {
    if (mean_out) mean_out[row] = mean;
    if (rstd_out) rstd_out[row] = rstd;
  }
}

// Rows longer than MAX_ROW: the same sums with the row read three times.
template <typename TX, typename TP>
__global__ void __launch_bounds__(MAX_THREADS)
    k_ln_forward_long(const TX *__restrict__ x, int32_t h, const TP *__restrict__ gamma,
                      const TP *__restrict__ beta, float eps, __half *__restrict__ y,
                      float *__restrict__ mean_out, float *__restrict__ rstd_out) {
  __shared__ float red[2][32];
  const int64_t row = blockIdx.x;
  const int nvec = h >> 3;
  const TX *xr = x + row * h;
  float sum = 0.0f;
  for (int c = threadIdx.x; c < nvec; c += blockDim.x) {
    Vec8<TX> v;
    v.load(xr + 8 * c);
    float f[8];
    v.get(f);
    sum += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
  }
  const float mean = block_sum(sum, red[0]) / (float)h;
  float sq = 0.0f;
  for (int c = threadIdx.x; c < nvec; c += blockDim.x) {
    Vec8<TX> v;
    v.load(xr + 8 * c);
    float f[8];
    v.get(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) sq = fmaf(f[e] - mean, f[e] - mean, sq);
  }
  const float rstd = 1.0f / sqrtf(block_sum(sq, red[1]) / (float)h + eps);
  __half *yr = y + row * h;
  for (int c = threadIdx.x; c < nvec; c += blockDim.x) {
    Vec8<TX> v;
    Vec8<TP> gv, bv;
    v.load(xr + 8 * c);
    gv.load(gamma + 8 * c);
    bv.zero();
    if (beta) bv.load(beta + 8 * c);
    float f[8], g[8], b[8];
    v.get(f);
    gv.get(g);
    bv.get(b);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = fmaf((f[e] - mean) * rstd, g[e], b[e]);
    store8(yr + 8 * c, f);
  }
  if (threadIdx.x == 0) {
    if (mean_out) mean_out[row] = mean;
    if (rstd_out) rstd_out[row] = rstd;
  }
}

// Backward: block b takes rows b, b + grid, ...; each thread owns NV vectors
// of columns and keeps their dgamma / dbeta sums in registers over the
// block's rows, so the column sums cost one write of `part` (fp32
// [grid][2][h]) per block. k_ln_reduce adds those in block order.
template <typename TX, typename TP, int NV>
__global__ void __launch_bounds__(MAX_THREADS)
    k_ln_backward(const __half *__restrict__ dy, const TX *__restrict__ x, int64_t s, int32_t h,
                  const TP *__restrict__ gamma, const float *__restrict__ mean,
                  const float *__restrict__ rstd, TX *__restrict__ dx, float *__restrict__ part) {
  __shared__ float2 red[2][32];
  const int nvec = h >> 3;
  float dg[NV][8], db[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[i][e] = db[i][e] = 0.0f;
  const float inv_h = 1.0f / (float)h;
  int par = 0;
  for (int64_t row = blockIdx.x; row < s; row += gridDim.x, par ^= 1) {
    const float m = mean[row], q = rstd[row];
    Vec8<TX> xv[NV];
    Vec8<__half> yv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      xv[i].zero();
      yv[i].zero();
      if (c < nvec) {
        xv[i].load(x + row * h + 8 * c);
        yv[i].load(dy + row * h + 8 * c);
      }
    }
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c >= nvec) continue;
      float xf[8], yf[8], g[8];
      Vec8<TP> gv;
      gv.load(gamma + 8 * c);
      xv[i].get(xf);
      yv[i].get(yf);
      gv.get(g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (xf[e] - m) * q;
        dg[i][e] = fmaf(yf[e], xh, dg[i][e]);
        db[i][e] += yf[e];
        const float gg = yf[e] * g[e];
        a += gg;
        b = fmaf(gg, xh, b);
      }
    }
    const float2 ab = block_sum2(a, b, red[par]);
    if (dx) {
      const float c1 = ab.x * inv_h, c2 = ab.y * inv_h;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nvec) continue;
        float xf[8], yf[8], g[8];
        Vec8<TP> gv;
        gv.load(gamma + 8 * c);
        xv[i].get(xf);
        yv[i].get(yf);
        gv.get(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xh = (xf[e] - m) * q;
          xf[e] = q * (yf[e] * g[e] - c1 - xh * c2);
        }
        store8(dx + row * h + 8 * c, xf);
      }
    }
  }
  if (!part) return;
  float *pg = part + (int64_t)blockIdx.x * 2 * h;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c >= nvec) continue;
    store8(pg + 8 * c, dg[i]);
    store8(pg + h + 8 * c, db[i]);
  }
}

// Rows longer than MAX_ROW: the row is read twice, the column sums live in
// this block's slice of `part`.
template <typename TX, typename TP>
__global__ void __launch_bounds__(MAX_THREADS)
    k_ln_backward_long(const __half *__restrict__ dy, const TX *__restrict__ x, int64_t s,
                       int32_t h, const TP *__restrict__ gamma, const float *__restrict__ mean,
                       const float *__restrict__ rstd, TX *__restrict__ dx,
                       float *__restrict__ part) {
  __shared__ float2 red[2][32];
  const int nvec = h >> 3;
  const float inv_h = 1.0f / (float)h;
  float *pg = part ? part + (int64_t)blockIdx.x * 2 * h : nullptr;
  int par = 0;
  for (int64_t row = blockIdx.x; row < s; row += gridDim.x, par ^= 1) {
    const float m = mean[row], q = rstd[row];
    float a = 0.0f, b = 0.0f;
    for (int c = threadIdx.x; c < nvec; c += blockDim.x) {
      float xf[8], yf[8], g[8];
      Vec8<TX> xv;
      Vec8<__half> yv;
      Vec8<TP> gv;
      xv.load(x + row * h + 8 * c);
      yv.load(dy + row * h + 8 * c);
      gv.load(gamma + 8 * c);
      xv.get(xf);
      yv.get(yf);
      gv.get(g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float gg = yf[e] * g[e];
        a += gg;
        b = fmaf(gg, (xf[e] - m) * q, b);
      }
    }
    const float2 ab = block_sum2(a, b, red[par]);
    const float c1 = ab.x * inv_h, c2 = ab.y * inv_h;
    const bool first = row == blockIdx.x;
    for (int c = threadIdx.x; c < nvec; c += blockDim.x) {
      float xf[8], yf[8], g[8], dg[8], db[8];
      Vec8<TX> xv;
      Vec8<__half> yv;
      Vec8<TP> gv;
      xv.load(x + row * h + 8 * c);
      yv.load(dy + row * h + 8 * c);
      gv.load(gamma + 8 * c);
      xv.get(xf);
      yv.get(yf);
      gv.get(g);
      Vec8<float> og, ob;
      og.zero();
      ob.zero();
      if (pg && !first) {
        og.load(pg + 8 * c);
        ob.load(pg + h + 8 * c);
      }
      og.get(dg);
      ob.get(db);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (xf[e] - m) * q;
        dg[e] = fmaf(yf[e], xh, dg[e]);
        db[e] += yf[e];
        xf[e] = q * (yf[e] * g[e] - c1 - xh * c2);
      }
      if (pg) {
        store8(pg + 8 * c, dg);
        store8(pg + h + 8 * c, db);
      }
      if (dx) store8(dx + row * h + 8 * c, xf);
    }
  }
}

// dgamma / dbeta = the blocks' partial sums, added in a fixed order: a block
// of 32 columns x 32 lanes of rows, then the lanes in order.
constexpr int RED_COLS = 32;
constexpr int RED_LANES = 32;
__global__ void __launch_bounds__(RED_COLS *RED_LANES)
    k_ln_reduce(const float *__restrict__ part, int32_t blocks, int32_t h,
                float *__restrict__ dgamma, float *__restrict__ dbeta) {
  __shared__ float sg[RED_LANES][RED_COLS + 1];
  grid_dependency_wait();
  const int64_t w = 2 * (int64_t)h;
  const int64_t col = (int64_t)blockIdx.x * RED_COLS + (threadIdx.x & 31);  // of 2h
  const int lane = threadIdx.x >> 5;
  float v = 0.0f;
  if (col < w)
    for (int b = lane; b < blocks; b += RED_LANES) v += part[(int64_t)b * w + col];
  sg[lane][threadIdx.x & 31] = v;
  __syncthreads();
  if (lane == 0 && col < w) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < RED_LANES; ++i) t += sg[i][threadIdx.x];
    if (col < h) {
      if (dgamma) dgamma[col] = t;
    } else if (dbeta) {
      dbeta[col - h] = t;
    }
  }
}

}  // namespace ln
}  // namespace llmint8

// Gradient of an LLM.int8() projection's input, through the frozen int8
// weight:
//
//   dX[i][k] = fp16(base[i][k] + sum_j dY[i][j] * W[k][j]),
//   W[k][j]  = wq[j][k] * aw[j] / 127
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "ptx_sm100.cuh"
#include "rows_common.cuh"

namespace llmint8 {
namespace igrad {

// 64 x 64 output tile per block of 256 threads, 16 output columns of W per
// step, 4 x 4 outputs per thread.
__global__ void __launch_bounds__(256)
    k_input_grad_simple(const __half *dY, int64_t s, int32_t h, int32_t o, const int8_t *wq,
                        const float *aw, const __half *base, __half *dX) {
  __shared__ float sY[16][68];
  __shared__ float sW[16][68];
  const int64_t i0 = (int64_t)blockIdx.y * 64;
  const int k0 = blockIdx.x * 64;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int j0 = 0; j0 < o; j0 += 16) {
    for (int e = threadIdx.x; e < 64 * 16; e += 256) {
      const int64_t i = i0 + e / 16;
      sY[e % 16][e / 16] = i < s ? __half2float(dY[i * o + j0 + e % 16]) : 0.0f;
      const int j = j0 + e / 64, k = k0 + e % 64;
      sW[e / 64][e % 64] = k < h ? (float)wq[(int64_t)j * h + k] * (aw[j] / 127.0f) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      float a[4], b[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        a[u] = sY[j][ty * 4 + u];
        b[u] = sW[j][tx * 4 + u];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int w = 0; w < 4; ++w) acc[u][w] = fmaf(a[u], b[w], acc[u][w]);
    }
    __syncthreads();
  }
  for (int u = 0; u < 4; ++u)
    for (int w = 0; w < 4; ++w) {
      const int64_t i = i0 + ty * 4 + u;
      const int k = k0 + tx * 4 + w;
      if (i < s && k < h) {
        const float b = base ? __half2float(base[i * h + k]) : 0.0f;
        dX[i * h + k] = __float2half_rn(b + acc[u][w]);
      }
    }
}

}  // namespace igrad
}  // namespace llmint8

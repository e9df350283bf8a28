// Device helpers of the row and reduction kernels: typed 8-element vectors and
// block-wide sums in a fixed order.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace llmint8 {

// Eight consecutive elements of a row (16-byte aligned for 16-bit types,
// 32-byte groups of two 16-byte halves for fp32), held as loaded.
template <typename T>
struct Vec8;

template <>
struct Vec8<__half> {
  uint4 q;
  __device__ __forceinline__ void load(const __half *p) { q = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void zero() { q = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
};

template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = *reinterpret_cast<const float4 *>(p);
    b = *reinterpret_cast<const float4 *>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store8(__half *p, const float (&f)[8]) {
  *reinterpret_cast<uint4 *>(p) = pack8(f);
}

__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
  *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Sum over the block, returned to every thread. `red` holds one word per
// warp and is not reused before the next barrier of the caller.
__device__ __forceinline__ float block_sum(float v, float *red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int nw = blockDim.x >> 5;
  float t = (int)(threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.0f;
  return warp_sum(t);
}

// Two sums at once, and whether `pred` holds in any thread.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2 *red, bool pred, bool *any) {
  a = warp_sum(a);
  b = warp_sum(b);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
  *any = __syncthreads_or(pred);
  const int nw = blockDim.x >> 5;
  const float2 t = (int)(threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : make_float2(0.f, 0.f);
  return make_float2(warp_sum(t.x), warp_sum(t.y));
}

__device__ __forceinline__ float2 block_sum2(float a, float b, float2 *red) {
  bool any;
  return block_sum2(a, b, red, false, &any);
}

}  // namespace llmint8

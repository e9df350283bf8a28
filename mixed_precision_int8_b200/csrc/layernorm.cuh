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
// Bound: bytes. A row is read once and kept in registers (forward; NV vectors
// of eight elements per thread) or shared memory (backward) between the sums
// and the store; rows too long for that are re-read from L2 by the *_long
// kernels. y may be x, and dx may be x or dy: every read of an element comes
// before its write, and none of these pointers is __restrict__.
#pragma once

#include <cstdint>

#include "ptx_finetune_sm100.cuh"
#include "rows_common.cuh"

namespace llmint8 {
namespace ln {

constexpr int MAX_THREADS = 512;
constexpr int MAX_VEC = 4;                            // vectors of 8 per thread
constexpr int64_t MAX_ROW = 8LL * MAX_VEC * MAX_THREADS;  // longest row held in registers

template <typename TX, typename TP, int NV>
__global__ void __launch_bounds__(MAX_THREADS)
    k_ln_forward(const TX *x, int32_t h, const TP *__restrict__ gamma,
                 const TP *__restrict__ beta, float eps, __half *y,
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
    k_ln_forward_long(const TX *x, int32_t h, const TP *__restrict__ gamma,
                      const TP *__restrict__ beta, float eps, __half *y,
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

// Backward: block b takes groups of RB rows b, b + grid, ..., which bulk
// copies bring into a ring in shared memory ahead of their use; each thread
// owns NU units of 16 bytes' worth of x's columns and keeps their gamma and
// dgamma / dbeta sums in registers over the block's rows, so the column sums
// cost one write of `part` (fp32 [grid][2][h]) per block. k_ln_reduce adds
// those in block order. What is left beside the bytes is a row's latency (two
// sums over the block): two rows share it where two and a ring of them fit,
// the next rows' statistics are loaded ahead, and the arithmetic is in packed
// pairs of fp32.
constexpr int BW_MAX_STAGES = 8;

// 16 bytes of x, and as many elements of another row or of gamma, from global
// or shared memory, as packed pairs.
template <int P>
__device__ __forceinline__ void pairs_of(const float *p, uint64_t (&f)[P]) {
#pragma unroll
  for (int i = 0; i < P; i += 2) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(p + 2 * i);
    f[i] = a.x;
    f[i + 1] = a.y;
  }
}
template <int P>
__device__ __forceinline__ void pairs_of(const __half *p, uint64_t (&f)[P]) {
  uint32_t w[P];
  if constexpr (P == 4) {
    const uint4 q = *reinterpret_cast<const uint4 *>(p);
    w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
  } else {
    const uint2 q = *reinterpret_cast<const uint2 *>(p);
    w[0] = q.x; w[1] = q.y;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    f[i] = f32x2_pack(v.x, v.y);
  }
}
__device__ __forceinline__ void store_pairs(float *p, const uint64_t *f, int pairs) {
#pragma unroll
  for (int i = 0; i < 4; i += 2)
    if (i < pairs)
      *reinterpret_cast<float4 *>(p + 2 * i) =
          make_float4(f32x2_lo(f[i]), f32x2_hi(f[i]), f32x2_lo(f[i + 1]), f32x2_hi(f[i + 1]));
}

template <typename TX, typename TP, int NU, int RB>
__global__ void __launch_bounds__(MAX_THREADS, NU * (int)(16 / sizeof(TX)) <= 8 ? 2 : 1)
    k_ln_backward(const __half *dy, const TX *x, int64_t s, int32_t h,
                  int32_t stages, const TP *__restrict__ gamma, const float *__restrict__ mean,
                  const float *__restrict__ rstd, TX *dx, float *__restrict__ part,
                  int32_t *status, uint64_t timeout_ns) {
  constexpr int U = 16 / (int)sizeof(TX), P = U / 2;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float2 red[2][RB][MAX_THREADS / 32];
  __shared__ uint64_t bars[BW_MAX_STAGES];
  __shared__ int abort_word;
  volatile int *abort_flag = &abort_word;
  grid_dependency_trigger();
  const int units = h / U;
  const uint32_t xbytes = RB * (uint32_t)h * sizeof(TX), stage_bytes = xbytes + 2 * RB * (uint32_t)h;
  const uint32_t bar0 = smem_u32(bars);
  const int64_t step = (int64_t)gridDim.x * RB;
  auto load_rows = [&](int64_t row, int st) {
    const uint32_t rows = (uint32_t)min((int64_t)RB, s - row);
    const uint32_t dst = smem_u32(ring) + st * stage_bytes;
    mbar_arrive_expect_tx(bar0 + 8u * st, rows * (uint32_t)h * (sizeof(TX) + 2));
    bulk_load_1d(dst, x + row * h, rows * (uint32_t)h * sizeof(TX), bar0 + 8u * st);
    bulk_load_1d(dst + xbytes, dy + row * h, rows * 2 * (uint32_t)h, bar0 + 8u * st);
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(bar0 + 8u * i, 1);
    abort_word = 0;
    fence_mbar_init();
    for (int i = 0; i < stages; ++i)
      if (blockIdx.x * (int64_t)RB + i * step < s) load_rows(blockIdx.x * (int64_t)RB + i * step, i);
  }
  __syncthreads();
  uint64_t g2[NU][P], dg[NU][P], db[NU][P];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
#pragma unroll
    for (int e = 0; e < P; ++e) g2[i][e] = dg[i][e] = db[i][e] = 0ull;
    if (c < units) pairs_of<P>(gamma + U * c, g2[i]);
  }
  const float inv_h = 1.0f / (float)h;
  int st = 0, prev = -1, par = 0;
  uint32_t phase = 0;
  float m[RB], q[RB];
  auto load_stats = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      m[k] = row + k < s ? mean[row + k] : 0.0f;
      q[k] = row + k < s ? rstd[row + k] : 0.0f;
    }
  };
  load_stats(blockIdx.x * (int64_t)RB);
  for (int64_t row = blockIdx.x * (int64_t)RB; row < s; row += step, par ^= 1) {
    const int rows = (int)min((int64_t)RB, s - row);
    // the rows' copies, or an abort of the whole block
    const bool ok = mbar_wait_bounded(bar0 + 8u * st, phase, abort_flag, status,
                                      LLMINT8_DEV_TIMEOUT_ROWS, timeout_ns);
    const TX *xs = reinterpret_cast<const TX *>(ring + st * stage_bytes);
    const __half *ys = reinterpret_cast<const __half *>(ring + st * stage_bytes + xbytes);
    uint64_t q2[RB], m2[RB];
    float a[RB], b[RB];
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      q2[k] = f32x2_pack(q[k], q[k]);
      m2[k] = f32x2_pack(-m[k], -m[k]);
      uint64_t a2 = 0ull, b2 = 0ull;
      if (k < rows) {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          const int c = threadIdx.x + i * blockDim.x;
          if (c >= units) continue;
          uint64_t xf[P], yf[P];
          pairs_of<P>(xs + k * h + U * c, xf);
          pairs_of<P>(ys + k * h + U * c, yf);
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const uint64_t xh = f32x2_mul(f32x2_add(xf[e], m2[k]), q2[k]);
            const uint64_t gg = f32x2_mul(yf[e], g2[i][e]);
            dg[i][e] = f32x2_fma(yf[e], xh, dg[i][e]);
            db[i][e] = f32x2_add(db[i][e], yf[e]);
            a2 = f32x2_add(a2, gg);
            b2 = f32x2_fma(gg, xh, b2);
          }
        }
      }
      a[k] = f32x2_lo(a2) + f32x2_hi(a2);
      b[k] = f32x2_lo(b2) + f32x2_hi(b2);
    }
    load_stats(row + step);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
      for (int k = 0; k < RB; ++k) {
        a[k] += __shfl_xor_sync(0xffffffffu, a[k], d);
        b[k] += __shfl_xor_sync(0xffffffffu, b[k], d);
      }
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < RB; ++k) red[par][k][threadIdx.x >> 5] = make_float2(a[k], b[k]);
    // (every thread gets here, whatever its wait said)
    if (__syncthreads_or(!ok)) break;
    // all threads are past the previous rows: their slot takes the next ones
    if (threadIdx.x == 0 && prev >= 0 && row + (stages - 1) * step < s)
      load_rows(row + (stages - 1) * step, prev);
    if (dx) {
#pragma unroll
      for (int k = 0; k < RB; ++k) {
        if (k >= rows) break;
        float c1 = 0.0f, c2 = 0.0f;
        for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
          const float2 t = red[par][k][w];
          c1 += t.x;
          c2 += t.y;
        }
        c1 *= -inv_h;
        c2 *= -inv_h;
        const uint64_t k1 = f32x2_pack(c1, c1), k2 = f32x2_pack(c2, c2);
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          const int c = threadIdx.x + i * blockDim.x;
          if (c >= units) continue;
          uint64_t xf[P], yf[P], d[P];
          pairs_of<P>(xs + k * h + U * c, xf);
          pairs_of<P>(ys + k * h + U * c, yf);
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const uint64_t xh = f32x2_mul(f32x2_add(xf[e], m2[k]), q2[k]);
            d[e] = f32x2_mul(q2[k], f32x2_fma(xh, k2, f32x2_fma(yf[e], g2[i][e], k1)));
          }
          TX *to = dx + (row + k) * h + U * c;
          if constexpr (U == 4) {
            store_pairs(to, d, P);
          } else {
            float o[8];
#pragma unroll
            for (int e = 0; e < P; ++e) {
              o[2 * e] = f32x2_lo(d[e]);
              o[2 * e + 1] = f32x2_hi(d[e]);
            }
            store8(to, o);
          }
        }
      }
    }
    prev = st;
    if (++st == stages) {
      st = 0;
      phase ^= 1u;
    }
  }
  if (*abort_flag) {  // copies in flight land before shared memory goes
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 200000u) __nanosleep(1000);
    return;
  }
  if (!part) return;
  float *pg = part + (int64_t)blockIdx.x * 2 * h;
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c >= units) continue;
    store_pairs(pg + U * c, dg[i], P);
    store_pairs(pg + h + U * c, db[i], P);
  }
}

// Rows longer than MAX_ROW: the row is read twice, the column sums live in
// this block's slice of `part`.
template <typename TX, typename TP>
__global__ void __launch_bounds__(MAX_THREADS)
    k_ln_backward_long(const __half *dy, const TX *x, int64_t s,
                       int32_t h, const TP *__restrict__ gamma, const float *__restrict__ mean,
                       const float *__restrict__ rstd, TX *dx,
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

// dgamma / dbeta = the blocks' partial sums, added in a fixed order: 32
// threads of four columns each by 32 lanes of blocks, then the lanes in order.
// (part is still being written when this kernel starts: not __restrict__, so
// that no read of it can move before the wait.)
constexpr int RED_COLS = 128;
constexpr int RED_LANES = 32;
__global__ void __launch_bounds__(RED_COLS / 4 * RED_LANES)
    k_ln_reduce(const float *part, int32_t blocks, int32_t h,
                float *__restrict__ dgamma, float *__restrict__ dbeta) {
  __shared__ float4 sums[RED_LANES][RED_COLS / 4];
  grid_dependency_wait();
  const int64_t w = 2 * (int64_t)h;
  const int64_t col = (int64_t)blockIdx.x * RED_COLS + (threadIdx.x & 31) * 4;  // of 2 h
  const int lane = threadIdx.x >> 5;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < w) {
#pragma unroll 4
    for (int b = lane; b < blocks; b += RED_LANES) {
      const float4 p = *reinterpret_cast<const float4 *>(part + (int64_t)b * w + col);
      v.x += p.x;
      v.y += p.y;
      v.z += p.z;
      v.w += p.w;
    }
  }
  sums[lane][threadIdx.x & 31] = v;
  __syncthreads();
  if (threadIdx.x < RED_COLS) {
    const int64_t c = (int64_t)blockIdx.x * RED_COLS + threadIdx.x;
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < RED_LANES; ++i)
      t += reinterpret_cast<const float *>(&sums[i][0])[threadIdx.x];
    if (c < h) {
      if (dgamma) dgamma[c] = t;
    } else if (c < w && dbeta) {
      dbeta[c - h] = t;
    }
  }
}

}  // namespace ln
}  // namespace llmint8

// The global norm of the gradients of many tensors, and clipping to it:
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   coef = min(1, max_norm / (norm + 1e-6))       out = g * coef
//
// Bound: bytes. The list of tensors is laid out once, on the device, as a
// table of entries with the running number of chunks (CHUNK_BYTES) before
// each. The chunks of all tensors are cut into equal contiguous ranges, one per
// block, so thousands of small tensors and a few large ones load the GPU
// alike; the table also holds the entry in which each range starts (a search
// for it in the kernel took 4 us of 256 entries). The norm kernel leaves one fp64 partial sum per block; the
// scaling kernel's blocks each add those partial sums in the same order, so
// the result does not depend on timing, and walk their ranges from the end.
// The norm kernel reads the last KEPT_CHUNKS of all ranges with the default L2
// policy and what lies before as data not needed again, as the scaling kernel
// does all it reads and writes: so those ends are still in L2 when it comes to
// them. Measured: 16 tensors of 420 MB (fp16) in 221 us, 229 with ranges walked
// forwards and no policy (5.7 TB/s over two reads and a write; the bytes alone
// 192 us), 233 backwards without the policy; 256 tensors of 67 MB (fp32) 40 us
// instead of 43. Chunks of 32 KB instead of 16: 233 and 43 us.
//
// Sums are fp64. The squares of a 16-byte vector are added in fp32 first
// (converting every element to fp64 took twice as long as its bytes), unless
// that sum shows that fp32 does not hold them: the square of an fp32 or bf16
// gradient above 2^64 or below 2^-75 has no fp32 value, and such vectors are
// squared in fp64.
#pragma once

#include <cstdint>

#include "ptx_finetune_sm100.cuh"
#include "rows_common.cuh"

namespace llmint8 {
namespace clip {

constexpr int THREADS = 512;
constexpr int CHUNK_BYTES = 16384;  // two vectors of 16 bytes per thread
constexpr int KEPT_CHUNKS = 5120;  // 80 MB of the 126 MB of L2
constexpr int MAX_BLOCKS = 1024;   // partial sums a list holds
constexpr int INIT_ENTRIES = 48;   // entries one launch of k_list_init carries
constexpr int INIT_STARTS = 512;   // range starts one launch of k_starts_init carries

struct Entry {
  const void *grad;
  void *out;
  int64_t n;
  int64_t chunk0;  // chunks of the tensors before this one
  int32_t type;
  int32_t pad;
};

// The table: MAX_BLOCKS partial sums, the blocks' first entries, the entries.
constexpr size_t kStartsOffset = MAX_BLOCKS * sizeof(double);
constexpr size_t kEntriesOffset = kStartsOffset + MAX_BLOCKS * sizeof(int32_t);

// Chunks [first, last) of block b of `blocks`.
__host__ __device__ inline int64_t range_start(int64_t chunks, int64_t b, int64_t blocks) {
  return chunks * b / blocks;
}

struct InitBatch {
  Entry e[INIT_ENTRIES];
};

__global__ void k_list_init(Entry *table, const __grid_constant__ InitBatch batch, int32_t n) {
  const int i = threadIdx.x;
  if (i < n) table[i] = batch.e[i];
}

struct StartBatch {
  int32_t first[INIT_STARTS];
};

__global__ void k_starts_init(int32_t *starts, const __grid_constant__ StartBatch batch,
                              int32_t n) {
  const int i = threadIdx.x;
  if (i < n) starts[i] = batch.first[i];
}

// Elements of a chunk of a type.
__host__ __device__ inline int chunk_elements(int32_t type) {
  return CHUNK_BYTES / (type == LLMINT8_F32 ? 4 : 2);
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float &d, float v) { d = v; }
__device__ __forceinline__ void from_f(__half &d, float v) { d = __float2half_rn(v); }
__device__ __forceinline__ void from_f(__nv_bfloat16 &d, float v) { d = __float2bfloat16_rn(v); }

template <typename T>
struct Pack {
  static constexpr int N = 16 / sizeof(T);
  union {
    uint4 q;
    T v[N];
  };
  __device__ __forceinline__ Pack() {}
};

// Sum of squares of one 16-byte vector. A sum between 2^-80 and 2^120 has lost
// at most its last bits: every square that matters to it is a normal number
// (one below 2^-126 is below 2^-46 of it), and none overflowed.
template <typename T>
__device__ __forceinline__ double vector_square_sum(const Pack<T> &p) {
  constexpr int N = Pack<T>::N;
  float f = 0.0f;
#pragma unroll
  for (int e = 0; e < N; ++e) f = fmaf(to_f(p.v[e]), to_f(p.v[e]), f);
  if (f > 8.2718061e-25f && f < 1.329228e36f) return (double)f;
  double acc = 0.0;
  if ((p.q.x | p.q.y | p.q.z | p.q.w) != 0) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const double d = (double)to_f(p.v[e]);
      acc = fma(d, d, acc);
    }
  }
  return acc;
}

// Sum of squares of elements [0, m) of g, at most a chunk; `again`: it should
// stay in L2.
template <typename T>
__device__ __forceinline__ double chunk_square_sum(const T *g, int m, bool again) {
  double acc = 0.0;
  constexpr int N = Pack<T>::N;
  constexpr int PER = CHUNK_BYTES / 16 / THREADS;  // vectors per thread in a full chunk
  int done = 0;
  if ((reinterpret_cast<uintptr_t>(g) & 15) == 0) {
    const int nv = m / N;
    if (nv == PER * THREADS) {
      Pack<T> p[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const uint4 *q = reinterpret_cast<const uint4 *>(g) + threadIdx.x + i * THREADS;
        p[i].q = again ? __ldg(q) : __ldcs(q);
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) acc += vector_square_sum(p[i]);
    } else {
      for (int i = threadIdx.x; i < nv; i += THREADS) {
        Pack<T> p;
        p.q = __ldg(reinterpret_cast<const uint4 *>(g) + i);
        acc += vector_square_sum(p);
      }
    }
    done = nv * N;
  }
  for (int i = done + threadIdx.x; i < m; i += THREADS) {
    const double d = (double)to_f(g[i]);
    acc = fma(d, d, acc);
  }
  return acc;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T *g, T *out, int m, float coef) {
  constexpr int N = Pack<T>::N;
  int done = 0;
  if (((reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(out)) & 15) == 0) {
    constexpr int PER = CHUNK_BYTES / 16 / THREADS;
    const int nv = m / N;
    if (nv == PER * THREADS) {
      Pack<T> p[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i)
        p[i].q = __ldcs(reinterpret_cast<const uint4 *>(g) + threadIdx.x + i * THREADS);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
#pragma unroll
        for (int e = 0; e < N; ++e) from_f(p[i].v[e], to_f(p[i].v[e]) * coef);
        __stcs(reinterpret_cast<uint4 *>(out) + threadIdx.x + i * THREADS, p[i].q);
      }
    } else {
      for (int i = threadIdx.x; i < nv; i += THREADS) {
        Pack<T> p;
        p.q = reinterpret_cast<const uint4 *>(g)[i];
#pragma unroll
        for (int e = 0; e < N; ++e) from_f(p.v[e], to_f(p.v[e]) * coef);
        reinterpret_cast<uint4 *>(out)[i] = p.q;
      }
    }
    done = nv * N;
  }
  for (int i = done + threadIdx.x; i < m; i += THREADS) from_f(out[i], to_f(g[i]) * coef);
}

__global__ void __launch_bounds__(THREADS)
    k_square_sums(const Entry *__restrict__ table, int64_t n, int64_t chunks,
                  const int32_t *__restrict__ starts, double *__restrict__ partial) {
  __shared__ double red[32];
  grid_dependency_trigger();
  const int64_t c0 = range_start(chunks, blockIdx.x, gridDim.x);
  const int64_t c1 = range_start(chunks, blockIdx.x + 1, gridDim.x);
  const int64_t kept = c1 - KEPT_CHUNKS / gridDim.x;
  double acc = 0.0;
  int64_t t = starts[blockIdx.x];
  for (int64_t c = c0; c < c1; ++c) {
    while (t + 1 < n && table[t + 1].chunk0 <= c) ++t;
    const Entry e = table[t];
    const int full = chunk_elements(e.type);
    const int64_t at = (c - e.chunk0) * full;
    const int m = (int)(e.n - at < full ? e.n - at : full);
    if (e.type == LLMINT8_F16)
      acc += chunk_square_sum(static_cast<const __half *>(e.grad) + at, m, c >= kept);
    else if (e.type == LLMINT8_BF16)
      acc += chunk_square_sum(static_cast<const __nv_bfloat16 *>(e.grad) + at, m, c >= kept);
    else
      acc += chunk_square_sum(static_cast<const float *>(e.grad) + at, m, c >= kept);
  }
  acc = warp_sum(acc);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x < 32) {
    const double v = warp_sum((int)threadIdx.x < THREADS / 32 ? red[threadIdx.x] : 0.0);
    if (threadIdx.x == 0) partial[blockIdx.x] = v;
  }
}

// (partial is still being written when this kernel starts: not __restrict__, so
// that no read of it can move before the wait.)
__global__ void __launch_bounds__(THREADS)
    k_clip_scale(const Entry *__restrict__ table, int64_t n, int64_t chunks,
                 const int32_t *__restrict__ starts, const double *partial,
                 int32_t n_partial, float max_norm, float *__restrict__ norm_out) {
  __shared__ double red[32];
  __shared__ float s_coef;
  grid_dependency_wait();
  double acc = 0.0;
  for (int i = threadIdx.x; i < n_partial; i += THREADS) acc += partial[i];
  acc = warp_sum(acc);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x < 32) {
    const double v = warp_sum((int)threadIdx.x < THREADS / 32 ? red[threadIdx.x] : 0.0);
    if (threadIdx.x == 0) {
      const double norm = sqrt(v);
      const double c = (double)max_norm / (norm + 1e-6);
      // max_norm = inf asks for the norm alone; a NaN norm gives a NaN coefficient
      s_coef = c > 1.0 || isinf(max_norm) ? 1.0f : (float)c;
      if (blockIdx.x == 0) *norm_out = (float)norm;
    }
  }
  __syncthreads();
  const float coef = s_coef;
  // from the end of the range
  const int64_t c0 = range_start(chunks, blockIdx.x, gridDim.x);
  const int64_t c1 = range_start(chunks, blockIdx.x + 1, gridDim.x);
  if (c0 == c1) return;
  int64_t t = blockIdx.x + 1 < gridDim.x ? starts[blockIdx.x + 1] : n - 1;
  for (int64_t c = c1 - 1; c >= c0; --c) {
    while (table[t].chunk0 > c) --t;
    const Entry e = table[t];
    if (coef == 1.0f && e.out == e.grad) continue;  // nothing to change in place
    const int full = chunk_elements(e.type);
    const int64_t at = (c - e.chunk0) * full;
    const int m = (int)(e.n - at < full ? e.n - at : full);
    if (e.type == LLMINT8_F16)
      chunk_scale(static_cast<const __half *>(e.grad) + at, static_cast<__half *>(e.out) + at, m,
                  coef);
    else if (e.type == LLMINT8_BF16)
      chunk_scale(static_cast<const __nv_bfloat16 *>(e.grad) + at,
                  static_cast<__nv_bfloat16 *>(e.out) + at, m, coef);
    else
      chunk_scale(static_cast<const float *>(e.grad) + at, static_cast<float *>(e.out) + at, m,
                  coef);
  }
}

}  // namespace clip
}  // namespace llmint8

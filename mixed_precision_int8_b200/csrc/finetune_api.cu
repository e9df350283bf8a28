// C ABI of the operators next to the projection (declared in
// include/llmint8.h): low-rank adapters, the gradient of the projection's
// input, layer norm and gradient clipping. Argument validation, workspace
// layout and launches; host code only enqueues work and never allocates
// device memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <mutex>
#include <vector>

#include "llmint8.h"
#include "finetune_host.cuh"
#include "adapters.cuh"
#include "adapters_sm100.cuh"
#include "grad_clip.cuh"
#include "input_grad_sm100.cuh"
#include "layernorm.cuh"

namespace {

using namespace llmint8;

template <typename TX, typename TP>
bool ln_backward_setup();

auto shrink_kernel(int32_t r) {
  return r <= 16   ? lora::k_shrink<2>
         : r <= 32 ? lora::k_shrink<4>
         : r <= 64 ? lora::k_shrink<8>
                   : lora::k_shrink<16>;
}

bool shrink_setup(cudaFuncAttribute attr, int value) {
  for (int32_t r : {16, 32, 64, 128})
    if (cudaFuncSetAttribute(shrink_kernel(r), attr, value) != cudaSuccess) return false;
  return true;
}

auto input_grad_kernel(int32_t mt, bool base) {
  return mt == 1 ? (base ? igrad::k_input_grad<1, true> : igrad::k_input_grad<1, false>)
                 : (base ? igrad::k_input_grad<2, true> : igrad::k_input_grad<2, false>);
}

size_t input_grad_smem(int32_t mt) {
  return mt == 1 ? igrad::Smem<1>::BYTES : igrad::Smem<2>::BYTES;
}

bool input_grad_setup() {
  for (int32_t mt : {1, 2})
    for (bool base : {false, true})
      if (cudaFuncSetAttribute(input_grad_kernel(mt, base),
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)input_grad_smem(mt)) != cudaSuccess)
        return false;
  return true;
}

struct Device {
  bool init = false;
  bool supported = false;
  int sm_count = 0;
  int max_pairs = 0;  // CTA pairs of k_input_grad that fit at once
  int shrink_split = 8;  // CTAs of a k_shrink cluster: 16 where the device runs such
};
Device g_device[kMaxDevices];
std::mutex g_device_mutex;

llmint8_status current_device(Device **out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return LLMINT8_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_device_mutex);
  Device &d = g_device[dev];
  if (!d.init) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return LLMINT8_ERR_CUDA;
    d.supported = major == 10 && minor == 0;
    if (d.supported) {
      if (!input_grad_setup() ||
          !shrink_setup(cudaFuncAttributeMaxDynamicSharedMemorySize, (int)lora::SMEM_LIMIT) ||
          cudaFuncSetAttribute(lora::k_expand, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)lora::SMEM_LIMIT) != cudaSuccess ||
          cudaFuncSetAttribute(lora::k_outer<2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)lora::SMEM_LIMIT) != cudaSuccess ||
          cudaFuncSetAttribute(lora::k_outer<4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)lora::SMEM_LIMIT) != cudaSuccess ||
          cudaFuncSetAttribute(lora::k_outer<8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)lora::SMEM_LIMIT) != cudaSuccess ||
          cudaFuncSetAttribute(lora::k_outer<16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)lora::SMEM_LIMIT) != cudaSuccess ||
          !ln_backward_setup<__half, __half>() || !ln_backward_setup<__half, float>() ||
          !ln_backward_setup<float, __half>() || !ln_backward_setup<float, float>())
        return LLMINT8_ERR_CUDA;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2 * (unsigned)(d.sm_count / 2));
      cfg.blockDim = dim3(igrad::NUM_THREADS);
      cfg.dynamicSmemBytes = igrad::Smem<2>::BYTES;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int clusters = 0;
      if (cudaOccupancyMaxActiveClusters(&clusters, igrad::k_input_grad<2, true>, &cfg) != cudaSuccess ||
          clusters < 1)
        return LLMINT8_ERR_CUDA;
      d.max_pairs = std::min({clusters, d.sm_count / 2, igrad::MAX_PAIRS});
      cfg.gridDim = dim3(lora::SH_MAX_SPLIT);
      cfg.blockDim = dim3(lora::SH_THREADS);
      cfg.dynamicSmemBytes = lora::SMEM_LIMIT;
      attr[0].val.clusterDim.x = lora::SH_MAX_SPLIT;
      if (shrink_setup(cudaFuncAttributeNonPortableClusterSizeAllowed, 1) &&
          cudaOccupancyMaxActiveClusters(&clusters, lora::k_shrink<16>, &cfg) == cudaSuccess &&
          clusters > 0)
        d.shrink_split = lora::SH_MAX_SPLIT;
      else
        (void)cudaGetLastError();
    }
    d.init = true;
  }
  if (!d.supported) return LLMINT8_ERR_UNSUPPORTED;
  *out = &d;
  return LLMINT8_OK;
}

// Row indices, rounded up to whole tiles, stay 32-bit numbers.
constexpr int64_t kMaxRows = (int64_t)INT32_MAX - 1023;

llmint8_status check_rows(int64_t s) {
  return s < 0 || s > kMaxRows ? LLMINT8_ERR_SHAPE : LLMINT8_OK;
}

llmint8_status check_width(int64_t h) {
  return h < 16 || h > kMaxH || (h % 16) != 0 ? LLMINT8_ERR_SHAPE : LLMINT8_OK;
}

unsigned blocks_for(int64_t work, int64_t per_block) {
  return (unsigned)((work + per_block - 1) / per_block);
}

// Whether [p, p + pn) and [q, q + qn) share a byte.
bool overlap(const void *p, size_t pn, const void *q, size_t qn) {
  if (!p || !q || pn == 0 || qn == 0) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + qn && b < a + pn;
}

struct Span {
  const void *p;
  size_t n;
};

// Whether `out` shares a byte with any of these tensors.
bool overlaps_any(Span out, std::initializer_list<Span> others) {
  for (const Span &t : others)
    if (overlap(out.p, out.n, t.p, t.n)) return true;
  return false;
}

// Whether `out` overlaps `in` without being the same tensor.
bool overlaps_partly(Span out, Span in) {
  return (out.p != in.p || out.n != in.n) && overlap(out.p, out.n, in.p, in.n);
}

// ------------------------------------------------------------- adapters

// The row kernels (adapters.cuh) take batches of at most one tile of rows while
// their work, s r (h + o), is small: it costs them time in proportion, and the
// tensor-core kernels, whose time it hardly changes, a pass per adapter held.
// Backward they also sum an adapter's rows one after another. Rows against
// tensor cores, us: 12288 -> 20480, rank 64, forward, one adapter 15 against 17
// at 32 rows, 22 against 18 at 48; four 22 against 25 at 48, 35 against 27 at
// 96; sixteen 54 against 62 at 128; backward, one 34 against 37 at 48, 43
// against 37 at 64; four 56 against 58 at 96, 71 against 57 at 128. 4096 ->
// 4096, rank 16, one adapter at 128 rows: forward 7 against 12, backward 27
// against 21 (17 against 18 at 64). Every adapter held was in those batches;
// which of them a batch uses is known on the device only, so that 128 rows of
// one of 64 adapters held take the row kernels too (forward 47 us, 23 if it is
// held alone). Widths leave at most kRowMaxSlices partial sums of a row.
constexpr int64_t kRowMaxSlices = 256;

bool use_row_kernels(int64_t s, const llmint8_adapters *ad, bool backward) {
  if (s > lora::RO_MAX_ROWS || std::max(ad->h, ad->o) > kRowMaxSlices * lora::RS_SLICE)
    return false;
  const int64_t n = ad->n, work = s * ad->r * (ad->h + ad->o);
  return backward ? s <= 64 * n && work <= (80 + 24 * n) << 20 : work <= (64 + 16 * n) << 20;
}

struct AdapterLayout {
  size_t v, g, vmax, gmax, amax, part, info, vpack, gpack, end;
};

int64_t row_slices(int64_t h) { return (h + lora::RS_SLICE - 1) / lora::RS_SLICE; }

AdapterLayout adapter_layout(int64_t s, int64_t h, int64_t o, int32_t n, int32_t r) {
  AdapterLayout L;
  const size_t sr = 4 * (size_t)s * r, s1 = 4 * (size_t)s;
  const size_t blocks = (size_t)((s + lora::OU_KB - 1) / lora::OU_KB);
  const size_t packed = blocks * lora::outer_p_bytes(r);
  L.v = kStateBytes;
  L.g = align256(L.v + sr);
  L.vmax = align256(L.g + sr);
  L.gmax = align256(L.vmax + s1);
  L.amax = align256(L.gmax + s1);  // [2][n]: v's, g's
  L.part = align256(L.amax + 8 * (size_t)n);
  const int64_t slices = std::min(row_slices(std::max(h, o)), kRowMaxSlices);
  L.info =
      align256(L.part + 4 * (size_t)(slices * std::min<int64_t>(s, lora::RO_MAX_ROWS)) * r);
  L.vpack = align256(L.info + 4 * blocks);
  L.gpack = align256(L.vpack + packed);
  L.end = align256(L.gpack + packed);
  return L;
}

llmint8_status check_adapter_sizes(int64_t s, int64_t h, int64_t o, int32_t n, int32_t r) {
  llmint8_status rc = check_hw(h, o);
  if (rc) return rc;
  if (n < 1 || n > 65535 || r < 8 || r > lora::MAX_R || r % 8 != 0) return LLMINT8_ERR_SHAPE;
  return check_rows(s);
}

llmint8_status check_adapters(const llmint8_adapters *ad, int64_t s) {
  if (!ad || !ad->a_dev || !ad->b_dev || !ad->scale_dev) return LLMINT8_ERR_NULL;
  llmint8_status rc = check_adapter_sizes(s, ad->h, ad->o, ad->n, ad->r);
  if (rc) return rc;
  if (!aligned(ad->a_dev, 16) || !aligned(ad->b_dev, 16) || !aligned(ad->scale_dev, 4) ||
      !aligned(ad->rank_dev, 4))
    return LLMINT8_ERR_ALIGN;
  return LLMINT8_OK;
}

Span factor_a(const llmint8_adapters *ad) {
  return {ad->a_dev, 2 * (size_t)ad->n * ad->r * ad->h};
}
Span factor_b(const llmint8_adapters *ad) {
  return {ad->b_dev, 2 * (size_t)ad->n * ad->r * ad->o};
}

const __half *as_half(const uint16_t *p) { return reinterpret_cast<const __half *>(p); }
__half *as_half(uint16_t *p) { return reinterpret_cast<__half *>(p); }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// v = X . F1^T over k features (kept in v_out, or null) and, unless out is
// null, out = base + scale * v . F2 over w features, by the row kernels.
llmint8_status enqueue_rows(const uint16_t *X, int64_t s, int64_t k, const uint16_t *F1, int64_t w,
                            const uint16_t *F2, const llmint8_adapters *ad, const int32_t *ids,
                            const uint16_t *base, uint16_t *out, float *v_out, float *part,
                            cudaStream_t st) {
  const int64_t slices = row_slices(k);
  if (launch(lora::k_rows_shrink, dim3((unsigned)slices, (unsigned)s), dim3(lora::RS_THREADS), 0,
             st, false, as_half(X), (int32_t)s, (int32_t)k, as_half(F1), ids, ad->rank_dev, ad->n,
             ad->r, part) != cudaSuccess ||
      launch(lora::k_rows_expand,
             dim3(out ? (unsigned)ceil_div(w, lora::RE_SLICE) : 1u, (unsigned)s),
             dim3(lora::RE_THREADS), 0, st, true, (const float *)part, (int32_t)slices, (int32_t)s,
             (int32_t)w, as_half(F2), ids, ad->scale_dev, ad->rank_dev, ad->n, ad->r,
             as_half(base), as_half(out), v_out) != cudaSuccess)
    return LLMINT8_ERR_CUDA;
  return LLMINT8_OK;
}

// How k_shrink's work is cut: CTAs of a cluster (over the features), clusters
// of a row tile (over the passes that mixed rows take).
struct ShrinkGrid {
  int split, y;
};

// Powers of two up to 8 CTAs per cluster that leave every CTA its place, then
// clusters for the passes, then clusters of 16 if there is still room (whole
// forward calls, 1000 rows of 16 adapters, rank 64, 12288 -> 12288: 80 us with 8
// CTAs and one cluster, 57 with 8 and 4, 61 with 16 and 2; 200 rows of one
// adapter, rank 64, 11456 -> 1104: 22 us with 8, 18 with 16). A pass of fewer
// than eight stages is over sooner than another cluster's start (221 rows of 5
// adapters, rank 16, 768 -> 768: 15.0 us, 15.6 with 2).
ShrinkGrid shrink_grid(int64_t s, int64_t k, const llmint8_adapters *ad, int n_jobs,
                       const Device &dev) {
  const int64_t room = (ad->r <= 64 ? 2 : 1) * dev.sm_count;  // two CTAs per SM up to r = 64
  const int64_t tiles = n_jobs * ceil_div(s, lora::TM);
  const int64_t limit = std::min<int64_t>(dev.shrink_split, ceil_div(k, 2 * lora::SH_KB));
  ShrinkGrid g = {1, 1};
  while (2 * g.split <= std::min<int64_t>(limit, 8) && tiles * 2 * g.split <= room) g.split *= 2;
  const int64_t passes =
      ceil_div(std::min<int64_t>(ad->n, lora::TM), lora::shrink_slots(ad->r));
  if (ceil_div(k, lora::SH_KB) >= 8 * g.split)
    g.y = (int)std::max<int64_t>(1, std::min(passes, room / (tiles * g.split)));
  if (g.split == 8 && limit >= 16 && tiles * 16 * g.y <= room) g.split = 16;
  return g;
}

// Shared memory of a CTA when an SM holds two.
constexpr uint32_t kHalfSmem = 113 * 1024;

// v = X . F^T with the largest values per row and per adapter (amax, or
// null); w, w_amax: another [s][r] array's per adapter.
bool shrink_job(lora::ShrinkJob *job, const uint16_t *X, int64_t s, int64_t k, const uint16_t *F,
                const llmint8_adapters *ad, const int32_t *ids, float *v, float *vmax,
                uint32_t *amax, const float *w, uint32_t *w_amax, int split, void *ws) {
  lora::ShrinkParams &p = job->p;
  p.s = (int32_t)s;
  p.k = (int32_t)k;
  p.n = ad->n;
  p.r = ad->r;
  p.split = split;
  p.slots = lora::shrink_slots(ad->r);
  p.stage_bytes = lora::shrink_stage_bytes(ad->r);
  // two CTAs per SM (four stages in half of its shared memory) up to r = 64,
  // one above
  const uint32_t limit = ad->r <= 64 ? kHalfSmem : lora::SMEM_LIMIT;
  p.stages = (int32_t)std::min<uint32_t>(lora::SH_MAX_STAGES,
                                         (limit - lora::SH_FIXED_BYTES) / p.stage_bytes);
  p.cols = lora::shrink_cols(ad->r);
  p.tmem_cols = 256;
  p.accs = std::min(lora::SH_MAX_ACC, p.tmem_cols / p.cols);
  p.ids = ids;
  p.rank = ad->rank_dev;
  p.v = v;
  p.vmax = vmax;
  p.amax = amax;
  p.w = w;
  p.w_amax = w_amax;
  p.status = static_cast<int32_t *>(ws);
  p.timeout_ns = kTimeoutNs;
  return make_tmap_f16(&job->x, const_cast<uint16_t *>(X), (uint64_t)k, (uint64_t)s, lora::SH_KB,
                       lora::TM) &&
         make_tmap_f16(&job->f, const_cast<uint16_t *>(F), (uint64_t)k,
                       (uint64_t)ad->n * ad->r, lora::SH_KB, (uint32_t)ad->r);
}

cudaError_t launch_shrink(const lora::ShrinkJob *jobs, int n_jobs, int y, cudaStream_t st) {
  const lora::ShrinkParams &p = jobs[0].p;
  const int64_t tiles = ceil_div(p.s, lora::TM);
  const uint32_t smem = lora::SH_FIXED_BYTES + p.stages * p.stage_bytes;
  return launch_clusters(shrink_kernel(p.r), dim3((unsigned)(tiles * p.split), (unsigned)y, n_jobs),
                         dim3(lora::SH_THREADS), smem, st, p.split, false, jobs[0],
                         jobs[n_jobs - 1]);
}

// out = base + scale * v . F
llmint8_status enqueue_expand(const float *v, const float *vmax, int64_t s, int64_t o,
                              const uint16_t *F, const llmint8_adapters *ad, const int32_t *ids,
                              const uint16_t *base, uint16_t *out, const lora::PackParams *pack,
                              void *ws, int sm_count, cudaStream_t st) {
  lora::ExpandParams p;
  p.s = (int32_t)s;
  p.o = (int32_t)o;
  p.n = ad->n;
  p.r = ad->r;
  p.steps = (int32_t)ceil_div(o, lora::EX_N);
  // two CTAs per SM while v's operand leaves room for their rings
  const int per_sm = ad->r <= 64 ? 2 : 1;
  const uint32_t limit = per_sm == 2 ? kHalfSmem : lora::SMEM_LIMIT;
  p.fbufs = ad->r <= 32 ? 4 : 2;
  p.ring = 2;
  while (p.ring < lora::EX_MAX_RING && lora::expand_bytes(ad->r, p.ring + 1, p.fbufs) <= limit)
    ++p.ring;
  // chunks of steps per row tile: the fewest CTA rounds for their length, a
  // CTA's start counted as three steps and one per octet of terms. In a single
  // round nothing overlaps the starts and the ends, which is counted as eight
  // steps more (4096 x 20480 at rank 16: 67 us with 9 chunks, 58 with 18; 4096
  // x 5120 at rank 64: 23 us with 9, 31 with 18).
  const int64_t tiles = ceil_div(s, lora::TM), room = (int64_t)per_sm * sm_count;
  int64_t best = INT64_MAX;
  for (int64_t c = 1; c <= std::min<int64_t>(p.steps, std::max<int64_t>(2 * room / tiles, 16));
       ++c) {
    const int64_t rounds = ceil_div(tiles * c, room);
    const int64_t cost = rounds * (ceil_div(p.steps, c) + 3 + ad->r / 8) + (rounds == 1 ? 8 : 0);
    if (cost < best) {
      best = cost;
      p.chunks = (int32_t)c;
    }
  }
  p.v = v;
  p.vmax = vmax;
  p.scale = ad->scale_dev;
  p.f = as_half(F);
  p.ids = ids;
  p.rank = ad->rank_dev;
  p.has_base = base != nullptr;
  p.status = static_cast<int32_t *>(ws);
  p.timeout_ns = kTimeoutNs;
  CUtensorMap tm_base, tm_out;
  if (!make_tmap_f16(&tm_out, out, (uint64_t)o, (uint64_t)s, lora::EX_N, lora::TM) ||
      !make_tmap_f16(&tm_base, const_cast<uint16_t *>(base ? base : out), (uint64_t)o, (uint64_t)s,
                     lora::EX_N, lora::TM))
    return LLMINT8_ERR_CUDA;
  const lora::PackParams none = {};
  const int64_t pack_blocks = pack ? (int64_t)pack->jobs * pack->blocks : 0;
  if (launch(lora::k_expand, dim3((unsigned)(tiles * p.chunks + pack_blocks)),
             dim3(lora::EX_THREADS), lora::expand_bytes(ad->r, p.ring, p.fbufs), st, true, tm_base,
             tm_out, p, pack ? *pack : none) != cudaSuccess)
    return LLMINT8_ERR_CUDA;
  return LLMINT8_OK;
}

// dF = scale * P^T . Q per adapter
bool outer_job(lora::OuterJob *job, const uint8_t *packed, const int32_t *info,
               const uint32_t *amax, const uint16_t *Q, int64_t s, int64_t w,
               const llmint8_adapters *ad, const int32_t *ids, float *out, void *ws) {
  lora::OuterParams &p = job->p;
  p.s = (int32_t)s;
  p.w = (int32_t)w;
  p.n = ad->n;
  p.r = ad->r;
  const int32_t r16 = lora::outer_r16(ad->r);
  p.stage_bytes = lora::OU_Q_BYTES + lora::outer_p_bytes(ad->r);
  // two CTAs per SM up to r = 64, one above
  const bool half = ad->r <= 64;
  p.stages = (int32_t)std::min<uint32_t>(
      lora::OU_MAX_STAGES,
      ((half ? kHalfSmem : lora::SMEM_LIMIT) - lora::OU_FIXED_BYTES) / p.stage_bytes);
  p.tmem_cols = 32;  // two accumulators for each of the two products
  while (p.tmem_cols < 4 * r16) p.tmem_cols *= 2;
  p.col_tiles = (int32_t)ceil_div(w, lora::OU_COLS);
  p.p = packed;
  p.info = info;
  p.amax = amax;
  p.ids = ids;
  p.rank = ad->rank_dev;
  p.scale = ad->scale_dev;
  p.out = out;
  p.status = static_cast<int32_t *>(ws);
  p.timeout_ns = kTimeoutNs;
  return make_tmap_f16(&job->q, const_cast<uint16_t *>(Q), (uint64_t)w, (uint64_t)s, 64,
                       lora::OU_KB);
}

cudaError_t launch_outer(lora::OuterJob *jobs, int n_jobs, int sm_count, cudaStream_t st) {
  int64_t tiles = 0;
  for (int i = 0; i < n_jobs; ++i) tiles += jobs[i].p.col_tiles;
  // the fewest rounds for their length (a CTA's start and end counted as
  // twelve blocks: at 4096 rows of 5120 and 20480 features and rank 64 a split
  // of 2 takes 116 us in all, 3 135, 4 128, 5 123)
  const lora::OuterParams &p = jobs[0].p;
  const int64_t blocks = ceil_div(p.s, lora::OU_KB);
  const int64_t room = p.r <= 64 ? 2 * sm_count : sm_count;
  int split = 1;
  int64_t best = INT64_MAX;
  for (int c = 1; c <= lora::OU_MAX_SPLIT && c <= blocks; ++c) {
    const int64_t cost = ceil_div(tiles * p.n * c, room) * (ceil_div(blocks, c) + 12);
    if (cost < best) {
      best = cost;
      split = c;
    }
  }
  for (int i = 0; i < n_jobs; ++i) jobs[i].p.split = split;
  auto *k = p.r <= 16   ? lora::k_outer<2>
            : p.r <= 32 ? lora::k_outer<4>
            : p.r <= 64 ? lora::k_outer<8>
                        : lora::k_outer<16>;
  return launch_clusters(k, dim3((unsigned)(tiles * split), 1, (unsigned)p.n),
                         dim3(lora::OU_THREADS),
                         lora::OU_FIXED_BYTES + p.stages * p.stage_bytes, st, split, true, jobs[0],
                         jobs[n_jobs - 1]);
}

// ---------------------------------------- gradient of the projection's input

// Tiles of 512 rows where there are more than 256 (each converted weight tile
// then serves two MMAs), of 256 else. Whole rounds of tiles first (one tile
// per pair); the tiles of the last, partial round are cut along the reduction
// into as many parts as make the rounds they then take shortest. A part costs
// an fp32 tile written and read back, counted here as two stages. Planned for
// MAX_PAIRS pairs on any device, so that the workspace size depends on the
// sizes alone.
igrad::Plan input_grad_plan(int64_t s, int64_t h, int64_t o) {
  igrad::Plan p;
  p.mt = s > 2 * igrad::BM ? 2 : 1;
  p.num_m = (int32_t)ceil_div(s, p.mt * 2 * igrad::BM);
  p.num_n = (int32_t)ceil_div(h, igrad::BN);
  p.num_k = (int32_t)ceil_div(o, igrad::BK);
  const int64_t tiles = (int64_t)p.num_m * p.num_n;
  p.whole = (int32_t)(tiles / igrad::MAX_PAIRS * igrad::MAX_PAIRS);
  p.rest = (int32_t)(tiles - p.whole);
  p.parts = 1;
  int64_t best = INT64_MAX;
  for (int32_t parts = 1; p.rest > 0 && parts <= p.num_k && p.rest * parts <= igrad::MAX_PARTS;
       ++parts) {
    const int64_t rounds = ceil_div(p.rest * parts, igrad::MAX_PAIRS);
    const int64_t cost = rounds * (ceil_div(p.num_k, parts) + (parts > 1 ? 2 : 0)) +
                         (parts > 1 ? 2 * parts : 0);
    if (cost < best) {
      best = cost;
      p.parts = parts;
    }
  }
  return p;
}

size_t input_grad_workspace(const igrad::Plan &p) {
  const size_t slots = p.parts > 1 ? (size_t)p.rest * p.parts : 0;
  return align256(kStateBytes + 4 * igrad::PART_ELEMS * p.mt * slots);
}

// ----------------------------------------------------------- layer norm

// Threads and vectors of eight per thread for a row of h <= ln::MAX_ROW. Two
// vectors from 256 threads on: half the threads meet in a row's sums (backward
// at 2047 x 4096 fp16: 24.6 us against 27.8 with 512 threads).
void ln_shape(int64_t h, int *threads, int *nv) {
  const int64_t vecs = h / 8;
  *nv = (int)((vecs + ln::MAX_THREADS - 1) / ln::MAX_THREADS);
  if (vecs > ln::MAX_THREADS / 2) *nv = std::max(*nv, 2);
  const int64_t t = (vecs + *nv - 1) / *nv;
  *threads = (int)((t + 31) / 32 * 32);
}

template <typename TX, typename TP>
cudaError_t ln_forward(const void *x, int64_t s, int64_t h, const void *gamma, const void *beta,
                       float eps, uint16_t *y, float *mean, float *rstd, cudaStream_t st) {
  const TX *xp = static_cast<const TX *>(x);
  const TP *gp = static_cast<const TP *>(gamma), *bp = static_cast<const TP *>(beta);
  const dim3 grid((unsigned)s);
  if (h > ln::MAX_ROW)
    return launch(ln::k_ln_forward_long<TX, TP>, grid, dim3(ln::MAX_THREADS), 0, st, false, xp,
                  (int32_t)h, gp, bp, eps, as_half(y), mean, rstd);
  int threads, nv;
  ln_shape(h, &threads, &nv);
  auto *k = nv == 1   ? ln::k_ln_forward<TX, TP, 1>
            : nv == 2 ? ln::k_ln_forward<TX, TP, 2>
            : nv == 3 ? ln::k_ln_forward<TX, TP, 3>
                      : ln::k_ln_forward<TX, TP, 4>;
  return launch(k, grid, dim3(threads), 0, st, false, xp, (int32_t)h, gp, bp, eps, as_half(y),
                mean, rstd);
}

// Blocks of the backward kernel, which keeps one partial sum of each column
// per block: as many as run at once (two or three per SM for the narrower
// rows), never more than rows.
constexpr int kLnMaxBlocks = 512;

int ln_blocks_per_sm(int64_t h) {
  if (h > ln::MAX_ROW) return 2;
  int threads, nv;
  ln_shape(h, &threads, &nv);
  return threads > 256 ? 1 : threads > 128 ? 2 : 3;
}

int64_t ln_blocks(int64_t s, int64_t h, int sm_count) {
  return std::max<int64_t>(1, std::min<int64_t>({s, (int64_t)ln_blocks_per_sm(h) * sm_count,
                                                 (int64_t)kLnMaxBlocks}));
}

// nv vectors of 8 columns per thread; two rows at a time or one.
template <typename TX, typename TP>
auto ln_backward_kernel(int nv, bool two) {
  constexpr int U = (int)sizeof(TX) / 2;  // units of 16 bytes in 8 columns
  return nv == 1   ? (two ? ln::k_ln_backward<TX, TP, U, 2> : ln::k_ln_backward<TX, TP, U, 1>)
         : nv == 2 ? (two ? ln::k_ln_backward<TX, TP, 2 * U, 2>
                          : ln::k_ln_backward<TX, TP, 2 * U, 1>)
         : nv == 3 ? ln::k_ln_backward<TX, TP, 3 * U, 1>
                   : ln::k_ln_backward<TX, TP, 4 * U, 1>;
}

constexpr uint32_t kLnSmemPerSm = 224 * 1024;

template <typename TX, typename TP>
bool ln_backward_setup() {
  for (int nv = 1; nv <= ln::MAX_VEC; ++nv)
    for (int two = 0; two < 2; ++two)
      if (cudaFuncSetAttribute(ln_backward_kernel<TX, TP>(nv, two != 0),
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)kLnSmemPerSm) != cudaSuccess)
        return false;
  return true;
}

template <typename TX, typename TP>
cudaError_t ln_backward(const uint16_t *dy, const void *x, int64_t s, int64_t h, const void *gamma,
                        const float *mean, const float *rstd, void *dx, float *part,
                        int64_t blocks, void *ws, cudaStream_t st) {
  const TX *xp = static_cast<const TX *>(x);
  const TP *gp = static_cast<const TP *>(gamma);
  TX *dxp = static_cast<TX *>(dx);
  const dim3 grid((unsigned)blocks);
  if (h > ln::MAX_ROW)
    return launch(ln::k_ln_backward_long<TX, TP>, grid, dim3(ln::MAX_THREADS), 0, st, false,
                  as_half(dy), xp, s, (int32_t)h, gp, mean, rstd, dxp, part);
  int threads, nv;
  ln_shape(h, &threads, &nv);
  uint32_t stage = (uint32_t)h * (sizeof(TX) + 2);
  const uint32_t limit = kLnSmemPerSm / ln_blocks_per_sm(h) - 2048;
  // two rows at a time where every block has them and three such stages fit
  const bool two = nv <= 2 && 3 * 2 * stage <= limit && s >= 2 * blocks;
  if (two) stage *= 2;
  const int stages = (int)std::min<uint32_t>(ln::BW_MAX_STAGES, limit / stage);
  return launch(ln_backward_kernel<TX, TP>(nv, two), grid, dim3(threads), stages * stage, st,
                false, as_half(dy), xp, s, (int32_t)h, stages, gp, mean, rstd, dxp, part,
                static_cast<int32_t *>(ws), kTimeoutNs);
}

// -------------------------------------------------------------- clipping

// As many blocks as fit the GPU at once, four per SM, and one at least.
int64_t clip_blocks(int64_t chunks, int sm_count) {
  return std::max<int64_t>(
      1, std::min<int64_t>({chunks, 4 * (int64_t)sm_count, clip::MAX_BLOCKS}));
}

// LLMINT8_ERR_ARG when two outputs share memory, or an output and another
// entry's gradient: blocks of one call would race on it.
llmint8_status check_grad_overlaps(const llmint8_grad *grads, int64_t n) {
  struct Range {
    uintptr_t begin, end;
    bool written;
  };
  try {
    std::vector<Range> spans;
    spans.reserve(2 * (size_t)n);
    for (int64_t i = 0; i < n; ++i) {
      const llmint8_grad &g = grads[i];
      if (g.n == 0) continue;
      const size_t bytes = (g.type == LLMINT8_F32 ? 4 : 2) * (size_t)g.n;
      const uintptr_t in = reinterpret_cast<uintptr_t>(g.grad_dev);
      const uintptr_t out = g.out_dev ? reinterpret_cast<uintptr_t>(g.out_dev) : in;
      spans.push_back({out, out + bytes, true});
      if (out != in) spans.push_back({in, in + bytes, false});
    }
    std::sort(spans.begin(), spans.end(),
              [](const Range &a, const Range &b) { return a.begin < b.begin; });
    uintptr_t read_end = 0, written_end = 0;
    for (const Range &s : spans) {
      if (s.begin < written_end || (s.written && s.begin < read_end)) return LLMINT8_ERR_ARG;
      uintptr_t &end = s.written ? written_end : read_end;
      end = std::max(end, s.end);
    }
  } catch (...) {  // no host memory for the check
    return LLMINT8_ERR_TOO_LARGE;
  }
  return LLMINT8_OK;
}

size_t type_size(int32_t type) { return type == LLMINT8_F32 ? 4 : 2; }

bool ln_types_ok(int32_t x_type, int32_t p_type) {
  return (x_type == LLMINT8_F16 || x_type == LLMINT8_F32) &&
         (p_type == LLMINT8_F16 || p_type == LLMINT8_F32);
}

}  // namespace

extern "C" {

size_t llmint8_adapters_workspace_size(int64_t s, int64_t h, int64_t o, int32_t n, int32_t r) {
  if (check_adapter_sizes(s, h, o, n, r)) return 0;
  return adapter_layout(s, h, o, n, r).end;
}

llmint8_status llmint8_adapters_forward(const uint16_t *X_dev, int64_t s,
                                        const llmint8_adapters *ad, const int32_t *ids_dev,
                                        const uint16_t *base_dev, uint16_t *out_dev, float *v_dev,
                                        void *ws_dev, size_t ws_bytes, void *stream) {
  llmint8_status rc = check_adapters(ad, s);
  if (rc) return rc;
  if (s == 0) return LLMINT8_OK;
  if (!X_dev || !ids_dev || !out_dev || !ws_dev) return LLMINT8_ERR_NULL;
  if (!aligned(X_dev, 16) || !aligned(ids_dev, 4) || !aligned(base_dev, 16) ||
      !aligned(out_dev, 16) || !aligned(v_dev, 16) || !aligned(ws_dev, 256))
    return LLMINT8_ERR_ALIGN;
  const Span X = {X_dev, 2 * (size_t)s * ad->h}, base = {base_dev, 2 * (size_t)s * ad->o};
  const Span out = {out_dev, base.n}, kept = {v_dev, 4 * (size_t)s * ad->r};
  const Span ids = {ids_dev, 4 * (size_t)s}, A = factor_a(ad), B = factor_b(ad);
  const Span scale = {ad->scale_dev, 4 * (size_t)ad->n}, rank = {ad->rank_dev, scale.n};
  if (overlaps_any(out, {X, kept, ids, A, B, scale, rank}) || overlaps_partly(out, base) ||
      overlaps_any(kept, {X, base, ids, A, B, scale, rank}))
    return LLMINT8_ERR_ARG;
  const AdapterLayout L = adapter_layout(s, ad->h, ad->o, ad->n, ad->r);
  if (ws_bytes < L.end) return LLMINT8_ERR_WORKSPACE;
  if (overlaps_any({ws_dev, L.end}, {X, base, out, kept, ids, A, B, scale, rank}))
    return LLMINT8_ERR_ARG;
  Device *dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  cudaStream_t st = as_stream(stream);
  uint8_t *wsb = static_cast<uint8_t *>(ws_dev);
  if (use_row_kernels(s, ad, false)) {
    if ((rc = enqueue_rows(X_dev, s, ad->h, ad->a_dev, ad->o, ad->b_dev, ad, ids_dev, base_dev,
                           out_dev, v_dev, reinterpret_cast<float *>(wsb + L.part), st)))
      return rc;
    return last_launch();
  }
  float *v = v_dev ? v_dev : reinterpret_cast<float *>(wsb + L.v);
  float *vmax = reinterpret_cast<float *>(wsb + L.vmax);
  const ShrinkGrid grid = shrink_grid(s, ad->h, ad, 1, *dev);
  lora::ShrinkJob job;
  if (!shrink_job(&job, X_dev, s, ad->h, ad->a_dev, ad, ids_dev, v, vmax, nullptr, nullptr,
                  nullptr, grid.split, ws_dev) ||
      launch_shrink(&job, 1, grid.y, st) != cudaSuccess)
    return LLMINT8_ERR_CUDA;
  if ((rc = enqueue_expand(v, vmax, s, ad->o, ad->b_dev, ad, ids_dev, base_dev, out_dev, nullptr,
                           ws_dev, dev->sm_count, st)))
    return rc;
  return last_launch();
}

llmint8_status llmint8_adapters_backward(const uint16_t *X_dev, const uint16_t *dY_dev, int64_t s,
                                         const llmint8_adapters *ad, const int32_t *ids_dev,
                                         const float *v_dev, const uint16_t *base_dev,
                                         uint16_t *dX_dev, float *dA_dev, float *dB_dev,
                                         void *ws_dev, size_t ws_bytes, void *stream) {
  llmint8_status rc = check_adapters(ad, s);
  if (rc) return rc;
  const bool need_v = dB_dev && !v_dev;
  if (s > 0 && (!dY_dev || !ids_dev || !ws_dev || ((dA_dev || need_v) && !X_dev)))
    return LLMINT8_ERR_NULL;
  if (!aligned(X_dev, 16) || !aligned(dY_dev, 16) || !aligned(ids_dev, 4) || !aligned(v_dev, 16) ||
      !aligned(base_dev, 16) || !aligned(dX_dev, 16) || !aligned(dA_dev, 16) ||
      !aligned(dB_dev, 16) || !aligned(ws_dev, 256))
    return LLMINT8_ERR_ALIGN;
  const Span X = {X_dev, 2 * (size_t)s * ad->h}, dY = {dY_dev, 2 * (size_t)s * ad->o};
  const Span base = {base_dev, X.n}, dX = {dX_dev, X.n}, kept = {v_dev, 4 * (size_t)s * ad->r};
  const Span ids = {ids_dev, 4 * (size_t)s}, A = factor_a(ad), B = factor_b(ad);
  const Span scale = {ad->scale_dev, 4 * (size_t)ad->n}, rank = {ad->rank_dev, scale.n};
  const Span dA = {dA_dev, 2 * A.n}, dB = {dB_dev, 2 * B.n};
  if (overlaps_any(dX, {X, dY, kept, ids, A, B, scale, rank}) || overlaps_partly(dX, base) ||
      overlaps_any(dA, {X, dY, base, dX, kept, ids, A, B, scale, rank}) ||
      overlaps_any(dB, {X, dY, base, dX, kept, ids, A, B, scale, rank, dA}))
    return LLMINT8_ERR_ARG;
  const AdapterLayout L = adapter_layout(s, ad->h, ad->o, ad->n, ad->r);
  if (s > 0 && ws_bytes < L.end) return LLMINT8_ERR_WORKSPACE;
  if (s > 0 && overlaps_any({ws_dev, L.end},
                            {X, dY, base, dX, kept, ids, A, B, scale, rank, dA, dB}))
    return LLMINT8_ERR_ARG;
  Device *dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  cudaStream_t st = as_stream(stream);
  const size_t factor = 4 * (size_t)ad->n * ad->r;
  if (s == 0) {  // no rows: empty sums
    if ((dA_dev && cudaMemsetAsync(dA_dev, 0, factor * ad->h, st) != cudaSuccess) ||
        (dB_dev && cudaMemsetAsync(dB_dev, 0, factor * ad->o, st) != cudaSuccess))
      return LLMINT8_ERR_CUDA;
    return LLMINT8_OK;
  }
  uint8_t *wsb = static_cast<uint8_t *>(ws_dev);
  float *v = reinterpret_cast<float *>(wsb + L.v), *g = reinterpret_cast<float *>(wsb + L.g);
  float *vmax = reinterpret_cast<float *>(wsb + L.vmax);
  float *gmax = reinterpret_cast<float *>(wsb + L.gmax);
  uint32_t *v_amax = reinterpret_cast<uint32_t *>(wsb + L.amax), *g_amax = v_amax + ad->n;
  const bool need_g = dX_dev || dA_dev;
  if (use_row_kernels(s, ad, true)) {
    float *part = reinterpret_cast<float *>(wsb + L.part);
    if (need_v && (rc = enqueue_rows(X_dev, s, ad->h, ad->a_dev, ad->o, ad->b_dev, ad, ids_dev,
                                     nullptr, nullptr, v, part, st)))
      return rc;
    if (need_g && (rc = enqueue_rows(dY_dev, s, ad->o, ad->b_dev, ad->h, ad->a_dev, ad, ids_dev,
                                     base_dev, dX_dev, g, part, st)))
      return rc;
    lora::RowsOuterJob jobs[2];
    int n_jobs = 0;
    if (dB_dev)
      jobs[n_jobs++] = {v_dev ? v_dev : v, as_half(dY_dev), dB_dev, (int32_t)ad->o};
    if (dA_dev) jobs[n_jobs++] = {g, as_half(X_dev), dA_dev, (int32_t)ad->h};
    if (n_jobs > 0) {
      const int64_t first = ceil_div(jobs[0].w, lora::RO_SLICE);
      const int64_t second = n_jobs > 1 ? ceil_div(jobs[1].w, lora::RO_SLICE) : 0;
      if (launch(lora::k_rows_outer,
                 dim3((unsigned)(first + second), (unsigned)ad->n,
                      (unsigned)ceil_div(ad->r, lora::RO_TERMS)),
                 dim3(lora::RO_THREADS), 0, st, need_g || need_v, jobs[0], jobs[n_jobs - 1],
                 (int32_t)first, (int32_t)s, ids_dev, ad->scale_dev, ad->rank_dev, ad->n,
                 ad->r) != cudaSuccess)
        return LLMINT8_ERR_CUDA;
    }
    return last_launch();
  }
  const bool own_v = dB_dev && v_dev;  // v as the caller kept it: only its maxima
  int32_t *info = reinterpret_cast<int32_t *>(wsb + L.info);
  lora::ShrinkJob shrink[2];
  lora::OuterJob outer[2];
  lora::PackParams pack = {};
  pack.blocks = (int32_t)ceil_div(s, lora::OU_KB);
  pack.s = (int32_t)s;
  pack.n = ad->n;
  pack.r = ad->r;
  pack.ids = ids_dev;
  pack.info = info;
  int n_shrink = 0, n_outer = 0;
  const int want = (need_g ? 1 : 0) + (need_v ? 1 : 0);
  const int64_t width = !need_v ? ad->o : !need_g ? ad->h : std::min(ad->h, ad->o);
  const ShrinkGrid grid = shrink_grid(s, width, ad, std::max(want, 1), *dev);
  if (need_g && !shrink_job(&shrink[n_shrink++], dY_dev, s, ad->o, ad->b_dev, ad, ids_dev, g, gmax,
                            dA_dev ? g_amax : nullptr, own_v ? v_dev : nullptr, v_amax, grid.split,
                            ws_dev))
    return LLMINT8_ERR_CUDA;
  if (need_v && !shrink_job(&shrink[n_shrink++], X_dev, s, ad->h, ad->a_dev, ad, ids_dev, v, vmax,
                            v_amax, nullptr, nullptr, grid.split, ws_dev))
    return LLMINT8_ERR_CUDA;
  if (dB_dev) {
    pack.job[n_outer] = {v_dev ? v_dev : v, v_amax, wsb + L.vpack};
    if (!outer_job(&outer[n_outer++], wsb + L.vpack, info, v_amax, dY_dev, s, ad->o, ad, ids_dev,
                   dB_dev, ws_dev))
      return LLMINT8_ERR_CUDA;
  }
  if (dA_dev) {
    pack.job[n_outer] = {g, g_amax, wsb + L.gpack};
    if (!outer_job(&outer[n_outer++], wsb + L.gpack, info, g_amax, X_dev, s, ad->h, ad, ids_dev,
                   dA_dev, ws_dev))
      return LLMINT8_ERR_CUDA;
  }
  if (n_outer > 0 && cudaMemsetAsync(v_amax, 0, 8 * (size_t)ad->n, st) != cudaSuccess)
    return LLMINT8_ERR_CUDA;
  if (n_shrink > 0) {
    if (launch_shrink(shrink, n_shrink, grid.y, st) != cudaSuccess) return LLMINT8_ERR_CUDA;
  } else if (own_v && launch(lora::k_adapter_max, dim3((unsigned)ceil_div(s, 8)), dim3(256), 0, st,
                             false, v_dev, s, ad->n, ad->r, ids_dev, v_amax) != cudaSuccess) {
    return LLMINT8_ERR_CUDA;
  }
  pack.jobs = n_outer;
  if (dX_dev) {
    if ((rc = enqueue_expand(g, gmax, s, ad->h, ad->a_dev, ad, ids_dev, base_dev, dX_dev,
                             n_outer > 0 ? &pack : nullptr, ws_dev, dev->sm_count, st)))
      return rc;
  } else if (n_outer > 0 &&
             launch(lora::k_pack, dim3((unsigned)(n_outer * pack.blocks)), dim3(lora::PK_THREADS),
                    0, st, true, pack) != cudaSuccess) {
    return LLMINT8_ERR_CUDA;
  }
  if (n_outer > 0 && launch_outer(outer, n_outer, dev->sm_count, st) != cudaSuccess)
    return LLMINT8_ERR_CUDA;
  return last_launch();
}

size_t llmint8_matmul_backward_workspace_size(int64_t s, int64_t h, int64_t o) {
  if (check_hw(h, o) || check_rows(s)) return 0;
  // up to MAX_PARTS fp32 tiles: the most that any smaller number of rows needs
  // (the plan repeats every MAX_PAIRS tiles of rows)
  size_t bytes = 0;
  const int64_t blocks = ceil_div(s, 2 * igrad::BM);
  for (int64_t m = 0; m < std::min<int64_t>(blocks, 2 * igrad::MAX_PAIRS); ++m)
    bytes = std::max(bytes,
                     input_grad_workspace(input_grad_plan((blocks - m) * 2 * igrad::BM, h, o)));
  if (blocks > 0) bytes = std::max(bytes, input_grad_workspace(input_grad_plan(1, h, o)));
  return std::max(bytes, kStateBytes);
}

llmint8_status llmint8_matmul_backward(const uint16_t *dY_dev, int64_t s, const llmint8_weight *w,
                                       const uint16_t *base_dev, uint16_t *dX_dev, void *ws_dev,
                                       size_t ws_bytes, void *stream) {
  if (!w || !w->wq_dev || !w->aw_dev) return LLMINT8_ERR_NULL;
  llmint8_status rc = check_hw(w->h, w->o);
  if (rc) return rc;
  if ((rc = check_rows(s))) return rc;
  if (!aligned(w->wq_dev, 16) || !aligned(w->aw_dev, 16)) return LLMINT8_ERR_ALIGN;
  if (s == 0) return LLMINT8_OK;
  if (!dY_dev || !dX_dev || !ws_dev) return LLMINT8_ERR_NULL;
  if (!aligned(dY_dev, 16) || !aligned(base_dev, 16) || !aligned(dX_dev, 16) ||
      !aligned(ws_dev, 256))
    return LLMINT8_ERR_ALIGN;
  const Span dX = {dX_dev, 2 * (size_t)s * w->h}, base = {base_dev, dX.n};
  const Span dY = {dY_dev, 2 * (size_t)s * w->o}, aw = {w->aw_dev, 4 * (size_t)w->o};
  const Span wq = {w->wq_dev, (size_t)w->h * w->o};
  if (overlaps_any(dX, {dY, wq, aw}) || overlaps_partly(dX, base)) return LLMINT8_ERR_ARG;
  const igrad::Plan plan = input_grad_plan(s, w->h, w->o);
  const size_t need = input_grad_workspace(plan);
  if (ws_bytes < need) return LLMINT8_ERR_WORKSPACE;
  if (overlaps_any({ws_dev, need}, {dX, base, dY, wq, aw})) return LLMINT8_ERR_ARG;
  Device *dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  igrad::Params p;
  p.s = (int32_t)s;
  p.h = (int32_t)w->h;
  p.o = (int32_t)w->o;
  p.plan = plan;
  p.wq = w->wq_dev;
  p.aw = w->aw_dev;
  p.base = as_half(base_dev);
  p.out = as_half(dX_dev);
  p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws_dev) + kStateBytes);
  p.status = static_cast<int32_t *>(ws_dev);
  p.timeout_ns = kTimeoutNs;
  CUtensorMap tmA, tmW;
  if (!make_tmap_i8_plain(&tmW, w->wq_dev, (uint64_t)w->h, (uint64_t)w->o, igrad::BNH,
                          igrad::BK) ||
      !make_tmap_f16(&tmA, const_cast<uint16_t *>(dY_dev), (uint64_t)w->o, (uint64_t)s, igrad::BK,
                     igrad::BM))
    return LLMINT8_ERR_CUDA;
  cudaStream_t st = as_stream(stream);
  const int64_t units = plan.whole + (int64_t)plan.rest * plan.parts;
  const unsigned ctas = 2 * (unsigned)std::min<int64_t>(units, dev->max_pairs);
  // (with parts, the base of the tiles cut is added by their sum)
  if (launch_pairs(input_grad_kernel(plan.mt, base_dev != nullptr), dim3(ctas),
                   dim3(igrad::NUM_THREADS), input_grad_smem(plan.mt), st, false, tmA, tmW,
                   p) != cudaSuccess)
    return LLMINT8_ERR_CUDA;
  if (plan.parts > 1 &&
      launch(igrad::k_input_grad_sum,
             dim3(blocks_for((int64_t)plan.rest * plan.mt * 2 * igrad::BM * (igrad::BN / 8),
                             igrad::SUM_THREADS)),
             dim3(igrad::SUM_THREADS), 0, st, true, p) != cudaSuccess)
    return LLMINT8_ERR_CUDA;
  return last_launch();
}

llmint8_status llmint8_layernorm_forward(const void *x_dev, int32_t x_type, int64_t s, int64_t h,
                                         const void *gamma_dev, const void *beta_dev,
                                         int32_t p_type, float eps, uint16_t *y_dev,
                                         float *mean_dev, float *rstd_dev, void *stream) {
  llmint8_status rc = check_width(h);
  if (rc) return rc;
  if ((rc = check_rows(s))) return rc;
  if (!ln_types_ok(x_type, p_type) || !std::isfinite(eps) || eps < 0.0f) return LLMINT8_ERR_ARG;
  if (s == 0) return LLMINT8_OK;
  if (!x_dev || !gamma_dev || !y_dev) return LLMINT8_ERR_NULL;
  if (!aligned(x_dev, 16) || !aligned(gamma_dev, 16) || !aligned(beta_dev, 16) ||
      !aligned(y_dev, 16) || !aligned(mean_dev, 4) || !aligned(rstd_dev, 4))
    return LLMINT8_ERR_ALIGN;
  // y in place of an fp16 x: a thread has read what it writes
  const Span x = {x_dev, type_size(x_type) * (size_t)s * h}, y = {y_dev, 2 * (size_t)s * h};
  const Span gamma = {gamma_dev, type_size(p_type) * (size_t)h}, beta = {beta_dev, gamma.n};
  const Span mean = {mean_dev, 4 * (size_t)s}, rstd = {rstd_dev, mean.n};
  if (overlaps_partly(y, x) || overlaps_any(y, {gamma, beta, mean, rstd}) ||
      overlaps_any(mean, {x, gamma, beta, rstd}) || overlaps_any(rstd, {x, gamma, beta}))
    return LLMINT8_ERR_ARG;
  Device *dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  cudaStream_t st = as_stream(stream);
  auto *f = x_type == LLMINT8_F16
                ? (p_type == LLMINT8_F16 ? ln_forward<__half, __half> : ln_forward<__half, float>)
                : (p_type == LLMINT8_F16 ? ln_forward<float, __half> : ln_forward<float, float>);
  if (f(x_dev, s, h, gamma_dev, beta_dev, eps, y_dev, mean_dev, rstd_dev, st) != cudaSuccess)
    return LLMINT8_ERR_CUDA;
  return last_launch();
}

size_t llmint8_layernorm_workspace_size(int64_t s, int64_t h) {
  if (check_width(h) || check_rows(s)) return 0;
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>(s, kLnMaxBlocks));
  return align256(kStateBytes + 8 * (size_t)blocks * h);
}

llmint8_status llmint8_layernorm_backward(const uint16_t *dy_dev, const void *x_dev,
                                          int32_t x_type, int64_t s, int64_t h,
                                          const void *gamma_dev, int32_t p_type,
                                          const float *mean_dev, const float *rstd_dev,
                                          void *dx_dev, float *dgamma_dev, float *dbeta_dev,
                                          void *ws_dev, size_t ws_bytes, void *stream) {
  llmint8_status rc = check_width(h);
  if (rc) return rc;
  if ((rc = check_rows(s))) return rc;
  if (!ln_types_ok(x_type, p_type)) return LLMINT8_ERR_ARG;
  if (s > 0 && (!dy_dev || !x_dev || !gamma_dev || !mean_dev || !rstd_dev || !ws_dev))
    return LLMINT8_ERR_NULL;
  if (!aligned(dy_dev, 16) || !aligned(x_dev, 16) || !aligned(gamma_dev, 16) ||
      !aligned(mean_dev, 4) || !aligned(rstd_dev, 4) || !aligned(dx_dev, 16) ||
      !aligned(dgamma_dev, 16) || !aligned(dbeta_dev, 16) || !aligned(ws_dev, 256))
    return LLMINT8_ERR_ALIGN;
  const size_t need = s > 0 ? llmint8_layernorm_workspace_size(s, h) : 0;
  if (ws_bytes < need) return LLMINT8_ERR_WORKSPACE;
  // dx in place of x or dy of its type: a row's block has read the row
  const Span x = {x_dev, type_size(x_type) * (size_t)s * h}, dy = {dy_dev, 2 * (size_t)s * h};
  const Span dx = {dx_dev, x.n}, gamma = {gamma_dev, type_size(p_type) * (size_t)h};
  const Span mean = {mean_dev, 4 * (size_t)s}, rstd = {rstd_dev, mean.n};
  const Span dgamma = {dgamma_dev, 4 * (size_t)h}, dbeta = {dbeta_dev, dgamma.n};
  if (overlaps_partly(dx, x) || overlaps_partly(dx, dy) ||
      overlaps_any(dx, {gamma, mean, rstd, dgamma, dbeta}) ||
      overlaps_any(dgamma, {x, dy, gamma, mean, rstd, dbeta}) ||
      overlaps_any(dbeta, {x, dy, gamma, mean, rstd}) ||
      overlaps_any({ws_dev, need}, {x, dy, gamma, mean, rstd, dx, dgamma, dbeta}))
    return LLMINT8_ERR_ARG;
  Device *dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  cudaStream_t st = as_stream(stream);
  if (s == 0) {  // no rows: empty sums
    if ((dgamma_dev && cudaMemsetAsync(dgamma_dev, 0, 4 * (size_t)h, st) != cudaSuccess) ||
        (dbeta_dev && cudaMemsetAsync(dbeta_dev, 0, 4 * (size_t)h, st) != cudaSuccess))
      return LLMINT8_ERR_CUDA;
    return LLMINT8_OK;
  }
  const int64_t blocks = ln_blocks(s, h, dev->sm_count);
  float *part = dgamma_dev || dbeta_dev
                    ? reinterpret_cast<float *>(static_cast<uint8_t *>(ws_dev) + kStateBytes)
                    : nullptr;
  auto *f = x_type == LLMINT8_F16
                ? (p_type == LLMINT8_F16 ? ln_backward<__half, __half> : ln_backward<__half, float>)
                : (p_type == LLMINT8_F16 ? ln_backward<float, __half> : ln_backward<float, float>);
  if (f(dy_dev, x_dev, s, h, gamma_dev, mean_dev, rstd_dev, dx_dev, part, blocks, ws_dev, st) !=
      cudaSuccess)
    return LLMINT8_ERR_CUDA;
  if (part && launch(ln::k_ln_reduce, dim3(blocks_for(2 * h, ln::RED_COLS)),
                     dim3(ln::RED_COLS / 4 * ln::RED_LANES), 0, st, true, (const float *)part,
                     (int32_t)blocks, (int32_t)h, dgamma_dev, dbeta_dev) != cudaSuccess)
    return LLMINT8_ERR_CUDA;
  return last_launch();
}

size_t llmint8_grad_list_size(int64_t n) {
  if (n < 0 || n > (int64_t)1 << 24) return 0;
  return align256(clip::kEntriesOffset + sizeof(clip::Entry) * (size_t)n);
}

llmint8_status llmint8_grad_list_init(const llmint8_grad *grads_host, int64_t n,
                                      llmint8_grad_list *list, void *stream) {
  if (!list || !list->table_dev || (n > 0 && !grads_host)) return LLMINT8_ERR_NULL;
  const size_t need = llmint8_grad_list_size(n);
  if (need == 0) return LLMINT8_ERR_SHAPE;
  if (!aligned(list->table_dev, 256)) return LLMINT8_ERR_ALIGN;
  if (list->table_bytes < need) return LLMINT8_ERR_WORKSPACE;
  int64_t chunks = 0;
  for (int64_t i = 0; i < n; ++i) {
    const llmint8_grad &g = grads_host[i];
    if (g.type != LLMINT8_F16 && g.type != LLMINT8_F32 && g.type != LLMINT8_BF16)
      return LLMINT8_ERR_ARG;
    if (g.n < 0 || g.n > (int64_t)1 << 40) return LLMINT8_ERR_SHAPE;
    if (g.n == 0) continue;
    if (!g.grad_dev) return LLMINT8_ERR_NULL;
    const uintptr_t size = g.type == LLMINT8_F32 ? 4 : 2;
    if (!aligned(g.grad_dev, size) || !aligned(g.out_dev, size)) return LLMINT8_ERR_ALIGN;
    const size_t bytes = size * (size_t)g.n;
    if ((g.out_dev != g.grad_dev && overlap(g.out_dev, bytes, g.grad_dev, bytes)) ||
        overlap(g.out_dev ? g.out_dev : g.grad_dev, bytes, list->table_dev, need))
      return LLMINT8_ERR_ARG;
    chunks += ceil_div(g.n, clip::chunk_elements(g.type));
  }
  llmint8_status rc = check_grad_overlaps(grads_host, n);
  if (rc) return rc;
  Device *dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  cudaStream_t st = as_stream(stream);
  clip::Entry *table = reinterpret_cast<clip::Entry *>(static_cast<uint8_t *>(list->table_dev) +
                                                       clip::kEntriesOffset);
  // the entry that holds each block's first chunk
  const int64_t blocks = clip_blocks(chunks, dev->sm_count);
  int32_t *starts = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(list->table_dev) +
                                                clip::kStartsOffset);
  int64_t entry = 0, before = 0;  // chunks before `entry`
  for (int64_t b = 0; b < blocks; b += clip::INIT_STARTS) {
    const int m = (int)std::min<int64_t>(clip::INIT_STARTS, blocks - b);
    clip::StartBatch batch = {};
    for (int k = 0; k < m; ++k) {
      const int64_t c = clip::range_start(chunks, b + k, blocks);
      while (entry + 1 < n) {
        const llmint8_grad &g = grads_host[entry];
        const int64_t mine = ceil_div(g.n, clip::chunk_elements(g.type));
        if (before + mine > c) break;
        before += mine;
        ++entry;
      }
      batch.first[k] = (int32_t)entry;
    }
    if (launch(clip::k_starts_init, dim3(1), dim3(clip::INIT_STARTS), 0, st, false, starts + b,
               batch, m) != cudaSuccess)
      return LLMINT8_ERR_CUDA;
  }
  int64_t at = 0;
  for (int64_t i = 0; i < n; i += clip::INIT_ENTRIES) {
    const int m = (int)std::min<int64_t>(clip::INIT_ENTRIES, n - i);
    clip::InitBatch batch = {};
    for (int k = 0; k < m; ++k) {
      const llmint8_grad &g = grads_host[i + k];
      clip::Entry &e = batch.e[k];
      e.grad = g.grad_dev;
      e.out = g.out_dev ? g.out_dev : const_cast<void *>(g.grad_dev);
      e.n = g.n;
      e.chunk0 = at;
      e.type = g.type;
      at += ceil_div(g.n, clip::chunk_elements(g.type));
    }
    if (launch(clip::k_list_init, dim3(1), dim3(64), 0, st, false, table + i, batch, m) !=
        cudaSuccess)
      return LLMINT8_ERR_CUDA;
  }
  list->n = n;
  list->chunks = chunks;
  return last_launch();
}

llmint8_status llmint8_clip_grads(const llmint8_grad_list *list, float max_norm, float *norm_dev,
                                  void *stream) {
  if (!list || !list->table_dev || !norm_dev) return LLMINT8_ERR_NULL;
  if (std::isnan(max_norm) || max_norm < 0.0f) return LLMINT8_ERR_ARG;
  const size_t need = llmint8_grad_list_size(list->n);
  if (need == 0 || list->chunks < 0) return LLMINT8_ERR_SHAPE;
  if (!aligned(list->table_dev, 256) || !aligned(norm_dev, 4)) return LLMINT8_ERR_ALIGN;
  if (list->table_bytes < need) return LLMINT8_ERR_WORKSPACE;
  if (overlap(norm_dev, sizeof(float), list->table_dev, need)) return LLMINT8_ERR_ARG;
  Device *dev = nullptr;
  llmint8_status rc = current_device(&dev);
  if (rc) return rc;
  cudaStream_t st = as_stream(stream);
  double *partial = static_cast<double *>(list->table_dev);
  const clip::Entry *table = reinterpret_cast<const clip::Entry *>(
      static_cast<const uint8_t *>(list->table_dev) + clip::kEntriesOffset);
  const int32_t *starts = reinterpret_cast<const int32_t *>(
      static_cast<const uint8_t *>(list->table_dev) + clip::kStartsOffset);
  const int64_t blocks = clip_blocks(list->chunks, dev->sm_count);
  if (launch(clip::k_square_sums, dim3((unsigned)blocks), dim3(clip::THREADS), 0, st, false, table,
             list->n, list->chunks, starts, partial) != cudaSuccess)
    return LLMINT8_ERR_CUDA;
  if (launch(clip::k_clip_scale, dim3((unsigned)blocks), dim3(clip::THREADS), 0, st, true, table,
             list->n, list->chunks, starts, (const double *)partial, (int32_t)blocks, max_norm,
             norm_dev) != cudaSuccess)
    return LLMINT8_ERR_CUDA;
  return last_launch();
}

}  // extern "C"

// Host-side helpers of finetune_api.cu: the shape and alignment rules of
// include/llmint8.h and the state block at the front of every workspace (as in
// llmint8_api.cu), TMA descriptor creation and kernel launches. Everything here
// has internal linkage.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <utility>

#include "llmint8.h"

namespace {

constexpr int64_t kMaxH = 133144;  // 127*127*h must fit int32
constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s per individual wait
constexpr int kMaxDevices = 64;

// ----------------------------------------------------- TMA descriptors
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 2-D int8 tensor [rows][inner] with row stride `inner` bytes, box
// [box_rows][box_inner] landing in shared memory row by row.
bool make_tmap_i8_plain(CUtensorMap *map, const void *ptr, uint64_t inner, uint64_t rows,
                        uint32_t box_inner, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, rows};
  cuuint64_t strides[1] = {inner};
  cuuint32_t box[2] = {box_inner, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(ptr), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D fp16 tensor [rows][inner] (row stride 2*inner bytes) in boxes of
// [box_rows][64] (128 bytes a row, 128-byte swizzle).
bool make_tmap_f16(CUtensorMap *map, void *ptr, uint64_t inner, uint64_t rows,
                   uint32_t box_inner, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, rows};
  cuuint64_t strides[1] = {2 * inner};
  cuuint32_t box[2] = {box_inner, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, ptr, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ------------------------------------------------------ workspaces
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// The state block at the front of a workspace, cleared by
// llmint8_workspace_init and kept by the kernels between calls: the status
// words, then the accumulation bitmask of the one-read activation pass
// (sized for the largest h), which that pass leaves zero on exit.
constexpr size_t kStateBytes = 256 + ((4 * (size_t)((kMaxH + 31) / 32) + 255) & ~size_t(255));
static_assert(kStateBytes == LLMINT8_WORKSPACE_STATE_BYTES, "state block size");

// --------------------------------------------------------- validation
bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

llmint8_status check_hw(int64_t h, int64_t o) {
  if (h < 16 || h > kMaxH || (h % 16) != 0) return LLMINT8_ERR_SHAPE;
  if (o < 16 || (o % 16) != 0 || o > (int64_t)INT32_MAX / 2) return LLMINT8_ERR_SHAPE;
  return LLMINT8_OK;
}

cudaStream_t as_stream(void *s) { return reinterpret_cast<cudaStream_t>(s); }

llmint8_status last_launch() {
  return cudaGetLastError() == cudaSuccess ? LLMINT8_OK : LLMINT8_ERR_CUDA;
}

// Launch with programmatic stream serialization when `pdl`: the kernel may
// be scheduled while its predecessor drains; it orders itself after the
// predecessor with griddepcontrol.wait before it reads the predecessor's
// results or writes anything.
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                   cudaStream_t st, bool pdl, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// The same for a kernel run by clusters of `cluster` CTAs along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                            cudaStream_t st, unsigned cluster, bool pdl, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pairs(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                         cudaStream_t st, bool pdl, Args &&...args) {
  return launch_clusters(kernel, grid, block, smem, st, 2, pdl, std::forward<Args>(args)...);
}

}  // namespace

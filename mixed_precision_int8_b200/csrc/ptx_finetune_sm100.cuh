// Further inline-PTX wrappers (beside ptx_sm100.cuh) for the operators next to
// the projection: untiled bulk copies, cp.async, MN-major and unswizzled
// matrix descriptors, distributed shared memory.
#pragma once

#include <cstdint>

#include "ptx_sm100.cuh"

namespace llmint8 {

// Whether the phase of parity `parity` of barrier `bar` has completed; never
// suspends the thread.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Contiguous bulk copy global -> shared of `bytes` bytes (both addresses
// 16-byte aligned, bytes a multiple of 16), completion counted in bytes on
// `bar`. No multicast.
__device__ __forceinline__ void bulk_load_1d(uint32_t dst, const void *src, uint32_t bytes,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

// Wait until no committed bulk group but the last one is still reading shared
// memory.
__device__ __forceinline__ void bulk_wait_group_read1() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}

// Warp-collective: lane i reads 8 consecutive 32-bit TMEM columns of TMEM lane
// (base lane of this warp's quarter + i).
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7])
      : "r"(taddr)
      : "memory");
}

// Shared-memory matrix descriptor for an MN-major operand tile (the reduction
// index outside, the M or N index contiguous) in 128-byte-swizzled blocks of
// 64 fp16 columns: each block's rows are 128 bytes, one per value of the
// reduction index, and blocks follow each other block_bytes apart. Leading
// byte offset: from one 64-column block to the next; stride byte offset: from
// one group of 8 reduction rows to the next (1024). Descriptor version 1,
// layout 2 = SWIZZLE_128B.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t block_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)(block_bytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// Shared-memory matrix descriptor for an operand tile of unswizzled core
// matrices (8 rows of 16 bytes, contiguous). K-major: a core matrix is 8 rows
// (M or N) of 8 reduction values; lead = bytes to the next one along K,
// stride = along M / N. MN-major: 8 reduction values' rows of 8 M / N columns;
// lead = bytes to the next one along K, stride = along M / N.
__device__ __forceinline__ uint64_t smem_desc_core(uint32_t saddr, uint32_t lead,
                                                   uint32_t stride) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)(lead >> 4) << 16;
  d |= (uint64_t)(stride >> 4) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}

// 16-byte asynchronous copy global -> shared; zeros when `valid` is false
// (src is then not read).
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// Wait until at most N committed groups are still under way.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Reads shared memory of a CTA of the cluster (shared::cluster address).
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Arrive on an mbarrier given by its shared::cluster address, with a release at
// cluster scope of accesses to this CTA's shared memory only: unlike
// mbar_arrive_cluster it does not wait for the thread's other writes to reach
// the cluster's point of coherence (a round trip to L2 under load). For signals
// about shared memory, whose waiter acquires at cluster scope.
__device__ __forceinline__ void mbar_arrive_smem(uint32_t cluster_bar) {
  asm volatile(
      "fence.release.sync_restrict::shared::cta.cluster;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
      : "memory");
}

// mbar_wait_bounded for a barrier on which threads of the other CTA arrive: what
// they released at cluster scope is acquired at cluster scope.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool mbar_wait_bounded_cluster(uint32_t bar, uint32_t parity,
                                                          volatile int *abort_flag, int *status,
                                                          int code, uint64_t limit_ns) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > limit_ns) {
      *abort_flag = 1;
      atomicOr(status, code);
      return false;
    }
  }
}

// Instruction descriptor of tcgen05.mma kind::f16 (idesc_f16_f32) with the
// operands' majors chosen: bit 15 (A) and 16 (B) set for MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32_mn(uint32_t M, uint32_t N, bool a_mn,
                                                        bool b_mn) {
  return idesc_f16_f32(M, N) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
}

}  // namespace llmint8

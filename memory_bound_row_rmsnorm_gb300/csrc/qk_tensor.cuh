// qk_tensor.cuh -- tcgen05 (5th-generation tensor core) and tensor-map TMA
// primitives for pairs of CTAs, as inline PTX.
//
// A cluster of two CTAs works on one 256-row tile: each CTA holds 128 rows of A
// and half of B's rows in its shared memory, one thread of the even CTA (the
// leader) issues the products for both, and each CTA's tensor memory (TMEM)
// receives its own 128 rows of fp32 sums, one row a lane.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "qk_device.cuh"

namespace qk {

// Tile loads of a 3-D tensor (inner, row, plane).  dst: this CTA's shared
// memory; bar: the barrier that counts the bytes, which may be the other CTA's.
// x is a multiple of 8 elements (16 bytes) at every call.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void prefetch_tensor_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// One arrival on a barrier of any CTA of the cluster (a shared::cluster
// address).  It tells that registers were loaded, which needs no release beyond
// this CTA: at cluster scope it would wait for the thread's global stores.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// TMEM columns for the pair: the same warp of both CTAs allocates and frees.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(columns)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t tmem, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns) : "memory");
}

__device__ __forceinline__ void tcgen05_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tcgen05_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D[tmem] (+)= A B^T for bf16 operands described by shared-memory descriptors.
__device__ __forceinline__ void mma_bf16_pair(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}
// Arrives on the barrier at this offset in both CTAs once every product issued
// so far is done.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(uint16_t(3))
      : "memory");
}

// 16 columns of this warp's 32 TMEM lanes: v[j] is column j of the lane's row.
// The loads of several calls are in flight together until tmem_load_wait().
__device__ __forceinline__ void tmem_load_16(uint32_t tmem, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(tmem)
      : "memory");
}
// Completes the loads before; their registers are only valid behind it, so they pass through.
__device__ __forceinline__ void tmem_load_wait(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}

// Shared-memory descriptor of an operand tile in 128-byte swizzled rows.
// K-major: rows of 64 k; 8-row groups follow each other at 1024 bytes (sbo).
// MN-major: rows of 64 m (or n), one row a k; 8-row groups at 1024 bytes (sbo),
// the next 64 m at `lbo` bytes.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lbo) {
  return uint64_t((addr >> 4) & 0x3fffu) | (uint64_t((lbo >> 4) & 0x3fffu) << 16) | (uint64_t(1024u >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// Instruction descriptor: bf16 x bf16 -> fp32, 256 rows a pair, n columns.
__host__ __device__ constexpr uint32_t instruction_desc(bool a_mn, bool b_mn, uint32_t n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) | ((n >> 3) << 17) |
         ((256u >> 4) << 24);
}

}  // namespace qk

// mxq_tc_ptx.cuh -- sm_103a helpers for the tensor-core products: tensor
// memory, block-scaled tcgen05.mma, its operand and instruction descriptors,
// and cluster synchronisation.
#pragma once

#include <cstdint>

#include "mxq_ptx.cuh"

namespace mxq {

// One thread of a converged warp.  The compiler then knows that the branch has
// one thread and issues tensor-core and copy instructions straight from uniform
// registers: 128 clocks a 128 x 256 x 32 instruction, the tensor cores' own
// rate, against 141 under `lane == 0`, and 95 against 141 for 128 x 128.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// ---------------------------------------------------------------------------
// Tensor memory
// ---------------------------------------------------------------------------

// In all of this a kernel keeps to one CTAS: 1, or 2 for pairs of CTAs that
// work on one tile (cta_group::2), where the pair's first CTA issues.

// Whole-warp allocation of `cols` columns (a power of two >= 32); the address
// is written to shared memory at `dst`.  With pairs, one warp of each CTA.
template <int CTAS>
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
  if constexpr (CTAS == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(dst), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(dst), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}

template <int CTAS>
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
  if constexpr (CTAS == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;"
                 :: "r"(addr), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                 :: "r"(addr), "r"(cols) : "memory");
}

// 32 lanes x 32 columns of fp32: lane i of the warp receives columns
// [col, col + 32) of tensor-memory lane 32 * (warp % 4) + i.
__device__ __forceinline__ void tmem_load_x32(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
        "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
        "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr));
}

// The values of every earlier tmem_load of this thread have arrived.
__device__ __forceinline__ void tmem_wait_load() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_before_sync() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_after_sync() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Descriptors
// ---------------------------------------------------------------------------

// A K-major operand tile in shared memory, rows of 128 bytes with the
// 128-byte swizzle: groups of 8 rows are 1024 bytes apart.  Advancing along K
// by 32 bytes adds 2 to the descriptor.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (1ull << 16) | (64ull << 32) |
         (1ull << 46) | (2ull << 61);
}

// A 512-byte scale tile (32 rows of 16 bytes, no swizzle): groups of 8 rows
// are 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (8ull << 32) | (1ull << 46);
}

// Instruction descriptor of kind::mxf8f6f4 with both operands E4M3 and K-major
// and E8M0 scales, for an m x n tile; `id` is the byte of each 32-bit scale
// word that holds this instruction's scales.
__host__ __device__ constexpr uint32_t mxf8_idesc(uint32_t m, uint32_t n, uint32_t id) {
  return (id << 4) | ((n >> 3) << 17) | (1u << 23) | ((m >> 7) << 27) | (id << 29);
}

// ---------------------------------------------------------------------------
// Asynchronous tensor-core work (issued by one thread; executed in order)
// ---------------------------------------------------------------------------

// Copies a scale tile to 4 tensor-memory columns (of each CTA, from its own
// shared memory): byte 16 r + 4 c + i goes to lane r (and r + 32, r + 64, r +
// 96), column c, byte i.
template <int CTAS>
__device__ __forceinline__ void tc_copy_scales(uint32_t tmem, uint64_t desc) {
  if constexpr (CTAS == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" :: "r"(tmem), "l"(desc)
                 : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(tmem), "l"(desc)
                 : "memory");
}

// D (+)= (A * scale_a) (B * scale_b)^T over 32 values of K.  With pairs each
// CTA holds half of A's rows (and of D's) and half of B's rows, and all of B's
// scales.
template <int CTAS>
__device__ __forceinline__ void tc_mma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            uint32_t scale_a, uint32_t scale_b, bool accumulate) {
  if constexpr (CTAS == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(scale_a), "r"(scale_b),
           "r"(static_cast<uint32_t>(accumulate)) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(scale_a), "r"(scale_b),
           "r"(static_cast<uint32_t>(accumulate)) : "memory");
}

// Arrives once on `bar` (with pairs: on both CTAs' barriers at this place) when
// everything this thread has issued has completed.
template <int CTAS>
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  if constexpr (CTAS == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" :: "r"(bar), "h"(static_cast<uint16_t>(3)) : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(bar) : "memory");
}

// ---------------------------------------------------------------------------
// Clusters, barriers and copies
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}

// The shared-memory address `addr` of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
  return at;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr(addr, rank))
               : "memory");
  return v;
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(cluster_addr(addr, rank))
               : "memory");
  return v;
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}

// Arrival on a barrier of the cluster (an address of cluster_addr).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(bar)
               : "memory");
}

// mbar_wait_bounded that also sees what the cluster's CTAs wrote before their
// arrivals.
__device__ __forceinline__ bool mbar_wait_bounded_cluster(uint32_t bar, uint32_t parity,
                                                          uint64_t timeout_ns) {
  uint64_t t0 = 0;
  while (true) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    if (done) return true;
    const uint64_t now = global_timer_ns();
    if (t0 == 0) t0 = now;
    else if (now - t0 > timeout_ns) return false;
  }
}

// 3-D TMA tile store that adds fp32 values to what is there.
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, uint32_t src, int x, int y,
                                           int z) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%2, %3, %4}], [%1];"
      :: "l"(map), "r"(src), "r"(x), "r"(y), "r"(z) : "memory");
}

// 3-D TMA tile load into this CTA's shared memory, completing on a barrier of
// the pair's first CTA (an address of cluster_addr).
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int x,
                                                 int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

// 3-D TMA tile load global -> shared, completing on `bar`.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

}  // namespace mxq

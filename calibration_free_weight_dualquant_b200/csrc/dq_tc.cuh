// dq_tc.cuh -- fifth-generation tensor-core primitives (tcgen05, sm_100a) of
// the block-scaled products: descriptors, tensor-memory allocation, the copy
// of block scales into tensor memory, the multiply-accumulate and its commit,
// and tensor-memory loads.
#pragma once

#include <cstdint>

#include "dq_device.cuh"

namespace dq {

// What the formats need of a block-scaled multiply-accumulate.  One K tile is
// 128 bytes of codes a row, four instructions of 32 bytes each.
template <int FMT>
struct TcFormat {
  static constexpr bool kByteCodes = FMT == FMT_MXFP8;
  static constexpr int kTileK = kByteCodes ? 128 : 256;                   // columns of a K tile
  static constexpr int kGroup = FMT == FMT_NVFP4 ? 16 : 32;
  static constexpr int kScaleBytes = kTileK / kGroup;                     // block scales of a row and K tile: 16, 8 or 4
  static constexpr int kAtoms = kScaleBytes / 4;                          // 4-byte scale words of a row and K tile
  // Instruction descriptor without the sizes' and scale ids' fields: operand
  // types (E4M3 0, or E2M1 1), E8M0 (1) or E4M3 (0) block scales.
  static constexpr uint32_t kIdesc =
      (kByteCodes ? 0u : (1u << 7) | (1u << 10)) | (FMT == FMT_NVFP4 ? 0u : 1u << 23);
  // scale word and byte within it of instruction k of a K tile
  __host__ __device__ static constexpr int atom(int k) { return k * kAtoms / 4; }
  __host__ __device__ static constexpr int byte(int k) { return kAtoms == 4 ? 0 : (kAtoms == 2 ? (k & 1) * 2 : k); }
};

// Instruction descriptor of an M x N tile whose scales start at byte `id` of
// their words.
template <int FMT>
__host__ __device__ constexpr uint32_t tc_idesc(int M, int N, int id) {
  return TcFormat<FMT>::kIdesc | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 7) << 27) | ((uint32_t)id << 29) |
         ((uint32_t)id << 4);
}

// Shared-memory descriptor of K-major rows of 128 bytes in the 128-byte
// swizzle (8-row atoms 1024 bytes apart).
__device__ __forceinline__ uint64_t tc_desc_sw128(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// Shared-memory descriptor of a 512-byte block of scale words: 32 rows of 16
// bytes, 8-row atoms 128 bytes apart, no swizzle.
__device__ __forceinline__ uint64_t tc_desc_scales(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (8ull << 32) | (1ull << 46);
}

template <int COLS>
__device__ __forceinline__ void tc_alloc(uint32_t smem_dst) {  // one whole warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(COLS) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
template <int COLS>
__device__ __forceinline__ void tc_dealloc(uint32_t taddr) {  // the warp that allocated
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(COLS));
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 512 bytes of scale words to 4 columns of all four lane quarters.
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <int FMT>
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t accumulate) {
  if (FMT == FMT_NVFP4)
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else if (FMT == FMT_MXFP4)
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Arrives on `bar` when everything this thread issued to the tensor core is done.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 16 consecutive columns of this warp's lane quarter, one lane a thread.
__device__ __forceinline__ void tc_load16(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tc_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// fp32 value at this CTA's shared address `addr` in the cluster's CTA `rank`.
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

}  // namespace dq

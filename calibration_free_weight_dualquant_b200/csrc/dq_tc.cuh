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
  static constexpr int kPiece = 8 / kAtoms;                               // K tiles of a 32-byte piece of a row's scales
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

// CG: CTAs that work on one tile (1, or the two of a pair).
template <int CG, int COLS>
__device__ __forceinline__ void tc_alloc(uint32_t smem_dst) {  // one whole warp (of each CTA)
  if (CG == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
}
template <int CG, int COLS>
__device__ __forceinline__ void tc_dealloc(uint32_t taddr) {  // the warp that allocated
  if (CG == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(COLS));
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(COLS));
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 512 bytes of scale words to 4 columns of all four lane quarters (of a pair:
// each CTA's own words, at the same place in its shared memory).
template <int CG>
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint64_t desc) {
  if (CG == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

#define DQ_TC_MMA(CGS, KIND)                                                                                            \
  asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"                                                              \
               "tcgen05.mma.cta_group::" CGS ".kind::" KIND " [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),            \
               "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                                          \
               : "memory")
template <int FMT, int CG>
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t accumulate) {
  if (CG == 1) {
    if (FMT == FMT_NVFP4)
      DQ_TC_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
    else if (FMT == FMT_MXFP4)
      DQ_TC_MMA("1", "mxf4.block_scale.scale_vec::2X");
    else
      DQ_TC_MMA("1", "mxf8f6f4.block_scale.scale_vec::1X");
  } else {
    if (FMT == FMT_NVFP4)
      DQ_TC_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
    else if (FMT == FMT_MXFP4)
      DQ_TC_MMA("2", "mxf4.block_scale.scale_vec::2X");
    else
      DQ_TC_MMA("2", "mxf8f6f4.block_scale.scale_vec::1X");
  }
}
#undef DQ_TC_MMA

// Arrives on `bar` (of a pair whose even CTA has the cluster rank `leader`: on
// both CTAs' barriers at that place) when everything this thread issued to the
// tensor core is done.
template <int CG>
__device__ __forceinline__ void tc_commit(uint64_t* bar, uint32_t leader = 0) {
  if (CG == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_u32(bar)),
                 "h"((uint16_t)(3u << leader))
                 : "memory");
}

// Brings a tensor map (a kernel parameter) close before its first copy.
__device__ __forceinline__ void tma_prefetch_map(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Tensor copy of a pair's CTA into its own shared memory, completing on the
// even CTA's barrier (the rank is bit 24 of a shared address in a cluster).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const void* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar) & 0xFEFFFFFFu)
      : "memory");
}

// Arrival on the barrier at this place in the cluster's CTA `rank`, released to
// the cluster: what it publishes are writes to this CTA's shared memory, so the
// fence is the one of that memory alone.  (A release of all memory waited for the
// warp's global traffic, about 1500 clocks: NVFP4 8192 x 14336 x 4096 470 us
// against 273 then.)  Waited for with mbar_try_wait_cluster.
__device__ __forceinline__ void mbar_arrive_cluster(uint64_t* bar, uint32_t rank) {
  asm volatile(
      "{\n.reg .b32 a;\nmapa.shared::cluster.u32 a, %0, %1;\n"
      "fence.release.sync_restrict::shared::cta.cluster;\n"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [a];\n}" ::"r"(smem_u32(bar)),
      "r"(rank)
      : "memory");
}
// mbar_try_wait on a barrier of this CTA that another CTA of the cluster arrives
// at or copies to: acquires the cluster's shared memory.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, unsigned parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n"
      "@p fence.acquire.sync_restrict::shared::cluster.cluster;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// `bytes` of a barrier's expected copies that will not come.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, unsigned bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
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
__device__ __forceinline__ void tc_load32(uint32_t taddr, uint32_t* v) {
  tc_load16(taddr, v);
  tc_load16(taddr + 16, v + 16);
}
// Waits for this thread's tensor-memory loads; v passes through, so that no use
// of the loaded values moves above the wait.
__device__ __forceinline__ void tc_load_wait16(uint32_t* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                 "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])::"memory");
}
__device__ __forceinline__ void tc_load_wait32(uint32_t* v) {
  tc_load_wait16(v);
  tc_load_wait16(v + 16);
}

// True in one lane of a converged warp.  The compiler keeps the operands of the
// tensor-core instructions under it in uniform registers; under `lane == 0` it
// moves every operand there first (measured: about 60 clocks an instruction).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The two halves of one more meeting of the cluster, before which nobody has written anything for the others.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// If `on`, a word to this CTA's shared address `addr` in the cluster's CTA `rank`.
__device__ __forceinline__ void st_cluster_if(bool on, uint32_t addr, uint32_t rank, uint32_t v) {
  asm volatile(
      "{\n.reg .b32 a;\n.reg .pred p;\nsetp.ne.b32 p, %3, 0;\n@p mapa.shared::cluster.u32 a, %0, %1;\n"
      "@p st.shared::cluster.b32 [a], %2;\n}" ::"r"(addr),
      "r"(rank), "r"(v), "r"((int)on)
      : "memory");
}
// Four fp32 values at this CTA's shared address `addr` in the cluster's CTA `rank`.
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

}  // namespace dq

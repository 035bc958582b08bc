// dq_matmul.cu -- the product of quantized activations and a quantized weight
// matrix, both microscaled in the same format:
//
//   Y[t][n] = s_x s_w sum_k (a_x[t][k/G] q_x[t][k]) (a_w[n][k/G] q_w[n][k])
//
// (DualQuant arXiv 2610.13767 summary, section 4.4: X W^T = (X D_b) Q^T D_a;
// the column scales b are in q_x already).  Sums are held in fp32, multiplied by
// the tensor scales in fp32 and rounded once more, to the output type.
#include <climits>

#include <cuda.h>
#include <cudaTypedefs.h>  // PFN_cuTensorMapEncodeTiled
#include <math_constants.h>

#include "dq.h"
#include "dq_device.cuh"
#include "dq_fast.cuh"
#include "dq_internal.h"
#include "dq_launch.h"
#include "dq_tc.cuh"

namespace dq {

struct MatmulProblem {
  const unsigned char* xq;
  const unsigned char* xs;  // [T][K/G]
  const float* x_sT;        // NULL: 1
  const unsigned char* wq;
  const unsigned char* ws;  // [N][K/G]
  const float* w_sT;
  void* y;
  int y_dt;
  int64_t T, N, K;
  unsigned* flags;  // the workspace's status word, or NULL
};

// The tensor scales' product as f1 * f2, applied one after the other: f2 is 1
// unless the product leaves fp32's normal range, and finite: beyond 2^255 the
// largest number does, since the smallest nonzero sum, 2^-20, leaves the range all
// the same and a zero sum stays zero.
__device__ __forceinline__ void tensor_factors(const MatmulProblem& p, float& f1, float& f2) {
  f1 = f2 = 1.f;
  if (p.x_sT == nullptr) return;
  const double s = (double)*p.x_sT * (double)*p.w_sT;
  const double a = fabs(s);
  if (a >= 0x1p-126 && a <= 0x1p127 || a == 0.0 || !(a <= 1.7976931348623157e308)) {
    f1 = (float)s;
  } else {
    const int e = ilogb(s) < 0 ? -126 : 127;
    f1 = scalbnf(1.f, e);
    const double top = 3.4028234663852886e38;
    f2 = (float)fmin(fmax(scalbn(s, -e), -top), top);
  }
}

__device__ __forceinline__ void y_store(void* y, int dt, int64_t i, float v) {
  if (dt == DT_F32)
    reinterpret_cast<float*>(y)[i] = v;
  else if (dt == DT_BF16)
    reinterpret_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
  else
    reinterpret_cast<__half*>(y)[i] = __float2half_rn(v);
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, int dt) {
  uint32_t r;
  if (dt == DT_BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four neighbouring outputs from element i, `n` of them inside the row.  vec:
// such fours start at multiples of their size.
__device__ __forceinline__ void y_store4(void* y, int dt, int64_t i, const float* v, int64_t n, bool vec) {
  if (vec && n >= 4) {
    if (dt == DT_F32) {
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(y) + i) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      const uint32_t a = pack16(v[0], v[1], dt), b = pack16(v[2], v[3], dt);
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(y) + i) = make_uint2(a, b);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) y_store(y, dt, i + k, v[k]);
  }
}

// Grid value of one code.
template <int FMT>
__device__ __forceinline__ float code_value(const unsigned char* q, int64_t at) {
  if (FMT == FMT_MXFP8) {
    const unsigned char c = q[at];
    const float v = (c & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FC00000u) : e4m3_value(c);
    return c & 0x80u ? -v : v;
  }
  const uint32_t c = (q[at >> 1] >> (4 * (at & 1))) & 15u;
  const uint32_t m = c & 7u;
  const float v = m < 4 ? 0.5f * m : (m == 4 ? 2.f : (m == 5 ? 3.f : (m == 6 ? 4.f : 6.f)));
  return c & 8u ? -v : v;
}

// Any shape and alignment: a 64 x 64 tile of Y per CTA, 16-column slices of
// both operands' codes decoded to fp32 in shared memory, 4 x 4 outputs per
// thread.  A slice lies within one block of each operand, so its sum of code
// products (exact for E2M1, whose products are multiples of 1/4 up to 36; fp32
// additions for E4M3) is multiplied by the two block scales at once; powers of
// two add their exponents, so that scales at the ends of their range do not
// overflow on the way.  Bound by fp32 arithmetic and the decoding:
// 200 x 400 x 400 NVFP4 87 us (0.7 TFLOP/s).
// Taken only where the copies of the tensor-core kernels cannot read the codes:
// rows of codes that do not start at multiples of 16 bytes (a 4-bit row length that
// is not a multiple of 32, or such an address).
template <int FMT>
__global__ void __launch_bounds__(256) k_matmul_any(MatmulProblem p) {
  constexpr int G = FMT == FMT_NVFP4 ? 16 : 32;
  __shared__ float xs[16][68], ws[16][68];
  __shared__ unsigned char xa[64], wa[64];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int64_t tiles_n = (p.N + 63) / 64, nb = p.K / G;
  const int64_t t0 = blockIdx.x / tiles_n * 64, n0 = blockIdx.x % tiles_n * 64;
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0 && tid == 0 && p.flags) *p.flags = 0;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < p.K; k0 += 16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (tid >> 4) + 16 * i, k = tid & 15;
      xs[k][r] = t0 + r < p.T ? code_value<FMT>(p.xq, (t0 + r) * p.K + k0 + k) : 0.f;
      ws[k][r] = n0 + r < p.N ? code_value<FMT>(p.wq, (n0 + r) * p.K + k0 + k) : 0.f;
    }
    if (tid < 64)
      xa[tid] = t0 + tid < p.T ? p.xs[(t0 + tid) * nb + k0 / G] : 0;
    else if (tid < 128)
      wa[tid - 64] = n0 + tid - 64 < p.N ? p.ws[(n0 + tid - 64) * nb + k0 / G] : 0;
    __syncthreads();
    float dot[4][4] = {};
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float4 a = *reinterpret_cast<const float4*>(&xs[k][4 * ty]), b = *reinterpret_cast<const float4*>(&ws[k][4 * tx]);
      const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) dot[i][j] = fmaf(av[i], bv[j], dot[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const unsigned ea = xa[4 * ty + i], ew = wa[4 * tx + j];
        float v;
        if (FMT == FMT_NVFP4) {
          v = dot[i][j] * (e4m3_value(ea & 0x7Fu) * e4m3_value(ew & 0x7Fu));
          if ((ea & 0x7Fu) == 0x7Fu || (ew & 0x7Fu) == 0x7Fu) v = __uint_as_float(0x7FC00000u);
        } else {
          v = ea == 255u || ew == 255u ? __uint_as_float(0x7FC00000u) : scalbnf(dot[i][j], (int)(ea + ew) - 254);
        }
        acc[i][j] += v;
      }
    __syncthreads();
  }
  float f1, f2;
  tensor_factors(p, f1, f2);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t t = t0 + 4 * ty + i, n = n0 + 4 * tx + j;
      if (t < p.T && n < p.N) y_store(p.y, p.y_dt, t * p.N + n, acc[i][j] * f1 * f2);
    }
}

// ---------------------------------------------------------------------------
// Tensor-core product: a CTA computes the tile of 128 output features and BN
// tokens, Y^T = W X^T, so that few tokens still fill the tensor core's 128
// rows.  Codes go by TMA into 128-byte-swizzled shared memory as they are
// stored; block scales are read as stored, one row's bytes of a K tile a lane,
// and written to shared memory transposed into the words that tcgen05.cp moves
// to tensor memory; tcgen05.mma multiplies codes and scales and sums in fp32
// in tensor memory.  Where there are fewer tiles than SMs the columns are
// split over the CTAs of a cluster, whose partial tiles are joined through
// distributed shared memory in rank order (no atomics: equal calls give equal
// bits).
//
// Up to 64 tokens the weight's bytes bound it, and below some 30 MB the fixed 3.5
// us of a tile's start, join and store.  1 token (GPU time): NVFP4 28672 x 4096
// 15.2 us = 4.3 TB/s, 4096 x 4096 5.4 us (1.8 TB/s); MXFP8 4096 x 14336 13.1 us =
// 4.6 TB/s.  16 tokens MXFP4 4096 x 14336: 8.1 us = 3.9 TB/s.  More tokens, as long
// as the tiles are few (tc_ns): 64 or 128 a tile; 1000 x 1001 x 1056 NVFP4 7.2 us,
// 12.1 with pairs of CTAs.
//
// Warps: 0 issues the copies, 1 the tensor-core work; 2 and 4 bring the
// weights' scales, 3 and 5 the tokens', and the four write the tile out (warp w
// reads tensor-memory lanes 32 (w % 4) ..).
constexpr int kMmThreads = 192;
constexpr int kMmMaxStages = 8;
constexpr int kMmSmem = 220 * 1024;  // most of a CTA

template <int FMT, int BN>
struct MmGeo {
  using F = TcFormat<FMT>;
  static_assert(BN <= 128, "one 128-row block of token scales");
  static constexpr int kA = 128 * 128, kB = BN * 128;
  static constexpr int kStage = kA + kB;
  static constexpr int kScales = 2 * 4096;  // a slot of the piece ring: 32 bytes of 128 features and of 128 tokens
  static constexpr int kAccCols = BN < 32 ? 32 : BN;
  static constexpr int kSfACol = kAccCols, kSfBCol = kAccCols + 16;
  static constexpr int kCols = kAccCols + 16 + 16;
  static constexpr int kAlloc = kCols <= 64 ? 64 : (kCols <= 128 ? 128 : (kCols <= 256 ? 256 : 512));
};

// Block scales of a lane's four rows (row0 + lane + 32 q): the 32-byte piece
// `piece` of each row, one memory sector where rows are aligned, as words
// w[q][0 .. 7]; zeros past the matrix.  U: what the address and the length of
// every row are multiples of, 32, 16, 8 or (1) nothing.  With 1, three aligned
// 16-byte reads are shifted into place, and pieces whose aligned window leaves the
// scales' memory are read by bytes afterwards.  All reads of the four rows are
// under way before the first is used.
template <int U>
__device__ __forceinline__ void load_scales(const unsigned char* s, int64_t row0, int64_t rows, int64_t nb, int64_t piece,
                                            uint32_t (*w)[8]) {
  unsigned here;  // keeps the loads, free among themselves, behind the wait for the grid before
  asm volatile("mov.u32 %0, 0;" : "=r"(here)::"memory");
  if constexpr (U > 1) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t r = row0 + (threadIdx.x & 31) + 32 * q;
      const unsigned char* p = s + r * nb + piece * 32;
      const int64_t left = r < rows ? nb - piece * 32 : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) w[q][j] = 0;
      if constexpr (U == 32) {
        if (left > 0)
          asm("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
              : "=r"(w[q][0]), "=r"(w[q][1]), "=r"(w[q][2]), "=r"(w[q][3]), "=r"(w[q][4]), "=r"(w[q][5]), "=r"(w[q][6]),
                "=r"(w[q][7])
              : "l"(p), "r"(here));
      } else if constexpr (U == 16) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (16 * i < left) {
            const uint4 v = reinterpret_cast<const uint4*>(p)[i];
            w[q][4 * i] = v.x, w[q][4 * i + 1] = v.y, w[q][4 * i + 2] = v.z, w[q][4 * i + 3] = v.w;
          }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (8 * i < left) {
            const uint2 v = reinterpret_cast<const uint2*>(p)[i];
            w[q][2 * i] = v.x, w[q][2 * i + 1] = v.y;
          }
      }
    }
  } else {
    uint4 v[4][3];
    const int64_t r0 = row0 + (threadIdx.x & 31);
    const unsigned char* const p0 = s + r0 * nb + piece * 32;
    const unsigned char* const end = s + rows * nb;
    const int have = (int)min((int64_t)32, nb - piece * 32);  // bytes of the piece that belong to a row
    bool bytes = false;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const unsigned char* p = p0 + 32 * q * nb;
      const unsigned char* a = p - ((uintptr_t)p & 15u);
      const bool on = r0 + 32 * q < rows, in = on && a >= s && a + 48 <= end;
#pragma unroll
      for (int i = 0; i < 3; ++i) v[q][i] = in ? reinterpret_cast<const uint4*>(a)[i] : make_uint4(0, 0, 0, 0);
      bytes |= on && !in;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const unsigned sh = (unsigned)(uintptr_t)(p0 + 32 * q * nb) & 15u;
      uint32_t t[12];
#pragma unroll
      for (int i = 0; i < 3; ++i) t[4 * i] = v[q][i].x, t[4 * i + 1] = v[q][i].y, t[4 * i + 2] = v[q][i].z, t[4 * i + 3] = v[q][i].w;
#pragma unroll
      for (int j = 0; j < 10; ++j) t[j] = sh & 8u ? t[j + 2] : t[j];
#pragma unroll
      for (int j = 0; j < 9; ++j) t[j] = sh & 4u ? t[j + 1] : t[j];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int more = have - 4 * j;
        const uint32_t x = __funnelshift_r(t[j], t[j + 1], 8 * (sh & 3u));
        w[q][j] = more >= 4 ? x : (more > 0 ? x & (0xFFFFFFFFu >> (32 - 8 * more)) : 0u);
      }
    }
    if (bytes) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const unsigned char* p = p0 + 32 * q * nb;
        const unsigned char* a = p - ((uintptr_t)p & 15u);
        if (r0 + 32 * q < rows && !(a >= s && a + 48 <= end)) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (4 * j + i < have) w[q][j] |= (uint32_t)p[4 * j + i] << (8 * i);
        }
      }
    }
  }
}

// How long waits last, and what a self-test withholds: a role of the CTA `rank` of
// every cluster stops as if its wait had run out, after `at` K tiles (role 0, the
// copies) or pieces of 32 bytes a row (1, the weights' scales; 2, the tokens').
// Eight bytes, for a launch's parameters are read from memory a 64-byte line at a time.
struct MmWait {
  unsigned limit_ns = (unsigned)kWaitLimitNs;
  unsigned stop = 0xFFFFFFFFu;  // rank, role and at, in 4, 2 and 26 bits
};
constexpr unsigned kStopAtBits = 26;
__host__ __device__ __forceinline__ unsigned stop_key(int rank, int role) { return (unsigned)rank << 2 | (unsigned)role; }
// The count at which this CTA's role stops.
__device__ __forceinline__ unsigned stop_of(const MmWait& w, int rank, int role) {
  return w.stop >> kStopAtBits == stop_key(rank, role) ? w.stop & ((1u << kStopAtBits) - 1) : 0xFFFFFFFFu;
}

// Bounded wait for a ring barrier, by the clock alone: the header's flags may
// still hold what the workspace held before this launch.  CLUSTER: another CTA
// signals the barrier too.
template <bool CLUSTER>
__device__ __forceinline__ bool mm_wait(uint64_t* bar, unsigned parity, unsigned limit_ns, unsigned* flags) {
  auto done = [&] { return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
  if (done()) return true;
  const unsigned long long t0 = global_ns();
  while (!done()) {
    if (global_ns() - t0 > limit_ns) {
      if (flags) atomicOr(flags, kFlagTimeout);
      return false;
    }
  }
  return true;
}

// mbar_drain where the phase is nearly always over: the clock is not read then.
__device__ __forceinline__ void mm_drain(uint64_t* bar, unsigned parity) {
  if (!mbar_try_wait(bar, parity)) mbar_drain(bar, parity);
}

// A place in the ring, kept by every role over all tiles of a CTA.
struct MmSlot {
  int slot = 0;
  unsigned phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++slot == stages) slot = 0, phase ^= 1;
  }
};

// Scales travel in pieces of 32 bytes a row, one memory sector: the scales of
// 2, 4 or 8 K tiles.  (Read a K tile at a time, the same sector would come from
// L2 every time, and every K tile would cost its own barriers.)  Each 128-row
// block has two warps that take turns, so that one reads while the other waits
// or writes: the proxy fence that publishes a piece waits for the warp's own
// reads in flight.  A slot is free when its piece's multiply-adds are done, and
// filling it takes longer than those of one K tile, so two slots do while a
// piece is 4 or 8 tiles, and the pairs' kernel has three for NVFP4's pieces of
// two (8192 x 14336 x 4096: 215 us against 222).  The kernel of few tokens waits
// for the weight's bytes and leaves the room to them.  (A warp may wait for a
// slot's barrier by parity: when it filled piece p - 2 it waited for p - 2 - SLOTS,
// so the phase two before the one that it waits for now is over.)
constexpr int kScaleSlots = 2;
struct ScaleTurn {
  int turn;            // 0 or 1
  unsigned piece = 0;  // pieces of the block so far, over all its tiles
};
// Slot and phase of a piece's use of the ring, for those who take every piece.
template <int SLOTS>
struct ScaleSlot {
  int slot = 0;
  unsigned phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == SLOTS) slot = 0, phase ^= 1;
  }
};

// A warp's share of one block's scales of the K tiles k0 .. k0 + n - 1.  Slot i
// of the ring starts at ring + i * slot_bytes; the words of K tile u of a piece
// and scale word j are the 512-byte block u * kAtoms + j, block_bytes apart.
// PAIR: the arrival goes to the cluster's CTA `leader`.
template <bool PAIR, int SLOTS, int U>
__device__ __forceinline__ bool scale_loop(ScaleTurn& t, int tiles_per_piece, const unsigned char* s, int64_t row0, int64_t rows,
                                           int64_t nb, int k0, int n, unsigned char* ring, int slot_bytes, int block_bytes,
                                           uint64_t* full, uint64_t* empty, unsigned limit_ns, unsigned* flags,
                                           unsigned stop, uint32_t leader) {
  const int lane = threadIdx.x & 31;
  const int last = (k0 + n - 1) / tiles_per_piece;
#pragma unroll 1
  for (int piece = k0 / tiles_per_piece; piece <= last; ++piece, ++t.piece) {
    if ((int)(t.piece & 1) != t.turn) continue;
    uint32_t w[4][8];
    load_scales<U>(s, row0, rows, nb, piece, w);
    if (t.piece >= stop) return false;
    const unsigned use = t.piece / SLOTS, slot = t.piece - use * SLOTS;
    if (!__all_sync(0xffffffffu, mm_wait<PAIR>(&empty[slot], (use & 1) ^ 1, limit_ns, flags))) return false;
    unsigned char* dst = ring + slot * slot_bytes + lane * 16;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      *reinterpret_cast<uint4*>(dst + j * block_bytes) = make_uint4(w[0][j], w[1][j], w[2][j], w[3][j]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (PAIR)
        mbar_arrive_cluster(&full[slot], leader);
      else
        mbar_arrive(&full[slot]);
    }
  }
  return true;
}
// `unit`: the largest power of two (32 at most) that divides the scales' address
// and the row's length.  WIDE kernels take units of 16 and 32, the others 8 and
// less: with all four in one kernel its registers spilled (NVFP4 1000 x 4096 x
// 11008: 28.5 us against 27.1).
template <bool PAIR, int SLOTS, bool WIDE>
__device__ __forceinline__ bool scale_warp(int unit, ScaleTurn& t, int tiles_per_piece, const unsigned char* s, int64_t row0,
                                           int64_t rows, int64_t nb, int k0, int n, unsigned char* ring, int slot_bytes,
                                           int block_bytes, uint64_t* full, uint64_t* empty, unsigned limit_ns, unsigned* flags,
                                           unsigned stop, uint32_t leader) {
#define DQ_SCALE_LOOP(U) \
  scale_loop<PAIR, SLOTS, U>(t, tiles_per_piece, s, row0, rows, nb, k0, n, ring, slot_bytes, block_bytes, full, empty,   \
                             limit_ns, flags, stop, leader)
  if (WIDE) return unit == 32 ? DQ_SCALE_LOOP(32) : DQ_SCALE_LOOP(16);
  return unit >= 8 ? DQ_SCALE_LOOP(8) : DQ_SCALE_LOOP(1);
#undef DQ_SCALE_LOOP
}

struct MmLaunch {
  int split;    // CTAs of a cluster, each with its share of the K tiles
  int stages;   // ring slots
  int unit_x, unit_w;  // powers of two that divide the scales' address and row
  int vec4;            // fours of outputs are aligned
  int early;           // the next grid may begin from the start on (else from the end of the multiply-adds on)
  MmWait wait;
};

template <int FMT, int BN, bool WIDE>
__global__ void __launch_bounds__(kMmThreads, WIDE ? 3 : 2)
    k_matmul_tc(const __grid_constant__ MatmulProblem p, const __grid_constant__ MmLaunch l,
                const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap) {
  using G = MmGeo<FMT, BN>;
  using F = TcFormat<FMT>;
  extern __shared__ unsigned char mm_smem[];
  __shared__ uint64_t full_t[kMmMaxStages], empty[kMmMaxStages], full_s[kScaleSlots], empty_s[kScaleSlots], acc_full, given_up;
  __shared__ uint32_t tmem_base;
  unsigned char* ring = reinterpret_cast<unsigned char*>(((uintptr_t)mm_smem + 1023) & ~(uintptr_t)1023);
  unsigned char* scales = ring + l.stages * G::kStage;
  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  const int64_t tiles_n = (p.N + 127) / 128;
  const int64_t tile = blockIdx.x / l.split;
  const uint32_t rank = blockIdx.x % l.split;
  const int64_t n0 = tile % tiles_n * 128, t0 = tile / tiles_n * BN;
  const int64_t nk = (p.K + F::kTileK - 1) / F::kTileK;
  const int64_t k0 = nk * rank / l.split;
  const int n = (int)(nk * (rank + 1) / l.split - k0);  // at least 1: split <= nk
  unsigned* const flags = p.flags;
  const unsigned limit_ns = l.wait.limit_ns;
  if (threadIdx.x == 0) {
    for (int i = 0; i < l.stages; ++i) {
      mbar_init(&full_t[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(&full_s[i], 2);
      mbar_init(&empty_s[i], 1);
    }
    mbar_init(&acc_full, 1);
    mbar_init(&given_up, 1);
    mbar_fence_init();
  }
  if (warp == 1) tc_alloc<1, G::kAlloc>(smem_u32(&tmem_base));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  if (warp == 0 && elect_one()) {
    tma_prefetch_map(&wmap);
    tma_prefetch_map(&xmap);
  }
  __syncwarp();
  if (l.split > 1) cluster_arrive();
  if (l.early) griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0 && flags) *reinterpret_cast<volatile unsigned*>(flags) = 0;
  float f1, f2;
  tensor_factors(p, f1, f2);

  int issued = 0;            // of the lane that issues copies
  uint64_t* last = nullptr;  // of the lane that issues multiply-adds: signalled when all are done
  if (warp == 0) {
    if (elect_one()) {
      int slot = 0;
      unsigned phase = 1;
      const unsigned stop = stop_of(l.wait, (int)rank, 0);
      for (; issued < n && (unsigned)issued < stop; ++issued) {
        if (!mm_wait<false>(&empty[slot], phase, limit_ns, flags)) break;
        unsigned char* st = ring + slot * G::kStage;
        mbar_arrive_expect_tx(&full_t[slot], G::kA + G::kB);
        tma_load_2d(st, &wmap, (int)((k0 + issued) * 128), (int)n0, &full_t[slot]);
        tma_load_2d(st + G::kA, &xmap, (int)((k0 + issued) * 128), (int)t0, &full_t[slot]);
        if (++slot == l.stages) slot = 0, phase ^= 1;
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      MmSlot at;
      ScaleSlot<kScaleSlots> piece;
      int it = 0;
      for (; it < n; ++it) {
        const int kt = (int)k0 + it, u = kt % F::kPiece;
        if ((it == 0 || u == 0) && !mm_wait<false>(&full_s[piece.slot], piece.phase, limit_ns, flags)) break;
        if (!mm_wait<false>(&full_t[at.slot], at.phase, limit_ns, flags)) break;
        tc_fence_after();
        const uint32_t st = smem_u32(ring + at.slot * G::kStage);
        const uint32_t sfa = smem_u32(scales + piece.slot * G::kScales) + 512 * u * F::kAtoms, sfb = sfa + 4096;
#pragma unroll
        for (int j = 0; j < F::kAtoms; ++j) {
          tc_copy_scales<1>(tmem + G::kSfACol + 4 * j, tc_desc_scales(sfa + 512 * j));
          tc_copy_scales<1>(tmem + G::kSfBCol + 4 * j, tc_desc_scales(sfb + 512 * j));
        }
        const uint64_t da = tc_desc_sw128(st), db = tc_desc_sw128(st + G::kA);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma<FMT, 1>(tmem, da + 2 * k, db + 2 * k, tc_idesc<FMT>(128, BN, F::byte(k)), tmem + G::kSfACol + 4 * F::atom(k),
                         tmem + G::kSfBCol + 4 * F::atom(k), it > 0 || k > 0);
        tc_commit<1>(&empty[at.slot]);
        if (u == F::kPiece - 1) {
          tc_commit<1>(&empty_s[piece.slot]);
          piece.next();
        }
        at.next(l.stages);
      }
      last = it == n ? &acc_full : &given_up;  // an unfinished tile's readers' wait runs out too
      tc_commit<1>(last);
    }
  } else {
    const bool of_w = (warp & 1) == 0;
    ScaleTurn t{(warp - 2) >> 1};
    scale_warp<false, kScaleSlots, WIDE>(of_w ? l.unit_w : l.unit_x, t, F::kPiece, of_w ? p.ws : p.xs, of_w ? n0 : t0, of_w ? p.N : p.T,
                      p.K / F::kGroup, (int)k0, n, scales + (of_w ? 0 : 4096), G::kScales, 512, full_s, empty_s, limit_ns, flags,
                      stop_of(l.wait, (int)rank, of_w ? 1 : 2), 0u);
  }
  __syncwarp();

  if (!l.early) griddep_launch_dependents();

  // the finished tile: tensor-memory lane = feature, column = token.  Of a split
  // tile every CTA sums its share of the tokens, in rank order; the others write
  // their parts into its shared memory.  (Reading them from there cost the latency
  // of that network once more: 1 x 4096 x 4096 MXFP8 6.2 us against 5.9.)
  const int tv = (int)min((int64_t)BN, p.T - t0);
  const int share = (tv + l.split - 1) / l.split;
  float* const parts = reinterpret_cast<float*>(scales + kScaleSlots * G::kScales);  // [rank][token][128 features]
  bool ok = true;
  if (l.split > 1) cluster_wait();  // every CTA of the cluster has begun
  if (warp >= 2) {
    ok = __all_sync(0xffffffffu, mm_wait<false>(&acc_full, 0, limit_ns, flags));
    tc_fence_after();
    const int q = warp & 3;
    const int64_t nn = n0 + 32 * q + lane;
    const uint32_t mine = smem_u32(parts) + 4 * ((int)rank * share * 128 + 32 * q + lane);
    int owner = 0, at = 0;  // of token c + i, and its place there
    constexpr int C = BN < 32 ? BN : 32;
#pragma unroll 1
    for (int c = 0; c < tv; c += C) {
      uint32_t v[C];
#pragma unroll
      for (int i = 0; i < C; i += 16) tc_load16(tmem + ((uint32_t)(32 * q) << 16) + c + i, v + i);
#pragma unroll
      for (int i = 0; i < C; i += 16) tc_load_wait16(v + i);
      if (!ok) {  // a wait ran out: no number that looks like a result
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = 0x7FC00000u;
      }
      // Branches outside, predicates within: one warp a scheduler hides no branch (with them 16 tokens took 1.1 us;
      // 64 x 4096 x 4096 NVFP4 10.3 us against 7.0).
      if (l.split > 1) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
          st_cluster_if(c + i < tv, mine + 512 * at, (uint32_t)owner, v[i]);
          ++at;
          owner += at == share;
          at = at == share ? 0 : at;
        }
      } else if (p.y_dt == DT_F32) {
        float* y = reinterpret_cast<float*>(p.y) + (t0 + c) * p.N + nn;
#pragma unroll
        for (int i = 0; i < C; ++i, y += p.N)
          if (c + i < tv && nn < p.N) *y = __uint_as_float(v[i]) * f1 * f2;
      } else {
        uint16_t* y = reinterpret_cast<uint16_t*>(p.y) + (t0 + c) * p.N + nn;
#pragma unroll
        for (int i = 0; i < C; ++i, y += p.N) {
          const uint16_t o = (uint16_t)pack16(__uint_as_float(v[i]) * f1 * f2, 0.f, p.y_dt);
          if (c + i < tv && nn < p.N) *y = o;
        }
      }
    }
    tc_fence_before();
  }
  // Whatever the waits did, all copies and multiply-adds that were issued are done before the CTA gives back its memory.
  // (A lane a slot: one after the other they took 0.2 us.)
  if (warp == 0) {
    issued = __reduce_max_sync(0xffffffffu, issued);
    if (lane < min(issued, l.stages)) mm_drain(&full_t[lane], ((issued - 1 - lane) / l.stages) & 1);
  }
  if (last) mm_drain(last, 0);
  __syncwarp();
  if (l.split > 1) {
    cluster_sync();
    const int first = (int)rank * share, total = min(share, tv - first) * 32;  // groups of four features
    for (int e = threadIdx.x; e < total; e += kMmThreads) {
      const float4* v = reinterpret_cast<const float4*>(parts) + e;
      float4 s = v[0];
      for (int r = 1; r < l.split; ++r) {
        const float4 o = v[r * share * 32];
        s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
      }
      const int64_t nn = n0 + 4 * (e & 31), at = (t0 + first + (e >> 5)) * p.N + nn;
      const float o[4] = {s.x * f1 * f2, s.y * f1 * f2, s.z * f1 * f2, s.w * f1 * f2};
      y_store4(p.y, p.y_dt, at, o, p.N - nn, l.vec4);
    }
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tc_dealloc<1, G::kAlloc>(tmem);
  }
}

// ---------------------------------------------------------------------------
// Tensor-core product of many tokens: pairs of CTAs (tcgen05 cta_group::2)
// compute tiles of 256 tokens x 256 features, persistently.  Each CTA of a
// pair holds 128 tokens and 128 features of a K tile, and the tensor cores of
// both read both halves of the features: half the shared-memory fill per
// multiply-add of a single CTA's 128 x 256 tile, which the L2's bandwidth
// would bound.  The even CTA issues the multiply-adds; copies and scale warps
// of both signal its barriers.
//
// Warps: 0 .. 7 write tiles out (lane quarter w % 4, column half w / 4), 8
// issues the copies, 9 the tensor-core work, 10 and 11 bring the tokens' scales,
// 12 .. 15 the features' (two warps a 128-row block).  A finished tile is read
// into registers, rounded to the output type and released before it is stored,
// so the next tile's multiply-adds wait for the tensor-memory reads alone.
//
// MXFP8 is bound by the tensor cores (the pipe is active 90 % of the time) and the
// last wave: 4096 x 4096 x 14336 181 us = 2.7 PFLOP/s.  NVFP4 and MXFP4 do the
// multiply-adds of the same bytes in half the time, and no unit is at its limit (NVFP4:
// tensor pipe 60 %, shared memory and L1 66 %, L2 41 %): between them stand
// the scales' way through shared memory and the wait of a tile's first multiply-adds
// for the reading of the tile before (two accumulators of 256 columns and the scales
// are more than tensor memory has).  NVFP4 8192 x 14336 x 4096 218 us = 4.4 PFLOP/s, MXFP4 8192 x 4096 x 4096
// 57 us = 4.8 PFLOP/s.  The 16-bit outputs of NVFP4 spill 16 bytes a thread.
constexpr int kPairThreads = 16 * 32;
constexpr int kPairEpilogue = 8;  // warps
constexpr int kPairStages = 5;

template <int FMT>
struct PairGeo {
  using F = TcFormat<FMT>;
  static constexpr int kA = 128 * 128, kB = 128 * 128;
  static constexpr int kStage = kA + kB;
  static constexpr int kScales = 3 * 4096;  // a slot of the piece ring: 32 bytes of 128 tokens and 256 features
  static constexpr int kSlots = F::kPiece == 2 ? 3 : 2;
  // Rows that a warp stores at a time: 32 where they fit (MXFP4 256 x 4096 x 4096: 9.9 us, 10.2 with 16).
  static constexpr int kRows = kSlots == 3 ? 16 : 32;
  static constexpr int kTurnWarp = kRows == 32 ? 32 * 32 * 4 : 32 * 17 * 4;  // a padded block of 32 x 16 words fits too
  static constexpr int kTurn = kPairEpilogue * kTurnWarp;
  static constexpr int kSmem = kPairStages * kStage + kSlots * kScales + kTurn + 1024;
  static constexpr int kScaleCols = 16 + 32;  // tensor-memory columns of one set of scales; two sets take turns
};

struct PairLaunch {
  unsigned tiles_m, tiles_n;  // their product is below 2^31
  unsigned first, end;        // the tiles of this launch
  int unit_x, unit_w;
  int rows16;  // rows of Y start at multiples of 16 bytes
  int vec4;   // fours of outputs are aligned
  int split;  // pairs of a cluster, each with its share of the K tiles of one tile
  MmWait wait;
};
constexpr int kPartPitch = 260;  // floats of a partial tile's row in shared memory: conflict-free both ways

// Tile order: bands of 8 token tiles, features within, so that the pairs at
// work at one time share operands in L2.
__device__ __forceinline__ void pair_tile(const PairLaunch& l, unsigned i, int64_t& m, int64_t& n) {
  const unsigned band = i / (8 * l.tiles_n), rest = i - band * 8 * l.tiles_n;
  const unsigned height = min(8u, l.tiles_m - band * 8), col = rest / height;
  m = band * 8 + (rest - col * height);
  n = col;
}

// Stores 32 rows x 128 bytes of a warp from (row t, column n) on, lane = row, v =
// its 32 words (16-bit outputs: two columns a word), through the warp's block of
// shared memory, so that lanes write neighbouring columns.  Rows of Y that start
// at multiples of 16 bytes: 16-byte chunks of a row at places that depend on the
// row (conflict-free both ways), ROWS at a time, whole 128-byte lines of 4 rows an
// instruction.  Others: half of the columns at a time in a padded block, an
// output a lane.  (An aligned word a lane, shifted into place, took longer: 15.9 us against 13.2 for 1000 x
// 1001 x 1056 NVFP4.)
template <bool OUT32, int ROWS>
__device__ __forceinline__ void store_rows(const MatmulProblem& p, uint4* stage, const uint32_t* v, int64_t t, int64_t n,
                                           bool rows16) {
  constexpr int ES = OUT32 ? 4 : 2, COLS = 128 / ES;
  const int lane = threadIdx.x & 31;
  const int rows = (int)max((int64_t)0, min((int64_t)32, p.T - t)), cols = (int)max((int64_t)0, min((int64_t)COLS, p.N - n));
  unsigned char* y = reinterpret_cast<unsigned char*>(p.y) + (t * p.N + n) * ES;
  const int64_t pitch = p.N * ES;
  if (rows16) {  // the row's end is a multiple of 16 bytes too
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += ROWS) {
      __syncwarp();
      if (ROWS == 32 || lane / ROWS == r0 / ROWS) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          stage[(lane & (ROWS - 1)) * 8 + (c ^ (lane & 7))] = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
      }
      __syncwarp();
      const int c = lane & 7;
#pragma unroll
      for (int i = 0; i < ROWS / 4; ++i) {
        const int r = 4 * i + (lane >> 3);
        if (r0 + r < rows && c * 16 < cols * ES)
          *reinterpret_cast<uint4*>(y + (r0 + r) * pitch + c * 16) = stage[r * 8 + (c ^ (r & 7))];
      }
    }
    return;
  }
  uint32_t* b = reinterpret_cast<uint32_t*>(stage);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 16; ++c) b[lane * 17 + c] = v[16 * half + c];
    __syncwarp();
    if (OUT32) {
      const int c = lane & 15, col = 16 * half + c;
      if (col < cols)
        for (int r = lane >> 4; r < rows; r += 2) *reinterpret_cast<uint32_t*>(y + r * pitch + col * 4) = b[r * 17 + c];
    } else {
      const int col = 32 * half + lane;
      if (col < cols)
        for (int r = 0; r < rows; ++r)
          *reinterpret_cast<uint16_t*>(y + r * pitch + col * 2) = reinterpret_cast<const uint16_t*>(b + r * 17)[lane];
    }
  }
}

// A wait ran out: this warp's part of the tiles i, i + pairs, ... becomes NaN, so
// that nothing looks like a result.
template <bool OUT32>
static __device__ __noinline__ void pair_give_up(const MatmulProblem& p, const PairLaunch& l, unsigned i, unsigned pairs,
                                                 int rank, int warp) {
  for (; i < l.end; i += pairs) {
    int64_t m, n;
    pair_tile(l, i, m, n);
    const int64_t t = m * 256 + rank * 128 + 32 * (warp & 3) + (threadIdx.x & 31), n0 = n * 256 + 128 * (warp >> 2);
    if (t < p.T)
      for (int64_t c = n0; c < p.N && c < n0 + 128; ++c) y_store(p.y, p.y_dt, t * p.N + c, __uint_as_float(0x7FC00000u));
  }
}

// Waits until the last copies of both CTAs of a pair that gave up have landed: tile i of `even` or `odd` copied so far
// went to slot i % kPairStages, both halves of `half` bytes reported to the even CTA's barrier `full`, which may lack
// the even CTA's arrival or one half.  (Neither is more than kPairStages tiles ahead: those need the other's to be
// consumed first.)
static __device__ __noinline__ void pair_drain(uint64_t* full, unsigned even, unsigned odd, unsigned half) {
  const unsigned last = max(even, odd);
  for (unsigned i = last > kPairStages ? last - kPairStages : 0; i < last; ++i) {
    uint64_t* bar = &full[i % kPairStages];
    if (i >= even)
      mbar_arrive_expect_tx(bar, half);
    else if (i >= odd)
      mbar_complete_tx(bar, half);
    mbar_drain(bar, i / kPairStages & 1);
  }
}

template <int FMT, bool OUT32, bool WIDE>
__global__ void __launch_bounds__(kPairThreads, 1)
    k_matmul_pair(const __grid_constant__ MatmulProblem p, const __grid_constant__ PairLaunch l, const __grid_constant__ CUtensorMap wmap,
                  const __grid_constant__ CUtensorMap xmap) {
  using G = PairGeo<FMT>;
  using F = TcFormat<FMT>;
  extern __shared__ unsigned char mm_smem[];
  __shared__ uint64_t full_t[kPairStages], empty[kPairStages], full_s[G::kSlots], empty_s[G::kSlots], acc_full, acc_empty,
      done;
  __shared__ uint32_t tmem_base;
  __shared__ unsigned failed, copied[2];  // a wait of the cluster ran out; K tiles that the pair's CTAs copied (in the even one)
  unsigned char* ring = reinterpret_cast<unsigned char*>(((uintptr_t)mm_smem + 1023) & ~(uintptr_t)1023);
  unsigned char* scales = ring + kPairStages * G::kStage;
  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  const int in_cluster = (int)cluster_rank(), rank = in_cluster & 1, share = in_cluster >> 1;
  const uint32_t leader = (uint32_t)in_cluster & ~1u;
  const unsigned pair = blockIdx.x / (2 * l.split), pairs = gridDim.x / (2 * l.split);
  const int all_k = (int)((p.K + F::kTileK - 1) / F::kTileK);
  const int k0 = (int)((int64_t)all_k * share / l.split), k1 = (int)((int64_t)all_k * (share + 1) / l.split);
  const int64_t nb = p.K / F::kGroup;
  unsigned* const flags = p.flags;
  const unsigned limit_ns = l.wait.limit_ns;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPairStages; ++i) {
      mbar_init(&full_t[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < G::kSlots; ++i) {
      mbar_init(&full_s[i], 2 * 3);
      mbar_init(&empty_s[i], 1);
    }
    mbar_init(&acc_full, 1);
    mbar_init(&done, 1);
    mbar_init(&acc_empty, 2 * kPairEpilogue);
    mbar_fence_init();
    failed = 0;
  }
  if (warp == 9) tc_alloc<2, 512>(smem_u32(&tmem_base));
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  if (warp == 8 && elect_one()) {
    tma_prefetch_map(&xmap);
    tma_prefetch_map(&wmap);
  }
  griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0 && flags && l.first == 0) *reinterpret_cast<volatile unsigned*>(flags) = 0;
  MmSlot at;
  // tells every CTA of the cluster (in a self-test too, where nothing runs out in the role that stops)
  auto give_up = [&] {
    for (int r = 0; r < 2 * l.split; ++r) st_cluster_if(true, smem_u32(&failed), (uint32_t)r, 1u);
  };

  if (warp == 8) {
    if (elect_one()) {
      bool ok = true;
      unsigned issued = 0;
      const unsigned stop = stop_of(l.wait, in_cluster, 0);
      for (unsigned i = l.first + pair; i < l.end && ok; i += pairs) {
        int64_t m, n;
        pair_tile(l, i, m, n);
        for (int kt = k0; kt < k1; ++kt, ++issued) {
          if (!(ok = issued < stop && mm_wait<true>(&empty[at.slot], at.phase ^ 1, limit_ns, flags))) break;
          unsigned char* st = ring + at.slot * G::kStage;
          if (rank == 0) mbar_arrive_expect_tx(&full_t[at.slot], 2 * (G::kA + G::kB));
          tma_load_2d_pair(st, &xmap, kt * 128, (int)(m * 256 + rank * 128), &full_t[at.slot]);
          tma_load_2d_pair(st + G::kA, &wmap, kt * 128, (int)(n * 256 + rank * 128), &full_t[at.slot]);
          at.next(kPairStages);
        }
      }
      st_cluster_if(true, smem_u32(&copied[rank]), leader, issued);
      if (!ok) give_up();
      for (unsigned i = issued > kPairStages ? issued - kPairStages : 0; ok && i < issued; ++i)  // the last slots' releases
        ok = mm_wait<true>(&empty[i % kPairStages], i / kPairStages & 1, limit_ns, flags);
    }
  } else if (warp == 9) {
    if (rank == 0 && elect_one()) {
      unsigned turn = 0, set = 0;
      ScaleSlot<G::kSlots> piece;
      bool ok = true;
      for (unsigned i = l.first + pair; i < l.end && ok; i += pairs, turn ^= 1) {
        if (!(ok = mm_wait<true>(&acc_empty, turn ^ 1, limit_ns, flags))) break;
        tc_fence_after();
        for (int kt = k0; kt < k1; ++kt, set ^= 1) {
          const int u = kt % F::kPiece;
          if ((u == 0 || kt == k0) && !(ok = mm_wait<true>(&full_s[piece.slot], piece.phase, limit_ns, flags))) break;
          if (!(ok = mm_wait<true>(&full_t[at.slot], at.phase, limit_ns, flags))) break;
          tc_fence_after();
          const uint32_t st = smem_u32(ring + at.slot * G::kStage);
          const uint32_t sa = smem_u32(scales + piece.slot * G::kScales) + 512 * u * F::kAtoms;
          const uint32_t sb = sa + 4096 + 512 * u * F::kAtoms;  // features' words: two blocks a scale word
          const uint32_t ca = tmem + 256 + set * G::kScaleCols, cb = ca + 16;
#pragma unroll
          for (int j = 0; j < F::kAtoms; ++j) {
            tc_copy_scales<2>(ca + 4 * j, tc_desc_scales(sa + 512 * j));
            tc_copy_scales<2>(cb + 8 * j, tc_desc_scales(sb + 1024 * j));
            tc_copy_scales<2>(cb + 8 * j + 4, tc_desc_scales(sb + 1024 * j + 512));
          }
          const uint64_t da = tc_desc_sw128(st), db = tc_desc_sw128(st + G::kA);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma<FMT, 2>(tmem, da + 2 * k, db + 2 * k, tc_idesc<FMT>(256, 256, F::byte(k)), ca + 4 * F::atom(k),
                           cb + 8 * F::atom(k), kt > k0 || k > 0);
          tc_commit<2>(&empty[at.slot], leader);
          if (u == F::kPiece - 1 || kt == k1 - 1) {
            tc_commit<2>(&empty_s[piece.slot], leader);
            piece.next();
          }
          at.next(kPairStages);
        }
        if (ok) tc_commit<2>(&acc_full, leader);
      }
      if (!ok) give_up();
      tc_commit<2>(&done, leader);
    }
  } else if (warp >= 10) {
    const int block = (warp - 10) >> 1;  // 0: the tokens, 1 and 2: the features' halves
    const bool of_x = block == 0;
    ScaleTurn t{warp & 1};
    bool ok = true;
    for (unsigned i = l.first + pair; i < l.end && ok; i += pairs) {
      int64_t m, n;
      pair_tile(l, i, m, n);
      ok = scale_warp<true, G::kSlots, WIDE>(of_x ? l.unit_x : l.unit_w, t, F::kPiece, of_x ? p.xs : p.ws,
                            of_x ? m * 256 + rank * 128 : n * 256 + (block - 1) * 128, of_x ? p.T : p.N, nb, k0, k1 - k0,
                            scales + (of_x ? 0 : 4096 + (block - 1) * 512), G::kScales, of_x ? 512 : 1024, full_s, empty_s,
                            limit_ns, flags, stop_of(l.wait, in_cluster, of_x ? 2 : 1), leader);
    }
    if (!ok && lane == 0) give_up();
  } else {
    float f1, f2_;
    tensor_factors(p, f1, f2_);
    const int q = warp & 3, half = warp >> 2;
    uint4* stage = reinterpret_cast<uint4*>(scales + G::kSlots * G::kScales) + warp * (G::kTurnWarp / 16);
    unsigned turn = 0;
    for (unsigned i = l.first + pair; i < l.end; i += pairs, turn ^= 1) {
      int64_t m, n;
      pair_tile(l, i, m, n);
      if (!__all_sync(0xffffffffu, mm_wait<true>(&acc_full, turn, limit_ns, flags))) {
        if (lane == 0) give_up();
        if (l.split == 1) pair_give_up<OUT32>(p, l, i, pairs, rank, warp);
        break;
      }
      tc_fence_after();
      const uint32_t src = tmem + ((uint32_t)(32 * q) << 16) + 128 * half;
      const int64_t t0 = m * 256 + rank * 128 + 32 * q, nn = n * 256 + 128 * half;
      if (l.split > 1) {  // the partial tile to the idle ring, joined below
        float* part = reinterpret_cast<float*>(ring) + (32 * q + lane) * kPartPitch + 128 * half;
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          uint32_t v[32];
          tc_load32(src + c, v);
          tc_load_wait32(v);
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(part + c + e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
      } else if (!OUT32) {
        uint32_t o[64];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t v[64];
          tc_load32(src + 64 * c, v);
          tc_load32(src + 64 * c + 32, v + 32);
          tc_load_wait32(v);
          tc_load_wait32(v + 32);
          if (c == 1) {  // everything is in registers: the next tile's multiply-adds may begin
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(&acc_empty, leader);
          }
          if (FMT == FMT_NVFP4 && f2_ != 1.f) {
#pragma unroll
            for (int e = 0; e < 64; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f2_);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float a = __uint_as_float(v[2 * e]), b = __uint_as_float(v[2 * e + 1]);
            if (FMT == FMT_NVFP4) a *= f1, b *= f1;
            o[32 * c + e] = pack16(a, b, p.y_dt);
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) store_rows<false, G::kRows>(p, stage, o + 32 * c, t0, nn + 64 * c, l.rows16);
      } else {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tc_load32(src + 32 * c, v);
          tc_load_wait32(v);
          if (c == 3) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(&acc_empty, leader);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f1 * f2_);
          store_rows<true, G::kRows>(p, stage, v, t0, nn + 32 * c, l.rows16);
        }
      }
    }
  }
  __syncwarp();
  if (l.split > 1) {
    // each CTA joins and stores its share of the 128 rows, as many as there are, that the pairs' CTAs of its rank hold, in pair order
    cluster_sync();
    const bool nothing = ld_volatile(&failed) != 0;  // a wait ran out: no number that looks like a result
    float f1, f2_;
    tensor_factors(p, f1, f2_);
    int64_t m, n;
    pair_tile(l, l.first + pair, m, n);
    const int tv = (int)max((int64_t)0, min((int64_t)128, p.T - m * 256 - rank * 128)), rows = (tv + l.split - 1) / l.split;
    const uint32_t part = smem_u32(ring);
    for (int e = threadIdx.x; e < min(rows, tv - share * rows) * 64; e += kPairThreads) {
      const int row = share * rows + (e >> 6), col = 4 * (e & 63);
      const int64_t t = m * 256 + rank * 128 + row, nn = n * 256 + col;
      if (nn >= p.N) continue;
      float4 v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < l.split) v[r] = ld_cluster_f4(part + 4 * (row * kPartPitch + col), 2 * r + rank);
      float4 sum = v[0];
#pragma unroll
      for (int r = 1; r < 4; ++r)
        if (r < l.split) sum.x += v[r].x, sum.y += v[r].y, sum.z += v[r].z, sum.w += v[r].w;
      if (nothing) sum = make_float4(CUDART_NAN_F, CUDART_NAN_F, CUDART_NAN_F, CUDART_NAN_F);
      const float o[4] = {sum.x * f1 * f2_, sum.y * f1 * f2_, sum.z * f1 * f2_, sum.w * f1 * f2_};
      y_store4(p.y, p.y_dt, t * p.N + nn, o, p.N - nn, l.vec4);
    }
  }
  // all multiply-adds that were issued are done, whether their readers waited for them or not
  if (warp == 0 && elect_one()) mm_drain(&done, 0);
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the other may still signal it or read its shared memory
  if (ld_volatile(&failed) != 0) {  // the same in all CTAs
    if (rank == 0 && warp == 8 && elect_one()) pair_drain(full_t, copied[0], copied[1], G::kA + G::kB);
    __syncwarp();
    cluster_sync();
  }
  if (warp == 9) {
    tc_fence_after();
    tc_dealloc<2, 512>(tmem);
  }
}

// What a call brings along on the host.
struct MmCall {
  int sms;
  cudaStream_t st;
  MmWait wait;
  dq_matmul_info* info;  // if given, what would run goes here and nothing does
};

// 2-D tensor map of a code matrix in bytes: boxes of 128 bytes x `box_rows`
// rows in the 128-byte swizzle, zeros outside.
static bool encode_codes(CUtensorMap* map, const unsigned char* q, int64_t row_bytes, int64_t rows, int box_rows) {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      return (PFN_cuTensorMapEncodeTiled_v12000) nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  const cuuint32_t elem_strides[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<unsigned char*>(q), dims, strides, box, elem_strides,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static int scale_unit(const unsigned char* s, int64_t nb) {
  const uintptr_t v = (uintptr_t)s | (uintptr_t)nb | 32u;
  return (int)(v & (~v + 1));
}

// Fours of neighbouring outputs start at multiples of their size.
static bool vec4_rows(const MatmulProblem& p) {
  return p.N % 4 == 0 && (uintptr_t)p.y % (p.y_dt == DT_F32 ? 16 : 8) == 0;
}

template <int FMT>
static cudaError_t matmul_any(const MatmulProblem& p, const MmCall& c) {
  const int64_t tiles = (p.T + 63) / 64 * ((p.N + 63) / 64);
  if (c.info) {
    *c.info = {DQ_MATMUL_ANY, 64, 0, tiles, 0, 1};
    return cudaSuccess;
  }
  return launch_early(k_matmul_any<FMT>, (unsigned)tiles, 256, 0, 1, c.st, p);
}

template <int FMT, int BN>
static cudaError_t matmul_tc(const MatmulProblem& p, const MmCall& c) {
  using G = MmGeo<FMT, BN>;
  CUtensorMap wmap, xmap;
  const int64_t row_bytes = FMT == FMT_MXFP8 ? p.K : p.K / 2;
  if (!encode_codes(&wmap, p.wq, row_bytes, p.N, 128) || !encode_codes(&xmap, p.xq, row_bytes, p.T, BN))
    return cudaErrorInvalidValue;
  const int64_t tiles = (p.N + 127) / 128 * ((p.T + BN - 1) / BN);
  const int64_t nk = (p.K + TcFormat<FMT>::kTileK - 1) / TcFormat<FMT>::kTileK;
  MmLaunch l;
  l.wait = c.wait;
  l.unit_x = scale_unit(p.xs, p.K / TcFormat<FMT>::kGroup);
  l.unit_w = scale_unit(p.ws, p.K / TcFormat<FMT>::kGroup);
  l.vec4 = vec4_rows(p);
  auto kern = l.unit_x >= 16 && l.unit_w >= 16 ? k_matmul_tc<FMT, BN, true> : k_matmul_tc<FMT, BN, false>;
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  // the same limit in every call: another thread's call may come between this and the launch
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMmSmem);
  if (e != cudaSuccess) return e;
  int smem = 0;
  // The largest split whose clusters all run at once (some SMs of a GPC are left
  // over by clusters that do not divide it: 132 of 148 SMs hold clusters of 4 or 6,
  // 120 of 8, 105 of 7; 40 x 2048 x 5632 MXFP4, 16 tiles: 15.2 us split in 7, 8.4 in 6).
  for (l.split = (int)min((int64_t)8, min(nk, max((int64_t)1, c.sms / tiles)));; --l.split) {
    const int64_t per = (nk + l.split - 1) / l.split;
    const int fixed = kScaleSlots * G::kScales + 1024 + (l.split > 1 ? (BN + l.split - 1) / l.split * l.split * 512 : 0);
    // one CTA an SM takes all shared memory, more tiles share an SM by three
    const int room = ((tiles * l.split <= c.sms ? kMmSmem : 74 * 1024) - fixed) / G::kStage;
    l.stages = (int)min((int64_t)kMmMaxStages, min(per, (int64_t)room));
    smem = l.stages * G::kStage + fixed;
    // A CTA takes at least its tensor memory's share of the SM's shared memory
    // (228 KB, 1 KB of it per CTA reserved).  Then tensor memory never runs out on
    // an SM before shared memory does, and no CTA of a cluster can wait for tensor
    // memory that is held by CTAs which wait for their own cluster.
    smem = max(smem, 228 * 1024 / 512 * G::kAlloc - 1024 - (int)fa.sharedSizeBytes);
    if (l.split <= 2) break;  // clusters of 2 fit everywhere
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute at;
    cluster_config(&cfg, &at, (unsigned)(tiles * l.split), kMmThreads, (size_t)smem, l.split);
    int clusters = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg)) != cudaSuccess) return e;
    if (clusters >= tiles) break;
  }
  if (c.info) {
    *c.info = {DQ_MATMUL_TILE, BN, l.unit_x >= 16 && l.unit_w >= 16, l.split > 1 ? 0 : tiles, l.split > 1 ? tiles : 0, l.split};
    return cudaSuccess;
  }
  // where an SM takes several CTAs, those of the next grid would take the places of this one unevenly
  l.early = tiles * l.split <= c.sms;
  return launch_early(kern, (unsigned)(tiles * l.split), kMmThreads, (size_t)smem, l.split, c.st, p, l, wmap, xmap);
}

// Whole waves of pairs first; the tiles left over, or all of them where they do
// not fill a wave, split their columns over the pairs of a cluster, if clusters
// that large have room for them at once and the wave saved is long enough.
// (1500 x 4096 x 14336 MXFP8, 96 tiles on 74 pairs: 82 us as two waves, 72 so;
// 2048 x 14336 x 4096 NVFP4, 448 tiles: 62 us as seven waves, 66 so.)
template <int FMT, bool OUT32>
static cudaError_t matmul_pair(const MatmulProblem& p, const MmCall& c) {
  using G = PairGeo<FMT>;
  CUtensorMap wmap, xmap;
  const int64_t row_bytes = FMT == FMT_MXFP8 ? p.K : p.K / 2;
  if (!encode_codes(&wmap, p.wq, row_bytes, p.N, 128) || !encode_codes(&xmap, p.xq, row_bytes, p.T, 128))
    return cudaErrorInvalidValue;
  PairLaunch l;
  l.wait = c.wait;
  l.tiles_m = (unsigned)((p.T + 255) / 256);
  l.tiles_n = (unsigned)((p.N + 255) / 256);
  l.unit_x = scale_unit(p.xs, p.K / TcFormat<FMT>::kGroup);
  l.unit_w = scale_unit(p.ws, p.K / TcFormat<FMT>::kGroup);
  l.rows16 = ((uintptr_t)p.y | (uintptr_t)(p.N * (OUT32 ? 4 : 2))) % 16 == 0;
  l.vec4 = vec4_rows(p);
  auto kern = l.unit_x >= 16 && l.unit_w >= 16 ? k_matmul_pair<FMT, OUT32, true> : k_matmul_pair<FMT, OUT32, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem);
  if (e != cudaSuccess) return e;
  const unsigned tiles = l.tiles_m * l.tiles_n, pairs = (unsigned)c.sms / 2;
  const int64_t nk = (p.K + TcFormat<FMT>::kTileK - 1) / TcFormat<FMT>::kTileK;
  const unsigned rest = tiles % pairs;
  int split = 1;
  for (int s = 4; s > 1 && split == 1 && rest > 0; --s) {
    // K tiles saved, about 0.3 us each, against the joining of the partial tiles (4 us) and a launch of its own (4 us)
    if (rest * s > pairs || nk * (s - 1) < (tiles > rest ? 28 : 12) * s) continue;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute at;
    cluster_config(&cfg, &at, rest * 2 * s, kPairThreads, (size_t)G::kSmem, 2 * s);
    int room = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&room, kern, &cfg)) != cudaSuccess) return e;
    if ((unsigned)room >= rest) split = s;
  }
  const unsigned whole = split > 1 ? tiles - rest : tiles;
  if (c.info) {
    *c.info = {DQ_MATMUL_PAIR, 256, l.unit_x >= 16 && l.unit_w >= 16, whole, tiles - whole, split};
    return cudaSuccess;
  }
  if (whole > 0) {
    l.first = 0;
    l.end = whole;
    l.split = 1;
    e = launch_early(kern, 2 * (whole < pairs ? whole : pairs), kPairThreads, (size_t)G::kSmem, 2, c.st, p, l, wmap, xmap);
    if (e != cudaSuccess || whole == tiles) return e;
  }
  l.first = whole;
  l.end = tiles;
  l.split = split;
  return launch_early(kern, rest * 2 * split, kPairThreads, (size_t)G::kSmem, 2 * split, c.st, p, l, wmap, xmap);
}

// About how long a product takes, in ns, to choose between the kernels: a fixed
// part, with the join of split tiles, and the K tiles that a CTA works on, each the
// time that its SM's operands take to arrive, whichever the kernel (measured: 70
// bytes a ns with a scale per 16, 90 with one per 32).  Chosen by this, the kernel
// was within 10 % of the fastest of the three in 260 of 264 products of 65 to 1500
// tokens, 17 % off at worst and 0.7 % on average; the pairs for all of them took 1.22
// times as long on average, 1.83 times at most (192 x 4096 x 1024 NVFP4: 64 tokens a tile
// 5.3 us, 128 8.2, pairs 6.9; 128 x 4096 x 14336: 15.9, 12.9 and 16.9; 300 x 4096 x
// 14336: 34.4, 25.3 and 20.5).
constexpr int tile_ns(int fmt, int bn) { return (128 + bn) * 128 / (fmt == FMT_NVFP4 ? 70 : 90); }
static int64_t tc_ns(const MatmulProblem& p, int fmt, int64_t nk, int bn, int sms) {
  const int64_t tiles = (p.N + 127) / 128 * ((p.T + bn - 1) / bn);
  const int64_t split = max((int64_t)1, min((int64_t)8, min(nk, sms / tiles)));
  return 3600 + (split > 1 ? 20 * bn : 0) + (tiles + sms - 1) / sms * ((nk + split - 1) / split) * tile_ns(fmt, bn);
}
static int64_t pair_ns(const MatmulProblem& p, int fmt, int64_t nk, int sms) {
  const int64_t tiles = (p.N + 255) / 256 * ((p.T + 255) / 256), pairs = sms / 2;
  int64_t split = 4;
  while (split > 1 && (tiles * split > pairs || nk * (split - 1) < 12 * split)) --split;
  return (split > 1 ? 9000 : 6000) + (tiles + pairs - 1) / pairs * ((nk + split - 1) / split) * tile_ns(fmt, 128);
}

template <int FMT>
static cudaError_t matmul_fmt(const MatmulProblem& p, const MmCall& c) {
  const int64_t row_bytes = FMT == FMT_MXFP8 ? p.K : p.K / 2;
  if (((uintptr_t)p.xq | (uintptr_t)p.wq | (uintptr_t)row_bytes) % 16 != 0) return matmul_any<FMT>(p, c);
  if (p.T <= 16) return matmul_tc<FMT, 16>(p, c);
  if (p.T <= 32) return matmul_tc<FMT, 32>(p, c);
  const int64_t nk = (p.K + TcFormat<FMT>::kTileK - 1) / TcFormat<FMT>::kTileK;
  const int64_t t64 = tc_ns(p, FMT, nk, 64, c.sms), t128 = tc_ns(p, FMT, nk, 128, c.sms), two = pair_ns(p, FMT, nk, c.sms);
  if (p.T <= 64 || (t64 <= t128 && t64 <= two)) return matmul_tc<FMT, 64>(p, c);
  // 128 tokens a tile leave no shared memory for a second CTA of an SM
  if ((p.N + 127) / 128 * ((p.T + 127) / 128) <= c.sms && t128 <= two) return matmul_tc<FMT, 128>(p, c);
  return p.y_dt == DT_F32 ? matmul_pair<FMT, true>(p, c) : matmul_pair<FMT, false>(p, c);
}

static int matmul_call(const dq_outputs* X, int64_t tokens, const dq_outputs* W, int64_t rows, int64_t cols, int format, int group,
                       void* Y, int y_dtype, void* workspace, size_t workspace_bytes, const MmWait& wait, dq_matmul_info* info,
                       void* stream) {
  if (tokens <= 0 || rows <= 0 || cols <= 0 || group <= 0 || cols % group != 0) return DQ_EINVAL;
  if (format < DQ_INT4 || format > DQ_MXFP8) return DQ_EINVAL;
  if (format != DQ_NVFP4 && format != DQ_MXFP4 && format != DQ_MXFP8) return DQ_EUNSUPPORTED;
  if (group != (format == DQ_NVFP4 ? 16 : 32)) return DQ_EUNSUPPORTED;
  if (y_dtype < DQ_F32 || y_dtype > DQ_F16) return DQ_EINVAL;
  // a tile's sum must end well within the waits' limit of 1 s: 2^27 columns take 0.4 s
  if (tokens > INT_MAX - 256 || rows > INT_MAX - 256 || cols > ((int64_t)1 << 27)) return DQ_EUNSUPPORTED;
  if ((tokens + 63) / 64 * ((rows + 63) / 64) > INT_MAX) return DQ_EUNSUPPORTED;
  if (!X || !W || !X->codes || !X->block_scales || !W->codes || !W->block_scales || !Y) return DQ_EINVAL;
  if (format == DQ_NVFP4 && (!X->tensor_scale || !W->tensor_scale || (uintptr_t)X->tensor_scale % 4 != 0 ||
                             (uintptr_t)W->tensor_scale % 4 != 0))
    return DQ_EINVAL;
  if ((uintptr_t)Y % (y_dtype == DQ_F32 ? 4 : 2) != 0) return DQ_EINVAL;
  if ((uintptr_t)workspace % 256 != 0) return DQ_EINVAL;
  if (workspace && workspace_bytes < DQ_MATMUL_WORKSPACE_BYTES) return DQ_EWORKSPACE;
  MatmulProblem p{};
  p.xq = static_cast<const unsigned char*>(X->codes);
  p.xs = static_cast<const unsigned char*>(X->block_scales);
  p.wq = static_cast<const unsigned char*>(W->codes);
  p.ws = static_cast<const unsigned char*>(W->block_scales);
  if (format == DQ_NVFP4) {
    p.x_sT = X->tensor_scale;
    p.w_sT = W->tensor_scale;
  }
  p.y = Y;
  p.y_dt = y_dtype;
  p.T = tokens;
  p.N = rows;
  p.K = cols;
  p.flags = workspace ? &static_cast<WsHeader*>(workspace)->flags : nullptr;
  MmCall c{0, static_cast<cudaStream_t>(stream), wait, info};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DQ_ECUDA;
  if (cudaDeviceGetAttribute(&c.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return DQ_ECUDA;
  const cudaError_t e = format == DQ_NVFP4   ? matmul_fmt<FMT_NVFP4>(p, c)
                        : format == DQ_MXFP4 ? matmul_fmt<FMT_MXFP4>(p, c)
                                             : matmul_fmt<FMT_MXFP8>(p, c);
  return e == cudaSuccess ? DQ_OK : DQ_ECUDA;
}

}  // namespace dq

extern "C" int dq_matmul(const dq_outputs* X, int64_t tokens, const dq_outputs* W, int64_t rows, int64_t cols, int format,
                         int group, void* Y, int y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return dq::matmul_call(X, tokens, W, rows, cols, format, group, Y, y_dtype, workspace, workspace_bytes, dq::MmWait(),
                         nullptr, stream);
}

extern "C" int dq_matmul_selftest(const dq_outputs* X, int64_t tokens, const dq_outputs* W, int64_t rows, int64_t cols,
                                  int format, int group, void* Y, int y_dtype, void* workspace, size_t workspace_bytes,
                                  unsigned wait_ns, int rank, int role, unsigned at, void* stream) {
  if (wait_ns < 1000000u || wait_ns > dq::kWaitLimitNs || rank < 0 || rank > 7 || role < 0 || role > 2 ||
      at >> dq::kStopAtBits != 0 || !workspace)
    return DQ_EINVAL;
  dq::MmWait wait;
  wait.limit_ns = wait_ns;
  wait.stop = dq::stop_key(rank, role) << dq::kStopAtBits | at;
  return dq::matmul_call(X, tokens, W, rows, cols, format, group, Y, y_dtype, workspace, workspace_bytes,
                         wait, nullptr, stream);
}

extern "C" int dq_matmul_kernel(const dq_outputs* X, int64_t tokens, const dq_outputs* W, int64_t rows, int64_t cols,
                                int format, int group, const void* Y, int y_dtype, dq_matmul_info* info) {
  if (!info) return DQ_EINVAL;
  return dq::matmul_call(X, tokens, W, rows, cols, format, group, const_cast<void*>(Y), y_dtype, nullptr, 0, dq::MmWait(), info,
                         nullptr);
}

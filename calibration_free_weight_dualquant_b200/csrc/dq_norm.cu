// dq_norm.cu -- the row quantizers around a quantized product: residual
// addition + root-mean-square norm + column scales + quantization
// (dq_norm_quant), and silu(gate) * up + column scales + quantization
// (dq_glu_quant), each in one pass over its inputs (NVFP4: a pass for the
// tensor scale first, in the same launch).
//
// Mathematics: with W ~ D_a Q D_b a product X W^T is (X D_b) Q^T D_a
// (DualQuant arXiv 2610.13767 summary, section 4.4), so whatever produces X
// multiplies its channels by b before the format's own row-wise quantization:
//   norm   h = round(x + r), x' = h / sqrt(mean(h^2) + eps) * g * b
//   glu    x' = gate / (1 + exp(-gate)) * up * b
//   a = Proj_Fa(max|x'| over the group / qmax), 1 for an all-zero group
//   q = Q(x' / a), ties to even, clipped
// x' is not rounded on the way: the decisions are those of the real numbers.
// fp32 values known to a relative 2^-20 settle nearly all of them: a code is
// certain where both ends of a bracket that wide convert to it, a block scale
// where the fp32 ratio is not next to a projection midpoint.  The rest is
// decided in fp64 from the stored inputs.
//
// A lane holds 16 consecutive elements: a whole NVFP4 group, or half a group of
// the MX formats.  (With 8 a lane, twice as many lanes repeated the scale's
// arithmetic, the votes and the address arithmetic: 34 and 58 instructions an
// element, measured, and the issue slots were the bound.)
#include <climits>
#include <math_constants.h>

#include "dq.h"
#include "dq_device.cuh"
#include "dq_fast.cuh"
#include "dq_internal.h"
#include "dq_launch.h"

namespace dq {

constexpr int kGluThreads = 256;   // dq_glu_quant's block; two an SM
constexpr int kGluMax = 512;       // ... its largest, in a call that one cluster takes
constexpr int kNormSmem = 4 * 512 * 64;  // g b of 4 chunks of 512 threads
constexpr float kFltMax = 3.402823466e38f;

struct RowProblem {
  const void* x;          // norm: hidden state; glu: gate
  const void* y;          // norm: residual or NULL; glu: up
  const void* g;          // norm weight or NULL
  const void* b_store;    // column inverse scales or NULL
  int col_dt;
  int b_vec;              // b_store is 16-byte aligned
  int wide;               // rows of x, y and h start at multiples of 32 bytes
  int codes_vec;          // codes is 16-byte aligned
  int64_t M, K, ld;       // rows, columns, row stride of x and y in elements
  float eps;
  void* h;                // residual sum out (aliases x or y at will) or NULL
  unsigned char* codes;
  unsigned char* scales;  // [M][nb] bytes
  float* sT_out;
  double* rstd;           // NVFP4 norm: 1/rms of every row between the passes
  WsHeader* hdr;
  int cluster;            // the grid is one cluster
};

__device__ __forceinline__ float2 h2_values(uint32_t u, int xdt) {
  return xdt == DT_BF16 ? make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u))
                        : __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// Sum of two packed pairs, rounded once (to nearest even).
template <int XDT>
__device__ __forceinline__ uint32_t h2_add(uint32_t a, uint32_t b) {
  uint32_t r;
  if (XDT == DT_BF16)
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 16 consecutive 16-bit elements of a lane.
struct V16 {
  uint32_t u[8];
};
__device__ __forceinline__ V16 zero16() {
  V16 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v.u[i] = 0;
  return v;
}
// An offset that no load can use before this point, which comes after the kernel's wait for
// the grid before.
__device__ __forceinline__ int64_t after_wait(int64_t off) {
  asm volatile("" : "+l"(off)::"memory");
  return off;
}

// An input of the call, read once: free to move above stores (a store of h to
// the input's own place depends on the value loaded from it), but not above the
// wait for the grid before: `off` comes out of after_wait.
__device__ __forceinline__ V16 load16(const void* base, int64_t off, bool wide) {
  const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + off;
  V16 v;
  if (wide) {
    asm("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(v.u[0]), "=r"(v.u[1]), "=r"(v.u[2]), "=r"(v.u[3]), "=r"(v.u[4]), "=r"(v.u[5]), "=r"(v.u[6]), "=r"(v.u[7])
        : "l"(p));
  } else {
    asm("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.u[0]), "=r"(v.u[1]), "=r"(v.u[2]), "=r"(v.u[3]) : "l"(p));
    asm("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.u[4]), "=r"(v.u[5]), "=r"(v.u[6]), "=r"(v.u[7])
        : "l"(p + 8));
  }
  return v;
}
// What this thread stored earlier, or an input read again after stores.
__device__ __forceinline__ V16 load16_again(const void* base, int64_t off) {
  const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + off;
  V16 v;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.u[4 * i]), "=r"(v.u[4 * i + 1]), "=r"(v.u[4 * i + 2]), "=r"(v.u[4 * i + 3])
                 : "l"(p + 8 * i)
                 : "memory");
  return v;
}
__device__ __forceinline__ void store16(void* base, int64_t off, bool wide, const V16& v) {
  uint16_t* p = reinterpret_cast<uint16_t*>(base) + off;
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.u[0]), "r"(v.u[1]), "r"(v.u[2]),
                 "r"(v.u[3]), "r"(v.u[4]), "r"(v.u[5]), "r"(v.u[6]), "r"(v.u[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(v.u[0], v.u[1], v.u[2], v.u[3]);
    *reinterpret_cast<uint4*>(p + 8) = make_uint4(v.u[4], v.u[5], v.u[6], v.u[7]);
  }
}
// All 16 are zeros (of either sign).
__device__ __forceinline__ bool zero_bits16(const V16& v) {
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) any |= v.u[i];
  return (any & 0x7FFF7FFFu) == 0;
}
// The elements as fp32 pairs.
template <int XDT>
__device__ __forceinline__ void pairs16(const V16& v, f2* x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = h2_values(v.u[i], XDT);
    x[i] = pk(f.x, f.y);
  }
}

// The 16 column scales at col (1 where there are none).
__device__ __forceinline__ void b16_values(const RowProblem& p, int64_t col, f2* b) {
  if (p.b_vec) {
    const V16 s = load16(p.b_store, after_wait(col), false);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = h2_values(s.u[i], p.col_dt);
      b[i] = pk(f.x, f.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      b[i] = p.b_store ? pk(b_decode(p.b_store, p.col_dt, col + 2 * i), b_decode(p.b_store, p.col_dt, col + 2 * i + 1))
                       : splat(1.f);
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Three-input maximum that propagates NaN.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Lanes of a group at 16 elements a lane.
__host__ __device__ constexpr int group_lanes(int fmt) { return fmt == FMT_NVFP4 ? 1 : 2; }
// 32-bit words of a lane's codes.
__host__ __device__ constexpr int code_words(int fmt) { return fmt == FMT_MXFP8 ? 4 : 2; }

// Magnitude code of |x'| = ax for the scale a (a = s_T e for NVFP4), decided in
// fp64: E2M1 midpoints times a are exact (3 + 28 significant bits), a division
// by a power of two is exact.
template <int FMT>
__device__ __forceinline__ uint32_t mag_code(double ax, double a) {
  if (FMT == FMT_MXFP8) {
    const double m = ax / a;
    if (m >= 448.0) return 0x7Eu;
    const int e = m < 0x1p-6 ? -6 : ilogb(m);
    return e4m3_bits(fmin(scalbn(rint(scalbn(m, 3 - e)), e - 3), 448.0));
  }
  return (ax > 0.25 * a) + (ax >= 0.75 * a) + (ax > 1.25 * a) + (ax >= 1.75 * a) + (ax > 2.5 * a) + (ax >= 3.5 * a) +
         (ax > 5.0 * a);
}

// Conversions of v[0 .. 15] times s: E4M3 bytes or E2M1 nibbles (hardware round
// to nearest even, saturating).
template <int FMT>
__device__ __forceinline__ void codes_fast(const f2* v, float s, uint32_t* cw) {
  const f2 ss = splat(s);
#pragma unroll
  for (int w = 0; w < code_words(FMT); ++w) {
    if (FMT == FMT_MXFP8) {
      const f2 a = mul2(v[2 * w], ss), b = mul2(v[2 * w + 1], ss);
      asm("{\n.reg .b16 l, h;\ncvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\ncvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n"
          "mov.b32 %0, {l, h};\n}"
          : "=r"(cw[w])
          : "f"(lo_of(a)), "f"(hi_of(a)), "f"(lo_of(b)), "f"(hi_of(b)));
    } else {
      f2 t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = mul2(v[4 * w + i], ss);
      asm("{\n.reg .b8 c0, c1, c2, c3;\n"
          "cvt.rn.satfinite.e2m1x2.f32 c0, %2, %1;\n"
          "cvt.rn.satfinite.e2m1x2.f32 c1, %4, %3;\n"
          "cvt.rn.satfinite.e2m1x2.f32 c2, %6, %5;\n"
          "cvt.rn.satfinite.e2m1x2.f32 c3, %8, %7;\n"
          "mov.b32 %0, {c0, c1, c2, c3};\n}"
          : "=r"(cw[w])
          : "f"(lo_of(t[0])), "f"(hi_of(t[0])), "f"(lo_of(t[1])), "f"(hi_of(t[1])), "f"(lo_of(t[2])), "f"(hi_of(t[2])),
            "f"(lo_of(t[3])), "f"(hi_of(t[3])));
    }
  }
}

// A zero magnitude has no sign.
template <int FMT>
__device__ __forceinline__ uint32_t no_negzero(uint32_t w) {
  if (FMT == FMT_MXFP8) return w & (((w & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | 0x7F7F7F7Fu);
  return w & (0x77777777u | (w << 1) | (w << 2) | (w << 3));
}

// fp64 value of x' at (row, col), from the stored inputs.
template <int XDT, bool GLU>
__device__ __forceinline__ double exact1(const RowProblem& p, int64_t row, int64_t col, double rstd) {
  const double h = (double)b_decode(GLU ? p.x : (p.y ? p.h : p.x), XDT, row * p.ld + col);
  const double b = p.b_store ? (double)b_decode(p.b_store, p.col_dt, col) : 1.0;
  if (GLU) return h / (1.0 + exp(-h)) * ((double)b_decode(p.y, XDT, row * p.ld + col) * b);
  return h * ((p.g ? (double)b_decode(p.g, XDT, col) : 1.0) * b) * rstd;
}

// The scale of the block that holds element `at` (row * K + column) to memory.
template <int FMT>
__device__ __forceinline__ void store_scale(const RowProblem& p, int64_t at, float a, bool bad) {
  unsigned char* s = p.scales + (at >> (FMT == FMT_NVFP4 ? 4 : 5));  // a row is a whole number of groups
  if (bad)
    *s = fmt_pow2(FMT) ? 0xFFu : 0x7Fu;
  else
    a_store_f<FMT>(s, 0, a);
}

// The group from element `first` decided in fp64 and stored, an element a lane:
// the cold path, out of line.  Every lane of the warp calls it with the same arguments.  A group
// with a value that is not finite in fp32 gets the format's NaN scale and zero
// codes; returns whether it did.
template <int FMT, int XDT, bool GLU>
static __device__ __noinline__ bool quant_exact(const RowProblem& p, int64_t first, double rstd, float sT) {
  constexpr int G = FMT == FMT_NVFP4 ? 16 : 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = first / p.K, col = first - row * p.K;
  const double x = lane < G ? exact1<XDT, GLU>(p, row, col + lane, rstd) : 0.0;
  double m = fabs(x) <= (double)kFltMax ? fabs(x) : CUDART_INF;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
  const bool bad = m > (double)kFltMax;
  const float a = m == 0.0 || bad ? 1.f : (float)a_project<FMT>(m / grid_qmax(FMT), (double)sT);
  uint32_t c = bad ? 0u : mag_code<FMT>(fabs(x), FMT == FMT_NVFP4 ? (double)sT * (double)a : (double)a);
  if (c != 0 && x < 0.0) c |= FMT == FMT_MXFP8 ? 0x80u : 8u;
  const int64_t at = first + lane;
  if (FMT == FMT_MXFP8) {
    p.codes[at] = (unsigned char)c;
  } else {
    const uint32_t high = __shfl_down_sync(0xffffffffu, c, 1);
    if (lane < G && (lane & 1) == 0) p.codes[at >> 1] = (unsigned char)(c | (high << 4));
  }
  if (lane == 0) store_scale<FMT>(p, first, a, bad);
  return bad;
}

__device__ __forceinline__ float absmax16(const f2* v) {
  float m = max_nan(fabsf(lo_of(v[0])), fabsf(hi_of(v[0])));
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max3_nan(m, fabsf(lo_of(v[i])), fabsf(hi_of(v[i])));
  return m;
}

// Quantizes and stores the 16 elements of a lane from element `at`.  v: fp32
// values of x' whose relative error, with the rounding of the scaled value, is
// below delta.  zero(): the lane's x' are zeros for certain (an fp32 zero alone
// may be an underflow).  `force` sends the lane's group to fp64.  Every lane of the
// warp calls it; `on` lanes hold data, the others zeros.  A group with an
// undecided lane is decided in fp64 by the whole warp, an element a lane (about
// one group in 1500; done by its own lanes, one element after the other, it took
// 5 us).  Returns whether one of the warp's groups is not finite.
template <int FMT, int XDT, bool GLU, class Zero>
__device__ __forceinline__ bool quant_store16(const RowProblem& p, int64_t at, bool on, const f2* v, float delta, float sT,
                                              float isT, Zero&& zero, bool force, double rstd) {
  constexpr int LG = group_lanes(FMT), CW = code_words(FMT);
  float m = absmax16(v);
#pragma unroll
  for (int o = 1; o < LG; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  bool redo = false;
  float a = a_fast<FMT>(m, (float)grid_qmax(FMT), isT, redo);  // flags a zero, a NaN or an infinity too
  const float ia = fmt_pow2(FMT) ? __uint_as_float(0x7F000000u - __float_as_uint(a)) : __frcp_rn(a);
  const float c = FMT == FMT_NVFP4 ? isT * ia : ia;
  uint32_t cw[CW], cl[CW], differ = 0;
  codes_fast<FMT>(v, c * (1.f - delta), cl);
  codes_fast<FMT>(v, c * (1.f + delta), cw);
#pragma unroll
  for (int w = 0; w < CW; ++w) differ |= cl[w] ^ cw[w];
  if (m == 0.f) redo = !zero();  // a is 1 then; differ is 0
  redo |= differ != 0 || force;
  redo &= on;
  const uint32_t lanes = __ballot_sync(0xffffffffu, redo);
  const uint32_t groups = LG == 1 ? lanes : (lanes | (lanes >> 1)) & 0x55555555u;  // bit of a group's first lane
  if (on && !(groups >> (threadIdx.x & 31 & ~(LG - 1)) & 1u)) {
#pragma unroll
    for (int w = 0; w < CW; ++w) cw[w] = no_negzero<FMT>(cw[w]);
    if (FMT == FMT_MXFP8) {
      if (p.codes_vec) {
        *reinterpret_cast<uint4*>(p.codes + at) = make_uint4(cw[0], cw[1], cw[2 % CW], cw[3 % CW]);
      } else {
        *reinterpret_cast<uint2*>(p.codes + at) = make_uint2(cw[0], cw[1]);
        *reinterpret_cast<uint2*>(p.codes + at + 8) = make_uint2(cw[2 % CW], cw[3 % CW]);
      }
    } else {
      *reinterpret_cast<uint2*>(p.codes + (at >> 1)) = make_uint2(cw[0], cw[1]);
    }
    if ((threadIdx.x & (LG - 1)) == 0) store_scale<FMT>(p, at, a, false);
  }
  bool bad = false;
  for (uint32_t rest = groups; rest != 0; rest &= rest - 1)
    bad |= quant_exact<FMT, XDT, GLU>(p, __shfl_sync(0xffffffffu, at, __ffs(rest) - 1), rstd, sT);
  return bad;
}

// Grid-wide barrier of a cooperative launch (bounded wait).
__device__ __forceinline__ void row_grid_barrier(WsHeader* hdr) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(&hdr->gbar, 1u);
    const unsigned long long t0 = global_ns();
    while (ld_acquire_gpu(&hdr->gbar) < gridDim.x)
      if (wait_expired(&hdr->flags, t0)) break;
  }
  __syncthreads();
}

__device__ __forceinline__ void row_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Start of a kernel: everything before it in the stream is done.  A grid of one
// CTA, or of one cluster, clears its own header (a cluster meets once more
// before anything is written there).
__device__ __forceinline__ void row_begin(const RowProblem& p) {
  griddep_launch_dependents();
  griddep_wait();
  if ((gridDim.x == 1 || p.cluster) && p.hdr) {
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      p.hdr->flags = 0;
      p.hdr->gbar = 0;
      p.hdr->amax_scaled = 0;
    }
    __syncthreads();
  }
}

// Tensor scale from the bits of max |x'| (fp64) over the call.
__device__ __forceinline__ float tensor_scale(unsigned long long bits) {
  const double amax = __longlong_as_double((long long)bits);
  if (amax == 0.0) return 1.f;
  const float s = __double2float_rn(amax / 2688.0);
  return s == 0.f ? 0x1p-149f : s;
}

// ---------------------------------------------------------------------------
// dq_norm_quant: a CTA takes rows grid-stride, thread t the 16-element chunks
// t, t + blockDim, ...  With NC > 0 a thread has at most NC chunks and keeps its
// part of the row in registers; with NC = 0 (rows longer than 4 x 512 chunks)
// the stored row is read again after the sum.  The sum of squares is held in
// fp64.

template <int XDT>
__device__ __forceinline__ void gb16(const RowProblem& p, int64_t col, f2* gb) {
  b16_values(p, col, gb);
  if (p.g) {
    f2 g[8];
    pairs16<XDT>(load16(p.g, after_wait(col), false), g);
#pragma unroll
    for (int i = 0; i < 8; ++i) gb[i] = mul2(gb[i], g[i]);  // exact: at most 22 significant bits
  }
}

// 1/rms of the row from the threads' partial sums of squares; NaN for a row
// with a non-finite value.  `red`: 33 doubles of shared memory.
__device__ __forceinline__ double row_rstd(double s, double* red, const RowProblem& p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) red[warp] = s;
  __syncthreads();
  if (warp == 0) {
    double t = lane < nw ? red[lane] : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0) {
      const double r = 1.0 / sqrt(t / (double)p.K + (double)p.eps);
      red[32] = t <= 1.7976931348623157e308 ? r : __longlong_as_double(0x7FF8000000000000ll);
    }
  }
  __syncthreads();
  return red[32];
}

// The tensor's amax (NVFP4), exact without fp64 for every element: a lane keeps
// the chunk with its largest fp32 maximum (a relative 2^-20 off) and at the end
// the CTA's largest are evaluated in fp64.  Chunks within 2^-18 of the lane's
// largest, and those about which the fp32 value says nothing (a NaN, an
// infinity, an underflow), are evaluated when they come.
struct Amax {
  double exact = 0.0;  // of the chunks evaluated so far
  float best = 0.f;
  int64_t at = 0;      // first element of the lane's best chunk
  double rstd = 0.0;   // its row's
};

// Raises a.exact to the largest finite |x'| of the 16-element chunks from `at`
// of the lanes in the mask, an element a lane; every lane of the warp calls it.
template <int XDT, bool GLU>
static __device__ __noinline__ double amax_exact(const RowProblem& p, int64_t at, uint32_t lanes, double rstd, double amax) {
  const int lane = threadIdx.x & 31;
  for (uint32_t rest = lanes; rest != 0; rest &= rest - 1) {
    const int from = __ffs(rest) - 1;
    const int64_t first = __shfl_sync(0xffffffffu, at, from), row = first / p.K;
    const double r = __shfl_sync(0xffffffffu, rstd, from);
    const double x = lane < 16 ? fabs(exact1<XDT, GLU>(p, row, first - row * p.K + lane, r)) : 0.0;
    if (x <= (double)kFltMax) amax = fmax(amax, x);
  }
  return amax;
}

template <int XDT, bool GLU>
__device__ __forceinline__ void amax_add(const RowProblem& p, Amax& a, float m, int64_t at, bool on, bool force, double rstd) {
  const bool plain = !force && m >= 0x1p-60f && m <= kFltMax;
  bool now = on && !plain;
  if (on && plain) {
    if (m > a.best * (1.f + 0x1p-18f)) {
      a.best = m;
      a.at = at;
      a.rstd = rstd;
    } else {
      now = m >= a.best * (1.f - 0x1p-18f);
    }
  }
  const uint32_t ask = __ballot_sync(0xffffffffu, now);
  if (ask) a.exact = amax_exact<XDT, GLU>(p, at, ask, rstd, a.exact);
}

// The call's amax from the threads' shares (bits of a double; a wait for the
// other CTAs that runs out sets the header's flag).
template <int XDT, bool GLU>
__device__ __forceinline__ unsigned long long amax_finish(const RowProblem& p, Amax& a) {
  __shared__ unsigned top;  // fp32 bits: positive floats order as integers
  __shared__ unsigned long long all;
  if (threadIdx.x == 0) top = 0, all = 0;
  __syncthreads();
  float m = a.best;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) atomicMax(&top, __float_as_uint(m));
  __syncthreads();
  const uint32_t ask = __ballot_sync(0xffffffffu, a.best > 0.f && a.best >= __uint_as_float(top) * (1.f - 0x1p-18f));
  if (ask) a.exact = amax_exact<XDT, GLU>(p, a.at, ask, a.rstd, a.exact);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a.exact = fmax(a.exact, __shfl_xor_sync(0xffffffffu, a.exact, o));
  if ((threadIdx.x & 31) == 0 && a.exact > 0.0) atomicMax(&all, (unsigned long long)__double_as_longlong(a.exact));
  __syncthreads();
  if (gridDim.x == 1) return all;
  if (p.cluster) {
    row_cluster_sync();
    unsigned long long most = 0;
    for (unsigned r = 0; r < gridDim.x; ++r) {
      unsigned long long v;
      asm volatile("{\n.reg .b32 a;\nmapa.shared::cluster.u32 a, %1, %2;\nld.shared::cluster.u64 %0, [a];\n}"
                   : "=l"(v)
                   : "r"(smem_u32(&all)), "r"(r)
                   : "memory");
      most = max(most, v);
    }
    row_cluster_sync();  // no CTA leaves while another reads its shared memory
    return most;
  }
  if (threadIdx.x == 0) atomicMax(&p.hdr->amax_scaled, all);
  row_grid_barrier(p.hdr);
  return *reinterpret_cast<volatile unsigned long long*>(&p.hdr->amax_scaled);
}

// A CTA takes one row at a time, NC chunks of 16 elements a thread in registers
// between the sum of squares and the quantization (NC 0: rows of more than 2048
// chunks, read twice).  The sum is in fp64: x' has to be known to 2^-20 and
// decided exactly where that is not enough, and one fp64 add an element is 7 % of
// that pipe.  8192 x 4096 with residual: MXFP8 50 us, 4.7 TB/s of the 7 bytes an
// element; MXFP4 44 us; NVFP4, which writes h, meets the grid and reads h again, 96 us.
// 1 x 4096 MXFP8: 4 us.  Bound by the latency of a row's loads and its two
// barriers, with the issue slots half used.  Spilled, bytes stored a thread, bf16 and
// fp16 inputs: NC 2 (held to 80 registers) MXFP8 40 and 114, MXFP4 36 and 110, NVFP4
// 270 and 270; NC 4 (128) MXFP8 0 and 174, MXFP4 0 and 166, NVFP4 34 and 34; others none.
__host__ __device__ constexpr int norm_threads(int nc) { return nc == 1 || nc == 4 ? 512 : 256; }

template <int FMT, int XDT, int NC>
__global__ void __launch_bounds__(norm_threads(NC), NC == 2 ? 3 : 1) k_norm(const __grid_constant__ RowProblem p) {
  __shared__ double red[33];
  // g b of the thread's own chunks (NC > 1), 16-byte pieces [c][piece][thread]: written and read by one thread
  extern __shared__ uint4 gb_kept[];
  constexpr int N = NC > 0 ? NC : 1;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int chunks = (int)(p.K / 16);
  const int trips = NC > 0 ? 1 : (chunks + nt - 1) / nt;
  const void* hsrc = p.y ? p.h : p.x;
  row_begin(p);
  Amax amax;
  float sT = 1.f, isT = 1.f;
  bool sT_ok = true, bad = false;
  // NVFP4: a CTA with one row has it in registers in the second pass too
  const bool kept = FMT == FMT_NVFP4 && NC > 0 && p.M <= gridDim.x;
  double rstd = 0.0;
  V16 hv[N], rv[N];  // zeros for good where the thread has no chunk
#pragma unroll
  for (int c = 0; c < N; ++c) hv[c] = rv[c] = zero16();
  f2 gb[8];
  auto get_gb = [&](int ch) {
#pragma unroll
    for (int i = 0; i < 8; ++i) gb[i] = 0ull;
    if (ch < chunks) gb16<XDT>(p, ch * 16, gb);
  };
  if (NC == 1) get_gb(tid);
  if (NC > 1) {
#pragma unroll 1
    for (int c = 0; c < N; ++c) {
      get_gb(tid + c * nt);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ulonglong2 q;
        q.x = gb[2 * i];
        q.y = gb[2 * i + 1];
        *reinterpret_cast<ulonglong2*>(&gb_kept[(c * 4 + i) * nt + tid]) = q;
      }
    }
  }
  // pass 0 (NVFP4): sums, 1/rms and the tensor's amax; pass 1: scales and codes
#pragma unroll 1
  for (int pass = FMT == FMT_NVFP4 ? 0 : 1; pass < 2; ++pass) {
    if (FMT == FMT_NVFP4 && pass == 1) {
      sT = tensor_scale(amax_finish<XDT, false>(p, amax));
      if (gridDim.x > 1 && !p.cluster && (ld_volatile(&p.hdr->flags) & kFlagTimeout)) return;
      isT = __frcp_rn(sT);
      sT_ok = in_range(isT);
    }
    int64_t row0 = after_wait(blockIdx.x * p.K + tid * 16);  // element of the thread's first chunk
#pragma unroll 1
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, row0 += gridDim.x * p.K) {
      if (FMT != FMT_NVFP4 || pass == 0) {
        double s[4] = {0.0, 0.0, 0.0, 0.0};  // four chains of additions
#pragma unroll 1
        for (int t = 0; t < trips; ++t) {
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const int i = (NC > 0 ? c : t) * nt;
            if (NC == 0) hv[c] = rv[c] = zero16();
            if (tid + i < chunks) {
              hv[c] = load16(p.x, row0 + i * 16, p.wide);
              if (p.y) rv[c] = load16(p.y, row0 + i * 16, p.wide);
            }
          }
          if (p.y) {
#pragma unroll
            for (int c = 0; c < N; ++c) {
              const int i = (NC > 0 ? c : t) * nt;
#pragma unroll
              for (int k = 0; k < 8; ++k) hv[c].u[k] = h2_add<XDT>(hv[c].u[k], rv[c].u[k]);
              if (tid + i < chunks) store16(p.h, row0 + i * 16, p.wide, hv[c]);
            }
          }
#pragma unroll
          for (int c = 0; c < N; ++c) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 h = h2_values(hv[c].u[i], XDT);
              s[2 * (i & 1)] = fma((double)h.x, (double)h.x, s[2 * (i & 1)]);
              s[2 * (i & 1) + 1] = fma((double)h.y, (double)h.y, s[2 * (i & 1) + 1]);
            }
          }
        }
        rstd = row_rstd((s[0] + s[1]) + (s[2] + s[3]), red, p);
        if (FMT == FMT_NVFP4 && tid == 0) p.rstd[row] = rstd;
      } else if (!kept) {
        rstd = p.rstd[row];
      }
      const float rs = (float)rstd;
      // x' = h (rs gb): with rs from 2^-30 on a product rs gb that loses bits below fp32's normal range leaves |x'| < 2^-80
      // (|h| rs <= sqrt(K)), a zero code in every group whose scale the fast path settles (from 2^-60 on); one beyond
      // the range shows as an infinity or a NaN.  (h rs) gb would bring a subnormal h rs back into range.
      const bool rs_ok = rs >= 0x1p-30f && rs <= 0x1p100f;
#pragma unroll 1
      for (int t = 0; t < trips; ++t) {
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const int i0 = (NC > 0 ? c : t) * nt;
          const bool on = tid + i0 < chunks;
          if (NC > 1 && (tid & ~31) + i0 >= chunks) break;  // the whole warp is past the row
          if (NC == 0 || (FMT == FMT_NVFP4 && pass == 1 && !kept)) hv[c] = on ? load16_again(hsrc, row0 + i0 * 16) : zero16();
          if (NC == 0) get_gb(tid + i0);
          if (NC > 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(&gb_kept[(c * 4 + i) * nt + tid]);
              gb[2 * i] = q.x;
              gb[2 * i + 1] = q.y;
            }
          }
          f2 v[8];
          pairs16<XDT>(hv[c], v);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], mul2(gb[i], splat(rs)));
          if (FMT == FMT_NVFP4 && pass == 0) {
            // values that are not finite have no share in the tensor scale
            amax_add<XDT, false>(p, amax, absmax16(v), row0 + i0 * 16, on && rstd == rstd && !zero_bits16(hv[c]), !rs_ok, rstd);
          } else {
            // relative error: 1/rms, two products, the scale's factor and the scaled value, 2^-24 each (NVFP4: three more)
            bad |= quant_store16<FMT, XDT, false>(p, row0 + i0 * 16, on, v, 0x1p-20f, sT, isT, [&] { return zero_bits16(hv[c]); },
                                                  !sT_ok || !rs_ok, rstd);
          }
        }
      }
    }
  }
  if (blockIdx.x == 0 && tid == 0 && p.sT_out) *p.sT_out = sT;
  if (bad && (tid & 31) == 0 && p.hdr) atomicOr(&p.hdr->flags, kFlagNonFinite);
}

// ---------------------------------------------------------------------------
// dq_glu_quant: elementwise but for the groups, so the warps of the grid take
// items of 32 x 16 consecutive columns of a row, row-major and grid-stride, and
// read the next item while they work on one.  The grid's warps are a multiple
// of a row's items where there are enough, so a warp keeps its columns and
// their scales.

// A lane's 16 column scales and their products with 16-bit values, exact in fp32:
// as stored, multiplied by mixed-precision fma, where the types agree.
template <bool BSAME>
struct GluCols {
  uint32_t w[BSAME ? 8 : 1];
  f2 f[BSAME ? 1 : 8];
  __device__ __forceinline__ void load(const RowProblem& p, int64_t col, bool on) {
    if (BSAME) {
      const uint16_t* b = reinterpret_cast<const uint16_t*>(p.b_store) + col;
#pragma unroll
      for (int i = 0; i < (BSAME ? 8 : 1); ++i) w[i] = on ? (uint32_t)b[2 * i] | (uint32_t)b[2 * i + 1] << 16 : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < (BSAME ? 1 : 8); ++i) f[i] = 0ull;
      if (on) b16_values(p, col, f);
    }
  }
  __device__ __forceinline__ void times(const V16& v, int xdt, f2* x) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (BSAME) {
        float lo, hi;
        if (xdt == DT_BF16)
          asm("{\n.reg .b16 x0, x1, b0, b1;\nmov.b32 {x0, x1}, %2;\nmov.b32 {b0, b1}, %3;\n"
              "fma.rn.f32.bf16 %0, x0, b0, 0f80000000;\nfma.rn.f32.bf16 %1, x1, b1, 0f80000000;\n}"
              : "=f"(lo), "=f"(hi)
              : "r"(v.u[i]), "r"(w[BSAME ? i : 0]));
        else
          asm("{\n.reg .b16 x0, x1, b0, b1;\nmov.b32 {x0, x1}, %2;\nmov.b32 {b0, b1}, %3;\n"
              "fma.rn.f32.f16 %0, x0, b0, 0f80000000;\nfma.rn.f32.f16 %1, x1, b1, 0f80000000;\n}"
              : "=f"(lo), "=f"(hi)
              : "r"(v.u[i]), "r"(w[BSAME ? i : 0]));
        x[i] = pk(lo, hi);
      } else {
        const float2 a = h2_values(v.u[i], xdt);
        x[i] = mul2(pk(a.x, a.y), f[BSAME ? 0 : i]);
      }
    }
  }
};

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Smallest and largest of a lane's 16-bit elements (NaN ignored).
template <int XDT>
__device__ __forceinline__ void range16(const V16& v, float& lo, float& hi) {
  uint32_t a = v.u[0], b = v.u[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    if (XDT == DT_BF16) {
      asm("min.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(v.u[i]));
      asm("max.bf16x2 %0, %0, %1;" : "+r"(b) : "r"(v.u[i]));
    } else {
      asm("min.f16x2 %0, %0, %1;" : "+r"(a) : "r"(v.u[i]));
      asm("max.f16x2 %0, %0, %1;" : "+r"(b) : "r"(v.u[i]));
    }
  }
  const float2 x = h2_values(a, XDT), y = h2_values(b, XDT);
  lo = fminf(x.x, x.y);
  hi = fmaxf(y.x, y.y);
}

// x' in fp32.  exp(-g) = 2^t (1 + ln2 r) with t = fp32(-g log2 e) and r what its
// rounding left out, formed by fma; ex2.approx is good to 2^-22.5, rcp.approx to
// 2^-23, and five further roundings give 2^-21 in all.  `far` marks gates whose
// exponential (below -80) or product with an underflowed up * b (above 2^40)
// leaves that bound; an up * b that overflows shows as an infinity or a NaN.
// (Otherwise an up * b below the normal range gives |x'| < 2^-86: a zero code in
// every group whose scale the fast path settles.)
template <int XDT, bool BSAME>
__device__ __forceinline__ void glu_fast16(const V16& gv, const V16& uv, const GluCols<BSAME>& b, f2* v, bool& far) {
  float lo, hi;
  range16<XDT>(gv, lo, hi);
  far = !(lo >= -80.f && hi <= 0x1p40f);
  f2 g[8], u[8];
  pairs16<XDT>(gv, g);
  b.times(uv, XDT, u);
  // log2(e) as the sum of two fp32 numbers
  const f2 l1 = splat(1.44269502f), m1 = splat(-1.44269502f), l2 = splat((float)(1.4426950408889634 - (double)1.44269502f));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const f2 t = mul2(g[i], m1);
    const f2 r = fma2(g[i], l2, fma2(g[i], l1, t));  // minus what t lacks
    f2 e = pk(ex2_approx(lo_of(t)), ex2_approx(hi_of(t)));
    e = fma2(e, mul2(r, splat(-0.693147181f)), e);
    const f2 d = add2(e, splat(1.f));
    const f2 s = pk(rcp_approx(lo_of(d)), rcp_approx(hi_of(d)));
    v[i] = mul2(mul2(g[i], s), u[i]);
  }
}

// A warp takes 512 columns of a row at a time, two such items in turn, so that one's
// loads are under way while the other is computed.  8192 x 14336 MXFP8: 114 us, 5.2
// TB/s of the 5 bytes an element; MXFP4 105 us; NVFP4, which reads and computes twice,
// 211 us.  16 x 14336 MXFP8: 4.7 us.  Bound by instructions (22 an
// element: the sigmoid's exponential and reciprocal, two conversions of the
// bracket's ends); a ring of asynchronous copies added to them: 168 us against the
// 133 of its time.
template <int FMT, int XDT, bool BSAME>
__global__ void __launch_bounds__(kGluMax, 1) k_glu(const __grid_constant__ RowProblem p) {
  const int lane = threadIdx.x & 31;
  const int64_t spans = (p.K + 511) / 512;  // 512-column pieces of a row
  const int64_t w0 = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t all = (int64_t)gridDim.x * (blockDim.x >> 5);
  const int64_t nw = all >= spans ? all / spans * spans : all;  // warps that take items
  const int drow = (int)(nw / spans), dspan = (int)(nw - drow * spans);  // the grid's stride as rows and spans
  // ... and as elements of the inputs and outputs, without and with a carry into the next row
  const int64_t din = drow * p.ld + dspan * 512, dout = drow * p.K + dspan * 512;
  const int64_t cin = p.ld - spans * 512, cout = p.K - spans * 512;
  row_begin(p);
  Amax amax;
  float sT = 1.f, isT = 1.f;
  bool sT_ok = true, bad = false;
  GluCols<BSAME> b;
  int have = -1;
  // NVFP4: a warp with one item has it in registers in the second pass too
  const bool kept = FMT == FMT_NVFP4 && p.M * spans <= nw;
  V16 g0 = zero16(), u0 = zero16(), g1 = zero16(), u1 = zero16();  // two items in turn: no copies of registers
#pragma unroll 1
  for (int pass = FMT == FMT_NVFP4 ? 0 : 1; pass < 2; ++pass) {
    if (FMT == FMT_NVFP4 && pass == 1) {
      sT = tensor_scale(amax_finish<XDT, true>(p, amax));
      if (gridDim.x > 1 && !p.cluster && (ld_volatile(&p.hdr->flags) & kFlagTimeout)) return;
      isT = __frcp_rn(sT);
      sT_ok = in_range(isT);
    }
    int64_t row = w0 < nw ? w0 / spans : p.M;
    int span = (int)(w0 - row * spans);
    int64_t in = after_wait(row * p.ld + (int64_t)span * 512 + lane * 16), at = row * p.K + (int64_t)span * 512 + lane * 16;
    auto read = [&](V16& g, V16& u) {
      if (row < p.M && (int64_t)span * 512 + lane * 16 < p.K) {
        g = load16(p.x, in, p.wide);
        u = load16(p.y, in, p.wide);
      }
    };
    // works on (gv, uv), the item at row and span, and reads the next one
    auto step = [&](const V16& gv, const V16& uv, V16& g, V16& u) {
      const int64_t col = (int64_t)span * 512 + lane * 16, here = at;
      const bool on = col < p.K;
      if (span != have) {
        b.load(p, col, on);
        have = span;
      }
      row += drow;
      span += dspan;
      in += din;
      at += dout;
      if (span >= spans) {
        span -= (int)spans;
        ++row;
        in += cin;
        at += cout;
      }
      if (!kept) read(g, u);
      f2 v[8];
      bool far;
      glu_fast16<XDT, BSAME>(gv, uv, b, v, far);
      if (FMT == FMT_NVFP4 && pass == 0) {
        // values that are not finite have no share in the tensor scale
        amax_add<XDT, true>(p, amax, absmax16(v), here, on && !zero_bits16(gv) && !zero_bits16(uv), far, 0.0);
      } else {
        // 2^-21 of x' and the roundings of the scaled value
        bad |= quant_store16<FMT, XDT, true>(p, here, on, v, 1.25f * 0x1p-20f, sT, isT,
                                             [&] { return zero_bits16(gv) || zero_bits16(uv); }, !sT_ok || far, 0.0);
      }
    };
    if (!(kept && pass == 1)) read(g0, u0);
#pragma unroll 1
    while (row < p.M) {
      step(g0, u0, g1, u1);
      if (row >= p.M) break;
      step(g1, u1, g0, u0);
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.sT_out) *p.sT_out = sT;
  if (bad && lane == 0 && p.hdr) atomicOr(&p.hdr->flags, kFlagNonFinite);
}

// ---------------------------------------------------------------------------
// Host side.

// One resident wave (the NVFP4 kernels wait for the whole grid: cooperative).
// A single CTA clears the header itself; more of them need it cleared before.
// Up to one CTA an SM is resident whatever the kernel's registers, so the
// occupancy is asked for beyond that only (a microsecond of the host's time).
static cudaError_t row_launch(void (*kern)(RowProblem), const RowProblem& p, bool coop, int64_t want, int threads,
                              size_t smem, int sms, cudaStream_t st) {
  cudaError_t e;
  // the same limit in every call: another thread's call may come between this and the launch
  if (smem > 48 * 1024 &&
      (e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem)) != cudaSuccess)
    return e;
  int grid = (int)(want < sms ? want : sms);
  if (coop && grid > 1 && grid <= 8) {  // the CTAs of a cluster need no cooperative launch and no clearing
    RowProblem one = p;
    one.cluster = 1;
    return launch_early(kern, (unsigned)grid, (unsigned)threads, smem, grid, st, one);
  }
  if (want > sms) {
    int per_sm = 0;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem)) != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    const int64_t most = (int64_t)sms * per_sm;
    grid = (int)(want < most ? want : most);
  }
  if (grid > 1 && p.hdr && (e = cudaMemsetAsync(p.hdr, 0, sizeof(WsHeader), st)) != cudaSuccess) return e;
  if (!coop || grid == 1)
    return launch_early(kern, (unsigned)grid, (unsigned)threads, smem, 1, st, p);
  RowProblem arg = p;
  void* args[] = {&arg};
  return cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kern), dim3(grid), dim3(threads), args, smem, st);
}

// Few rows: a chunk a thread, for latency.  From 4 rows an SM on: 2 chunks a
// thread at 80 registers and their spills, for 24 warps an SM (8192 x 4096 MXFP8: 53 us
// with 1 chunk a thread, 50 with 2, 51 with 4 at 126 registers).  What bounds it then is
// latency, not the memory: bringing the next row into shared memory meanwhile
// took longer (56 us).
template <int FMT, int XDT>
static cudaError_t norm_launch(const RowProblem& p, int sms, cudaStream_t st) {
  const int64_t chunks = p.K / 16;
  int nc, threads;
  if (chunks > 512)
    nc = chunks <= 4 * 512 ? 4 : 0;
  else
    nc = p.M >= 4 * (int64_t)sms ? 2 : 1;
  threads = nc == 0 ? 256 : (int)(((chunks + nc - 1) / nc + 31) / 32 * 32);
  void (*kern)(RowProblem) = nc == 1   ? k_norm<FMT, XDT, 1>
                             : nc == 2 ? k_norm<FMT, XDT, 2>
                             : nc == 4 ? k_norm<FMT, XDT, 4>
                                       : k_norm<FMT, XDT, 0>;
  return row_launch(kern, p, FMT == FMT_NVFP4, p.M, threads, nc > 1 ? (size_t)nc * threads * 64 : 0, sms, st);
}

template <int FMT, int XDT>
static cudaError_t glu_launch(const RowProblem& p, int sms, cudaStream_t st) {
  void (*kern)(RowProblem) = p.b_store && p.col_dt == XDT ? k_glu<FMT, XDT, true> : k_glu<FMT, XDT, false>;
  const int64_t items = p.M * ((p.K + 511) / 512);
  // NVFP4, few items: one cluster with an item a warp, whose two passes need no grid barrier and whose header no clearing
  if (FMT == FMT_NVFP4 && items <= 8 * (kGluMax / 32)) {
    const int threads = items <= 32 ? 128 : (items <= 64 ? 256 : kGluMax);
    return row_launch(kern, p, true, (items + threads / 32 - 1) / (threads / 32), threads, 0, sms, st);
  }
  return row_launch(kern, p, FMT == FMT_NVFP4, (items + 7) / 8, kGluThreads, 0, sms, st);
}

// Checks shared by the two entry points.
static int row_check(int64_t rows, int64_t cols, int x_dtype, const void* col_scales, int col_dtype, int format, int group,
                     const dq_outputs* out, const void* workspace) {
  if (rows <= 0 || cols <= 0 || group <= 0 || cols % group != 0) return DQ_EINVAL;
  if (format < DQ_INT4 || format > DQ_MXFP8) return DQ_EINVAL;
  if (format != DQ_NVFP4 && format != DQ_MXFP4 && format != DQ_MXFP8) return DQ_EUNSUPPORTED;
  if (group != (format == DQ_NVFP4 ? 16 : 32)) return DQ_EUNSUPPORTED;
  if (x_dtype != DQ_BF16 && x_dtype != DQ_F16) return DQ_EUNSUPPORTED;
  if (col_scales && col_dtype != DQ_BF16 && col_dtype != DQ_F16) return DQ_EUNSUPPORTED;
  if (rows > ((int64_t)1 << 40) / cols || cols > INT_MAX) return DQ_EUNSUPPORTED;
  if ((uintptr_t)col_scales % 2 != 0) return DQ_EINVAL;
  if (!out || !out->codes || !out->block_scales || (uintptr_t)out->codes % 8 != 0 ||
      (format == DQ_NVFP4 && !out->tensor_scale) || (uintptr_t)out->tensor_scale % 4 != 0)
    return DQ_EINVAL;
  if ((!workspace && format == DQ_NVFP4) || (uintptr_t)workspace % 256 != 0) return DQ_EINVAL;
  return DQ_OK;
}

static int row_sms(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DQ_ECUDA;
  return cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? DQ_OK : DQ_ECUDA;
}

static void row_fill(RowProblem* p, int64_t rows, int64_t cols, const void* col_scales, int col_dtype,
                     const dq_outputs* out, void* workspace) {
  p->b_store = col_scales;
  p->col_dt = col_dtype;
  p->b_vec = col_scales != nullptr && (uintptr_t)col_scales % 16 == 0;
  p->codes_vec = (uintptr_t)out->codes % 16 == 0;
  p->M = rows;
  p->K = cols;
  p->codes = static_cast<unsigned char*>(out->codes);
  p->scales = static_cast<unsigned char*>(out->block_scales);
  p->sT_out = out->tensor_scale;
  p->hdr = static_cast<WsHeader*>(workspace);
}

}  // namespace dq

extern "C" size_t dq_norm_workspace_bytes(int64_t rows, int64_t cols, int format, int group) {
  if (rows <= 0 || cols <= 0 || group <= 0 || cols % group != 0 || rows > ((int64_t)1 << 40) / cols || cols > INT_MAX) return 0;
  if (format != DQ_NVFP4 && format != DQ_MXFP4 && format != DQ_MXFP8) return 0;
  if (group != (format == DQ_NVFP4 ? 16 : 32)) return 0;
  return DQ_ACT_WORKSPACE_BYTES + (format == DQ_NVFP4 ? (size_t)rows * sizeof(double) : 0);
}

extern "C" int dq_norm_quant(const void* X, const void* residual, int x_dtype, int64_t rows, int64_t cols,
                             const void* weight, float eps, const void* col_scales, int col_dtype, int format, int group,
                             const dq_outputs* out, void* residual_out, void* workspace, size_t workspace_bytes,
                             void* stream) {
  int st = dq::row_check(rows, cols, x_dtype, col_scales, col_dtype, format, group, out, workspace);
  if (st != DQ_OK) return st;
  if (!X || (uintptr_t)X % 16 != 0 || (uintptr_t)residual % 16 != 0 || (uintptr_t)weight % 16 != 0) return DQ_EINVAL;
  if (residual ? (!residual_out || (uintptr_t)residual_out % 16 != 0) : residual_out != nullptr) return DQ_EINVAL;
  if (!(eps >= 0.f && eps <= dq::kFltMax)) return DQ_EINVAL;
  if (workspace && workspace_bytes < dq_norm_workspace_bytes(rows, cols, format, group)) return DQ_EWORKSPACE;
  int sms = 0;
  if ((st = dq::row_sms(&sms)) != DQ_OK) return st;
  dq::RowProblem p{};
  dq::row_fill(&p, rows, cols, col_scales, col_dtype, out, workspace);
  p.x = X;
  p.y = residual;
  p.g = weight;
  p.ld = cols;
  p.eps = eps;
  p.h = residual_out;
  p.wide = ((uintptr_t)X | (uintptr_t)residual | (uintptr_t)residual_out) % 32 == 0;  // a row is a multiple of 32 bytes
  if (format == DQ_NVFP4) p.rstd = reinterpret_cast<double*>(static_cast<unsigned char*>(workspace) + DQ_ACT_WORKSPACE_BYTES);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (format == DQ_NVFP4)
    e = x_dtype == DQ_BF16 ? dq::norm_launch<dq::FMT_NVFP4, dq::DT_BF16>(p, sms, s) : dq::norm_launch<dq::FMT_NVFP4, dq::DT_F16>(p, sms, s);
  else if (format == DQ_MXFP4)
    e = x_dtype == DQ_BF16 ? dq::norm_launch<dq::FMT_MXFP4, dq::DT_BF16>(p, sms, s) : dq::norm_launch<dq::FMT_MXFP4, dq::DT_F16>(p, sms, s);
  else
    e = x_dtype == DQ_BF16 ? dq::norm_launch<dq::FMT_MXFP8, dq::DT_BF16>(p, sms, s) : dq::norm_launch<dq::FMT_MXFP8, dq::DT_F16>(p, sms, s);
  return e == cudaSuccess ? DQ_OK : DQ_ECUDA;
}

extern "C" int dq_glu_quant(const void* gate, const void* up, int x_dtype, int64_t rows, int64_t cols, int64_t ld,
                            const void* col_scales, int col_dtype, int format, int group, const dq_outputs* out,
                            void* workspace, size_t workspace_bytes, void* stream) {
  int st = dq::row_check(rows, cols, x_dtype, col_scales, col_dtype, format, group, out, workspace);
  if (st != DQ_OK) return st;
  if (!gate || !up || (uintptr_t)gate % 16 != 0 || (uintptr_t)up % 16 != 0) return DQ_EINVAL;
  if (ld < cols || ld % 8 != 0 || rows > ((int64_t)1 << 40) / ld) return DQ_EINVAL;
  if (workspace && workspace_bytes < DQ_ACT_WORKSPACE_BYTES) return DQ_EWORKSPACE;
  int sms = 0;
  if ((st = dq::row_sms(&sms)) != DQ_OK) return st;
  dq::RowProblem p{};
  dq::row_fill(&p, rows, cols, col_scales, col_dtype, out, workspace);
  p.x = gate;
  p.y = up;
  p.ld = ld;
  p.wide = ((uintptr_t)gate | (uintptr_t)up | (uintptr_t)(2 * ld)) % 32 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (format == DQ_NVFP4)
    e = x_dtype == DQ_BF16 ? dq::glu_launch<dq::FMT_NVFP4, dq::DT_BF16>(p, sms, s) : dq::glu_launch<dq::FMT_NVFP4, dq::DT_F16>(p, sms, s);
  else if (format == DQ_MXFP4)
    e = x_dtype == DQ_BF16 ? dq::glu_launch<dq::FMT_MXFP4, dq::DT_BF16>(p, sms, s) : dq::glu_launch<dq::FMT_MXFP4, dq::DT_F16>(p, sms, s);
  else
    e = x_dtype == DQ_BF16 ? dq::glu_launch<dq::FMT_MXFP8, dq::DT_BF16>(p, sms, s) : dq::glu_launch<dq::FMT_MXFP8, dq::DT_F16>(p, sms, s);
  return e == cudaSuccess ? DQ_OK : DQ_ECUDA;
}

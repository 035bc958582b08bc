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
// fp32 values known to a relative 2^-20 (norm) or 2^-19 (glu) settle nearly
// all of them: a code is certain where both ends of that bracket convert to
// it, a block scale where the fp32 ratio is not next to a projection midpoint.
// The rest is decided in fp64 from the stored inputs.
#include <climits>
#include <math_constants.h>

#include "dq.h"
#include "dq_device.cuh"
#include "dq_fast.cuh"
#include "dq_internal.h"

namespace dq {

constexpr int kGluThreads = 256;
constexpr float kFltMax = 3.402823466e38f;

struct RowProblem {
  const void* x;          // norm: hidden state; glu: gate
  const void* y;          // norm: residual or NULL; glu: up
  const void* g;          // norm weight or NULL
  const void* b_store;    // column inverse scales or NULL
  int col_dt;
  int b_vec;              // b_store is 16-byte aligned
  int64_t M, K, ld;       // rows, columns, row stride of x and y in elements
  float eps;
  void* h;                // residual sum out (aliases x or y at will) or NULL
  unsigned char* codes;
  unsigned char* scales;  // [M][nb] bytes
  int64_t nb;
  float* sT_out;
  double* rstd;           // NVFP4 norm: 1/rms of every row between the passes
  WsHeader* hdr;
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

template <int XDT>
__device__ __forceinline__ void h8_values(const uint4& v, float* x) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = h2_values(u[i], XDT);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// The 8 column scales at col (1 where there are none).
__device__ __forceinline__ void b8_values(const RowProblem& p, int64_t col, float* b) {
  if (p.b_vec) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.b_store) + col));
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = h2_values(u[i], p.col_dt);
      b[2 * i] = f.x;
      b[2 * i + 1] = f.y;
    }
  } else if (p.b_store) {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = b_decode(p.b_store, p.col_dt, col + i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = 1.f;
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

// Lanes of a group at 8 elements a lane.
__host__ __device__ constexpr int group_lanes(int fmt) { return fmt == FMT_NVFP4 ? 2 : 4; }

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

// Codes of 8 elements from their fp64 values: 8 bytes, or 8 nibbles in cw[0].
template <int FMT>
__device__ __forceinline__ void codes_exact(const double* x, double a, uint32_t* cw) {
  cw[0] = cw[1] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t m = mag_code<FMT>(fabs(x[i]), a);
    const uint32_t neg = m != 0 && x[i] < 0.0;
    if (FMT == FMT_MXFP8)
      cw[i >> 2] |= (m | (neg << 7)) << (8 * (i & 3));
    else
      cw[0] |= (m | (neg << 3)) << (4 * i);
  }
}

// Eight packed conversions of v[0..7] times s: E4M3 bytes or E2M1 nibbles
// (hardware round to nearest even, saturating).
template <int FMT>
__device__ __forceinline__ void codes_fast(const f2* v, float s, uint32_t* cw) {
  const f2 ss = splat(s);
  f2 t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = mul2(v[i], ss);
  if (FMT == FMT_MXFP8) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
      asm("{\n.reg .b16 l, h;\ncvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\ncvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n"
          "mov.b32 %0, {l, h};\n}"
          : "=r"(cw[c])
          : "f"(lo_of(t[2 * c])), "f"(hi_of(t[2 * c])), "f"(lo_of(t[2 * c + 1])), "f"(hi_of(t[2 * c + 1])));
  } else {
    asm("{\n.reg .b8 c0, c1, c2, c3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 c0, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 c1, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 c2, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 c3, %8, %7;\n"
        "mov.b32 %0, {c0, c1, c2, c3};\n}"
        : "=r"(cw[0])
        : "f"(lo_of(t[0])), "f"(hi_of(t[0])), "f"(lo_of(t[1])), "f"(hi_of(t[1])), "f"(lo_of(t[2])), "f"(hi_of(t[2])),
          "f"(lo_of(t[3])), "f"(hi_of(t[3])));
    cw[1] = 0;
  }
}

// A zero magnitude has no sign.
template <int FMT>
__device__ __forceinline__ uint32_t no_negzero(uint32_t w) {
  if (FMT == FMT_MXFP8) return w & (((w & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | 0x7F7F7F7Fu);
  return w & (0x77777777u | (w << 1) | (w << 2) | (w << 3));
}

// fp64 values of 8 elements of x' at (row, col), from the stored inputs.
template <int XDT, bool GLU>
__device__ __forceinline__ void exact8(const RowProblem& p, int64_t row, int64_t col, double rstd, double* x) {
  const uint16_t* src = reinterpret_cast<const uint16_t*>(GLU ? p.x : (p.y ? p.h : p.x));
  float h[8], b[8], g[8];
  h8_values<XDT>(*reinterpret_cast<const uint4*>(src + row * p.ld + col), h);
  b8_values(p, col, b);
  if (GLU) {
    h8_values<XDT>(*reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.y) + row * p.ld + col), g);
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      const double d = (double)h[i];
      x[i] = d / (1.0 + exp(-d)) * ((double)g[i] * (double)b[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = 1.f;
    if (p.g) h8_values<XDT>(__ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.g) + col)), g);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (double)h[i] * ((double)g[i] * (double)b[i]) * rstd;
  }
}

// The lane's codes (8 bytes, or 4 in cw[0]) and its group's scale to memory.
template <int FMT>
__device__ __forceinline__ void store8(const RowProblem& p, int64_t row, int64_t col, const uint32_t* cw, float a, bool bad) {
  constexpr int LG = group_lanes(FMT);
  const int64_t at = row * p.K + col;
  if (FMT == FMT_MXFP8)
    *reinterpret_cast<uint2*>(p.codes + at) = make_uint2(cw[0], cw[1]);
  else
    *reinterpret_cast<uint32_t*>(p.codes + (at >> 1)) = cw[0];
  if ((threadIdx.x & (LG - 1)) == 0) {
    unsigned char* s = p.scales + row * p.nb + col / (8 * LG);
    if (bad)
      *s = fmt_pow2(FMT) ? 0xFFu : 0x7Fu;
    else
      a_store_f<FMT>(s, 0, a);
  }
}

// A warp's 32 x 8 elements decided in fp64 throughout and stored: the cold path,
// out of line.  A group with a value that is not finite in fp32 gets the
// format's NaN scale and zero codes; returns whether the lane's group did.
template <int FMT, int XDT, bool GLU>
static __device__ __noinline__ bool quant_exact(const RowProblem& p, int64_t row, int64_t col, bool on, double rstd, float sT) {
  constexpr int LG = group_lanes(FMT);
  double x[8], m = 0.0;
  if (on) {
    exact8<XDT, GLU>(p, row, col, rstd, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmax(m, fabs(x[i]) <= (double)kFltMax ? fabs(x[i]) : CUDART_INF);
  }
#pragma unroll
  for (int o = 1; o < LG; o <<= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!on) return false;
  const bool bad = m > (double)kFltMax;
  const float a = m == 0.0 || bad ? 1.f : (float)a_project<FMT>(m / grid_qmax(FMT), (double)sT);
  uint32_t cw[2] = {0u, 0u};
  if (!bad) codes_exact<FMT>(x, FMT == FMT_NVFP4 ? (double)sT * (double)a : (double)a, cw);
  store8<FMT>(p, row, col, cw, a, bad);
  return bad;
}

// Quantizes and stores the 8 elements of a lane at (row, col).  v: fp32 values
// of x' known to a relative delta/2.  `force` sends the warp to fp64.  Every
// lane of the warp calls it; `on` lanes hold data, the others zeros.  One
// undecided lane sends the whole warp to fp64 (about one call in 100 at most):
// zeros go there too, as their scale is 1 only if no product underflowed.
template <int FMT, int XDT, bool GLU>
__device__ __forceinline__ bool quant_store8(const RowProblem& p, int64_t row, int64_t col, bool on, const f2* v, float delta,
                                             float sT, float isT, bool force, double rstd) {
  constexpr int LG = group_lanes(FMT);
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max3_nan(m, fabsf(lo_of(v[i])), fabsf(hi_of(v[i])));
#pragma unroll
  for (int o = 1; o < LG; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  bool redo = force;
  const float a = a_fast<FMT>(m, (float)grid_qmax(FMT), isT, redo);  // flags a NaN or an infinity too
  const float ia = fmt_pow2(FMT) ? __uint_as_float(0x7F000000u - __float_as_uint(a)) : __frcp_rn(a);
  const float c = FMT == FMT_NVFP4 ? isT * ia : ia;
  uint32_t cw[2], cl[2];
  codes_fast<FMT>(v, c * (1.f - delta), cl);
  codes_fast<FMT>(v, c * (1.f + delta), cw);
  redo |= cl[0] != cw[0] || cl[1] != cw[1];
  if (__any_sync(0xffffffffu, redo && on)) return quant_exact<FMT, XDT, GLU>(p, row, col, on, rstd, sT);
  if (on) {
    cw[0] = no_negzero<FMT>(cw[0]);
    if (FMT == FMT_MXFP8) cw[1] = no_negzero<FMT>(cw[1]);
    store8<FMT>(p, row, col, cw, a, false);
  }
  return false;
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

// Tensor scale from the bits of max |x'| (fp64) over the call.
__device__ __forceinline__ float tensor_scale(unsigned long long bits) {
  const double amax = __longlong_as_double((long long)bits);
  if (amax == 0.0) return 1.f;
  const float s = __double2float_rn(amax / 2688.0);
  return s == 0.f ? 0x1p-149f : s;
}

// Block-wide maximum of a non-negative double into hdr->amax_scaled.
__device__ __forceinline__ void amax_to_header(WsHeader* hdr, double amax) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmax(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0 && amax > 0.0)
    atomicMax(&hdr->amax_scaled, (unsigned long long)__double_as_longlong(amax));
}

// ---------------------------------------------------------------------------
// dq_norm_quant: a CTA takes rows grid-stride, thread t the 8-element chunks
// t, t + blockDim, ...  With NC = 1, 2 or 4 a thread has at most NC chunks and
// keeps its part of the row in registers; with NC = 1 and 2 it also reads the
// next row while it works on this one, and with NC = 1 it keeps g b.  NC = 0
// is for rows longer than 4 x 1024 chunks: the stored row is read again after
// the sum.  The sum of squares is held in fp64.

template <int XDT>
__device__ __forceinline__ void gb8(const RowProblem& p, int64_t col, float* gb) {
  b8_values(p, col, gb);
  if (p.g) {
    float g[8];
    h8_values<XDT>(__ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.g) + col)), g);
#pragma unroll
    for (int i = 0; i < 8; ++i) gb[i] *= g[i];  // exact: at most 22 significant bits
  }
}

__device__ __forceinline__ uint4 load16(const void* base, int64_t off) {
  return *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + off);
}

// h = x + r, rounded to the input type.
template <int XDT>
__device__ __forceinline__ uint4 add8(const uint4& x, const uint4& r) {
  return make_uint4(h2_add<XDT>(x.x, r.x), h2_add<XDT>(x.y, r.y), h2_add<XDT>(x.z, r.z), h2_add<XDT>(x.w, r.w));
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

// Largest finite |x'| of a lane's 8 elements, in fp64.
template <int XDT, bool GLU>
static __device__ __noinline__ double amax_exact(const RowProblem& p, int64_t row, int64_t col, double rstd) {
  double x[8], m = 0.0;
  exact8<XDT, GLU>(p, row, col, rstd, x);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (fabs(x[i]) <= (double)kFltMax) m = fmax(m, fabs(x[i]));
  return m;
}

template <int FMT, int XDT, int NC>
__global__ void __launch_bounds__(NC == 1 || NC == 2 ? 512 : 1024, NC == 1 || NC == 2 ? 2 : 1)
    k_norm(const __grid_constant__ RowProblem p) {
  __shared__ double red[33];
  constexpr int N = NC > 0 ? NC : 1;
  constexpr bool AHEAD = NC == 1 || NC == 2, KEEP = NC == 1;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int chunks = (int)(p.K / 8);
  const int trips = NC > 0 ? 1 : (chunks + nt - 1) / nt;
  const void* hsrc = p.y ? p.h : p.x;
  float gb[N][8];
  auto get_gb = [&](int c, int ch) {
#pragma unroll
    for (int i = 0; i < 8; ++i) gb[c][i] = 0.f;
    if (ch < chunks) gb8<XDT>(p, ch * 8, gb[c]);
  };
  uint4 xv[N], rv[N];  // the next row's inputs
  auto read = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const int ch = tid + c * nt;
      xv[c] = rv[c] = make_uint4(0, 0, 0, 0);
      if (row < p.M && ch < chunks) {
        xv[c] = load16(p.x, row * p.K + ch * 8);
        if (p.y) rv[c] = load16(p.y, row * p.K + ch * 8);
      }
    }
  };
  if (AHEAD) {
    read(blockIdx.x);
    if (KEEP) get_gb(0, tid);
  }
  double amax = 0.0;
  float sT = 1.f, isT = 1.f;
  bool sT_ok = true, bad = false;
  uint4 hv[N];
  // pass 0 (NVFP4): sums, 1/rms and the tensor's amax; pass 1: scales and codes
#pragma unroll 1
  for (int pass = FMT == FMT_NVFP4 ? 0 : 1; pass < 2; ++pass) {
    if (FMT == FMT_NVFP4 && pass == 1) {
      amax_to_header(p.hdr, amax);
      row_grid_barrier(p.hdr);
      if (ld_volatile(&p.hdr->flags) & kFlagTimeout) return;
      sT = tensor_scale(*reinterpret_cast<volatile unsigned long long*>(&p.hdr->amax_scaled));
      isT = __frcp_rn(sT);
      sT_ok = in_range(isT);
    }
#pragma unroll 1
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
      double rstd;
      if (FMT != FMT_NVFP4 || pass == 0) {
        double s = 0.0;
#pragma unroll 1
        for (int t = 0; t < trips; ++t) {
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const int ch = tid + (NC > 0 ? c : t) * nt;
            if (!AHEAD) {
              xv[c] = rv[c] = make_uint4(0, 0, 0, 0);
              if (ch < chunks) {
                xv[c] = load16(p.x, row * p.K + ch * 8);
                if (p.y) rv[c] = load16(p.y, row * p.K + ch * 8);
              }
            }
          }
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const int ch = tid + (NC > 0 ? c : t) * nt;
            hv[c] = xv[c];
            if (p.y) {
              hv[c] = add8<XDT>(xv[c], rv[c]);
              if (ch < chunks)
                *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.h) + row * p.K + ch * 8) = hv[c];
            }
            float h[8];
            h8_values<XDT>(hv[c], h);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fma((double)h[i], (double)h[i], s);
          }
        }
        if (AHEAD) read(row + gridDim.x);
        rstd = row_rstd(s, red, p);
        if (FMT == FMT_NVFP4 && tid == 0) p.rstd[row] = rstd;
      } else {
        rstd = p.rstd[row];
      }
      const float rs = (float)rstd;
      const bool rs_ok = rs >= 0x1p-100f && rs <= 0x1p100f;
#pragma unroll 1
      for (int t = 0; t < trips; ++t) {
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const int ch = tid + (NC > 0 ? c : t) * nt;
          const bool on = ch < chunks;
          if (NC == 0 || (FMT == FMT_NVFP4 && pass == 1))
            hv[c] = on ? load16(hsrc, row * p.K + ch * 8) : make_uint4(0, 0, 0, 0);
          if (!KEEP) get_gb(c, ch);
          float h[8];
          h8_values<XDT>(hv[c], h);
          f2 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = on ? mul2(mul2(pk(h[2 * i], h[2 * i + 1]), splat(rs)), pk(gb[c][2 * i], gb[c][2 * i + 1])) : 0ull;
          if (FMT == FMT_NVFP4 && pass == 0) {
            // values that are not finite have no share in the tensor scale
            if (on && rstd == rstd) {
              float mf = 0.f;
#pragma unroll
              for (int i = 0; i < 4; ++i) mf = max3_nan(mf, fabsf(lo_of(v[i])), fabsf(hi_of(v[i])));
              // fp64 only where the fp32 value could raise the maximum
              if (!((double)mf * (1.0 + 0x1p-18) < amax) || !rs_ok || (mf < 0x1p-60f && amax < 0x1p-59))
                amax = fmax(amax, amax_exact<XDT, false>(p, row, ch * 8, rstd));
            }
          } else {
            bad |= quant_store8<FMT, XDT, false>(p, row, ch * 8, on, v, 0x1p-20f, sT, isT, !sT_ok || !rs_ok, rstd);
          }
        }
      }
    }
  }
  if (blockIdx.x == 0 && tid == 0 && p.sT_out) *p.sT_out = sT;
  if (__any_sync(0xffffffffu, bad) && (tid & 31) == 0) atomicOr(&p.hdr->flags, kFlagNonFinite);
}

// ---------------------------------------------------------------------------
// dq_glu_quant: elementwise but for the groups, so the warps of the grid take
// items of 32 x 8 consecutive columns of a row, row-major and grid-stride, and
// read the next item while they work on one.

// x' in fp32: relative error below 10 * 2^-24 (expf within 2 ulp, six further
// roundings) while exp(-gate) and up * b stay in range; `far` marks the rest.
// (An up * b below fp32's normal range gives |x'| < 2^-86 here: a zero code in
// every group whose scale the fast path settles.)
template <int XDT>
__device__ __forceinline__ void glu_fast8(const uint4& gv, const uint4& uv, const float* b, f2* v, bool& far) {
  float g[8], u[8];
  h8_values<XDT>(gv, g);
  h8_values<XDT>(uv, u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float r[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float gg = g[2 * i + k], ub = u[2 * i + k] * b[2 * i + k];
      far |= !(gg >= -80.f && gg <= 0x1p40f) || !(fabsf(ub) <= kFltMax);
      r[k] = gg * __frcp_rn(1.f + expf(-gg)) * ub;
    }
    v[i] = pk(r[0], r[1]);
  }
}

template <int FMT, int XDT>
__global__ void __launch_bounds__(kGluThreads, 4) k_glu(const __grid_constant__ RowProblem p) {
  const int lane = threadIdx.x & 31;
  const int64_t spans = (p.K + 255) / 256;  // 256-column pieces of a row
  const int64_t w0 = (int64_t)blockIdx.x * (kGluThreads / 32) + (threadIdx.x >> 5);
  const int64_t nw = (int64_t)gridDim.x * (kGluThreads / 32);
  const int64_t drow = nw / spans, dspan = nw - drow * spans;  // the grid's stride as rows and spans
  double amax = 0.0;
  float sT = 1.f, isT = 1.f;
  bool sT_ok = true, bad = false;
#pragma unroll 1
  for (int pass = FMT == FMT_NVFP4 ? 0 : 1; pass < 2; ++pass) {
    if (FMT == FMT_NVFP4 && pass == 1) {
      amax_to_header(p.hdr, amax);
      row_grid_barrier(p.hdr);
      if (ld_volatile(&p.hdr->flags) & kFlagTimeout) return;
      sT = tensor_scale(*reinterpret_cast<volatile unsigned long long*>(&p.hdr->amax_scaled));
      isT = __frcp_rn(sT);
      sT_ok = in_range(isT);
    }
    int64_t row = w0 / spans, span = w0 - row * spans;
    uint4 gn, un;
    auto read = [&]() {
      const int64_t col = span * 256 + lane * 8;
      gn = un = make_uint4(0, 0, 0, 0);
      if (row < p.M && col < p.K) {
        gn = load16(p.x, row * p.ld + col);
        un = load16(p.y, row * p.ld + col);
      }
    };
    read();
#pragma unroll 1
    while (row < p.M) {
      const int64_t r = row, col = span * 256 + lane * 8;
      const bool on = col < p.K;
      const uint4 gv = gn, uv = un;
      row += drow;
      span += dspan;
      if (span >= spans) {
        span -= spans;
        ++row;
      }
      read();
      float b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = 0.f;
      if (on) b8_values(p, col, b);
      f2 v[4];
      bool far = false;
      glu_fast8<XDT>(gv, uv, b, v, far);
      if (FMT == FMT_NVFP4 && pass == 0) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max3_nan(m, fabsf(lo_of(v[i])), fabsf(hi_of(v[i])));
        // fp64 only where the fp32 value could raise the maximum; values that
        // are not finite have no share in it
        if (on && (far || !((double)m * (1.0 + 0x1p-18) < amax) || (m < 0x1p-60f && amax < 0x1p-59)))
          amax = fmax(amax, amax_exact<XDT, true>(p, r, col, 0.0));
      } else {
        bad |= quant_store8<FMT, XDT, true>(p, r, col, on, v, 0x1p-19f, sT, isT, !sT_ok || far, 0.0);
      }
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.sT_out) *p.sT_out = sT;
  if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&p.hdr->flags, kFlagNonFinite);
}

// ---------------------------------------------------------------------------
// Host side.

// One resident wave (the NVFP4 kernels wait for the whole grid: cooperative).
static cudaError_t row_launch(void (*kern)(RowProblem), const RowProblem& p, bool coop, int64_t want, int threads,
                              int sms, cudaStream_t st) {
  int per_sm = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, 0);
  if (e != cudaSuccess) return e;
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  const int64_t most = (int64_t)sms * per_sm;
  const int grid = (int)(want < most ? want : most);
  if (!coop) {
    kern<<<grid, threads, 0, st>>>(p);
    return cudaGetLastError();
  }
  RowProblem arg = p;
  void* args[] = {&arg};
  return cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kern), dim3(grid), dim3(threads), args, (size_t)0, st);
}

template <int FMT, int XDT>
static cudaError_t norm_launch(const RowProblem& p, int sms, cudaStream_t st) {
  const int64_t chunks = p.K / 8;
  const int nc = chunks <= 512 ? 1 : (chunks <= 1024 ? 2 : (chunks <= 4096 ? 4 : 0));
  const int64_t per = nc > 0 ? (chunks + nc - 1) / nc : 1024;
  const int threads = (int)((per + 31) / 32 * 32);
  void (*kern)(RowProblem) = nc == 1   ? k_norm<FMT, XDT, 1>
                             : nc == 2 ? k_norm<FMT, XDT, 2>
                             : nc == 4 ? k_norm<FMT, XDT, 4>
                                       : k_norm<FMT, XDT, 0>;
  return row_launch(kern, p, FMT == FMT_NVFP4, p.M, threads, sms, st);
}

template <int FMT, int XDT>
static cudaError_t glu_launch(const RowProblem& p, int sms, cudaStream_t st) {
  const int64_t items = p.M * ((p.K + 255) / 256);
  return row_launch(k_glu<FMT, XDT>, p, FMT == FMT_NVFP4, (items + 7) / 8, kGluThreads, sms, st);
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
  if (rows > ((int64_t)1 << 40) / cols) return DQ_EUNSUPPORTED;
  if ((uintptr_t)col_scales % 2 != 0) return DQ_EINVAL;
  if (!out || !out->codes || !out->block_scales || (uintptr_t)out->codes % 8 != 0 ||
      (format == DQ_NVFP4 && !out->tensor_scale) || (uintptr_t)out->tensor_scale % 4 != 0)
    return DQ_EINVAL;
  if (!workspace || (uintptr_t)workspace % 256 != 0) return DQ_EINVAL;
  return DQ_OK;
}

static int row_sms(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DQ_ECUDA;
  return cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? DQ_OK : DQ_ECUDA;
}

static void row_fill(RowProblem* p, int64_t rows, int64_t cols, const void* col_scales, int col_dtype, int group,
                     const dq_outputs* out, void* workspace) {
  p->b_store = col_scales;
  p->col_dt = col_dtype;
  p->b_vec = col_scales != nullptr && (uintptr_t)col_scales % 16 == 0;
  p->M = rows;
  p->K = cols;
  p->codes = static_cast<unsigned char*>(out->codes);
  p->scales = static_cast<unsigned char*>(out->block_scales);
  p->nb = cols / group;
  p->sT_out = out->tensor_scale;
  p->hdr = static_cast<WsHeader*>(workspace);
}

}  // namespace dq

extern "C" size_t dq_norm_workspace_bytes(int64_t rows, int64_t cols, int format, int group) {
  if (rows <= 0 || cols <= 0 || group <= 0 || cols % group != 0 || rows > ((int64_t)1 << 40) / cols) return 0;
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
  if (workspace_bytes < dq_norm_workspace_bytes(rows, cols, format, group)) return DQ_EWORKSPACE;
  int sms = 0;
  if ((st = dq::row_sms(&sms)) != DQ_OK) return st;
  dq::RowProblem p{};
  dq::row_fill(&p, rows, cols, col_scales, col_dtype, group, out, workspace);
  p.x = X;
  p.y = residual;
  p.g = weight;
  p.ld = cols;
  p.eps = eps;
  p.h = residual_out;
  p.rstd = reinterpret_cast<double*>(static_cast<unsigned char*>(workspace) + DQ_ACT_WORKSPACE_BYTES);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, sizeof(dq::WsHeader), s) != cudaSuccess) return DQ_ECUDA;
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
  if (workspace_bytes < DQ_ACT_WORKSPACE_BYTES) return DQ_EWORKSPACE;
  int sms = 0;
  if ((st = dq::row_sms(&sms)) != DQ_OK) return st;
  dq::RowProblem p{};
  dq::row_fill(&p, rows, cols, col_scales, col_dtype, group, out, workspace);
  p.x = gate;
  p.y = up;
  p.ld = ld;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, sizeof(dq::WsHeader), s) != cudaSuccess) return DQ_ECUDA;
  cudaError_t e;
  if (format == DQ_NVFP4)
    e = x_dtype == DQ_BF16 ? dq::glu_launch<dq::FMT_NVFP4, dq::DT_BF16>(p, sms, s) : dq::glu_launch<dq::FMT_NVFP4, dq::DT_F16>(p, sms, s);
  else if (format == DQ_MXFP4)
    e = x_dtype == DQ_BF16 ? dq::glu_launch<dq::FMT_MXFP4, dq::DT_BF16>(p, sms, s) : dq::glu_launch<dq::FMT_MXFP4, dq::DT_F16>(p, sms, s);
  else
    e = x_dtype == DQ_BF16 ? dq::glu_launch<dq::FMT_MXFP8, dq::DT_BF16>(p, sms, s) : dq::glu_launch<dq::FMT_MXFP8, dq::DT_F16>(p, sms, s);
  return e == cudaSuccess ? DQ_OK : DQ_ECUDA;
}

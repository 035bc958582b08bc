// dq_matmul.cu -- the product of quantized activations and a quantized weight
// matrix, both microscaled in the same format:
//
//   Y[t][n] = s_x s_w sum_k (a_x[t][k/G] q_x[t][k]) (a_w[n][k/G] q_w[n][k])
//
// (DualQuant arXiv 2610.13767 summary, section 4.4: X W^T = (X D_b) Q^T D_a;
// the column scales b are in q_x already).  Sums are held in fp32 and rounded
// once, after the tensor scales, to the output type.
#include <climits>

#include "dq.h"
#include "dq_device.cuh"
#include "dq_fast.cuh"
#include "dq_internal.h"

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
  WsHeader* hdr;
};

// The tensor scales' product as f1 * f2, applied one after the other: f2 is 1
// unless the product leaves fp32's normal range.
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
    f2 = (float)scalbn(s, -e);
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
// products (exact: 16 products of at most 18 significant bits) is multiplied
// by the two block scales at once; powers of two add their exponents, so that
// scales at the ends of their range do not overflow on the way.  Bound by
// fp32 arithmetic and the decoding.
template <int FMT>
__global__ void __launch_bounds__(256) k_matmul_any(MatmulProblem p) {
  constexpr int G = FMT == FMT_NVFP4 ? 16 : 32;
  __shared__ float xs[16][68], ws[16][68];
  __shared__ unsigned char xa[64], wa[64];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int64_t tiles_n = (p.N + 63) / 64, nb = p.K / G;
  const int64_t t0 = blockIdx.x / tiles_n * 64, n0 = blockIdx.x % tiles_n * 64;
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

template <int FMT>
static cudaError_t matmul_any(const MatmulProblem& p, cudaStream_t st) {
  const int64_t tiles = (p.T + 63) / 64 * ((p.N + 63) / 64);
  k_matmul_any<FMT><<<(unsigned)tiles, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace dq

extern "C" int dq_matmul(const dq_outputs* X, int64_t tokens, const dq_outputs* W, int64_t rows, int64_t cols, int format,
                         int group, void* Y, int y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (tokens <= 0 || rows <= 0 || cols <= 0 || group <= 0 || cols % group != 0) return DQ_EINVAL;
  if (format < DQ_INT4 || format > DQ_MXFP8) return DQ_EINVAL;
  if (format != DQ_NVFP4 && format != DQ_MXFP4 && format != DQ_MXFP8) return DQ_EUNSUPPORTED;
  if (group != (format == DQ_NVFP4 ? 16 : 32)) return DQ_EUNSUPPORTED;
  if (y_dtype < DQ_F32 || y_dtype > DQ_F16) return DQ_EINVAL;
  if (tokens > INT_MAX - 256 || rows > INT_MAX - 256 || cols > INT_MAX - 256) return DQ_EUNSUPPORTED;
  if ((tokens + 63) / 64 * ((rows + 63) / 64) > INT_MAX) return DQ_EUNSUPPORTED;
  if (!X || !W || !X->codes || !X->block_scales || !W->codes || !W->block_scales || !Y) return DQ_EINVAL;
  if (format == DQ_NVFP4 && (!X->tensor_scale || !W->tensor_scale || (uintptr_t)X->tensor_scale % 4 != 0 ||
                             (uintptr_t)W->tensor_scale % 4 != 0))
    return DQ_EINVAL;
  if ((uintptr_t)Y % (y_dtype == DQ_F32 ? 4 : 2) != 0) return DQ_EINVAL;
  if (!workspace || (uintptr_t)workspace % 256 != 0) return DQ_EINVAL;
  if (workspace_bytes < DQ_MATMUL_WORKSPACE_BYTES) return DQ_EWORKSPACE;
  dq::MatmulProblem p{};
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
  p.hdr = static_cast<dq::WsHeader*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, sizeof(dq::WsHeader), s) != cudaSuccess) return DQ_ECUDA;
  const cudaError_t e = format == DQ_NVFP4   ? dq::matmul_any<dq::FMT_NVFP4>(p, s)
                        : format == DQ_MXFP4 ? dq::matmul_any<dq::FMT_MXFP4>(p, s)
                                             : dq::matmul_any<dq::FMT_MXFP8>(p, s);
  return e == cudaSuccess ? DQ_OK : DQ_ECUDA;
}

// mxfp4_gemm.cu -- products with MXFP4 weights: y[m][n] = sum_k x[m][k] w[n][k]
// (+ bias[n]) (+ residual[m][n]), and silu(x g^T) * (x u^T); x is fp16, or MXFP4
// like the weights.  Weights are fp16 numbers exactly, sums fp32, one rounding to
// fp16 at the end (SiLU's two sums are not rounded before it).
#include <algorithm>

#include "mxfp4.cuh"
#include "kernels.h"

namespace w4 {

constexpr int MXS_N = 64, MXS_M = 64, MXS_K = 32;

// 8 values of row r, elements k .. k + 7, into column r of t[k][r]
__device__ __forceinline__ void mxs_unpack(float (*t)[MXS_N + 1], int col, int kl, uint32_t code, float s) {
  const uint4 v = mx_values(code);
  const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    t[kl + 2 * j][col] = f.x * s;
    t[kl + 2 * j + 1][col] = f.y * s;
  }
}
__device__ __forceinline__ uint32_t mxs_word(const MxWeights& w, int r, int rows, int k, int K, float* s) {
  *s = 0.f;
  if (r >= rows) return 0u;
  *s = mx_scale(w.scales[mx_scale_at(r, k >> 7, K >> 7) + ((k >> 5) & 3)]);
  return w.codes[(size_t)r * (K / 8) + (k >> 3)];
}

// 64 x 64 outputs a CTA of 256 threads, 4 x 4 a thread
template <bool SILU>
__global__ void __launch_bounds__(256) w4pg_mxfp4_tile(const MxArgs a) {
  pdl_wait_then_trigger();
  constexpr int NW = SILU ? 2 : 1;
  __shared__ float ws[NW][MXS_K][MXS_N + 1], xs[MXS_K][MXS_M + 1];
  const int n0 = blockIdx.x * MXS_N, m0 = blockIdx.y * MXS_M, K = a.K;
  const int tid = threadIdx.x, tn = (tid & 15) * 4, tm = (tid >> 4) * 4;
  const int col = tid >> 2, kl = (tid & 3) * 8;  // loads: a row, 8 elements
  float acc[NW][4][4] = {};
  for (int k0 = 0; k0 < K; k0 += MXS_K) {
    float s;
#pragma unroll
    for (int g = 0; g < NW; ++g) {
      const uint32_t c = mxs_word(a.w[g], n0 + col, a.N, k0 + kl, K, &s);
      if (a.x != nullptr) s = __half2float(__float2half_rn(s));  // beside fp16 x, weights are fp16 numbers
      mxs_unpack(ws[g], col, kl, c, s);
    }
    if (a.x == nullptr) {
      const uint32_t c = mxs_word(a.xq, m0 + col, a.M, k0 + kl, K, &s);
      mxs_unpack(xs, col, kl, c, s);
    } else {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (m0 + col < a.M) v = *reinterpret_cast<const uint4*>(a.x + (size_t)(m0 + col) * K + k0 + kl);
      const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
        xs[kl + 2 * j][col] = f.x;
        xs[kl + 2 * j + 1][col] = f.y;
      }
    }
    __syncthreads();
#pragma unroll 4
    for (int k = 0; k < MXS_K; ++k) {
      float xv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) xv[j] = xs[k][tm + j];
#pragma unroll
      for (int g = 0; g < NW; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float wv = ws[g][k][tn + i];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[g][i][j] = fmaf(wv, xv[j], acc[g][i][j]);
        }
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int m = m0 + tm + j;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + tn + i;
      if (m >= a.M || n >= a.N) continue;
      float v = acc[0][i][j];
      if (SILU) v = v / (1.f + expf(-v)) * acc[NW - 1][i][j];
      if (a.bias) v += __half2float(a.bias[n]);
      if (a.residual) v += __half2float(a.residual[(size_t)m * a.N + n]);
      a.y[(size_t)m * a.N + n] = __float2half_rn(v);
    }
  }
}

static int launch_mxfp4(const MxArgs& a, bool silu, cudaStream_t s) {
  if (a.x && mxfp4_matvec_serves(a.M, a.K)) return launch_mxfp4_matvec(a, silu, s);
  if (a.x) return launch_mxfp4_a16(a, silu, s);
  const dim3 grid((a.N + MXS_N - 1) / MXS_N, (a.M + MXS_M - 1) / MXS_M);
  const cudaError_t e = silu ? launch_pdl(w4pg_mxfp4_tile<true>, grid, dim3(256), 0, s, a)
                             : launch_pdl(w4pg_mxfp4_tile<false>, grid, dim3(256), 0, s, a);
  if (e != cudaSuccess) return set_error(W4A16_ERR_CUDA, "mxfp4 product launch: %s", cudaGetErrorString(e));
  return W4A16_OK;
}

}  // namespace w4

// ---------------------------------------------------------------------------
// C ABI
// ---------------------------------------------------------------------------
using namespace w4;

static int mx_product_checks(const char* what, const MxArgs& a) {
  W4_CHECK_ARG(a.y, "%s: null y", what);
  W4_CHECK_ARG(a.M >= 1 && a.N >= 1 && a.K >= 1, "%s: sizes must be positive", what);
  W4_CHECK_SHAPE(a.K % 128 == 0, "%s: K=%d must be a multiple of 128", what, a.K);
  W4_CHECK_SHAPE(a.K <= W4A16_MXFP4_MAX_K, "%s: K=%d > %d", what, a.K, W4A16_MXFP4_MAX_K);
  W4_CHECK_SHAPE(a.M <= W4A16_MXFP4_MAX_ROWS && a.N <= W4A16_MXFP4_MAX_ROWS, "%s: M=%d N=%d > %d", what, a.M, a.N,
                 W4A16_MXFP4_MAX_ROWS);
  W4_CHECK_ALIGN(a.x, 128, "x");
  W4_CHECK_ALIGN(a.xq.codes, 128, "x_codes");
  W4_CHECK_ALIGN(a.xq.scales, 128, "x_scales");
  for (const MxWeights& w : a.w) {
    W4_CHECK_ALIGN(w.codes, 128, "codes");
    W4_CHECK_ALIGN(w.scales, 128, "scales");
  }
  W4_CHECK_ALIGN(a.bias, 128, "bias");
  W4_CHECK_ALIGN(a.residual, 128, "residual");
  W4_CHECK_ALIGN(a.y, 128, "y");
  W4_CHECK_ALIGN(a.workspace, 128, "workspace");
  return W4A16_OK;
}

extern "C" size_t w4a16_gemm_mxfp4_workspace_size(int M, int K, int N, int silu) {
  if (M < 1 || K < 128 || N < 1) return 0;
  return mxfp4_matvec_serves(M, K) ? 256 : mxfp4_a16_workspace(M, N, K, silu != 0);
}
extern "C" size_t w4a4_gemm_mxfp4_workspace_size(int M, int K, int N) { return 256; }

extern "C" int w4a16_gemm_mxfp4(const uint16_t* x, int M, int K, const uint32_t* codes, const uint8_t* scales, int N,
                                const uint16_t* bias, const uint16_t* residual, uint16_t* y, void* workspace,
                                size_t workspace_bytes, int32_t* err_flag, w4a16_stream_t stream) {
  W4_CHECK_ARG(x && codes && scales, "w4a16_gemm_mxfp4: null pointer");
  MxArgs a = {};
  a.x = reinterpret_cast<const __half*>(x);
  a.w[0] = {codes, scales};
  a.bias = reinterpret_cast<const __half*>(bias);
  a.residual = reinterpret_cast<const __half*>(residual);
  a.y = reinterpret_cast<__half*>(y);
  a.M = M;
  a.N = N;
  a.K = K;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  a.err_flag = err_flag;
  if (const int rc = mx_product_checks("w4a16_gemm_mxfp4", a)) return rc;
  return launch_mxfp4(a, false, (cudaStream_t)stream);
}

extern "C" int w4a16_gemm_silu_mul_mxfp4(const uint16_t* x, int M, int K, const uint32_t* codes_gate,
                                         const uint8_t* scales_gate, const uint32_t* codes_up,
                                         const uint8_t* scales_up, int N, uint16_t* y, void* workspace,
                                         size_t workspace_bytes, int32_t* err_flag, w4a16_stream_t stream) {
  W4_CHECK_ARG(x && codes_gate && scales_gate && codes_up && scales_up, "w4a16_gemm_silu_mul_mxfp4: null pointer");
  MxArgs a = {};
  a.x = reinterpret_cast<const __half*>(x);
  a.w[0] = {codes_gate, scales_gate};
  a.w[1] = {codes_up, scales_up};
  a.y = reinterpret_cast<__half*>(y);
  a.M = M;
  a.N = N;
  a.K = K;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  a.err_flag = err_flag;
  if (const int rc = mx_product_checks("w4a16_gemm_silu_mul_mxfp4", a)) return rc;
  return launch_mxfp4(a, true, (cudaStream_t)stream);
}

extern "C" int w4a4_gemm_mxfp4(const uint32_t* x_codes, const uint8_t* x_scales, int M, int K, const uint32_t* codes,
                               const uint8_t* scales, int N, const uint16_t* bias, const uint16_t* residual,
                               uint16_t* y, void* workspace, size_t workspace_bytes, int32_t* err_flag,
                               w4a16_stream_t stream) {
  W4_CHECK_ARG(x_codes && x_scales && codes && scales, "w4a4_gemm_mxfp4: null pointer");
  MxArgs a = {};
  a.xq = {x_codes, x_scales};
  a.w[0] = {codes, scales};
  a.bias = reinterpret_cast<const __half*>(bias);
  a.residual = reinterpret_cast<const __half*>(residual);
  a.y = reinterpret_cast<__half*>(y);
  a.M = M;
  a.N = N;
  a.K = K;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  a.err_flag = err_flag;
  if (const int rc = mx_product_checks("w4a4_gemm_mxfp4", a)) return rc;
  return launch_mxfp4(a, false, (cudaStream_t)stream);
}

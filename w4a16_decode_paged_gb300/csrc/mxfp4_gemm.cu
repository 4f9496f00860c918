// mxfp4_gemm.cu -- products with MXFP4 weights: y[m][n] = sum_k x[m][k] w[n][k]
// (+ bias[n]) (+ residual[m][n]), and silu(x g^T) * (x u^T); x is fp16, or MXFP4
// like the weights.  Weights are fp16 numbers exactly, sums fp32, one rounding to
// fp16 at the end (SiLU's two sums are not rounded before it).
#include <algorithm>

#include "mxfp4.cuh"
#include "kernels.h"

namespace w4 {

static int launch_mxfp4(const MxArgs& a, bool silu, cudaStream_t s) {
  if (a.x == nullptr) return launch_mxfp4_a4(a, s);
  if (mxfp4_matvec_serves(a.M, a.K)) return launch_mxfp4_matvec(a, silu, s);
  return launch_mxfp4_a16(a, silu, s);
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
extern "C" size_t w4a4_gemm_mxfp4_workspace_size(int M, int K, int N) {
  return M < 1 || K < 128 || N < 1 ? 0 : mxfp4_a4_workspace(M, N, K);
}

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

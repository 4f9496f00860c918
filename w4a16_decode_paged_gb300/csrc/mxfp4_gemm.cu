// mxfp4_gemm.cu -- products with MXFP4 weights: y[m][n] = sum_k x[m][k] w[n][k]
// (+ bias[n]) (+ residual[m][n]), and silu(x g^T) * (x u^T); x is fp16, or MXFP4
// like the weights.  Weights are fp16 numbers exactly, sums fp32, one rounding to
// fp16 at the end (SiLU's two sums are not rounded before it).
#include <algorithm>

#include "mxfp4_tc.cuh"

namespace w4 {

// The sums of tiles that were split along K: a thread adds the parts of four
// neighbouring outputs, in order.
__global__ void __launch_bounds__(256) w4pg_mxfp4_join(const __grid_constant__ MtJoin j) {
  pdl_wait_then_trigger();
  const int width = (j.silu ? 128 : j.tn) / 4;     // threads along a row
  const int i = blockIdx.x * 256 + threadIdx.x, c = i % width * 4, row = i / width % j.tm, t = i / width / j.tm;
  if (t >= j.tiles) return;
  const int tile = j.first + t, m = tile % j.mtiles * j.tm + row, n = tile / j.mtiles * j.tstep + c;
  if (m >= j.a.M || n >= j.a.N) return;
  const size_t part = (size_t)j.tm * j.tn;
  const float* p = j.parts + (size_t)t * j.split * part + (size_t)row * j.tn + c;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f), u = v;
#pragma unroll 8
  for (int q = 0; q < j.split; ++q) {
    const float4 w = __ldcg(reinterpret_cast<const float4*>(p + q * part));
    v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    if (j.silu) {
      const float4 z = __ldcg(reinterpret_cast<const float4*>(p + q * part + 128));
      u.x += z.x, u.y += z.y, u.z += z.z, u.w += z.w;
    }
  }
  float o[4] = {v.x, v.y, v.z, v.w};
  const float up[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (n + k >= j.a.N) break;
    const size_t at = (size_t)m * j.a.N + n + k;
    if (j.silu) o[k] = o[k] / (1.f + expf(-o[k])) * up[k];
    if (j.a.bias) o[k] += __half2float(j.a.bias[n + k]);
    if (j.a.residual) o[k] += __half2float(j.a.residual[at]);
    j.a.y[at] = __float2half_rn(o[k]);
  }
}

int launch_mxfp4_join(const MtJoin& j, cudaStream_t s) {
  const long long threads = (long long)j.tiles * j.tm * (j.silu ? 128 : j.tn) / 4;
  const cudaError_t e = launch_pdl(w4pg_mxfp4_join, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, j);
  if (e != cudaSuccess) return set_error(W4A16_ERR_CUDA, "mxfp4 join launch: %s", cudaGetErrorString(e));
  return W4A16_OK;
}

static int launch_mxfp4(const MxArgs& a, bool silu, cudaStream_t s) {
  if (a.x == nullptr) return launch_mxfp4_a4(a, s);
  if (mxfp4_matvec_serves(a.M, a.N, a.K, silu)) return launch_mxfp4_matvec(a, silu, s);
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
  return mxfp4_matvec_serves(M, N, K, silu != 0) ? 256 : mxfp4_a16_workspace(M, N, K, silu != 0);
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

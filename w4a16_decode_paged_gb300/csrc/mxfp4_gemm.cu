// mxfp4_gemm.cu -- products with MXFP4 weights: y[m][n] = sum_k x[m][k] w[n][k]
// (+ bias[n]) (+ residual[m][n]), and silu(x g^T) * (x u^T); x is fp16, or MXFP4
// like the weights.  Weights are fp16 numbers exactly, sums fp32, one rounding to
// fp16 at the end (SiLU's two sums are not rounded before it).
#include <algorithm>

#include "mxfp4_tc.cuh"

namespace w4 {

// The sums of tiles that were split along K: a thread adds, in order, the parts of
// four neighbouring outputs in each of R rows; R times MJ_LOADS / R parts are asked
// for at once, so that few parts (a prompt's tiles) and many (a decode batch's) both
// keep eight loads in flight.  (One row a thread, only its own
// parts in flight: 2048 rows, 3584 x 3584
// 53.9 us, so 50.9; 32 rows, 512 x 3584 9.1 us, so 6.6.)
constexpr int MJ_LOADS = 8;

template <bool SILU, int R>
__global__ void __launch_bounds__(256) w4pg_mxfp4_join(const __grid_constant__ MtJoin j) {
  constexpr int AHEAD = MJ_LOADS / R;
  pdl_wait_then_trigger();
  const int width = (SILU ? 128 : j.tn) / 4;       // threads along a row
  const int i = blockIdx.x * 256 + threadIdx.x, row0 = i / width, c = (i - row0 * width) * 4, rstep = j.tm / R;
  const int tile = j.first + blockIdx.y, nt = tile / j.mtiles, n = nt * j.tstep + c;
  const int N = j.a.N, m0 = (tile - nt * j.mtiles) * j.tm + row0;
  if (row0 >= rstep || n >= N) return;
  const size_t part = (size_t)j.tm * j.tn / 4;
  const float4* p = reinterpret_cast<const float4*>(j.parts) + (size_t)blockIdx.y * j.split * part + (row0 * j.tn + c) / 4;
  const bool wide = N % 4 == 0;                    // four outputs lie on 8 bytes
  uint2 res[R];
  if (wide && j.a.residual) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (m0 + r * rstep < j.a.M) res[r] = *reinterpret_cast<const uint2*>(j.a.residual + (size_t)(m0 + r * rstep) * N + n);
  }
  auto sums = [&](float (&v)[R][4], const float4* p) {
#pragma unroll
    for (int r = 0; r < R; ++r) v[r][0] = v[r][1] = v[r][2] = v[r][3] = 0.f;
    for (int q = 0; q < j.split; q += AHEAD) {
      float4 a[R][AHEAD];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
          if (q + k < j.split && m0 + r * rstep < j.a.M) a[r][k] = __ldcg(p + (q + k) * part + (size_t)r * rstep * j.tn / 4);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
          if (q + k < j.split) v[r][0] += a[r][k].x, v[r][1] += a[r][k].y, v[r][2] += a[r][k].z, v[r][3] += a[r][k].w;
    }
  };
  float v[R][4];
  sums(v, p);
  if (SILU) {
    float u[R][4];
    sums(u, p + 32);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[r][k] = v[r][k] / (1.f + expf(-v[r][k])) * u[r][k];
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int m = m0 + r * rstep;
    if (m >= j.a.M) break;
    const size_t at = (size_t)m * N + n;
    if (wide && j.a.residual) {
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&res[r].x)), b = __half22float2(*reinterpret_cast<const __half2*>(&res[r].y));
      v[r][0] += a.x, v[r][1] += a.y, v[r][2] += b.x, v[r][3] += b.y;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (n + k >= N) break;
      if (j.a.bias) v[r][k] += __half2float(j.a.bias[n + k]);
      if (!wide) {
        if (j.a.residual) v[r][k] += __half2float(j.a.residual[at + k]);
        j.a.y[at + k] = __float2half_rn(v[r][k]);
      }
    }
    if (wide) {
      const __half2 h[2] = {__floats2half2_rn(v[r][0], v[r][1]), __floats2half2_rn(v[r][2], v[r][3])};
      *reinterpret_cast<uint2*>(j.a.y + at) = *reinterpret_cast<const uint2*>(h);
    }
  }
}

template <bool SILU, int R>
static cudaError_t mj_launch(const MtJoin& j, cudaStream_t s) {
  const dim3 grid((unsigned)((j.tm / R * (SILU ? 128 : j.tn) / 4 + 255) / 256), (unsigned)j.tiles);
  return launch_pdl(w4pg_mxfp4_join<SILU, R>, grid, dim3(256), 0, s, j);
}

int launch_mxfp4_join(const MtJoin& j, cudaStream_t s) {
  // four parts and fewer: several rows a thread
  cudaError_t e;
  if (j.silu) e = j.split > 4 ? mj_launch<true, 1>(j, s) : j.split > 2 ? mj_launch<true, 2>(j, s) : mj_launch<true, 4>(j, s);
  else e = j.split > 4 ? mj_launch<false, 1>(j, s) : j.split > 2 ? mj_launch<false, 2>(j, s) : mj_launch<false, 4>(j, s);
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
  return mxfp4_matvec_serves(M, N, K, silu != 0) ? 0 : mxfp4_a16_workspace(M, N, K, silu != 0);
}
extern "C" size_t w4a4_gemm_mxfp4_workspace_size(int M, int K, int N) {
  return M < 1 || K < 128 || N < 1 ? 0 : mxfp4_a4_workspace(M, N, K);
}

extern "C" size_t mxfp4_workspace_size(void) {
  // a deal has at most as many parts as there are CTAs (mt_deal)
  return TC_TICKET_BYTES + (size_t)ATW_SMS * std::max(mxfp4_a16_largest_tile(), mxfp4_a4_largest_tile()) * 4;
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

extern "C" int w4a16_debug_mxfp4_plan(int kind, int M, int K, int N, size_t workspace_bytes, int sms, int32_t* plan) {
  W4_CHECK_ARG(plan && kind >= 0 && kind <= 2 && sms >= 0, "w4a16_debug_mxfp4_plan: arguments");
  W4_CHECK_SHAPE(M >= 1 && M <= W4A16_MXFP4_MAX_ROWS && N >= 1 && N <= W4A16_MXFP4_MAX_ROWS && K >= 128 && K % 128 == 0 &&
                     K <= W4A16_MXFP4_MAX_K,
                 "w4a16_debug_mxfp4_plan: M=%d N=%d K=%d", M, N, K);
  const int slots = sms ? sms : num_sms();
  if (kind == 2) mxfp4_a4_plan(M, N, K, workspace_bytes, slots, plan);
  else if (mxfp4_matvec_serves(M, N, K, kind == 1)) mxfp4_matvec_plan(M, N, K, kind == 1, plan);
  else mxfp4_a16_plan(M, N, K, kind == 1, workspace_bytes, slots, plan);
  return W4A16_OK;
}

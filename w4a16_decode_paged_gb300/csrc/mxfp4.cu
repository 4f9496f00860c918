// mxfp4.cu -- MXFP4 matrices: quantising fp16 rows, reading them back, and the
// C ABI of the products (kernels in mxfp4_*.cu).
//
// Quantising, per 32 consecutive elements: a = max |x|, e = floor(log2 a) - 2
// (so that a 2^-e is in [4, 8); the microscaling format's rule), at least -23;
// code = x 2^-e (exact) rounded to the nearest E2M1 number, ties to even, 6 at
// most; scale byte e + 127.  With e >= -23 the least code step, 2^(e-1), is a
// multiple of fp16's 2^-24, and with fp16 input e <= 13, so every value read
// back is an fp16 number exactly.  An infinity or a NaN among the 32: byte 255,
// codes 0.
#include <algorithm>

#include "mxfp4.cuh"
#include "kernels.h"

namespace w4 {

// Both kernels: 16 lanes have 128 elements of a row (a scale tile's width), 8
// each; a CTA of 256 threads has `kx` (a power of two) such units along K and
// 16 / kx rows, MXQ_ROWS times over, all loads ahead of the first use.
// 2048 x 18944, 98 MB each way: quantised in 18.5 us (5.3 TB/s, 0.80 of a plain copy), read
// back in 17.0 (5.8), each in a row of such calls; one behind the other 31.7, as the codes
// are still in L2.  In the quantiser the warps issue at 0.71 of the slots and the integer
// pipe is at 0.67 (reader: 0.71, 0.53), so that memory and instructions are near one
// another.  A row of 3584 takes 1.25 and 1.0 us, the launch.
constexpr int MXQ_ROWS = 4;
constexpr int MXQ_THREADS = 256;

struct MxqPlace {
  int kt, row, rstep;
  bool live;
};
__device__ __forceinline__ MxqPlace mxq_place(int K, int kx_log2) {
  const int u = threadIdx.x >> 4, ry = (MXQ_THREADS / 16) >> kx_log2;
  MxqPlace p;
  p.kt = (blockIdx.y << kx_log2) + (u & ((1 << kx_log2) - 1));
  p.row = blockIdx.x * (ry * MXQ_ROWS) + (u >> kx_log2);
  p.rstep = ry;
  p.live = p.kt < K / 128;
  return p;
}

__global__ void __launch_bounds__(MXQ_THREADS)
    w4pg_mxfp4_quantize(const __half* __restrict__ x, uint32_t* __restrict__ codes, uint8_t* __restrict__ scales, int M,
                        int K, int kx_log2) {
  pdl_wait_then_trigger();
  const MxqPlace p = mxq_place(K, kx_log2);
  const int lane = threadIdx.x & 15;
  uint4 v[MXQ_ROWS];
#pragma unroll
  for (int i = 0; i < MXQ_ROWS; ++i) {
    const int r = p.row + i * p.rstep;
    v[i] = make_uint4(0, 0, 0, 0);
    if (p.live && r < M) v[i] = ldg_stream(x + (size_t)r * K + p.kt * 128 + lane * 8);
  }
#pragma unroll
  for (int i = 0; i < MXQ_ROWS; ++i) {
    const int r = p.row + i * p.rstep;
    // the largest magnitude of 32 elements: fp16 magnitudes order as integers
    const uint32_t a0 = __vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu);
    const uint32_t a1 = __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu);
    uint32_t a = __vmaxu2(a0, a1);
    a = max(a & 0xFFFFu, a >> 16);
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    const bool bad = a >= 0x7C00u;
    // floor(log2 a) is the fp32 exponent (fp16's subnormals are normal there)
    const uint32_t ex = __float_as_uint(__half2float(__ushort_as_half((unsigned short)a))) >> 23;
    const uint32_t byte = max((int)ex - 2, MX_MIN_BYTE);
    const float inv = __uint_as_float((254u - byte) << 23);
    uint32_t w = 0;
    const uint32_t h[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      uint32_t q;  // two codes, the first in the low nibble
      asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
          : "=r"(q)
          : "f"(f.y * inv), "f"(f.x * inv));
      w |= q << (8 * j);
    }
    // the four scale bytes of the unit, from lanes 0, 4, 8, 12
    uint32_t s = bad ? 255u : byte;
    s |= __shfl_down_sync(0xffffffffu, s, 4, 16) << 8;
    s |= __shfl_down_sync(0xffffffffu, s, 8, 16) << 16;
    if (p.live && r < M) {
      codes[(size_t)r * (K / 8) + p.kt * 16 + lane] = bad ? 0u : w;
      if (lane == 0) *reinterpret_cast<uint32_t*>(scales + mx_scale_at(r, p.kt, K / 128)) = s;
    }
  }
}

__global__ void __launch_bounds__(MXQ_THREADS)
    w4pg_mxfp4_dequantize(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                          __half* __restrict__ y, int M, int K, int kx_log2) {
  pdl_wait_then_trigger();
  const MxqPlace p = mxq_place(K, kx_log2);
  const int lane = threadIdx.x & 15;
  uint32_t w[MXQ_ROWS], s[MXQ_ROWS];
#pragma unroll
  for (int i = 0; i < MXQ_ROWS; ++i) {
    const int r = p.row + i * p.rstep;
    w[i] = s[i] = 0;
    if (p.live && r < M) {
      w[i] = codes[(size_t)r * (K / 8) + p.kt * 16 + lane];
      s[i] = scales[mx_scale_at(r, p.kt, K / 128) + (lane >> 2)];
    }
  }
#pragma unroll
  for (int i = 0; i < MXQ_ROWS; ++i) {
    const int r = p.row + i * p.rstep;
    if (!p.live || r >= M) continue;
    // in fp32, so that any scale byte is served: one rounding to fp16
    const float sc = mx_scale(s[i]);
    const uint4 c = mx_values(w[i]);
    const uint32_t h[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      const __half2 g = __floats2half2_rn(f.x * sc, f.y * sc);
      o[j] = *reinterpret_cast<const uint32_t*>(&g);
    }
    *reinterpret_cast<uint4*>(y + (size_t)r * K + p.kt * 128 + lane * 8) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// units along K per CTA: as many as leave the fewest idle
static int mxq_kx_log2(int ktiles) {
  int best = 0, waste = 1 << 30;
  for (int l = 4; l >= 0; --l) {
    const int w = ((ktiles + (1 << l) - 1) >> l << l) - ktiles;
    if (w < waste) {
      waste = w;
      best = l;
    }
  }
  return best;
}

template <class Kern, class... Args>
static int launch_mxq(const char* what, Kern kern, int M, int K, cudaStream_t s, Args... args) {
  const int kx = mxq_kx_log2(K / 128), rows = ((MXQ_THREADS / 16) >> kx) * MXQ_ROWS;
  const dim3 grid((M + rows - 1) / rows, (K / 128 + (1 << kx) - 1) >> kx);
  const cudaError_t e = launch_pdl(kern, grid, dim3(MXQ_THREADS), 0, s, args..., M, K, kx);
  if (e != cudaSuccess) return set_error(W4A16_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
  return W4A16_OK;
}

}  // namespace w4

// ---------------------------------------------------------------------------
// C ABI
// ---------------------------------------------------------------------------
using namespace w4;

static int mx_matrix_checks(const char* what, int rows, int K) {
  W4_CHECK_ARG(rows >= 1 && K >= 1, "%s: sizes must be positive", what);
  W4_CHECK_SHAPE(K % 128 == 0, "%s: K=%d must be a multiple of 128", what, K);
  W4_CHECK_SHAPE(K <= W4A16_MXFP4_MAX_K, "%s: K=%d > %d", what, K, W4A16_MXFP4_MAX_K);
  W4_CHECK_SHAPE(rows <= W4A16_MXFP4_MAX_ROWS, "%s: %d rows > %d", what, rows, W4A16_MXFP4_MAX_ROWS);
  return W4A16_OK;
}

extern "C" size_t mxfp4_scales_size(int rows, int K) {
  return rows < 1 || K < 128 || K % 128 ? 0 : mx_tiles(rows, K) * MX_TILE;
}

extern "C" int mxfp4_quantize(const uint16_t* x, int M, int K, uint32_t* codes, uint8_t* scales,
                              w4a16_stream_t stream) {
  W4_CHECK_ARG(x && codes && scales, "mxfp4_quantize: null pointer");
  if (const int rc = mx_matrix_checks("mxfp4_quantize", M, K)) return rc;
  W4_CHECK_ALIGN(x, 128, "x");
  W4_CHECK_ALIGN(codes, 128, "codes");
  W4_CHECK_ALIGN(scales, 128, "scales");
  return launch_mxq("mxfp4_quantize", w4pg_mxfp4_quantize, M, K, (cudaStream_t)stream,
                    reinterpret_cast<const __half*>(x), codes, scales);
}

extern "C" int mxfp4_dequantize(const uint32_t* codes, const uint8_t* scales, int M, int K, uint16_t* y,
                                w4a16_stream_t stream) {
  W4_CHECK_ARG(codes && scales && y, "mxfp4_dequantize: null pointer");
  if (const int rc = mx_matrix_checks("mxfp4_dequantize", M, K)) return rc;
  W4_CHECK_ALIGN(codes, 128, "codes");
  W4_CHECK_ALIGN(scales, 128, "scales");
  W4_CHECK_ALIGN(y, 128, "y");
  return launch_mxq("mxfp4_dequantize", w4pg_mxfp4_dequantize, M, K, (cudaStream_t)stream, codes, scales,
                    reinterpret_cast<__half*>(y));
}

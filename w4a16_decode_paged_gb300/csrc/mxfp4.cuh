// mxfp4.cuh -- the MXFP4 matrix format, shared by its kernels.
//
// value = c * 2^(b - 127): c an E2M1 code (sign, then 0, 0.5, 1, 1.5, 2, 3, 4,
// 6), b one byte per 32 consecutive elements of a row (255: NaN).  Codes:
// uint32 [rows][K/8], the lowest nibble first.  Scale bytes: tiles of 128 rows
// x 128 elements, 512 bytes each, [rows/128 rounded up][K/128]; row r, block j
// of a tile at byte 16 (r % 32) + 4 (r / 32) + j.  That is the order in which
// the tensor core takes its scales (32 lanes of four 32-bit columns), so that
// they go there by plain copies; a thread that wants one row's scales reads
// the 4 bytes of 128 elements at once.
#pragma once

#include "common.cuh"

namespace w4 {

constexpr int MX_TILE = 512;          // bytes of a scale tile (128 rows x 4 blocks)
constexpr int MX_MIN_BYTE = 104;      // least scale written: 2^-23, whose half is the last fp16 bit
__host__ __device__ inline size_t mx_tiles(int rows, int K) { return (size_t)((rows + 127) / 128) * (K / 128); }

// byte offset of the four scales of row r, elements 128 kt .. 128 kt + 127
__host__ __device__ __forceinline__ size_t mx_scale_at(int r, int kt, int ktiles) {
  return ((size_t)(r >> 7) * ktiles + kt) * MX_TILE + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// the eight values of a code word as fp16 pairs (0 1) (2 3) (4 5) (6 7)
__device__ __forceinline__ uint4 mx_values(uint32_t w) {
  uint4 v;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "r"(w));
  return v;
}

// 2^(byte - 127) in fp32 (byte 0: zero); inf * 0 + inf makes the 255 a NaN
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  const float f = __uint_as_float(byte << 23);
  return fmaf(f, 0.f, f);
}

// What a weight's scale bytes stand for in the products with fp16 rows, two at a
// time (in bits 0..7 and 16..23), as a pair of bf16 numbers: 2^(byte - 127) for the
// bytes under which every value is an fp16 number (104..140, as the quantiser
// writes), zero below, NaN above.  One meaning for every kernel: what an operand in
// fp16 cannot hold does not depend on how many rows of x there are.
__device__ __forceinline__ uint32_t mx_weight_scales(uint32_t bytes) {
  const uint32_t e = bytes << 7;  // (255 is an infinity here)
  uint32_t least, above;
  asm("set.ge.u32.bf16x2 %0, %1, %2;" : "=r"(least) : "r"(e), "r"(0x34003400u));
  asm("set.gt.u32.bf16x2 %0, %1, %2;" : "=r"(above) : "r"(e), "r"(0x46004600u));
  return (e & least) | above;
}

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// One product (mxfp4_gemm): y[m][n] = sum_k x[m][k] w[n][k] (+ bias[n])
// (+ residual[m][n]), or silu(x g^T) * (x u^T) with two weight matrices.
struct MxWeights {
  const uint32_t* codes;   // [N][K/8]
  const uint8_t* scales;   // tiles
};
struct MxArgs {
  const __half* x;         // [M][K], or
  MxWeights xq;            // x in MXFP4 (x null)
  MxWeights w[2];          // w, or gate and up
  const __half* bias;      // [N] or null
  const __half* residual;  // [M][N] or null
  __half* y;               // [M][N]
  int M, N, K;
  void* workspace;
  size_t workspace_bytes;
  int32_t* err_flag;
};
// eight fp16 numbers added to eight sums
__device__ __forceinline__ void mx_add8(float4& lo, float4& hi, const uint4& r) {
  const float2 r0 = __half22float2(*reinterpret_cast<const __half2*>(&r.x)), r1 = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
  const float2 r2 = __half22float2(*reinterpret_cast<const __half2*>(&r.z)), r3 = __half22float2(*reinterpret_cast<const __half2*>(&r.w));
  lo.x += r0.x, lo.y += r0.y, lo.z += r1.x, lo.w += r1.y;
  hi.x += r2.x, hi.y += r2.y, hi.z += r3.x, hi.w += r3.y;
}
__device__ __forceinline__ uint4 mx_round8(const float4& lo, const float4& hi) {
  const __half2 h[4] = {__floats2half2_rn(lo.x, lo.y), __floats2half2_rn(lo.z, lo.w), __floats2half2_rn(hi.x, hi.y),
                        __floats2half2_rn(hi.z, hi.w)};
  return *reinterpret_cast<const uint4*>(h);
}
bool mxfp4_matvec_serves(int M, int N, int K, bool silu);
int launch_mxfp4_matvec(const MxArgs& a, bool silu, cudaStream_t s);
int launch_mxfp4_a16(const MxArgs& a, bool silu, cudaStream_t s);
int launch_mxfp4_a4(const MxArgs& a, cudaStream_t s);
size_t mxfp4_a4_workspace(int M, int N, int K);
size_t mxfp4_a16_workspace(int M, int N, int K, bool silu);
int mxfp4_a4_largest_tile();   // outputs
int mxfp4_a16_largest_tile();
// what w4a16_debug_mxfp4_plan tells
void mxfp4_matvec_plan(int M, int N, int K, bool silu, int32_t* plan);
void mxfp4_a16_plan(int M, int N, int K, bool silu, size_t bytes, int slots, int32_t* plan);
void mxfp4_a4_plan(int M, int N, int K, size_t bytes, int slots, int32_t* plan);

}  // namespace w4

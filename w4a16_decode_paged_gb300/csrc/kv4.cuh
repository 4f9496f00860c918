// kv4.cuh -- INT4 KV pages: the format, its quantiser and its unpacking.
//
// A (page, kv head) slice is 1088 bytes: 1024 bytes of codes (16 tokens x 128
// dims, two per byte, element d in nibble d % 2, lowest first, offset binary
// u = q + 8 with q in [-7, 7]) and 64 scale bytes (one per token and 32 dims).
//   value = q * s,  s = the fp16 number whose bits are byte << 7
// so a scale has 5 exponent and 3 fraction bits (4 significant bits, byte 0 = 0).
// A page holds bytes up to 0xE7 (15360; the quantiser's largest is 10240), as far
// as the unpacking goes, and 0xFF for a group that is no number.  A code has 3
// significant bits and a sign: every product is exact in fp16, in fp32 and
// against a scale that was divided by 64 (multiples of 2^-23).
// Quantising 32 values: s = the smallest scale with 7 s >= amax, q = x / s
// rounded to nearest even.  A group with an infinity or a NaN takes byte 0xFF
// and reads back as NaN throughout.
//
// Where the bytes sit follows from the attention's matrix fragments:
//   K codes   token t, dims 4i..4i+3 at 64 t + 2 i: a lane's 16 bytes are the 32
//             dims of one scale of one token
//   K scales  token t, group c at 1024 + 8 (t % 8) + 2 c + t / 8: the bytes of
//             tokens t and t + 8, which one lane needs, are neighbours
//   V codes   token t, dims 4i..4i+3 at 128 (t / 2) + 4 i + 2 (t % 2): the two
//             tokens of a pair alternate by halfwords, so that the nibbles at
//             one place of a word's two halves are one dim of both tokens
//   V scales  token t, group c at 1024 + 16 c + 4 (t % 8 / 2) + 2 (t / 8) + t % 2
// Each token's bytes are its own: appends of different tokens never meet.
#pragma once

#include "common.cuh"

namespace w4 {

constexpr int KV4_D = 128;
constexpr int KV4_PAGE = 16;
constexpr int KV4_GROUP = 32;                       // dims per scale
constexpr int KV4_CODES = KV4_PAGE * KV4_D / 2;     // 1024
constexpr uint32_t KV4_MAX_SCALE = 0xE7;            // largest scale byte of a page but for 0xFF (NaN)
constexpr int KV4_SLICE = KV4_CODES + KV4_PAGE * KV4_D / KV4_GROUP;  // 1088

// byte offsets in a slice of dims 4i..4i+3 (a halfword) and of group c's scale
__device__ __forceinline__ int kv4_k_code(int t, int i) { return 64 * t + 2 * i; }
__device__ __forceinline__ int kv4_v_code(int t, int i) { return 128 * (t >> 1) + 4 * i + 2 * (t & 1); }
__device__ __forceinline__ int kv4_k_scale(int t, int c) { return KV4_CODES + 8 * (t & 7) + 2 * c + (t >> 3); }
__device__ __forceinline__ int kv4_v_scale(int t, int c) {
  return KV4_CODES + 16 * c + 4 * ((t & 7) >> 1) + 2 * (t >> 3) + (t & 1);
}

// Scale byte of a group whose largest magnitude has the fp16 bits `bits`: the
// smallest scale s with 7 s >= amax.  amax / 7 is taken a little too small
// (times 1/7 rounded down): where it is a scale exactly, rounding up brings it
// back; elsewhere amax, of 11 bits, is 2^-12 or more away from 7 s, of 7 bits.
__device__ __forceinline__ uint32_t kv4_scale_byte(uint32_t bits) {
  if (bits >= 0x7C00u) return 0xFFu;  // an infinity or a NaN
  const float r = __half2float(__ushort_as_half((unsigned short)bits)) * __uint_as_float(0x3E124924u);
  // the 3 leading fraction bits rounded up (a carry moves the exponent on);
  // below fp16's normal range multiples of 2^-17
  if (r < 0x1p-14f) return (uint32_t)ceilf(r * 0x1p17f);
  return ((__float_as_uint(r) + 0xFFFFFu) >> 20) - (112u << 3);
}

__device__ __forceinline__ float kv4_scale_value(uint32_t byte) {
  return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

// Rows of 128 fp16 values, eight per lane (dims 8 c .. 8 c + 7 of lane c of a
// half-warp, packed in x) -> this lane's eight codes, lowest nibble first, and
// the scale byte of its group of four lanes.  Warp-wide: two rows at once.
__device__ __forceinline__ void kv4_quantise(const uint4& x, uint32_t& codes, uint32_t& byte) {
  // magnitudes compare as integers, NaN and infinity above every number
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __vmaxu2(m, (&x.x)[i] & 0x7FFF7FFFu);
  m = max(m & 0xFFFFu, m >> 16);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  byte = kv4_scale_byte(m);
  const bool live = byte != 0u && byte != 0xFFu;
  // q = x / s to nearest even, without a division per value: y = x (1/s) is off
  // by 2^-20 at most (two roundings of 2^-24 of |q| <= 7).  x / s is a tie n + 1/2
  // exactly or 2^-12 or more away from one (x has 11 bits, (n + 1/2) s has 8), so
  // rounding y to multiples of 2^-14 first (the sum with 768 and back) makes ties
  // exact and moves no other across.  The sum with 1.5 * 2^23 then leaves q in the
  // low bits.
  const float inv = live ? __frcp_rn(kv4_scale_value(byte)) : 0.f;
  codes = 0x88888888u - 0x4B400000u * 0x11111111u;  // (q + 8) 16^e, summed modulo 2^32
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float v = __half2float(__ushort_as_half((unsigned short)((&x.x)[e >> 1] >> (16 * (e & 1)))));
    float y = live ? __fmul_rn(v, inv) : 0.f;
    y = __fsub_rn(__fadd_rn(y, 768.0f), 768.0f);
    codes += __float_as_uint(__fadd_rn(y, 12582912.0f)) << (4 * e);
  }
}

// This lane's codes and (first lane of a group) scale into token t of a slice.
__device__ __forceinline__ void kv4_put(uint8_t* slice, bool is_k, int t, int c, uint32_t codes, uint32_t byte) {
  if (is_k) {
    *reinterpret_cast<uint32_t*>(slice + kv4_k_code(t, 2 * c)) = codes;
  } else {
    *reinterpret_cast<uint16_t*>(slice + kv4_v_code(t, 2 * c)) = (uint16_t)codes;
    *reinterpret_cast<uint16_t*>(slice + kv4_v_code(t, 2 * c + 1)) = (uint16_t)(codes >> 16);
  }
  if ((c & 3) == 0) slice[is_k ? kv4_k_scale(t, c >> 2) : kv4_v_scale(t, c >> 2)] = (uint8_t)byte;
}

// Rotate-half RoPE of rows held eight dims per lane (as above): the partner
// dims i +- 64 sit eight lanes away.  cs, sn: 64 cosines and sines.  Products
// and their sum are rounded one by one, so every caller gets the same bits.
// (Two to an instruction, mul.rn.f32x2 and add.rn.f32x2, came out fused and
// rounded once; the products alone in pairs saved no time.)
// This lane's eight cosines and sines of one position, the sines with the sign
// that the lane's half of the row takes them with: the low half rotates to
// x c - y s, the high half to x c + y s (x its own, y the partner's).
struct RopeLane {
  float c[8], s[8];
  __device__ __forceinline__ void load(const float* cs, const float* sn, int lane) {
    const int i = 8 * (lane & 7);
    const float sign = (lane & 8) == 0 ? -1.f : 1.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = cs[i + e];
      s[e] = sign * sn[i + e];
    }
  }
};
__device__ __forceinline__ void rope_rows(uint4& x, const RopeLane& t) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, (&x.x)[w], 8);
    float r[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float own = __half2float(__ushort_as_half((unsigned short)((&x.x)[w] >> (16 * e))));
      const float other = __half2float(__ushort_as_half((unsigned short)(y >> (16 * e))));
      r[e] = __fadd_rn(__fmul_rn(own, t.c[2 * w + e]), __fmul_rn(other, t.s[2 * w + e]));
    }
    const __half2 h = __floats2half2_rn(r[0], r[1]);
    (&x.x)[w] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

// ---------------------------------------------------------------------------
// Unpacking.  A nibble u at bits b..b+3 of a half, or-ed under an exponent
// that makes bit b worth 1, is the fp16 number 2^(10-b) + u; one fused
// multiply-add takes the bias off and applies the scale:
//   q s' = (2^(10-b) + u) s' - (2^(10-b) + 8) s',   s' = s / 64
// exactly, because the bias times a scale still fits fp16's 11 bits at b = 2
// and 6 (264 and 24).  264 s' stays in fp16's range up to s = 15360, the largest
// that a page may hold (264 / 64 times the next, 16384, does not), and the
// smallest s', 2^-23, is an fp16 number (2^-17 / 256 were not).  Callers multiply
// by 64.
// ---------------------------------------------------------------------------
struct Kv4Scale {
  uint32_t s, c264, c24;  // packed pairs
};
__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hfma2_u(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// two: the scales' fp16 bits (s, s)
__device__ __forceinline__ Kv4Scale kv4_scale_pair(uint32_t two) {
  Kv4Scale r;
  r.s = hmul2_u(two, 0x24002400u);     // 1 / 64
  r.c264 = hmul2_u(two, 0xC420C420u);  // -264 / 64
  r.c24 = hmul2_u(two, 0xB600B600u);   // -24 / 64
  return r;
}
// The exponents, kept in registers: an instruction takes one immediate, which
// the mask is, and a compiler that may re-create a constant does so at each use.
struct Kv4Bias {
  uint32_t e256, e16;
  __device__ __forceinline__ Kv4Bias() {
    asm volatile("mov.u32 %0, 0x5C005C00;" : "=r"(e256));
    asm volatile("mov.u32 %0, 0x4C004C00;" : "=r"(e16));
  }
};

// Eight codes of a word: x[n] = nibbles n of the low and of the high half.
__device__ __forceinline__ void kv4_unpack(uint32_t w, const Kv4Scale& k, const Kv4Bias& e, uint32_t (&x)[4]) {
  const uint32_t l = w << 2, r = w >> 6;  // nibbles 0, 1 and 2, 3 at bits 2 and 6
  x[0] = hfma2_u(and_or(l, 0x003C003Cu, e.e256), k.s, k.c264);
  x[1] = hfma2_u(and_or(l, 0x03C003C0u, e.e16), k.s, k.c24);
  x[2] = hfma2_u(and_or(r, 0x003C003Cu, e.e256), k.s, k.c264);
  x[3] = hfma2_u(and_or(r, 0x03C003C0u, e.e16), k.s, k.c24);
}

}  // namespace w4

// attn_window.cu -- paged GQA decode attention over INT4 pages, and with a
// sliding window and sinks over fp16, FP8 (E4M3) and INT4 pages.
//
// One query token per sequence at position L - 1 sees token t < L if t < sinks
// or t >= L - window.  Its pages are the sinks' pages, then the window's: a
// list of n "visible" pages (plain attention: all of them), cut into chunks of
// equal length over the CTAs of a (sequence, kv head) pair, and within a CTA
// over its warps.
//
// A page is a dense contraction for the G = Hq / Hkv query heads that share
// the kv head.  Tokens are the rows and heads the columns of the warp-level
// mma.sync m16n8k16 products (fp16 in, fp32 accumulate):
//   S^T[16 tokens][8 heads]  = K Q^T
//   O^T[128 dims][8 heads]  += V^T P^T
// so both products use all 16 rows (heads as rows would leave half of them
// zero), the accumulators of 8 heads x 128 dims are 32 registers a lane, and a
// lane's K rows and V dims are contiguous: a page's (page, kv head) slices go
// whole, 512 bytes per asynchronous copy, into the warp's ring in shared memory,
// are read back with 16-byte loads free of bank conflicts, and are widened in
// registers.  (Bulk copies to mbarriers measured the same for INT4 pages, and
// slower for the others, whose rows they cannot permute; copies straight to
// registers had too little in flight.)  P^T is the scores' accumulator
// transposed 8x8 by 8x8 with movmatrix.
//
// Softmax: p = exp2(s - m) with a reference m per head that lies ATW_HEAD (log2)
// under the running maximum as of the last time a score passed it by more than
// ATW_SLACK; only then are the sums rescaled (a warp-wide vote, no shuffles
// otherwise).  Sums and outputs are fp32.  P is rounded to fp16 once: the tensor
// cores' fp32-accumulating products take fp16.  With a head of 13 the largest
// p is 2^15, fp16's largest power of two; weights down to 2^-27 of the largest
// are normal numbers (rounded by 2^-11 of themselves, as much as the output)
// and smaller ones are off by 2^-38 of the largest at most.  (With p <= 1 the
// many small weights beside a few large ones are lost from 2^-14 down, while
// their sum keeps them: a quarter of the output where 32768 tokens lie e^-18 below
// a sink without a value, emulated.)  P's rest in a second product would bring the
// error from up to 1.35 times that of 32-bit sums down to theirs, at 7 % of the time
// over INT4 pages, 4 % over FP8 and 1 % over fp16 ones: not kept, as the output's
// own rounding is as large.
// K and V enter exactly: fp16 as they are, INT4 values (kv4.cuh) as fp16 numbers,
// FP8 codes as the fp16 numbers that they name.  K's row scales multiply the
// scores; V's go into P before its rounding, where a product p s of a small s
// would leave fp16's range as small weights do.  So the FP8 outputs have a
// reference of their own, which follows log2(p s) as m follows log2(p): P is
// p s 2^(m - mo) <= 2^15 for any row scales, and the warps' outputs go from mo
// to m where they are merged.  (A fixed factor of 64 lost 4 % of an output of
// 4e-6.)
//
// Rows that nothing attends to (an empty window, length 0) give zeros; masked
// tokens of a visible page take no part whatever their bytes hold: their
// scores are -inf and their V rows are zeroed.
//
// What bounds it (GB300, device time of one call among others): a chain of
// about 3 us before the first page is there (lengths, block table, page), the
// pages, and about 3 us to join the parts of a sequence.  fp16 and FP8 pages are
// waited for (32 sequences, window 1000, fp16: 58 MB in 13.4 us, 4.3 TB/s; batch
// 8, window 4096, FP8: 70 MB in 16.6 us, 4.2 TB/s).  INT4 pages (4 x 32768 tokens:
// 71 MB in 20.6 us, 3.5 TB/s) wait for their own instructions: 346 a page all
// told, 9 us of issue slots of the 20.6; 0.53 of a cycle's slot is used, no pipe
// is full, and a warp's next instruction most often waits for its last at 16
// warps per SM.  Measured beside two CTAs of eight warps per SM on that case:
// three CTAs leave 85 registers and spill (29 us and more), 1.5 and 2 times the
// CTAs pay the chain again (30 and 32 us), three, four or six pages in flight 21.8
// us and more.
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "attn_core.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace w4 {

constexpr int ATW_PITCH = ATT_D + 4;   // floats per head in the warps' merge
constexpr float ATW_SLACK = 2.0f;
constexpr float ATW_LOWEST = -3.402823466e38f;  // reference of heads that have met no score: under every finite one
constexpr float ATW_HEAD = 13.0f;      // log2: how far references lie under the scores that set them
constexpr float ATW_MOST = 100.0f;     // log2: bound of FP8's factor on p and row scale (they may be zero)

__device__ __forceinline__ uint4 ldcg16(const void* p) { return __ldcg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// D (16 x 8) += A (16 x 16) B (16 x 8), fp16 in, fp32 accumulate (registers as
// mma_16816_full; free to move, so that independent chains interleave).
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ float lg2(float x) {
  float d;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}
// to fp16, numbers beyond its range to its largest: a reference that is itself
// rounded (scores beyond 2^24) may leave P at 2^16
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// ---------------------------------------------------------------------------
// Page kinds.  Lane (g, t4) = (lane / 4, lane % 4) loads of a page
//   K: tokens g and g + 8, a quarter of the dims (dims in the order qdim gives)
//   V: tokens 2 t4, 2 t4 + 1 and 8 + those, 16 dims (in the order odim gives)
// k_frag gives the A fragments of MMA step st (st of 8), v_frag those of the
// 16 dims of block mt (mt of 8).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// What a lane copies from starts here, for page 0 and this kv head; pages lie
// `pitch` bytes apart (FP8: their row scales spitch).
struct LanePtrs {
  const unsigned char *k, *v, *s;
  uint32_t pitch, spitch;
  static __device__ __forceinline__ const unsigned char* at(const unsigned char* p, int page, uint32_t pitch) {
    return p + (uint64_t)(uint32_t)page * pitch;
  }
};

template <int KIND>
struct Page;

template <>
struct Page<ATW_F16> {
  static constexpr int NW = 8;      // warps per CTA
  static constexpr int MIN_CTAS = 1;
  static constexpr int MIN_PAGES = 8;
  static constexpr int V = 4096;    // V's offset in a page's slot
  static constexpr int SLOT = 8192;
  // dim of element e (0, 1) of query register r (0, 1) in step st
  static __device__ __forceinline__ int qdim(int st, int t4, int r, int e) {
    return 64 * (st >> 2) + 16 * t4 + 8 * ((st >> 1) & 1) + 4 * (st & 1) + 2 * r + e;
  }
  static __device__ __forceinline__ int odim(int mt, int g) { return 64 * (mt >> 2) + 8 * g + 2 * (mt & 3); }
  // Rows of 256 bytes, copied 512 bytes per instruction; the 16-byte chunks of
  // each half row are permuted by the row (chunk ^ row % 8), so that neither
  // the K reads (two rows, every other chunk) nor the V reads (four rows, one
  // chunk) of eight lanes meet in a bank.
  static __device__ __forceinline__ LanePtrs lane_ptrs(const AtwArgs& a, int kvh, int lane) {
    const size_t at = (size_t)kvh * 4096 + 16 * lane;
    return {static_cast<const unsigned char*>(a.k) + at, static_cast<const unsigned char*>(a.v) + at, nullptr,
            (uint32_t)a.Hkv * 4096u, 0u};
  }
  static __device__ __forceinline__ void fetch(const LanePtrs& lp, int page, uint32_t slot, int lane) {
    const unsigned char *k = LanePtrs::at(lp.k, page, lp.pitch), *v = LanePtrs::at(lp.v, page, lp.pitch);
    const int row = lane >> 4, c = lane & 15;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t at = slot + 512 * i + 256 * row + 16 * (c ^ ((2 * i + row) & 7));
      copy16(at, k + 512 * i);
      copy16(at + V, v + 512 * i);
    }
  }
  // S^T += K Q^T of one page, scaled where the kind has K row scales
  static __device__ __forceinline__ void scores(const unsigned char* slot, int g, int t4, const Kv4Bias&,
                                                const uint32_t (&qb)[8][2], float (&s)[4]) {
    const unsigned char* p = slot + 256 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = 128 * (i >> 1) + 16 * ((2 * t4 + (i & 1)) ^ g);
      const uint4 x = *reinterpret_cast<const uint4*>(p + at), y = *reinterpret_cast<const uint4*>(p + 2048 + at);
      mma(s, x.x, y.x, x.y, y.y, qb[2 * i][0], qb[2 * i][1]);
      mma(s, x.z, y.z, x.w, y.w, qb[2 * i + 1][0], qb[2 * i + 1][1]);
    }
  }
  // O^T += V^T P^T; MASK: bit r of live says that token r is seen, V rows of
  // others count as zero whatever they hold
  template <bool MASK>
  static __device__ __forceinline__ void output(const unsigned char* slot, int g, int t4, const Kv4Bias& bias, uint32_t live,
                                                uint32_t b0, uint32_t b1, float (&o)[8][4]) {
    const unsigned char* p = slot + V + 512 * t4;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4 w[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        w[r] = *reinterpret_cast<const uint4*>(p + 256 * (r & 1) + 2048 * (r >> 1) + 128 * i +
                                               16 * (g ^ (2 * t4 + (r & 1))));
        if (MASK && !((live >> (2 * t4 + (r & 1) + 8 * (r >> 1))) & 1u)) w[r] = make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = (&w[0].x)[j], b = (&w[1].x)[j], c = (&w[2].x)[j], d = (&w[3].x)[j];
        mma(o[4 * i + j], prmt(a, b, 0x5410), prmt(a, b, 0x7632), prmt(c, d, 0x5410), prmt(c, d, 0x7632), b0,
                       b1);
      }
    }
  }
};

template <>
struct Page<ATW_F8> {
  static constexpr int NW = 8;
  static constexpr int MIN_CTAS = 2;
  static constexpr int MIN_PAGES = 16;
  static constexpr int V = 2048, KS = 4096, VS = 4160;
  static constexpr int SLOT = 4224;
  static __device__ __forceinline__ int qdim(int st, int t4, int r, int e) {
    return 32 * t4 + 16 * (st >> 2) + 4 * (st & 3) + 2 * r + e;
  }
  static __device__ __forceinline__ int odim(int mt, int g) { return 16 * g + 2 * mt; }
  // (rows of 128 bytes, their chunks permuted as those of fp16 pages)
  static __device__ __forceinline__ LanePtrs lane_ptrs(const AtwArgs& a, int kvh, int lane) {
    const size_t at = (size_t)kvh * 2048 + 16 * lane;
    const float* s = (lane < 4 ? a.ks : a.vs) + (size_t)kvh * ATT_PAGE + 4 * (lane & 3);  // (lanes 0-7)
    return {static_cast<const unsigned char*>(a.k) + at, static_cast<const unsigned char*>(a.v) + at,
            reinterpret_cast<const unsigned char*>(s), (uint32_t)a.Hkv * 2048u, (uint32_t)a.Hkv * 64u};
  }
  static __device__ __forceinline__ void fetch(const LanePtrs& lp, int page, uint32_t slot, int lane) {
    const unsigned char *k = LanePtrs::at(lp.k, page, lp.pitch), *v = LanePtrs::at(lp.v, page, lp.pitch);
    const int row = lane >> 3, c = lane & 7;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t at = slot + 512 * i + 128 * row + 16 * (c ^ ((4 * i + row) & 7));
      copy16(at, k + 512 * i);
      copy16(at + V, v + 512 * i);
    }
    if (lane < 8) copy16(slot + KS + 16 * lane, LanePtrs::at(lp.s, page, lp.spitch));
  }
  static __device__ __forceinline__ void scores(const unsigned char* slot, int g, int t4, const Kv4Bias&,
                                                const uint32_t (&qb)[8][2], float (&s)[4]) {
    const unsigned char* p = slot + 128 * g;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = 16 * ((2 * t4 + i) ^ g);
      const uint4 x = *reinterpret_cast<const uint4*>(p + at), y = *reinterpret_cast<const uint4*>(p + 1024 + at);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t a0, a1, a2, a3;
        e4m3x4_to_h2x2((&x.x)[w], a0, a2);
        e4m3x4_to_h2x2((&y.x)[w], a1, a3);
        mma(s, a0, a1, a2, a3, qb[4 * i + w][0], qb[4 * i + w][1]);
      }
    }
    const float* ks = reinterpret_cast<const float*>(slot + KS);
    const float f0 = ks[g], f1 = ks[g + 8];
    s[0] *= f0;
    s[1] *= f0;
    s[2] *= f1;
    s[3] *= f1;
  }
  // V row scales of tokens g and g + 8 (0: not seen)
  template <bool MASK>
  static __device__ __forceinline__ void v_scales(const unsigned char* slot, int g, uint32_t live, float& f0, float& f1) {
    const float* vs = reinterpret_cast<const float*>(slot + VS);
    f0 = vs[g];
    f1 = vs[g + 8];
    if (MASK && !((live >> g) & 1u)) f0 = 0.f;
    if (MASK && !((live >> (g + 8)) & 1u)) f1 = 0.f;
  }
  template <bool MASK>
  static __device__ __forceinline__ void output(const unsigned char* slot, int g, int t4, const Kv4Bias& bias, uint32_t live,
                                                uint32_t b0, uint32_t b1, float (&o)[8][4]) {
    const unsigned char* p = slot + V + 256 * t4;
    uint4 w[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      w[r] = *reinterpret_cast<const uint4*>(p + 128 * (r & 1) + 1024 * (r >> 1) + 16 * (g ^ (2 * t4 + (r & 1))));
      if (MASK && !((live >> (2 * t4 + (r & 1) + 8 * (r >> 1))) & 1u)) w[r] = make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = (&w[0].x)[j], b = (&w[1].x)[j], c = (&w[2].x)[j], d = (&w[3].x)[j];
      uint32_t x[4], y[4];
      e4m3x4_to_h2x2(prmt(a, b, 0x5140), x[0], x[1]);
      e4m3x4_to_h2x2(prmt(a, b, 0x7362), x[2], x[3]);
      e4m3x4_to_h2x2(prmt(c, d, 0x5140), y[0], y[1]);
      e4m3x4_to_h2x2(prmt(c, d, 0x7362), y[2], y[3]);
      mma(o[2 * j], x[0], x[1], y[0], y[1], b0, b1);
      mma(o[2 * j + 1], x[2], x[3], y[2], y[3], b0, b1);
    }
  }
};

template <>
struct Page<ATW_I4> {
  static constexpr int NW = 8;
  static constexpr int MIN_CTAS = 2;
  static constexpr int MIN_PAGES = 32;
  static constexpr int V = 1024, KS = 2048, VS = 2112;
  static constexpr int SLOT = 2 * KV4_SLICE;
  static __device__ __forceinline__ int qdim(int st, int t4, int r, int e) {
    return 32 * t4 + 8 * (st >> 1) + 2 * (st & 1) + r + 4 * e;
  }
  static __device__ __forceinline__ int odim(int mt, int g) { return 16 * g + 2 * mt; }
  // K rows as they are (a lane reads the chunks it copied); the 16-byte chunks
  // of a V pair's 128 bytes permuted by the pair, so that the reads of eight
  // lanes (four pairs, two chunks) do not meet in a bank
  static __device__ __forceinline__ LanePtrs lane_ptrs(const AtwArgs& a, int kvh, int lane) {
    const size_t at = (size_t)kvh * KV4_SLICE + 16 * lane;
    const unsigned char *k = static_cast<const unsigned char*>(a.k) + at, *v = static_cast<const unsigned char*>(a.v) + at;
    return {k, v, (lane < 4 ? k : v - 64) + KV4_CODES, (uint32_t)a.Hkv * KV4_SLICE, 0u};  // (scales: lanes 0-7)
  }
  static __device__ __forceinline__ void fetch(const LanePtrs& lp, int page, uint32_t slot, int lane) {
    const unsigned char *k = LanePtrs::at(lp.k, page, lp.pitch), *v = LanePtrs::at(lp.v, page, lp.pitch);
    const int pair = lane >> 3, c = lane & 7;
    const uint32_t kd = slot + 16 * lane, vd = slot + V + 128 * pair + 16 * (c ^ (2 * pair));
    copy16(kd, k);
    copy16(kd + 512, k + 512);
    copy16(vd, v);
    copy16(vd + 512, v + 512);
    if (lane < 8) copy16(slot + KS + 16 * lane, LanePtrs::at(lp.s, page, lp.pitch));
  }
  static __device__ __forceinline__ void scores(const unsigned char* slot, int g, int t4, const Kv4Bias& bias,
                                                const uint32_t (&qb)[8][2], float (&s)[4]) {
    const uint4 k0 = *reinterpret_cast<const uint4*>(slot + kv4_k_code(g, 8 * t4));
    const uint4 k1 = *reinterpret_cast<const uint4*>(slot + kv4_k_code(g + 8, 8 * t4));
    const uint32_t ks = *reinterpret_cast<const uint16_t*>(slot + KS - KV4_CODES + kv4_k_scale(g, t4));  // tokens g and g + 8
    const Kv4Scale s0 = kv4_scale_pair((ks & 0xFFu) * 0x00800080u), s1 = kv4_scale_pair((ks >> 8) * 0x00800080u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t x[4], y[4];
      kv4_unpack((&k0.x)[i], s0, bias, x);
      kv4_unpack((&k1.x)[i], s1, bias, y);
      mma(s, x[0], y[0], x[1], y[1], qb[2 * i][0], qb[2 * i][1]);
      mma(s, x[2], y[2], x[3], y[3], qb[2 * i + 1][0], qb[2 * i + 1][1]);
    }
  }
  template <bool MASK>
  static __device__ __forceinline__ void output(const unsigned char* slot, int g, int t4, const Kv4Bias& bias, uint32_t live,
                                                uint32_t b0, uint32_t b1, float (&o)[8][4]) {
    const unsigned char* p = slot + V + 128 * t4 + 16 * (g ^ (2 * t4));
    const uint4 v0 = *reinterpret_cast<const uint4*>(p), v1 = *reinterpret_cast<const uint4*>(p + 512);
    // scale bytes of tokens 2 t4, 2 t4 + 1, 8 + 2 t4, 9 + 2 t4; a zero scale makes every code zero
    uint32_t vs = *reinterpret_cast<const uint32_t*>(slot + VS - KV4_CODES + kv4_v_scale(2 * t4, g >> 1));
    if (MASK) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (!((live >> (2 * t4 + (r & 1) + 8 * (r >> 1))) & 1u)) vs &= ~(0xFFu << (8 * r));
    }
    const Kv4Scale s0 = kv4_scale_pair(prmt(vs, 0u, 0x4140) << 7), s1 = kv4_scale_pair(prmt(vs, 0u, 0x4342) << 7);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t x[4], y[4];
      kv4_unpack((&v0.x)[j], s0, bias, x);
      kv4_unpack((&v1.x)[j], s1, bias, y);
      mma(o[2 * j], x[0], x[1], y[0], y[1], b0, b1);
      mma(o[2 * j + 1], x[2], x[3], y[2], y[3], b0, b1);
    }
  }
  // the new token's rows over what was copied (warp-wide)
  static __device__ __forceinline__ void patch(unsigned char* slot, const uint16_t (&codes)[2][32],
                                               const uint8_t (&scales)[2][4], int t, int lane) {
    *reinterpret_cast<uint16_t*>(slot + kv4_k_code(t, lane)) = codes[0][lane];
    const int pair = t >> 1;  // (dims 4 lane .. are in chunk lane / 4 of the pair)
    *reinterpret_cast<uint16_t*>(slot + V + 128 * pair + 16 * ((lane >> 2) ^ (2 * pair & 7)) + 4 * (lane & 3) +
                                 2 * (t & 1)) = codes[1][lane];
    if (lane < 4) slot[KS - KV4_CODES + kv4_k_scale(t, lane)] = scales[0][lane];
    else if (lane < 8) slot[VS - KV4_CODES + kv4_v_scale(t, lane - 4)] = scales[1][lane - 4];
  }
};

// factor of the accumulated scores and outputs
template <int KIND>
__device__ __forceinline__ constexpr float atw_s_factor() { return KIND == ATW_I4 ? 64.f : 1.f; }
template <int KIND>
__device__ __forceinline__ constexpr float atw_o_factor() { return KIND == ATW_I4 ? 64.f : 1.f; }

// ---------------------------------------------------------------------------
// Which pages a CTA takes.  A (sequence, kv head) pair with n visible pages is
// cut into ceil(n / per) equal parts, one CTA each, where `per` is what the
// whole batch's pages come to per CTA that fits the GPU at once (at least
// min_pages: below that a second CTA costs more than it saves).  CTAs are
// numbered in the order (sequence, kv head, part), so a CTA finds its place by
// a prefix sum over the sequences' part counts, which follow from the lengths.
// With equal lengths parts come out whole for a number of CTAs that is a
// multiple of the pairs (fit); where that leaves more parts than fit at once
// (slots), lengths are mixed and a pair rounds up by half a part on average.
// ---------------------------------------------------------------------------
struct AtwShare {
  int b, kvh, part, parts;     // b -1: nothing to do
  int L, w0, S, n, nsp, wp;    // L: the length, up to max_context
  int fits, len;               // whether the length is no longer than that; the length
};

// the visible pages of a sequence of this length
__device__ __forceinline__ AtwShare atw_visible(const AtwArgs& a, int len) {
  AtwShare r;
  r.fits = len <= a.max_context;
  r.len = len;
  r.L = max(min(len, a.max_context), 0);
  r.w0 = a.window >= r.L ? 0 : r.L - a.window;  // first token of the window
  r.S = min(a.sinks, r.L);                      // sinks
  if (r.w0 <= r.S) r.w0 = r.S = 0;              // they meet: everything is seen
  r.nsp = (r.S + ATT_PAGE - 1) / ATT_PAGE;
  r.wp = max(r.w0 / ATT_PAGE, r.nsp);           // the window's first page that is not a sink page
  r.n = r.nsp + (r.w0 < r.L ? max((r.L + ATT_PAGE - 1) / ATT_PAGE - r.wp, 0) : 0);
  return r;
}

// a / b rounded up, 0 <= a <= 2^20: (a - 1/2) / b is 1 / (2 b) away from every
// whole number, which the quotient's error (2^-22 of it) does not bridge
__device__ __forceinline__ int atw_div_up(int a, int b) {
  return a > 0 ? (int)__fdividef((float)a - 0.5f, (float)b) + 1 : 0;
}
__device__ __forceinline__ int atw_parts(int n, int per) {
  return min(max(atw_div_up(n, per), 1), ATW_MAX_PARTITIONS);
}
// Pages per part for `pages` in all over `fit` parts: a little more than their
// quotient at times, never less (the grid has no CTAs for more parts).  The
// host refuses contexts from 2^24 tokens on, and batches whose pages, times the
// kv heads, pass 2^30.
__device__ __forceinline__ int atw_per(unsigned pages, int fit, int min_pages) {
  return min(max((int)(__fdividef((float)pages, (float)fit) * 1.000001f) + 1, min_pages), 1 << 20);
}

// Up to 32 sequences: one warp's work (every warp's own would be eight times
// the requests for the same line of lengths).
__device__ __forceinline__ AtwShare atw_share_warp(const AtwArgs& a, int min_pages) {
  const int lane = threadIdx.x & 31, cta = blockIdx.x;
  const int len = lane < a.B ? __ldcg(&a.context_lens[lane]) : 0;
  const int n = lane < a.B ? atw_visible(a, len).n : 0;
  const unsigned all = __reduce_add_sync(0xffffffffu, (unsigned)n) * (unsigned)a.Hkv;
  int per = atw_per(all, a.fit, min_pages);
  int p = lane < a.B ? atw_parts(n, per) : 0;
  if (__reduce_add_sync(0xffffffffu, (unsigned)p) * (unsigned)a.Hkv > (unsigned)a.slots) {
    per = atw_per(all, a.fit_mixed, min_pages);
    p = lane < a.B ? atw_parts(n, per) : 0;
  }
  int hi = p * a.Hkv;  // inclusive prefix sum
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, hi, d);
    if (lane >= d) hi += t;
  }
  AtwShare r;
  const unsigned past = __ballot_sync(0xffffffffu, lane < a.B && hi > cta);  // sequences that end behind this CTA
  if (past == 0u) {
    r.b = -1;
    return r;
  }
  const int b = __ffs(past) - 1;
  r = atw_visible(a, __shfl_sync(0xffffffffu, len, b));
  r.b = b;
  r.parts = __shfl_sync(0xffffffffu, p, b);
  const int i = cta - (__shfl_sync(0xffffffffu, hi, b) - r.parts * a.Hkv);
  r.kvh = i / r.parts;
  r.part = i - r.kvh * r.parts;
  return r;
}

// More: CTA-wide; s: 24 ints of shared memory.
template <int NW>
__device__ __noinline__ AtwShare atw_share_cta(const AtwArgs& a, int min_pages, int* s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x;
  auto sum_over = [&](auto term) {  // of every sequence
    unsigned v = 0;
    for (int i = tid; i < a.B; i += NW * 32) v += term(atw_visible(a, __ldcg(&a.context_lens[i])).n);
    v = __reduce_add_sync(0xffffffffu, v);
    if (lane == 0) s[warp] = (int)v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += (unsigned)s[w];
    __syncthreads();
    return v;
  };
  const unsigned all = sum_over([](int n) { return (unsigned)n; }) * (unsigned)a.Hkv;
  int per = atw_per(all, a.fit, min_pages);
  if (sum_over([&](int n) { return (unsigned)atw_parts(n, per); }) * (unsigned)a.Hkv > (unsigned)a.slots)
    per = atw_per(all, a.fit_mixed, min_pages);
  // the sequence whose CTAs hold this one
  int base = 0;  // CTAs of the sequences before this round's
  int* found = s + 16;  // b, first CTA of b, parts
  if (tid == 0) found[0] = -1;
  for (int i0 = 0; i0 < a.B; i0 += NW * 32) {
    const int i = i0 + tid;
    const int p = i < a.B ? atw_parts(atw_visible(a, __ldcg(&a.context_lens[i])).n, per) : 0;
    int sum = p * a.Hkv;  // inclusive prefix sum over the threads
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += t;
    }
    if (lane == 31) s[warp] = sum;
    __syncthreads();
    int before = base, after = base;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < warp) before += s[w];
      after += s[w];
    }
    const int hi = before + sum, lo = hi - p * a.Hkv;
    if (p > 0 && cta >= lo && cta < hi) {
      found[0] = i;
      found[1] = lo;
      found[2] = p;
    }
    __syncthreads();
    base = after;
    if (cta < base) break;
  }
  AtwShare r;
  r.b = found[0];
  if (r.b < 0) return r;
  const int b = found[0], lo = found[1], p = found[2];
  r = atw_visible(a, __ldcg(&a.context_lens[b]));
  r.b = b;
  r.parts = p;
  r.kvh = (cta - lo) / p;
  r.part = (cta - lo) - r.kvh * p;
  return r;
}

constexpr int ATW_STAGES = 2;  // pages in flight per warp (more only make the first pages of all CTAs wait for each other)
template <int KIND>
constexpr size_t atw_ring_bytes() { return (size_t)Page<KIND>::NW * ATW_STAGES * Page<KIND>::SLOT; }
template <int KIND>
constexpr size_t atw_smem() { return std::max(atw_ring_bytes<KIND>(), (size_t)Page<KIND>::NW * 8 * ATW_PITCH * 4); }

template <int KIND, bool FUSE>
__global__ void __launch_bounds__(Page<KIND>::NW * 32, Page<KIND>::MIN_CTAS)
    w4pg_attn_window(const __grid_constant__ AtwArgs a) {
  using PG = Page<KIND>;
  constexpr int NW = PG::NW, STAGES = ATW_STAGES;
  extern __shared__ __align__(128) unsigned char smraw[];  // the warps' rings, then their merge
  __shared__ __align__(16) __half s_q[8][ATT_D + 8];
  __shared__ float s_ml[NW * 8 * 2];
  __shared__ float s_mo[KIND == ATW_F8 ? NW * 8 : 1];  // FP8: the references of the warps' outputs
  __shared__ __align__(16) float s_cos[FUSE ? ATT_D / 2 : 4], s_sin[FUSE ? ATT_D / 2 : 4];
  __shared__ __align__(16) uint16_t s_new[2][32];  // codes of the new K and V rows (fused)
  __shared__ uint8_t s_news[2][4];
  __shared__ int s_scan[24];
  __shared__ __align__(16) AtwShare s_share;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int G = a.G;
  W4_TRACE_SCOPE(a.tag);
  pdl_wait_then_trigger();
  W4_TRACE_WAITED();

  // ---- which (sequence, kv head) and which part of its pages ------------------
  AtwShare sh;
  if (a.B <= 32) {
    if (warp == 0) {
      const AtwShare r = atw_share_warp(a, PG::MIN_PAGES);
      if (lane == 0) s_share = r;
    }
    __syncthreads();
    sh = s_share;
  } else {
    sh = atw_share_cta<NW>(a, PG::MIN_PAGES, s_scan);
  }
  if (sh.b < 0) return;
  const int b = sh.b, kvh = sh.kvh, pc = sh.part, active = sh.parts;
  const int L = sh.L, w0 = sh.w0, S = sh.S, n = sh.n, nsp = sh.nsp, wp = sh.wp;
  const bool fits = sh.fits != 0;
  if (!fits && pc == 0 && tid == 0 && a.err_flag) atomicOr(a.err_flag, 1);
  const __half* qrow = a.q + (size_t)b * a.q_stride + (size_t)kvh * G * ATT_D;
  uint4 qw = make_uint4(0u, 0u, 0u, 0u);
  const int chunk = atw_div_up(n, active);
  const int v0 = pc * chunk, v1 = min(n, v0 + chunk);
  // The rows that become queries, and (fused, in the CTA of the last page) the
  // new K and V rows 8 and 9: half a warp per row.  They are asked for before
  // any page: behind the first pages' copies they would wait for them all.
  const int r = 2 * warp + (lane >> 4), c = lane & 15;
  const bool last = v0 < n && v1 == n;
  if (r < G) qw = ldcg16(qrow + r * ATT_D + 8 * c);
  else if (FUSE && last && (r == 8 || r == 9))
    qw = ldcg16(a.q + (size_t)b * a.q_stride + (size_t)(a.Hq + (r - 8) * a.Hkv + kvh) * ATT_D + 8 * c);
  const int pos = fits ? L - 1 : -1;  // the new token's (fused); a length past the bound appends nothing
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks;
  auto page_no = [&](int v) { return v < nsp ? v : v - nsp + wp; };

  // this warp takes every NW-th page
  const int wv0 = v0 + warp;
  const int steps = wv0 < v1 ? (v1 - wv0 + NW - 1) / NW : 0;
  auto table = [&](int i) {  // pool page of the warp's i-th page (-1: none, or not in the pool)
    const int v = wv0 + i * NW;
    if (v >= v1) return -1;
    const int pn = page_no(v);
    const int id = pn < a.max_blocks ? __ldcg(&bt[pn]) : -1;
    if (id < 0 || id >= a.num_pages) {
      if (a.err_flag) atomicOr(a.err_flag, 1);
      return -1;
    }
    return id;
  };
  // 32 page ids at a time, one per lane: `ids` holds those of the pages being
  // copied (32 k .. of the warp's list), ids_next the 32 after
  int ids = table(lane), ids_next = -1;
  unsigned have = 0;  // bit `stage`: its page was copied
  unsigned char* ring = smraw + (size_t)warp * STAGES * PG::SLOT;
  const LanePtrs lp = PG::lane_ptrs(a, kvh, lane);
  // copies the warp's page i into a stage (warp-wide; pages come in order)
  auto issue = [&](int i, int stage) {
    if ((i & 31) == 0 && i > 0) ids = ids_next;
    if ((i & 31) == 1) ids_next = table(i + 31 + lane);
    const int id = __shfl_sync(0xffffffffu, ids, i & 31);
    have &= ~(1u << stage);
    if (id >= 0) {
      PG::fetch(lp, id, smem_u32(ring) + stage * PG::SLOT, lane);
      have |= 1u << stage;
    }
  };
  if (FUSE && tid < ATT_D / 2) sincosf(__fmul_rn((float)max(sh.len - 1, 0), a.inv_freq[tid]), &s_sin[tid], &s_cos[tid]);
#pragma unroll
  for (int st = 0; st < STAGES; ++st) {
    if (st < steps) issue(st, st);
    cp_async_commit();  // (a group per page, empty behind the last)
  }
  // pages some of whose tokens are masked: the last of the sinks, the first of
  // the window, the last of the sequence (-1: none; fused: the new token's)
  const int part_s = S % ATT_PAGE ? nsp - 1 : -1;
  const int part_w = nsp < n && wp * ATT_PAGE < w0 ? nsp : -1;
  const int part_l = FUSE || L % ATT_PAGE ? n - 1 : -1;

  // ---- queries ----------------------------------------------------------------
  if (FUSE) {
    __syncthreads();  // the sines and cosines
    if (warp < (last ? 5 : 4)) {
      uint4 w = qw;
      RopeLane rope;
      rope.load(s_cos, s_sin, lane);
      rope_rows(w, rope);
      if (r < 8) {
        *reinterpret_cast<uint4*>(&s_q[r][8 * c]) = w;
      } else {
        const bool is_k = r == 8;
        if (!is_k) w = qw;
        uint32_t codes, byte;
        kv4_quantise(w, codes, byte);
        *reinterpret_cast<uint32_t*>(&s_new[r - 8][2 * c]) = codes;
        if ((c & 3) == 0) s_news[r - 8][c >> 2] = (uint8_t)byte;
        const int blk = max(pos, 0) / ATT_PAGE;
        const int id = pos >= 0 && blk < a.max_blocks ? __ldcg(&bt[blk]) : -1;
        if (id >= 0 && id < a.num_pages)
          kv4_put(static_cast<uint8_t*>(const_cast<void*>(is_k ? a.k : a.v)) + ((size_t)id * a.Hkv + kvh) * KV4_SLICE,
                  is_k, pos % ATT_PAGE, c, codes, byte);
      }
    }
  } else if (r < 8) {
    *reinterpret_cast<uint4*>(&s_q[r][8 * c]) = qw;
  }
  __syncthreads();
  uint32_t qb[8][2];
#pragma unroll
  for (int st = 0; st < 8; ++st)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const __half lo = s_q[g][PG::qdim(st, t4, r, 0)], hi = s_q[g][PG::qdim(st, t4, r, 1)];
      qb[st][r] = ((uint32_t)__half_as_ushort(lo) | ((uint32_t)__half_as_ushort(hi) << 16)) ^
                  (a.scale_log2 < 0.f ? 0x80008000u : 0u);
    }
  W4_TRACE_MARK(0);

  // ---- pages --------------------------------------------------------------------
  const float scale = fabsf(a.scale_log2) * atw_s_factor<KIND>();  // (its sign is in the queries)
  // references of heads 2 t4 and 2 t4 + 1 (log2 domain, ATW_HEAD under the scores
  // that set them).  Finite from the start:
  // a score of -inf (an infinity in a K row) under it weighs zero, not NaN
  float m0 = ATW_LOWEST, m1 = ATW_LOWEST;
  float l0 = 0.f, l1 = 0.f;              // this lane's part of their sums
  float o[8][4];                         // rows: dims odim(mt, g) + {0, 1}, columns: the two heads
#pragma unroll
  for (int mt = 0; mt < 8; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;

  const Kv4Bias bias;
  float t0 = ATW_LOWEST, t1 = ATW_LOWEST;  // scores above these move the references
  // FP8: the outputs' references, the sums log2(p s) that move them, and the
  // factors 2^(m - mo) of p s
  float mo0 = ATW_LOWEST, mo1 = ATW_LOWEST, fo0 = 0.f, fo1 = 0.f;
  // one page; MASK: some token of it is not seen
  auto attend = [&](auto mask, const int stage, int v) {
    constexpr bool MASK = decltype(mask)::value;
    unsigned char* slot = ring + stage * PG::SLOT;
    uint32_t live = 0u;  // bit r: token r of the page is seen: t < L, and t >= w0 or t < S
    if (MASK && (have >> stage) & 1u) {
      const int first = page_no(v) * ATT_PAGE;
      auto below = [&](int t) { return (1u << min(max(t - first, 0), ATT_PAGE)) - 1u; };
      live = below(L) & (~below(w0) | below(S));
    }
    const bool a0 = (live >> g) & 1u, a1 = (live >> (g + 8)) & 1u;  // this lane's tokens (MASK)
    if constexpr (FUSE) {
      if constexpr (MASK) {  // (the new token's page counts as masked)
        if (v == n - 1 && pos >= 0) PG::patch(slot, s_new, s_news, pos & 15, lane);
        __syncwarp();
      }
    }
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    PG::scores(slot, g, t4, bias, qb, s);
    // (log2 domain; rounded before a reference is taken off, not after it: the
    // largest of scores beyond 2^24 would come out a multiple of their spacing
    // above or below its own reference)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = __fmul_rn(s[i], scale);
    if (MASK) {
      if (!a0) s[0] = s[1] = -INFINITY;
      if (!a1) s[2] = s[3] = -INFINITY;
    }
    float x0 = fmaxf(s[0], s[2]), x1 = fmaxf(s[1], s[3]);
    bool move = x0 > t0 || x1 > t1;
    float v0 = 0.f, v1 = 0.f, y0 = 0.f, y1 = 0.f;  // FP8: V's row scales, the largest log2(p s)
    if constexpr (KIND == ATW_F8) {
      PG::template v_scales<MASK>(slot, g, live, v0, v1);
      const float e0 = lg2(fabsf(v0)), e1 = lg2(fabsf(v1));
      y0 = fmaxf(s[0] + e0, s[2] + e1);
      y1 = fmaxf(s[1] + e0, s[3] + e1);
      move = move || y0 - mo0 > ATW_HEAD + ATW_SLACK || y1 - mo1 > ATW_HEAD + ATW_SLACK;
    }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
        if constexpr (KIND == ATW_F8) {
          y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, d));
          y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, d));
        }
      }
      x0 = fmaxf(m0, x0 - ATW_HEAD);
      x1 = fmaxf(m1, x1 - ATW_HEAD);
      float c0 = x0 == m0 ? 1.f : ex2(m0 - x0), c1 = x1 == m1 ? 1.f : ex2(m1 - x1);
      m0 = x0;
      m1 = x1;
      t0 = m0 + (ATW_HEAD + ATW_SLACK);
      t1 = m1 + (ATW_HEAD + ATW_SLACK);
      l0 *= c0;
      l1 *= c1;
      if constexpr (KIND == ATW_F8) {
        y0 = fmaxf(mo0, y0 - ATW_HEAD);
        y1 = fmaxf(mo1, y1 - ATW_HEAD);
        c0 = y0 == mo0 ? 1.f : ex2(mo0 - y0);
        c1 = y1 == mo1 ? 1.f : ex2(mo1 - y1);
        mo0 = y0;
        mo1 = y1;
        fo0 = ex2(fminf(m0 - mo0, ATW_MOST));
        fo1 = ex2(fminf(m1 - mo1, ATW_MOST));
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        o[mt][0] *= c0;
        o[mt][1] *= c1;
        o[mt][2] *= c0;
        o[mt][3] *= c1;
      }
    }
    float p[4];
    p[0] = ex2(s[0] - m0);
    p[1] = ex2(s[1] - m1);
    p[2] = ex2(s[2] - m0);
    p[3] = ex2(s[3] - m1);
    l0 += p[0] + p[2];
    l1 += p[1] + p[3];
    if constexpr (KIND == ATW_F8) {
      p[0] *= v0 * fo0;
      p[1] *= v0 * fo1;
      p[2] *= v1 * fo0;
      p[3] *= v1 * fo1;
    }
    const uint32_t b0 = movmatrix_trans(pack_h2(p[0], p[1])), b1 = movmatrix_trans(pack_h2(p[2], p[3]));
    PG::template output<MASK>(slot, g, t4, bias, live, b0, b1, o);
  };
  auto one = [&](int i, auto which) {  // the stage is a constant: addresses and masks fold
    constexpr int stage = decltype(which)::value;
    const int v = wv0 + i * NW;   // the visible page
    cp_async_wait<STAGES - 1>();  // this lane's copies,
    __syncwarp();                 // and every other's
    if (((have >> stage) & 1u) && v != part_s && v != part_w && v != part_l) attend(std::false_type{}, stage, v);
    else attend(std::true_type{}, stage, v);
    __syncwarp();  // every lane has read the stage
    if (i + STAGES < steps) issue(i + STAGES, stage);
    cp_async_commit();
  };
  static_assert(STAGES == 2, "pages alternate between two stages");
  for (int i = 0; i < steps; i += 2) {
    one(i, std::integral_constant<int, 0>{});
    if (i + 1 < steps) one(i + 1, std::integral_constant<int, 1>{});
  }
  cp_async_wait<0>();
  __syncthreads();  // the rings become the merge's buffer
  W4_TRACE_MARK(1);

  // ---- the warps' states, merged in shared memory ------------------------------------
  float* s_o = reinterpret_cast<float*>(smraw);  // [warp][head][128 + 4], dims in the order (mt, g, e)
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, d);
    l1 += __shfl_xor_sync(0xffffffffu, l1, d);
  }
#pragma unroll
  for (int mt = 0; mt < 8; ++mt) {
    float* p = s_o + (warp * 8 + 2 * t4) * ATW_PITCH + 16 * mt + 2 * g;
    *reinterpret_cast<float2*>(p) = make_float2(o[mt][0], o[mt][2]);
    *reinterpret_cast<float2*>(p + ATW_PITCH) = make_float2(o[mt][1], o[mt][3]);
  }
  if (g == 0) {
    float* ml = s_ml + (warp * 8 + 2 * t4) * 2;
    ml[0] = m0;
    ml[1] = l0;
    ml[2] = m1;
    ml[3] = l1;
    if constexpr (KIND == ATW_F8) {
      s_mo[warp * 8 + 2 * t4] = mo0;
      s_mo[warp * 8 + 2 * t4 + 1] = mo1;
    }
  }
  __syncthreads();
  const size_t qh0 = (size_t)b * a.Hq + (size_t)kvh * G;
  auto write_out = [&](int h, int i4, float4 acc) {  // positions 4 i4 .. 4 i4 + 3 of the order (mt, g, e)
    const int mt = i4 >> 2, g0 = 2 * (i4 & 3);
    __half* out = a.out + (qh0 + h) * ATT_D;
    *reinterpret_cast<__half2*>(out + PG::odim(mt, g0)) = __floats2half2_rn(acc.x, acc.y);
    *reinterpret_cast<__half2*>(out + PG::odim(mt, g0 + 1)) = __floats2half2_rn(acc.z, acc.w);
  };
  static_assert(8 % NW == 0, "a warp per head, or for a few heads");
  const int i4 = lane;
  const bool single = active == 1;
  for (int h = warp; h < G; h += NW) {
    float M = ATW_LOWEST;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, s_ml[(w * 8 + h) * 2]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float mw = s_ml[(w * 8 + h) * 2], lw = s_ml[(w * 8 + h) * 2 + 1];
      const float f = ex2(mw - M);
      const float fo = KIND == ATW_F8 ? ex2(s_mo[KIND == ATW_F8 ? w * 8 + h : 0] - M) : f;
      const float4 v = *reinterpret_cast<const float4*>(s_o + (w * 8 + h) * ATW_PITCH + 4 * i4);
      acc.x = fmaf(v.x, fo, acc.x);
      acc.y = fmaf(v.y, fo, acc.y);
      acc.z = fmaf(v.z, fo, acc.z);
      acc.w = fmaf(v.w, fo, acc.w);
      den = fmaf(lw, f, den);
    }
    if (single) {
      const float inv = den == 0.f ? 0.f : atw_o_factor<KIND>() / den;
      write_out(h, i4, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
      continue;
    }
    // ---- this head's partials of all the parts: the last warp to finish its
    // adds them up, in the order of the parts ---------------------------------
    const size_t mine = (size_t)blockIdx.x * G + h;
    __stcg(reinterpret_cast<float4*>(a.ws_o + mine * ATT_D) + i4, acc);
    if (lane == 0) __stcg(reinterpret_cast<float2*>(a.ws_ml) + mine, make_float2(M, den));
    __syncwarp();
    unsigned* counter = a.counters + qh0 + h;
    unsigned ticket = 0;
    if (lane == 0)  // releases the warp's partial with the ticket; for the last, acquires the others'
      asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(ticket) : "l"(counter) : "memory");
    ticket = __shfl_sync(0xffffffffu, ticket, 0);
    __syncwarp();
    if (ticket != (unsigned)(active - 1)) continue;
    if (lane == 0) *counter = 0u;  // ready for the next call
    // one round trip for the first partials and all (max, sum) pairs.  FLIGHT: as
    // many partials as go into the registers that the page loop has (32 spill)
    constexpr int FLIGHT = 20;
    const size_t first = (size_t)(blockIdx.x - pc) * G + h;  // the parts are consecutive CTAs
    const float4* src = reinterpret_cast<const float4*>(a.ws_o) + first * (ATT_D / 4) + i4;
    const size_t pitch = (size_t)G * (ATT_D / 4);
    float4 pv[FLIGHT];
#pragma unroll
    for (int j = 0; j < FLIGHT; ++j)
      if (j < active) pv[j] = __ldcg(src + (size_t)j * pitch);
    constexpr int PER_LANE = (ATW_MAX_PARTITIONS + 31) / 32;  // parts lane, 32 + lane, ..
    float2 e[PER_LANE];
#pragma unroll
    for (int k = 0; k < PER_LANE; ++k)
      e[k] = 32 * k + lane < active ? __ldcg(reinterpret_cast<const float2*>(a.ws_ml) + first + (size_t)(32 * k + lane) * G)
                                    : make_float2(ATW_LOWEST, 0.f);
    float top = e[0].x;
#pragma unroll
    for (int k = 1; k < PER_LANE; ++k) top = fmaxf(top, e[k].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    float f[PER_LANE], sum = 0.f;  // weights
#pragma unroll
    for (int k = 0; k < PER_LANE; ++k) {
      f[k] = ex2(e[k].x - top);
      sum = fmaf(e[k].y, f[k], sum);
    }
    sum = warp_sum(sum);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = 0;;) {  // (the rest FLIGHT at a time: 64 parts of 32768 tokens, 4 heads 16.3 -> 13.5 us)
#pragma unroll
      for (int j = 0; j < FLIGHT; ++j) {
        if (j0 + j >= active) break;
        float mine = f[0];
#pragma unroll
        for (int k = 1; k < PER_LANE; ++k)
          if ((j0 + j) >> 5 == k) mine = f[k];
        const float w = __shfl_sync(0xffffffffu, mine, (j0 + j) & 31);
        acc.x = fmaf(pv[j].x, w, acc.x);
        acc.y = fmaf(pv[j].y, w, acc.y);
        acc.z = fmaf(pv[j].z, w, acc.z);
        acc.w = fmaf(pv[j].w, w, acc.w);
      }
      j0 += FLIGHT;
      if (j0 >= active) break;
#pragma unroll
      for (int j = 0; j < FLIGHT; ++j)
        if (j0 + j < active) pv[j] = __ldcg(src + (size_t)(j0 + j) * pitch);
    }
    const float inv = sum == 0.f ? 0.f : atw_o_factor<KIND>() / sum;
    write_out(h, i4, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  }
}

// Pages that a sequence can see.
static long long atw_most_pages(int max_context, int window, int sinks) {
  const long long all = ((long long)max_context + ATT_PAGE - 1) / ATT_PAGE;
  const long long seen = ((long long)std::min(sinks, max_context) + ATT_PAGE - 1) / ATT_PAGE +
                         ((long long)window + ATT_PAGE - 2) / ATT_PAGE + 1;
  return std::min(all, seen);
}

template <class F>
static auto atw_of_kind(int kind, F f) {
  if (kind == ATW_F16) return f(Page<ATW_F16>{});
  if (kind == ATW_F8) return f(Page<ATW_F8>{});
  return f(Page<ATW_I4>{});
}

// The split's figures (see above) and the CTAs of the grid: no more than either
// every pair's pages in parts of min_pages, or the shared-out parts and one
// part of rounding up per pair, can need.
void atw_plan(AtwArgs& a, int kind, int B, int Hq, int Hkv, int max_context, int window, int sinks) {
  const long long groups = (long long)B * Hkv;
  const long long n = atw_most_pages(max_context, window, sinks);
  const int min_pages = atw_of_kind(kind, [](auto p) { return (int)p.MIN_PAGES; });
  a.slots = ATW_SMS * atw_of_kind(kind, [](auto p) { return (int)p.MIN_CTAS; });
  a.fit = groups <= a.slots ? (int)(a.slots / groups * groups) : a.slots;
  a.fit_mixed = (int)std::max(a.slots - groups / 2, a.slots / 2ll);
  a.ctas = (int)std::min(groups * std::min((n + min_pages - 1) / min_pages, (long long)ATW_MAX_PARTITIONS),
                         std::max(a.fit, a.fit_mixed) + groups);
  if (B * (long long)Hq * 4 > (long long)ATT_TICKET_BYTES) {  // no ticket for every query head: no splitting
    a.fit = a.fit_mixed = 1;
    a.ctas = (int)groups;
  }
}

// CTAs that no call over up to B sequences, any kind of page and up to this
// context, window and sinks exceeds where it splits (atw_plan's fit, fit_mixed
// <= slots): a workspace for a batch serves smaller ones, which may have more
// parts (Hkv 4: 380 CTAs for 39 sequences, 456 for 38).
int atw_most_ctas(int B, int Hq, int Hkv, int max_context, int window, int sinks) {
  const long long tickets = (long long)ATT_TICKET_BYTES / 4 / (Hq / Hkv);  // pairs that split calls can have
  const long long groups = std::min((long long)B * Hkv, tickets);
  const long long n = atw_most_pages(max_context, window, sinks);
  long long most = 0;
  for (int kind : {ATW_F16, ATW_F8, ATW_I4})
    most = std::max(most, atw_of_kind(kind, [&](auto p) {
      return std::min(groups * std::min((n + p.MIN_PAGES - 1) / p.MIN_PAGES, (long long)ATW_MAX_PARTITIONS),
                      (long long)ATW_SMS * p.MIN_CTAS + groups);
    }));
  return (int)most;
}

template <int KIND, bool FUSE>
static int launch_atw(const AtwArgs& a, cudaStream_t s) {
  static PerDeviceOnce once;
  constexpr size_t smem = atw_smem<KIND>();
  auto kern = w4pg_attn_window<KIND, FUSE>;
  once_per_device(once, [&] { cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem); });
  cudaError_t e = launch_pdl(kern, dim3(a.ctas), dim3(Page<KIND>::NW * 32), smem, s, a);
  if (e != cudaSuccess) return set_error(W4A16_ERR_CUDA, "paged attention launch: %s", cudaGetErrorString(e));
  return W4A16_OK;
}

int launch_attn_window(const AtwArgs& a, cudaStream_t s) {
  if (a.G > 8) return set_error(W4A16_ERR_SHAPE, "paged attention: Hq/Hkv=%d > 8", a.G);
  if (a.kind == ATW_F16) return launch_atw<ATW_F16, false>(a, s);
  if (a.kind == ATW_F8) return launch_atw<ATW_F8, false>(a, s);
  return a.fuse_rope_append ? launch_atw<ATW_I4, true>(a, s) : launch_atw<ATW_I4, false>(a, s);
}

}  // namespace w4

using namespace w4;

// The checks and the set-up that every entry shares.  who: the entry's name.
static int atw_call(AtwArgs& a, const uint16_t* q, int q_stride, int num_pages, const int32_t* block_table, int max_blocks,
                    const int32_t* context_lens, int max_context, int window, int sinks, int B, int Hq, int Hkv, int D,
                    float theta, float sm_scale, void* workspace, size_t workspace_bytes, uint16_t* out,
                    int32_t* err_flag, cudaStream_t stream, const char* who) {
  W4_CHECK_ARG(q && a.k && a.v && block_table && context_lens && out, "%s: null tensor pointer", who);
  W4_CHECK_ARG(B >= 1 && Hq >= 1 && Hkv >= 1 && num_pages >= 1 && max_blocks >= 1 && max_context >= 1,
               "%s: sizes must be positive", who);
  W4_CHECK_ARG(window >= 0 && sinks >= 0, "%s: window=%d sinks=%d", who, window, sinks);
  W4_CHECK_SHAPE(D == ATT_D, "%s: D=%d, only 128 is built", who, D);
  W4_CHECK_SHAPE(Hq % Hkv == 0 && Hq / Hkv <= 8, "%s: Hq=%d Hkv=%d", who, Hq, Hkv);
  W4_CHECK_SHAPE(Hkv <= (1 << 16), "%s: Hkv=%d > 65536", who, Hkv);  // (a page of all heads: below 2^32 bytes)
  W4_CHECK_SHAPE((long long)B * Hkv <= (1 << 24) && max_context < (1 << 24) &&
                     (long long)B * Hkv * (max_context / ATT_PAGE + 1) <= (1 << 30),
                 "%s: B=%d x Hkv=%d x max_context %d is too large", who, B, Hkv, max_context);
  W4_CHECK_SHAPE((long long)max_context <= (long long)max_blocks * ATT_PAGE, "%s: max_context %d > max_blocks*16", who,
                 max_context);
  const bool fuse = a.fuse_rope_append;
  if (fuse) W4_CHECK_ARG(theta > 0.f, "%s: theta must be positive", who);
  const int min_stride = (fuse ? Hq + 2 * Hkv : Hq) * D;
  if (q_stride == 0) q_stride = min_stride;
  W4_CHECK_ARG(q_stride >= min_stride && q_stride % 8 == 0, "%s: bad q_stride", who);
  W4_CHECK_ALIGN(q, 128, "q");
  W4_CHECK_ALIGN(a.k, 128, "k_pool");
  W4_CHECK_ALIGN(a.v, 128, "v_pool");
  W4_CHECK_ALIGN(out, 128, "out");
  atw_plan(a, a.kind, B, Hq, Hkv, max_context, window, sinks);
  if (a.ctas > B * Hkv) {
    const size_t need = atw_workspace_bytes(a.ctas, Hq / Hkv);
    W4_CHECK_ARG(workspace != nullptr && workspace_bytes >= need, "%s: workspace of %zu bytes needed", who, need);
    W4_CHECK_ALIGN(workspace, 128, "workspace");
    atw_workspace(a, workspace, a.ctas, Hq / Hkv);
  }
  a.q = reinterpret_cast<const __half*>(q);
  a.block_table = block_table;
  a.context_lens = context_lens;
  a.out = reinterpret_cast<__half*>(out);
  a.err_flag = err_flag;
  a.q_stride = q_stride;
  a.num_pages = num_pages;
  a.max_blocks = max_blocks;
  a.max_context = max_context;
  a.window = window;
  a.sinks = sinks;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  if (fuse) rope_inv_freq_table(theta, D, a.inv_freq);
  return launch_attn_window(a, stream);
}

extern "C" size_t paged_gqa_decode_window_workspace_size(int B, int Hq, int Hkv, int max_context, int window,
                                                         int sinks, int D) {
  (void)D;
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_context < 1 || window < 0 || sinks < 0 ||
      (long long)B * Hkv > (1 << 24))
    return 0;
  return atw_workspace_bytes(atw_most_ctas(B, Hq, Hkv, max_context, window, sinks), Hq / Hkv);
}

extern "C" int paged_gqa_decode_window(const uint16_t* q, int q_stride, const uint16_t* k_pool, const uint16_t* v_pool,
                                       int num_pages, const int32_t* block_table, int max_blocks,
                                       const int32_t* context_lens, int max_context, int window, int sinks, int B,
                                       int Hq, int Hkv, int D, float sm_scale, void* workspace, size_t workspace_bytes,
                                       uint16_t* out, int32_t* err_flag, w4a16_stream_t stream) {
  AtwArgs a = {};
  a.kind = ATW_F16;
  a.k = k_pool;
  a.v = v_pool;
  return atw_call(a, q, q_stride, num_pages, block_table, max_blocks, context_lens, max_context, window, sinks, B, Hq,
                  Hkv, D, 0.f, sm_scale, workspace, workspace_bytes, out, err_flag, (cudaStream_t)stream,
                  "paged_gqa_decode_window");
}

extern "C" int paged_gqa_decode_window_fp8(const uint16_t* q, int q_stride, const uint8_t* k_pool,
                                           const uint8_t* v_pool, const float* k_scale, const float* v_scale,
                                           int num_pages, const int32_t* block_table, int max_blocks,
                                           const int32_t* context_lens, int max_context, int window, int sinks, int B,
                                           int Hq, int Hkv, int D, float sm_scale, void* workspace,
                                           size_t workspace_bytes, uint16_t* out, int32_t* err_flag,
                                           w4a16_stream_t stream) {
  W4_CHECK_ARG(k_scale && v_scale, "paged_gqa_decode_window_fp8: null scale pointer");
  W4_CHECK_ALIGN(k_scale, 128, "k_scale");
  W4_CHECK_ALIGN(v_scale, 128, "v_scale");
  AtwArgs a = {};
  a.kind = ATW_F8;
  a.k = k_pool;
  a.v = v_pool;
  a.ks = k_scale;
  a.vs = v_scale;
  return atw_call(a, q, q_stride, num_pages, block_table, max_blocks, context_lens, max_context, window, sinks, B, Hq,
                  Hkv, D, 0.f, sm_scale, workspace, workspace_bytes, out, err_flag, (cudaStream_t)stream,
                  "paged_gqa_decode_window_fp8");
}

extern "C" int paged_gqa_decode_window_int4(const uint16_t* q, int q_stride, const uint8_t* k_pool,
                                            const uint8_t* v_pool, int num_pages, const int32_t* block_table,
                                            int max_blocks, const int32_t* context_lens, int max_context, int window,
                                            int sinks, int B, int Hq, int Hkv, int D, float sm_scale, void* workspace,
                                            size_t workspace_bytes, uint16_t* out, int32_t* err_flag,
                                            w4a16_stream_t stream) {
  AtwArgs a = {};
  a.kind = ATW_I4;
  a.k = k_pool;
  a.v = v_pool;
  return atw_call(a, q, q_stride, num_pages, block_table, max_blocks, context_lens, max_context, window, sinks, B, Hq,
                  Hkv, D, 0.f, sm_scale, workspace, workspace_bytes, out, err_flag, (cudaStream_t)stream,
                  "paged_gqa_decode_window_int4");
}

extern "C" int paged_gqa_decode_int4(const uint16_t* q, int q_stride, const uint8_t* k_pool, const uint8_t* v_pool,
                                     int num_pages, const int32_t* block_table, int max_blocks,
                                     const int32_t* context_lens, int max_context, int B, int Hq, int Hkv, int D,
                                     float sm_scale, void* workspace, size_t workspace_bytes, uint16_t* out,
                                     int32_t* err_flag, w4a16_stream_t stream) {
  AtwArgs a = {};
  a.kind = ATW_I4;
  a.k = k_pool;
  a.v = v_pool;
  return atw_call(a, q, q_stride, num_pages, block_table, max_blocks, context_lens, max_context, max_context, 0, B, Hq,
                  Hkv, D, 0.f, sm_scale, workspace, workspace_bytes, out, err_flag, (cudaStream_t)stream,
                  "paged_gqa_decode_int4");
}

extern "C" int paged_gqa_decode_rope_append_int4(const uint16_t* qkv, int qkv_stride, uint8_t* k_pool, uint8_t* v_pool,
                                                 int num_pages, const int32_t* block_table, int max_blocks,
                                                 const int32_t* context_lens, int max_context, int B, int Hq, int Hkv,
                                                 int D, float theta, float sm_scale, void* workspace,
                                                 size_t workspace_bytes, uint16_t* out, int32_t* err_flag,
                                                 w4a16_stream_t stream) {
  AtwArgs a = {};
  a.kind = ATW_I4;
  a.k = k_pool;
  a.v = v_pool;
  a.fuse_rope_append = 1;
  return atw_call(a, qkv, qkv_stride, num_pages, block_table, max_blocks, context_lens, max_context, max_context, 0, B,
                  Hq, Hkv, D, theta, sm_scale, workspace, workspace_bytes, out, err_flag, (cudaStream_t)stream,
                  "paged_gqa_decode_rope_append_int4");
}

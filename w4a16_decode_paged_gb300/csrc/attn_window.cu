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
// lane's K rows and V dims are contiguous in memory: the cache goes from global
// memory to registers with 16-byte loads and is widened there, without shared
// memory.  The next page's K is requested when the scores have consumed this
// page's, its V after the second product.  P^T is the scores' accumulator
// transposed 8x8 by 8x8 with movmatrix.
//
// Softmax: p = exp2(s - m) with a reference m per head that is the running
// maximum as of the last time a score passed it by more than 2^ATW_SLACK;
// only then are the sums rescaled (a warp-wide vote, no shuffles otherwise).
// p stays <= 2^ATW_SLACK, sums and outputs are fp32, P is rounded to fp16 once.
//
// Rows that nothing attends to (an empty window, length 0) give zeros; masked
// tokens of a visible page take no part whatever their bytes hold: their
// scores are -inf and their V rows are zeroed.
#include <algorithm>
#include <cmath>

#include "attn_core.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace w4 {

constexpr int ATW_NW = 8;              // warps per CTA
constexpr int ATW_PITCH = ATT_D + 4;   // floats per head in the warps' merge
constexpr float ATW_SLACK = 2.0f;
constexpr float ATW_V8 = 64.0f;        // FP8: factor that keeps p * (V row scale) in fp16's normal range

__device__ __forceinline__ uint4 ldcg16(const void* p) { return __ldcg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---------------------------------------------------------------------------
// Page kinds.  Lane (g, t4) = (lane / 4, lane % 4) loads of a page
//   K: tokens g and g + 8, a quarter of the dims (dims in the order qdim gives)
//   V: tokens 2 t4, 2 t4 + 1 and 8 + those, 16 dims (in the order odim gives)
// k_frag gives the A fragments of MMA step st (st of 8), v_frag those of the
// 16 dims of block mt (mt of 8).
// ---------------------------------------------------------------------------
template <int KIND>
struct Page;

// Where a lane reads in slice 0 of this (kv head's) pools, and the bytes from
// one page to the next; kc / vc codes or values, ks / vs scales.
struct LanePtrs {
  const uint8_t *kc, *vc, *ks, *vs;
  uint32_t pitch, spitch;
  __device__ __forceinline__ const uint8_t* at(const uint8_t* p, int page) const {
    return p + (uint64_t)(uint32_t)page * pitch;
  }
  __device__ __forceinline__ const uint8_t* at_scale(const uint8_t* p, int page) const {
    return p + (uint64_t)(uint32_t)page * spitch;
  }
};

template <>
struct Page<ATW_F16> {
  static constexpr int BATCH = 1;  // pages per step of a warp
  uint4 k[2][4], v[4][2];
  // dim of element e (0, 1) of query register r (0, 1) in step st
  static __device__ __forceinline__ int qdim(int st, int t4, int r, int e) {
    return 32 * (st >> 1) + 8 * t4 + 4 * (st & 1) + 2 * r + e;
  }
  static __device__ __forceinline__ int odim(int mt, int g) { return 64 * (mt >> 2) + 8 * g + 2 * (mt & 3); }
  static __device__ __forceinline__ LanePtrs lane_ptrs(const AtwArgs& a, int kvh, int g, int t4) {
    const uint8_t* k = static_cast<const uint8_t*>(a.k) + (size_t)kvh * ATT_SLICE * 2;
    const uint8_t* v = static_cast<const uint8_t*>(a.v) + (size_t)kvh * ATT_SLICE * 2;
    return {k + g * 256 + 16 * t4, v + 2 * t4 * 256 + 16 * g, nullptr, nullptr, (uint32_t)(a.Hkv * ATT_SLICE * 2), 0u};
  }
  __device__ __forceinline__ void load_k(const LanePtrs& lp, int page) {
    const uint8_t* p = lp.at(lp.kc, page);
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) k[r][i] = ldcg16(p + r * 2048 + 64 * i);
  }
  __device__ __forceinline__ void load_v(const LanePtrs& lp, int page) {
    const uint8_t* p = lp.at(lp.vc, page);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < 2; ++i) v[r][i] = ldcg16(p + ((r & 1) + 8 * (r >> 1)) * 256 + 128 * i);
  }
  // V rows of tokens that are not seen (bit r of live: token r is) become zero
  __device__ __forceinline__ void mask_v(uint32_t live, int, int t4) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (!((live >> (2 * t4 + (r & 1) + 8 * (r >> 1))) & 1u)) v[r][0] = v[r][1] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void scores(const uint32_t (&qb)[8][2], float (&s)[4]) const {
#pragma unroll
    for (int st = 0; st < 8; ++st) {
      const uint32_t* k0 = &k[0][st >> 1].x + 2 * (st & 1);
      const uint32_t* k1 = &k[1][st >> 1].x + 2 * (st & 1);
      mma_16816_full(s, k0[0], k1[0], k0[1], k1[1], qb[st][0], qb[st][1]);
    }
  }
  __device__ __forceinline__ void score_scale(float (&)[4]) const {}
  __device__ __forceinline__ void p_scale(float (&)[4]) const {}
  __device__ __forceinline__ void output(uint32_t b0, uint32_t b1, float (&o)[8][4]) const {
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      const int i = mt >> 2, j = mt & 3;
      const uint32_t a = (&v[0][i].x)[j], b = (&v[1][i].x)[j], c = (&v[2][i].x)[j], d = (&v[3][i].x)[j];
      mma_16816_full(o[mt], prmt(a, b, 0x5410), prmt(a, b, 0x7632), prmt(c, d, 0x5410), prmt(c, d, 0x7632), b0, b1);
    }
  }
};

template <>
struct Page<ATW_F8> {
  static constexpr int BATCH = 1;
  uint4 k[2][2], v[4];
  float ks[2], vs[2];
  static __device__ __forceinline__ int qdim(int st, int t4, int r, int e) {
    return 64 * (st >> 2) + 16 * t4 + 4 * (st & 3) + 2 * r + e;
  }
  static __device__ __forceinline__ int odim(int mt, int g) { return 16 * g + 2 * mt; }
  static __device__ __forceinline__ LanePtrs lane_ptrs(const AtwArgs& a, int kvh, int g, int t4) {
    const uint8_t* k = static_cast<const uint8_t*>(a.k) + (size_t)kvh * ATT_SLICE;
    const uint8_t* v = static_cast<const uint8_t*>(a.v) + (size_t)kvh * ATT_SLICE;
    return {k + g * 128 + 16 * t4, v + 2 * t4 * 128 + 16 * g,
            reinterpret_cast<const uint8_t*>(a.ks + (size_t)kvh * ATT_PAGE + g),
            reinterpret_cast<const uint8_t*>(a.vs + (size_t)kvh * ATT_PAGE + g), (uint32_t)(a.Hkv * ATT_SLICE),
            (uint32_t)(a.Hkv * ATT_PAGE * 4)};
  }
  __device__ __forceinline__ void load_k(const LanePtrs& lp, int page) {
    const uint8_t* p = lp.at(lp.kc, page);
    const float* q = reinterpret_cast<const float*>(lp.at_scale(lp.ks, page));
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int i = 0; i < 2; ++i) k[r][i] = ldcg16(p + r * 1024 + 64 * i);
      ks[r] = __ldcg(q + 8 * r);
    }
  }
  __device__ __forceinline__ void load_v(const LanePtrs& lp, int page) {
    const uint8_t* p = lp.at(lp.vc, page);
    const float* q = reinterpret_cast<const float*>(lp.at_scale(lp.vs, page));
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = ldcg16(p + ((r & 1) + 8 * (r >> 1)) * 128);
#pragma unroll
    for (int r = 0; r < 2; ++r) vs[r] = __ldcg(q + 8 * r);
  }
  __device__ __forceinline__ void mask_v(uint32_t live, int g, int t4) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (!((live >> (2 * t4 + (r & 1) + 8 * (r >> 1))) & 1u)) v[r] = make_uint4(0u, 0u, 0u, 0u);
    if (!((live >> g) & 1u)) vs[0] = 0.f;
    if (!((live >> (g + 8)) & 1u)) vs[1] = 0.f;
  }
  __device__ __forceinline__ void scores(const uint32_t (&qb)[8][2], float (&s)[4]) const {
#pragma unroll
    for (int st = 0; st < 8; ++st) {
      uint32_t a0, a1, a2, a3;
      e4m3x4_to_h2x2((&k[0][st >> 2].x)[st & 3], a0, a2);
      e4m3x4_to_h2x2((&k[1][st >> 2].x)[st & 3], a1, a3);
      mma_16816_full(s, a0, a1, a2, a3, qb[st][0], qb[st][1]);
    }
  }
  __device__ __forceinline__ void score_scale(float (&s)[4]) const {
    s[0] *= ks[0];
    s[1] *= ks[0];
    s[2] *= ks[1];
    s[3] *= ks[1];
  }
  // V row scales go into P before its rounding
  __device__ __forceinline__ void p_scale(float (&p)[4]) const {
    const float f0 = vs[0] * ATW_V8, f1 = vs[1] * ATW_V8;
    p[0] *= f0;
    p[1] *= f0;
    p[2] *= f1;
    p[3] *= f1;
  }
  __device__ __forceinline__ void output(uint32_t b0, uint32_t b1, float (&o)[8][4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = (&v[0].x)[j], b = (&v[1].x)[j], c = (&v[2].x)[j], d = (&v[3].x)[j];
      uint32_t x[4], y[4];
      e4m3x4_to_h2x2(prmt(a, b, 0x5140), x[0], x[1]);
      e4m3x4_to_h2x2(prmt(a, b, 0x7362), x[2], x[3]);
      e4m3x4_to_h2x2(prmt(c, d, 0x5140), y[0], y[1]);
      e4m3x4_to_h2x2(prmt(c, d, 0x7362), y[2], y[3]);
      mma_16816_full(o[2 * j], x[0], x[1], y[0], y[1], b0, b1);
      mma_16816_full(o[2 * j + 1], x[2], x[3], y[2], y[3], b0, b1);
    }
  }
};

template <>
struct Page<ATW_I4> {
  static constexpr int BATCH = 2;
  uint4 k[2], v[2];
  uint32_t ks, vs;  // scale bytes: K tokens g, g + 8; V tokens 2 t4, 2 t4 + 1, 8 + 2 t4, 9 + 2 t4
  static __device__ __forceinline__ int qdim(int st, int t4, int r, int e) {
    return 32 * t4 + 8 * (st >> 1) + 2 * (st & 1) + r + 4 * e;
  }
  static __device__ __forceinline__ int odim(int mt, int g) { return 16 * g + 2 * mt; }
  static __device__ __forceinline__ LanePtrs lane_ptrs(const AtwArgs& a, int kvh, int g, int t4) {
    const uint8_t* k = static_cast<const uint8_t*>(a.k) + (size_t)kvh * KV4_SLICE;
    const uint8_t* v = static_cast<const uint8_t*>(a.v) + (size_t)kvh * KV4_SLICE;
    return {k + kv4_k_code(g, 8 * t4), v + kv4_v_code(2 * t4, 4 * g), k + kv4_k_scale(g, t4),
            v + kv4_v_scale(2 * t4, g >> 1), (uint32_t)(a.Hkv * KV4_SLICE), (uint32_t)(a.Hkv * KV4_SLICE)};
  }
  __device__ __forceinline__ void load_k(const LanePtrs& lp, int page) {
    const uint8_t* p = lp.at(lp.kc, page);
    k[0] = ldcg16(p);
    k[1] = ldcg16(p + 512);
    ks = __ldcg(reinterpret_cast<const unsigned short*>(lp.at(lp.ks, page)));
  }
  __device__ __forceinline__ void load_v(const LanePtrs& lp, int page) {
    const uint8_t* p = lp.at(lp.vc, page);
    v[0] = ldcg16(p);
    v[1] = ldcg16(p + 512);
    vs = __ldcg(reinterpret_cast<const unsigned int*>(lp.at(lp.vs, page)));
  }
  // a zero scale makes every code zero
  __device__ __forceinline__ void mask_v(uint32_t live, int, int t4) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (!((live >> (2 * t4 + (r & 1) + 8 * (r >> 1))) & 1u)) vs &= ~(0xFFu << (8 * r));
  }
  __device__ __forceinline__ void scores(const uint32_t (&qb)[8][2], float (&s)[4]) const {
    const Kv4Scale s0 = kv4_scale_pair((ks & 0xFFu) * 0x00800080u), s1 = kv4_scale_pair((ks >> 8) * 0x00800080u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t x[4], y[4];
      kv4_unpack((&k[0].x)[i], s0, x);
      kv4_unpack((&k[1].x)[i], s1, y);
      mma_16816_full(s, x[0], y[0], x[1], y[1], qb[2 * i][0], qb[2 * i][1]);
      mma_16816_full(s, x[2], y[2], x[3], y[3], qb[2 * i + 1][0], qb[2 * i + 1][1]);
    }
  }
  __device__ __forceinline__ void score_scale(float (&)[4]) const {}
  __device__ __forceinline__ void p_scale(float (&)[4]) const {}
  __device__ __forceinline__ void output(uint32_t b0, uint32_t b1, float (&o)[8][4]) const {
    const Kv4Scale s0 = kv4_scale_pair(prmt(vs, 0u, 0x4140) << 7), s1 = kv4_scale_pair(prmt(vs, 0u, 0x4342) << 7);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t x[4], y[4];
      kv4_unpack((&v[0].x)[j], s0, x);
      kv4_unpack((&v[1].x)[j], s1, y);
      mma_16816_full(o[2 * j], x[0], x[1], y[0], y[1], b0, b1);
      mma_16816_full(o[2 * j + 1], x[2], x[3], y[2], y[3], b0, b1);
    }
  }
  // the new token's row (codes and scales in shared memory) over what was loaded
  __device__ __forceinline__ void patch_k(const uint16_t* codes, const uint8_t* scale, int slot, int g, int t4) {
    if ((slot & 7) != g) return;
    const uint4 w = *reinterpret_cast<const uint4*>(codes + 8 * t4);
    if (slot < 8) k[0] = w;
    else k[1] = w;
    const int sh = 8 * (slot >> 3);
    ks = (ks & ~(0xFFu << sh)) | ((uint32_t)scale[t4] << sh);
  }
  __device__ __forceinline__ void patch_v(const uint16_t* codes, const uint8_t* scale, int slot, int g, int t4) {
    if (((slot & 7) >> 1) != t4) return;
    const uint32_t sel = (slot & 1) ? 0x5410u : 0x3254u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t c = codes[4 * g + j];
      if (slot < 8) (&v[0].x)[j] = prmt((&v[0].x)[j], c, sel);
      else (&v[1].x)[j] = prmt((&v[1].x)[j], c, sel);
    }
    const int sh = 8 * (2 * (slot >> 3) + (slot & 1));
    vs = (vs & ~(0xFFu << sh)) | ((uint32_t)scale[g >> 1] << sh);
  }
};

// factor of the accumulated scores and outputs
template <int KIND>
__device__ __forceinline__ constexpr float atw_s_factor() { return KIND == ATW_I4 ? 64.f : 1.f; }
template <int KIND>
__device__ __forceinline__ constexpr float atw_o_factor() { return KIND == ATW_I4 ? 64.f : (KIND == ATW_F8 ? 1.f / ATW_V8 : 1.f); }

template <int KIND, bool FUSE>
__global__ void __launch_bounds__(ATW_NW * 32, KIND == ATW_F16 ? 1 : 2) w4pg_attn_window(const __grid_constant__ AtwArgs a) {
  constexpr int NW = ATW_NW, BATCH = Page<KIND>::BATCH;
  __shared__ __align__(16) __half s_q[8][ATT_D + 8];
  __shared__ __align__(16) float s_o[NW * 8 * ATW_PITCH];  // [warp][head][128 + 4], dims in the order (mt, g, e)
  __shared__ float s_ml[NW * 8 * 2];
  __shared__ float s_cos[FUSE ? ATT_D / 2 : 1], s_sin[FUSE ? ATT_D / 2 : 1];
  __shared__ __align__(16) uint16_t s_new[FUSE ? 2 : 1][32];  // codes of the new K and V rows
  __shared__ uint8_t s_news[FUSE ? 2 : 1][4];
  __shared__ int s_last;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int pc = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int G = a.G;
  W4_TRACE_SCOPE(a.tag);
  pdl_wait_then_trigger();
  W4_TRACE_WAITED();

  // ---- the visible pages and this CTA's share -------------------------------
  int L = __ldcg(&a.context_lens[b]);
  const bool fits = L <= a.max_context;
  if (!fits) {
    if (pc == 0 && tid == 0 && a.err_flag) atomicOr(a.err_flag, 1);
    L = a.max_context;
  }
  L = max(L, 0);
  int w0 = a.window >= L ? 0 : L - a.window;  // first token of the window
  int S = min(a.sinks, L);                    // sinks
  if (w0 <= S) w0 = S = 0;                    // they meet: everything is seen
  const int nsp = (S + ATT_PAGE - 1) / ATT_PAGE;
  const int wp = max(w0 / ATT_PAGE, nsp);     // the window's first page that is not a sink page
  const int n = nsp + (w0 < L ? max((L + ATT_PAGE - 1) / ATT_PAGE - wp, 0) : 0);
  const int chunk = max((n + a.PC - 1) / a.PC, NW * BATCH);
  const int active = max((n + chunk - 1) / chunk, 1);
  if (pc >= active) return;
  const int v0 = pc * chunk, v1 = min(n, v0 + chunk);
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks;
  auto page_no = [&](int v) { return v < nsp ? v : v - nsp + wp; };

  // this warp takes BATCH consecutive pages of every NW * BATCH
  const int wv0 = v0 + warp * BATCH;
  const int steps = wv0 < v1 ? (v1 - wv0 + NW * BATCH - 1) / (NW * BATCH) : 0;
  auto table = [&](int i) {  // pool page of the warp's i-th page (-1: none, or not in the pool)
    const int v = wv0 + (i / BATCH) * NW * BATCH + i % BATCH;
    if (v >= v1) return -1;
    const int pn = page_no(v);
    const int id = pn < a.max_blocks ? __ldcg(&bt[pn]) : -1;
    if (id < 0 || id >= a.num_pages) {
      if (a.err_flag) atomicOr(a.err_flag, 1);
      return -1;
    }
    return id;
  };
  // 32 page ids at a time, one per lane
  int ids = table(lane), ids_next = -1;
  const LanePtrs lp = Page<KIND>::lane_ptrs(a, kvh, g, t4);

  // (a missing page loads page 0 in its place: its tokens are masked)
  Page<KIND> pg[BATCH];
  int cur[BATCH];
  auto fetch_ids = [&](int step) {
#pragma unroll
    for (int j = 0; j < BATCH; ++j) cur[j] = __shfl_sync(0xffffffffu, ids, (step * BATCH + j) & 31);
  };
  if (steps > 0) {
    fetch_ids(0);
#pragma unroll
    for (int j = 0; j < BATCH; ++j) pg[j].load_k(lp, max(cur[j], 0));
#pragma unroll
    for (int j = 0; j < BATCH; ++j) pg[j].load_v(lp, max(cur[j], 0));
  }
  // pages some of whose tokens are masked: the last of the sinks, the first of
  // the window, the last of the sequence (-1: none)
  const int part_s = S % ATT_PAGE ? nsp - 1 : -1;
  const int part_w = nsp < n && wp * ATT_PAGE < w0 ? nsp : -1;
  const int part_l = L % ATT_PAGE ? n - 1 : -1;

  // ---- queries ----------------------------------------------------------------
  const __half* qrow = a.q + (size_t)b * a.q_stride + (size_t)kvh * G * ATT_D;
  const int pos = fits ? L - 1 : -1;  // the new token's (fused); a length past the bound appends nothing
  if (FUSE) {
    if (tid < ATT_D / 2) sincosf(__fmul_rn((float)max(pos, 0), a.inv_freq[tid]), &s_sin[tid], &s_cos[tid]);
    __syncthreads();
    // a warp per query head; the CTA of the last page also takes the new K and V rows
    const bool last = pc == active - 1;
    for (int r = warp; r < 8 + (last ? 2 : 0); r += NW) {
      uint2 x = make_uint2(0u, 0u);
      const __half* src = r < 8 ? qrow + r * ATT_D
                                : a.q + (size_t)b * a.q_stride + (size_t)(a.Hq + (r - 8) * a.Hkv + kvh) * ATT_D;
      if (r < G || r >= 8) x = __ldcg(reinterpret_cast<const uint2*>(src) + lane);
      if (r != 9) rope_row4(x.x, x.y, s_cos, s_sin, lane);
      if (r < 8) {
        *reinterpret_cast<uint2*>(&s_q[r][4 * lane]) = x;
      } else {
        uint32_t codes, byte;
        kv4_quantise(x.x, x.y, codes, byte);
        s_new[r - 8][lane] = (uint16_t)codes;
        if ((lane & 7) == 0) s_news[r - 8][lane >> 3] = (uint8_t)byte;
        const int blk = max(pos, 0) / ATT_PAGE, slot = max(pos, 0) % ATT_PAGE;
        const int id = pos >= 0 && blk < a.max_blocks ? __ldcg(&bt[blk]) : -1;
        if (id >= 0 && id < a.num_pages) {
          uint8_t* sl = static_cast<uint8_t*>(const_cast<void*>(r == 8 ? a.k : a.v)) +
                        ((size_t)id * a.Hkv + kvh) * KV4_SLICE;
          *reinterpret_cast<uint16_t*>(sl + (r == 8 ? kv4_k_code(slot, lane) : kv4_v_code(slot, lane))) = (uint16_t)codes;
          if ((lane & 7) == 0)
            sl[r == 8 ? kv4_k_scale(slot, lane >> 3) : kv4_v_scale(slot, lane >> 3)] = (uint8_t)byte;
        }
      }
    }
  } else if (tid < 8 * ATT_D / 8) {
    const int h = tid / (ATT_D / 8), c = tid % (ATT_D / 8);
    *reinterpret_cast<uint4*>(&s_q[h][8 * c]) = h < G ? ldcg16(qrow + h * ATT_D + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();
  uint32_t qb[8][2];
#pragma unroll
  for (int st = 0; st < 8; ++st)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const __half lo = s_q[g][Page<KIND>::qdim(st, t4, r, 0)], hi = s_q[g][Page<KIND>::qdim(st, t4, r, 1)];
      qb[st][r] = ((uint32_t)__half_as_ushort(lo) | ((uint32_t)__half_as_ushort(hi) << 16)) ^
                  (a.scale_log2 < 0.f ? 0x80008000u : 0u);
    }
  W4_TRACE_MARK(0);

  // ---- pages --------------------------------------------------------------------
  const float scale = fabsf(a.scale_log2) * atw_s_factor<KIND>();  // (its sign is in the queries)
  float m0 = -INFINITY, m1 = -INFINITY;  // references of heads 2 t4 and 2 t4 + 1 (log2 domain)
  float l0 = 0.f, l1 = 0.f;              // this lane's part of their sums
  float o[8][4];                         // rows: dims odim(mt, g) + {0, 1}, columns: the two heads
#pragma unroll
  for (int mt = 0; mt < 8; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;

  for (int step = 0; step < steps; ++step) {
    const int v = wv0 + step * NW * BATCH;  // first visible page of this step
    // does any of these pages have masked tokens?
    bool masked = false;
#pragma unroll
    for (int j = 0; j < BATCH; ++j)
      masked |= cur[j] < 0 || v + j == part_s || v + j == part_w || v + j == part_l;
    uint32_t live[BATCH];  // bit r: token r of the page is seen
    if (masked) {
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        live[j] = 0u;
        const int t0 = page_no(v + j) * ATT_PAGE;
        if (cur[j] >= 0) {
          for (int r = 0; r < ATT_PAGE; ++r)
            live[j] |= (t0 + r < L && (t0 + r >= w0 || t0 + r < S) ? 1u : 0u) << r;
        }
      }
    }
    bool fresh[BATCH];  // fused: the page of the new token
    float s[BATCH][4];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      if constexpr (FUSE) {
        fresh[j] = v + j == n - 1 && pos >= 0;
        if (fresh[j]) pg[j].patch_k(s_new[0], s_news[0], pos & 15, g, t4);
      }
      s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
      pg[j].scores(qb, s[j]);
      pg[j].score_scale(s[j]);
    }
    const bool more = step + 1 < steps;
    if (more) {
      const int i = (step + 1) * BATCH;
      if ((i & 31) == 0) ids = ids_next;
      if ((i & 31) == BATCH) ids_next = table((i & ~31) + 32 + lane);
      fetch_ids(step + 1);
#pragma unroll
      for (int j = 0; j < BATCH; ++j) pg[j].load_k(lp, max(cur[j], 0));
    }
    if (masked) {
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        if (!((live[j] >> g) & 1u)) s[j][0] = s[j][1] = -INFINITY;
        if (!((live[j] >> (g + 8)) & 1u)) s[j][2] = s[j][3] = -INFINITY;
      }
    }
    float x0 = fmaxf(s[0][0], s[0][2]), x1 = fmaxf(s[0][1], s[0][3]);
#pragma unroll
    for (int j = 1; j < BATCH; ++j) {
      x0 = fmaxf(x0, fmaxf(s[j][0], s[j][2]));
      x1 = fmaxf(x1, fmaxf(s[j][1], s[j][3]));
    }
    x0 *= scale;
    x1 *= scale;
    if (__any_sync(0xffffffffu, x0 > m0 + ATW_SLACK || x1 > m1 + ATW_SLACK)) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
      }
      x0 = fmaxf(m0, x0);
      x1 = fmaxf(m1, x1);
      const float c0 = x0 == m0 ? 1.f : ex2(m0 - x0), c1 = x1 == m1 ? 1.f : ex2(m1 - x1);
      m0 = x0;
      m1 = x1;
      l0 *= c0;
      l1 *= c1;
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        o[mt][0] *= c0;
        o[mt][1] *= c1;
        o[mt][2] *= c0;
        o[mt][3] *= c1;
      }
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      s[j][0] = ex2(fmaf(s[j][0], scale, -m0));
      s[j][1] = ex2(fmaf(s[j][1], scale, -m1));
      s[j][2] = ex2(fmaf(s[j][2], scale, -m0));
      s[j][3] = ex2(fmaf(s[j][3], scale, -m1));
    }
    if (masked) {  // (-inf under a reference still at -inf is no number)
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        if (!((live[j] >> g) & 1u)) s[j][0] = s[j][1] = 0.f;
        if (!((live[j] >> (g + 8)) & 1u)) s[j][2] = s[j][3] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      l0 += s[j][0] + s[j][2];
      l1 += s[j][1] + s[j][3];
      if constexpr (FUSE) {
        if (fresh[j]) pg[j].patch_v(s_new[1], s_news[1], pos & 15, g, t4);
      }
    }
    if (masked) {
#pragma unroll
      for (int j = 0; j < BATCH; ++j) pg[j].mask_v(live[j], g, t4);
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      pg[j].p_scale(s[j]);
      const uint32_t b0 = movmatrix_trans(pack_h2(s[j][0], s[j][1])), b1 = movmatrix_trans(pack_h2(s[j][2], s[j][3]));
      pg[j].output(b0, b1, o);
    }
    if (more) {
#pragma unroll
      for (int j = 0; j < BATCH; ++j) pg[j].load_v(lp, max(cur[j], 0));
    }
  }
  W4_TRACE_MARK(1);

  // ---- the warps' states, merged in shared memory ------------------------------------
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
  }
  __syncthreads();
  const size_t qh0 = (size_t)b * a.Hq + (size_t)kvh * G;
  auto write_out = [&](int h, int i4, float4 acc) {  // positions 4 i4 .. 4 i4 + 3 of the order (mt, g, e)
    const int mt = i4 >> 2, g0 = 2 * (i4 & 3);
    __half* out = a.out + (qh0 + h) * ATT_D;
    *reinterpret_cast<__half2*>(out + Page<KIND>::odim(mt, g0)) = __floats2half2_rn(acc.x, acc.y);
    *reinterpret_cast<__half2*>(out + Page<KIND>::odim(mt, g0 + 1)) = __floats2half2_rn(acc.z, acc.w);
  };
  const bool single = active == 1;
  for (int idx = tid; idx < G * 32; idx += NW * 32) {
    const int h = idx >> 5, i4 = idx & 31;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, s_ml[(w * 8 + h) * 2]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float mw = s_ml[(w * 8 + h) * 2], lw = s_ml[(w * 8 + h) * 2 + 1];
      const float f = mw == -INFINITY ? (lw == 0.f ? 0.f : 1.f) : exp2f(mw - M);
      const float4 v = *reinterpret_cast<const float4*>(s_o + (w * 8 + h) * ATW_PITCH + 4 * i4);
      acc.x = fmaf(v.x, f, acc.x);
      acc.y = fmaf(v.y, f, acc.y);
      acc.z = fmaf(v.z, f, acc.z);
      acc.w = fmaf(v.w, f, acc.w);
      den = fmaf(lw, f, den);
    }
    if (single) {
      const float inv = den == 0.f ? 0.f : atw_o_factor<KIND>() / den;
      write_out(h, i4, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    } else {
      *reinterpret_cast<float4*>(a.ws_o + ((qh0 + h) * a.PC + pc) * ATT_D + 4 * i4) = acc;
      if (i4 == 0) *reinterpret_cast<float2*>(a.ws_ml + ((qh0 + h) * a.PC + pc) * 2) = make_float2(M, den);
    }
  }
  if (single) return;

  // ---- the CTAs' partials: the last to finish adds them up, in order ----------------
  __threadfence();
  __syncthreads();
  if (tid == 0) s_last = atomicAdd(&a.counters[(size_t)b * a.Hkv + kvh], 1u) == (unsigned)(active - 1);
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  for (int idx = tid; idx < G * 32; idx += NW * 32) {
    const int h = idx >> 5, i4 = idx & 31;
    const float2* ml = reinterpret_cast<const float2*>(a.ws_ml + (qh0 + h) * a.PC * 2);
    float M = -INFINITY;
    for (int j = 0; j < active; ++j) M = fmaxf(M, __ldcg(ml + j).x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
    const float4* src = reinterpret_cast<const float4*>(a.ws_o + (qh0 + h) * a.PC * ATT_D) + i4;
#pragma unroll 4
    for (int j = 0; j < active; ++j) {
      const float2 e = __ldcg(ml + j);
      const float f = e.x == -INFINITY ? (e.y == 0.f ? 0.f : 1.f) : exp2f(e.x - M);
      const float4 v = __ldcg(src + (size_t)j * (ATT_D / 4));
      acc.x = fmaf(v.x, f, acc.x);
      acc.y = fmaf(v.y, f, acc.y);
      acc.z = fmaf(v.z, f, acc.z);
      acc.w = fmaf(v.w, f, acc.w);
      den = fmaf(e.y, f, den);
    }
    const float inv = den == 0.f ? 0.f : atw_o_factor<KIND>() / den;
    write_out(h, i4, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  }
  if (tid == 0) a.counters[(size_t)b * a.Hkv + kvh] = 0u;  // ready for the next call
}

// CTAs per (sequence, kv head): enough for two per SM over the batch, no more
// than the visible pages can feed with a step for every warp.
int atw_partitions(int B, int Hkv, int max_context, int window, int sinks) {
  const long long all = ((long long)max_context + ATT_PAGE - 1) / ATT_PAGE;
  const long long seen = ((long long)std::min(sinks, max_context) + ATT_PAGE - 1) / ATT_PAGE +
                         ((long long)window + ATT_PAGE - 2) / ATT_PAGE + 1;
  const long long n = std::min(all, seen);
  const long long want = (2ll * ATW_SMS + (long long)B * Hkv - 1) / ((long long)B * Hkv);
  const long long most = (n + ATW_NW - 1) / ATW_NW;
  return (int)std::max(1ll, std::min(std::min(want, most), (long long)ATW_MAX_PARTITIONS));
}

template <int KIND, bool FUSE>
static int launch_atw(const AtwArgs& a, cudaStream_t s) {
  cudaError_t e = launch_pdl(w4pg_attn_window<KIND, FUSE>, dim3(a.PC, a.Hkv, a.B), dim3(ATW_NW * 32), 0, s, a);
  if (e != cudaSuccess) return set_error(W4A16_ERR_CUDA, "paged attention launch: %s", cudaGetErrorString(e));
  return W4A16_OK;
}

int launch_attn_window(const AtwArgs& a, cudaStream_t s) {
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
  W4_CHECK_SHAPE(B <= 65535 && Hkv <= 65535, "%s: B=%d Hkv=%d", who, B, Hkv);
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
  a.PC = atw_partitions(B, Hkv, max_context, window, sinks);
  if (a.PC > 1) {
    const size_t need = attention_workspace_bytes(B, Hq, Hkv, a.PC);
    W4_CHECK_ARG(workspace != nullptr && workspace_bytes >= need, "%s: workspace of %zu bytes needed", who, need);
    W4_CHECK_ALIGN(workspace, 128, "workspace");
    atw_workspace(a, workspace, B, Hq);
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
  if (B < 1 || Hq < 1 || Hkv < 1 || max_context < 1 || window < 0 || sinks < 0) return 0;
  return attention_workspace_bytes(B, Hq, Hkv, atw_partitions(B, Hkv, max_context, window, sinks));
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

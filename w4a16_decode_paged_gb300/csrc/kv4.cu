// kv4.cu -- writing INT4 KV pages (RoPE + quantised append) and reading them
// back.  Format and quantiser: kv4.cuh.
//
// Both only move data: an appended row is Hq + 2 Hkv head rows of 256 bytes in,
// Hq of them out again and 2 Hkv x 68 bytes of codes and scales; a token read
// back is 136 bytes in and 512 out per kv head.  A few rows are bound by the
// chain of latencies (length, table entry, page: 2.5 us a call), a prompt's
// rows by that chain and their instructions one after the other (2048 rows are
// 512 CTAs, resident at once and in step: loads, sines, rotation; 0.58 of the
// issue slots used), a whole cache read back by one burst of stores behind that chain
// (9 MB in, 33.5 MB out in 9.5 us, 4.5 TB/s; half the instructions, with whole
// pages stored unchecked, measured the same).
#include "kernels.h"
#include "kv4.cuh"

namespace w4 {

// ---------------------------------------------------------------------------
// RoPE + INT4 append: R rows (of the batch or the prompt) per CTA, 8 / R warps
// each.  A row's head rows -- q (rotated), k (rotated, quantised), v
// (quantised) -- are taken two at a time by a warp, eight dims per lane.  The
// values do not depend on the position, so the first of them are asked for
// before the length and the table entry are read and the sines computed; the
// next are asked for as these are finished.
// ---------------------------------------------------------------------------
constexpr int APPEND_WARPS = 8;
constexpr int APPEND_AHEAD = 3;  // row pairs a warp loads ahead

template <int R>
__global__ void __launch_bounds__(APPEND_WARPS * 32, 4) w4pg_rope_append_int4(const __grid_constant__ Kv4AppendArgs a) {
  constexpr int PER = APPEND_WARPS / R;  // warps per row
  __shared__ __align__(16) float s_cos[R][KV4_D / 2], s_sin[R][KV4_D / 2];
  __shared__ int s_slot[R], s_page[R];  // page -1: none; slot -1: a row of length 0
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int u = warp / PER, w0 = warp % PER;
  const int c = lane & 15, half = lane >> 4;
  const size_t b = (size_t)blockIdx.x * R + u;
  const int rows = b < (size_t)a.B ? a.Hq + 2 * a.Hkv : 0;
  const __half* qb = a.q + b * a.stride_q + 8 * c;
  const __half* kb = a.k + b * a.stride_kv + 8 * c;
  const __half* vb = a.v + b * a.stride_kv + 8 * c;
  auto load = [&](int r) -> uint4 {
    if (r >= rows) return make_uint4(0u, 0u, 0u, 0u);
    const __half* src = r < a.Hq ? qb + (size_t)r * KV4_D
                                 : (r < a.Hq + a.Hkv ? kb + (size_t)(r - a.Hq) * KV4_D
                                                     : vb + (size_t)(r - a.Hq - a.Hkv) * KV4_D);
    return __ldcg(reinterpret_cast<const uint4*>(src));
  };
  pdl_wait_then_trigger();
  uint4 x[APPEND_AHEAD];
#pragma unroll
  for (int k = 0; k < APPEND_AHEAD; ++k) x[k] = load(2 * (w0 + k * PER) + half);
  for (int i = tid; i < R * (KV4_D / 2); i += APPEND_WARPS * 32) {
    const int v = i / (KV4_D / 2), f = i % (KV4_D / 2), bv = blockIdx.x * R + v;
    const int pos = bv < a.B ? max(__ldcg(&a.context_lens[bv]), 0) - 1 : -1;
    if (f == 0) {
      const int blk = pos / KV4_PAGE;
      const int page = pos >= 0 && blk < a.max_blocks ? __ldcg(&a.block_table[(size_t)bv * a.max_blocks + blk]) : -1;
      const bool ok = page >= 0 && page < a.num_pages;
      if (pos >= 0 && !ok && a.err_flag) atomicOr(a.err_flag, 1);
      s_page[v] = ok ? page : -1;
      s_slot[v] = pos >= 0 ? pos % KV4_PAGE : -1;
    }
    sincosf(__fmul_rn((float)max(pos, 0), a.inv_freq[f]), &s_sin[v][f], &s_cos[v][f]);
  }
  __syncthreads();
  const int slot = s_slot[u], page = s_page[u];
  if (slot < 0) return;
  RopeLane rope;
  rope.load(s_cos[u], s_sin[u], lane);
  for (int r0 = 2 * w0; r0 < rows; r0 += 2 * PER * APPEND_AHEAD) {
#pragma unroll
    for (int k = 0; k < APPEND_AHEAD; ++k) {
      const int pair = r0 + 2 * k * PER, r = pair + half;
      if (pair >= rows) break;
      const bool is_q = r < a.Hq, is_k = !is_q && r < a.Hq + a.Hkv;
      // (a warp's two rows may be of two kinds)
      uint4 w = x[k];
      if (pair < a.Hq + a.Hkv) rope_rows(w, rope);
      if (!is_q && !is_k) w = x[k];
      uint32_t codes = 0u, byte = 0u;
      if (pair + 1 >= a.Hq) kv4_quantise(w, codes, byte);
      if (is_q) {
        *reinterpret_cast<uint4*>(a.q_out + b * a.stride_qo + (size_t)r * KV4_D + 8 * c) = w;
      } else if (page >= 0 && r < rows) {
        const int h = is_k ? r - a.Hq : r - a.Hq - a.Hkv;
        kv4_put((is_k ? a.k_pool : a.v_pool) + ((size_t)page * a.Hkv + h) * KV4_SLICE, is_k, slot, c, codes, byte);
      }
      x[k] = load(r + 2 * PER * APPEND_AHEAD);
    }
  }
}

// One row per CTA as long as two per SM hold them (a decode batch: the shortest
// chain of latencies, 2.5 us); four where a prompt's rows would queue behind each
// other's chains (2048 rows of 28 + 2 x 4 heads, with the read back of them all:
// 20.3 us with one row per CTA, 14.6 with two, 13.2 with four).
int launch_rope_append_int4(const Kv4AppendArgs& a, cudaStream_t s) {
  cudaError_t e;
  if (a.B <= 2 * num_sms()) e = launch_pdl(w4pg_rope_append_int4<1>, dim3(a.B), dim3(APPEND_WARPS * 32), 0, s, a);
  else e = launch_pdl(w4pg_rope_append_int4<4>, dim3((a.B + 3) / 4), dim3(APPEND_WARPS * 32), 0, s, a);
  if (e != cudaSuccess) return set_error(W4A16_ERR_CUDA, "int4 rope/append launch: %s", cudaGetErrorString(e));
  return W4A16_OK;
}

// ---------------------------------------------------------------------------
// Read back: a warp per (page, kv head).  A lane takes eight dims, so that a
// warp's stores are whole rows of 256 bytes; a page's 2176 bytes are asked for
// at once (16384 tokens x 4 heads: 9.5 us; 14.5 with the loads beside their use).
// ---------------------------------------------------------------------------
struct Kv4ReadArgs {
  const uint8_t *k_pool, *v_pool;
  const int32_t *block_table, *starts, *context_lens;
  __half *k_out, *v_out;  // [B][T][Hkv][D]
  int32_t* err_flag;
  int num_pages, max_blocks, T, Hkv, pages_max;  // pages_max: pages that T rows can touch
  int clear;  // rows that hold no token become zero
};

// a word of codes times its scale(s): the pairs (n, n + 4) of its nibbles as
// fp16 values.  two: the fp16 bits of the low and the high half's scale.
__device__ __forceinline__ void kv4_values(uint32_t word, const Kv4Scale& k, const Kv4Bias& e, uint32_t (&x)[4]) {
  kv4_unpack(word, k, e, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = hmul2_u(x[i], 0x54005400u);  // 64: the unpacking's scales are s / 64
}
__device__ __forceinline__ uint32_t lows(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t highs(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

__global__ void __launch_bounds__(256) w4pg_read_int4(const __grid_constant__ Kv4ReadArgs a) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait_then_trigger();
  const int h = (int)(item % a.Hkv);
  const long long pi = item / a.Hkv;
  if (pi >= a.pages_max) return;
  const long long L = __ldcg(&a.context_lens[b]);
  const long long first = a.starts ? __ldcg(&a.starts[b]) : 0;
  const long long blk = (first >> 4) + pi;  // (rounds down for negative starts too)
  const long long lo = blk * KV4_PAGE, hi = lo + KV4_PAGE;
  if (lo >= first + a.T) return;
  const bool live = lo < L && hi > 0;  // the page holds a token of the sequence
  if (!live && !a.clear) return;
  const int page = live && blk < a.max_blocks ? __ldcg(&a.block_table[(size_t)b * a.max_blocks + blk]) : -1;
  const bool ok = page >= 0 && page < a.num_pages;
  if (live && !ok) {
    if (lane == 0 && a.err_flag) atomicOr(a.err_flag, 1);
    if (!a.clear) return;
  }
  const size_t off = ((size_t)(ok ? page : 0) * a.Hkv + h) * KV4_SLICE;
  const uint8_t* ks = a.k_pool + off;
  const uint8_t* vs = a.v_pool + off;
  const int c = lane & 15, half = lane >> 4;  // dims 8 c .. 8 c + 7
  const size_t pitch = (size_t)a.Hkv * KV4_D;
  const size_t out0 = ((size_t)b * a.T * a.Hkv + h) * KV4_D + 8 * c;
  // everything the lane needs of the page, in one go: K words of eight dims of
  // tokens 2 i + half, V word pairs of the token pairs 4 i + 2 half, and the
  // scale bytes (K: those of tokens t and t + 8; V: of two token pairs)
  uint32_t kw[8], ksc[4], vsc[2];
  uint2 vw[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) kw[i] = __ldcg(reinterpret_cast<const uint32_t*>(ks + kv4_k_code(2 * i + half, 2 * c)));
#pragma unroll
  for (int i = 0; i < 4; ++i) vw[i] = __ldcg(reinterpret_cast<const uint2*>(vs + kv4_v_code(4 * i + 2 * half, 2 * c)));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    ksc[i] = __ldcg(reinterpret_cast<const unsigned short*>(ks + kv4_k_scale(2 * i + half, c >> 2)));
#pragma unroll
  for (int i = 0; i < 2; ++i) vsc[i] = __ldcg(reinterpret_cast<const uint32_t*>(vs + kv4_v_scale(4 * i + 2 * half, c >> 2)));
  const Kv4Bias bias;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  // row of token t of the page: the token's value, zero, or left alone
  auto put = [&](__half* out, int t, uint4 value) {
    const long long tok = lo + t, row = tok - first;
    if (row < 0 || row >= a.T) return;
    const bool holds = ok && tok >= 0 && tok < L;
    if (holds || a.clear) *reinterpret_cast<uint4*>(out + out0 + (size_t)row * pitch) = holds ? value : zero;
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t s = i < 4 ? ksc[i] & 0xFFu : ksc[i - 4] >> 8;
    uint32_t x[4];
    kv4_values(kw[i], kv4_scale_pair(s * 0x00800080u), bias, x);
    put(a.k_out, 2 * i + half, make_uint4(lows(x[0], x[1]), lows(x[2], x[3]), highs(x[0], x[1]), highs(x[2], x[3])));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 4 * i + 2 * half;
    const uint32_t s = vsc[i & 1] >> (i < 2 ? 0 : 16);
    const Kv4Scale k = kv4_scale_pair(((s & 0xFFu) << 7) | ((s & 0xFF00u) << 15));
    uint32_t x[4], y[4];
    kv4_values(vw[i].x, k, bias, x);
    kv4_values(vw[i].y, k, bias, y);
    put(a.v_out, t, make_uint4(lows(x[0], x[1]), lows(x[2], x[3]), lows(y[0], y[1]), lows(y[2], y[3])));
    put(a.v_out, t + 1, make_uint4(highs(x[0], x[1]), highs(x[2], x[3]), highs(y[0], y[1]), highs(y[2], y[3])));
  }
}

}  // namespace w4

using namespace w4;

extern "C" int kv_append_rope_int4(uint16_t* q, const uint16_t* k, const uint16_t* v, int row_stride, uint16_t* q_out,
                                   uint8_t* k_pool, uint8_t* v_pool, int num_pages, const int32_t* block_table,
                                   int max_blocks, const int32_t* context_lens, int B, int Hq, int Hkv, int D,
                                   float theta, int32_t* err_flag, w4a16_stream_t stream) {
  W4_CHECK_ARG(q && k && v && k_pool && v_pool && block_table && context_lens, "kv_append_rope_int4: null pointer");
  W4_CHECK_ARG(B >= 1 && Hq >= 1 && Hkv >= 1 && num_pages >= 1 && max_blocks >= 1, "kv_append_rope_int4: sizes");
  W4_CHECK_SHAPE(D == KV4_D, "kv_append_rope_int4: D=%d, only 128 is built", D);
  W4_CHECK_SHAPE(Hq % Hkv == 0 && Hq <= (1 << 20), "kv_append_rope_int4: Hq=%d Hkv=%d", Hq, Hkv);
  W4_CHECK_ARG(theta > 0.f, "kv_append_rope_int4: theta must be positive");
  W4_CHECK_ARG(row_stride == 0 || (row_stride % 8 == 0 && row_stride >= Hq * D),
               "kv_append_rope_int4: row_stride must be 0 or a multiple of 8 that holds a q row");
  W4_CHECK_ALIGN(q, 128, "q");
  W4_CHECK_ALIGN(k, 128, "k");
  W4_CHECK_ALIGN(v, 128, "v");
  W4_CHECK_ALIGN(q_out, 128, "q_out");
  W4_CHECK_ALIGN(k_pool, 128, "k_pool");
  W4_CHECK_ALIGN(v_pool, 128, "v_pool");
  Kv4AppendArgs a = {};
  a.q = reinterpret_cast<const __half*>(q);
  a.k = reinterpret_cast<const __half*>(k);
  a.v = reinterpret_cast<const __half*>(v);
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.block_table = block_table;
  a.context_lens = context_lens;
  a.err_flag = err_flag;
  a.stride_q = row_stride ? row_stride : Hq * D;
  a.stride_kv = row_stride ? row_stride : Hkv * D;
  a.q_out = reinterpret_cast<__half*>(q_out ? q_out : q);
  a.stride_qo = q_out ? Hq * D : a.stride_q;
  a.num_pages = num_pages;
  a.max_blocks = max_blocks;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  rope_inv_freq_table(theta, D, a.inv_freq);
  return launch_rope_append_int4(a, (cudaStream_t)stream);
}

extern "C" int kv_read_int4(const uint8_t* k_pool, const uint8_t* v_pool, int num_pages, const int32_t* block_table,
                            int max_blocks, const int32_t* starts, const int32_t* context_lens, int T, int B, int Hkv,
                            int D, uint16_t* k_out, uint16_t* v_out, int clear, int32_t* err_flag,
                            w4a16_stream_t stream) {
  W4_CHECK_ARG(clear == 0 || clear == 1, "kv_read_int4: clear=%d", clear);
  W4_CHECK_ARG(k_pool && v_pool && block_table && context_lens && k_out && v_out, "kv_read_int4: null pointer");
  W4_CHECK_ARG(T >= 1 && B >= 1 && Hkv >= 1 && num_pages >= 1 && max_blocks >= 1, "kv_read_int4: sizes");
  W4_CHECK_SHAPE(D == KV4_D, "kv_read_int4: D=%d, only 128 is built", D);
  W4_CHECK_SHAPE(B <= 65535, "kv_read_int4: B=%d > 65535", B);
  W4_CHECK_ALIGN(k_pool, 128, "k_pool");
  W4_CHECK_ALIGN(v_pool, 128, "v_pool");
  W4_CHECK_ALIGN(k_out, 128, "k_out");
  W4_CHECK_ALIGN(v_out, 128, "v_out");
  Kv4ReadArgs a = {};
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.block_table = block_table;
  a.starts = starts;
  a.context_lens = context_lens;
  a.k_out = reinterpret_cast<__half*>(k_out);
  a.v_out = reinterpret_cast<__half*>(v_out);
  a.err_flag = err_flag;
  a.num_pages = num_pages;
  a.max_blocks = max_blocks;
  a.T = T;
  a.Hkv = Hkv;
  a.clear = clear;
  a.pages_max = (int)(((long long)T + KV4_PAGE - 2) / KV4_PAGE + 1);  // that T consecutive tokens can touch
  const long long ctas = ((long long)a.pages_max * Hkv + 7) / 8;
  W4_CHECK_SHAPE(ctas <= 0x7FFFFFFFll, "kv_read_int4: T=%d x Hkv=%d is too large", T, Hkv);
  cudaError_t e = launch_pdl(w4pg_read_int4, dim3((unsigned)ctas, (unsigned)B), dim3(256), 0, (cudaStream_t)stream, a);
  if (e != cudaSuccess) return set_error(W4A16_ERR_CUDA, "kv_read_int4 launch: %s", cudaGetErrorString(e));
  return W4A16_OK;
}

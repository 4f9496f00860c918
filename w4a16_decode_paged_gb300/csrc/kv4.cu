// kv4.cu -- writing INT4 KV pages (RoPE + quantised append) and reading them
// back.  Format and quantiser: kv4.cuh.
#include "kernels.h"
#include "kv4.cuh"

namespace w4 {

// ---------------------------------------------------------------------------
// RoPE + INT4 append: one CTA per row.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) w4pg_rope_append_int4(const __grid_constant__ Kv4AppendArgs a) {
  __shared__ float s_cos[KV4_D / 2], s_sin[KV4_D / 2];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait_then_trigger();
  const int pos = __ldcg(&a.context_lens[b]) - 1;
  if (pos < 0) return;
  if (tid < KV4_D / 2) sincosf(__fmul_rn((float)pos, a.inv_freq[tid]), &s_sin[tid], &s_cos[tid]);
  const int blk = pos / KV4_PAGE, slot = pos % KV4_PAGE;
  const int page = blk < a.max_blocks ? __ldcg(&a.block_table[(size_t)b * a.max_blocks + blk]) : -1;
  const bool ok = page >= 0 && page < a.num_pages;
  if (!ok && tid == 0 && a.err_flag) atomicOr(a.err_flag, 1);
  __syncthreads();
  // rows: q heads (rotated), k heads (rotated, quantised), v heads (quantised),
  // one warp each, four dims per lane
  const int rows = a.Hq + 2 * a.Hkv;
  for (int r = warp; r < rows; r += 8) {
    const bool is_q = r < a.Hq, is_k = !is_q && r < a.Hq + a.Hkv;
    if (!is_q && !ok) break;
    const int h = is_q ? r : (is_k ? r - a.Hq : r - a.Hq - a.Hkv);
    const __half* src = is_q ? a.q + (size_t)b * a.stride_q : (is_k ? a.k : a.v) + (size_t)b * a.stride_kv;
    uint2 x = *reinterpret_cast<const uint2*>(src + (size_t)h * KV4_D + 4 * lane);
    if (is_q || is_k) rope_row4(x.x, x.y, s_cos, s_sin, lane);
    if (is_q) {
      *reinterpret_cast<uint2*>(a.q_out + (size_t)b * a.stride_qo + (size_t)h * KV4_D + 4 * lane) = x;
      continue;
    }
    uint32_t codes, byte;
    kv4_quantise(x.x, x.y, codes, byte);
    uint8_t* sl = (is_k ? a.k_pool : a.v_pool) + ((size_t)page * a.Hkv + h) * KV4_SLICE;
    *reinterpret_cast<uint16_t*>(sl + (is_k ? kv4_k_code(slot, lane) : kv4_v_code(slot, lane))) = (uint16_t)codes;
    if ((lane & 7) == 0)
      sl[is_k ? kv4_k_scale(slot, lane >> 3) : kv4_v_scale(slot, lane >> 3)] = (uint8_t)byte;
  }
}

int launch_rope_append_int4(const Kv4AppendArgs& a, cudaStream_t s) {
  cudaError_t e = launch_pdl(w4pg_rope_append_int4, dim3(a.B), dim3(256), 0, s, a);
  if (e != cudaSuccess) return set_error(W4A16_ERR_CUDA, "int4 rope/append launch: %s", cudaGetErrorString(e));
  return W4A16_OK;
}

// ---------------------------------------------------------------------------
// Read back: a warp per (page, kv head).  A lane takes eight dims, so that a
// warp's stores are whole rows of 256 bytes.
// ---------------------------------------------------------------------------
struct Kv4ReadArgs {
  const uint8_t *k_pool, *v_pool;
  const int32_t *block_table, *starts, *context_lens;
  __half *k_out, *v_out;  // [B][T][Hkv][D]
  int32_t* err_flag;
  int num_pages, max_blocks, T, Hkv, pages_max;  // pages_max: pages that T rows can touch
  int clear;  // rows that hold no token become zero
};

// eight dims of one token (two code halfwords) times their scale, as 16 bytes
__device__ __forceinline__ uint4 kv4_eight(uint32_t lo4, uint32_t hi4, float s) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = ((i < 2 ? lo4 : hi4) >> (8 * (i & 1))) & 0xFFu;
    const __half2 h = __floats2half2_rn(((int)(c & 15u) - 8) * s, ((int)(c >> 4) - 8) * s);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

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
    const int t = 2 * i + half;  // K: two tokens per step
    const uint32_t w = *reinterpret_cast<const uint32_t*>(ks + kv4_k_code(t, 2 * c));
    put(a.k_out, t, kv4_eight(w & 0xFFFFu, w >> 16, kv4_scale_value(ks[kv4_k_scale(t, c >> 2)])));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 4 * i + 2 * half;  // V: two token pairs per step
    const uint2 w = *reinterpret_cast<const uint2*>(vs + kv4_v_code(t, 2 * c));
    put(a.v_out, t, kv4_eight(w.x & 0xFFFFu, w.y & 0xFFFFu, kv4_scale_value(vs[kv4_v_scale(t, c >> 2)])));
    put(a.v_out, t + 1, kv4_eight(w.x >> 16, w.y >> 16, kv4_scale_value(vs[kv4_v_scale(t + 1, c >> 2)])));
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
  W4_CHECK_SHAPE(Hq % Hkv == 0, "kv_append_rope_int4: Hq %% Hkv != 0");
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

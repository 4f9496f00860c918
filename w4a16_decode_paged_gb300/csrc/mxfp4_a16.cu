// mxfp4_a16.cu -- products of many fp16 rows (a decode batch, a prompt) with MXFP4
// weights on the 5th-generation tensor cores.
//
// y[m][n] = sum_k x[m][k] w[n][k], w = c 2^(b - 127) an fp16 number exactly, so the
// MMA's operands are x as it is and the weights expanded: the expander warps
// convert codes (hardware E2M1 to fp16 pairs), apply the block's scale with one
// packed multiplication, and store the tile in tensor memory, from which the MMA
// takes its A operand (weights as rows: D[n][m], 128 lanes x NC columns, fp32).
// The whole of K is summed in tensor memory; nothing is read out before the end.
//
// A CTA's tile is 2 x 128 weight rows (two neighbouring tiles, or gate and up) x
// NC rows of x, so that a stage (128 k) of x, its largest operand, serves 256
// weight rows: at NC = 128 49 KB for 1024 cycles of MMAs.  NC = 32 and 64 are for
// decode batches and short prompts, where the weights' bytes decide.
//
// Roles (18 warps), meeting only at mbarriers: a producer lane copies codes,
// scales and x into a ring; two sets of 8 expander warps (lane quadrant, tile) take
// the stages in turn and fill one of NAB tensor-memory A buffers each, so that one
// set's waits lie under the other's work; one warp issues the MMAs; the expander
// warps run the epilogue, turning 8 columns at a time through shared memory, so
// that stores (and the residual's loads) are 16 bytes of a row of y.  Tiles are
// dealt by mt_deal.
//
// What bounds it, by copies that leave work out: a stage of 32 rows of x takes 0.51 us in
// a call of 28 stages (0.45 between 28 and 56, 5.9 TB/s),
// 0.42 without the conversions, which is the DRAM's rate (38 conversions and more a clock
// and SM would be 0.21 alone; no pipe is over 0.39, and the warps' largest stall is
// waiting for shared and tensor memory, 2.8 of 9.2 cycles); of 64 rows 0.61, 0.54 without
// the conversions and 0.48 without the stores as well; of 128 rows 0.80 to 0.83, 0.74
// without both, where a bf16 product of that size takes 0.65 at the rate of a large one.
// 32 rows, 18944 x 3584 twice, with SiLU 19.0 us; 2048 rows, 3584 x 3584 49.5 us, 18944
// x 3584 199 us (1397 TFLOP/s).  A tile's first two stages under the one before's last
// MMAs and ahead of its epilogue: 203.9 us to 198.1 there, 47.8 to 42.0 at 4096 rows, 8960
// x 256; where a CTA has one tile only it costs up to 2 % (300 rows, 3584 x 3584 16.7 us to
// 17.0).  A stage handed over by halves 0.67 (32 rows) and 0.83
// us; direct 2-byte stores 5.4 us an epilogue, turned 4.3.
#include "mxfp4_tc.cuh"

namespace w4 {

constexpr int MA_K = 128;                    // k of a stage: one scale tile's width
constexpr int MA_EXP = 16;                   // expander warps
constexpr int MA_THREADS = 64 + 32 * MA_EXP;
constexpr uint32_t MA_W = 128 * MA_K / 2;    // bytes of a tile's codes per stage

template <int NC>
struct MaShape {
  static constexpr uint32_t XHALF = NC * 128;                         // 64 k of x, 128-byte rows
  static constexpr uint32_t WAT = 2 * XHALF, SAT = WAT + 2 * MA_W;    // a slot: x, codes, scales
  static constexpr uint32_t SLOT = SAT + 2 * MX_TILE;
  static constexpr int S = 204800 / SLOT;
  static constexpr size_t SMEM = S * SLOT + MA_EXP * 1024 + 1024;     // + a warp's 8 columns x 32 rows, fp32
  static constexpr int NAB = (512 - 2 * NC) / 128 > 3 ? 3 : (512 - 2 * NC) / 128;
  static constexpr int TA = 2 * NC;                                   // tensor memory: sums, then A buffers
  static constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(NC >> 3) << 17) | ((128u >> 4) << 24);
  static_assert(SLOT % 1024 == 0 && NAB >= 2 && S >= 4, "swizzled tiles start on 1024-byte boundaries");
};

struct MaArgs {
  MxArgs a;
  int silu, mtiles, ntiles, whole, split, items;   // ntiles: of 128 weight rows; items as mt_deal
  float* parts;
  CUtensorMap tm_w[2], tm_x;
};

__device__ __forceinline__ void mx_tmem_ld8(float (&v)[8], uint32_t taddr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "r"(taddr));
}

template <int NC>
__global__ void __launch_bounds__(MA_THREADS, 1) w4pg_mxfp4_a16(const __grid_constant__ MaArgs p) {
  using SH = MaShape<NC>;
  constexpr int S = SH::S, NAB = SH::NAB;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const unsigned char* ringp = smem_raw + (ring - smem_u32(smem_raw));
  __shared__ __align__(8) uint64_t full[S], empty[S], afull[NAB], aempty[NAB], dfull, dempty, drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int s_fail;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int K = p.a.K, stages = K / MA_K, KT = K / 128;

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 32) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], MA_EXP / 2 + 1);
    }
    for (int i = 0; i < NAB; ++i) {
      mbar_init(&afull[i], MA_EXP / 2);
      mbar_init(&aempty[i], 1);
    }
    mbar_init(&dfull, 1);
    mbar_init(&dempty, MA_EXP);
    mbar_init(&drain, 1);
    s_fail = 0;
    fence_mbar_init();
  }
  mt_fence_before();
  __syncthreads();
  mt_fence_after();
  const uint32_t tmem = tmem_slot;

  // item -> its m tile, first 128-row weight tile (and the second's distance), part, k range
  auto item = [&](int i, int* mt, int* nt, int* part, int* k0, int* k1) {
    int tile;
    mt_item(i, p.whole, p.split, stages, &tile, part, k0, k1);
    *mt = tile % p.mtiles;
    *nt = tile / p.mtiles * (p.silu ? 1 : 2);
    return tile;
  };

  if (warp == 0) {
    // ---- producer ----
    if (mt_elect()) {
      mt_prefetch_map(&p.tm_w[0]);
      if (p.silu) mt_prefetch_map(&p.tm_w[1]);
      mt_prefetch_map(&p.tm_x);
      int mt, nt, part, k0, k1;
      if (blockIdx.x < p.items) {
        // weights may come from the call just before: into L2 ahead of the wait, read behind it
        item(blockIdx.x, &mt, &nt, &part, &k0, &k1);
        for (int k = k0; k < min(k1, k0 + S); ++k)
          for (int g = 0; g < 2; ++g) mt_prefetch_2d(&p.tm_w[p.silu ? g : 0], k * (MA_K / 8), (p.silu ? nt : nt + g) * 128);
      }
      pdl_wait_then_trigger();
      uint32_t s = 0;
      bool ok = true;
      for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x) {
        item(i, &mt, &nt, &part, &k0, &k1);
        for (int k = k0; k < k1; ++k, ++s) {
          const int slot = s % S;
          if (s >= S && !(ok = mt_wait(&empty[slot], (s / S - 1) & 1, &s_fail))) break;
          const uint32_t sl = ring + slot * SH::SLOT;
          mbar_arrive_expect_tx(&full[slot], SH::SLOT);
          for (int g = 0; g < 2; ++g) {
            const int t = p.silu ? nt : nt + g;  // (past the last tile: zeros, under the last tile's scales)
            mt_load_2d(sl + SH::WAT + g * MA_W, &p.tm_w[p.silu ? g : 0], k * (MA_K / 8), t * 128, &full[slot]);
            mt_load(sl + SH::SAT + g * MX_TILE, p.a.w[p.silu ? g : 0].scales + ((size_t)min(t, p.ntiles - 1) * KT + k) * MX_TILE,
                    MX_TILE, &full[slot]);
          }
          for (int h = 0; h < 2; ++h) mt_load_2d(sl + h * SH::XHALF, &p.tm_x, k * MA_K + h * 64, mt * NC, &full[slot]);
        }
      }
      // shared memory is given back only when the copies into it are done, also where
      // another role gives up behind this one's end (the last S: the others were waited for)
      for (uint32_t i = s > S ? s - S : 0; i < s; ++i) (void)mt_wait(&full[i % S], (i / S) & 1, nullptr);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- MMA issue ----
    pdl_wait_then_trigger();
    uint32_t s = 0, n = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x, ++n) {
      int mt, nt, part, k0, k1;
      item(i, &mt, &nt, &part, &k0, &k1);
      if (n > 0) ok = __all_sync(0xffffffffu, mt_wait(&dempty, (n - 1) & 1, &s_fail));
      for (int k = k0; k < k1 && ok; ++k, ++s) {
        const int slot = s % S, ab = s % NAB;
        ok = mt_wait(&full[slot], (s / S) & 1, &s_fail) && mt_wait(&afull[ab], (s / NAB) & 1, &s_fail);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        mt_fence_after();
        if (mt_elect()) {
          const uint64_t b0 = mt_desc(ring + slot * SH::SLOT), b1 = mt_desc(ring + slot * SH::SLOT + SH::XHALF);
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int kk = 0; kk < MA_K / 16; ++kk) {
              const uint64_t b = (kk < 4 ? b0 : b1) + (uint64_t)((kk & 3) * 2);
              const uint32_t at = tmem + SH::TA + (uint32_t)((ab * 2 + g) * 64 + kk * 8);
              asm volatile(
                  "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                  "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem + (uint32_t)(g * NC)),
                  "r"(at), "l"(b), "r"(SH::IDESC), "r"(k > k0 || kk > 0 ? 1u : 0u)
                  : "memory");
            }
          mt_commit(&empty[slot]);
          mt_commit(&aempty[ab]);
          if (k == k1 - 1) mt_commit(&dfull);
        }
        __syncwarp();
      }
    }
    // tensor memory is freed only when every MMA issued is done, whatever happened elsewhere
    if (s > 0) {
      if (mt_elect()) mt_commit(&drain);
      __syncwarp();
      (void)mt_wait(&drain, 0, nullptr);
    }
  } else {
    // ---- expanders and epilogue ----
    pdl_wait_then_trigger();
    const int e = warp - 2, quad = warp & 3, g = (e >> 2) & 1, set = e >> 3;
    const int row = 32 * quad + lane;  // of the tile; the tensor-memory lane
    const int sw = (row >> 1) & 3;     // 16-byte chunk c of a row's codes is at c ^ sw
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    uint32_t s = 0, n = 0;
    int early = 0;                     // stages of this item done under the one before
    bool ok = true;
    for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x, ++n) {
      int mt, nt, part, k0, k1, ahead = 0;
      // Behind the item's stages the next one's first two, one of each set: they
      // lie under the item's last MMAs, and the next one's first need not wait.  (Their
      // buffers are left by MMAs of this item: none of them waits for the epilogue below.)
      if (i + (int)gridDim.x < p.items) {
        item(i + gridDim.x, &mt, &nt, &part, &k0, &k1);
        ahead = min(k1 - k0, 2);
      }
      int tile = item(i, &mt, &nt, &part, &k0, &k1);
      for (int left = k1 - k0 - early + ahead; left > 0; --left, ++s) {
        if ((s & 1) != set) continue;
        const int slot = s % S, ab = s % NAB;
        ok = __all_sync(0xffffffffu, mt_wait(&full[slot], (s / S) & 1, &s_fail));
        if (!ok) break;
        const unsigned char* w = ringp + slot * SH::SLOT + SH::WAT + g * MA_W + row * 64;
        uint4 c[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) c[q] = *reinterpret_cast<const uint4*>(w + ((q ^ sw) << 4));
        const uint32_t sc = *reinterpret_cast<const uint32_t*>(ringp + slot * SH::SLOT + SH::SAT + g * MX_TILE + lane * 16 + quad * 4);
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
        uint32_t v[64];
        const uint32_t s01 = mx_weight_scales(__byte_perm(sc, 0, 0x4140)), s23 = mx_weight_scales(__byte_perm(sc, 0, 0x4342));
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t bf = b < 2 ? s01 : s23, cw[4] = {c[b].x, c[b].y, c[b].z, c[b].w};
          const __half2 sh = __float2half2_rn(__uint_as_float(b & 1 ? bf & 0xFFFF0000u : bf << 16));
          const uint32_t sb = *reinterpret_cast<const uint32_t*>(&sh);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 f = mx_values(cw[j]);
            v[16 * b + 4 * j] = hmul2_u32(f.x, sb);
            v[16 * b + 4 * j + 1] = hmul2_u32(f.y, sb);
            v[16 * b + 4 * j + 2] = hmul2_u32(f.z, sb);
            v[16 * b + 4 * j + 3] = hmul2_u32(f.w, sb);
          }
        }
        ok = __all_sync(0xffffffffu, s < NAB || mt_wait(&aempty[ab], (s / NAB - 1) & 1, &s_fail));
        if (!ok) break;
        mt_fence_after();
        const uint32_t ta = lanes + SH::TA + (uint32_t)((ab * 2 + g) * 64);
#pragma unroll
        for (int h = 0; h < 64; h += 32)
          asm volatile(
              "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
              "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(ta + h),
              "r"(v[h]), "r"(v[h + 1]), "r"(v[h + 2]), "r"(v[h + 3]), "r"(v[h + 4]), "r"(v[h + 5]), "r"(v[h + 6]),
              "r"(v[h + 7]), "r"(v[h + 8]), "r"(v[h + 9]), "r"(v[h + 10]), "r"(v[h + 11]), "r"(v[h + 12]), "r"(v[h + 13]),
              "r"(v[h + 14]), "r"(v[h + 15]), "r"(v[h + 16]), "r"(v[h + 17]), "r"(v[h + 18]), "r"(v[h + 19]), "r"(v[h + 20]),
              "r"(v[h + 21]), "r"(v[h + 22]), "r"(v[h + 23]), "r"(v[h + 24]), "r"(v[h + 25]), "r"(v[h + 26]), "r"(v[h + 27]),
              "r"(v[h + 28]), "r"(v[h + 29]), "r"(v[h + 30]), "r"(v[h + 31])
              : "memory");
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        mt_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&afull[ab]);
      }
      if (!ok) break;
      early = ahead;
      // Where the item lies is found again below 128 columns, as registers are short above
      // (18944 x 3584 twice of 32 rows 18.9 us, 19.4 without; of 128 columns, 2048 rows of
      // 18944 x 3584, 206 us with it and 199 without).
      if (NC < 128) tile = item(i, &mt, &nt, &part, &k0, &k1);
      // epilogue: warp e has columns [e / 4 * NC / 4, ..) of both tiles' rows of its quadrant
      ok = __all_sync(0xffffffffu, mt_wait(&dfull, n & 1, &s_fail));
      if (!ok) break;
      mt_fence_after();
      float* turn = reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw)) + S * SH::SLOT) + e * 256;
      const int M = p.a.M, N = p.a.N;
      const bool wide = N % 8 == 0;      // rows of y (and of the residual) start on 16 bytes
      constexpr int CW = NC / 4, PC = CW / 8;
      const int col0 = (e >> 2) * CW;
      const bool parts = i >= p.whole && p.split > 1;
      float* mine = parts ? p.parts + ((size_t)(tile - p.whole) * p.split + part) * (NC * 256) : nullptr;
      const int rounds = p.silu && !parts ? PC : 2 * PC;  // silu takes both tiles' columns at once
#pragma unroll 1
      for (int pc = 0; pc < rounds; ++pc) {
        const int gg = pc >= PC ? 1 : 0, c0 = col0 + (pc - gg * PC) * 8, m0 = mt * NC + c0;
        const int n0 = (nt + gg) * 128 + 32 * quad;      // the quadrant's first weight row
        float v[8], u[8];
        __syncwarp();  // tensor memory is read, and waited for, by whole warps
        mx_tmem_ld8(v, lanes + (uint32_t)(gg * NC + c0));
        if (p.silu && !parts) mx_tmem_ld8(u, lanes + (uint32_t)(NC + c0));
        // this lane's share of the turned outputs: row m, 8 weight rows from nn
        const int m = m0 + (lane >> 2), nn = n0 + (lane & 3) * 8;
        const bool inside = m < M && nn < N && !parts;
        const size_t at = (size_t)m * N + nn;
        uint4 add = make_uint4(0, 0, 0, 0);
        if (wide && inside && p.a.residual) add = *reinterpret_cast<const uint4*>(p.a.residual + at);
        const float bias = p.a.bias && n0 + lane < N ? __half2float(p.a.bias[n0 + lane]) : 0.f;
        __syncwarp();
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        if (pc == rounds - 1) {
          mt_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&dempty);
        }
        if (parts) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (m0 + c < M) mine[(c0 + c) * 256 + gg * 128 + row] = v[c];
          continue;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (p.silu) v[c] = v[c] / (1.f + expf(-v[c])) * u[c];
          v[c] += bias;
        }
        if (wide) {
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 8; ++c) turn[c * 32 + lane] = v[c];
          __syncwarp();
          float4 lo = *reinterpret_cast<const float4*>(turn + lane * 8), hi = *reinterpret_cast<const float4*>(turn + lane * 8 + 4);
          if (p.a.residual) mx_add8(lo, hi, add);
          const uint4 o = mx_round8(lo, hi);
          if (inside) *reinterpret_cast<uint4*>(p.a.y + at) = o;
        } else if (n0 + lane < N) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (m0 + c >= M) break;
            const size_t at = (size_t)(m0 + c) * N + n0 + lane;
            if (p.a.residual) v[c] += __half2float(p.a.residual[at]);
            p.a.y[at] = __float2half_rn(v[c]);
          }
        }
      }
    }
  }
  mt_fence_before();
  __syncthreads();
  if (s_fail && tid == 0 && p.a.err_flag) atomicOr(p.a.err_flag, 2);
  __syncwarp();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem_slot) : "memory");
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
bool mt_map(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t rows, uint64_t row_bytes,
            uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle sw) {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {inner, rows}, strides[1] = {row_bytes};
  const cuuint32_t box[2] = {box_inner, box_rows}, es[2] = {1, 1};
  return enc(m, dt, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static int ma_cols(int M) { return M <= 32 ? 32 : M <= 64 ? 64 : 128; }
static int ma_tiles(int M, int N, bool silu) {
  const int nc = ma_cols(M), nt = (N + 127) / 128;
  return (M + nc - 1) / nc * (silu ? nt : (nt + 1) / 2);
}
constexpr int MA_SPLIT = 16;

// The deal for these sizes with room for `bytes` of workspace: the split along K,
// or none, whose busiest CTA has least to do, in cycles as measured (a stage 980,
// 1150, 1580 for 32, 64, 128 rows; a tile's epilogue 2000 to 8000; the join 5000).
static MtDeal ma_deal(int M, int N, int K, bool silu, size_t bytes, int slots) {
  const int nc = ma_cols(M), tiles = ma_tiles(M, N, silu), stages = K / MA_K;
  const double stage = nc == 32 ? 980 : nc == 64 ? 1150 : 1580, tail = 62.0 * nc;
  MtDeal best = mt_deal(tiles, stages, slots, 1);
  double cost = (double)((tiles + slots - 1) / slots) * (stages * stage + tail);
  for (int most = 2; most <= MA_SPLIT; ++most) {
    const MtDeal d = mt_deal(tiles, stages, slots, most);
    if (d.split != most || mt_workspace(d, nc, 256) > bytes) continue;
    const double v = (double)(d.whole / slots) * (stages * stage + tail) + (stages + most - 1) / most * stage + tail + 5000;
    if (v < cost) {
      cost = v;
      best = d;
    }
  }
  return best;
}

size_t mxfp4_a16_workspace(int M, int N, int K, bool silu) {
  // for the split of a GB300's 152 SMs, so that it can be asked for where there is no GPU
  return mt_workspace(ma_deal(M, N, K, silu, ~(size_t)0, ATW_SMS), ma_cols(M), 256);
}

int mxfp4_a16_largest_tile() { return 128 * 256; }

void mxfp4_a16_plan(int M, int N, int K, bool silu, size_t bytes, int slots, int32_t* plan) {
  mt_tell(ma_deal(M, N, K, silu, bytes, slots), ma_cols(M), 256, slots, plan);
}

template <int NC>
static int ma_launch(MaArgs& p, int slots, cudaStream_t s) {
  using SH = MaShape<NC>;
  static PerDeviceOnce once;
  once_per_device(once, [] {
    cudaFuncSetAttribute(w4pg_mxfp4_a16<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SH::SMEM);
  });
  const MxArgs& a = p.a;
  bool ok = mt_map(&p.tm_x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.x, a.K, a.M, (uint64_t)a.K * 2, 64, NC,
                   CU_TENSOR_MAP_SWIZZLE_128B);
  for (int g = 0; g < (p.silu ? 2 : 1); ++g)
    ok = ok && mt_map(&p.tm_w[g], CU_TENSOR_MAP_DATA_TYPE_UINT32, a.w[g].codes, a.K / 8, a.N, (uint64_t)a.K / 2, MA_K / 8, 128,
                      CU_TENSOR_MAP_SWIZZLE_64B);
  if (!ok) return set_error(W4A16_ERR_CUDA, "mxfp4 product: no tensor maps for the operands");
  const cudaError_t e = launch_pdl(w4pg_mxfp4_a16<NC>, dim3(std::min(p.items, slots)), dim3(MA_THREADS), SH::SMEM, s, p);
  if (e != cudaSuccess) return set_error(W4A16_ERR_CUDA, "mxfp4 product launch: %s", cudaGetErrorString(e));
  return W4A16_OK;
}

int launch_mxfp4_a16(const MxArgs& a, bool silu, cudaStream_t s) {
  MaArgs p = {};
  const int nc = ma_cols(a.M), slots = num_sms();
  const MtDeal d = ma_deal(a.M, a.N, a.K, silu, a.workspace ? a.workspace_bytes : 0, slots);
  p.a = a;
  p.silu = silu;
  p.mtiles = (a.M + nc - 1) / nc;
  p.ntiles = (a.N + 127) / 128;
  p.whole = d.whole;
  p.split = d.split;
  p.items = d.items;
  if (d.split > 1) p.parts = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + TC_TICKET_BYTES);
  const int rc = nc == 32 ? ma_launch<32>(p, slots, s) : nc == 64 ? ma_launch<64>(p, slots, s) : ma_launch<128>(p, slots, s);
  if (rc || d.split < 2) return rc;
  return launch_mxfp4_join({a, p.parts, d.whole, (d.items - d.whole) / d.split, d.split, nc, 256, p.mtiles, silu ? 128 : 256, silu},
                           s);
}

}  // namespace w4

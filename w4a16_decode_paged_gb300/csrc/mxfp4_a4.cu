// mxfp4_a4.cu -- products of two MXFP4 matrices (a prompt's activations, quantised,
// with the weights) on the 5th-generation tensor cores' block-scaled 4-bit MMAs.
//
// y[m][n] = sum over blocks of 32 k of 2^(bx + bw - 254) sum cx cw: kind::mxf4 MMAs
// take both operands' codes packed as they are in memory (K-major rows, 128-byte
// swizzle) and one scale byte per 32 k and row from tensor memory, and sum in
// fp32.  The scale tiles (mxfp4.cuh) have the order in which tcgen05.cp spreads
// them: 32 lanes of four 32-bit columns, repeated for the four lane quadrants.
//
// A CTA's tile is 2 x 128 weight rows (lanes of D) x NC rows of x (its columns).
// A stage is 256 k: 128-byte rows of codes and two scale tiles per 128 rows; at
// NC = 192 60 KB for 768 cycles of MMAs.
//
// Roles: a producer lane, one warp that issues the scales' copies and the MMAs
// (these run in the order issued, so one set of scale columns serves), 8 epilogue
// warps.  Tiles are dealt by mt_deal, parts along K meet as in mxfp4_a16.cu.
#include "mxfp4_tc.cuh"

namespace w4 {

constexpr int MB_K = 256;                     // k of a stage
constexpr int MB_EPI = 8;                     // epilogue warps
constexpr int MB_THREADS = 64 + 32 * MB_EPI;
constexpr uint32_t MB_W = 128 * MB_K / 2;     // bytes of a weight tile per stage

template <int NC>
struct MbShape {
  static constexpr uint32_t X = NC * MB_K / 2;
  static constexpr uint32_t XAT = 2 * MB_W, SAT = XAT + X;            // a slot: two weight tiles, x, scales (w, w, x, x)
  static constexpr uint32_t SLOT = SAT + 4 * 2 * MX_TILE;
  static constexpr int S = 225 * 1024 / SLOT;
  static constexpr size_t SMEM = S * SLOT + 1024;
  static constexpr uint32_t TS = 2 * NC;                              // tensor memory: sums, weight scales, x scales
  static constexpr uint32_t IDESC =
      (1u << 7) | (1u << 10) | ((uint32_t)(NC >> 3) << 17) | (1u << 23) | ((128u >> 4) << 24);
  static_assert(SLOT % 1024 == 0 && TS + 32 <= 512 && S >= 3, "swizzled tiles start on 1024-byte boundaries");
};

struct MbArgs {
  MxArgs a;
  int mtiles, ntiles, whole, split, items;
  float* parts;
  unsigned int* tickets;
  CUtensorMap tm_w, tm_x;
};

// shared-memory descriptor of a scale tile: rows of 16 bytes, 8 to a 128-byte unit
__device__ __forceinline__ uint64_t mb_scale_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
}
__device__ __forceinline__ void mb_copy_scales(uint32_t taddr, uint32_t saddr) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(mb_scale_desc(saddr)) : "memory");
}

template <int NC>
__global__ void __launch_bounds__(MB_THREADS, 1) w4pg_mxfp4_a4(const __grid_constant__ MbArgs p) {
  using SH = MbShape<NC>;
  constexpr int S = SH::S;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  __shared__ __align__(8) uint64_t full[S], empty[S], dfull, dempty, drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int s_last;
  __shared__ volatile int s_fail;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int K = p.a.K, KT = K / 128, stages = (K + MB_K - 1) / MB_K;

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 32) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&dfull, 1);
    mbar_init(&dempty, MB_EPI);
    mbar_init(&drain, 1);
    s_fail = 0;
    fence_mbar_init();
  }
  mt_fence_before();
  __syncthreads();
  mt_fence_after();
  const uint32_t tmem = tmem_slot;

  auto item = [&](int i, int* mt, int* nt, int* part, int* k0, int* k1) {
    int tile;
    mt_item(i, p.whole, p.split, stages, &tile, part, k0, k1);
    *mt = tile % p.mtiles;
    *nt = tile / p.mtiles * 2;
    return tile;
  };

  if (warp == 0) {
    // ---- producer ----
    if (mt_elect()) {
      int mt, nt, part, k0, k1;
      if (blockIdx.x < p.items) {
        // weights may come from the call just before: into L2 ahead of the wait, read behind it
        item(blockIdx.x, &mt, &nt, &part, &k0, &k1);
        for (int k = k0; k < min(k1, k0 + S); ++k)
          for (int g = 0; g < 2; ++g) mt_prefetch_2d(&p.tm_w, k * (MB_K / 2), (nt + g) * 128);
      }
      pdl_wait_then_trigger();
      uint32_t s = 0;
      bool ok = true;
      const int xtiles = (p.a.M + 127) / 128;
      for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x) {
        item(i, &mt, &nt, &part, &k0, &k1);
        for (int k = k0; k < k1; ++k, ++s) {
          const int slot = s % S;
          if (s >= S && !(ok = mt_wait(&empty[slot], (s / S - 1) & 1, &s_fail))) break;
          const uint32_t sl = ring + slot * SH::SLOT;
          const uint32_t sb = (2 * k + 2 <= KT ? 2 : 1) * MX_TILE;  // scales: an odd last tile is half a stage
          mbar_arrive_expect_tx(&full[slot], 2 * MB_W + SH::X + 4 * sb);
          for (int g = 0; g < 2; ++g) {
            // (past the last tile: zeros, under the last tile's scales)
            mt_load_2d(sl + g * MB_W, &p.tm_w, k * (MB_K / 2), (nt + g) * 128, &full[slot]);
            mt_load(sl + SH::SAT + g * 2 * MX_TILE,
                    p.a.w[0].scales + ((size_t)min(nt + g, p.ntiles - 1) * KT + 2 * k) * MX_TILE, sb, &full[slot]);
            mt_load(sl + SH::SAT + (2 + g) * 2 * MX_TILE,
                    p.a.xq.scales + ((size_t)min(mt * NC / 128 + g, xtiles - 1) * KT + 2 * k) * MX_TILE, sb, &full[slot]);
          }
          mt_load_2d(sl + SH::XAT, &p.tm_x, k * (MB_K / 2), mt * NC, &full[slot]);
        }
      }
      // shared memory is given back only when the copies into it are done
      for (uint32_t i = s > S ? s - S : 0; i < s && s_fail; ++i) (void)mt_wait(&full[i % S], (i / S) & 1, nullptr);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- scales and MMAs ----
    pdl_wait_then_trigger();
    uint32_t s = 0, n = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x, ++n) {
      int mt, nt, part, k0, k1;
      item(i, &mt, &nt, &part, &k0, &k1);
      if (n > 0) ok = __all_sync(0xffffffffu, mt_wait(&dempty, (n - 1) & 1, &s_fail));
      mt_fence_after();
      const uint32_t xoff = (uint32_t)(mt * NC % 128) / 32;  // the first row's scale column in its tile
      for (int k = k0; k < k1 && ok; ++k, ++s) {
        const int slot = s % S;
        ok = __all_sync(0xffffffffu, mt_wait(&full[slot], (s / S) & 1, &s_fail));
        if (!ok) break;
        mt_fence_after();
        if (mt_elect()) {
          const uint32_t sl = ring + slot * SH::SLOT, ts = tmem + SH::TS;
          const int halves = 2 * k + 2 <= KT ? 2 : 1;
          // columns: weights tile g, half j at 8 g + 4 j; x half j, tile g at 16 + 8 j + 4 g
          for (int j = 0; j < halves; ++j)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              mb_copy_scales(ts + 8 * g + 4 * j, sl + SH::SAT + (2 * g + j) * MX_TILE);
              mb_copy_scales(ts + 16 + 8 * j + 4 * g, sl + SH::SAT + (4 + 2 * g + j) * MX_TILE);
            }
          for (int j = 0; j < halves; ++j)
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
              for (int kk = 0; kk < 2; ++kk) {
                const uint64_t ad = mt_desc(sl + g * MB_W) + (uint64_t)(4 * j + 2 * kk);
                const uint64_t bd = mt_desc(sl + SH::XAT) + (uint64_t)(4 * j + 2 * kk);
                const uint32_t id = SH::IDESC | ((uint32_t)(2 * kk) << 29) | ((uint32_t)(2 * kk) << 4);
                asm volatile(
                    "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
                    "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                        tmem + (uint32_t)(g * NC)),
                    "l"(ad), "l"(bd), "r"(id), "r"(ts + 8 * g + 4 * j), "r"(ts + 16 + 8 * j + xoff),
                    "r"(k > k0 || j > 0 || kk > 0 ? 1u : 0u)
                    : "memory");
              }
          mt_commit(&empty[slot]);
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
    // ---- epilogue ----
    pdl_wait_then_trigger();
    const int e = warp - 2, quad = warp & 3, row = 32 * quad + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    constexpr int CW = NC / 2;  // columns of a warp, both weight tiles
    const int col0 = (e >> 2) * CW, M = p.a.M, N = p.a.N;
    uint32_t n = 0;
    for (int i = blockIdx.x; i < p.items; i += gridDim.x, ++n) {
      int mt, nt, part, k0, k1;
      const int tile = item(i, &mt, &nt, &part, &k0, &k1);
      if (!__all_sync(0xffffffffu, mt_wait(&dfull, n & 1, &s_fail))) break;
      mt_fence_after();
      const bool parts = i >= p.whole && p.split > 1;
      const int t = tile - p.whole, m0 = mt * NC + col0;
      float* mine = parts ? p.parts + ((size_t)t * p.split + part) * (2 * NC * 128) : nullptr;
      auto out = [&](int nn, int m, float v, float bias) {
        const size_t at = (size_t)m * N + nn;
        v += bias;
        if (p.a.residual) v += __half2float(p.a.residual[at]);
        p.a.y[at] = __float2half_rn(v);
      };
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int nn = (nt + g) * 128 + row;
        const float bias = !parts && p.a.bias && nn < N ? __half2float(p.a.bias[nn]) : 0.f;
#pragma unroll
        for (int c0 = 0; c0 < CW; c0 += 32) {
          uint32_t v[32];
#pragma unroll
          for (int c = 0; c < 32; c += 8)
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(v[c]), "=r"(v[c + 1]), "=r"(v[c + 2]), "=r"(v[c + 3]), "=r"(v[c + 4]), "=r"(v[c + 5]),
                           "=r"(v[c + 6]), "=r"(v[c + 7])
                         : "r"(lanes + (uint32_t)(g * NC + col0 + c0 + c)));
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
          if (g == 1 && c0 + 32 == CW) {
            mt_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&dempty);
          }
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            if (m0 + c0 + c >= M) break;
            const float f = __uint_as_float(v[c]);
            if (parts) mine[(g * NC + col0 + c0 + c) * 128 + row] = f;
            else if (nn < N) out(nn, m0 + c0 + c, f, bias);
          }
        }
      }
      if (!parts) continue;
      __threadfence();
      asm volatile("bar.sync 1, %0;" ::"n"(32 * MB_EPI) : "memory");
      if (e == 0 && lane == 0) s_last = atomicAdd(&p.tickets[t], 1u) == (unsigned int)(p.split - 1);
      asm volatile("bar.sync 1, %0;" ::"n"(32 * MB_EPI) : "memory");
      if (!s_last) continue;
      __threadfence();
      if (e == 0 && lane == 0) p.tickets[t] = 0u;
      const float* all = p.parts + (size_t)t * p.split * (2 * NC * 128);
      for (int g = 0; g < 2; ++g) {
        const int nn = (nt + g) * 128 + row;
        if (nn >= N) break;
        const float bias = p.a.bias ? __half2float(p.a.bias[nn]) : 0.f;
#pragma unroll 4
        for (int c = 0; c < CW; ++c) {
          if (m0 + c >= M) break;
          float v = 0.f;
          for (int q = 0; q < p.split; ++q) v += __ldcg(&all[(size_t)q * (2 * NC * 128) + (g * NC + col0 + c) * 128 + row]);
          out(nn, m0 + c, v, bias);
        }
      }
    }
  }
  mt_fence_before();
  __syncthreads();
  if (s_fail && tid == 0 && p.a.err_flag) atomicOr(p.a.err_flag, 2);
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem_slot) : "memory");
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
static int mb_cols(int M) { return M <= 64 ? 64 : M <= 128 ? 128 : 192; }
static int mb_tiles(int M, int N) {
  const int nc = mb_cols(M);
  return (M + nc - 1) / nc * ((N + 255) / 256);
}
constexpr int MB_SPLIT = 16;

static MtDeal mb_deal(int M, int N, int K, size_t bytes, int slots) {
  const size_t part = (size_t)2 * 128 * mb_cols(M) * 4;
  const int stages = (K + MB_K - 1) / MB_K;
  for (int most = MB_SPLIT; most > 1; --most) {
    const MtDeal d = mt_deal(mb_tiles(M, N), stages, slots, most);
    const int over = d.items == d.whole ? 0 : (d.items - d.whole) / d.split;
    if (over <= (int)(TC_TICKET_BYTES / 4) && (over == 0 || TC_TICKET_BYTES + (size_t)over * d.split * part <= bytes)) return d;
  }
  return mt_deal(mb_tiles(M, N), stages, slots, 1);
}

size_t mxfp4_a4_workspace(int M, int N, int K) {
  const MtDeal d = mb_deal(M, N, K, ~(size_t)0, ATW_SMS);
  return TC_TICKET_BYTES + (size_t)(d.items - d.whole) * 2 * 128 * mb_cols(M) * 4;
}

template <int NC>
static int mb_launch(MbArgs& p, int slots, cudaStream_t s) {
  using SH = MbShape<NC>;
  static PerDeviceOnce once;
  once_per_device(once, [] {
    cudaFuncSetAttribute(w4pg_mxfp4_a4<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SH::SMEM);
  });
  const MxArgs& a = p.a;
  const bool ok = mt_map(&p.tm_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.xq.codes, a.K / 2, a.M, (uint64_t)a.K / 2, MB_K / 2, NC,
                         CU_TENSOR_MAP_SWIZZLE_128B) &&
                  mt_map(&p.tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w[0].codes, a.K / 2, a.N, (uint64_t)a.K / 2, MB_K / 2, 128,
                         CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return set_error(W4A16_ERR_CUDA, "mxfp4 product: no tensor maps for the operands");
  const cudaError_t e = launch_pdl(w4pg_mxfp4_a4<NC>, dim3(std::min(p.items, slots)), dim3(MB_THREADS), SH::SMEM, s, p);
  if (e != cudaSuccess) return set_error(W4A16_ERR_CUDA, "mxfp4 product launch: %s", cudaGetErrorString(e));
  return W4A16_OK;
}

int launch_mxfp4_a4(const MxArgs& a, cudaStream_t s) {
  MbArgs p = {};
  const int nc = mb_cols(a.M), slots = num_sms();
  const MtDeal d = mb_deal(a.M, a.N, a.K, a.workspace ? a.workspace_bytes : 0, slots);
  p.a = a;
  p.mtiles = (a.M + nc - 1) / nc;
  p.ntiles = (a.N + 127) / 128;
  p.whole = d.whole;
  p.split = d.split;
  p.items = d.items;
  p.tickets = static_cast<unsigned int*>(a.workspace);
  if (d.split > 1) p.parts = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + TC_TICKET_BYTES);
  return nc == 64 ? mb_launch<64>(p, slots, s) : nc == 128 ? mb_launch<128>(p, slots, s) : mb_launch<192>(p, slots, s);
}

}  // namespace w4

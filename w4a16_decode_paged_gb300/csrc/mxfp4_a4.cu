// mxfp4_a4.cu -- products of two MXFP4 matrices (a prompt's activations, quantised,
// with the weights) on the 5th-generation tensor cores' block-scaled 4-bit MMAs.
//
// y[m][n] = sum over blocks of 32 k of 2^(bx + bw - 254) sum cx cw: kind::mxf4 MMAs
// take both operands' codes packed as they are in memory (K-major rows, 128-byte
// swizzle) and one scale byte per 32 k and row from tensor memory, and sum in
// fp32.  The scale tiles (mxfp4.cuh) have the order in which tcgen05.cp spreads
// them: 32 lanes of four 32-bit columns, repeated for the four lane quadrants.
//
// A CTA's tile is NA x 128 rows of x (lanes of D) x NC weight rows (its columns), so
// that a thread of the epilogue has neighbouring outputs of one row.  Where tensor
// memory holds the tile's sums twice (DB = 2), its epilogue lies under the next
// tile's MMAs.  A stage is 256 k: 128-byte rows of codes, two scale tiles per 128
// rows.  NC = 192 starts in the middle of a scale tile every other time, which is two
// columns further on in tensor memory (scales have to start on an even column, so
// that NC is a multiple of 64).
//
// What bounds it is not settled.  A stage takes 1170 to 1200 cycles at 2 x 192 (0.58 us,
// 4096 x 3584 by two lengths of K, SM clock sampled at 2.02 to 2.07 GHz) and 690 to 720
// at 1 x 192 (0.34 us); its MMAs at their nominal rate (128 x NC x 64 in NC / 2 cycles)
// would be 768 and 384.  Two accounts fit all shapes: shared memory at 128 bytes a clock
// (per 64 k an MMA reads 4 KB of x and NC / 32 KB of weights, and as much is copied in:
// 1088 and 640 cycles), or the MMAs and a constant of 290 to 430 cycles, for which the scale
// columns are a candidate: there is one set, so that a stage's copies into it wait for
// the MMAs before them.  256 x 192 by pairs of CTAs, each with half of the weight rows,
// has less to read and copy than 1 x 192 and took as long a stage (0.38 us where 1 x 192
// took 0.38 as well; two CTAs of 2 x 192 get through as much in 0.30: not kept), which
// speaks for the second.
//
// Roles: a producer lane, one warp that issues the scales' copies and the MMAs
// (these run in the order issued, so one set of scale columns serves), 8 epilogue
// warps.  Tiles are dealt by mt_deal.
#include "mxfp4_tc.cuh"

namespace w4 {

constexpr int MB_K = 256;                     // k of a stage
constexpr int MB_EPI = 8;                     // epilogue warps
constexpr int MB_THREADS = 64 + 32 * MB_EPI;
constexpr uint32_t MB_X = 128 * MB_K / 2;     // bytes of 128 rows of x per stage
constexpr int MB_SPLIT = 16;
constexpr int MB_TURN = 32 * 32 * 4;          // a warp's 32 x 32 outputs, fp32: four columns c of row r at c ^ r % 8

template <int NA, int NC, int DB>
struct MbShape {
  static constexpr int NB = NC == 128 ? 1 : 2;                        // weight scale tiles that NC rows can touch
  static constexpr uint32_t W = NC * MB_K / 2;
  static constexpr uint32_t WAT = NA * MB_X, SAT = WAT + W;           // a slot: x, weights, scales of x, of the weights
  static constexpr uint32_t SLOT = (SAT + (NA + NB) * 2 * MX_TILE + 1023) / 1024 * 1024;
  static constexpr int S = (225 * 1024 - MB_EPI * MB_TURN) / SLOT;
  static constexpr size_t SMEM = S * SLOT + MB_EPI * MB_TURN + 1024;
  static constexpr uint32_t TS = DB * NA * NC;                        // tensor memory: sums, scales of x, of the weights
  static constexpr uint32_t IDESC =
      (1u << 7) | (1u << 10) | ((uint32_t)(NC >> 3) << 17) | (1u << 23) | ((128u >> 4) << 24);
  static_assert(NC % 64 == 0 && NC <= 256 && TS + 8 * (NA + NB) <= 512 && S >= 3, "tensor memory, ring");
};

struct MbArgs {
  MxArgs a;
  int mtiles, ntiles, whole, split, items;  // ntiles: scale tiles of the weights
  float* parts;
  CUtensorMap tm_w, tm_x;
};

// shared-memory descriptor of a scale tile: rows of 16 bytes, 8 to a 128-byte unit
__device__ __forceinline__ uint64_t mb_scale_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
}
__device__ __forceinline__ void mb_copy_scales(uint32_t taddr, uint32_t saddr) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(mb_scale_desc(saddr)) : "memory");
}

template <int NA, int NC, int DB>
__global__ void __launch_bounds__(MB_THREADS, 1) w4pg_mxfp4_a4(const __grid_constant__ MbArgs p) {
  using SH = MbShape<NA, NC, DB>;
  constexpr int S = SH::S, NB = SH::NB;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  __shared__ __align__(8) uint64_t full[S], empty[S], dfull[DB], dempty[DB][NA], drain;
  __shared__ uint32_t tmem_slot;
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
    for (int b = 0; b < DB; ++b) {
      mbar_init(&dfull[b], 1);
      for (int g = 0; g < NA; ++g) mbar_init(&dempty[b][g], MB_EPI);
    }
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
    *nt = tile / p.mtiles;
    return tile;
  };

  if (warp == 0) {
    // ---- producer ----
    if (mt_elect()) {
      mt_prefetch_map(&p.tm_w);
      mt_prefetch_map(&p.tm_x);
      int mt, nt, part, k0, k1;
      if (blockIdx.x < p.items) {
        // weights may come from the call just before: into L2 ahead of the wait, read behind it
        item(blockIdx.x, &mt, &nt, &part, &k0, &k1);
        for (int k = k0; k < min(k1, k0 + S); ++k) mt_prefetch_2d(&p.tm_w, k * (MB_K / 2), nt * NC);
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
          mbar_arrive_expect_tx(&full[slot], NA * MB_X + SH::W + (NA + NB) * sb);
          mt_load_2d(sl + SH::WAT, &p.tm_w, k * (MB_K / 2), nt * NC, &full[slot]);
#pragma unroll
          for (int g = 0; g < NA; ++g) {
            // (past the last rows: zeros, under the last tile's scales)
            mt_load_2d(sl + g * MB_X, &p.tm_x, k * (MB_K / 2), (mt * NA + g) * 128, &full[slot]);
            mt_load(sl + SH::SAT + g * 2 * MX_TILE,
                    p.a.xq.scales + ((size_t)min(mt * NA + g, xtiles - 1) * KT + 2 * k) * MX_TILE, sb, &full[slot]);
          }
#pragma unroll
          for (int g = 0; g < NB; ++g)
            mt_load(sl + SH::SAT + (NA + g) * 2 * MX_TILE,
                    p.a.w[0].scales + ((size_t)min(nt * NC / 128 + g, p.ntiles - 1) * KT + 2 * k) * MX_TILE, sb, &full[slot]);
        }
      }
      // shared memory is given back only when the copies into it are done, also where
      // another role gives up behind this one's end (the last S: the others were waited for)
      for (uint32_t i = s > S ? s - S : 0; i < s; ++i) (void)mt_wait(&full[i % S], (i / S) & 1, nullptr);
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
      const uint32_t woff = (uint32_t)(nt * NC % 128) / 32;  // the first weight row's scale column in its tile
      const int buf = DB == 2 ? n & 1 : 0;
      for (int k = k0; k < k1; ++k, ++s) {
        const int slot = s % S;
        ok = __all_sync(0xffffffffu, mt_wait(&full[slot], (s / S) & 1, &s_fail));
        if (!ok) break;
        const uint32_t sl = ring + slot * SH::SLOT, ts = tmem + SH::TS;
        mt_fence_after();
        // columns: x tile g, half j at 8 g + 4 j; the weights' half j, tile g behind them at 4 NB j + 4 g
        auto scales = [&](int j) {
#pragma unroll
          for (int g = 0; g < NA; ++g) mb_copy_scales(ts + 8 * g + 4 * j, sl + SH::SAT + (2 * g + j) * MX_TILE);
#pragma unroll
          for (int g = 0; g < NB; ++g)
            mb_copy_scales(ts + 8 * NA + 4 * NB * j + 4 * g, sl + SH::SAT + (2 * (NA + g) + j) * MX_TILE);
        };
        auto mmas = [&](int g, int j) {
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            const uint64_t ad = mt_desc(sl + g * MB_X) + (uint64_t)(4 * j + 2 * kk);
            const uint64_t bd = mt_desc(sl + SH::WAT) + (uint64_t)(4 * j + 2 * kk);
            const uint32_t id = SH::IDESC | ((uint32_t)(2 * kk) << 29) | ((uint32_t)(2 * kk) << 4);
            asm volatile(
                "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
                "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                    tmem + (uint32_t)((buf * NA + g) * NC)),
                "l"(ad), "l"(bd), "r"(id), "r"(ts + 8 * g + 4 * j), "r"(ts + 8 * NA + 4 * NB * j + woff),
                "r"(k > k0 || j > 0 || kk > 0 ? 1u : 0u)
                : "memory");
          }
        };
        const bool both = 2 * k + 2 <= KT;
#pragma unroll
        for (int g = 0; g < NA; ++g) {
          // an earlier tile has left these columns of tensor memory
          if (k == k0 && n >= DB) {
            ok = __all_sync(0xffffffffu, mt_wait(&dempty[buf][g], (n / DB - 1) & 1, &s_fail));
            if (!ok) break;
            mt_fence_after();
          }
          if (mt_elect()) {
            if (g == 0) {
              scales(0);
              if (both) scales(1);
            }
            mmas(g, 0);
            if (both) mmas(g, 1);
          }
          __syncwarp();
        }
        if (mt_elect()) {
          mt_commit(&empty[slot]);
          if (k == k1 - 1) mt_commit(&dfull[buf]);
        }
        __syncwarp();
        if (!ok) { ++s; break; }
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
    const int e = warp - 2, quad = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    const int M = p.a.M, N = p.a.N;
    const bool wide = N % 8 == 0;  // rows of y (and of the residual) start on 16 bytes
    float4* turn = reinterpret_cast<float4*>(smem_raw + (ring - smem_u32(smem_raw)) + S * SH::SLOT + e * MB_TURN);
    uint32_t n = 0;
    for (int i = blockIdx.x; i < p.items; i += gridDim.x, ++n) {
      int mt, nt, part, k0, k1;
      const int tile = item(i, &mt, &nt, &part, &k0, &k1);
      const int buf = DB == 2 ? n & 1 : 0;
      if (!__all_sync(0xffffffffu, mt_wait(&dfull[buf], (n / DB) & 1, &s_fail))) break;
      mt_fence_after();
      const bool parts = i >= p.whole && p.split > 1;
      // pieces of 32 rows x 32 columns, the two halves of the warps in turn
      constexpr int PC = NC / 32;
#pragma unroll 1
      for (int pc = e >> 2; pc < NA * PC; pc += 2) {
        const int g = NA == 2 && pc >= PC ? 1 : 0, c0 = (pc - g * PC) * 32;
        const int r = g * 128 + 32 * quad, m = mt * NA * 128 + r, nn = nt * NC + c0;  // first row, first column
        float v[32];
        __syncwarp();  // tensor memory is read, and waited for, by whole warps
#pragma unroll
        for (int c = 0; c < 32; c += 8)
          asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                       : "=f"(v[c]), "=f"(v[c + 1]), "=f"(v[c + 2]), "=f"(v[c + 3]), "=f"(v[c + 4]), "=f"(v[c + 5]),
                         "=f"(v[c + 6]), "=f"(v[c + 7])
                       : "r"(lanes + (uint32_t)((buf * NA + g) * NC + c0 + c)));
        // This lane's share of the turned outputs: 8 columns from n8 of rows m + lane / 4
        // + 8 h.  What is added to them is asked for ahead; nothing branches between the
        // loads and the stores, whose latencies are all a tile's epilogue is (4 rows at a
        // time behind branches: 0.65 us a piece).
        const int q = (lane & 3) * 8, n8 = nn + q, r8 = lane >> 2;
        const bool inside = n8 < N && !parts;
        const size_t at = (size_t)(m + r8) * N + n8;
        uint4 add[4], bias = make_uint4(0, 0, 0, 0);
        if (wide && inside) {
          if (p.a.bias) bias = *reinterpret_cast<const uint4*>(p.a.bias + n8);
          if (p.a.residual) {
#pragma unroll
            for (int h = 0; h < 4; ++h)
              if (m + r8 + 8 * h < M) add[h] = *reinterpret_cast<const uint4*>(p.a.residual + at + (size_t)(8 * h) * N);
          }
        }
        __syncwarp();
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        if (pc + 2 >= (g + 1) * PC) {  // this warp's last piece of these 128 rows
          mt_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&dempty[buf][g]);
        }
        // turned in shared memory: 4 lanes have 32 columns of a row, 8 rows a store
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          turn[lane * 8 + (c ^ (lane & 7))] = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
        __syncwarp();
        if (parts || wide) {
          float4 lo[4], hi[4];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            lo[h] = turn[(r8 + 8 * h) * 8 + ((q / 4) ^ r8)];
            hi[h] = turn[(r8 + 8 * h) * 8 + ((q / 4 + 1) ^ r8)];
          }
          if (parts) {
            float* mine = p.parts + ((size_t)(tile - p.whole) * p.split + part) * (NA * 128 * NC) + (size_t)(r + r8) * NC + c0 + q;
#pragma unroll
            for (int h = 0; h < 4; ++h)
              if (m + r8 + 8 * h < M) {
                *reinterpret_cast<float4*>(mine + 8 * h * NC) = lo[h];
                *reinterpret_cast<float4*>(mine + 8 * h * NC + 4) = hi[h];
              }
          } else {
            if (p.a.bias) {
#pragma unroll
              for (int h = 0; h < 4; ++h) mx_add8(lo[h], hi[h], bias);
            }
            if (p.a.residual) {
#pragma unroll
              for (int h = 0; h < 4; ++h) mx_add8(lo[h], hi[h], add[h]);
            }
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const uint4 o = mx_round8(lo[h], hi[h]);
              if (inside && m + r8 + 8 * h < M) *reinterpret_cast<uint4*>(p.a.y + at + (size_t)(8 * h) * N) = o;
            }
          }
        } else if (nn + lane < N) {
          const float bias = p.a.bias ? __half2float(p.a.bias[nn + lane]) : 0.f;
#pragma unroll 4
          for (int rr = 0; rr < 32 && m + rr < M; ++rr) {
            const size_t at = (size_t)(m + rr) * N + nn + lane;
            float f = reinterpret_cast<const float*>(turn)[rr * 32 + (((lane >> 2) ^ (rr & 7)) << 2) + (lane & 3)] + bias;
            if (p.a.residual) f += __half2float(p.a.residual[at]);
            p.a.y[at] = __float2half_rn(f);
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
// A call's tile shape and deal: of the shapes built, and with and without the
// split along K, the one whose busiest CTA has least to do, in cycles with every SM at
// work: a stage, what a tile's epilogue keeps the next one's MMAs from, and the join.
// (Stages measured: see above; 1 x 128 680 at 1000 x 2432, where copies are not
// shared by many CTAs.)
struct MbTile {
  int na, nc, db;
  double stage, tail;
};
constexpr MbTile MB_TILES[] = {
    {2, 192, 1, 1160, 5900}, {1, 256, 1, 800, 4200}, {1, 192, 2, 730, 3500}, {1, 128, 2, 570, 2500}};
constexpr double MB_JOIN = 5000;
struct MbPlan {
  int na, nc, mtiles;
  MtDeal d;
};
static MbPlan mb_plan(int M, int N, int K, size_t bytes, int slots) {
  const int stages = (K + MB_K - 1) / MB_K;
  MbPlan best = {};
  double cost = 0;
  for (const MbTile& t : MB_TILES) {
    if (t.na == 2 && M <= 128) continue;
    const int mtiles = (M + 128 * t.na - 1) / (128 * t.na), tiles = mtiles * ((N + t.nc - 1) / t.nc);
    for (int most = 1; most <= MB_SPLIT; ++most) {
      const MtDeal d = mt_deal(tiles, stages, slots, most);
      if (most > 1 && (d.split != most || mt_workspace(d, 128 * t.na, t.nc) > bytes)) continue;
      // two sets of sums: the epilogue costs time of its own only behind the last tile
      const double tile = t.db == 2 ? std::max(stages * t.stage, t.tail) : stages * t.stage + t.tail;
      const double last = t.db == 2 ? t.tail : 0;
      double v;
      if (d.split > 1) v = d.whole / slots * tile + (stages + d.split - 1) / d.split * t.stage + t.tail + MB_JOIN;
      else v = (tiles + slots - 1) / slots * tile + last;
      if (best.na == 0 || v < cost) {
        cost = v;
        best = {t.na, t.nc, mtiles, d};
      }
    }
  }
  return best;
}

size_t mxfp4_a4_workspace(int M, int N, int K) {
  // for the split of a GB300's 152 SMs, so that it can be asked for where there is no GPU
  const MbPlan b = mb_plan(M, N, K, ~(size_t)0, ATW_SMS);
  return mt_workspace(b.d, 128 * b.na, b.nc);
}

int mxfp4_a4_largest_tile() {
  int n = 0;
  for (const MbTile& t : MB_TILES) n = std::max(n, 128 * t.na * t.nc);
  return n;
}

void mxfp4_a4_plan(int M, int N, int K, size_t bytes, int slots, int32_t* plan) {
  const MbPlan b = mb_plan(M, N, K, bytes, slots);
  mt_tell(b.d, 128 * b.na, b.nc, slots, plan);
}

template <int NA, int NC, int DB>
static int mb_launch(MbArgs& p, int slots, cudaStream_t s) {
  using SH = MbShape<NA, NC, DB>;
  static PerDeviceOnce once;
  once_per_device(once, [] {
    cudaFuncSetAttribute(w4pg_mxfp4_a4<NA, NC, DB>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SH::SMEM);
  });
  const MxArgs& a = p.a;
  const bool ok = mt_map(&p.tm_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.xq.codes, a.K / 2, a.M, (uint64_t)a.K / 2, MB_K / 2, 128,
                         CU_TENSOR_MAP_SWIZZLE_128B) &&
                  mt_map(&p.tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w[0].codes, a.K / 2, a.N, (uint64_t)a.K / 2, MB_K / 2, NC,
                         CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return set_error(W4A16_ERR_CUDA, "mxfp4 product: no tensor maps for the operands");
  const cudaError_t e = launch_pdl(w4pg_mxfp4_a4<NA, NC, DB>, dim3(std::min(p.items, slots)), dim3(MB_THREADS), SH::SMEM, s, p);
  if (e != cudaSuccess) return set_error(W4A16_ERR_CUDA, "mxfp4 product launch: %s", cudaGetErrorString(e));
  return W4A16_OK;
}

int launch_mxfp4_a4(const MxArgs& a, cudaStream_t s) {
  MbArgs p = {};
  const int slots = num_sms();
  const MbPlan b = mb_plan(a.M, a.N, a.K, a.workspace ? a.workspace_bytes : 0, slots);
  const MtDeal& d = b.d;
  p.a = a;
  p.mtiles = b.mtiles;
  p.ntiles = (a.N + 127) / 128;
  p.whole = d.whole;
  p.split = d.split;
  p.items = d.items;
  if (d.split > 1) p.parts = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + TC_TICKET_BYTES);
  const int rc = b.na == 2     ? mb_launch<2, 192, 1>(p, slots, s)
                 : b.nc == 256 ? mb_launch<1, 256, 1>(p, slots, s)
                 : b.nc == 192 ? mb_launch<1, 192, 2>(p, slots, s)
                               : mb_launch<1, 128, 2>(p, slots, s);
  if (rc || d.split < 2) return rc;
  return launch_mxfp4_join({a, p.parts, d.whole, (d.items - d.whole) / d.split, d.split, 128 * b.na, b.nc, b.mtiles, b.nc, 0}, s);
}

}  // namespace w4

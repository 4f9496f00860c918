// mxfp4_matvec.cu -- products of a few fp16 rows (decode steps of up to 4
// sequences) with MXFP4 weights.
//
// y[m][n] = sum_k x[m][k] c[n][k] 2^(b[n][k/32] - 127).  At these M the weights'
// bytes are all the time there is (4.25 bits a weight), so the kernel is a stream
// of 16-byte loads with as little work per code as possible.  A lane's 16 bytes
// are one scale block; the hardware conversion makes fp16 pairs of its codes, and
// m16n8k16 MMAs (16 weight rows) take them as they are: the order of k within an
// MMA is free as long as x's fragments follow it.  The MMA's 8 columns are 2 rows
// of x times 4 scale blocks: column 4 m + j holds x[m] in block j and zeros in
// the other three, so that a column's sum over 128 k is one block's, unscaled,
// and the scales enter as 4 fp32 FMAs per 128 k (32 packed multiplications of
// the codes otherwise).  Codes and products are exact, sums fp32.
//
// Split: one persistent CTA of 16 warps per SM; clusters of C CTAs split K (the
// sums meet through distributed shared memory); a cluster's 16-row groups times
// its CTA's scale tiles along K are one stream of units that the 16 warps share
// out evenly, each keeping MV_D units of loads in flight across group borders.
// A warp parks its sum of a group, or of a piece of one, in shared memory; at the
// end the pieces are added in the order of K, whatever the timing.
#include <algorithm>

#include "mxfp4.cuh"
#include "kernels.h"

namespace w4 {

constexpr int MV_WARPS = 16;
constexpr int MV_THREADS = 32 * MV_WARPS;
constexpr int MV_ROWS = 16;
constexpr int MV_GROUPS = 32;    // groups of a cluster between two joins
constexpr int MV_SMEM = 220 * 1024;

__device__ __forceinline__ void mv_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ uint32_t word_of(const uint4& v, int q) { return q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w; }

// a float at the same shared-memory offset in CTA `rank` of the cluster (between
// two cluster barriers: not to be moved)
__device__ __forceinline__ float ld_cluster(const float* p, int rank) {
  uint32_t remote;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
  return v;
}

// a scale beside fp16 activations: bytes that fp16 cannot hold count as zero
__device__ __forceinline__ float mv_scale(uint32_t byte) { return byte < 103 ? 0.f : mx_scale(byte); }

// shared memory: x of this CTA's K in the MMA's order, this CTA's sums of the
// groups, the pieces of them
template <int NW, int MS>
struct MvShape {
  static constexpr int MT = 2 * MS;                      // rows of x
  static constexpr int PIECE = NW * MT * MV_ROWS;        // floats
  static constexpr int D = NW == 2 ? 3 : 6;              // units in flight per warp
  static size_t smem(int ktiles, int groups) {
    const int n = std::min(groups, MV_GROUPS);
    return (size_t)ktiles * 16 * MT * 16 + (size_t)(n + n + MV_WARPS) * PIECE * 4;
  }
};

// NW weight matrices (2: gate and up); MS MMAs per 16 k, 2 rows of x each
template <int NW, int MS>
__global__ void __launch_bounds__(MV_THREADS, 1)
    w4pg_mxfp4_matvec(const __grid_constant__ MxArgs a, int csize, int groups, int gcap) {
  using SH = MvShape<NW, MS>;
  constexpr int MT = SH::MT, PIECE = SH::PIECE, D = SH::D;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int ubegin[MV_WARPS + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % csize, cluster = blockIdx.x / csize, clusters = gridDim.x / csize;
  const int K = a.K, KT = K / 128;
  const int c0 = KT * rank / csize, kc = KT * (rank + 1) / csize - c0;  // this CTA's scale tiles along K
  uint4* xs = reinterpret_cast<uint4*>(smem);
  float* sums = reinterpret_cast<float*>(smem + (size_t)((KT + csize - 1) / csize) * 16 * MT * 16);
  float* pieces = sums + gcap * PIECE;

  const int ngroups = (groups - cluster + clusters - 1) / clusters;  // of this cluster: cluster, cluster + clusters, ..
  const uint4* wp[NW][2];
  const uint8_t* sp[NW];
  // lane's rows g and g + 8 of a group: its 16 rows are four times four, 32 apart,
  // so that their scales are 64 contiguous bytes of a tile; rows past the last
  // read the last one
  auto point = [&](int i) {
    const int group = cluster + i * clusters, row0 = (group >> 3) * 128 + (group & 7) * 4;
    const int r0 = min(row0 + (g & 3) + 32 * (g >> 2), a.N - 1), r1 = min(row0 + (g & 3) + 32 * (g >> 2) + 64, a.N - 1);
    const size_t at = ((size_t)(group >> 3) * KT + c0) * MX_TILE + (group & 7) * 64 + (g & 3) * 16 + (g >> 2) * 4 + 2 * (t & 1);
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      wp[j][0] = reinterpret_cast<const uint4*>(a.w[j].codes + (size_t)r0 * (K / 8)) + 4 * c0 + t;
      wp[j][1] = reinterpret_cast<const uint4*>(a.w[j].codes + (size_t)r1 * (K / 8)) + 4 * c0 + t;
      sp[j] = a.w[j].scales + at;
    }
  };

  uint4 wv[D][NW][2];
  uint16_t sv[D][NW][2];
  float acc[NW][MS][2];
  const bool mine = t == (g & 3);
  const uint4* xl = xs + (g >> 2) * 4 + t;
  const int rounds = (groups + clusters * gcap - 1) / (clusters * gcap);  // as many for every cluster
  for (int round = 0; round < rounds; ++round) {
    const int g0 = round * gcap, ng = min(gcap, max(0, ngroups - g0)), units = ng * kc;
    const int u0 = units * warp / MV_WARPS, u1 = units * (warp + 1) / MV_WARPS;
    if (tid <= MV_WARPS) ubegin[tid] = units * tid / MV_WARPS;
    int li = u0 / kc, lk = u0 - li * kc, lu = u0;  // next unit to load: group, tile
    if (lu < u1) point(g0 + li);
    auto load = [&](int d) {
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        wv[d][j][0] = ldg_stream(wp[j][0] + 4 * lk);
        wv[d][j][1] = ldg_stream(wp[j][1] + 4 * lk);
        const uint8_t* s = sp[j] + (size_t)lk * MX_TILE;
        sv[d][j][0] = *reinterpret_cast<const uint16_t*>(s);
        sv[d][j][1] = *reinterpret_cast<const uint16_t*>(s + 8);
      }
      ++lu;
      if (++lk == kc) {
        lk = 0;
        ++li;
        if (lu < u1) point(g0 + li);
      }
    };
    if (round == 0) {
      // the weights may come from the call just before: into L2 ahead of the wait, read behind it
      if (t == 0) {
#pragma unroll
        for (int d = 0; d < D; ++d)
          if (lu + d < u1 && lk + d < kc) {
#pragma unroll
            for (int j = 0; j < NW; ++j) {
              prefetch_l2(wp[j][0] + 4 * (lk + d));
              prefetch_l2(wp[j][1] + 4 * (lk + d));
            }
          }
      }
      pdl_wait_then_trigger();
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (lu < u1) load(d);
    if (round == 0) {
      // 16 bytes (8 k) of x[m], block t, quarter q of tile kt at [kt][q][m][t]
      for (int i = tid; i < kc * 16 * MT; i += MV_THREADS) {
        const int m = i % MT, c = i / MT;
        if (m < a.M)
          cp_async16(&xs[(((c >> 4) * 4 + (c & 3)) * MT + m) * 4 + ((c >> 2) & 3)], a.x + (size_t)m * K + (c0 * 16 + c) * 8);
      }
      cp_async_commit();
      cp_async_wait<0>();
    }
    __syncthreads();

    int ci = u0 / kc, ck = u0 - ci * kc;  // the unit to add up
#pragma unroll
    for (int j = 0; j < NW; ++j)
#pragma unroll
      for (int s = 0; s < MS; ++s) acc[j][s][0] = acc[j][s][1] = 0.f;
    for (int u = u0; u < u1;) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (u < u1) {
          float c[NW][MS][4] = {};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint4 xv[MS];
#pragma unroll
            for (int s = 0; s < MS; ++s) {
              xv[s] = make_uint4(0, 0, 0, 0);
              if (mine && 2 * s + (g >> 2) < a.M) xv[s] = xl[((ck * 4 + q) * MT + 2 * s) * 4];
            }
#pragma unroll
            for (int j = 0; j < NW; ++j) {
              const uint4 v0 = mx_values(word_of(wv[d][j][0], q)), v1 = mx_values(word_of(wv[d][j][1], q));
#pragma unroll
              for (int s = 0; s < MS; ++s) {
                mv_mma(c[j][s], v0.x, v1.x, v0.y, v1.y, xv[s].x, xv[s].y);
                mv_mma(c[j][s], v0.z, v1.z, v0.w, v1.w, xv[s].z, xv[s].w);
              }
            }
          }
          // columns 2 t, 2 t + 1 of this lane: blocks 2 (t & 1) and the next of row m = t / 2
#pragma unroll
          for (int j = 0; j < NW; ++j) {
            const float a0 = mv_scale(sv[d][j][0] & 255u), a1 = mv_scale(sv[d][j][0] >> 8);
            const float b0 = mv_scale(sv[d][j][1] & 255u), b1 = mv_scale(sv[d][j][1] >> 8);
#pragma unroll
            for (int s = 0; s < MS; ++s) {
              acc[j][s][0] = fmaf(a1, c[j][s][1], fmaf(a0, c[j][s][0], acc[j][s][0]));
              acc[j][s][1] = fmaf(b1, c[j][s][3], fmaf(b0, c[j][s][2], acc[j][s][1]));
            }
          }
          if (lu < u1) load(d);
          ++u;
          if (++ck == kc || u == u1) {
            // a group's, or a piece's, end: piece (warp, group) is number group + warp
            float* p = pieces + (ci + warp) * PIECE;
#pragma unroll
            for (int j = 0; j < NW; ++j)
#pragma unroll
              for (int s = 0; s < MS; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float v = acc[j][s][h] + __shfl_xor_sync(0xffffffffu, acc[j][s][h], 1);
                  if (!(t & 1)) p[(j * MT + 2 * s + (t >> 1)) * MV_ROWS + g + 8 * h] = v;
                  acc[j][s][h] = 0.f;
                }
            ck = 0;
            ++ci;
          }
        }
      }
    }
    __syncthreads();
    // this CTA's sums, each group's pieces in the order of K
    for (int i = tid; i < ng * PIECE; i += MV_THREADS) {
      const int grp = i / PIECE, e = i % PIECE, ua = grp * kc, ub = ua + kc;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < MV_WARPS; ++w)
        if (max(ubegin[w], ua) < min(ubegin[w + 1], ub)) v += pieces[(grp + w) * PIECE + e];
      sums[i] = v;
    }
    if (csize > 1) cluster_sync();
    else __syncthreads();
    // the cluster's: its CTAs take the groups in turn
    for (int i = tid; i < ng * MT * MV_ROWS; i += MV_THREADS) {
      const int grp = i / (MT * MV_ROWS), e = i % (MT * MV_ROWS), m = e / MV_ROWS, r = e % MV_ROWS;
      if (grp % csize != rank || m >= a.M) continue;
      const int group = cluster + (g0 + grp) * clusters;
      const int n = (group >> 3) * 128 + (group & 7) * 4 + (r & 3) + 32 * (r >> 2);
      if (n >= a.N) continue;
      const float* p = sums + grp * PIECE + e;
      float v = 0.f, w = 0.f;
      if (csize == 1) {
        v = p[0];
        if (NW == 2) w = p[MT * MV_ROWS];
      } else {
        for (int c = 0; c < csize; ++c) {
          v += ld_cluster(p, c);
          if (NW == 2) w += ld_cluster(p + MT * MV_ROWS, c);
        }
      }
      if (NW == 2) v = v / (1.f + expf(-v)) * w;
      if (a.bias) v += __half2float(a.bias[n]);
      if (a.residual) v += __half2float(a.residual[(size_t)m * a.N + n]);
      a.y[(size_t)m * a.N + n] = __float2half_rn(v);
    }
    // the sums are read, the pieces' and the sums' places are free
    if (csize > 1) cluster_sync();
    else if (round + 1 < rounds) __syncthreads();
  }
}

// How a call is split: clusters of csize CTAs over K, `clusters` of them.
struct MvPlan {
  int groups, csize, clusters, gcap;
  size_t smem;
};

template <int NW, int MS>
static int mv_max_clusters(int csize, size_t smem) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(csize);
  cfg.blockDim = dim3(MV_THREADS);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = csize;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, w4pg_mxfp4_matvec<NW, MS>, &cfg) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    n = std::max(1, num_sms() / csize - 2);
  }
  return n;
}

// The busiest CTA's units decide, with some MV_JOIN units' time for a join
// through the cluster.
constexpr double MV_JOIN = 16;

template <int NW, int MS>
static MvPlan mv_plan(int N, int K) {
  using SH = MvShape<NW, MS>;
  static PerDeviceOnce once;
  static int room[64][4];  // clusters of 1, 2, 4, 8 CTAs that the device holds at once
  const int dev = device_index() & 63;
  once_per_device(once, [&] {
    cudaFuncSetAttribute(w4pg_mxfp4_matvec<NW, MS>, cudaFuncAttributeMaxDynamicSharedMemorySize, MV_SMEM);
    room[dev][0] = num_sms();
    for (int l = 1; l < 4; ++l) room[dev][l] = mv_max_clusters<NW, MS>(1 << l, MV_SMEM);
  });
  const int groups = N / 128 * 8 + std::min(8, (N % 128 + 3) / 4);  // (those of the last tile that have rows)
  const int ktiles = K / 128;
  MvPlan best = {};
  double cost = 0;
  for (int l = 0; l < 4; ++l) {
    const int c = 1 << l;
    if (c > ktiles && l > 0) break;
    const int clusters = std::min(groups, room[dev][l]);
    const int n = (groups + clusters - 1) / clusters, kc = (ktiles + c - 1) / c, gcap = std::min(n, MV_GROUPS);
    const size_t smem = SH::smem(kc, gcap);
    if (smem > MV_SMEM) continue;
    const double v = (double)n * kc + (l ? MV_JOIN : 0);
    if (best.csize == 0 || v < cost) {
      cost = v;
      best = {groups, c, clusters, gcap, smem};
    }
  }
  return best;
}

template <int NW, int MS>
static int mv_launch(const MxArgs& a, cudaStream_t s) {
  const MvPlan p = mv_plan<NW, MS>(a.N, a.K);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.clusters * p.csize);
  cfg.blockDim = dim3(MV_THREADS);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.csize;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.csize > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, w4pg_mxfp4_matvec<NW, MS>, a, p.csize, p.groups, p.gcap);
  if (e != cudaSuccess) return set_error(W4A16_ERR_CUDA, "mxfp4 product launch: %s", cudaGetErrorString(e));
  return W4A16_OK;
}

bool mxfp4_matvec_serves(int M, int) { return M <= 4; }

int launch_mxfp4_matvec(const MxArgs& a, bool silu, cudaStream_t s) {
  if (silu) return a.M <= 2 ? mv_launch<2, 1>(a, s) : mv_launch<2, 2>(a, s);
  return a.M <= 2 ? mv_launch<1, 1>(a, s) : mv_launch<1, 2>(a, s);
}

}  // namespace w4

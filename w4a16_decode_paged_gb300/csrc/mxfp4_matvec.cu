// mxfp4_matvec.cu -- products of a few fp16 rows (decode steps of one or two
// sequences, of up to 8 where the weights are small) with MXFP4 weights.
//
// y[m][n] = sum_k x[m][k] c[n][k] 2^(b[n][k/32] - 127).  At these M the weights'
// bytes are all the time there is (4.25 bits a weight), so the kernel is a stream of
// 16-byte copies with as little work per code as possible.  A lane's 16 bytes are
// one scale block; the hardware conversion makes fp16 pairs of its codes, and
// m16n8k16 MMAs (16 weight rows) take them as they are: the order of k within an
// MMA is free as long as x's fragments follow it.  The MMA's 8 columns are 2 rows
// of x times 4 scale blocks: column 4 m + j holds x[m] in block j and zeros in
// the other three, so that a column's sum over 128 k is one block's, unscaled,
// and the scales enter as 4 fp32 FMAs per 128 k (32 packed multiplications of
// the codes otherwise).  Codes and products are exact, sums fp32.
//
// Split: one persistent CTA of 16 warps per SM (two for long streams, MV_TWO);
// clusters of C CTAs split K (the sums meet through distributed shared memory); a
// cluster's 16-row groups times its CTA's scale tiles along K are one stream of
// units that its warps share out evenly, each keeping D units of copies in flight
// across group borders, x among them (staged once a CTA ahead of everything, it
// cost 2 us of a call).  A warp parks its sum of a group, or of a piece of one, in
// shared memory; at the end the pieces are added in the order of K, whatever the
// timing.
//
// What bounds it: a call of next to no bytes takes 2.4 us (one row, 512 x 3584:
// launch, one chain of copies, the join), and the stream behind that runs at 5.5 TB/s
// (one row, 152064 x 3584, 52.4 us; a plain copy reaches 6.7): one row of 18944 x 3584
// twice 16.0 us, of 3584 x 18944 9.0 us.  Why the stream stops there is not settled: of
// 145 instructions a unit of 1088 bytes the warps issue at 0.53 of the slots, the
// fullest pipe (integer, which the conversions share) is at 0.47, and no stall stands
// out (13.7 cycles an instruction: 2.7 for the shared-memory queue, 2.2 not chosen, 1.8
// fixed latencies, 1.7 copies).  The conversions alone would be 108 cycles at most of the
// 273 that a unit takes its scheduler (38 and more a clock and SM, registers only).  Two
// chains of MMAs a unit lost 5 %.
#include <algorithm>

#include "mxfp4.cuh"
#include "kernels.h"

namespace w4 {

constexpr int MV_WARPS = 16;
constexpr int MV_THREADS = 32 * MV_WARPS;
constexpr int MV_ROWS = 16;
constexpr int MV_GROUPS = 32;    // groups of a cluster between two joins
template <int MS>
constexpr int MV_D = MS <= 2 ? 4 : 3;  // units in flight per warp

template <bool FIRST>  // FIRST: d = a b, else d += a b
__device__ __forceinline__ void mv_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  if (FIRST)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ uint32_t word_of(const uint4& v, int q) { return q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w; }

// store a float at the same shared-memory offset in CTA `rank` of the cluster
__device__ __forceinline__ void st_cluster(float* p, int rank, float v) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint16_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cpa16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// through L1: x, which the next groups read again
__device__ __forceinline__ void cpa16_ca(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// two scale bytes as fp32
__device__ __forceinline__ float2 mv_scales(uint16_t bytes) {
  const uint32_t v = mx_weight_scales(__byte_perm(bytes, 0, 0x4140));
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

// shared memory: the rings, zeros, this cluster's sums of the groups, this CTA's
// pieces of them
template <int MS>
struct MvShape {
  static constexpr int MT = 2 * MS;                      // rows of x
  static constexpr int PIECE = MT * MV_ROWS;             // floats
  static constexpr int D = MV_D<MS>;
  static constexpr int XAT = 1088;                       // a unit: 16 rows x (64 bytes of codes, 4 of scales), x
  static constexpr int UNIT = XAT + MT * 256;
  static constexpr int RING = MV_WARPS * D * UNIT;
  static constexpr int ZEROS = 4 * MT * 64;              // bytes
  static size_t smem(int groups) {                       // groups: of a round
    return (size_t)RING + ZEROS + (size_t)(groups + 16 + groups + MV_WARPS) * PIECE * 4;
  }
};

// NW weight matrices (2: gate and up, their groups in turn); MS MMAs per 16 k, 2
// rows of x each.  Up to 2 rows 64 registers, so that the next kernel's CTA fits
// beside this one.
template <int NW, int MS>
__global__ void __launch_bounds__(MV_THREADS, MS == 1 ? 2 : 1)
    w4pg_mxfp4_matvec(const __grid_constant__ MxArgs a, int clog, int groups, int gcap) {
  using SH = MvShape<MS>;
  constexpr int MT = SH::MT, PIECE = SH::PIECE, D = SH::D;
  W4_TRACE_SCOPE(0);
  if (clog > 0) cluster_arrive();
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int first[MV_GROUPS], last[MV_GROUPS];  // the warps that have a group's pieces
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int csize = 1 << clog, rank = blockIdx.x & (csize - 1), cluster = blockIdx.x >> clog, clusters = gridDim.x >> clog;
  const int K = a.K, KT = K / 128;
  const int c0 = KT * rank >> clog, kc = (KT * (rank + 1) >> clog) - c0;  // this CTA's scale tiles along K
  const uint32_t ring = smem_u32(smem) + warp * D * SH::UNIT;
  uint4* zeros = reinterpret_cast<uint4*>(smem + SH::RING);
  float* sums = reinterpret_cast<float*>(smem + SH::RING + SH::ZEROS);
  float* pieces = sums + (gcap + 16) * PIECE;

  // the cluster's groups: cluster, cluster + clusters, .., of each matrix in turn
  const int ngroups = NW * ((groups - cluster + clusters - 1) / clusters);
  const uint4 *wp0, *wp1;
  const uint8_t* sp;
  // lane's rows g and g + 8 of a group: its 16 rows are four times four, 32 apart,
  // so that their scales are 64 contiguous bytes of a tile; rows past the last
  // read the last one
  auto point = [&](int i, int kt) {
    const int group = cluster + i / NW * clusters, row0 = (group >> 3) * 128 + (group & 7) * 4 + (g & 3) + 32 * (g >> 2);
    const MxWeights& w = a.w[NW == 2 ? i & 1 : 0];
    const int at = 4 * (c0 + kt) + t;
    wp0 = reinterpret_cast<const uint4*>(w.codes + (size_t)min(row0, a.N - 1) * (K / 8)) + at;
    wp1 = reinterpret_cast<const uint4*>(w.codes + (size_t)min(row0 + 64, a.N - 1) * (K / 8)) + at;
    sp = w.scales + ((size_t)(group >> 3) * KT + c0 + kt) * MX_TILE + (group & 7) * 64 + (lane & 3) * 16;
  };

  // this lane's places in a unit: its codes, the two rows' scales, x.  Column g of
  // the MMA's B is block g % 4 of x's row g / 4 (+ 2 s), read by lane t = g % 4; zeros elsewhere
  const uint32_t rl = ring + lane * 16, rs = ring + 1024 + (g & 3) * 16 + (g >> 2) * 4 + 2 * (t & 1);
  uint32_t rx[MS], xstep[MS];
#pragma unroll
  for (int s = 0; s < MS; ++s) {
    const bool live = t == (g & 3) && 2 * s + (g >> 2) < a.M;
    rx[s] = live ? ring + SH::XAT + ((2 * s + (g >> 2)) * 4 + t) * 16 : smem_u32(zeros);
    xstep[s] = live ? SH::UNIT : 0;
  }
  for (int i = tid; i < SH::ZEROS / 16; i += MV_THREADS) zeros[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  // copies of x: 16 bytes (8 k) of row m, block b, quarter q at [q][m][b]
  const int xc = lane & 15, xm = lane >> 4;
  const uint32_t xto = ring + SH::XAT + (((xc & 3) * MT + xm) * 4 + (xc >> 2)) * 16;
  const __half* const x0 = a.x + (size_t)min(xm, a.M - 1) * K + c0 * 128 + xc * 8;
  const size_t xrows = (size_t)2 * K;  // from one set's rows to the next one's
  bool xlive[MS];
#pragma unroll
  for (int s = 0; s < MS; ++s) xlive[s] = 2 * s + xm < a.M;
  const int most = NW * ((groups + clusters - 1) / clusters), rounds = (most + gcap - 1) / gcap;  // alike in every cluster
  for (int round = 0; round < rounds; ++round) {
    const int g0 = round * gcap, ng = min(gcap, max(0, ngroups - g0)), units = ng * kc;
    const int nw = min(MV_WARPS, max(1, units));  // warps with work: unit u is warp (nw (u + 1) - 1) / units's
    const int u0 = units * min(warp, nw) / nw, u1 = units * min(warp + 1, nw) / nw;
    // next unit to load: its group, the units until the group's or this warp's end, those behind
    int li = u0 / kc, left = min(kc - (u0 - li * kc), u1 - u0), rest = u1 - u0 - left;
    const __half* xp = x0 + (u0 - li * kc) * 128;
    if (left > 0) point(g0 + li, u0 - li * kc);
    auto load = [&](int d) {
      // (a group is committed for every unit, also past the last, so that the
      // wait below counts units)
      if (left > 0) {
        cpa16(rl + d * SH::UNIT, wp0);
        cpa16(rl + d * SH::UNIT + 512, wp1);
        if (lane < 4) cpa16(rl + d * SH::UNIT + 1024, sp);
#pragma unroll
        for (int s = 0; s < MS; ++s)
          if (xlive[s]) cpa16_ca(xto + d * SH::UNIT + s * 128, xp + s * xrows);
        wp0 += 4;
        wp1 += 4;
        sp += MX_TILE;
        xp += 128;
        if (--left == 0 && rest > 0) {
          left = min(kc, rest);
          rest -= left;
          xp = x0;
          point(g0 + ++li, 0);
        }
      }
      cp_async_commit();
    };
    if (round == 0) {
      // the weights may come from the call just before: into L2 ahead of the wait, read behind it
      if (t == 0) {
#pragma unroll
        for (int d = 0; d < 2 * D; d += 2)  // (128 bytes: two tiles)
          if (d < left) {
            prefetch_l2(wp0 + 4 * d);
            prefetch_l2(wp1 + 4 * d);
          }
      }
      pdl_wait_then_trigger();
      W4_TRACE_WAITED();
    }
#pragma unroll
    for (int d = 0; d < D; ++d) load(d);
    W4_TRACE_MARK(0);

    int ci = u0 / kc, togo = u1 - u0;                  // the unit to add up: its group
    int ck = kc - (u0 - ci * kc);                      // units until the group's end
    bool fresh = ck == kc;                             // from its group's first tile
    float acc[MS][2];
#pragma unroll
    for (int s = 0; s < MS; ++s) acc[s][0] = acc[s][1] = 0.f;
#pragma unroll 1
    while (togo > 0) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        float c[MS][4];
        cp_async_wait<D - 1>();
        __syncwarp();
        const uint4 w0 = lds128(rl + d * SH::UNIT), w1 = lds128(rl + d * SH::UNIT + 512);
        const float2 s0 = mv_scales(lds16(rs + d * SH::UNIT)), s1 = mv_scales(lds16(rs + d * SH::UNIT + 8));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint4 v0 = mx_values(word_of(w0, q)), v1 = mx_values(word_of(w1, q));
#pragma unroll
          for (int s = 0; s < MS; ++s) {
            const uint4 xv = lds128(rx[s] + d * xstep[s] + q * MT * 64);
            if (q == 0) mv_mma<true>(c[s], v0.x, v1.x, v0.y, v1.y, xv.x, xv.y);
            else mv_mma<false>(c[s], v0.x, v1.x, v0.y, v1.y, xv.x, xv.y);
            mv_mma<false>(c[s], v0.z, v1.z, v0.w, v1.w, xv.z, xv.w);
          }
        }
        // columns 2 t, 2 t + 1 of this lane: blocks 2 (t & 1) and the next of row m = t / 2
#pragma unroll
        for (int s = 0; s < MS; ++s) {
          acc[s][0] = fmaf(s0.y, c[s][1], fmaf(s0.x, c[s][0], acc[s][0]));
          acc[s][1] = fmaf(s1.y, c[s][3], fmaf(s1.x, c[s][2], acc[s][1]));
        }
        __syncwarp();  // (the scales are read by other lanes than copied them)
        load(d);
        --togo;
        if (--ck == 0 || togo == 0) {
          // a group's, or a piece's, end: piece (warp, group) is number group + warp
          float* p = pieces + (ci + warp) * PIECE;
          if (lane == 0) {
            if (fresh) first[ci] = warp;
            if (ck == 0) last[ci] = warp;
          }
          fresh = true;
#pragma unroll
          for (int s = 0; s < MS; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float v = acc[s][h] + __shfl_xor_sync(0xffffffffu, acc[s][h], 1);
              if (!(t & 1)) p[(2 * s + (t >> 1)) * MV_ROWS + g + 8 * h] = v;
              acc[s][h] = 0.f;
            }
          ck = kc;
          ++ci;
          if (togo == 0) break;
        }
      }
    }
    // this thread's first output, and what is added to it, asked for ahead of the join
    struct Out {
      bool live;
      size_t at;
      float add;
    };
    auto place_of = [&](int i) {
      const int e = i % PIECE, m = e / MV_ROWS, r = e % MV_ROWS, pair = (i / PIECE << clog) + rank;
      const int group = cluster + (g0 / NW + pair) * clusters;
      const int n = (group >> 3) * 128 + (group & 7) * 4 + (r & 3) + 32 * (r >> 2);
      Out o = {pair * NW < ng && m < a.M && n < a.N, (size_t)m * a.N + n, 0.f};
      if (o.live && a.bias) o.add = __half2float(a.bias[n]);
      if (o.live && a.residual) o.add += __half2float(a.residual[o.at]);
      return o;
    };
    Out o = place_of(tid);
    __syncthreads();
    W4_TRACE_MARK(1);
    // this CTA's sums, each group's pieces in the order of K
    if (csize > 1) cluster_wait();  // every CTA of the cluster has started, and read its sums of the round before
    for (int i = tid; i < ng * PIECE; i += MV_THREADS) {
      const int grp = i / PIECE, e = i % PIECE;
      float v = 0.f;
      for (int w = first[grp]; w <= last[grp]; ++w) v += pieces[(grp + w) * PIECE + e];
      // to the CTA of the cluster that joins this group (they take them in turn, gate and up together)
      const int pair = grp / NW, owner = pair & (csize - 1), place = (pair - owner + rank) * NW + grp % NW;
      if (csize == 1) sums[place * PIECE + e] = v;
      else st_cluster(sums + place * PIECE + e, owner, v);
    }
    __syncwarp();  // the cluster's barriers are for whole warps
    if (csize > 1) cluster_sync();
    else __syncthreads();
    W4_TRACE_MARK(2);
    for (int i = tid;;) {
      if (!o.live) break;
      const float* p = sums + (i / PIECE << clog) * NW * PIECE + i % PIECE;
      float v = 0.f, w = 0.f;
      for (int c = 0; c < csize; ++c) {
        v += p[c * NW * PIECE];
        if (NW == 2) w += p[c * NW * PIECE + PIECE];
      }
      if (NW == 2) v = v / (1.f + expf(-v)) * w;
      a.y[o.at] = __float2half_rn(v + o.add);
      o = place_of(i += MV_THREADS);
    }
    if (round + 1 < rounds) {
      __syncwarp();  // lanes leave the loop above at different turns
      if (csize > 1) cluster_arrive();
      __syncthreads();
    }
  }
}

// How a call is split: clusters of csize CTAs over K, `clusters` of them.
struct MvPlan {
  int groups, clog, clusters, gcap;
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
// From so many units per warp two CTAs share an SM instead of leaving room for the
// next kernel's: b1 gate|up (28) 15.8 us against 16.4, down (14) 10.7 against 9.0
// (before the scales below 104 and above 140 were told apart, 0.2 and 0.1 us).
constexpr int MV_TWO = 20;

template <int NW, int MS>
static MvPlan mv_plan(int N, int K) {
  using SH = MvShape<MS>;
  static PerDeviceOnce once;
  static int room[64][4];  // clusters of 1, 2, 4, 8 CTAs that the device holds at once
  const int dev = device_index() & 63;
  once_per_device(once, [&] {
    cudaFuncSetAttribute(w4pg_mxfp4_matvec<NW, MS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SH::smem(MV_GROUPS));
    room[dev][0] = 2 * num_sms();
    for (int l = 1; l < 4; ++l) room[dev][l] = mv_max_clusters<NW, MS>(1 << l, SH::smem(MV_GROUPS));
  });
  const int groups = N / 128 * 8 + std::min(8, (N % 128 + 3) / 4);  // (those of the last tile that have rows)
  const int ktiles = K / 128, sms = num_sms();
  const int per = MS == 1 && (long long)NW * groups * ktiles >= (long long)MV_TWO * MV_WARPS * sms ? 2 : 1;
  MvPlan best = {};
  double cost = 0;
  for (int l = 0; l < 4; ++l) {
    const int c = 1 << l;
    if (c > ktiles || c > per * sms) break;  // (no device: one SM is assumed, and the launch fails)
    const int clusters = std::min(groups, std::min(room[dev][l], per * sms / c));
    const int n = NW * ((groups + clusters - 1) / clusters), kc = (ktiles + c - 1) / c, gcap = std::min(n, MV_GROUPS);
    const double v = (double)n * kc + (l ? MV_JOIN : 0);
    if (best.groups == 0 || v < cost) {
      cost = v;
      best = {groups, l, clusters, gcap, SH::smem(gcap)};
    }
  }
  return best;
}

template <int NW, int MS>
static int mv_launch(const MxArgs& a, cudaStream_t s) {
  const MvPlan p = mv_plan<NW, MS>(a.N, a.K);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.clusters << p.clog);
  cfg.blockDim = dim3(MV_THREADS);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1 << p.clog;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.clog > 0 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, w4pg_mxfp4_matvec<NW, MS>, a, p.clog, p.groups, p.gcap);
  if (e != cudaSuccess) return set_error(W4A16_ERR_CUDA, "mxfp4 product launch: %s", cudaGetErrorString(e));
  return W4A16_OK;
}

// Up to 2 rows always (gate|up 17.6 us against 19.7 on the tensor cores).  3 and 4
// take twice the MMAs a unit, 5 to 8 four times, and win while the tensor-core
// kernel's start and join decide: up to so many scale tiles of weights.  4 rows,
// 3584 x 3584 (784 tiles): 4.9 us against 8.3, 18944 x 3584 twice (8288): 25 against
// 19.7; 8 rows, 784 tiles: 7.5 against 8.4, 1568 tiles: 11.5 against 10.9.
constexpr long long MV_TILES4 = 4096, MV_TILES8 = 1200;
bool mxfp4_matvec_serves(int M, int N, int K, bool silu) {
  const long long tiles = (long long)((N + 127) / 128) * (K / 128) * (silu ? 2 : 1);
  return M <= 2 || (M <= 8 && tiles <= (M <= 4 ? MV_TILES4 : MV_TILES8));
}

void mxfp4_matvec_plan(int M, int N, int K, bool silu, int32_t* plan) {
  const MvPlan p = silu ? (M <= 2 ? mv_plan<2, 1>(N, K) : M <= 4 ? mv_plan<2, 2>(N, K) : mv_plan<2, 4>(N, K))
                        : (M <= 2 ? mv_plan<1, 1>(N, K) : M <= 4 ? mv_plan<1, 2>(N, K) : mv_plan<1, 4>(N, K));
  const int most = (silu ? 2 : 1) * ((p.groups + p.clusters - 1) / p.clusters);
  plan[0] = 0;
  plan[1] = 1 << p.clog;
  plan[2] = p.clusters;
  plan[3] = most;
  plan[4] = (most + p.gcap - 1) / p.gcap;
  plan[5] = plan[6] = 0;
}

int launch_mxfp4_matvec(const MxArgs& a, bool silu, cudaStream_t s) {
  if (silu) return a.M <= 2 ? mv_launch<2, 1>(a, s) : a.M <= 4 ? mv_launch<2, 2>(a, s) : mv_launch<2, 4>(a, s);
  return a.M <= 2 ? mv_launch<1, 1>(a, s) : a.M <= 4 ? mv_launch<1, 2>(a, s) : mv_launch<1, 4>(a, s);
}

}  // namespace w4

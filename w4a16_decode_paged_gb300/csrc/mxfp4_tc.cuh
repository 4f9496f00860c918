// mxfp4_tc.cuh -- what the MXFP4 tensor-core products share: bounded barrier
// waits, bulk-tensor copies and their maps, tcgen05 descriptors, and how a
// product's output tiles are dealt to CTAs.
#pragma once

#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "mxfp4.cuh"
#include "kernels.h"

namespace w4 {

constexpr long long MT_TIMEOUT_CYCLES = 4000000000ll;  // 2 s at the highest clock

// One lane of a converged warp.  (Chosen by elect.sync, and with the warp's number
// taken from one lane, so that what follows is known to be uniform: with MMAs behind
// `lane == 0` a stage took 1.03 us where it takes 0.51 now (fp16, 32 rows of x), and
// 0.86 where it takes 0.61 (4-bit, 2 x 128 x 192).)
__device__ __forceinline__ bool mt_elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Bounded wait; gives up as well once another role of the CTA has (*fail).
// fail null: only its own bound counts (drains).
__device__ __forceinline__ bool mt_wait(uint64_t* bar, uint32_t parity, volatile int* fail) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (fail && *fail) return false;
    if (clock64() - t0 > MT_TIMEOUT_CYCLES) {
      if (fail) *fail = 1;
      return false;
    }
  }
}

__device__ __forceinline__ void mt_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void mt_prefetch_2d(const CUtensorMap* map, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void mt_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// `bytes` (a multiple of 16) in one piece
__device__ __forceinline__ void mt_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void mt_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mt_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void mt_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor of a K-major tile with 128-byte rows in the
// 128-byte swizzle (8-row atoms of 1024 bytes); 32 bytes of a row further on is
// two more in its address field.
__device__ __forceinline__ uint64_t mt_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// 2-D map over rows of `inner` elements, `row_bytes` apart; boxes of box_inner x
// box_rows (what lies outside reads as zeros)
bool mt_map(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t rows, uint64_t row_bytes,
            uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle sw);

// How T output tiles of `stages` steps along K are dealt to `slots` CTAs: whole
// rounds of tiles as they are, and what is left over split along K, so that the
// last round is as full as the others.  The parts' fp32 sums go to the workspace
// and a second kernel adds them in order (launch_mxfp4_join).
struct MtDeal {
  int whole;      // tiles that are not split: items 0 .. whole - 1
  int split;      // parts of each other tile
  int items;
};
inline MtDeal mt_deal(int tiles, int stages, int slots, int most_split) {
  MtDeal d = {tiles, 1, tiles};
  const int over = tiles % slots;
  if (over == 0 || most_split < 2) return d;
  const int split = std::min(std::min(slots / over, stages / 2), most_split);
  if (split < 2) return d;
  d.whole = tiles - over;
  d.split = split;
  d.items = d.whole + over * split;
  return d;
}
inline void mt_tell(const MtDeal& d, int tm, int tn, int slots, int32_t* plan) {
  plan[0] = 1;
  plan[1] = tm;
  plan[2] = tn;
  plan[3] = d.whole;
  plan[4] = d.split > 1 ? (d.items - d.whole) / d.split : 0;
  plan[5] = d.split;
  plan[6] = std::min(d.items, slots);
}
// Parts in the workspace lie behind the block that the other split-K calls keep
// their tickets in; a part is [rows of x][weight rows] of its tile, fp32.
inline size_t mt_workspace(const MtDeal& d, int tm, int tn) {
  return d.split > 1 ? TC_TICKET_BYTES + (size_t)(d.items - d.whole) * tm * tn * 4 : 0;
}
struct MtJoin {
  MxArgs a;
  const float* parts;
  int first, tiles, split;   // the split tiles: numbers first .. first + tiles - 1, in `split` parts each
  int tm, tn, mtiles;        // tile t covers rows tm (t % mtiles) .., weight rows tstep (t / mtiles) ..
  int tstep, silu;           // silu: a part's columns are 128 gate, 128 up
};
int launch_mxfp4_join(const MtJoin& j, cudaStream_t s);

__device__ __host__ __forceinline__ void mt_item(int i, int whole, int split, int stages, int* tile, int* part, int* k0,
                                                  int* k1) {
  *tile = i < whole ? i : whole + (i - whole) / split;
  *part = i < whole ? 0 : (i - whole) % split;
  *k0 = i < whole ? 0 : (int)((long long)stages * *part / split);
  *k1 = i < whole ? stages : (int)((long long)stages * (*part + 1) / split);
}

}  // namespace w4

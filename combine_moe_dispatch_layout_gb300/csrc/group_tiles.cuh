// group_tiles.cuh -- the row offsets and the tile prefix of a grouped problem,
// built in shared memory by every CTA from the device's row counts.
#pragma once

#include "moe_ep_internal.cuh"

namespace moe_ep {

// Rows of group g (a negative count is reported and read as 0); without counts
// there is one group of every row.
__device__ __forceinline__ int group_count(const LinearArgs& p, int g, int32_t* dev_status) {
  if (!p.group_rows) return static_cast<int>(p.a_rows);
  const int c = p.group_rows[g];
  if (c < 0 && dev_status) set_status(dev_status, MOE_ERR_INVALID_ARG);
  return c < 0 ? 0 : c;
}

// Blocks of at most `block` rows in a group of cnt rows.
__device__ __forceinline__ int row_blocks(int cnt, int block) {
  return static_cast<int>((int64_t(cnt) + block - 1) / block);
}

__device__ __forceinline__ int smem_load(uint32_t a) {
  int v;
  asm volatile("ld.shared.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void smem_store(uint32_t a, int v) {
  asm volatile("st.shared.s32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// goff[g] = first row of group g, tpre[g] = tiles before it (shared-memory
// addresses of G + 1 words each; the last ones are the totals), a group having
// row_blocks(rows, block) * ntn tiles.  More rows than the buffer holds set
// MOE_ERR_CAPACITY and leave no tiles.  s_scan: 12 * THREADS bytes, 8-aligned (a caller whose
// bulk or tensor copies write there later fences the proxies first, in every thread).
// All THREADS threads take part; the tables are ready after the caller's next
// __syncthreads().
template <int THREADS>
__device__ __forceinline__ void build_group_tables(const LinearArgs& p, int block, int ntn,
                                                   void* s_scan, uint32_t goff, uint32_t tpre,
                                                   int32_t* dev_status) {
  const int tid = threadIdx.x, lane = tid & 31;
  const int per = (p.G + THREADS - 1) / THREADS;
  const int g0 = min(tid * per, p.G), g1 = min(g0 + per, p.G);
  int64_t rsum = 0;
  int tsum = 0;
  for (int g = g0; g < g1; ++g) {
    const int c = group_count(p, g, dev_status);
    rsum += c;
    tsum += row_blocks(c, block) * ntn;
  }
  int64_t* s_r = static_cast<int64_t*>(s_scan);
  int* s_t = reinterpret_cast<int*>(s_r + THREADS);
  s_r[tid] = rsum;
  s_t[tid] = tsum;
  __syncthreads();
  if (tid < 32) {             // exclusive scan of the threads' sums
    constexpr int kPer = THREADS / 32;
    int64_t r = 0;
    int tt = 0;
    for (int i = 0; i < kPer; ++i) {
      r += s_r[lane * kPer + i];
      tt += s_t[lane * kPer + i];
    }
    int64_t ri = r;
    int ti = tt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, ri, d);
      const int b = __shfl_up_sync(0xffffffffu, ti, d);
      if (lane >= d) {
        ri += a;
        ti += b;
      }
    }
    int64_t re = ri - r;
    int te = ti - tt;
    for (int i = 0; i < kPer; ++i) {
      const int64_t a = s_r[lane * kPer + i];
      const int b = s_t[lane * kPer + i];
      s_r[lane * kPer + i] = re;
      s_t[lane * kPer + i] = te;
      re += a;
      te += b;
    }
    if (lane == 31) {
      const bool over = re > p.a_rows;
      if (over) set_status(dev_status, MOE_ERR_CAPACITY);
      smem_store(goff + 4 * p.G, over ? 0 : static_cast<int>(re));
      smem_store(tpre + 4 * p.G, over ? 0 : te);
    }
  }
  __syncthreads();
  int64_t r = s_r[tid];
  int tt = s_t[tid];
  for (int g = g0; g < g1; ++g) {
    smem_store(goff + 4 * g, static_cast<int>(min(r, p.a_rows)));
    smem_store(tpre + 4 * g, tt);
    const int c = group_count(p, g, nullptr);
    r += c;
    tt += row_blocks(c, block) * ntn;
  }
}

// The group that tile t belongs to: the largest g with tpre[g] <= t.
__device__ __forceinline__ int group_of_tile(int t, uint32_t tpre, int G) {
  int lo = 0, hi = G;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (smem_load(tpre + 4 * mid) <= t) lo = mid; else hi = mid;
  }
  return lo;
}

}  // namespace moe_ep

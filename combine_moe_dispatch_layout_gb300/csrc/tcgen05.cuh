// tcgen05.cuh -- thin wrappers over the tensor-core, TMEM, tensor-copy and
// cluster instructions of sm_103a used by the 8-bit matrix product.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "moe_ep_internal.cuh"

namespace moe_ep {

// True in one lane of a converged warp.  Loops around tensor copies and products
// run in the whole warp and issue under this predicate: the operands then stay
// in uniform registers (under a per-lane condition, an issue took 200 cycles).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// ---- mbarriers by 32-bit shared-memory address (half the registers of
// generic pointers) -------------------------------------------------
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool bar_poll(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for phase `parity` at most kGemmSpin polls; false on timeout.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
  for (uint32_t i = 0; i < kGemmSpin; ++i)
    if (bar_poll(bar, parity)) return true;
  return false;
}
// The same for a whole converged warp, which stays so (a lane's own loop made the compiler
// guard every wait against divergence, and spill what it keeps for that).  Every lane has to
// see the phase itself: one that has not has acquired nothing of what lies behind it.
__device__ __forceinline__ bool warp_bar_wait(uint32_t bar, uint32_t parity) {
  for (uint32_t i = 0; i < kGemmSpin; ++i)
    if (__all_sync(0xffffffffu, bar_poll(bar, parity))) return true;
  return false;
}
// Waits for phase `parity` of three barriers and `pd` of a fourth, a whole converged warp,
// with their polls in flight together (one after the other they took 90 clocks each though
// the phases were complete).
__device__ __forceinline__ bool warp_bar_wait4(uint32_t a, uint32_t b, uint32_t c, uint32_t parity,
                                               uint32_t d, uint32_t pd) {
  for (uint32_t i = 0; i < kGemmSpin; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q, r, s;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %4;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 q, [%2], %4;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 r, [%3], %4;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 s, [%5], %6;\n\t"
        "and.pred p, p, q;\n\tand.pred r, r, s;\n\tand.pred p, p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(a), "r"(b), "r"(c), "r"(parity), "r"(d), "r"(pd)
        : "memory");
    if (__all_sync(0xffffffffu, ok != 0)) return true;
  }
  return false;
}
// 2-D tensor copy global -> shared, completion counted on `bar`.
__device__ __forceinline__ void tensor_load_2d(uint32_t sdst, const CUtensorMap* map, int x,
                                               int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(sdst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// 2-D tensor copy shared -> global (tracked by bulk groups); what lies outside the map is
// left out.
__device__ __forceinline__ void tensor_store_2d(const CUtensorMap* map, int x, int y,
                                                uint32_t ssrc) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
               ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(ssrc) : "memory");
}

__device__ __forceinline__ void tensor_map_prefetch(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Descriptor of a K-major operand tile in shared memory: rows of 128 bytes,
// 128-byte swizzle, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
  uint64_t d = uint64_t((saddr & 0x3FFFFu) >> 4);
  d |= uint64_t(1) << 16;
  d |= uint64_t(1024 >> 4) << 32;
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}

// fp16 x fp16 -> fp32, both operands K-major; m, n: the instruction's shape.
__device__ __forceinline__ uint32_t f16_mma_desc(int m, int n) {
  return (1u << 4) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 4 consecutive TMEM columns of this warp's 32 lanes (more at once would cost
// registers where sums fill them).
__device__ __forceinline__ void tmem_load4(uint32_t taddr, uint32_t (&v)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// 8 consecutive TMEM columns of this warp's 32 lanes: the load starts here, and v may be
// read after tmem_wait8(v) alone (which names the registers, so that no use of them can
// be moved before it).
__device__ __forceinline__ void tmem_start8(uint32_t taddr, float (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                 "=f"(v[6]), "=f"(v[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait8(float (&v)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7])
               :
               : "memory");
}

// ---- clusters -------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int cluster_id() {        // which cluster, of how many
  int r;
  asm("mov.s32 %0, %%clusterid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int cluster_count() {
  int r;
  asm("mov.s32 %0, %%nclusterid.x;" : "=r"(r));
  return r;
}
// Every thread of every CTA of the cluster; earlier writes (also to another
// CTA's shared memory) are visible after it.
__device__ __forceinline__ void cluster_arrive_all() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
// The same without waiting for earlier writes: enough where all that the others need to see
// is barriers set up before a fence_mbar_init().
__device__ __forceinline__ void cluster_arrive_all_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_all() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive_all();
  cluster_wait_all();
}
// The same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
__device__ __forceinline__ void cluster_store(uint32_t caddr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(caddr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_store16(uint32_t caddr, const int32_t* v) {
  asm volatile("st.shared::cluster.v4.s32 [%0], {%1,%2,%3,%4};" ::"r"(caddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// One arrival on an mbarrier of any CTA of the cluster (address from
// cluster_addr).  The data that such an arrival announces here is read by the
// tensor core of the CTA that wrote it, after that CTA's own proxy fence, so
// the default (CTA-scope) release is enough; a cluster-scope release made
// every arrival wait over 1000 cycles for the CTA's stores in flight.
__device__ __forceinline__ void cluster_arrive(uint32_t caddr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(caddr) : "memory");
}

// The same from the lanes where `lane` holds, without a branch.
__device__ __forceinline__ void cluster_arrive_if(bool lane, uint32_t caddr) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(caddr), "r"(uint32_t(lane))
      : "memory");
}

// The products of one instruction (K = 16) of a pair of CTAs, issued by the
// pair's first CTA alone; each CTA holds half of both operands.
__device__ __forceinline__ void pair_mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}
// The same for 8-bit floats (K = 32), both e4m3; the instruction descriptor is that of
// f16_mma_desc, whose type fields are 0 for fp16 and for e4m3 alike.
__device__ __forceinline__ void pair_mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}
// Arrives on `bar` in the CTAs of `mask` (ranks in the cluster), at the same
// offset, once every product issued so far by this thread is done.
__device__ __forceinline__ void pair_commit(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
      ".b64 [%0], %1;" ::"r"(bar), "h"(mask) : "memory");
}
// TMEM columns of a pair: one warp of each of its CTAs takes part.
__device__ __forceinline__ void pair_tmem_alloc(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
               "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_free(uint32_t tmem, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
               : "memory");
}

// The same of a CTA by itself.
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar) : "memory");
}
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
               "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
               : "memory");
}

// Registers of this warpgroup (all four warps): more, or fewer.
template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_fewer() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Host: a 2-D map of `rows` rows of `cols` bytes, `stride` bytes apart, copied
// in boxes of 128 x box_rows with the 128-byte swizzle; bytes outside read as 0.
cudaError_t encode_bytes_2d(CUtensorMap* map, const void* base, int64_t rows, int64_t cols,
                            int64_t stride, uint32_t box_rows);

}  // namespace moe_ep

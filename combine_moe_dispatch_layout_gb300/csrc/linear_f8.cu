// linear_f8.cu -- matrix product of e4m3 rows and weights with a scale per 128 codes of a
// row and per 128 x 128 block of a weight matrix, rows grouped by expert
// (include/moe_ep.h, moe_linear_f8).
//
// Mathematics.  c[m][n] = sum over blocks b of 128 codes of
//   (a_scale[m][b] * w_scale[n / 128][b]) * sum_{j in b} a[m][j] w[n][j]   (+ bias[n]).
// The inner sums are the tensor cores' (fp32); their scales differ from block to block, so
// every block's sums leave TMEM and meet their scale in one fused multiply-add in fp32
// registers.
//
// Tile: a pair of CTAs (two SMs of a cluster) takes 256 tokens (the MMA's M, 128 TMEM
// lanes on each SM) x up to 256 channels (its N); each SM holds its 128 token rows and half
// of the weight rows.  Tokens are on the lanes so that a draining thread has one token:
// its scale is one register, and the multiply-adds take two columns per instruction.
// Warps of a CTA (one CTA per SM, persistent):
//   warp 0   copies its 128 token rows, 128 bytes of each, into a ring of stages (tensor
//            copies, 128-byte swizzle), and warp 2 its half of the weight rows (one warp
//            for both took 400 clocks a stage, which shows in narrow tiles)
//   warp 1   of the pair's first CTA: issues tcgen05.mma (K = 32), four per 128-code
//            block, into the TMEM accumulators in turn (two for 256 channels); of its
//            second CTA: tells the first which of its stages have landed
//   8 warps  drain a block's sums, scale and add them, and store the tile
// (kPair.)  Groups of few rows are taken by CTAs by themselves, 128 tokens x 256 channels
// (kSingle).  Where there are few tiles a cluster of two pairs splits K (kHalves): each pair
// sends its sums of one half of a CTA's rows to the other one's shared memory, adds what it
// gets to its own sums of the other half, and stores those.
// Every wait is bounded: a timeout sets MOE_ERR_TIMEOUT, the CTA stops issuing work and
// drains what is in flight.
//
// What bounds it.  A block of 128 codes is 512 clocks of products for a full tile (596 with
// its copies, which share the shared memory's port), and its accumulator stays taken through
// them, the commit's way to the draining warps, the drain (its 32,768 multiply-adds are 256
// clocks of the SM's pipes; the last column is loaded some 350 after the first) and the
// arrival's way back: with two accumulators 876 clocks a block (8192 x 4096 x 7168, ncu).
// Looped for longer than 20 ms the board is at its power limit and lowers the clock, so
// energy counts more than clocks: 166 us in bursts, 183 to 188 looped (a library product
// without block scales 127 and 144).  Measured beside it: 32,768 x 7168 x 2048 in 32 uneven
// groups 417 us, 1024 x 4096 x 4096 19.8, 256 x 4096 x 7168 16.1, 8192 rows over 256 groups
// of 4096 x 7168 1111 (6.85 TB/s, kSingle), 197 x 1001 x 1992 in fp32 10.6 to 12.  Slower for the
// first: four accumulators of 128 columns (the products read the token rows twice: 210), 16
// draining warps (178), TMEM loads of 4, 16 or 32 columns (198, 169, 210; of 8 here), scalar
// multiply-adds (215), single CTAs instead of pairs (as many clocks, 3% more energy).
#include <cuda.h>

#include <algorithm>

#include "group_tiles.cuh"
#include "moe_ep_internal.cuh"
#include "row_codes.cuh"
#include "tcgen05.cuh"

namespace moe_ep {

// linear_f8_polls.cu compiles this file a second time, for tests of the waits that run
// out: with role waits of its own, and without the function that others call.
#ifndef MOE_LINEAR_F8_POLLS
namespace {
// A role's waits for its next work; false after kGemmSpin polls.
__device__ __forceinline__ bool warp_role_wait(uint32_t bar, uint32_t parity) {
  return warp_bar_wait(bar, parity);
}
__device__ __forceinline__ bool warp_role_wait2(uint32_t a, uint32_t b, uint32_t parity) {
  return warp_bar_wait4(a, b, b, parity, a, parity);
}
__device__ __forceinline__ bool warp_role_wait4(uint32_t a, uint32_t b, uint32_t c,
                                                uint32_t parity, uint32_t d, uint32_t pd) {
  return warp_bar_wait4(a, b, c, parity, d, pd);
}
}  // namespace
#endif

namespace {

enum Form { kPair, kHalves, kSingle };       // two CTAs to a tile, two pairs, one CTA
__host__ __device__ constexpr int ctas_of(int form) {        // that multiply together
  return form == kSingle ? 1 : 2;
}
constexpr int TM = 128;              // tokens per CTA
constexpr int BK = kCodeBlock;       // codes per stage: one 128-byte row
constexpr int kRasterTokens = 8;     // token blocks per raster band (weights reused from L2)
constexpr int kEpiWarps = 8, kCtrlWarps = 4;
constexpr int kThreads = 32 * (kCtrlWarps + kEpiWarps);
// Registers per thread: 168 at launch, handed out again by role.
constexpr int kEpiRegs = 216, kCtrlRegs = 72;
static_assert(32 * (kEpiWarps * kEpiRegs + kCtrlWarps * kCtrlRegs) <= kThreads * 168,
              "no more registers than the launch has");
constexpr uint32_t kTmemCols = 512;
constexpr int kTurn = 4;             // blocks per turn of a draining thread, see load_scales
constexpr int kMaxStages = 10;
constexpr uint32_t kBoxBytes = 32 * 128;             // a warp's 32 rows of 128 output bytes
// (a CTA by itself has the second box's memory for another stage)
__host__ __device__ constexpr int boxes_of(int form) { return form == kSingle ? 1 : 2; }
constexpr int kMaxTable = 64;                        // a cluster's first tiles, decoded ahead

struct Maps {
  CUtensorMap w, a, c;       // weights, token rows, the result
};

// NT: channels per tile.
template <int NT, int FORM>
struct Stages {
  // Accumulators: what TMEM holds.  (A block's way from its products' commit to the drain
  // and back takes some 800 clocks, four times as long as a narrow tile's products.)
  static constexpr int kAccs = kTmemCols / NT;
  static constexpr uint32_t kBytes = (TM + NT / ctas_of(FORM)) * BK;
  static constexpr uint32_t kOutBytes = kEpiWarps * boxes_of(FORM) * kBoxBytes;
  static constexpr uint32_t kBarBytes = 464;
  // the other pair's sums of half the rows
  static constexpr uint32_t kSumBytes = FORM == kHalves ? TM / 2 * NT * 4 : 0;
  static size_t bytes(int stages, int table, int G) {
    return 1024 + size_t(stages) * kBytes + kOutBytes + kSumBytes + kBarBytes +
           size_t(table) * 16 + size_t(G + 1) * 8;
  }
};

struct Tile {
  int g;           // group
  int n0;          // first output channel
  int row0;        // first token row
  int rows;        // tokens of the group from there on, at most a tile's
};

template <int NT, int FORM>
__device__ __forceinline__ Tile decode_tile(int t, uint32_t goff, uint32_t tpre, int G, int ntn) {
  constexpr int CG = ctas_of(FORM);
  const int lo = group_of_tile(t, tpre, G);
  const int off = smem_load(goff + 4 * lo);
  const int cnt = smem_load(goff + 4 * lo + 4) - off;
  const int local = t - smem_load(tpre + 4 * lo);
  const int blocks = row_blocks(cnt, CG * TM);
  // bands of kRasterTokens token blocks (the last band takes the remainder); inside a
  // band the token block is fastest, so the CTAs in flight share weight tiles and a
  // bounded number of token blocks
  const int nband = max(blocks / kRasterTokens, 1), per_band = kRasterTokens * ntn;
  const int band = min(local / per_band, nband - 1);
  const int width = band < nband - 1 ? kRasterTokens : blocks - band * kRasterTokens;
  const int r = local - band * per_band;
  const int nblk = r / width, mblk = band * kRasterTokens + r - nblk * width;
  Tile tl;
  tl.g = lo;
  tl.n0 = nblk * NT;
  tl.row0 = off + mblk * (CG * TM);
  tl.rows = min(CG * TM, cnt - mblk * (CG * TM));
  return tl;
}

template <int OUT>
__device__ __forceinline__ uint32_t narrow_pair(float lo, float hi) {
  uint32_t h;
  if constexpr (OUT == MOE_BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
  return h;
}

// Blocks of K of the first of two parts: whole turns of a draining thread.
__host__ __device__ __forceinline__ int first_blocks(int K) {
  return static_cast<int>(align_up((code_blocks(K) + 1) / 2, kTurn));
}

template <int NT, int OUT, int FORM>
__global__ void __launch_bounds__(kThreads, 1)
linear_f8_tile_kernel(const __grid_constant__ Maps maps, const LinearArgs p, bool wide_scales,
                      int stages, int entries, int32_t* dev_status) {
  using St = Stages<NT, FORM>;
  constexpr int CG = ctas_of(FORM);
  constexpr bool SPLIT = FORM == kHalves;      // two pairs to a cluster, which takes one tile
  constexpr int kCols = NT / (kEpiWarps / 4);          // columns per draining thread
  constexpr int kAccs = St::kAccs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t outs = sbase + stages * St::kBytes, sums = outs + St::kOutBytes;
  const uint32_t bars = sums + St::kSumBytes;
  // A stage's token rows (0) and weight rows (1) of this CTA landed: a barrier for each warp
  // that copies, which after a timeout waits for its own copies whatever the other has done.
  auto full = [&](int of, int s) { return bars + 8 * (of * kMaxStages + s); };
  auto peer = [&](int s) { return bars + 8 * (2 * kMaxStages + s); };   // ... the other CTA's
  auto empty = [&](int s) { return bars + 8 * (3 * kMaxStages + s); };  // multiplied
  constexpr int kT0 = 4 * kMaxStages;
  auto tfull = [&](int b) { return bars + 8 * (kT0 + b); };             // accumulator final
  auto tempty = [&](int b) { return bars + 8 * (kT0 + kAccs + b); };    // ... drained
  const uint32_t tmem_slot = bars + 8 * (kT0 + 2 * kAccs), abort_flag = tmem_slot + 4;
  const uint32_t issued = abort_flag + 4;    // the pair's commits: of stages, of accumulators
  static_assert(8 * (kT0 + 2 * kAccs) + 16 <= St::kBarBytes, "barriers fit");
  const uint32_t table = bars + St::kBarBytes;
  const uint32_t goff = table + entries * 16, tpre = goff + 4 * (p.G + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ntn = (p.N + NT - 1) / NT;
  // rank in the pair; the pair's first CTA in the cluster; which part of K, and its blocks
  auto pair_rank = []() { return static_cast<int>(cluster_rank() % CG); };
  auto pair_leader = []() { return SPLIT ? static_cast<int>(cluster_rank() / CG * CG) : 0; };
  auto k_part = []() { return SPLIT ? static_cast<int>(cluster_rank() / CG) : 0; };
  auto first_part = [&]() { return first_blocks(p.K); };
  auto blocks_of_k = [&]() {
    const int all = code_blocks(p.K);
    return !SPLIT ? all : k_part() ? all - first_part() : first_part();
  };

  wait_for_stream();
  let_next_start();
  if (p.group_rows) {        // the scan borrows the stages, which are not in use yet
    build_group_tables<kThreads>(p, CG * TM, ntn, smem, goff, tpre, dev_status);
    fence_proxy_async_smem();      // (before the copies that write there)
  } else if (tid == 64) {
    const int rows = static_cast<int>(p.a_rows);
    smem_store(goff, 0);
    smem_store(goff + 4, rows);
    smem_store(tpre, 0);
    smem_store(tpre + 4, row_blocks(rows, CG * TM) * ntn);
  }
  if (warp == 0) {           // barriers: one lane each
    if (lane < stages) {
      bar_init(full(0, lane), 1);
      bar_init(full(1, lane), 1);
      bar_init(peer(lane), 1);
      bar_init(empty(lane), 1);
    }
    if (lane < kAccs) {
      bar_init(tfull(lane), 1);
      bar_init(tempty(lane), CG * kEpiWarps);
    }
    if (lane == 0) {
      smem_store(abort_flag, 0);
      smem_store(issued, 0);
      smem_store(issued + 4, 0);
      tensor_map_prefetch(&maps.w);
      tensor_map_prefetch(&maps.a);
      tensor_map_prefetch(&maps.c);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    if constexpr (CG == 2) pair_tmem_alloc(tmem_slot, kTmemCols);
    else tmem_alloc(tmem_slot, kTmemCols);
  }
  __syncthreads();
  if (tid >= kThreads - entries) {
    const int i = tid - (kThreads - entries), t = cluster_id() + i * cluster_count();
    if (t < smem_load(tpre + 4 * p.G)) {
      const Tile tl = decode_tile<NT, FORM>(t, goff, tpre, p.G, ntn);
      smem_store(table + i * 16, tl.g);
      smem_store(table + i * 16 + 4, tl.n0);
      smem_store(table + i * 16 + 8, tl.row0);
      smem_store(table + i * 16 + 12, tl.rows);
    }
  }
  tc_fence_before();
  __syncthreads();
  // The copies start at once; a role waits for the other CTA before it first reaches
  // into it (its barriers must have been set up).
  cluster_arrive_all_relaxed();
  tc_fence_after();

  // (each role reads what it needs: registers are short in some)
  auto tile_count = [&]() { return smem_load(tpre + 4 * p.G); };
  // The cluster's i-th tile, t = cluster_id() + i * cluster_count().  (The search for its
  // group and the divisions took some 400 clocks at the start of every tile.)
  auto tile_at = [&](int i, int t) {
    if (i >= entries) return decode_tile<NT, FORM>(t, goff, tpre, p.G, ntn);
    Tile tl;
    asm volatile("ld.shared.v4.s32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(tl.g), "=r"(tl.n0), "=r"(tl.row0), "=r"(tl.rows)
                 : "r"(table + i * 16) : "memory");
    return tl;
  };
  // Waits for the last commit on each of this CTA's barriers, once all of them are
  // issued: ncommit of stages, nacc of accumulators.  A barrier's n-th commit is issued
  // only after this CTA's threads have seen its n-1-th, so at most one is outstanding and
  // the parity tells.  Also after a timeout.
  auto await_commits = [&](uint32_t ncommit, uint32_t nacc) {
    bool ok = true;
    const uint32_t ns = stages;
#pragma unroll 1
    for (uint32_t i = ncommit > ns ? ncommit - ns : 0; i < ncommit; ++i)
      ok &= bar_wait(empty(i % ns), (i / ns) & 1u);
#pragma unroll 1
    for (uint32_t i = nacc > kAccs ? nacc - kAccs : 0; i < nacc; ++i)
      ok &= bar_wait(tfull(i % kAccs), (i / kAccs) & 1u);
    if (!ok) set_status(dev_status, MOE_ERR_TIMEOUT);
  };

  if (warp < kCtrlWarps) {
    regs_fewer<kCtrlRegs>();
    const int rank = pair_rank(), nk = blocks_of_k();
    if (warp == 0 || warp == 2) {
      // ---- copies -------------------------------------------------------------------
      const bool issue = elect_one();
      const int of = warp / 2;                 // 0: token rows, 1: weight rows
      const uint32_t bytes = of ? (NT / CG) * BK : TM * BK;
      const CUtensorMap* map = of ? &maps.w : &maps.a;
      const int kb0 = k_part() * first_part();
      int s = 0;
      uint32_t phase = 0, nload = 0;
      bool ok = true;
      int i = 0;
      for (int t = cluster_id(); ok && t < tile_count(); t += cluster_count(), ++i) {
        const Tile tl = tile_at(i, t);
        const int row = of ? tl.g * p.N + tl.n0 + rank * (NT / CG) : tl.row0 + rank * TM;
        for (int kb = 0; kb < nk; ++kb) {
          // (the ring's first round finds it empty)
          if (nload >= uint32_t(stages) && !warp_role_wait(empty(s), phase ^ 1u)) {
            ok = false;
            break;
          }
          if (issue) {
            bar_expect(full(of, s), bytes);
            tensor_load_2d(sbase + s * St::kBytes + of * (TM * BK), map, (kb0 + kb) * BK,
                           row, full(of, s));
          }
          ++nload;
          if (++s == stages) { s = 0; phase ^= 1u; }
        }
        ok = ok && !smem_load(abort_flag);
      }
      if (!ok) {
        if (issue) set_status(dev_status, MOE_ERR_TIMEOUT);
        smem_store(abort_flag, 1);
      }
      // no copy may land once the CTA has gone (only after a timeout are there any that
      // nobody waited for)
      const uint32_t ns = stages;
      for (uint32_t i = nload > ns ? nload - ns : 0; issue && i < nload; ++i)
        bar_wait(full(of, i % ns), (i / ns) & 1u);
      cluster_wait_all();
    } else if (CG == 2 && warp == 1 && rank == 1) {
      // ---- which stages of this CTA have landed ---------------------------------------
      cluster_wait_all();
      int s = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = cluster_id(); ok && t < tile_count(); t += cluster_count()) {
        for (int kb = 0; kb < nk; ++kb) {
          if (!warp_role_wait2(full(0, s), full(1, s), phase)) {
            ok = false;
            break;
          }
          cluster_arrive_if(lane == 0, cluster_addr(peer(s), pair_leader()));
          if (++s == stages) { s = 0; phase ^= 1u; }
        }
        ok = ok && !smem_load(abort_flag);
      }
      if (!ok) {
        if (lane == 0) set_status(dev_status, MOE_ERR_TIMEOUT);
        smem_store(abort_flag, 1);
      }
    } else if (warp == 1) {
      // ---- products of the pair ---------------------------------------------------------
      cluster_wait_all();
      const bool issue = elect_one();
      const uint32_t tmem = smem_load(tmem_slot);
      constexpr int kM = CG * TM;
      const uint32_t idesc = f16_mma_desc(kM, NT);
      int s = 0;
      uint32_t phase = 0, nacc = 0;
      bool ok = true;
      for (int t = cluster_id(); ok && t < tile_count(); t += cluster_count()) {
        for (int kb = 0; kb < nk; ++kb) {
          const uint32_t b = nacc % kAccs;
          const uint32_t other = CG == 2 ? peer(s) : full(1, s);
          if (!warp_role_wait4(full(0, s), full(1, s), other, phase, tempty(b),
                               ((nacc / kAccs) & 1u) ^ 1u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (issue) {
            const uint32_t st = sbase + s * St::kBytes;
            const uint64_t da = operand_desc(st), db = operand_desc(st + TM * BK);
            const uint32_t d = tmem + b * NT;
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk) {   // + 32 bytes along K per step
              if constexpr (CG == 2) pair_mma_f8(d, da + 2 * kk, db + 2 * kk, idesc, kk != 0);
              else mma_f8(d, da + 2 * kk, db + 2 * kk, idesc, kk != 0);
            }
            if constexpr (CG == 2) {
              pair_commit(tfull(b), uint16_t(3 << pair_leader()));
              pair_commit(empty(s), uint16_t(3 << pair_leader()));
            } else {
              mma_commit(tfull(b));
              mma_commit(empty(s));
            }
          }
          ++nacc;
          if (++s == stages) { s = 0; phase ^= 1u; }
        }
        ok = ok && !smem_load(abort_flag);
      }
      if (!ok) {
        if (issue) set_status(dev_status, MOE_ERR_TIMEOUT);
        smem_store(abort_flag, 1);
      }
      // the pair's other CTA, whose barriers the commits arrive on too, learns how many
      // there were; it waits for them after the closing barrier
      if (issue) {
        await_commits(nacc, nacc);
        if constexpr (CG == 2) {
          const uint32_t to = cluster_addr(issued, pair_leader() + 1);
          cluster_store(to, nacc);
          cluster_store(to + 4, nacc);
        }
      }
    } else {
      cluster_wait_all();
    }
    __syncwarp();
    if constexpr (SPLIT) cluster_sync();       // (the draining warps')
  } else {
    // ---- blocks' sums -> scaled sums -> stores --------------------------------------------
    regs_more<kEpiRegs>();
    const int rank = pair_rank(), nk = blocks_of_k();
    const int q = warp & 3;                  // TMEM lanes 32 q ..
    const int col0 = ((warp - kCtrlWarps) >> 2) * kCols;
    const uint32_t base = smem_load(tmem_slot) + (uint32_t(q * 32) << 16) + col0;
    const uint32_t drained = cluster_addr(tempty(0), pair_leader());
    constexpr int kWarpBoxes = boxes_of(FORM);
    const uint32_t box = outs + (warp - kCtrlWarps) * kWarpBoxes * kBoxBytes;
    const int nblocks = code_blocks(p.N);
    cluster_wait_all();
    // What the drain of a tile needs: its scales' places, and those of its first turn.
    // kTurn blocks a turn, their scales loaded a turn ahead (the first ones before the tile
    // ahead is stored): the token's 16 bytes at once (every load of a warp touches 32 lines,
    // and takes as many of the L1 cycles that the products need to read shared memory:
    // 8192 x 4096 x 7168 took 182 us by loads of 4 bytes, 174 by these, 197 with tensor
    // copies of 128 x 16 bytes, which hold up the operands' copies, and 187 with a warp that
    // loads for the others)
    const unsigned char* as = nullptr;
    const float* ws = nullptr;
    bool work = false;
    float ra[kTurn], rw[kTurn];
    auto load_scales = [&](int kb) {
      const float* from = reinterpret_cast<const float*>(as) + kb;
      if (work && wide_scales && kb + kTurn <= nk) {
        const float4 v = *reinterpret_cast<const float4*>(from);
        ra[0] = v.x; ra[1] = v.y; ra[2] = v.z; ra[3] = v.w;
#pragma unroll
        for (int i = 0; i < kTurn; ++i) rw[i] = ws[kb + i];
      } else {
#pragma unroll
        for (int i = 0; i < kTurn; ++i) {
          const bool in = work && kb + i < nk;
          ra[i] = in ? from[i] : 0.0f;
          rw[i] = in ? ws[kb + i] : 0.0f;
        }
      }
    };
    auto aim = [&](const Tile& tl) {
      const int row = tl.row0 + rank * TM + q * 32 + lane, n0 = tl.n0 + col0;
      work = tl.rows > rank * TM + q * 32 && n0 < p.N;
      as = p.row_scale + min(int64_t(row), p.a_rows - 1) * p.row_scale_stride;
      ws = p.col_scale +
           (int64_t(tl.g) * nblocks + min(n0 / kCodeBlock, nblocks - 1)) * code_blocks(p.K);
      if constexpr (SPLIT) {
        as += 4 * k_part() * first_part();
        ws += k_part() * first_part();
      }
      load_scales(0);
      // the tile's bias, which the store would otherwise wait for (197 x 1001 x 1992: 1 us)
      if (p.bias && lane * 32 < kCols && n0 + lane * 32 < p.N)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.bias + int64_t(tl.g) * p.N + n0 +
                                                      lane * 32));
    };
    uint32_t nacc = 0;
    bool ok = true, joined = false;          // the parts' sums
    int index = 0, t = cluster_id();
    Tile tl{};
    if (t < tile_count()) {
      tl = tile_at(0, t);
      aim(tl);
    }
    while (ok && t < tile_count()) {
      const int first_row = tl.row0 + rank * TM + q * 32;   // of the warp; a lane's token is
      const int rows = tl.rows - rank * TM - q * 32;        // first_row + lane, rows there are
      const int n0 = tl.n0 + col0, g = tl.g;
      float2 acc[kCols / 2];
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
      for (int kb = 0; ok && kb < nk; kb += kTurn) {
        float sc[kTurn];
#pragma unroll
        for (int i = 0; i < kTurn; ++i) sc[i] = __fmul_rn(ra[i], rw[i]);
        load_scales(kb + kTurn);
#pragma unroll
        for (int turn = 0; turn < kTurn; ++turn) {
          if (kb + turn >= nk) break;
          const uint32_t b = nacc % kAccs;
          ok = warp_role_wait(tfull(b), (nacc / kAccs) & 1u);
          if (!ok) break;
          ++nacc;
          tc_fence_after();
          auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            cluster_arrive_if(lane == 0, drained + 8 * b);
          };
          if (!work) {
            release();
            continue;
          }
          const float2 s2 = bcast2(sc[turn]);
          const uint32_t from = base + b * NT;
          constexpr int kParts = kCols / 8;
          float v[2][8];
          tmem_start8(from, v[0]);
#pragma unroll
          for (int i = 0; i < kParts; ++i) {
            tmem_wait8(v[i & 1]);
            if (i + 1 < kParts) tmem_start8(from + 8 * (i + 1), v[(i + 1) & 1]);
            else release();
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[4 * i + j] = fma2_rn(make_float2(v[i & 1][2 * j], v[i & 1][2 * j + 1]), s2,
                                       acc[4 * i + j]);
          }
        }
      }
      ok = ok && !smem_load(abort_flag);
      if (!ok) {
        if (lane == 0) set_status(dev_status, MOE_ERR_TIMEOUT);
        smem_store(abort_flag, 1);
        if (SPLIT) cluster_store(cluster_addr(abort_flag, (1 - k_part()) * CG + rank), 1);
        break;
      }
      t += cluster_count();
      if (!SPLIT && t < tile_count()) {
        tl = tile_at(++index, t);
        aim(tl);
      }
      auto add_bias = [&]() {
        if (!p.bias) return;
        const float* bias = p.bias + int64_t(g) * p.N + n0;
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j) {
          if (n0 + 2 * j < p.N) acc[j].x = __fadd_rn(acc[j].x, bias[2 * j]);
          if (n0 + 2 * j + 1 < p.N) acc[j].y = __fadd_rn(acc[j].y, bias[2 * j + 1]);
        }
      };
      if constexpr (SPLIT) {
        // Rows 0 .. 63 of a CTA are the first part's to finish, the others the second's: a
        // thread sends its sums to the other part's, or adds those to its own.
        const int part = q >> 1;
        const uint32_t slot =
            sums + ((((warp - kCtrlWarps) >> 2) * 2 + (q & 1)) * 32 + lane) * 16;
        constexpr uint32_t kPitch = 32 * (kEpiWarps / 2) * 16;
        const bool there = rows > 0 && n0 < p.N;
        if (there && part != k_part()) {
          const uint32_t to = cluster_addr(slot, part * CG + rank);
#pragma unroll
          for (int j = 0; j < kCols / 4; ++j)
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(to + j * kPitch),
                         "f"(acc[2 * j].x), "f"(acc[2 * j].y), "f"(acc[2 * j + 1].x),
                         "f"(acc[2 * j + 1].y) : "memory");
        } else if (there) {
          add_bias();        // (the prefetch does not outlive the barrier: 0.8 us)
        }
        cluster_sync();
        joined = true;
        if (part != k_part() || smem_load(abort_flag)) break;    // (not all of them came)
        if (there) {
#pragma unroll
          for (int j = 0; j < kCols / 4; ++j) {
            float4 v;
            asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(slot + j * kPitch)
                         : "memory");
            acc[2 * j] = add2_rn(acc[2 * j], make_float2(v.x, v.y));
            acc[2 * j + 1] = add2_rn(acc[2 * j + 1], make_float2(v.z, v.w));
          }
        }
      }
      if (rows <= 0 || n0 >= p.N) continue;
      if (!SPLIT) add_bias();
      constexpr int kItem = OUT == MOE_FP32 ? 4 : 2, kVec = 16 / kItem;     // per 16 bytes
      auto piece = [&](int j) {                // columns j .. j + kVec - 1, narrowed
        if constexpr (OUT == MOE_FP32)
          return make_uint4(__float_as_uint(acc[j / 2].x), __float_as_uint(acc[j / 2].y),
                            __float_as_uint(acc[j / 2 + 1].x),
                            __float_as_uint(acc[j / 2 + 1].y));
        else
          return make_uint4(narrow_pair<OUT>(acc[j / 2].x, acc[j / 2].y),
                            narrow_pair<OUT>(acc[j / 2 + 1].x, acc[j / 2 + 1].y),
                            narrow_pair<OUT>(acc[j / 2 + 2].x, acc[j / 2 + 2].y),
                            narrow_pair<OUT>(acc[j / 2 + 3].x, acc[j / 2 + 3].y));
      };
      constexpr int kBoxCols = kCols * kItem < 128 ? kCols : 128 / kItem;
      constexpr int kBoxes = kCols / kBoxCols;
      // kBoxCols columns of the warp's 32 rows into shared memory, 16-byte pieces swizzled as
      // a tensor copy reads them
      auto stage = [&](int j, uint32_t at) {
#pragma unroll
        for (int i = 0; i < kBoxCols / kVec; ++i) {
          const uint4 o = piece(j + i * kVec);
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                           at + lane * 128 + ((i ^ (lane & 7)) << 4)),
                       "r"(o.x), "r"(o.y), "r"(o.z), "r"(o.w) : "memory");
        }
      };
      if (p.N % kVec == 0) {
        if (kBoxCols * kItem == 128 && rows >= 32) {       // whole rows: out by tensor copies
#pragma unroll
          for (int j = 0; j < kCols; j += kBoxCols) {
            const uint32_t at = box + (j / kBoxCols % kWarpBoxes) * kBoxBytes;
            // (this buffer's last copy)
            if (lane == 0) bulk_wait_read<kBoxes == 1 || kWarpBoxes == 1 ? 0 : 1>();
            __syncwarp();
            stage(j, at);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (n0 + j < p.N) tensor_store_2d(&maps.c, (n0 + j) * kItem, first_row, at);
              bulk_commit();
            }
          }
        } else if (lane < rows) {
          const int64_t at = (int64_t(first_row) + lane) * p.N + n0;
#pragma unroll
          for (int j = 0; j < kCols; j += kVec) {
            const uint4 o = piece(j);
            if (n0 + j < p.N)
              *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.c) + (at + j) * kItem) = o;
          }
        }
      } else {
        // rows of c that do not start on 16 bytes: a row at a time by neighbouring lanes
        // (a lane storing its own row by elements touches 32 lines an instruction: 197 x
        // 1001 x 1992 in fp32 16.6 us, and 11.8 this way)
#pragma unroll
        for (int j = 0; j < kCols; j += kBoxCols) {
          stage(j, box);
          __syncwarp();
          constexpr int kLanes = kBoxCols * kItem / 4;       // lanes per row, 4 bytes each
          constexpr int kRows = 32 / kLanes, kBatch = 8;
          const int word = lane % kLanes, n = n0 + j + word * (4 / kItem);
          for (int r0 = lane / kLanes; r0 < min(rows, 32); r0 += kBatch * kRows) {
            uint32_t v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const int r = r0 + i * kRows;                  // (at most 31)
              v[i] = static_cast<uint32_t>(
                  smem_load(box + r * 128 + (((word >> 2) ^ (r & 7)) << 4) + (word & 3) * 4));
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const int r = r0 + i * kRows;
              if (r >= rows || n >= p.N) continue;
              const int64_t to = int64_t(first_row + r) * p.N + n;
              if constexpr (OUT == MOE_FP32) {
                static_cast<uint32_t*>(p.c)[to] = v[i];
              } else {
                uint16_t* c = static_cast<uint16_t*>(p.c) + to;
                c[0] = static_cast<uint16_t>(v[i]);
                if (n + 1 < p.N) c[1] = static_cast<uint16_t>(v[i] >> 16);
              }
            }
          }
          __syncwarp();
        }
      }
      __syncwarp();
    }
    if (SPLIT && !joined) cluster_sync();      // a timeout, or no tile: the others wait
    if (lane == 0) bulk_wait_all<0>();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  // no CTA of a pair goes while the other's threads may still arrive on its barriers ...
  cluster_sync();
  if (warp == 1) {
    // ... nor while a commit may (the first CTA's role has waited for its own)
    await_commits(smem_load(issued), smem_load(issued + 4));
    __syncwarp();
    tc_fence_after();
    if constexpr (CG == 2) pair_tmem_free(smem_load(tmem_slot), kTmemCols);
    else tmem_free(smem_load(tmem_slot), kTmemCols);
  }
}

struct Plan {
  int nt;          // channels per tile
  Form form;
  int clusters;
  bool wide_scales;          // every row's scales start on 16 bytes
};

template <int NT, int OUT, Form FORM>
cudaError_t launch_kernel(const Maps& maps, const LinearArgs& p, const Plan& plan,
                          int32_t* dev_status, int optin, cudaStream_t st) {
  using S = Stages<NT, FORM>;
  int stages = kMaxStages;
  while (stages > 2 && S::bytes(stages, 0, p.G) > size_t(optin)) --stages;
  // (a table in what the stages leave)
  const size_t least = S::bytes(stages, 0, p.G);
  const int table = static_cast<int>(
      std::min<size_t>(kMaxTable, (std::max(size_t(optin), least) - least) / 16));
  const size_t smem = S::bytes(stages, table, p.G);
  auto kernel = linear_f8_tile_kernel<NT, OUT, FORM>;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  const unsigned size = FORM == kSingle ? 1 : FORM == kPair ? 2 : 4;       // of a cluster
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(plan.clusters) * size);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = size;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;      // see launch_early
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, maps, p, plan.wide_scales, stages, table, dev_status);
}

template <int NT, Form FORM>
cudaError_t launch_out(const Maps& maps, const LinearArgs& p, const Plan& plan,
                       int32_t* dev_status, int optin, cudaStream_t st) {
  switch (p.c_dtype) {
    case MOE_BF16: return launch_kernel<NT, MOE_BF16, FORM>(maps, p, plan, dev_status, optin, st);
    case MOE_FP16: return launch_kernel<NT, MOE_FP16, FORM>(maps, p, plan, dev_status, optin, st);
    default: return launch_kernel<NT, MOE_FP32, FORM>(maps, p, plan, dev_status, optin, st);
  }
}

// Blocks of `rows` token rows: at most so many for any group sizes, and with even ones.
int64_t most_blocks(const LinearArgs& p, int rows) {
  return p.G == 1 ? (p.a_rows + rows - 1) / rows
                  : p.a_rows / rows + std::min<int64_t>(p.G, p.a_rows);
}
int64_t even_blocks(const LinearArgs& p, int rows) {
  return std::min(most_blocks(p, rows), p.G * (((p.a_rows + p.G - 1) / p.G + rows - 1) / rows));
}
// Tiles of a CTA by itself.
int64_t single_tiles(const LinearArgs& p) { return even_blocks(p, TM) * ((p.N + 255) / 256); }

// Whether the kernel that streams weights to the warps' own products is the faster one.
// A few rows of a plain product: up to 8 a weight byte meets one instruction (8 rows of 4096 x
// 7168 take 8.0 us there and 18.6 here), up to 16 two, which bound it (16 rows of 4096 x 7168
// 14.4 and 15 to 19, of 16,384 x 4096 29.9 and 21.4; 20 rows 23.9 and 15.1).  A few rows of
// few groups, which have not a tile for every SM: 16 rows in 8 groups of 4096 x 4096 27.4 and
// 30.3, 64 in 32 of 1024 x 1024 9.7 and 11.5, but 48 in 8 of 4096 x 4096 34.3 and 28.0; with
// more tiles 256 in 256 of 4096 x 7168 733 and 721, 1024 uneven ones 1105 and 854, 80 in 40
// of 2048 x 2048 31.8 and 29.7, and with a K of one block 80 in 138 of 4096 x 64 24.3 and
// 16.6, 512 in 256 of 2048 x 64 46.4 and 23.5.  Small products, where this kernel's start (barriers, TMEM,
// clusters) is most of its time: 256 x 512 x 512 4.8 and 5.8, 128 x 1024 x 2048 (at both
// limits) 9.1 and 9.2, 64 x 7168 x 256 (past the first) 10.1 and 7.0, 240 rows in 40 groups of
// 512 x 512 7.5 and 7.3.
bool use_few(const LinearArgs& p, int sms) {
  const int64_t outputs = p.a_rows * p.N;
  const bool few = p.G > 1 ? p.a_rows <= 3 * int64_t(p.G) && single_tiles(p) < sms
                           : p.a_rows <= (int64_t(p.N) * p.K <= 1 << 25 ? 16 : 8);
  return few || (outputs <= (1 << 17) && outputs * p.K <= (1 << 28));
}

// The form that is expected to take the least time: rounds of tiles over the pairs of SMs,
// each of so much a block of K (0.26, 0.24 and 0.40 us at 64, 128 and 256 channels) with its
// start as three blocks more, and the store, which is long where it is not by tensor copies of
// 16-bit values.  K in two parts costs 2 us for the exchange and a second pair's start; 36
// clusters of four CTAs run at once on 152 SMs (with a 37th 256 x 4736 x 4096 takes
// 21.7 us).  Measured in us at 64, 128 and 256 channels whole, 64 and 128 in parts:
//   bf16    33 x 4096 x 1024    9.9   7.9   8.4     -   8.4
//           64 x 4096 x 4096   14.0  12.8  16.9     -  11.6
//          256 x 1024 x 7168   18.9  18.3  26.1  13.7  14.7
//          256 x 4096 x 7168   20.3  19.3  26.9     -  16.4
//          512 x 4096 x 7168   32.3  20.5  27.2     -     -
//         1024 x 4096 x 7168   56.4  34.2  28.6     -     -
//         1280 x 4096 x 7168   68.2  47.3  50.3     -     -
//         2048 x 4096 x 7168   94.4  62.7  52.5     -     -
//          129 x 1500 x  700    7.5   9.0  12.6     -     -
//   fp32   300 x 1000 x 1025    8.9   9.7  13.3     -     -
//          197 x 1001 x 1992   10.6  12.5     -  10.6  13.1
//          512 x 4096 x 4096   22.1  16.9  23.2     -     -
//         4096 x 4096 x 4096    113  77.4  81.7     -     -
// Groups of up to 512 rows that have enough tiles: CTAs by themselves (256 channels).  For a
// tile of up to 128 rows both a pair's SMs would multiply rows that do not count, and two
// tiles' weights are on their way where the pair's SMs have one's: in pairs and singly 2048 or
// 8192 rows of 256 groups of 4096 x 7168 1456 and 1104, 1494 and 1123 (6.8 TB/s), 32,768 1580
// and 1375; 4096 of 8 groups (512 each) 152 and 120; 2048 of 16 groups of 1032 x 1100 (80
// tiles) 14.6 and 12.1; 8192 of 8 (1024 each) 195 and 203, 65,536 of 32 of 2048 x 2048 238 and
// 268.  With a tile for fewer than all SMs a long K waits for its few stages: 1000 rows of 8
// groups of 4096 x 7168 57 and 63.
Plan make_plan(const LinearArgs& p, int sms) {
  const int64_t pairs = std::max(1, sms / 2), fours = sms * 36 / 152, kb = code_blocks(p.K);
  const bool long_store = p.c_dtype == MOE_FP32 || p.N % 8 != 0;
  Plan plan{};
  const int64_t tiles = single_tiles(p);
  if (p.G > 1 && p.a_rows <= 512 * int64_t(p.G) &&
      (tiles >= sms || (2 * tiles >= sms && p.a_rows * kb <= 2048 * int64_t(p.G)))) {
    plan.nt = 256;
    plan.form = kSingle;
    plan.clusters = static_cast<int>(
        std::min<int64_t>(most_blocks(p, TM) * ((p.N + 255) / 256), sms));
    return plan;
  }
  int64_t least = INT64_MAX;             // 1/100 us
  auto take = [&](int nt, Form form, int64_t cost, int64_t clusters) {
    if (cost >= least) return;
    least = cost;
    plan.nt = nt;
    plan.form = form;
    plan.clusters = static_cast<int>(clusters);
  };
  for (int nt : {128, 256, 64}) {
    const int64_t columns = (p.N + nt - 1) / nt, first = first_blocks(p.K);
    const int64_t block = nt == 256 ? 40 : nt == 128 ? 24 : 26;
    const int64_t store = !long_store ? 0 : nt == 256 ? 450 : nt == 128 ? 200 : 60;
    const int64_t joined = !long_store ? 0 : nt == 128 ? 200 : 130;       // by half the warps
    const int64_t most = most_blocks(p, 2 * TM) * columns;
    const int64_t rounds = (even_blocks(p, 2 * TM) * columns + pairs - 1) / pairs;
    take(nt, kPair, (nt == 64 ? 570 : 480) + rounds * ((kb + 3) * block + store),
         std::min(most, pairs));
    if (nt <= 128 && p.G == 1 && kb - first >= kTurn && most <= fours)
      take(nt, kHalves, (nt == 64 ? 650 : 680) + (first + 3) * 24 + joined, most);
  }
  return plan;
}

cudaError_t make_maps(const LinearArgs& p, Plan* plan, Maps* maps) {
  cudaError_t e =
      encode_bytes_2d(&maps->w, p.w, int64_t(p.G) * p.N, p.K, p.w_stride,
                      plan->nt / ctas_of(plan->form));
  if (e == cudaSuccess) e = encode_bytes_2d(&maps->a, p.a, p.a_rows, p.K, p.a_stride, TM);
  // (rows of c that do not start on 16 bytes are stored without the map)
  const int64_t pitch = int64_t(p.N) * (p.c_dtype == MOE_FP32 ? 4 : 2);
  maps->c = maps->a;
  if (e == cudaSuccess && pitch % 16 == 0)
    e = encode_bytes_2d(&maps->c, p.c, p.a_rows, pitch, pitch, 32);
  plan->wide_scales = reinterpret_cast<uintptr_t>(p.row_scale) % 16 == 0 &&
                      (p.a_rows == 1 || p.row_scale_stride % 16 == 0);
  return e;
}

}  // namespace

#ifndef MOE_LINEAR_F8_POLLS
cudaError_t launch_linear_f8(const LinearArgs& p, int32_t* dev_status, cudaStream_t st) {
  int dev = 0, sms = 0, optin = 0;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  if (use_few(p, sms)) return launch_linear_f8_few(p, dev_status, st);
  e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e != cudaSuccess) return e;
  Plan plan = make_plan(p, sms);
  Maps maps;
  e = make_maps(p, &plan, &maps);
  if (e != cudaSuccess) return e;
  if (plan.form == kSingle) return launch_out<256, kSingle>(maps, p, plan, dev_status, optin, st);
  if (plan.form == kHalves)
    return plan.nt == 128 ? launch_out<128, kHalves>(maps, p, plan, dev_status, optin, st)
                          : launch_out<64, kHalves>(maps, p, plan, dev_status, optin, st);
  return plan.nt == 256   ? launch_out<256, kPair>(maps, p, plan, dev_status, optin, st)
         : plan.nt == 128 ? launch_out<128, kPair>(maps, p, plan, dev_status, optin, st)
                          : launch_out<64, kPair>(maps, p, plan, dev_status, optin, st);
}
#endif

}  // namespace moe_ep

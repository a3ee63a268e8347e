// linear_i8.cu -- matrix product of 8-bit codes with a scale per row and per
// output column, rows grouped by expert (include/moe_ep.h, moe_linear_i8).
//
// Mathematics.  acc[m][n] = sum_j a[m][j] w[g][n][j] in int32 (K <= 65536, so
// |acc| <= 2^30: exact), then c = ((fp32(acc) * col) * row) + bias, one
// rounding each, then one rounding to the output type.  sm_103a has no INT8
// tensor-core product, so the codes are widened to fp16 inside the kernel
// (exact, |code| <= 128) and multiplied with fp32 accumulation in chunks of
// 1024 products: a chunk's partial sums are integers of at most 1024 * 2^14 =
// 2^24, all exact in fp32; chunks are added in int32.
//
// Widening costs no memory traffic: both operands travel as bytes from HBM to
// shared memory.  A code byte b, xor 0x80, put under the high byte 0x64 is the
// fp16 number 1024 + (b + 128); subtracting 1152 leaves b: five instructions
// for four codes.
//
// Tile: a pair of CTAs (on two SMs of a cluster) takes 256 output channels (the
// MMA's M, 128 TMEM lanes on each SM) x up to 256 tokens (the MMA's N), so each
// SM widens 128 weight rows and half the tokens, and few tokens make narrow, cheap
// instructions while every weight is still read once.  Warps of a CTA (one CTA
// per SM, persistent):
//   warp 0        copies 128 weight rows and its half of the token rows, 128 bytes
//                 of each, into a ring of byte stages (tensor copies, 128-byte swizzle)
//   warp 1        of the pair's first CTA: issues tcgen05.mma (K = 16) from fp16
//                 stages of both SMs into one of two TMEM accumulators,
//                 alternating per chunk
//   16 warps      widen byte stages into fp16 stages (64 codes, 128-byte swizzle)
//   8 warps       drain finished chunks into int32 registers (one channel per
//                 thread), then scale and store: a warp's stores for one token
//                 are 32 neighbouring channels
// When there are fewer tiles than pairs of SMs, a cluster of 2 to 4 pairs splits
// K; the partial sums (integers, so any order gives the same result) meet in
// shared memory across the cluster, each CTA finishing its share of the tile's
// tokens.
// Every wait is bounded: a timeout sets MOE_ERR_TIMEOUT, the CTA stops issuing
// work and drains what is in flight.
//
// What bounds it.  A 64-code step of a full tile is 512 clocks of MMA on an SM, and
// 384 of its load and store unit (16 KB of bytes read, 32 KB of fp16 written, 128
// bytes a clock) beside the copies' and the MMA's own traffic; so large tiles run
// at the tensor cores' rate and tiles of fewer tokens at that of shared memory
// (128 weight rows are widened for however few tokens).  The store of a tile adds
// shuffles and stores to the same unit, which shows where K is short.  Measured (in
// a graph, SM clock at its maximum; boxes differ by 3%): 8192 x 4096 x 7168 253 to 260
// us, a library bf16 product's rate; 4096 x 4096 x 7168 145 to 148, 1640 TFLOP/s (304
// tiles of 224 tokens, four for each of 76 pairs: 4% of the columns are empty);
// 32,768 x 7168 x 2048 590, 1630; in 32 uneven groups (half of them under 512 rows, so
// of two narrower tiles) 671.  Without the store's arithmetic and stores the last two
// took 9% and 4% less.  Tried and slower for the whole product: two channels per store
// after an exchange between lanes (3%), row scales through shared memory instead of
// shuffles (the same), both paths of the store in one loop (11%).
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "group_tiles.cuh"
#include "moe_ep_internal.cuh"
#include "tcgen05.cuh"

namespace moe_ep {

// linear_i8_polls.cu compiles this file a second time, for tests of the waits that run
// out: with role_wait of its own, and without the two functions that others call.
#ifndef MOE_LINEAR_I8_POLLS
namespace {
// A role's wait for its next work; false after kGemmSpin polls.
__device__ __forceinline__ bool role_wait(uint32_t bar, uint32_t parity) {
  return bar_wait(bar, parity);
}
}  // namespace

cudaError_t encode_bytes_2d(CUtensorMap* map, const void* base, int64_t rows, int64_t cols,
                            int64_t stride, uint32_t box_rows) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::atomic<void*> known{nullptr};     // the driver's function, looked up once
  void* fn = known.load(std::memory_order_relaxed);
  if (fn == nullptr) {
    cudaDriverEntryPointQueryResult q;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                     cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || fn == nullptr) return cudaErrorNotSupported;
    known.store(fn, std::memory_order_relaxed);
  }
  const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(stride)};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  auto encode = [&]() {
    return reinterpret_cast<Encode>(fn)(
        map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  if (r != CUDA_SUCCESS) {
    // The driver's function needs a context, and a host thread that has made no runtime
    // call of its own yet has none: make its device's current, as the runtime would.
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaSetDevice(dev);
    if (e != cudaSuccess) return e;
    r = encode();
  }
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
#endif

namespace {

constexpr int BM = 128;              // output channels per CTA
constexpr int CG = 2;                // CTAs per tile (a pair)
constexpr int BK = 64;               // codes per fp16 stage: one 128-byte row
constexpr int kHalves = 2;           // fp16 stages per byte stage (128-byte rows both)
constexpr int BKB = kHalves * BK;
constexpr int kChunk = 1024 / BKB;   // byte stages per chunk: 1024 products, exact in fp32
constexpr int kMaxSplit = 4;         // pairs that may share a tile's K
constexpr int kRasterTokens = 8;     // token blocks per raster band (weights reused from L2)
// 28 warps: 4 that copy and multiply (two of them idle), 16 that widen, in groups
// of four on different stages, and 8 that drain and store.  (With 8 widening and
// 16 draining warps, 16384 x 7168 x 2048 took 317 us; this way 294.)
constexpr int kGroupWarps = 4, kConvWarps = 16, kEpiWarps = 8;
constexpr int kConvGroups = kConvWarps / kGroupWarps;
constexpr int kTurns = kConvGroups / kHalves;      // groups take byte stages in turns
static_assert(kTurns == 2, "turns");
constexpr int kThreads = 128 + 32 * (kConvWarps + kEpiWarps);
// Registers per thread: 72 at launch.  With pairs, whose draining threads hold 128
// sums, they are handed out again by role: 256 x 152 + 512 x 40 + 128 x 40 = 64512
// = 896 x 72.
constexpr int kEpiRegs = 152, kConvRegs = 40, kCtrlRegs = 40;
static_assert(32 * (kEpiWarps * kEpiRegs + kConvWarps * kConvRegs + 4 * kCtrlRegs) <=
                  kThreads * 72, "no more registers than the launch has");
// Tiles of up to 128 tokens hold 64 sums per draining thread and leave 8 registers
// more to a widening one (with 40 it spilled).
constexpr int kEpiRegs128 = 136, kConvRegs128 = 48;
static_assert(32 * (kEpiWarps * kEpiRegs128 + kConvWarps * kConvRegs128 + 4 * kCtrlRegs) <=
                  kThreads * 72, "no more registers than the launch has");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kAccCols = 256;   // column offset of the second accumulator
constexpr int kMaxByteStages = 12, kMaxF16Stages = 6;
static_assert(kTurns * kMaxByteStages <= 32, "a lane sets up each barrier");

// LT: token rows that one CTA holds (a pair of CTAs shares the tile's tokens).
template <int LT>
struct Stages {
  static constexpr int kF16 = 4;                                  // fp16 stages
  static constexpr uint32_t kF16Bytes = (BM + LT) * BK * 2;
  static constexpr uint32_t kByteBytes = (BM + LT) * BKB;
  static constexpr uint32_t kOffBytes = kF16 * kF16Bytes;
  // barriers and flags, then the group tables, follow the byte stages
  static constexpr uint32_t kBarBytes = 512;
  static size_t bytes(int nbyte, int G) {
    return 1024 + kOffBytes + size_t(nbyte) * kByteBytes + kBarBytes + size_t(G + 1) * 8;
  }
};

struct Tile {
  int g;           // group
  int n0;          // first output channel
  int row0;        // first token row
  int rows;        // tokens stored
  int cols;        // tokens computed: rows rounded up to the MMA's step
};

// A pair shares a tile of CG * BM channels; token counts are multiples of 32 (the
// MMA's step).
__device__ __forceinline__ Tile decode_tile(int t, uint32_t goff, uint32_t tpre, int G,
                                            int ntn, int block) {
  const int lo = group_of_tile(t, tpre, G);
  const int off = smem_load(goff + 4 * lo);
  const int cnt = smem_load(goff + 4 * lo + 4) - off;
  const uint32_t local = t - smem_load(tpre + 4 * lo);
  constexpr uint32_t kStep = 16 * CG;
  uint32_t per = (cnt + kStep - 1) / kStep * kStep, nblk = local, mblk = 0;   // one block
  if (cnt > block) {
    const uint32_t blocks = static_cast<uint32_t>(row_blocks(cnt, block));   // equal ones
    per = ((cnt + blocks - 1) / blocks + kStep - 1) / kStep * kStep;
    // bands of kRasterTokens token blocks (the last band takes the remainder);
    // inside a band the token block is fastest, so the CTAs in flight share
    // weight tiles and a bounded number of token blocks
    const uint32_t nband = max(blocks / kRasterTokens, 1u), per_band = kRasterTokens * ntn;
    const uint32_t band = min(local / per_band, nband - 1);
    const uint32_t width = band < nband - 1 ? kRasterTokens : blocks - band * kRasterTokens;
    const uint32_t r = local - band * per_band;
    nblk = r / width;
    mblk = band * kRasterTokens + r - nblk * width;
  }
  Tile tl;
  tl.g = lo;
  tl.n0 = static_cast<int>(nblk * (CG * BM));
  const int first = static_cast<int>(mblk * per);
  tl.row0 = off + first;
  tl.rows = max(0, min(static_cast<int>(per), cnt - first));
  tl.cols = max(kStep, (tl.rows + kStep - 1) / kStep * kStep);
  return tl;
}

// 16 codes -> 16 fp16 numbers (exact), low to high.
__device__ __forceinline__ void widen16(const uint4& v, uint4 (&o)[2]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = w[i] ^ 0x80808080u;
    const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140);   // 0x64b1 64b0
    const uint32_t hi = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r[2 * i]) : "r"(lo), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r[2 * i + 1]) : "r"(hi), "r"(0x64806480u));
  }
  o[0] = make_uint4(r[0], r[1], r[2], r[3]);
  o[1] = make_uint4(r[4], r[5], r[6], r[7]);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w) : "memory");
}

// Scales and bias of channel n of group g, and of row m (int32 outputs take none).
template <int OUT>
__device__ __forceinline__ float col_scale(const LinearArgs& p, int g, int n) {
  return OUT == MOE_INT32 ? 0.0f : p.col_scale[int64_t(g) * p.N + n];
}
template <int OUT>
__device__ __forceinline__ float row_scale(const LinearArgs& p, int64_t m) {
  return OUT == MOE_INT32
             ? 0.0f
             : *reinterpret_cast<const float*>(p.row_scale + m * p.row_scale_stride);
}
__device__ __forceinline__ float bias_of(const LinearArgs& p, int g, int n) {
  return p.bias[int64_t(g) * p.N + n];
}

// One output: its scales, its bias, its rounding.
template <int OUT, bool BIAS>
__device__ __forceinline__ void store_out(void* c, int64_t at, int32_t acc, float col, float row,
                                          float bias) {
  if constexpr (OUT == MOE_INT32) {
    static_cast<int32_t*>(c)[at] = acc;
  } else {
    float v = __fmul_rn(__fmul_rn(__int2float_rn(acc), col), row);
    if constexpr (BIAS) v = __fadd_rn(v, bias);
    if constexpr (OUT == MOE_FP32) static_cast<float*>(c)[at] = v;
    else static_cast<uint16_t*>(c)[at] = static_cast<uint16_t>(narrow_rn<OUT>(v));
  }
}

// Two tokens of one channel at once, N elements apart, by the same operations
// (packed; nz is -0, see mul2_rn): the full tiles' way, half the instructions.
template <int OUT, bool BIAS>
__device__ __forceinline__ void store_pair(uint8_t* at, uint32_t pitch, int32_t a0, int32_t a1,
                                           float col, float r0, float r1, float bias, float nz) {
  if constexpr (OUT == MOE_INT32) {
    *reinterpret_cast<int32_t*>(at) = a0;
    *reinterpret_cast<int32_t*>(at + pitch) = a1;
  } else {
    float2 v = make_float2(__int2float_rn(a0), __int2float_rn(a1));
    v = mul2_rn(mul2_rn(v, bcast2(col), nz), make_float2(r0, r1), nz);
    if constexpr (BIAS) v = add2_rn(v, bcast2(bias));
    if constexpr (OUT == MOE_FP32) {
      *reinterpret_cast<float*>(at) = v.x;
      *reinterpret_cast<float*>(at + pitch) = v.y;
    } else {
      uint32_t h;
      if constexpr (OUT == MOE_BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(v.y), "f"(v.x));
      else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(v.y), "f"(v.x));
      *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(h);
      *reinterpret_cast<uint16_t*>(at + pitch) = static_cast<uint16_t>(h >> 16);
    }
  }
}

// NT: tokens per tile at most.  SPLIT: the cluster's pairs split K (one tile per
// cluster).
template <int NT, int OUT, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
linear_i8_tile_kernel(const __grid_constant__ CUtensorMap map_w,
                      const __grid_constant__ CUtensorMap map_a, const LinearArgs p, int block,
                      int box_rows, int nbyte, int stages, int extra, float nz,
                      int32_t* dev_status) {
  constexpr int LT = NT / CG;
  using St = Stages<LT>;
  constexpr int NF = St::kF16;
  // every widening group starts on a stage of its own
  static_assert(NF >= kConvGroups && NF <= kMaxF16Stages && kConvGroups % kHalves == 0, "stages");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bars = sbase + St::kOffBytes + nbyte * St::kByteBytes;
  // Byte stage filled: one barrier per stage and turn (load i: barrier i modulo 2 nbyte,
  // stage i modulo nbyte).  Were there one per stage, both turns of widening groups
  // would wait on it where nbyte is odd, each skipping the other's phases; when loads
  // land out of order, a group would take the parity of a phase two back for its own
  // and read what the stage held before (seen with 3 stages and rows just copied: one
  // call in 200).
  auto bfull = [&](int i) { return bars + 8 * i; };
  auto bempty = [&](int s) { return bars + 8 * (kTurns * kMaxByteStages + s); };   // ... widened
  constexpr int kF0 = (kTurns + 1) * kMaxByteStages, kT0 = kF0 + 2 * kMaxF16Stages;
  auto ffull = [&](int f) { return bars + 8 * (kF0 + f); };                // fp16 stage written
  auto fempty = [&](int f) { return bars + 8 * (kF0 + kMaxF16Stages + f); };  // ... multiplied
  auto tfull = [&](int b) { return bars + 8 * (kT0 + b); };                // accumulator final
  auto tempty = [&](int b) { return bars + 8 * (kT0 + 2 + b); };           // ... drained
  const uint32_t tmem_slot = bars + 8 * (kT0 + 4), abort_flag = tmem_slot + 4;
  auto srows = [&](int s) { return abort_flag + 4 + 4 * s; };   // rows in byte stage s
  const uint32_t issued = srows(kMaxByteStages);   // the pair's commits: of stages, of chunks
  static_assert(8 * (kT0 + 5) + 4 * kMaxByteStages + 8 <= St::kBarBytes, "barriers fit");
  const uint32_t goff = bars + St::kBarBytes, tpre = goff + 4 * (p.G + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ntn = (p.N + CG * BM - 1) / (CG * BM);
  const int crank = static_cast<int>(cluster_rank());
  const int rank = crank % CG, part = SPLIT ? crank / CG : 0;    // in the pair; of K
  const int split = SPLIT ? static_cast<int>(cluster_size()) / CG : 1;      // a power of two
  const int leader = crank - rank;             // the pair's first CTA, in the cluster

  wait_for_stream();
  let_next_start();
  if (p.group_rows) {        // the scan borrows the stages, which are not in use yet
    build_group_tables<kThreads>(p, block, ntn, smem, goff, tpre, dev_status);
  } else if (tid == 64) {
    const int rows = static_cast<int>(p.a_rows);
    smem_store(goff, 0);
    smem_store(goff + 4, rows);
    smem_store(tpre, 0);
    smem_store(tpre + 4, row_blocks(rows, block) * ntn);
  }
  if (warp == 0) {           // barriers: one lane each
    if (lane < kTurns * nbyte) bar_init(bfull(lane), 1);
    if (lane < nbyte) bar_init(bempty(lane), kHalves * kGroupWarps);
    if (lane < NF) {
      bar_init(ffull(lane), CG * kGroupWarps);
      bar_init(fempty(lane), 1);
    }
    if (lane < 2) {
      bar_init(tfull(lane), 1);
      bar_init(tempty(lane), CG * kEpiWarps);
    }
    if (lane == 0) {
      smem_store(abort_flag, 0);
      tensor_map_prefetch(&map_w);
      tensor_map_prefetch(&map_a);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    pair_tmem_alloc(tmem_slot, kTmemCols);
  }
  tc_fence_before();
  __syncthreads();
  // The copies start at once; a role waits for the rest of the cluster before it
  // first reaches into another CTA (its barriers must have been set up).
  cluster_arrive_all();
  tc_fence_after();

  // (each role reads what it needs: registers are short in some)
  auto tile_count = [&]() { return smem_load(tpre + 4 * p.G); };
  // byte stages of K (zeros past it): every part of a split has `stages`, the first
  // `extra` parts one more
  auto stage_begin = [&]() { return part * stages + min(part, extra); };
  auto stage_count = [&]() { return stages + (part < extra ? 1 : 0); };
  auto chunk_count = [&](int nk) { return (nk + kChunk - 1) / kChunk; };
  // Waits for the last commit on each of this CTA's barriers, once all of them are
  // issued: ncommit of fp16 stages, nchunk of accumulators.  A barrier's n-th commit
  // is issued only after this CTA's threads have seen its n-1-th, so at most one is
  // outstanding and the parity tells (it would not while commits are still to be
  // issued: a phase two uses back looks the same).  Also after a timeout.
  auto await_commits = [&](uint32_t ncommit, uint32_t nchunk) {
    bool ok = true;
#pragma unroll 1
    for (uint32_t i = ncommit > uint32_t(NF) ? ncommit - NF : 0; i < ncommit; ++i)
      ok &= bar_wait(fempty(i % NF), (i / NF) & 1u);
#pragma unroll 1
    for (uint32_t i = nchunk > 2 ? nchunk - 2 : 0; i < nchunk; ++i)
      ok &= bar_wait(tfull(i & 1u), (i >> 1) & 1u);
    if (!ok) set_status(dev_status, MOE_ERR_TIMEOUT);
  };

  if (warp < 4) {
    regs_fewer<kCtrlRegs>();
    const int tiles = tile_count();
    const int nk = stage_count(), first = cluster_id(), step = cluster_count();
    if (warp == 0) {
      // ---- copies -------------------------------------------------------------------
      const bool issue = elect_one();
      int s = 0, full = 0;
      uint32_t phase = 0, nload = 0;
      bool ok = true;
      for (int t = first; ok && t < tiles; t += step) {
        const Tile tl = decode_tile(t, goff, tpre, p.G, ntn, block);
        const int rows = tl.cols / CG;                   // this CTA's token rows
        const int boxes = (rows + box_rows - 1) / box_rows;
        const int wrow = tl.g * p.N + tl.n0 + rank * BM;
        const int arow = tl.row0 + rank * rows;
        const int kb0 = stage_begin();
        for (int kb = kb0; kb < kb0 + nk; ++kb) {
          if (!role_wait(bempty(s), phase ^ 1u)) {
            ok = false;
            break;
          }
          if (issue) {
            const uint32_t dst = sbase + St::kOffBytes + s * St::kByteBytes;
            smem_store(srows(s), BM + rows);       // weight rows, then token rows
            bar_expect(bfull(full), (BM + boxes * box_rows) * BKB);
            tensor_load_2d(dst, &map_w, kb * BKB, wrow, bfull(full));
            for (int b = 0; b < boxes; ++b)
              tensor_load_2d(dst + (BM + b * box_rows) * BKB, &map_a, kb * BKB,
                             arow + b * box_rows, bfull(full));
          }
          ++nload;
          if (++s == nbyte) { s = 0; phase ^= 1u; }
          if (++full == kTurns * nbyte) full = 0;
        }
        ok = ok && !smem_load(abort_flag);
      }
      if (!ok) {
        if (issue) set_status(dev_status, MOE_ERR_TIMEOUT);
        smem_store(abort_flag, 1);
      }
      // no copy may land once the CTA has gone (the widening warps wait for all of
      // them, unless one of them has given up); the issuing lane's count is the true one
      for (uint32_t i = nload > uint32_t(nbyte) ? nload - nbyte : 0; issue && i < nload; ++i)
        bar_wait(bfull(i % (kTurns * nbyte)), (i / (kTurns * nbyte)) & 1u);
      cluster_wait_all();
    } else if (warp == 1 && rank == 0) {
      // ---- products (of the pair, by its first CTA) -----------------------------------
      cluster_wait_all();
      const bool issue = elect_one();
      const uint32_t tmem = smem_load(tmem_slot);
      int f = 0;
      uint32_t phase = 0, chunk = 0, ncommit = 0;
      bool ok = true;
      for (int t = first; ok && t < tiles; t += step) {
        const Tile tl = decode_tile(t, goff, tpre, p.G, ntn, block);
        const uint32_t idesc = f16_mma_desc(CG * BM, tl.cols);
        const int nchunks = chunk_count(nk);
        for (int c = 0; ok && c < nchunks; ++c, ++chunk) {
          const uint32_t b = chunk & 1u, use = (chunk >> 1) & 1u;
          if (!role_wait(tempty(b), use ^ 1u) || smem_load(abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + b * kAccCols;
          const int n = min(kChunk, nk - c * kChunk) * kHalves;
          for (int kb = 0; kb < n; ++kb) {
            if (!role_wait(ffull(f), phase)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (issue) {
              const uint32_t st = sbase + f * St::kF16Bytes;
              const uint64_t da = operand_desc(st), db = operand_desc(st + BM * BK * 2);
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk)     // + 32 bytes along K per step
                pair_mma_f16(d, da + 2 * kk, db + 2 * kk, idesc, kb != 0 || kk != 0);
              pair_commit(fempty(f), uint16_t(3 << leader));
            }
            ++ncommit;
            if (++f == NF) { f = 0; phase ^= 1u; }
          }
          if (!ok) break;
          if (issue) pair_commit(tfull(b), uint16_t(3 << leader));
        }
      }
      if (!ok) {
        if (issue) set_status(dev_status, MOE_ERR_TIMEOUT);
        smem_store(abort_flag, 1);
      }
      // the pair's other CTA, whose barriers the commits arrive on too, learns how
      // many there were; it waits for them after the closing barrier
      if (issue) {
        await_commits(ncommit, chunk);
        const uint32_t to = cluster_addr(issued, leader + 1);
        cluster_store(to, ncommit);
        cluster_store(to + 4, chunk);
        smem_store(issued, 0);            // none left for this one
        smem_store(issued + 4, 0);
      }
    } else {
      cluster_wait_all();
    }
    __syncwarp();
    if constexpr (SPLIT) {
      cluster_sync();
      cluster_sync();
    }
  } else if (warp < 4 + kConvWarps) {
    // ---- bytes -> fp16 ------------------------------------------------------------------
    regs_fewer<NT == 128 ? kConvRegs128 : kConvRegs>();
    // groups of four warps, each on one 64-code half of every other byte stage:
    // one group's waits and fences overlap the others' widening.  A thread takes
    // 16 codes (quarter uc of the half) of one row in kRows.  Eight neighbouring
    // threads share rows r and r ^ 5: their swizzled byte quarters lie in
    // different halves of the banks (bit 2 of the row differs), and so do their
    // fp16 pieces (even and odd ones: bit 0 differs), so loads and stores are
    // free of bank conflicts.
    constexpr int kGroupThreads = 32 * kGroupWarps;
    constexpr int kRows = kGroupThreads / 4;            // rows per pass: a multiple of 8, so
    constexpr int kPasses = (BM + LT) / kRows;          // every pass has one swizzle key
    // passes loaded before widening
    constexpr int kBatch = 2;
    const int grp = (tid - 128) / kGroupThreads, u = (tid - 128) % kGroupThreads;
    const int half = grp % kHalves, turn = grp / kHalves;
    const int uq = u >> 2, uc = u & 3;
    const int ur = (uq & ~7) + (((uq >> 1) & 3) ^ ((uq & 1) * 5));
    const uint32_t in = ur * BKB + (((half * 4 + uc) ^ (ur & 7)) << 4);
    const uint32_t out0 = ur * (BK * 2) + (((2 * uc) ^ (ur & 7)) << 4);
    cluster_wait_all();
    int load = turn, f = grp;            // load: modulo 2 nbyte
    uint32_t bphase = 0, fphase = 0;
    bool ok = true;
    const int tiles = tile_count(), first = cluster_id(), step = cluster_count();
    const int total = first < tiles ? ((tiles - first + step - 1) / step) * stage_count() : 0;
    for (int i = turn; i < total; i += kTurns) {
      ok = __all_sync(0xffffffffu, role_wait(bfull(load), bphase));
      if (!ok) break;
      const int s = load < nbyte ? load : load - nbyte;
      const int rows = smem_load(srows(s));
      const uint32_t src = sbase + St::kOffBytes + s * St::kByteBytes + in;
      const uint32_t dst = sbase + f * St::kF16Bytes + out0;   // and dst ^ 16
      auto widen = [&](auto full) {       // full: every token row of the tile is there
        auto has = [&](int i) {
          return decltype(full)::value || (i + 1) * kRows <= BM || i * kRows + ur < rows;
        };
#pragma unroll
        for (int i0 = 0; i0 < kPasses; i0 += kBatch) {
          uint4 v[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            v[i] = has(i0 + i) ? lds128(src + (i0 + i) * kRows * BKB) : make_uint4(0u, 0u, 0u, 0u);
          if (i0 + kBatch >= kPasses) {
            // This half of the stage is read: hand it back to the copies.  The
            // arrival's address depends on the loaded words (meeting a 0 that the compiler
            // cannot see: nz is -0), so no load can still be pending, or be moved
            // by the compiler to a point after it, when the copies overwrite them.  (Wrong
            // products were seen without this, but before every turn had barriers of its
            // own, which may have been their cause too.)
            uint32_t words = 0;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) words |= v[i].x;
            __syncwarp();
            if (lane == 0) bar_arrive(bempty(s) + (words & (__float_as_uint(nz) << 1)));
          }
          if (i0 == 0) {                              // the fp16 stage is free
            ok = __all_sync(0xffffffffu, role_wait(fempty(f), fphase ^ 1u));
            if (!ok) return;
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            if (has(i0 + i)) {
              uint4 o[2];
              widen16(v[i], o);
              sts128(dst + (i0 + i) * kRows * BK * 2, o[0]);
              sts128((dst ^ 16) + (i0 + i) * kRows * BK * 2, o[1]);
            }
        }
      };
      if (rows == BM + LT) widen(std::true_type());
      else widen(std::false_type());
      if (!ok) break;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) cluster_arrive(cluster_addr(ffull(f), leader));
      if ((load += kTurns) >= kTurns * nbyte) {
        load -= kTurns * nbyte;
        bphase ^= 1u;
      }
      for (f += kConvGroups; f >= NF; f -= NF) fphase ^= 1u;
    }
    if (!ok) {
      if (lane == 0) set_status(dev_status, MOE_ERR_TIMEOUT);
      smem_store(abort_flag, 1);
    }
    if constexpr (SPLIT) {
      cluster_sync();
      cluster_sync();
    }
  } else {
    // ---- chunk sums -> int32, scales, stores ----------------------------------------------
    regs_more<NT == 128 ? kEpiRegs128 : kEpiRegs>();
    constexpr int kParts = kEpiWarps / 4, kCols = NT / kParts;   // columns per thread
    const int q = warp & 3;                  // TMEM lanes 32 q ..
    const int col0 = ((warp - 4 - kConvWarps) >> 2) * kCols;
    const uint32_t base = smem_load(tmem_slot) + (uint32_t(q * 32) << 16) + col0;
    cluster_wait_all();
    uint32_t chunk = 0;
    bool ok = true;
    for (int t = cluster_id(); ok && t < tile_count(); t += cluster_count()) {
      Tile tl = decode_tile(t, goff, tpre, p.G, ntn, block);
      const int live = tl.cols - col0;       // columns of this thread that are computed
      auto wait = [&]() {                    // for the next chunk
        const bool got = role_wait(tfull(chunk & 1u), (chunk >> 1) & 1u) &&
                         !smem_load(abort_flag);
        ok = __all_sync(0xffffffffu, got);
        tc_fence_after();
        return ok;
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) cluster_arrive(cluster_addr(tempty(chunk & 1u), leader));
        ++chunk;
      };
      int32_t acc[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j) acc[j] = 0;
      // every chunk but the last: into the sums
      for (int c = chunk_count(stage_count()) - 1; c > 0; --c) {
        if (!wait()) break;
#pragma unroll
        for (int cb = 0; cb < kCols / 4; ++cb)
          if (cb * 4 < live) {
            uint32_t v[4];
            tmem_load4(base + (chunk & 1u) * kAccCols + cb * 4, v);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[cb * 4 + j] += __float2int_rn(__uint_as_float(v[j]));
          }
        release();
      }
      // the last one: four columns at a time, through the scales to memory or, where
      // K is split, to the CTA that adds them up (the tile is decoded again: the
      // sums leave no registers to hold it)
      if (!ok || !wait()) {
        if (lane == 0) set_status(dev_status, MOE_ERR_TIMEOUT);
        smem_store(abort_flag, 1);
        break;
      }
      auto drain = [&](auto&& emit) {
#pragma unroll
        for (int cb = 0; cb < kCols / 4; ++cb)
          if (cb * 4 < live) {
            uint32_t v[4];
            tmem_load4(base + (chunk & 1u) * kAccCols + cb * 4, v);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[cb * 4 + j] += __float2int_rn(__uint_as_float(v[j]));
            emit(cb * 4, &acc[cb * 4]);
          }
        release();
      };
      if constexpr (!SPLIT) {
        tl = decode_tile(t, goff, tpre, p.G, ntn, block);
        const int n = tl.n0 + rank * BM + q * 32 + lane;
        const int lim = n < p.N ? tl.rows - col0 : 0;    // tokens of this thread to store
        const float col = lim > 0 ? col_scale<OUT>(p, tl.g, n) : 0.0f;
        constexpr int kItem = OUT == MOE_BF16 || OUT == MOE_FP16 ? 2 : 4;
        const uint32_t pitch = p.N * kItem;
        uint8_t* at = static_cast<uint8_t*>(p.c) +
                      (int64_t(tl.row0 + col0) * p.N + n) * kItem;
        auto finish = [&](auto is_full, auto has_bias) {
          constexpr bool kFull = decltype(is_full)::value, kBias = decltype(has_bias)::value;
          const float bias = kBias && lim > 0 ? bias_of(p, tl.g, n) : 0.0f;
          float rs = 0.0f;                  // lane l: the scale of token l of 32
          drain([&](int j0, const int32_t* sum) {
            if (j0 % 32 == 0 && col0 + j0 + lane < tl.rows)
              rs = row_scale<OUT>(p, tl.row0 + col0 + j0 + lane);
#pragma unroll
            for (int j = 0; j < 4; j += 2, at += 2 * pitch) {
              const float r0 = __shfl_sync(0xffffffffu, rs, (j0 + j) % 32);
              const float r1 = __shfl_sync(0xffffffffu, rs, (j0 + j + 1) % 32);
              if constexpr (kFull) {
                store_pair<OUT, kBias>(at, pitch, sum[j], sum[j + 1], col, r0, r1, bias, nz);
              } else {
                if (j0 + j < lim) store_out<OUT, kBias>(at, 0, sum[j], col, r0, bias);
                if (j0 + j + 1 < lim)
                  store_out<OUT, kBias>(at + pitch, 0, sum[j + 1], col, r1, bias);
              }
            }
          });
        };
        const std::true_type yes;
        const std::false_type no;
        const bool is_full = tl.rows == NT && tl.n0 + rank * BM + BM <= p.N;
        if (p.bias) is_full ? finish(yes, yes) : finish(no, yes);
        else is_full ? finish(yes, no) : finish(no, no);
      } else {
        // part d finishes `share` of each thread's live columns, from d * share on
        const int share = (max(min(live, kCols), 0) + 4 * split - 1) / (4 * split) * 4;
        cluster_sync();                     // every CTA is done with its stages
        const int eth = tid - 128 - 32 * kConvWarps;   // epilogue thread
        drain([&](int j0, const int32_t* sum) {
          const int d = (j0 >= share) + (j0 >= 2 * share) + (j0 >= 3 * share);
          const uint32_t to = sbase + ((part * share + j0 - d * share) / 4 * 256 + eth) * 16;
          cluster_store16(cluster_addr(to, d * CG + rank), sum);
        });
        tl = decode_tile(t, goff, tpre, p.G, ntn, block);
        const int mine0 = part * share;               // this part's first column
        float rs[kCols / 64];                         // lane l: token col0 + mine0 + 32 i + l
#pragma unroll
        for (int i = 0; i < kCols / 64; ++i) {
          const int j = col0 + mine0 + 32 * i + lane;
          rs[i] = 32 * i + lane < share && j < tl.rows ? row_scale<OUT>(p, tl.row0 + j) : 0.0f;
        }
        const int n = tl.n0 + rank * BM + q * 32 + lane;
        const float col = n < p.N ? col_scale<OUT>(p, tl.g, n) : 0.0f;
        const float bias = OUT != MOE_INT32 && p.bias && n < p.N ? bias_of(p, tl.g, n) : 0.0f;
        cluster_sync();                     // every part's sums are here
        const int last = min(share, min(kCols, tl.rows - col0) - mine0);   // tokens to store
        constexpr int kItem = OUT == MOE_BF16 || OUT == MOE_FP16 ? 2 : 4;
        const uint32_t pitch = p.N * kItem;
        uint8_t* at = static_cast<uint8_t*>(p.c) +
                      (int64_t(tl.row0 + col0 + mine0) * p.N + n) * kItem;
#pragma unroll
        for (int i = 0; i < kCols / 64; ++i)
#pragma unroll 2
          for (int jj = 32 * i; jj < min(last, 32 * i + 32); jj += 4) {
            uint4 v[kMaxSplit];
#pragma unroll
            for (int r = 0; r < kMaxSplit; ++r)
              v[r] = r < split ? lds128(sbase + ((r * share + jj) / 4 * 256 + eth) * 16)
                               : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t sum[4] = {v[0].x + v[1].x + v[2].x + v[3].x,
                                     v[0].y + v[1].y + v[2].y + v[3].y,
                                     v[0].z + v[1].z + v[2].z + v[3].z,
                                     v[0].w + v[1].w + v[2].w + v[3].w};
#pragma unroll
            for (int k = 0; k < 4; ++k, at += pitch) {
              const float row = __shfl_sync(0xffffffffu, rs[i], (jj + k) & 31);
              if (jj + k >= last || n >= p.N) continue;
              if (p.bias) store_out<OUT, true>(at, 0, static_cast<int>(sum[k]), col, row, bias);
              else store_out<OUT, false>(at, 0, static_cast<int>(sum[k]), col, row, 0.0f);
            }
          }
      }
    }
    if (SPLIT && (cluster_id() >= tile_count() || !ok)) {   // no tile, or a timeout: the peers wait
      cluster_sync();
      cluster_sync();
    }
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
    pair_tmem_free(smem_load(tmem_slot), kTmemCols);
  }
}

struct Plan {
  int nt;          // the kernel's token limit per tile: 128 or 256
  int block;       // tokens per tile at most
  int box_rows;    // token rows per copy
  int split;       // pairs that share a tile's K
  int clusters;
};

template <int NT, int OUT, bool SPLIT>
cudaError_t launch_kernel(const CUtensorMap& mw, const CUtensorMap& ma, const LinearArgs& p,
                          const Plan& plan, int32_t* dev_status, int optin, cudaStream_t st) {
  using S = Stages<NT / CG>;
  int nbyte = kMaxByteStages;    // at least kConvGroups / kHalves = 2
  while (nbyte > 2 && S::bytes(nbyte, p.G) > size_t(optin)) --nbyte;
  const size_t smem = S::bytes(nbyte, p.G);
  auto kernel = linear_i8_tile_kernel<NT, OUT, SPLIT>;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(plan.clusters * CG * plan.split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(CG * plan.split);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;      // see launch_early
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, mw, ma, p, plan.block, plan.box_rows, nbyte,
                            (p.K + BKB - 1) / BKB / plan.split,
                            (p.K + BKB - 1) / BKB % plan.split, -0.0f, dev_status);
}

template <int NT, int OUT>
cudaError_t launch_out(const CUtensorMap& mw, const CUtensorMap& ma, const LinearArgs& p,
                       const Plan& plan, int32_t* dev_status, int optin, cudaStream_t st) {
  return plan.split > 1 ? launch_kernel<NT, OUT, true>(mw, ma, p, plan, dev_status, optin, st)
                        : launch_kernel<NT, OUT, false>(mw, ma, p, plan, dev_status, optin, st);
}

template <int NT>
cudaError_t launch_nt(const CUtensorMap& mw, const CUtensorMap& ma, const LinearArgs& p,
                      const Plan& plan, int32_t* dev_status, int optin, cudaStream_t st) {
  switch (p.c_dtype) {
    case MOE_BF16: return launch_out<NT, MOE_BF16>(mw, ma, p, plan, dev_status, optin, st);
    case MOE_FP16: return launch_out<NT, MOE_FP16>(mw, ma, p, plan, dev_status, optin, st);
    case MOE_FP32: return launch_out<NT, MOE_FP32>(mw, ma, p, plan, dev_status, optin, st);
    default: return launch_out<NT, MOE_INT32>(mw, ma, p, plan, dev_status, optin, st);
  }
}

// Whether the kernel that streams weights through integer dot products is the
// faster one.  A few rows of a plain product: 8 rows of 4096 x 7168 take 11.0 us
// there and 16.4 on the tensor cores, 9 rows 16.8 and 16.6.  A few per group on
// average: with 3, 256 groups of 4096 x 7168 take 1313 and 1281 us, 64 309 and
// 354, 32 of 7168 x 2048 89 and 102; with 4 1583 and 1334, 349 and 358, 105 and
// 102.  Small products, where the tile kernel's start-up (barriers, TMEM, clusters)
// is most of its time: 64 x 512 x 2048 takes 6.0 and 9.0 us, 512 x 256 x 1024 (at
// both limits) 9.0 and 9.3, 64 x 7168 x 256 (past the second) 16.9 and 7.4.  The rule
// does not see K below 1024 or how rows fall to the groups: 8 x 65,536 x 64 takes 18 us
// and would take 13 on the tensor cores, 512 rows over 256 groups of 2048 x 128 72 and
// 65, and 3 G rows that all fall to one group pass over its weights once per four rows.
bool use_few(const LinearArgs& p) {
  const int64_t outputs = p.a_rows * p.N;
  return p.a_rows <= (p.G == 1 ? 8 : 3 * p.G) ||
         (outputs <= (1 << 17) && outputs * p.K <= (1 << 27));
}

// Tokens per tile and pairs per K.  A plain product's tiles are known: the
// cheapest of the block sizes (multiples of 32) and splits by the time of the
// slowest pair, in clocks: a 64-code step takes 2 clocks a token in the MMA, or
// about 2 clocks per row (128 channels and half the tokens) to widen, whichever
// is more; a tile about 1500 besides, an exchange of partial sums 3000 more.
// Groups (sizes known on the device only): blocks that hold a group somewhat
// above the mean.
Plan make_plan(const LinearArgs& p, int sms) {
  const int64_t ntn = (p.N + CG * BM - 1) / (CG * BM);
  const int64_t stages = (p.K + BKB - 1) / BKB;
  const int64_t mean = (p.a_rows + p.G - 1) / p.G;
  Plan best{};
  double best_cost = 0.0;
  const int64_t least = (mean + 255) / 256;
  for (int64_t blocks = least; blocks <= 2 * least + 3 && blocks * 32 < mean + 32; ++blocks) {
    const int block = p.G > 1 ? (mean * 5 / 4 <= 128 ? 128 : 256)
                              : static_cast<int>(((mean + blocks - 1) / blocks + 31) / 32 * 32);
    // at most this many tiles, for any group sizes
    const int64_t tiles = p.G == 1
                              ? (p.a_rows + block - 1) / block * ntn
                              : (p.a_rows / block + std::min<int64_t>(p.G, p.a_rows)) * ntn;
    for (int split = 1; split <= kMaxSplit; ++split) {
      // clusters that run at once: larger ones leave SMs of a GPU cluster unused
      // (152 SMs hold 76 clusters of 2, 36 of 4, 23 of 6, 15 of 8)
      const int64_t room = sms * (split == 1 ? 76 : split == 2 ? 36 : split == 3 ? 23 : 15) / 152;
      if (split > 1 && (tiles > room || stages < 2 * split)) break;
      const double waves = static_cast<double>((tiles + room - 1) / room);
      const double step = std::max(2.0 * block, 2.05 * (BM + block / 2));
      const double cost =
          waves * (step * kHalves * ((stages + split - 1) / split) + 1500) + (split > 1) * 3000;
      if (best.nt == 0 || cost < best_cost) {
        best_cost = cost;
        best.block = block;
        best.split = split;
        best.clusters = static_cast<int>(std::min(tiles, room));
        best.nt = block <= 128 ? 128 : 256;
      }
    }
    if (p.G > 1) break;
  }
  const int64_t tokens = p.G > 1 ? mean : best.block;       // a CTA copies half of them
  best.box_rows = tokens > 64 ? 64 : tokens > 32 ? 32 : 16;
  return best;
}

}  // namespace

#ifndef MOE_LINEAR_I8_POLLS
cudaError_t launch_linear_i8(const LinearArgs& p, int32_t* dev_status, cudaStream_t st) {
  if (use_few(p)) return launch_linear_i8_few(p, dev_status, st);
  int dev = 0, sms = 0, optin = 0;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e != cudaSuccess) return e;
  const Plan plan = make_plan(p, sms);
  CUtensorMap mw, ma;
  e = encode_bytes_2d(&mw, p.w, int64_t(p.G) * p.N, p.K, p.w_stride, BM);
  if (e == cudaSuccess)
    e = encode_bytes_2d(&ma, p.a, p.a_rows, p.K, p.a_stride, plan.box_rows);
  if (e != cudaSuccess) return e;
  return plan.nt == 256 ? launch_nt<256>(mw, ma, p, plan, dev_status, optin, st)
                        : launch_nt<128>(mw, ma, p, plan, dev_status, optin, st);
}
#endif

}  // namespace moe_ep

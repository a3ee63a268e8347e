// linear_f8_few.cu -- the e4m3 product for groups of a few rows (decoding: one token, or
// a few tokens per expert).
//
// With few rows the product is a stream of the weights' bytes, and the arithmetic only
// has to keep up: a warp's matrix instruction multiplies 16 weight rows x 32 codes with
// 8 tokens (fp32 sums), four of them a 128-code block, whose sums then get the block's
// scales, one fused multiply-add each.  The sum over K does not care which code stands
// where as long as both operands agree, so a lane takes 16 consecutive bytes of its rows
// as four words of the instructions' fragments and nothing is shuffled.
//
// What bounds it is the weights' way from memory, and that wants long runs and many bytes
// on their way: loads of 64 or 128 bytes a row reached 6.1 TB/s, of 256 or 512 7.1, with
// 130 KB of an SM in flight 6.5 and with 190 7.05.  So a step of a warp is 256 codes of 16
// rows, copied asynchronously into a ring of kDepth steps of its own in shared memory (no
// barrier but the warp's own stands between copy and use), four CTAs to an SM.  The ring
// runs on over tile ends.  Tokens and scales come through L1, a step ahead, in registers.
// (With the weights a block ahead in registers too they came at 3.3 TB/s.)
//
// Measured (in a graph): one token by 4096 x 7168 7.1 to 7.5 us (29 MB, 4.3 us at a copy's
// rate; the rest is the launch, the first bytes' way and the sums), 8 tokens 8.4, 16 tokens
// 14.2 (each weight byte meets two instructions), 16 in 8 groups of 4096 x 4096 27.5.  Many
// groups are linear_f8.cu's: 256 tokens over 256 experts of 4096 x 7168 take 734 us here and
// 721 there; with 8 rows a group the tokens' way through L1 is the longer one.
//
// A warp takes 16 channels and up to 8 TB tokens; `parts` warps of a CTA split K where
// there are too few channels to fill the GPU (their sums are added in order).  A
// persistent grid walks (group, channels, token block), a group's token blocks fastest, so
// a second block finds the weights in L2.
#include <algorithm>

#include "group_tiles.cuh"
#include "moe_ep_internal.cuh"
#include "row_codes.cuh"

namespace moe_ep {
namespace {

constexpr int kChannels = 16;        // weight rows per warp
constexpr int kStep = 256;           // codes of K per step: two blocks
constexpr int kDepth = 3;            // steps in a warp's ring
constexpr uint32_t kStepBytes = kChannels * kStep;
__host__ __device__ constexpr size_t ring_bytes(int warps) {
  return size_t(warps) * kDepth * kStepBytes;
}

__device__ __forceinline__ void mma_f8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first `bytes` (0 to 16) of a 16-byte piece to shared memory, zeros behind them;
// reads those bytes alone.
__device__ __forceinline__ void copy_piece(uint32_t to, const uint8_t* from, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ uint4 read_piece(uint32_t from) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(from) : "memory");
  return v;
}

// The first n bytes of a 16-byte piece of a token row, zeros behind them; reads those n
// alone: the row may end there, and the buffer with it.
__device__ __forceinline__ uint4 token_piece(const uint8_t* p, int n) {
  if (n >= 16) return *reinterpret_cast<const uint4*>(p);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < n) w[i / 4] |= uint32_t(p[i]) << (8 * (i % 4));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

struct Tile {
  int g, n0, row0, tokens;
};

template <int TB>
struct Tokens {                      // a step as a lane holds it
  uint4 x[TB][4];                    // tokens gid of each eight: pieces tig, tig + 4, ...
  float s[TB][2][2];                 // scales of tokens 2 tig and 2 tig + 1, of both blocks
};

// TB: tokens per block / 8.
template <int TB, int kWarps>
__global__ void __launch_bounds__(32 * kWarps)
linear_f8_few_kernel(const LinearArgs p, int parts, int32_t* dev_status) {
  constexpr int kThreads = 32 * kWarps;
  extern __shared__ __align__(16) uint8_t s_ring[];          // the rings, then the group tables
  __shared__ int64_t s_scan[kThreads * 12 / 8];
  __shared__ float s_sums[kWarps][8 * TB][kChannels];
  wait_for_stream();
  let_next_start();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const int part = warp % parts, slot = warp / parts;
  const int chans = kWarps / parts * kChannels;          // channels per CTA
  const int ntn = (p.N + chans - 1) / chans;
  const int kblocks = code_blocks(p.K), nblocks = code_blocks(p.N);
  const int steps = (p.K + kStep - 1) / kStep;
  const uint32_t goff = smem_addr(s_ring) + ring_bytes(kWarps), tpre = goff + 4 * (p.G + 1);
  const bool grouped = p.group_rows != nullptr;
  int tiles = row_blocks(static_cast<int>(p.a_rows), 8 * TB) * ntn;
  if (grouped) {
    build_group_tables<kThreads>(p, 8 * TB, ntn, s_scan, goff, tpre, dev_status);
    __syncthreads();
    tiles = smem_load(tpre + 4 * p.G);
  }
  auto decode = [&](int t) {
    int g = 0, local = t, off = 0, end = static_cast<int>(p.a_rows);
    if (grouped) {
      g = group_of_tile(t, tpre, p.G);
      local = t - smem_load(tpre + 4 * g);
      off = smem_load(goff + 4 * g);
      end = smem_load(goff + 4 * g + 4);
    }
    const int blocks = row_blocks(end - off, 8 * TB);
    Tile tl;
    tl.g = g;
    tl.n0 = local / blocks * chans;
    tl.row0 = off + local % blocks * (8 * TB);
    tl.tokens = min(8 * TB, end - tl.row0);
    return tl;
  };

  // ---- copies of weights, kDepth - 1 steps ahead of the products --------------------------
  // Copy j takes rows 2 j and 2 j + 1, a half warp 256 bytes of each.  16-byte piece q of row
  // r lies at q ^ 4 (r & 1), so that the reads of two rows' pieces meet no bank twice.
  const uint32_t ring = smem_addr(s_ring) + warp * kDepth * kStepBytes;
  const int crow = lane >> 4, cpiece = lane & 15;
  const uint32_t cto = ring + crow * kStep + ((cpiece ^ (crow << 2)) << 4);
  int load_tile = blockIdx.x, load_step = part, load_slot = 0;
  const uint8_t* w = nullptr;          // of the tile's first row, this lane's piece
  int last = 0;                        // rows past the last channel repeat that one
  auto aim = [&]() {
    if (load_tile >= tiles) return;
    const Tile tl = decode(load_tile);
    const int n = min(tl.n0 + slot * kChannels, p.N - 1);
    w = static_cast<const uint8_t*>(p.w) + (int64_t(tl.g) * p.N + n) * p.w_stride;
    last = p.N - 1 - n;
  };
  auto copy_step = [&]() {
    if (load_tile < tiles) {
      const int at = load_step * kStep + 16 * cpiece;
      const int bytes = max(0, min(16, p.K - at));
      const uint8_t* from = w + (bytes ? at : 0);
      const uint32_t to = cto + load_slot * kStepBytes;
#pragma unroll
      for (int j = 0; j < kChannels / 2; ++j)
        copy_piece(to + 2 * j * kStep, from + min(2 * j + crow, last) * p.w_stride, bytes);
      load_step += parts;
      if (load_step >= steps) {        // (every warp has a step in every tile)
        load_step = part;
        load_tile += gridDim.x;
        aim();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++load_slot == kDepth) load_slot = 0;
  };
  aim();
  for (int i = 0; i < kDepth - 1; ++i) copy_step();

  int use_slot = 0;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const Tile tl = decode(t);
    const int n = min(tl.n0 + slot * kChannels, p.N - 1);
    const float* col = p.col_scale + (int64_t(tl.g) * nblocks + n / kCodeBlock) * kblocks;
    const unsigned char* rs = p.row_scale + int64_t(tl.row0) * p.row_scale_stride;
    const uint8_t* a = static_cast<const uint8_t*>(p.a) + int64_t(tl.row0) * p.a_stride + 16 * tig;
    auto load_tokens = [&](int step, Tokens<TB>& v) {     // tokens past the last repeat it
      float c[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) c[b] = 2 * step + b < kblocks ? col[2 * step + b] : 0.0f;
#pragma unroll
      for (int i = 0; i < TB; ++i) {
        const uint8_t* x = a + min(8 * i + gid, tl.tokens - 1) * p.a_stride + step * kStep;
        const int left = p.K - step * kStep - 16 * tig;
#pragma unroll
        for (int q = 0; q < 4; ++q) v.x[i][q] = token_piece(x + 64 * q, left - 64 * q);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float* r = reinterpret_cast<const float*>(
              rs + min(8 * i + 2 * tig + j, tl.tokens - 1) * p.row_scale_stride) + 2 * step;
          v.s[i][0][j] = __fmul_rn(r[0], c[0]);
          v.s[i][1][j] = 2 * step + 1 < kblocks ? __fmul_rn(r[1], c[1]) : 0.0f;
        }
      }
    };
    float acc[TB][4] = {};
    Tokens<TB> cur, next;
    load_tokens(part, cur);
    for (int step = part; step < steps; step += parts) {
      if (step + parts < steps) load_tokens(step + parts, next);
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
      __syncwarp();
      const uint32_t from =
          ring + use_slot * kStepBytes + gid * kStep + ((tig ^ ((gid & 1) << 2)) << 4);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint4 u[2][2];                 // rows gid and gid + 8, pieces tig and tig + 4
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          u[r][0] = read_piece(from + r * 8 * kStep + b * 128);
          u[r][1] = read_piece((from ^ 64) + r * 8 * kStep + b * 128);
        }
#pragma unroll
        for (int i = 0; i < TB; ++i) {
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 v = cur.x[i][2 * b + h];
            mma_f8(c, u[0][h].x, u[1][h].x, u[0][h].y, u[1][h].y, v.x, v.y);
            mma_f8(c, u[0][h].z, u[1][h].z, u[0][h].w, u[1][h].w, v.z, v.w);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = __fmaf_rn(c[j], cur.s[i][b][j & 1], acc[i][j]);
        }
      }
      if (++use_slot == kDepth) use_slot = 0;
      __syncwarp();
      copy_step();               // into the slot of the step before this one
      cur = next;
    }
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s_sums[warp][8 * i + 2 * tig + (j & 1)][gid + 8 * (j >> 1)] = acc[i][j];
    __syncthreads();
    for (int o = tid; o < tl.tokens * chans; o += kThreads) {
      const int tk = o / chans, ch = o - tk * chans, nn = tl.n0 + ch;
      if (nn >= p.N) continue;
      float v = 0.0f;
      for (int i = 0; i < parts; ++i)
        v = __fadd_rn(v, s_sums[ch / kChannels * parts + i][tk][ch % kChannels]);
      if (p.bias) v = __fadd_rn(v, p.bias[int64_t(tl.g) * p.N + nn]);
      const int64_t at = int64_t(tl.row0 + tk) * p.N + nn;
      if (p.c_dtype == MOE_FP32)
        static_cast<float*>(p.c)[at] = v;
      else
        static_cast<uint16_t*>(p.c)[at] = static_cast<uint16_t>(
            p.c_dtype == MOE_BF16 ? narrow_rn<MOE_BF16>(v) : narrow_rn<MOE_FP16>(v));
    }
    __syncthreads();
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Whether it was launched (parts of K: all kWarps of a CTA where `all`, which then has to
// leave all CTAs running at once; else as many as that allows).
template <int TB, int kWarps>
cudaError_t launch_few(const LinearArgs& p, bool all, bool* done, int32_t* dev_status,
                       cudaStream_t st) {
  const size_t smem = ring_bytes(kWarps) + size_t(p.G + 1) * 8;
  auto kernel = linear_f8_few_kernel<TB, kWarps>;
  const void* fn = reinterpret_cast<const void*>(kernel);
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e == cudaSuccess) e = kernel_blocks_per_sm(fn, 32 * kWarps, smem, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t blocks = p.G == 1
                             ? (p.a_rows + 8 * TB - 1) / (8 * TB)
                             : p.a_rows / (8 * TB) + std::min<int64_t>(p.G, p.a_rows);
  const int64_t room = int64_t(std::max(1, per_sm)) * sms;
  const int pieces = (p.K + kStep - 1) / kStep;
  auto ctas = [&](int parts) {
    const int chans = kWarps / parts * kChannels;
    return blocks * ((p.N + chans - 1) / chans);
  };
  int parts = 1;
  while (parts < kWarps && parts * 2 <= pieces && ctas(parts * 2) <= room) parts *= 2;
  *done = !all || parts == kWarps;
  if (!*done) return cudaSuccess;
  if (ctas(parts) > INT32_MAX) return cudaErrorInvalidValue;
  return launch_early(kernel, std::min(ctas(parts), room), 32 * kWarps, smem, st, p, parts,
                      dev_status);
}

}  // namespace

// Eight warps to a CTA where they can split K eight ways (one token by 4096 x 7168 7.4 us,
// with four warps 8.5), else four (100 rows in 200 groups of 300 x 300 7.9 and with eight
// 8.4).  More than 8 rows a group: two blocks of 8 share the weights' way (16 rows of 4096 x
// 7168 14.3 us).
cudaError_t launch_linear_f8_few(const LinearArgs& p, int32_t* dev_status, cudaStream_t st) {
  bool done = false;
  if ((p.a_rows + p.G - 1) / p.G > 8) return launch_few<2, 4>(p, false, &done, dev_status, st);
  const cudaError_t e = launch_few<1, 8>(p, true, &done, dev_status, st);
  if (done || e != cudaSuccess) return e;
  return launch_few<1, 4>(p, false, &done, dev_status, st);
}

}  // namespace moe_ep

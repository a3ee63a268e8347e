// linear_f8_few.cu -- the e4m3 product for groups of a few rows (decoding: one token, or
// a few tokens per expert).
//
// With few rows the product is a stream of the weights' bytes, and the arithmetic only
// has to keep up: a warp's matrix instruction multiplies 16 weight rows x 32 codes with
// 8 tokens (fp32 sums), four of them a 128-code block, whose sums then get the block's
// scales, one fused multiply-add each.  The sum over K does not care which code stands
// where as long as both operands agree, so a lane takes 16 consecutive bytes of its rows
// as four words of the instructions' fragments and nothing is shuffled: weights go from
// memory to registers, 64 consecutive bytes of 8 rows per load.
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

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChannels = 16;        // weight rows per warp

__device__ __forceinline__ void mma_f8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first n bytes of a 16-byte piece, zeros behind them, reading those n alone where
// EXACT (a row of a may end there, and the buffer with it), else the whole piece if n > 0.
template <bool EXACT>
__device__ __forceinline__ uint4 first_bytes(const uint8_t* p, int n) {
  if (n >= 16) return EXACT ? *reinterpret_cast<const uint4*>(p) : ld_once_16(p);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (n > 0) {
    if constexpr (EXACT) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) w[i / 4] |= uint32_t(p[i]) << (8 * (i % 4));
    } else {
      const uint4 v = ld_once_16(p);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int keep = n - 4 * i;
        w[i] = keep >= 4 ? u[i] : keep <= 0 ? 0u : u[i] & ((1u << (8 * keep)) - 1u);
      }
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int TB>
struct Block {                       // a 128-code block as a lane holds it
  uint4 w[2][2];                     // weight rows gid and gid + 8, pieces tig and tig + 4
  uint4 x[TB][2];                    // tokens gid of each eight
  float row[TB][2];                  // scales of tokens 2 tig and 2 tig + 1 of each eight
  float col;
};

// TB: tokens per block / 8.
template <int TB>
__global__ void __launch_bounds__(kThreads)
linear_f8_few_kernel(const LinearArgs p, int parts, int32_t* dev_status) {
  extern __shared__ int s_tables[];
  __shared__ int64_t s_scan[kThreads * 12 / 8];
  __shared__ float s_sums[kWarps][8 * TB][kChannels];
  wait_for_stream();
  let_next_start();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const int part = warp % parts, slot = warp / parts;
  const int chans = kWarps / parts * kChannels;          // channels per CTA
  const int ntn = (p.N + chans - 1) / chans;
  const int kblocks = code_blocks(p.K), nblocks = code_blocks(p.N), whole = p.K / kCodeBlock;
  const uint32_t goff = smem_addr(s_tables), tpre = goff + 4 * (p.G + 1);
  const bool grouped = p.group_rows != nullptr;
  int tiles = row_blocks(static_cast<int>(p.a_rows), 8 * TB) * ntn;
  if (grouped) {
    build_group_tables<kThreads>(p, 8 * TB, ntn, s_scan, goff, tpre, dev_status);
    __syncthreads();
    tiles = smem_load(tpre + 4 * p.G);
  }
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    int g = 0, local = t, off = 0, end = static_cast<int>(p.a_rows);
    if (grouped) {
      g = group_of_tile(t, tpre, p.G);
      local = t - smem_load(tpre + 4 * g);
      off = smem_load(goff + 4 * g);
      end = smem_load(goff + 4 * g + 4);
    }
    const int blocks = row_blocks(end - off, 8 * TB);
    const int row0 = off + local % blocks * (8 * TB), n0 = local / blocks * chans;
    const int tokens = min(8 * TB, end - row0);
    // rows past the last channel or token repeat that one; their sums go nowhere
    const int n = n0 + slot * kChannels, last = p.N - 1;
    const uint8_t* wbase = static_cast<const uint8_t*>(p.w) + int64_t(g) * p.N * p.w_stride;
    const uint8_t* w0 = wbase + min(n + gid, last) * p.w_stride;
    const uint8_t* w1 = wbase + min(n + gid + 8, last) * p.w_stride;
    const float* col = p.col_scale +
                       (int64_t(g) * nblocks + min(n, last) / kCodeBlock) * kblocks;
    const uint8_t* a = static_cast<const uint8_t*>(p.a) + int64_t(row0) * p.a_stride;
    const uint8_t* rs = p.row_scale + int64_t(row0) * p.row_scale_stride;

    auto load = [&](Block<TB>& b, int kb) {
      const int at = kb * kCodeBlock + 16 * tig;
      if (kb < whole) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          b.w[0][h] = ld_once_16(w0 + at + 64 * h);
          b.w[1][h] = ld_once_16(w1 + at + 64 * h);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          b.w[0][h] = first_bytes<false>(w0 + at + 64 * h, p.K - at - 64 * h);
          b.w[1][h] = first_bytes<false>(w1 + at + 64 * h, p.K - at - 64 * h);
        }
      }
      b.col = col[kb];
#pragma unroll
      for (int i = 0; i < TB; ++i) {
        const uint8_t* x = a + min(8 * i + gid, tokens - 1) * p.a_stride + at;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          b.x[i][h] = kb < whole ? *reinterpret_cast<const uint4*>(x + 64 * h)
                                 : first_bytes<true>(x + 64 * h, p.K - at - 64 * h);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          b.row[i][j] = *reinterpret_cast<const float*>(
              rs + min(8 * i + 2 * tig + j, tokens - 1) * p.row_scale_stride + 4 * kb);
      }
    };
    float acc[TB][4] = {};
    auto use = [&](const Block<TB>& b) {
#pragma unroll
      for (int i = 0; i < TB; ++i) {
        float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mma_f8(c, b.w[0][h].x, b.w[1][h].x, b.w[0][h].y, b.w[1][h].y, b.x[i][h].x,
                 b.x[i][h].y);
          mma_f8(c, b.w[0][h].z, b.w[1][h].z, b.w[0][h].w, b.w[1][h].w, b.x[i][h].z,
                 b.x[i][h].w);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __fmaf_rn(c[j], __fmul_rn(b.row[i][j & 1], b.col), acc[i][j]);
      }
    };
    // the next block is on its way while this one is used
    Block<TB> cur, next;
    int kb = part;
    if (kb < kblocks) load(cur, kb);
    while (kb < kblocks) {
      const int then = kb + parts;
      if (then < kblocks) load(next, then);
      use(cur);
      cur = next;
      kb = then;
    }
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s_sums[warp][8 * i + 2 * tig + (j & 1)][gid + 8 * (j >> 1)] = acc[i][j];
    __syncthreads();
    for (int o = tid; o < tokens * chans; o += kThreads) {
      const int tk = o / chans, ch = o - tk * chans, nn = n0 + ch;
      if (nn >= p.N) continue;
      float v = 0.0f;
      for (int i = 0; i < parts; ++i)
        v = __fadd_rn(v, s_sums[ch / kChannels * parts + i][tk][ch % kChannels]);
      if (p.bias) v = __fadd_rn(v, p.bias[int64_t(g) * p.N + nn]);
      const int64_t at = int64_t(row0 + tk) * p.N + nn;
      if (p.c_dtype == MOE_FP32)
        static_cast<float*>(p.c)[at] = v;
      else
        static_cast<uint16_t*>(p.c)[at] = static_cast<uint16_t>(
            p.c_dtype == MOE_BF16 ? narrow_rn<MOE_BF16>(v) : narrow_rn<MOE_FP16>(v));
    }
    __syncthreads();
  }
}

template <int TB>
cudaError_t launch_few(const LinearArgs& p, int32_t* dev_status, cudaStream_t st) {
  const size_t smem = size_t(p.G + 1) * 8;
  auto kernel = linear_f8_few_kernel<TB>;
  const void* fn = reinterpret_cast<const void*>(kernel);
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e == cudaSuccess) e = kernel_blocks_per_sm(fn, kThreads, smem, &per_sm);
  if (e != cudaSuccess) return e;
  // Split K over more warps while all CTAs still run at once.
  const int64_t blocks = p.G == 1
                             ? (p.a_rows + 8 * TB - 1) / (8 * TB)
                             : p.a_rows / (8 * TB) + std::min<int64_t>(p.G, p.a_rows);
  const int64_t room = int64_t(std::max(1, per_sm)) * sms;
  const int pieces = code_blocks(p.K);
  int parts = 1;
  auto ctas = [&](int parts) {
    const int chans = kWarps / parts * kChannels;
    return blocks * ((p.N + chans - 1) / chans);
  };
  while (parts < kWarps && parts * 2 <= pieces && ctas(parts * 2) <= room) parts *= 2;
  if (ctas(parts) > INT32_MAX) return cudaErrorInvalidValue;
  return launch_early(kernel, std::min(ctas(parts), room), kThreads, smem, st, p, parts,
                      dev_status);
}

}  // namespace

cudaError_t launch_linear_f8_few(const LinearArgs& p, int32_t* dev_status, cudaStream_t st) {
  const int64_t mean = (p.a_rows + p.G - 1) / p.G;
  return mean <= 8 ? launch_few<1>(p, dev_status, st) : mean <= 16
             ? launch_few<2>(p, dev_status, st) : launch_few<4>(p, dev_status, st);
}

}  // namespace moe_ep

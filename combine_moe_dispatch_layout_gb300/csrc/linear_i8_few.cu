// linear_i8_few.cu -- the 8-bit matrix product for groups of a few rows
// (decoding: one token, or a few tokens per expert).
//
// With few rows the product is a stream of the weights' bytes, and the
// arithmetic that keeps up with it is the four-way integer dot product: one
// instruction takes 4 codes of a weight row and of a token, no widening, exact
// int32 sums.  (Measured on this GPU: 265 products per clock and SM, against 23
// weight bytes per clock and SM from memory.)
//
// A warp takes kChannels weight rows and a block of up to 4 tokens; its lanes
// take neighbouring 16-byte pieces of K, so a load instruction reads 512
// consecutive bytes of one weight row.  The token codes come through L1 (the
// CTA's warps share them), the weights go past it.  A lane's sums are added over
// the warp by halving exchanges (15 shuffles and one step for 16 sums), and,
// where there are too few weight rows to fill the GPU, over the warps that split
// K.  A persistent grid walks (group, channels, token block); the token blocks
// of a group are fastest, so a second block finds the weights in L2.  (Blocks of
// 8 tokens were slower: 32 sums a lane leave no registers for loads in flight.)
//
// Measured: one token by 4096 x 7168 4.7 us in a graph, weights partly in L2, and 7.4 to
// 8.0 call by call (29 MB: 4.3 us at a copy's rate; the rest is the launch, the first
// load's way and the sums), 164 of 256 experts' 4096 x 7168 for 256 tokens 667 to 720
// us, 6.7 to 7.2 TB/s: bound by memory.  Seven CTAs of 128 threads to an SM spread 1024
// quads of channels more evenly over 152 SMs than three of 256 did (8.4 and 725 us).
// Short K leaves lanes without a piece: 80 rows in 138 groups of 4096 x 64 take 35 us,
// of 4096 x 256 38.
#include <algorithm>
#include <type_traits>

#include "group_tiles.cuh"
#include "moe_ep_internal.cuh"

namespace moe_ep {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kChannels = 4;         // weight rows per warp
constexpr int kTokens = 4;           // tokens per block at most
constexpr int kPiece = 512;          // bytes of K per warp step
constexpr unsigned kAll = 0xffffffffu;

// Sums V values per lane over the warp: afterwards lane l holds the totals of
// values l * V/32 .. (V >= 32), or of value l >> (5 - log2 V).
template <int V>
__device__ __forceinline__ void warp_totals(int (&v)[V], int lane) {
  int n = V;
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool upper = lane & d;
#pragma unroll
      for (int i = 0; i < V / 2; ++i)
        if (i < n) {
          const int send = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
          v[i] = keep + __shfl_xor_sync(kAll, send, d);
        }
    } else {
      v[0] += __shfl_xor_sync(kAll, v[0], d);
    }
  }
}

// The first n (0 < n < 16) bytes of a 16-byte piece, zeros behind them.  Reads those n
// alone: a row of a may end there, and the buffer with it.
__device__ __forceinline__ uint4 first_bytes(const uint8_t* p, int n) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = 0u;
    if (4 * i + 4 <= n) {
      w[i] = *reinterpret_cast<const uint32_t*>(p + 4 * i);
    } else {
#pragma unroll
      for (int b = 0; b < 3; ++b)
        if (4 * i + b < n) w[i] |= uint32_t(p[4 * i + b]) << (8 * b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int c) {
  c = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), c);
  c = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), c);
  c = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), c);
  return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), c);
}

// Totals of kChannels weight rows x TB tokens over this warp's pieces of K into
// sums[channel * kTokens + token].  w, a: the first rows; rows past the last
// channel (last, from the first) or the last token repeat that one.
template <int TB>
__device__ __forceinline__ void channels_by_tokens(const uint8_t* w, int64_t w_stride,
                                                   int last, const uint8_t* a,
                                                   int64_t a_stride, int tokens, int K,
                                                   int part, int parts, int lane, int* sums) {
  auto weights = [&](int r, int j) { return ld_once_16(w + min(r, last) * w_stride + j); };
  constexpr int CH = kChannels;
  int acc[CH * TB];
#pragma unroll
  for (int i = 0; i < CH * TB; ++i) acc[i] = 0;
  const int step = parts * kPiece;
  int j = part * kPiece + lane * 16;
  // one token: the next step's weights are on their way while this one's are used
  // (with more, the sums take those registers and the longer arithmetic of the
  // other warps covers the loads)
  constexpr bool kAhead = TB < 2;
  uint4 next[CH];
  if (kAhead) {
#pragma unroll
    for (int r = 0; r < CH; ++r) next[r] = j < K ? weights(r, j) : make_uint4(0u, 0u, 0u, 0u);
  }
  for (; j < K; j += step) {
    uint4 cur[CH];
#pragma unroll
    for (int r = 0; r < CH; ++r) cur[r] = kAhead ? next[r] : weights(r, j);
    if (kAhead && j + step < K) {
#pragma unroll
      for (int r = 0; r < CH; ++r) next[r] = weights(r, j + step);
    }
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      // (a weight row's bytes past K meet zeros here)
      const uint8_t* at = a + (t < tokens ? t : tokens - 1) * a_stride + j;
      const uint4 x = j + 16 <= K ? *reinterpret_cast<const uint4*>(at) : first_bytes(at, K - j);
#pragma unroll
      for (int r = 0; r < CH; ++r) acc[r * TB + t] = dot16(cur[r], x, acc[r * TB + t]);
    }
  }
  warp_totals<CH * TB>(acc, lane);
  constexpr int V = CH * TB, kLog = V == 4 ? 2 : V == 8 ? 3 : 4;
  static_assert(V == 1 << kLog, "4, 8 or 16 sums");
  const int idx = lane >> (5 - kLog);
  if ((lane & ((1 << (5 - kLog)) - 1)) == 0) sums[idx / TB * kTokens + idx % TB] = acc[0];
}

// parts: warps that split K (a divisor of kWarps).
__global__ void __launch_bounds__(kThreads, 7)
linear_i8_few_kernel(const LinearArgs p, int parts, int32_t* dev_status) {
  extern __shared__ int s_tables[];
  __shared__ int64_t s_scan[kThreads * 12 / 8];
  __shared__ int s_sums[kWarps][kChannels * kTokens];
  wait_for_stream();
  let_next_start();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = warp % parts, slot = warp / parts;
  const int chans = kWarps / parts * kChannels;          // channels per CTA
  const int ntn = (p.N + chans - 1) / chans;
  const uint32_t goff = smem_addr(s_tables), tpre = goff + 4 * (p.G + 1);
  const bool grouped = p.group_rows != nullptr;
  int tiles = row_blocks(static_cast<int>(p.a_rows), kTokens) * ntn;
  if (grouped) {
    build_group_tables<kThreads>(p, kTokens, ntn, s_scan, goff, tpre, dev_status);
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
    const int blocks = row_blocks(end - off, kTokens);
    const int row0 = off + local % blocks * kTokens, n0 = local / blocks * chans;
    const int tokens = min(kTokens, end - row0);
    const uint8_t* a = static_cast<const uint8_t*>(p.a) + int64_t(row0) * p.a_stride;
    const int n = min(n0 + slot * kChannels, p.N - 1), last = p.N - 1 - n;
    const uint8_t* w = static_cast<const uint8_t*>(p.w) + (int64_t(g) * p.N + n) * p.w_stride;
    int* sums = s_sums[warp];
    auto run = [&](auto tb) {
      channels_by_tokens<decltype(tb)::value>(w, p.w_stride, last, a, p.a_stride, tokens, p.K,
                                              part, parts, lane, sums);
    };
    if (tokens == 1) run(std::integral_constant<int, 1>());
    else if (tokens == 2) run(std::integral_constant<int, 2>());
    else run(std::integral_constant<int, 4>());
    __syncthreads();
    for (int o = tid; o < tokens * chans; o += kThreads) {
      const int tk = o / chans, ch = o - tk * chans, n = n0 + ch;
      if (n >= p.N) continue;
      int acc = 0;
      for (int i = 0; i < parts; ++i)
        acc += s_sums[ch / kChannels * parts + i][ch % kChannels * kTokens + tk];
      const int64_t m = row0 + tk, at = m * p.N + n, gn = int64_t(g) * p.N + n;
      if (p.c_dtype == MOE_INT32) {
        static_cast<int32_t*>(p.c)[at] = acc;
        continue;
      }
      const float row =
          *reinterpret_cast<const float*>(p.row_scale + m * p.row_scale_stride);
      float v = __fmul_rn(__fmul_rn(__int2float_rn(acc), p.col_scale[gn]), row);
      if (p.bias) v = __fadd_rn(v, p.bias[gn]);
      if (p.c_dtype == MOE_FP32)
        static_cast<float*>(p.c)[at] = v;
      else
        static_cast<uint16_t*>(p.c)[at] = static_cast<uint16_t>(
            p.c_dtype == MOE_BF16 ? narrow_rn<MOE_BF16>(v) : narrow_rn<MOE_FP16>(v));
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_linear_i8_few(const LinearArgs& p, int32_t* dev_status, cudaStream_t st) {
  const size_t smem = size_t(p.G + 1) * 8;
  const void* fn = reinterpret_cast<const void*>(linear_i8_few_kernel);
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e == cudaSuccess) e = kernel_blocks_per_sm(fn, kThreads, smem, &per_sm);
  if (e != cudaSuccess) return e;
  // Split K over more warps while all CTAs still run at once.
  const int64_t blocks = p.G == 1 ? (p.a_rows + kTokens - 1) / kTokens
                                  : p.a_rows / kTokens + std::min<int64_t>(p.G, p.a_rows);
  const int64_t room = int64_t(std::max(1, per_sm)) * sms;
  const int pieces = (p.K + kPiece - 1) / kPiece;
  int parts = 1;
  auto ctas = [&](int parts) {
    const int chans = kWarps / parts * kChannels;
    return blocks * ((p.N + chans - 1) / chans);
  };
  while (parts < kWarps && parts * 2 <= pieces && ctas(parts * 2) <= room)
    parts *= 2;
  if (ctas(parts) > INT32_MAX) return cudaErrorInvalidValue;
  const int64_t grid = std::min(ctas(parts), room);
  return launch_early(linear_i8_few_kernel, grid, kThreads, smem, st, p, parts, dev_status);
}

}  // namespace moe_ep

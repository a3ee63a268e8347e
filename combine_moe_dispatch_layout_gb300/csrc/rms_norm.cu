// rms_norm.cu -- residual addition, root-mean-square norm and 8-bit row images in one
// pass, and the norm's gradient (include/moe_ep.h, moe_rms_norm).
//
// Mathematics.  s = x + r rounded to the token type (the residual stream as it is
// stored, and so what the norm is of), rstd = (mean(s^2) + eps)^-1/2 in fp32,
// y = (s * rstd) * gamma.  The 16-bit rows and the codes are both rounded from the
// fp32 y, once each.  Gradient, with xh = s * rstd and a = gamma * dy:
//   dx = rstd * (a - xh * mean(a * xh)) + d_sum,   d_gamma = sum over rows of dy * xh.
//
// Both are bound by memory.  A row is read once, by TPR threads that keep it in
// registers (16-bit, NV chunks of 8 values each) over the reduction; thread t holds
// chunks t, t + TPR, ..., so every access of a warp is 512 consecutive bytes and a
// half warp holds the 128 values of an e4m3 block.  Measured: 32,768 x 7168 with its residual
// 271 us, 103% of a copy's rate, with codes too 319 (98%); 24,251 x 1000 to codes 17.3 (63%:
// instructions, and one stream of loads a warp); the gradient of 32,768 x 7168 290 (97%).
// INT8 codes wait for a second reduction, the row's maximum: 330 us for the first (95%), 20.0
// for the narrow rows.
#include <algorithm>

#include "row_codes.cuh"

namespace moe_ep {

// rms_norm_polls.cu compiles the gradient's kernel a second time, for tests of the waits that
// run out: with a wait of its own, and without the functions that others call.
#ifndef MOE_RMS_NORM_POLLS
namespace {
// A thread's wait for its team's next row; false after kGemmSpin polls.
__device__ __forceinline__ bool row_wait(uint64_t* bar, uint32_t parity) {
  return mbar_wait_bounded(bar, parity, kGemmSpin);
}
}  // namespace
#endif

namespace {

constexpr int kNoCodes = -1;
constexpr unsigned kAll = 0xffffffffu;

__host__ __device__ constexpr int block_threads(int tpr) { return tpr < 64 ? 128 : tpr; }

// Over the TPR threads of a row, in an order fixed by TPR alone; every thread gets
// the result.  part: this row's TPR / 32 words of shared memory, not in use by an
// earlier call that a thread may still be reading from.
template <int TPR, class T, class Op>
__device__ __forceinline__ T row_reduce(T v, T* part, int t, Op op) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = op(v, __shfl_xor_sync(kAll, v, d));
  if constexpr (TPR > 32) {
    if (t % 32 == 0) part[t / 32] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int i = 1; i < TPR / 32; ++i) v = op(v, part[i]);
  }
  return v;
}

struct Add {
  __device__ float operator()(float a, float b) const { return __fadd_rn(a, b); }
};
struct Max {
  __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return max(a, b); }
};

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

template <int DT, int TPR, int NV, int CODE>
__global__ void __launch_bounds__(block_threads(TPR))
rms_norm_kernel(const NormArgs p) {
  __shared__ float s_sum[32];
  __shared__ uint32_t s_max[32];
  wait_for_stream();
  let_next_start();
  constexpr int kRows = block_threads(TPR) / TPR;
  const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  const int64_t row = int64_t(blockIdx.x) * kRows + slot;
  if (row >= p.T) return;            // (a whole warp; TPR > 32 has one row per CTA)
  const int chunks = p.H / 8;
  const uint16_t* x = static_cast<const uint16_t*>(p.x) + row * p.x_stride;
  uint4 v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * TPR + t;
    v[i] = c < chunks ? ld_once_16(x + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
  }
  if (p.residual) {
    const uint16_t* r = static_cast<const uint16_t*>(p.residual) + row * p.residual_stride;
    uint16_t* sum = static_cast<uint16_t*>(p.sum) + row * p.sum_stride;
    uint4 u[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * TPR + t;
      u[i] = c < chunks ? ld_once_16(r + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a[8], b[8];
      unpack8<DT>(v[i], a);
      unpack8<DT>(u[i], b);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = __fadd_rn(a[j], b[j]);
      v[i] = pack8<DT>(a);
      const int c = i * TPR + t;
      if (c < chunks) *reinterpret_cast<uint4*>(sum + 8 * c) = v[i];
    }
  }
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float a[8];
    unpack8<DT>(v[i], a);
#pragma unroll
    for (int j = 0; j < 8; ++j) sq = __fmaf_rn(a[j], a[j], sq);
  }
  sq = row_reduce<TPR>(sq, s_sum, t, Add());
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sq, float(p.H)), p.eps)));
  if (p.rstd && t == 0) p.rstd[row] = rstd;

  auto scaled = [&](int i, float (&y)[8]) {       // the fp32 y of chunk i
    const int c = i * TPR + t;
    float g[8] = {};
    unpack8<DT>(v[i], y);
    if (c < chunks) load8(p.gamma + 8 * c, g);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 z = mul_pair(mul_pair(make_float2(y[j], y[j + 1]), make_float2(rstd, rstd)),
                                make_float2(g[j], g[j + 1]));
      y[j] = z.x;
      y[j + 1] = z.y;
    }
  };
  uint16_t* out = p.out ? static_cast<uint16_t*>(p.out) + row * p.out_stride : nullptr;
  const int padded = static_cast<int>(align_up(p.H, 32)) / 8;     // chunks with the zeros
  if constexpr (CODE == MOE_CODE_I8) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float y[8];
      scaled(i, y);
      if (i * TPR + t < chunks) top = max(top, abs_max_bits(y));
    }
    top = row_reduce<TPR>(top, s_max, t, Max());
    const float scale = __fdiv_rn(127.0f, __fadd_rn(__uint_as_float(top), 1e-12f));
    uint8_t* codes = static_cast<uint8_t*>(p.codes) + row * (padded * 8 + 32);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * TPR + t;
      float y[8];
      scaled(i, y);
      if (out && c < chunks) *reinterpret_cast<uint4*>(out + 8 * c) = pack8<DT>(y);
      if (c < padded)
        *reinterpret_cast<uint2*>(codes + 8 * c) =
            c < chunks ? i8_codes(y, scale) : make_uint2(0u, 0u);
    }
    if (t < 8)
      reinterpret_cast<float*>(codes + padded * 8)[t] = t ? 0.0f : __fdiv_rn(1.0f, scale);
  } else {
    const int nb = code_blocks(p.H);
    uint8_t* codes = nullptr;
    float* scales = nullptr;
    if constexpr (CODE == MOE_CODE_F8) {
      codes = static_cast<uint8_t*>(p.codes) + row * f8_row_bytes(p.H);
      scales = reinterpret_cast<float*>(codes + f8_scales_at(p.H));
      if (t < 8 && nb + t < align_up(nb, 8)) scales[nb + t] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * TPR + t;
      float y[8];
      scaled(i, y);
      if (out && c < chunks) *reinterpret_cast<uint4*>(out + 8 * c) = pack8<DT>(y);
      if constexpr (CODE == MOE_CODE_F8) {
        const F8Scale sc = f8_scale(block_max_bits(c < chunks ? abs_max_bits(y) : 0u));
        if (c < padded)
          *reinterpret_cast<uint2*>(codes + 8 * c) =
              c < chunks ? f8_codes(y, sc.inv) : make_uint2(0u, 0u);
        if (t % 16 == 0 && c < chunks) scales[c / 16] = sc.scale;
      }
    }
  }
}

// ---- gradient --------------------------------------------------------------------

// CTAs walk over rows and keep d_gamma's sums of their columns in registers; their
// partial sums go to the workspace, and a second kernel adds them in order.  Rows (of d_out,
// of x and of d_sum) come by bulk copies into a ring of `depth` rows a team of TPR threads,
// so that the next rows are on their way while one is reduced and written; both passes over
// a row read it from there.  (By loads into registers a CTA waited for every row: 32,768 x
// 7168 440 us.)  Where a wait runs out in any thread its team does not write that row, asks
// for no further one, and leaves once the copies on their way have landed.
constexpr int kMaxDepth = 4;
__host__ __device__ constexpr int backward_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

template <int DT, int TPR, int NV>
__global__ void __launch_bounds__(backward_threads(TPR))
rms_norm_backward_kernel(const NormBackwardArgs p, int depth) {
  constexpr int kRows = backward_threads(TPR) / TPR;
  constexpr bool kKeepGamma = NV < 4;            // in registers
  extern __shared__ __align__(16) uint8_t s_ring[];
  __shared__ __align__(8) uint64_t s_full[kRows][kMaxDepth];
  // a reduction's sums; behind them, read along, 1 where a thread's wait ran out
  constexpr int kGaveUp = TPR / 32;
  __shared__ __align__(16) float s_part[2][kGaveUp + 4];
  wait_for_stream();
  let_next_start();
  const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  const int chunks = p.H / 8;
  const uint32_t row_bytes = 2 * p.H, parts = p.d_sum ? 3 : 2;
  uint8_t* ring = s_ring + size_t(slot) * depth * parts * row_bytes;
  uint64_t* full = s_full[slot];
  if (t == 0) {
    if constexpr (TPR > 32) s_part[0][kGaveUp] = s_part[1][kGaveUp] = 0.0f;
    for (int i = 0; i < depth; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  auto team_sync = [&]() {
    if constexpr (TPR == 32) __syncwarp();
    else __syncthreads();
  };
  const int64_t first = int64_t(blockIdx.x) * kRows + slot, stride = int64_t(gridDim.x) * kRows;
  auto fetch = [&](int64_t row, int at) {          // one thread
    if (row >= p.T) return;
    uint8_t* to = ring + size_t(at) * parts * row_bytes;
    mbar_arrive_expect_tx(&full[at], parts * row_bytes);
    bulk_load(to, static_cast<const uint16_t*>(p.d_out) + row * p.d_out_stride, row_bytes,
              &full[at]);
    bulk_load(to + row_bytes, static_cast<const uint16_t*>(p.x) + row * p.x_stride, row_bytes,
              &full[at]);
    if (p.d_sum)
      bulk_load(to + 2 * row_bytes, static_cast<const uint16_t*>(p.d_sum) + row * p.d_sum_stride,
                row_bytes, &full[at]);
  };
  float acc[NV][8], kept[kKeepGamma ? NV : 1][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * TPR + t;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      acc[i][j] = 0.0f;
      if constexpr (kKeepGamma) kept[i][j] = 0.0f;
    }
    if constexpr (kKeepGamma)
      if (c < chunks) load8(p.gamma + 8 * c, kept[i]);
  }
  auto gamma_of = [&](int i, float (&g)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = kKeepGamma ? kept[kKeepGamma ? i : 0][j] : 0.0f;
    if constexpr (!kKeepGamma) load8(p.gamma + 8 * (i * TPR + t), g);
  };
  team_sync();
  if (t == 0)
    for (int i = 0; i < depth; ++i) fetch(first + i * stride, i);
  int at = 0, turn = 0;
  uint32_t phase = 0;
  bool ok = true;                     // the team's: no wait ran out
  float rstd_next = first < p.T ? p.rstd[first] : 0.0f;
  int64_t row = first;
  for (; row < p.T; row += stride, turn ^= 1) {
    const float rstd = rstd_next;
    if (row + stride < p.T) rstd_next = p.rstd[row + stride];
    ok = row_wait(&full[at], phase);
    if constexpr (TPR == 32) {
      ok = __all_sync(kAll, ok);
    } else if (!ok) {
      s_part[turn][kGaveUp] = 1.0f;    // (the others learn of it behind the next barrier)
    }
    const uint4* dv = reinterpret_cast<const uint4*>(ring + size_t(at) * parts * row_bytes);
    const uint4 *xv = dv + chunks, *sv = xv + chunks;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * TPR + t;
      if (c >= chunks) break;
      float d[8], xh[8], g[8];
      unpack8<DT>(dv[c], d);
      unpack8<DT>(xv[c], xh);
      gamma_of(i, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[j] = __fmul_rn(xh[j], rstd);
        dot = __fmaf_rn(__fmul_rn(d[j], g[j]), xh[j], dot);
        acc[i][j] = __fmaf_rn(d[j], xh[j], acc[i][j]);
      }
    }
    const float mean = __fdiv_rn(row_reduce<TPR>(dot, s_part[turn], t, Add()), float(p.H));
    if constexpr (TPR > 32) ok = s_part[turn][kGaveUp] == 0.0f;
    if (!ok) break;
    // every thread is done with the row before this one: its place is free
    if (TPR == 32) __syncwarp();
    if (t == 0 && row != first) {
      const int prev = at == 0 ? depth - 1 : at - 1;
      fetch(row + (depth - 1) * stride, prev);
    }
    uint16_t* dx = static_cast<uint16_t*>(p.d_x) + row * p.d_x_stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * TPR + t;
      if (c >= chunks) break;
      float d[8], xh[8], s[8] = {}, g[8];
      unpack8<DT>(dv[c], d);
      unpack8<DT>(xv[c], xh);
      if (p.d_sum) unpack8<DT>(sv[c], s);
      gamma_of(i, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[j] = __fmul_rn(xh[j], rstd);
        const float a = __fmul_rn(d[j], g[j]);
        d[j] = __fmaf_rn(__fmaf_rn(-xh[j], mean, a), rstd, s[j]);
      }
      *reinterpret_cast<uint4*>(dx + 8 * c) = pack8<DT>(d);
    }
    if (++at == depth) {
      at = 0;
      phase ^= 1u;
    }
  }
  if (!ok) {
    set_status(p.dev_status, MOE_ERR_TIMEOUT);
    // No copy may land once the CTA has gone: the rows asked for from this one on, one fewer
    // than the ring holds behind the first.
    for (int left = row == first ? depth : depth - 1; left > 0 && row < p.T;
         --left, row += stride) {
      mbar_wait_bounded(&full[at], phase, kGemmSpin);
      if (++at == depth) {
        at = 0;
        phase ^= 1u;
      }
    }
  }
  float* part = p.parts + int64_t(blockIdx.x) * p.H;
  auto put = [&](int c, const float (&f)[8]) {
    if (c >= chunks) return;
    *reinterpret_cast<float4*>(part + 8 * c) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(part + 8 * c + 4) = make_float4(f[4], f[5], f[6], f[7]);
  };
  if constexpr (kRows == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) put(i * TPR + t, acc[i]);
  } else {                       // the CTA's warps first, in order
    constexpr int kCols = TPR * NV * 8;
    float* s_cols = reinterpret_cast<float*>(s_ring);        // the rings are done with
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s_cols[slot * kCols + (i * 8 + j) * TPR + t] = acc[i][j];
    __syncthreads();
    if (slot == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[j] = acc[i][j];
          for (int r = 1; r < kRows; ++r)
            f[j] = __fadd_rn(f[j], s_cols[r * kCols + (i * 8 + j) * TPR + t]);
        }
        put(i * TPR + t, f);
      }
    }
  }
}

constexpr int kSumCols = 32, kSumGroups = 32;

// d_gamma[h] = the partial sums of column h, those of a group in order, then the
// groups in order.
__global__ void __launch_bounds__(kSumCols* kSumGroups)
rms_norm_columns_kernel(const float* parts, int nparts, int H, float* d_gamma) {
  __shared__ float s[kSumGroups][kSumCols];
  wait_for_stream();
  let_next_start();
  const int col = threadIdx.x % kSumCols, grp = threadIdx.x / kSumCols;
  const int h = blockIdx.x * kSumCols + col;
  float v = 0.0f;
  if (h < H)
    for (int i = grp; i < nparts; i += kSumGroups) v = __fadd_rn(v, parts[int64_t(i) * H + h]);
  s[grp][col] = v;
  __syncthreads();
  if (grp == 0 && h < H) {
    for (int i = 1; i < kSumGroups; ++i) v = __fadd_rn(v, s[i][col]);
    d_gamma[h] = v;
  }
}

// ---- rows of more than kMaxWidth values ------------------------------------------------
// One CTA per row that reads it once per pass (from L2 but for the first): no registers
// hold it.

constexpr int kWide = 1024;

template <int DT, int CODE>
__global__ void __launch_bounds__(kWide, 1)
rms_norm_wide_kernel(const NormArgs p) {
  __shared__ float s_sum[32];
  __shared__ uint32_t s_max[32];
  wait_for_stream();
  let_next_start();
  const int t = threadIdx.x, chunks = p.H / 8;
  const int64_t row = blockIdx.x;
  const uint16_t* x = static_cast<const uint16_t*>(p.x) + row * p.x_stride;
  const uint16_t* res =
      p.residual ? static_cast<const uint16_t*>(p.residual) + row * p.residual_stride : nullptr;
  uint16_t* sum = p.residual ? static_cast<uint16_t*>(p.sum) + row * p.sum_stride : nullptr;
  float sq = 0.0f;
  for (int c = t; c < chunks; c += kWide) {
    uint4 v = *reinterpret_cast<const uint4*>(x + 8 * c);
    float a[8];
    unpack8<DT>(v, a);
    if (res) {
      float b[8];
      unpack8<DT>(*reinterpret_cast<const uint4*>(res + 8 * c), b);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = __fadd_rn(a[j], b[j]);
      v = pack8<DT>(a);
      *reinterpret_cast<uint4*>(sum + 8 * c) = v;
      unpack8<DT>(v, a);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sq = __fmaf_rn(a[j], a[j], sq);
  }
  sq = row_reduce<kWide>(sq, s_sum, t, Add());
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sq, float(p.H)), p.eps)));
  if (p.rstd && t == 0) p.rstd[row] = rstd;
  const uint16_t* s = res ? sum : x;          // (a thread reads what it wrote itself)
  auto scaled = [&](int c, float (&y)[8]) {
    float g[8];
    unpack8<DT>(*reinterpret_cast<const uint4*>(s + 8 * c), y);
    load8(p.gamma + 8 * c, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(__fmul_rn(y[j], rstd), g[j]);
  };
  uint16_t* out = p.out ? static_cast<uint16_t*>(p.out) + row * p.out_stride : nullptr;
  const int padded = static_cast<int>(align_up(p.H, 32)) / 8;
  float scale = 0.0f;
  uint8_t* codes = nullptr;
  if constexpr (CODE == MOE_CODE_I8) {
    uint32_t top = 0;
    for (int c = t; c < chunks; c += kWide) {
      float y[8];
      scaled(c, y);
      top = max(top, abs_max_bits(y));
    }
    top = row_reduce<kWide>(top, s_max, t, Max());
    scale = __fdiv_rn(127.0f, __fadd_rn(__uint_as_float(top), 1e-12f));
    codes = static_cast<uint8_t*>(p.codes) + row * (padded * 8 + 32);
    if (t < 8)
      reinterpret_cast<float*>(codes + padded * 8)[t] = t ? 0.0f : __fdiv_rn(1.0f, scale);
  }
  float* scales = nullptr;
  if constexpr (CODE == MOE_CODE_F8) {
    const int nb = code_blocks(p.H);
    codes = static_cast<uint8_t*>(p.codes) + row * f8_row_bytes(p.H);
    scales = reinterpret_cast<float*>(codes + f8_scales_at(p.H));
    if (t < 8 && nb + t < align_up(nb, 8)) scales[nb + t] = 0.0f;
  }
  // (every thread of a warp takes each turn, for the shuffles)
  for (int c0 = 0; c0 < padded; c0 += kWide) {
    const int c = c0 + t;
    const bool in = c < chunks;
    float y[8] = {};
    if (in) scaled(c, y);
    if constexpr (CODE == MOE_CODE_F8) {
      const F8Scale sc = f8_scale(block_max_bits(abs_max_bits(y)));
      if (c < padded)
        *reinterpret_cast<uint2*>(codes + 8 * c) = in ? f8_codes(y, sc.inv) : make_uint2(0u, 0u);
      if (in && t % 16 == 0) scales[c / 16] = sc.scale;
    }
    if constexpr (CODE == MOE_CODE_I8) {
      if (c < padded)
        *reinterpret_cast<uint2*>(codes + 8 * c) = in ? i8_codes(y, scale) : make_uint2(0u, 0u);
    }
    if (in && out) *reinterpret_cast<uint4*>(out + 8 * c) = pack8<DT>(y);
  }
}

// d_x of a row.
template <int DT>
__global__ void __launch_bounds__(kWide, 1)
rms_norm_backward_wide_kernel(const NormBackwardArgs p) {
  __shared__ float s_part[32];
  wait_for_stream();
  let_next_start();
  const int t = threadIdx.x, chunks = p.H / 8;
  const int64_t row = blockIdx.x;
  const uint16_t* dy = static_cast<const uint16_t*>(p.d_out) + row * p.d_out_stride;
  const uint16_t* x = static_cast<const uint16_t*>(p.x) + row * p.x_stride;
  const uint16_t* ds =
      p.d_sum ? static_cast<const uint16_t*>(p.d_sum) + row * p.d_sum_stride : nullptr;
  uint16_t* dx = static_cast<uint16_t*>(p.d_x) + row * p.d_x_stride;
  const float rstd = p.rstd[row];
  float mean = 0.0f;
  for (int pass = 0; pass < 2; ++pass) {
    float dot = 0.0f;
    for (int c = t; c < chunks; c += kWide) {
      float d[8], xh[8], g[8], s[8] = {};
      unpack8<DT>(*reinterpret_cast<const uint4*>(dy + 8 * c), d);
      unpack8<DT>(*reinterpret_cast<const uint4*>(x + 8 * c), xh);
      load8(p.gamma + 8 * c, g);
      if (pass && ds) unpack8<DT>(*reinterpret_cast<const uint4*>(ds + 8 * c), s);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[j] = __fmul_rn(xh[j], rstd);
        const float a = __fmul_rn(d[j], g[j]);
        dot = __fmaf_rn(a, xh[j], dot);
        d[j] = __fmaf_rn(__fmaf_rn(-xh[j], mean, a), rstd, s[j]);
      }
      if (pass) *reinterpret_cast<uint4*>(dx + 8 * c) = pack8<DT>(d);
    }
    if (!pass) mean = __fdiv_rn(row_reduce<kWide>(dot, s_part, t, Add()), float(p.H));
  }
}

// Partial sums of d_gamma: CTA (i, j) takes rows j, j + gridDim.y, ... of kGammaCols columns.
constexpr int kGammaThreads = 128, kGammaCols = kGammaThreads * 8, kGammaParts = 32;

template <int DT>
__global__ void __launch_bounds__(kGammaThreads)
rms_norm_gamma_kernel(const NormBackwardArgs p) {
  wait_for_stream();
  let_next_start();
  const int c = blockIdx.x * kGammaThreads + threadIdx.x;
  if (8 * c >= p.H) return;
  float acc[8] = {};
  for (int64_t row = blockIdx.y; row < p.T; row += gridDim.y) {
    float d[8], xh[8];
    unpack8<DT>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.d_out) +
                                                row * p.d_out_stride + 8 * c), d);
    unpack8<DT>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) +
                                                row * p.x_stride + 8 * c), xh);
    const float rstd = p.rstd[row];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = __fmaf_rn(d[j], __fmul_rn(xh[j], rstd), acc[j]);
  }
  float* part = p.parts + int64_t(blockIdx.y) * p.H + 8 * c;
#pragma unroll
  for (int j = 0; j < 8; ++j) part[j] = acc[j];
}

// Calls f(TPR, NV) with the threads per row and chunks per thread of a row of H.
template <class F>
cudaError_t by_width(int H, F&& f) {
  const int chunks = H / 8;
  using std::integral_constant;
  auto go = [&](auto tpr, auto nv) { return f(tpr, nv); };
  if (chunks <= 64) return go(integral_constant<int, 32>(), integral_constant<int, 2>());
  if (chunks <= 128) return go(integral_constant<int, 32>(), integral_constant<int, 4>());
  if (chunks <= 512) return go(integral_constant<int, 256>(), integral_constant<int, 2>());
  if (chunks <= 1024) return go(integral_constant<int, 512>(), integral_constant<int, 2>());
  return go(integral_constant<int, 512>(), integral_constant<int, 4>());
}
constexpr int kMaxWidth = 512 * 4 * 8;      // wider rows: the kernels that read a row again

// The norm's own: many rows want 64 bytes of loads a thread under way (65,536 rows of 2048:
// 81 us with 4 chunks a thread, 125 with one), few rows many threads each.
template <class F>
cudaError_t by_width_and_rows(int H, int64_t T, F&& f) {
  const int chunks = H / 8;
  using std::integral_constant;
  if (T > 256 && chunks > 128) {
    if (chunks <= 256) return f(integral_constant<int, 64>(), integral_constant<int, 4>());
    if (chunks <= 512) return f(integral_constant<int, 128>(), integral_constant<int, 4>());
    if (chunks <= 1024) return f(integral_constant<int, 256>(), integral_constant<int, 4>());
  }
  return by_width(H, f);
}

template <int DT>
cudaError_t launch_norm(const NormArgs& p, cudaStream_t st) {
  if (p.H > kMaxWidth)
    return !p.codes ? launch_early(rms_norm_wide_kernel<DT, kNoCodes>, p.T, kWide, 0, st, p)
           : p.code_type == MOE_CODE_I8
               ? launch_early(rms_norm_wide_kernel<DT, MOE_CODE_I8>, p.T, kWide, 0, st, p)
               : launch_early(rms_norm_wide_kernel<DT, MOE_CODE_F8>, p.T, kWide, 0, st, p);
  return by_width_and_rows(p.H, p.T, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    constexpr int kBlock = block_threads(TPR), kRows = kBlock / TPR;
    const int64_t grid = (p.T + kRows - 1) / kRows;
    if (!p.codes)
      return launch_early(rms_norm_kernel<DT, TPR, NV, kNoCodes>, grid, kBlock, 0, st, p);
    if (p.code_type == MOE_CODE_I8)
      return launch_early(rms_norm_kernel<DT, TPR, NV, MOE_CODE_I8>, grid, kBlock, 0, st, p);
    return launch_early(rms_norm_kernel<DT, TPR, NV, MOE_CODE_F8>, grid, kBlock, 0, st, p);
  });
}

// CTAs that an SM's shared memory and registers are shared by: two, so that one's
// reductions overlap the other's; rows of which two do not fit twice have an SM alone.
// (32,768 x 7168 with one CTA an SM and twice its ring 326 us, with two 288 to 290.)
template <int TPR, int NV>
constexpr int kCtasPerSm = TPR * NV <= 1024 ? 2 : 1;
template <int TPR, int NV>
constexpr int kRingRoom = 196 * 1024 / kCtasPerSm<TPR, NV>;

constexpr int kMaxParts = 304;          // two CTAs for each of 152 SMs

int backward_parts(int64_t T, int H) {
  if (H > kMaxWidth)
    return static_cast<int>(std::min<int64_t>(kGammaParts, std::max<int64_t>(1, T)));
  int rows = 1, most = kMaxParts;
  by_width(H, [&](auto tpr, auto nv) {
    rows = backward_threads(decltype(tpr)::value) / decltype(tpr)::value;
    most = kMaxParts / 2 * kCtasPerSm<decltype(tpr)::value, decltype(nv)::value>;
    return cudaSuccess;
  });
  return static_cast<int>(std::min<int64_t>(most, std::max<int64_t>(1, (T + rows - 1) / rows)));
}

// The ring's rows: as many as fit.
template <int TPR, int NV>
int ring_depth(const NormBackwardArgs& p, size_t* smem) {
  constexpr int kTeams = backward_threads(TPR) / TPR;
  const size_t row = size_t(kTeams) * 2 * p.H * (p.d_sum ? 3 : 2);
  int depth = kMaxDepth;
  while (depth > 2 && row * depth > size_t(kRingRoom<TPR, NV>)) --depth;
  *smem = std::max(row * depth, kTeams > 1 ? sizeof(float) * kTeams * TPR * NV * 8 : size_t(0));
  return depth;
}

template <int DT>
cudaError_t launch_backward(const NormBackwardArgs& p, int parts, cudaStream_t st) {
  if (p.H > kMaxWidth) {          // d_gamma first: d_x may lie where the inputs do
    const int cols = (p.H + kGammaCols - 1) / kGammaCols;
    const cudaError_t e = launch_early(rms_norm_gamma_kernel<DT>, dim3(cols, parts), kGammaThreads,
                                       0, st, p);
    if (e != cudaSuccess) return e;
    return launch_early(rms_norm_backward_wide_kernel<DT>, p.T, kWide, 0, st, p);
  }
  return by_width(p.H, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    size_t smem = 0;
    const int depth = ring_depth<TPR, NV>(p, &smem);
    auto kernel = rms_norm_backward_kernel<DT, TPR, NV>;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
    return launch_early(kernel, parts, backward_threads(TPR), smem, st, p, depth);
  });
}

}  // namespace

#ifndef MOE_RMS_NORM_POLLS
cudaError_t launch_rms_norm(const NormArgs& p, cudaStream_t st) {
  return p.dtype == MOE_BF16 ? launch_norm<MOE_BF16>(p, st) : launch_norm<MOE_FP16>(p, st);
}

size_t rms_norm_backward_workspace_bytes(int64_t T, int H) {
  return size_t(backward_parts(T, H)) * H * sizeof(float);
}

cudaError_t launch_rms_norm_backward(const NormBackwardArgs& p, float* d_gamma,
                                     cudaStream_t st) {
  const int parts = backward_parts(p.T, p.H);
  const cudaError_t e = p.dtype == MOE_BF16 ? launch_backward<MOE_BF16>(p, parts, st)
                                            : launch_backward<MOE_FP16>(p, parts, st);
  if (e != cudaSuccess) return e;
  return launch_early(rms_norm_columns_kernel, (p.H + kSumCols - 1) / kSumCols,
                      kSumCols * kSumGroups, 0, st, p.parts, parts, p.H, d_gamma);
}
#endif

}  // namespace moe_ep

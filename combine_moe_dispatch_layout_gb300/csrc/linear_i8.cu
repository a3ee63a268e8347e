// linear_i8.cu -- matrix product of 8-bit codes with a scale per row and per
// output column, rows grouped by expert (include/moe_ep.h, moe_linear_i8).
//
// Mathematics.  acc[m][n] = sum_j a[m][j] w[g][n][j] in int32 (K <= 65536, so
// |acc| <= 2^30: exact), then c = ((fp32(acc) * col) * row) + bias, one
// rounding each, then one rounding to the output type.
//
// 64 x 64 output tile per CTA, K in steps of 64 bytes through shared memory,
// four-way integer dot products.
#include <algorithm>

#include "moe_ep_internal.cuh"

namespace moe_ep {
namespace {

constexpr int BM = 64, BN = 64, BK = 64, kThreads = 256;

// 16 bytes at column j of a row of K codes; zeros past K.
__device__ __forceinline__ uint4 load_codes(const uint8_t* row, int j, int K) {
  if (j + 16 <= K) return __ldg(reinterpret_cast<const uint4*>(row + j));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (j + i < K) w[i >> 2] |= uint32_t(__ldg(row + j + i)) << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(kThreads)
linear_i8_kernel(const LinearArgs p, int32_t* dev_status) {
  __shared__ uint32_t sa[BM][BK / 4 + 1], sw[BN][BK / 4 + 1];
  __shared__ int64_t s_row0, s_rows;
  __shared__ int s_g, s_n0;
  const int tid = threadIdx.x;
  if (tid == 0) {
    const int64_t ntn = (p.N + BN - 1) / BN;
    int64_t t = blockIdx.x, off = 0;
    s_g = -1;
    for (int g = 0; g < p.G; ++g) {
      int64_t n = p.group_rows ? __ldg(p.group_rows + g) : p.a_rows;
      if (n < 0) {
        set_status(dev_status, MOE_ERR_INVALID_ARG);
        n = 0;
      }
      const int64_t tiles = (n + BM - 1) / BM * ntn;
      if (s_g < 0 && t < tiles) {
        s_g = g;
        s_row0 = off + t / ntn * BM;
        s_rows = min(int64_t(BM), n - t / ntn * BM);
        s_n0 = static_cast<int>(t % ntn) * BN;
      }
      t -= tiles;
      off += n;
    }
    if (off > p.a_rows) {
      set_status(dev_status, MOE_ERR_CAPACITY);
      s_g = -1;
    }
  }
  __syncthreads();
  const int g = s_g;
  if (g < 0) return;
  const int64_t row0 = s_row0;
  const int rows = static_cast<int>(s_rows), n0 = s_n0;
  const uint8_t* a = static_cast<const uint8_t*>(p.a) + row0 * p.a_stride;
  const uint8_t* w = static_cast<const uint8_t*>(p.w) + (int64_t(g) * p.N + n0) * p.w_stride;
  const int lr = tid >> 2, lc = (tid & 3) * 16;      // this thread's 16 bytes of a tile
  const int ty = tid >> 4, tx = tid & 15;
  int acc[4][4] = {};
  for (int j = 0; j < p.K; j += BK) {
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    const uint4 va = lr < rows && j + lc < p.K ? load_codes(a + lr * p.a_stride, j + lc, p.K) : z;
    const uint4 vw = n0 + lr < p.N && j + lc < p.K
                         ? load_codes(w + lr * p.w_stride, j + lc, p.K) : z;
    __syncthreads();
    const uint32_t ua[4] = {va.x, va.y, va.z, va.w}, uw[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sa[lr][lc / 4 + i] = ua[i];
      sw[lr][lc / 4 + i] = uw[i];
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < BK / 4; ++c)
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          acc[y][x] = __dp4a(static_cast<int>(sa[ty + 16 * y][c]),
                             static_cast<int>(sw[tx + 16 * x][c]), acc[y][x]);
  }
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const int r = ty + 16 * y;
    if (r >= rows) continue;
    const int64_t m = row0 + r;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int n = n0 + tx + 16 * x;
      if (n >= p.N) continue;
      const int64_t at = m * p.N + n, gn = int64_t(g) * p.N + n;
      if (p.c_dtype == MOE_INT32) {
        static_cast<int32_t*>(p.c)[at] = acc[y][x];
        continue;
      }
      const float ts = __ldg(reinterpret_cast<const float*>(p.row_scale + m * p.row_scale_stride));
      float v = __fmul_rn(__fmul_rn(__int2float_rn(acc[y][x]), __ldg(p.col_scale + gn)), ts);
      if (p.bias) v = __fadd_rn(v, __ldg(p.bias + gn));
      if (p.c_dtype == MOE_FP32) static_cast<float*>(p.c)[at] = v;
      else
        static_cast<uint16_t*>(p.c)[at] = static_cast<uint16_t>(
            p.c_dtype == MOE_BF16 ? narrow_rn<MOE_BF16>(v) : narrow_rn<MOE_FP16>(v));
    }
  }
}

}  // namespace

cudaError_t launch_linear_i8(const LinearArgs& p, int32_t* dev_status, cudaStream_t st) {
  const int64_t ntn = (p.N + BN - 1) / BN;
  const int64_t tiles = (p.a_rows / BM + p.G) * ntn;   // at least the groups' tiles
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  linear_i8_kernel<<<static_cast<unsigned>(tiles), kThreads, 0, st>>>(p, dev_status);
  return cudaGetLastError();
}

}  // namespace moe_ep

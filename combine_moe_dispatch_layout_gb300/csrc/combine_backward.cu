// combine_backward.cu -- gradient of the combine (include/moe_ep.h,
// moe_combine_backward).
//
// Mathematics.  out[g] = sum_k w[g][k] y[row(g,k)], so the gradient of row
// (g, k) is w[g][k] d_out[g] and that of the weight is <d_out[g], y[row]>.
// Both take one pass: each expert row is read once and its gradient row
// written once, P*H elements each way, and d_out[g] stays in registers for
// the token's k rows.  Memory-bound: (T + 2P) rows of 2H bytes.
//
// Rows of more than 1024 elements: a persistent grid walks the tokens.  The last
// warp resolves the next token's rows and weights into the other half of a
// double-buffered table while the compute warps work on this one; each compute
// thread owns two 16-byte chunks of the hidden dimension, issues the loads of
// kBatch rows before using them, writes the gradient rows and adds up its part
// of the k dot products.  Dot products go over a warp by shuffles and over the
// CTA through shared memory, warps in ascending order: a fixed order.
//
// Measured (32,768 tokens, k = 8, H = 7168, bf16: 8.0 GB): 1211 us, 6.6 TB/s,
// 97% of a copy's rate, which is what bounds it.  Batches of 8 rows leave one CTA
// per SM: 17% slower; four chunks per thread: 25%; the next token's rows
// prefetched into L2 (which helps the combine, where nothing is written): 20%;
// write-back instead of streaming stores: 1%.
//
// Shorter rows: one warp per token (below).
#include <algorithm>

#include "moe_ep_internal.cuh"

namespace moe_ep {
namespace {

constexpr int kBatch = 4;          // rows loaded before they are used
constexpr int kMaxThreads = 512;
constexpr int kTokenWarps = 4;     // of the kernel for short rows
constexpr unsigned kAll = 0xffffffffu;

template <int DT>
__global__ void __launch_bounds__(kMaxThreads, 2)
combine_backward_kernel(const uint4* d_out, const uint4* y, int64_t y_rows,
                        const int32_t* topk_idx, const float* weights, const int32_t* send_idx,
                        const int32_t* put_offset, const int64_t* rank_recv_base, int R, int bs,
                        int k, int epr, int H, int64_t T, uint4* d_y, float* d_weights,
                        int32_t* dev_status) {
  __shared__ int64_t s_rows[2][MOE_EP_MAX_TOPK];
  __shared__ float s_w[2][MOE_EP_MAX_TOPK];
  __shared__ float s_dot[2][kMaxThreads / 32][MOE_EP_MAX_TOPK];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ncomp = blockDim.x - 32, nwarps = ncomp >> 5;
  const bool producer = tid >= ncomp;
  const int nch = H / 8;

  wait_for_stream();
  let_next_start();
  int64_t g = blockIdx.x;
  if (producer)
    resolve_token<true>(g, topk_idx, weights, send_idx, put_offset, rank_recv_base, R, bs, k, epr,
                        y_rows, s_rows[0], s_w[0], dev_status, lane);
  __syncthreads();

  for (int it = 0; g < T; ++it, g += gridDim.x) {
    const int buf = it & 1;
    if (producer) {
      const int64_t gn = g + gridDim.x;
      if (gn < T)
        resolve_token<true>(gn, topk_idx, weights, send_idx, put_offset, rank_recv_base, R, bs, k,
                            epr, y_rows, s_rows[buf ^ 1], s_w[buf ^ 1], dev_status, lane);
    } else {
      for (int k0 = 0; k0 < k; k0 += kBatch) {
        float dot[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) dot[b] = 0.0f;
        for (int c = tid; c < nch; c += ncomp) {
          uint4 v[kBatch];
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int64_t row = k0 + b < k ? s_rows[buf][k0 + b] : -1;
            v[b] = row >= 0 ? ld_once_16(y + row * nch + c) : make_uint4(0u, 0u, 0u, 0u);
          }
          float d[8];
          unpack8<DT>(d_out[g * nch + c], d);
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int64_t row = k0 + b < k ? s_rows[buf][k0 + b] : -1;
            if (row >= 0) {
              const float w = s_w[buf][k0 + b];
              float f[8], o[8];
              unpack8<DT>(v[b], f);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                dot[b] = __fmaf_rn(d[j], f[j], dot[b]);
                o[j] = __fmul_rn(w, d[j]);
              }
              __stcs(d_y + row * nch + c, pack8<DT>(o));   // written once, read by a later kernel
            }
          }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
#pragma unroll
          for (int s = 16; s; s >>= 1)
            dot[b] = __fadd_rn(dot[b], __shfl_xor_sync(kAll, dot[b], s));
          if (lane == 0 && k0 + b < k) s_dot[buf][warp][k0 + b] = dot[b];
        }
      }
    }
    __syncthreads();   // dots are in; this token's table is free, the next is ready
    // (the next token's dots go to the other half: no second barrier)
    if (tid < k) {
      float sum = 0.0f;
      for (int w = 0; w < nwarps; ++w) sum = __fadd_rn(sum, s_dot[buf][w][tid]);
      d_weights[g * k + tid] = sum;
    }
  }
}

// Rows of up to 32 * CH chunks (H <= 1024): one warp per token, its row of d_out in
// registers, kRows rows loaded before they are used; no CTA-wide barrier per token.
// Against the kernel above: 65,536 x 6 x 512 133 us instead of 190, 32,768 x 6 x 256
// 35 instead of 56, 4096 x 8 x 1024 20 instead of 24.  At H = 2048 the two meet (343 and
// 348 us at 32,768 tokens) and few tokens are slower (9.0 and 5.4 us at 128): it
// stays with the kernel above, which puts a whole CTA's threads on a token.  CH = 4
// with 2 rows at a time took 22 us, CH = 1 with 16 45.  Rows of less than 256 elements
// leave lanes without a chunk: 131,072 x 6 x 64 takes 101 us, x 128 112, 65,536 x 6 x 256 72.
template <int DT, int CH>
__global__ void __launch_bounds__(kTokenWarps * 32)
combine_backward_warp_kernel(const uint4* d_out, const uint4* y, int64_t y_rows,
                             const int32_t* topk_idx, const float* weights, const int32_t* send_idx,
                             const int32_t* put_offset, const int64_t* rank_recv_base, int R, int bs,
                             int k, int epr, int H, int64_t T, uint4* d_y, float* d_weights,
                             int32_t* dev_status) {
  constexpr int kRows = CH == 1 ? 8 : 4;
  __shared__ int64_t s_rows[kTokenWarps][MOE_EP_MAX_TOPK];
  __shared__ float s_w[kTokenWarps][MOE_EP_MAX_TOPK];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nch = H / 8;
  const int64_t g = int64_t(blockIdx.x) * kTokenWarps + warp;
  wait_for_stream();
  let_next_start();
  if (g >= T) return;
  uint4 q[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c)
    q[c] = lane + 32 * c < nch ? d_out[g * nch + lane + 32 * c] : make_uint4(0u, 0u, 0u, 0u);
  resolve_token<true>(g, topk_idx, weights, send_idx, put_offset, rank_recv_base, R, bs, k, epr,
                      y_rows, s_rows[warp], s_w[warp], dev_status, lane);
  __syncwarp();
  for (int k0 = 0; k0 < k; k0 += kRows) {
    uint4 v[kRows][CH];
#pragma unroll
    for (int b = 0; b < kRows; ++b) {
      const int64_t row = k0 + b < k ? s_rows[warp][k0 + b] : -1;
#pragma unroll
      for (int c = 0; c < CH; ++c)
        v[b][c] = row >= 0 && lane + 32 * c < nch ? ld_once_16(y + row * nch + lane + 32 * c)
                                                  : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int b = 0; b < kRows; ++b) {
      if (k0 + b >= k) break;
      const int64_t row = s_rows[warp][k0 + b];
      const float w = s_w[warp][k0 + b];
      float dot = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (row < 0 || lane + 32 * c >= nch) continue;
        float d[8], f[8], o[8];
        unpack8<DT>(q[c], d);
        unpack8<DT>(v[b][c], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dot = __fmaf_rn(d[j], f[j], dot);
          o[j] = __fmul_rn(w, d[j]);
        }
        __stcs(d_y + row * nch + lane + 32 * c, pack8<DT>(o));
      }
#pragma unroll
      for (int s = 16; s; s >>= 1) dot = __fadd_rn(dot, __shfl_xor_sync(kAll, dot, s));
      if (lane == 0) d_weights[g * k + k0 + b] = dot;
    }
  }
}

template <int DT>
cudaError_t launch_t(const Shape& s, const void* d_out, const void* y, int64_t y_rows,
                     const int32_t* topk_idx, const float* weights, const int32_t* send_idx,
                     const int32_t* put_offset, const int64_t* rank_recv_base, void* d_y,
                     float* d_weights, int32_t* dev_status, cudaStream_t st) {
  const int nch = s.H / 8;
  auto by_warps = [&](auto kernel) {
    return launch_early(kernel, (s.T() + kTokenWarps - 1) / kTokenWarps, kTokenWarps * 32, 0, st,
                        static_cast<const uint4*>(d_out), static_cast<const uint4*>(y), y_rows,
                        topk_idx, weights, send_idx, put_offset, rank_recv_base, s.R, s.bs, s.k,
                        s.epr, s.H, s.T(), static_cast<uint4*>(d_y), d_weights, dev_status);
  };
  // (H alone decides, so a sum's order depends on nothing else)
  if (nch <= 32) return by_warps(combine_backward_warp_kernel<DT, 1>);
  if (nch <= 64) return by_warps(combine_backward_warp_kernel<DT, 2>);
  if (nch <= 128) return by_warps(combine_backward_warp_kernel<DT, 4>);
  // two 16-byte chunks per compute thread; thread j finishes slot j's dot product
  int threads = std::max((nch + 1) / 2, s.k);
  threads = std::min(kMaxThreads - 32, (threads + 31) / 32 * 32) + 32;
  auto kernel = combine_backward_kernel<DT>;
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e == cudaSuccess)
    e = kernel_blocks_per_sm(reinterpret_cast<const void*>(kernel), threads, 0, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t grid = std::min<int64_t>(s.T(), int64_t(std::max(1, per_sm)) * sms);
  return launch_early(kernel, grid, threads, 0, st, static_cast<const uint4*>(d_out),
                      static_cast<const uint4*>(y), y_rows, topk_idx, weights, send_idx,
                      put_offset, rank_recv_base, s.R, s.bs, s.k, s.epr, s.H, s.T(),
                      static_cast<uint4*>(d_y), d_weights, dev_status);
}

}  // namespace

cudaError_t launch_combine_backward(const Shape& s, const void* d_out, const void* y,
                                    int64_t y_rows, const int32_t* topk_idx,
                                    const float* weights, const int32_t* send_idx,
                                    const int32_t* put_offset, const int64_t* rank_recv_base,
                                    void* d_y, float* d_weights, int32_t* dev_status,
                                    cudaStream_t st) {
  if (s.dtype == MOE_BF16)
    return launch_t<MOE_BF16>(s, d_out, y, y_rows, topk_idx, weights, send_idx, put_offset,
                              rank_recv_base, d_y, d_weights, dev_status, st);
  return launch_t<MOE_FP16>(s, d_out, y, y_rows, topk_idx, weights, send_idx, put_offset,
                            rank_recv_base, d_y, d_weights, dev_status, st);
}

}  // namespace moe_ep

// route_backward.cu -- gradient of the gate weights -> gradient of the logits
// (include/moe_ep.h, moe_route_backward).
//
// Mathematics.  With s the scores of the chosen experts, w = s / sum s and
// g = d_weights * scale, the chain rule gives, before the score function,
// ds_j = (g_j - sum_i w_i g_i) / sum s (renormalised) or ds_j = g_j; a sigmoid
// multiplies by s_j (1 - s_j), a softmax takes p_e (ds_e - sum_j p_j ds_j).
// Renormalised softmax weights are a softmax over the chosen logits alone:
// the second sum is then zero, and so is the gradient of every other expert.
// So only plain softmax needs the whole row of logits; every other form reads
// k of them, and the cost is the write of d_logits (mostly zeros).
//
// One warp per token: lane j works out the value of slot j (and j + 32); the
// row is written in 16-byte pieces (zeros, or -p_e * sum), and after a warp
// barrier, which orders the warp's own stores, the k chosen elements are
// stored over it, while the row's lines are still in L2.
#include <algorithm>

#include "moe_ep_internal.cuh"

namespace moe_ep {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kMaxF = 3.402823466e38f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kWarps = 8;   // tokens per CTA at a time

template <int DT>
struct Elem { using T = uint16_t; };
template <>
struct Elem<MOE_FP32> { using T = float; };

template <int DT>
__device__ __forceinline__ float load_logit(const typename Elem<DT>::T* p) {
  float l;
  if constexpr (DT == MOE_FP32) l = __ldg(p);
  else l = widen<DT>(__ldg(p));
  return l != l ? kNegInf : fminf(l, kMaxF);
}
template <int DT>
__device__ __forceinline__ typename Elem<DT>::T to_elem(float f) {
  if constexpr (DT == MOE_FP32) return f;
  else return static_cast<uint16_t>(narrow_rn<DT>(f));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kAll, v, d));
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}

// DENSE: plain softmax.  vec: rows of logits are 16-byte aligned and E is a
// multiple of a 16-byte piece (rows of d_logits then are aligned too).
template <int DT, bool DENSE>
__global__ void __launch_bounds__(kWarps * 32)
route_backward_kernel(const RouteArgs r, bool vec, const int32_t* __restrict__ idx,
                      const float* __restrict__ d_weights,
                      typename Elem<DT>::T* __restrict__ d_logits, int32_t* dev_status) {
  using T = typename Elem<DT>::T;
  constexpr int kPer16 = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  for (int64_t t = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); t < r.T;
       t += int64_t(gridDim.x) * kWarps) {
    const T* row = static_cast<const T*>(r.logits) + t * r.stride;
    T* out = d_logits + t * r.E;

    // ---- the chosen slots: id, logit, incoming gradient -------------------------
    int e[2];
    float l[2], g[2], s[2], v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = lane + 32 * h;
      e[h] = j < r.k ? __ldg(idx + t * r.k + j) : -1;
      if (e[h] < -1 || e[h] >= r.E) {
        set_status(dev_status, MOE_ERR_EXPERT_ID);
        e[h] = -1;
      }
      l[h] = e[h] >= 0 ? load_logit<DT>(row + e[h]) : kNegInf;
      g[h] = e[h] >= 0 ? __fmul_rn(__ldg(d_weights + t * r.k + j), r.scale) : 0.0f;
    }

    // ---- scores ------------------------------------------------------------------
    float m = 0.0f, inv_sum = 1.0f;
    if (DENSE) {
      m = kNegInf;
      if (vec) {
        for (int c = lane; c < r.E / kPer16; c += 32) {
          const uint4 q = __ldg(reinterpret_cast<const uint4*>(row) + c);
          const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (DT == MOE_FP32) {
              m = fmaxf(m, __uint_as_float(w[i]));
            } else {
              m = fmaxf(m, fmaxf(widen<DT>(w[i] & 0xffffu), widen<DT>(w[i] >> 16)));
            }
          }
        }
      } else {
        for (int i = lane; i < r.E; i += 32) m = fmaxf(m, load_logit<DT>(row + i));
      }
      m = fmaxf(fminf(warp_max(m), kMaxF), -kMaxF);
      float sum = 0.0f;
      for (int i = lane; i < r.E; i += 32)
        sum = __fadd_rn(sum, expf(__fsub_rn(load_logit<DT>(row + i), m)));
      sum = warp_sum(sum);
      inv_sum = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
    } else if (r.score == MOE_SOFTMAX) {
      m = fmaxf(warp_max(fmaxf(l[0], l[1])), -kMaxF);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (e[h] < 0) s[h] = 0.0f;
      else if (r.score == MOE_SOFTMAX) s[h] = __fmul_rn(expf(__fsub_rn(l[h], m)), inv_sum);
      else s[h] = __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-l[h])));
    }

    // ---- the slots' gradients ------------------------------------------------------
    float back = 0.0f;                 // what every expert loses (plain softmax)
    if (r.renormalise) {
      const float d = warp_sum(__fadd_rn(s[0], s[1]));
      const float inv = d > 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
      const float w0 = __fmul_rn(s[0], inv), w1 = __fmul_rn(s[1], inv);
      const float mean = warp_sum(__fadd_rn(__fmul_rn(w0, g[0]), __fmul_rn(w1, g[1])));
      v[0] = __fmul_rn(w0, __fsub_rn(g[0], mean));
      v[1] = __fmul_rn(w1, __fsub_rn(g[1], mean));
    } else {
      v[0] = __fmul_rn(s[0], g[0]);
      v[1] = __fmul_rn(s[1], g[1]);
      if (DENSE) back = warp_sum(__fadd_rn(v[0], v[1]));
    }
    if (r.score == MOE_SIGMOID) {
#pragma unroll
      for (int h = 0; h < 2; ++h)      // 1 - s as the sigmoid of -l: no cancellation
        v[h] = e[h] >= 0 ? __fmul_rn(v[h], __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(l[h])))) : 0.0f;
    }
    // a repeated id gets the sum of its slots, in slot order, from its first
    bool first[2] = {e[0] >= 0, e[1] >= 0};
    float total[2] = {0.0f, 0.0f};
    for (int j = 0; j < r.k; ++j) {
      const int ej = __shfl_sync(kAll, j < 32 ? e[0] : e[1], j & 31);
      const float vj = __shfl_sync(kAll, j < 32 ? v[0] : v[1], j & 31);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (ej == e[h]) {
          total[h] = __fadd_rn(total[h], vj);
          if (j < lane + 32 * h) first[h] = false;
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (DENSE) total[h] = __fsub_rn(total[h], __fmul_rn(s[h], back));

    // ---- the row ---------------------------------------------------------------------
    if (vec) {
      for (int c = lane; c < r.E / kPer16; c += 32) {
        uint4 o = make_uint4(0u, 0u, 0u, 0u);
        if (DENSE) {
          const uint4 q = __ldg(reinterpret_cast<const uint4*>(row) + c);
          if constexpr (DT == MOE_FP32) {
            const float x[4] = {__uint_as_float(q.x), __uint_as_float(q.y),
                                __uint_as_float(q.z), __uint_as_float(q.w)};
            float y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float li = x[i] != x[i] ? kNegInf : fminf(x[i], kMaxF);
              y[i] = -__fmul_rn(__fmul_rn(expf(__fsub_rn(li, m)), inv_sum), back);
            }
            o = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]),
                           __float_as_uint(y[2]), __float_as_uint(y[3]));
          } else {
            float x[8];
            unpack8<DT>(q, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float li = x[i] != x[i] ? kNegInf : fminf(x[i], kMaxF);
              x[i] = -__fmul_rn(__fmul_rn(expf(__fsub_rn(li, m)), inv_sum), back);
            }
            o = pack8<DT>(x);
          }
        }
        reinterpret_cast<uint4*>(out)[c] = o;
      }
    } else {
      for (int i = lane; i < r.E; i += 32)
        out[i] = to_elem<DT>(
            DENSE ? -__fmul_rn(__fmul_rn(expf(__fsub_rn(load_logit<DT>(row + i), m)), inv_sum),
                               back)
                  : 0.0f);
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (first[h]) out[e[h]] = to_elem<DT>(total[h]);
  }
}

template <int DT, bool DENSE>
cudaError_t launch_t(const RouteArgs& r, const int32_t* idx, const float* d_weights,
                     void* d_logits, int32_t* dev_status, cudaStream_t st) {
  using T = typename Elem<DT>::T;
  const bool vec = reinterpret_cast<uintptr_t>(r.logits) % 16 == 0 &&
                   r.stride * sizeof(T) % 16 == 0 && r.E * sizeof(T) % 16 == 0;
  auto kernel = route_backward_kernel<DT, DENSE>;
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e == cudaSuccess)
    e = kernel_blocks_per_sm(reinterpret_cast<const void*>(kernel), kWarps * 32, 0, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t grid =
      std::min<int64_t>((r.T + kWarps - 1) / kWarps, int64_t(std::max(1, per_sm)) * sms);
  kernel<<<static_cast<unsigned>(grid), kWarps * 32, 0, st>>>(
      r, vec, idx, d_weights, static_cast<T*>(d_logits), dev_status);
  return cudaGetLastError();
}

template <int DT>
cudaError_t launch_dt(const RouteArgs& r, const int32_t* idx, const float* d_weights,
                      void* d_logits, int32_t* dev_status, cudaStream_t st) {
  if (r.score == MOE_SOFTMAX && !r.renormalise)
    return launch_t<DT, true>(r, idx, d_weights, d_logits, dev_status, st);
  return launch_t<DT, false>(r, idx, d_weights, d_logits, dev_status, st);
}

}  // namespace

cudaError_t launch_route_backward(const RouteArgs& r, const int32_t* topk_idx,
                                  const float* d_weights, void* d_logits,
                                  int32_t* dev_status, cudaStream_t st) {
  switch (r.dtype) {
    case MOE_BF16:
      return launch_dt<MOE_BF16>(r, topk_idx, d_weights, d_logits, dev_status, st);
    case MOE_FP16:
      return launch_dt<MOE_FP16>(r, topk_idx, d_weights, d_logits, dev_status, st);
    default:
      return launch_dt<MOE_FP32>(r, topk_idx, d_weights, d_logits, dev_status, st);
  }
}

}  // namespace moe_ep

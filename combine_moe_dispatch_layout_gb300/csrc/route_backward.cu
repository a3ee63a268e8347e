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
// stored over it, while the row's lines are still in L2.  Plain softmax keeps
// the row's exponentials in registers between its two sums and the write.
#include <algorithm>
#include <type_traits>

#include "moe_ep_internal.cuh"
#include "route_math.cuh"

namespace moe_ep {
namespace {

constexpr int kWarps = 8;   // tokens per CTA at a time

// A logit as moe_route reads it: NaN as -inf, +inf as the largest finite number.
template <int DT>
__device__ __forceinline__ float clean_logit(const typename Elem<DT>::T* p) {
  const float l = load_logit<DT>(p);
  return l != l ? kNegInf : fminf(l, kMaxF);
}
template <int DT>
__device__ __forceinline__ typename Elem<DT>::T to_elem(float f) {
  if constexpr (DT == MOE_FP32) return f;
  else return static_cast<uint16_t>(narrow_rn<DT>(f));
}

// CHUNKS: 16-byte pieces of a row per lane, kept in registers (plain softmax, rows
// of logits 16-byte aligned, E a whole number of pieces); 0: any E and alignment,
// element by element where plain softmax needs the row.  DENSE: plain softmax.
// H: slots per lane (1 for k <= 32, else 2).  vec: 16-byte stores.
template <int DT, bool DENSE, int CHUNKS, int H>
__global__ void __launch_bounds__(kWarps * 32)
route_backward_kernel(const RouteArgs r, bool vec, const int32_t* __restrict__ idx,
                      const float* __restrict__ d_weights,
                      typename Elem<DT>::T* __restrict__ d_logits, float nz,
                      int32_t* dev_status) {
  using T = typename Elem<DT>::T;
  constexpr int kPer16 = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  for (int64_t t = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); t < r.T;
       t += int64_t(gridDim.x) * kWarps) {
    const T* row = static_cast<const T*>(r.logits) + t * r.stride;
    T* out = d_logits + t * r.E;

    // ---- the chosen slots: id, logit, incoming gradient -------------------------
    int e[H];
    float l[H], g[H], s[H], v[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int j = lane + 32 * h;
      e[h] = j < r.k ? __ldg(idx + t * r.k + j) : -1;
      g[h] = j < r.k ? __fmul_rn(__ldg(d_weights + t * r.k + j), r.scale) : 0.0f;
      if (e[h] < -1 || e[h] >= r.E) {
        set_status(dev_status, MOE_ERR_EXPERT_ID);
        e[h] = -1;
      }
      l[h] = e[h] >= 0 ? clean_logit<DT>(row + e[h]) : kNegInf;
      if (e[h] < 0) g[h] = 0.0f;
    }

    // ---- scores ------------------------------------------------------------------
    float m = 0.0f, inv_sum = 1.0f;
    constexpr int kVals = CHUNKS > 0 ? CHUNKS * kPer16 : 2;
    float x[kVals];                    // the lane's logits, then their exponentials
    if (DENSE && CHUNKS > 0) {
      const int pieces = r.E / kPer16;
      float probe = 0.0f;
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        const int at = lane + 32 * c;
        const uint4 q = at < pieces ? __ldg(reinterpret_cast<const uint4*>(row) + at)
                                    : make_uint4(0u, 0u, 0u, 0u);
        float* xc = x + c * kPer16;
        unpack_logits<DT>(q, xc);
#pragma unroll
        for (int i = 0; i < kPer16; ++i) probe = __fmaf_rn(xc[i], 0.0f, probe);
      }
      if (__any_sync(kAll, probe != probe)) {      // infinities and NaN, as moe_route
#pragma unroll
        for (int i = 0; i < kVals; ++i) x[i] = x[i] != x[i] ? kNegInf : fminf(x[i], kMaxF);
      }
      m = kNegInf;
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c)
        if (lane + 32 * c < pieces) {
#pragma unroll
          for (int i = 0; i < kPer16; ++i) m = fmaxf(m, x[c * kPer16 + i]);
        }
      m = fmaxf(warp_max(m), -kMaxF);
      float2 sum2 = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c)
        if (lane + 32 * c < pieces) {
#pragma unroll
          for (int i = 0; i < kPer16; i += 2) {
            float* p = x + c * kPer16 + i;
            const float2 ex = exp_neg2(add2_rn(make_float2(p[0], p[1]), bcast2(-m)), nz);
            p[0] = ex.x;
            p[1] = ex.y;
            sum2 = add2_rn(sum2, ex);
          }
        }
      const float sum = warp_sum(__fadd_rn(sum2.x, sum2.y));
      inv_sum = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
    } else if (DENSE) {
      m = kNegInf;
      for (int i = lane; i < r.E; i += 32) m = fmaxf(m, clean_logit<DT>(row + i));
      m = fmaxf(warp_max(m), -kMaxF);
      float sum = 0.0f;
      for (int i = lane; i < r.E; i += 32)
        sum = __fadd_rn(sum, expf(__fsub_rn(clean_logit<DT>(row + i), m)));
      sum = warp_sum(sum);
      inv_sum = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
    } else if (r.score == MOE_SOFTMAX) {
      m = fmaxf(warp_max(H > 1 ? fmaxf(l[0], l[H - 1]) : l[0]), -kMaxF);
    }
    float rest[H];                     // 1 - s of a sigmoid (of -l: no cancellation)
#pragma unroll
    for (int h = 0; h < H; ++h) {
      rest[h] = 1.0f;
      if (r.score == MOE_SOFTMAX) {
        s[h] = e[h] >= 0 ? __fmul_rn(expf(__fsub_rn(l[h], m)), inv_sum) : 0.0f;
      } else {                         // e^-|l| serves both sides
        const float ex = expf(-fabsf(l[h])), inv = __fdiv_rn(1.0f, __fadd_rn(1.0f, ex));
        const float small = __fmul_rn(ex, inv);
        s[h] = e[h] < 0 ? 0.0f : l[h] >= 0.0f ? inv : small;
        rest[h] = l[h] >= 0.0f ? small : inv;
      }
    }

    // ---- the slots' gradients ------------------------------------------------------
    float back = 0.0f;                 // what every expert loses (plain softmax)
    if (r.renormalise) {
      const float d = warp_sum(H > 1 ? __fadd_rn(s[0], s[H - 1]) : s[0]);
      const float inv = d > 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
      float part = 0.0f;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        v[h] = __fmul_rn(s[h], inv);
        part = __fmaf_rn(v[h], g[h], part);
      }
      const float mean = warp_sum(part);
#pragma unroll
      for (int h = 0; h < H; ++h) v[h] = __fmul_rn(v[h], __fsub_rn(g[h], mean));
    } else {
      float part = 0.0f;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        v[h] = __fmul_rn(s[h], g[h]);
        part = __fadd_rn(part, v[h]);
      }
      if (DENSE) back = warp_sum(part);
    }
    bool first[H];
    float total[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      if (r.score == MOE_SIGMOID) v[h] = __fmul_rn(v[h], rest[h]);
      first[h] = e[h] >= 0;
      total[h] = v[h];
    }
    // a repeated id gets the sum of its slots, in slot order, from its first one
    // (distinct ids, the rule, are recognised by one match; empty slots differ)
    bool repeated = true;
    if (H == 1) {
      const unsigned same = __match_any_sync(kAll, e[0] >= 0 ? e[0] : -1 - lane);
      repeated = __any_sync(kAll, (same & (same - 1)) != 0);
    }
    if (repeated) {
#pragma unroll
      for (int h = 0; h < H; ++h) total[h] = 0.0f;
      for (int j = 0; j < r.k; ++j) {
        const int ej = __shfl_sync(kAll, j < 32 ? e[0] : e[H - 1], j & 31);
        const float vj = __shfl_sync(kAll, j < 32 ? v[0] : v[H - 1], j & 31);
#pragma unroll
        for (int h = 0; h < H; ++h)
          if (ej == e[h]) {
            total[h] = __fadd_rn(total[h], vj);
            if (j < lane + 32 * h) first[h] = false;
          }
      }
    }
    if (DENSE) {
#pragma unroll
      for (int h = 0; h < H; ++h) total[h] = __fsub_rn(total[h], __fmul_rn(s[h], back));
    }

    // ---- the row ---------------------------------------------------------------------
    if (DENSE && CHUNKS > 0) {
      const float f = -__fmul_rn(inv_sum, back);
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        const int at = lane + 32 * c;
        if (at >= r.E / kPer16) continue;
        float y[kPer16];
#pragma unroll
        for (int i = 0; i < kPer16; i += 2) {
          const float2 q = mul2_rn(make_float2(x[c * kPer16 + i], x[c * kPer16 + i + 1]),
                                   bcast2(f), nz);
          y[i] = q.x;
          y[i + 1] = q.y;
        }
        uint4 o;
        if constexpr (DT == MOE_FP32)
          o = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                         __float_as_uint(y[3]));
        else
          o = pack8<DT>(y);
        reinterpret_cast<uint4*>(out)[at] = o;
      }
    } else if (!DENSE && vec) {
      for (int c = lane; c < r.E / kPer16; c += 32)
        reinterpret_cast<uint4*>(out)[c] = make_uint4(0u, 0u, 0u, 0u);
    } else {
      for (int i = lane; i < r.E; i += 32)
        out[i] = to_elem<DT>(
            DENSE ? -__fmul_rn(__fmul_rn(expf(__fsub_rn(clean_logit<DT>(row + i), m)), inv_sum),
                               back)
                  : 0.0f);
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (first[h]) out[e[h]] = to_elem<DT>(total[h]);
  }
}

template <int DT, bool DENSE, int CHUNKS, int H>
cudaError_t launch_kernel(const RouteArgs& r, bool vec, const int32_t* idx,
                          const float* d_weights, void* d_logits, int32_t* dev_status,
                          cudaStream_t st) {
  auto kernel = route_backward_kernel<DT, DENSE, CHUNKS, H>;
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e == cudaSuccess)
    e = kernel_blocks_per_sm(reinterpret_cast<const void*>(kernel), kWarps * 32, 0, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t grid =
      std::min<int64_t>((r.T + kWarps - 1) / kWarps, int64_t(std::max(1, per_sm)) * sms);
  kernel<<<static_cast<unsigned>(grid), kWarps * 32, 0, st>>>(
      r, vec, idx, d_weights, static_cast<typename Elem<DT>::T*>(d_logits), -0.0f, dev_status);
  return cudaGetLastError();
}

template <int DT, bool DENSE, int H>
cudaError_t launch_t(const RouteArgs& r, const int32_t* idx, const float* d_weights,
                     void* d_logits, int32_t* dev_status, cudaStream_t st) {
  constexpr int kPer16 = 16 / sizeof(typename Elem<DT>::T);
  const bool whole = r.E % kPer16 == 0;            // rows of d_logits are aligned too
  const bool vec = whole && reinterpret_cast<uintptr_t>(r.logits) % 16 == 0 &&
                   r.stride % kPer16 == 0;
  auto launch = [&](auto chunks) {
    return launch_kernel<DT, DENSE, decltype(chunks)::value, H>(
        r, whole, idx, d_weights, d_logits, dev_status, st);
  };
  const int pieces = (r.E / kPer16 + 31) / 32;     // per lane
  if constexpr (DENSE) {
    if (vec && pieces <= 1) return launch(std::integral_constant<int, 1>());
    if (vec && pieces <= 2) return launch(std::integral_constant<int, 2>());
    if (vec && pieces <= 3) return launch(std::integral_constant<int, 3>());
    if (vec && pieces <= 4) return launch(std::integral_constant<int, 4>());
    if constexpr (DT == MOE_FP32)
      if (vec && pieces <= 8) return launch(std::integral_constant<int, 8>());
  }
  return launch(std::integral_constant<int, 0>());
}

template <int DT>
cudaError_t launch_dt(const RouteArgs& r, const int32_t* idx, const float* d_weights,
                      void* d_logits, int32_t* dev_status, cudaStream_t st) {
  const bool dense = r.score == MOE_SOFTMAX && !r.renormalise;
  if (r.k <= 32)
    return dense ? launch_t<DT, true, 1>(r, idx, d_weights, d_logits, dev_status, st)
                 : launch_t<DT, false, 1>(r, idx, d_weights, d_logits, dev_status, st);
  return dense ? launch_t<DT, true, 2>(r, idx, d_weights, d_logits, dev_status, st)
               : launch_t<DT, false, 2>(r, idx, d_weights, d_logits, dev_status, st);
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

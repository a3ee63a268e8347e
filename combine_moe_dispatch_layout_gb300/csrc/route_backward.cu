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
// A lane holds the value of one slot (two for k > 32); a token takes as many
// lanes as it has slots, rounded up to 8, 16 or 32.  The rows are written in
// 16-byte pieces (zeros, or -p_e * sum), and after a warp barrier, which orders
// the warp's own stores, the k chosen elements are stored over them, while the
// lines are still in L2.  Plain softmax keeps the row's exponentials in registers
// between its two sums and the write.
//
// Measured (in a graph): 32,768 x 256 fp32, renormalised sigmoid, k = 8: 8.1 us (4.2
// TB/s of writes; 12.5 with a warp per token, zeros after the sums: the chain id ->
// logit -> sums was paid four times as often).  49,152 x 768 bf16, plain softmax: 30 us,
// 5.0 TB/s both ways; the exponentials' instructions (75% of the issue slots) are what
// keeps it from a copy's 23 us.  Rows of any other length or alignment are read three
// times, element by element: 49,152 x 767 77 us, 32,768 x 250 fp32 27 (x 256: 17).
#include <type_traits>

#include "moe_ep_internal.cuh"
#include "route_math.cuh"

namespace moe_ep {
namespace {

constexpr int kWarps = 2;   // per CTA (wide rows: 2 31.0 us, 4 31.5, 8 32.4)

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

// What a lane knows of its H slots (j and j + 32 of a token with W lanes).
template <int H>
struct Slots {
  int e[H];            // expert, -1: none
  float l[H], g[H];    // logit, gradient of the unscaled weight
};

// at: the token, there: it exists.
template <int DT, int W, int H>
__device__ __forceinline__ Slots<H> load_slots(const RouteArgs& r, int64_t at, bool there,
                                               int j0, const int32_t* idx,
                                               const float* d_weights, int32_t* dev_status) {
  using T = typename Elem<DT>::T;
  const T* row = static_cast<const T*>(r.logits) + at * r.stride;
  Slots<H> s;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int j = j0 + 32 * h;
    const bool mine = there && j < r.k;
    s.e[h] = mine ? idx[at * r.k + j] : -1;
    s.g[h] = mine ? __fmul_rn(d_weights[at * r.k + j], r.scale) : 0.0f;
    if (s.e[h] < -1 || s.e[h] >= r.E) {
      set_status(dev_status, MOE_ERR_EXPERT_ID);
      s.e[h] = -1;
    }
    s.l[h] = s.e[h] >= 0 ? clean_logit<DT>(row + s.e[h]) : kNegInf;
    if (s.e[h] < 0) s.g[h] = 0.0f;
  }
  return s;
}

// total: the slots' own gradients; where a token names an expert twice, the sum of
// its slots, in slot order, at the first of them, which alone keeps first set.
// Distinct ids, the rule, are recognised by one match.
template <int W, int H>
__device__ __forceinline__ void join_repeated(const Slots<H>& s, int k, int lane, int j0,
                                              float* total, bool* first) {
#pragma unroll
  for (int h = 0; h < H; ++h) first[h] = s.e[h] >= 0;
  if constexpr (H == 1) {              // empty slots differ from one another
    const int token = lane & -W;
    const unsigned same =
        __match_any_sync(kAll, s.e[0] >= 0 ? token * MOE_EP_MAX_EXPERTS + s.e[0] : -1 - lane);
    if (!__any_sync(kAll, (same & (same - 1)) != 0)) return;
  }
  float v[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    v[h] = total[h];
    total[h] = 0.0f;
  }
  for (int j = 0; j < k; ++j) {
    const int ej = __shfl_sync(kAll, j < 32 ? s.e[0] : s.e[H - 1], j & 31, W);
    const float vj = __shfl_sync(kAll, j < 32 ? v[0] : v[H - 1], j & 31, W);
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (ej == s.e[h]) {
        total[h] = __fadd_rn(total[h], vj);
        if (j < j0 + 32 * h) first[h] = false;
      }
  }
}

// Every form but plain softmax.  W lanes per token, 32 / W neighbouring tokens per
// warp: their rows of d_logits follow one another, and the zeros, which wait for
// nothing, are on their way before the first load.  vec: 16-byte stores.
template <int DT, int W, int H>
__global__ void __launch_bounds__(kWarps * 32)
route_backward_sparse_kernel(const RouteArgs r, bool vec, const int32_t* idx,
                             const float* d_weights, typename Elem<DT>::T* d_logits,
                             int32_t* dev_status) {
  using T = typename Elem<DT>::T;
  constexpr int kPer16 = 16 / sizeof(T);
  constexpr int kTokens = 32 / W;
  const int lane = threadIdx.x & 31, j0 = lane & (W - 1);
  const int64_t t0 = (int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kTokens;
  wait_for_stream();
  let_next_start();
  if (t0 >= r.T) return;
  const int64_t t = t0 + lane / W;

  T* out = d_logits + t0 * r.E;
  const int fill = static_cast<int>(min(r.T - t0, int64_t(kTokens))) * r.E;
  const int pieces = vec ? fill / kPer16 : 0;
  for (int c = lane; c < pieces; c += 32)
    reinterpret_cast<uint4*>(out)[c] = make_uint4(0u, 0u, 0u, 0u);
  for (int i = pieces * kPer16 + lane; i < fill; i += 32) out[i] = to_elem<DT>(0.0f);

  const Slots<H> s = load_slots<DT, W, H>(r, t, t < r.T, j0, idx, d_weights, dev_status);
  // score (scaled by a common factor where it is renormalised), and 1 - score of a sigmoid
  float p[H], rest[H], v[H];
  float m = 0.0f;
  if (r.renormalise)
    m = fmaxf(lanes_max<W>(H > 1 ? fmaxf(s.l[0], s.l[H - 1]) : s.l[0]), -kMaxF);
  if (r.score == MOE_SOFTMAX) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      p[h] = s.e[h] >= 0 ? expf(__fsub_rn(s.l[h], m)) : 0.0f;
      rest[h] = 1.0f;
    }
  } else {
    m = fminf(m, 0.0f);
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const float sig = sigmoid_scaled(s.l[h], m, &rest[h]);
      p[h] = s.e[h] >= 0 ? sig : 0.0f;
    }
  }
  if (r.renormalise) {
    const float d = lanes_sum<W>(H > 1 ? __fadd_rn(p[0], p[H - 1]) : p[0]);
    const float inv = d > 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
    float part = 0.0f;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      v[h] = __fmul_rn(p[h], inv);
      part = __fmaf_rn(v[h], s.g[h], part);
    }
    const float mean = lanes_sum<W>(part);
#pragma unroll
    for (int h = 0; h < H; ++h) v[h] = __fmul_rn(v[h], __fsub_rn(s.g[h], mean));
  } else {
#pragma unroll
    for (int h = 0; h < H; ++h) v[h] = __fmul_rn(p[h], s.g[h]);
  }
  bool first[H];
#pragma unroll
  for (int h = 0; h < H; ++h) v[h] = __fmul_rn(v[h], rest[h]);
  join_repeated<W, H>(s, r.k, lane, j0, v, first);
  __syncwarp();                        // the zeros come first
#pragma unroll
  for (int h = 0; h < H; ++h)
    if (first[h]) d_logits[t * r.E + s.e[h]] = to_elem<DT>(v[h]);
}

// Plain softmax.  CHUNKS: 16-byte pieces of a row per lane, kept in registers (rows
// of logits 16-byte aligned, E a whole number of pieces); 0: any E and alignment,
// element by element.  H: slots per lane (1 for k <= 32, else 2).
template <int DT, int CHUNKS, int H>
__global__ void __launch_bounds__(kWarps * 32)
route_backward_dense_kernel(const RouteArgs r, const int32_t* idx,
                            const float* d_weights, typename Elem<DT>::T* d_logits, float nz,
                            int32_t* dev_status) {
  using T = typename Elem<DT>::T;
  constexpr int kPer16 = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  const int64_t t = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  wait_for_stream();
  let_next_start();
  if (t >= r.T) return;
  const T* row = static_cast<const T*>(r.logits) + t * r.stride;
  T* out = d_logits + t * r.E;

  // ---- the row's maximum and sum -----------------------------------------------
  float m = kNegInf, sum = 0.0f;
  float x[CHUNKS > 0 ? CHUNKS * kPer16 : 1];   // the lane's logits, then exponentials
  if constexpr (CHUNKS > 0) {
    const int pieces = r.E / kPer16;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int at = lane + 32 * c;
      const uint4 q = at < pieces ? reinterpret_cast<const uint4*>(row)[at] : make_uint4(0u, 0u, 0u, 0u);
      unpack_logits<DT>(q, x + c * kPer16);
    }
  }
  const Slots<H> s = load_slots<DT, 32, H>(r, t, true, lane, idx, d_weights, dev_status);
  if constexpr (CHUNKS > 0) {
    const int pieces = r.E / kPer16;
    float probe = 0.0f;
#pragma unroll
    for (int i = 0; i < CHUNKS * kPer16; ++i) probe = __fmaf_rn(x[i], 0.0f, probe);
    if (__any_sync(kAll, probe != probe)) {      // infinities and NaN, as moe_route
#pragma unroll
      for (int i = 0; i < CHUNKS * kPer16; ++i)
        x[i] = x[i] != x[i] ? kNegInf : fminf(x[i], kMaxF);
    }
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
    sum = __fadd_rn(sum2.x, sum2.y);
  } else {
    for (int i = lane; i < r.E; i += 32) m = fmaxf(m, clean_logit<DT>(row + i));
    m = fmaxf(warp_max(m), -kMaxF);
    for (int i = lane; i < r.E; i += 32)
      sum = __fadd_rn(sum, expf(__fsub_rn(clean_logit<DT>(row + i), m)));
  }
  sum = warp_sum(sum);
  const float inv_sum = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;

  // ---- the slots' gradients, and what every expert loses ---------------------------
  float p[H], v[H], part = 0.0f;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    p[h] = s.e[h] >= 0 ? __fmul_rn(expf(__fsub_rn(s.l[h], m)), inv_sum) : 0.0f;
    v[h] = __fmul_rn(p[h], s.g[h]);
    part = __fadd_rn(part, v[h]);
  }
  const float back = warp_sum(part);
  bool first[H];
  join_repeated<32, H>(s, r.k, lane, lane, v, first);

  // ---- the row ---------------------------------------------------------------------
  const float f = -__fmul_rn(inv_sum, back);
  if constexpr (CHUNKS > 0) {
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
  } else {
    for (int i = lane; i < r.E; i += 32)
      out[i] = to_elem<DT>(__fmul_rn(expf(__fsub_rn(clean_logit<DT>(row + i), m)), f));
  }
  __syncwarp();
#pragma unroll
  for (int h = 0; h < H; ++h)
    if (first[h])
      out[s.e[h]] = to_elem<DT>(__fsub_rn(v[h], __fmul_rn(p[h], back)));
}

template <int DT, int W, int H>
cudaError_t launch_sparse(const RouteArgs& r, const int32_t* idx, const float* d_weights,
                          void* d_logits, int32_t* dev_status, cudaStream_t st) {
  using T = typename Elem<DT>::T;
  constexpr int kTokens = kWarps * 32 / W;         // per CTA
  const bool vec = r.E * sizeof(T) * (32 / W) % 16 == 0;   // each warp's first row is aligned
  return launch_early(route_backward_sparse_kernel<DT, W, H>, (r.T + kTokens - 1) / kTokens,
                      kWarps * 32, 0, st, r, vec, idx, d_weights, static_cast<T*>(d_logits),
                      dev_status);
}

template <int DT, int CHUNKS, int H>
cudaError_t launch_dense(const RouteArgs& r, const int32_t* idx, const float* d_weights,
                         void* d_logits, int32_t* dev_status, cudaStream_t st) {
  return launch_early(route_backward_dense_kernel<DT, CHUNKS, H>, (r.T + kWarps - 1) / kWarps,
                      kWarps * 32, 0, st, r, idx, d_weights,
                      static_cast<typename Elem<DT>::T*>(d_logits), -0.0f, dev_status);
}

template <int DT, int H>
cudaError_t launch_h(const RouteArgs& r, const int32_t* idx, const float* d_weights,
                     void* d_logits, int32_t* dev_status, cudaStream_t st) {
  if (r.score != MOE_SOFTMAX || r.renormalise) {
    if constexpr (H == 1) {
      if (r.k <= 8)
        return launch_sparse<DT, 8, 1>(r, idx, d_weights, d_logits, dev_status, st);
      if (r.k <= 16)
        return launch_sparse<DT, 16, 1>(r, idx, d_weights, d_logits, dev_status, st);
    }
    return launch_sparse<DT, 32, H>(r, idx, d_weights, d_logits, dev_status, st);
  }
  constexpr int kPer16 = 16 / sizeof(typename Elem<DT>::T);
  const bool vec = r.E % kPer16 == 0 && reinterpret_cast<uintptr_t>(r.logits) % 16 == 0 &&
                   r.stride % kPer16 == 0;
  auto launch = [&](auto chunks) {
    return launch_dense<DT, decltype(chunks)::value, H>(r, idx, d_weights, d_logits,
                                                        dev_status, st);
  };
  const int pieces = (r.E / kPer16 + 31) / 32;     // per lane
  if (vec && pieces <= 1) return launch(std::integral_constant<int, 1>());
  if (vec && pieces <= 2) return launch(std::integral_constant<int, 2>());
  if (vec && pieces <= 3) return launch(std::integral_constant<int, 3>());
  if (vec && pieces <= 4) return launch(std::integral_constant<int, 4>());
  if constexpr (DT == MOE_FP32)
    if (vec && pieces <= 8) return launch(std::integral_constant<int, 8>());
  return launch(std::integral_constant<int, 0>());
}

template <int DT>
cudaError_t launch_dt(const RouteArgs& r, const int32_t* idx, const float* d_weights,
                      void* d_logits, int32_t* dev_status, cudaStream_t st) {
  return r.k <= 32 ? launch_h<DT, 1>(r, idx, d_weights, d_logits, dev_status, st)
                   : launch_h<DT, 2>(r, idx, d_weights, d_logits, dev_status, st);
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

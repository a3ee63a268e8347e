// route_math.cuh -- what routing and its gradient share: logits of any type, warp
// reductions, exponentials.
#pragma once

#include "moe_ep_internal.cuh"

namespace moe_ep {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kMaxF = 3.402823466e38f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.44269502f;      // log2(e), and what that leaves out
constexpr float kLog2eLo = 1.92596299e-8f;
constexpr float kLn2 = 0.693147181f;

template <int DT>
struct Elem { using T = uint16_t; };
template <>
struct Elem<MOE_FP32> { using T = float; };

// A logit as fp32.
template <int DT>
__device__ __forceinline__ float load_logit(const typename Elem<DT>::T* p) {
  if constexpr (DT == MOE_FP32) return *p;
  else return widen<DT>(*p);
}
// The 16 / sizeof(T) logits of a 16-byte piece.
template <int DT>
__device__ __forceinline__ void unpack_logits(const uint4& v, float* l) {
  if constexpr (DT == MOE_FP32) {
    l[0] = __uint_as_float(v.x);
    l[1] = __uint_as_float(v.y);
    l[2] = __uint_as_float(v.z);
    l[3] = __uint_as_float(v.w);
  } else {
    float f[8];
    unpack8<DT>(v, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) l[i] = f[i];
  }
}

// Order-preserving key of a float; -0 reads as +0.  Keys of numbers above
// -inf are never 0.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t b = __float_as_uint(__fadd_rn(f, 0.0f));
  return b ^ ((b & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kAll, v, d));
  return v;
}
// The maximum over the warp, by the integer reduction (one instruction; the
// floating one is slower).
__device__ __forceinline__ float warp_max(float v) {
  const uint32_t k = __reduce_max_sync(kAll, order_key(v));
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

// Sum and maximum over the W lanes of a token.
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int d = W / 2; d; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kAll, v, d));
  return v;
}
template <int W>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (W == 32) {
    return warp_max(v);
  } else {
#pragma unroll
    for (int d = W / 2; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
    return v;
  }
}

__device__ __forceinline__ float exp2_approx(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
  return e;
}
// e^x for x <= 0 to about 2 ulp (0 below -120): x log2(e) in two parts, the
// second one (with |part| < 2^-16) to first order.
__device__ __forceinline__ float exp_neg(float x) {
  x = fmaxf(x, -120.0f);
  const float t = __fmul_rn(x, kLog2e);
  const float r = __fmaf_rn(x, kLog2eLo, __fmaf_rn(x, kLog2e, -t));
  const float e = exp2_approx(t);
  return __fmaf_rn(e, __fmul_rn(r, kLn2), e);
}
// The same of two numbers, packed.  nz: -0 (see mul2_rn).
__device__ __forceinline__ float2 exp_neg2(float2 x, float nz) {
  x = make_float2(fmaxf(x.x, -120.0f), fmaxf(x.y, -120.0f));
  const float2 t = mul2_rn(x, bcast2(kLog2e), nz);
  const float2 r = fma2_rn(x, bcast2(kLog2eLo),
                           fma2_rn(x, bcast2(kLog2e), make_float2(-t.x, -t.y)));
  const float2 e = make_float2(exp2_approx(t.x), exp2_approx(t.y));
  return fma2_rn(e, mul2_rn(r, bcast2(kLn2), nz), e);
}

// Sigmoid of x times e^-m = e^(min(x, 0) - m) / (1 + e^-|x|), m the smaller of 0 and
// the largest chosen logit of the token.  No exponential exceeds 1, so nothing
// overflows, and the largest of a token's scaled scores is at least 1/2, however far
// below 0 its logits are (the scores alone are subnormal from -87 on and 0 from -104).
// m = 0: the sigmoid itself.  rest: 1 - sigmoid(x), without cancellation.
__device__ __forceinline__ float sigmoid_scaled(float x, float m, float* rest) {
  const float ex = expf(-fabsf(x)), d = __fadd_rn(1.0f, ex);
  const float top = x >= 0.0f ? 1.0f : m < 0.0f ? expf(__fsub_rn(x, m)) : ex;
  *rest = __fdiv_rn(x >= 0.0f ? ex : 1.0f, d);
  return __fdiv_rn(top, d);
}

}  // namespace moe_ep

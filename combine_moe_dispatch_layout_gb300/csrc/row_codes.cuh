// row_codes.cuh -- rows of 8-bit codes with their scales (row images), as the norm
// and the SwiGLU step write them and the 8-bit products read them.
#pragma once

#include "moe_ep_internal.cuh"

namespace moe_ep {

constexpr int kCodeBlock = 128;                  // values that share an e4m3 scale
constexpr float kTinyMax = 1e-12f;               // a block's largest magnitude is at least this
constexpr float kF8Max = 448.0f;                 // the largest e4m3 number

__host__ __device__ constexpr int code_blocks(int H) {
  return (H + kCodeBlock - 1) / kCodeBlock;
}
// An e4m3 row image: H codes, zeros up to a multiple of 32 bytes, a fp32 scale per
// 128 codes, zeros up to a multiple of 32 bytes.
__host__ __device__ constexpr int64_t f8_scales_at(int H) { return align_up(H, 32); }
__host__ __device__ constexpr int64_t f8_row_bytes(int H) {
  return f8_scales_at(H) + align_up(4 * int64_t(code_blocks(H)), 32);
}

// The largest magnitude of 8 values as bits (ordered as unsigned numbers; a NaN is
// above every number, so it reaches the scale and the whole block).
__device__ __forceinline__ uint32_t abs_max_bits(const float (&y)[8]) {
  float m = fabsf(y[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(y[j])));
  return __float_as_uint(m) & 0x7fffffffu;
}

// 1 / x within 1 ulp for normal x (a number that comes out subnormal is 0).
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Over the 16 lanes of a half warp, which hold a block's 128 values.
__device__ __forceinline__ uint32_t block_max_bits(uint32_t m) {
#pragma unroll
  for (int d = 8; d; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}

// Two products in one instruction, each rounded once (no sum follows that the compiler
// could merge it with).
__device__ __forceinline__ float2 mul_pair(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 pa, pb, pd;\n\tmov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\t"
      "mul.rn.f32x2 pd, pa, pb;\n\tmov.b64 {%0, %1}, pd;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// The block's scale, and what its values are multiplied by.
struct F8Scale {
  float scale, inv;
};
__device__ __forceinline__ F8Scale f8_scale(uint32_t max_bits) {
  const float top = __uint_as_float(max(max_bits, __float_as_uint(kTinyMax)));
  const float scale = __fmul_rn(top, 1.0f / kF8Max);
  // (of the scale, whose reciprocal is a normal number for every finite block; that of a
  // block's maximum beyond 2^126 is not, and would be 0)
  return {scale, reciprocal(scale)};
}

// 8 values -> 8 e4m3 codes, nearest even (a product that rounding took past 448 is
// 448; NaN stays NaN).
__device__ __forceinline__ uint2 f8_codes(const float (&y)[8], float inv) {
  uint16_t c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 q = mul_pair(make_float2(y[2 * j], y[2 * j + 1]), make_float2(inv, inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c[j]) : "f"(q.y), "f"(q.x));
  }
  return make_uint2(c[0] | uint32_t(c[1]) << 16, c[2] | uint32_t(c[3]) << 16);
}

// 8 values -> 8 INT8 codes, half to even.
__device__ __forceinline__ uint2 i8_codes(const float (&y)[8], float scale) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = max(-127, min(127, __float2int_rn(__fmul_rn(y[j], scale))));
    w[j / 4] |= uint32_t(c & 0xff) << (8 * (j % 4));
  }
  return make_uint2(w[0], w[1]);
}

}  // namespace moe_ep

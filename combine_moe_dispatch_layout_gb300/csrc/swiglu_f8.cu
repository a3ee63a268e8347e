// swiglu_f8.cu -- the step between the two products of an e4m3 MoE layer: [gate | up]
// rows -> e4m3 row images of silu(gate) * up (include/moe_ep.h, moe_swiglu_f8).
//
// h = gate / (1 + exp(-gate)) * up in fp32, a scale per 128 values, one rounding to
// e4m3.  A half warp takes kBlocks neighbouring blocks of a row, lane l the 8 values from
// 8 l of each, so all its loads are under way at once and its scales leave in one store.
// Bound by memory, with the arithmetic close behind: at 31 instructions a value (IEEE
// division and exponential, maxima of integers) the issue slots were 84% busy and 262,144 x
// 2048 took 492 us; as written here 391 to 408, 98 to 102% of a copy's rate.
#include "row_codes.cuh"

namespace moe_ep {
namespace {

constexpr int kThreads = 256;
template <int DT>
struct Raw8 {                           // 8 values as they lie in memory
  uint4 v[DT == MOE_FP32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* row, int64_t at) {
    const char* p = static_cast<const char*>(row) + at * (DT == MOE_FP32 ? 4 : 2);
    v[0] = ld_once_16(p);
    if constexpr (DT == MOE_FP32) v[1] = ld_once_16(p + 16);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (DT == MOE_FP32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(v[i].x);
        f[4 * i + 1] = __uint_as_float(v[i].y);
        f[4 * i + 2] = __uint_as_float(v[i].z);
        f[4 * i + 3] = __uint_as_float(v[i].w);
      }
    } else {
      unpack8<DT>(v[0], f);
    }
  }
};

// 1 / (1 + exp(-x)): the exponential as 2^(-x log2 e), within 2^-21 and |x| 2^-23 of itself
// (the argument's rounding).  From x = -126 ln 2, about -87.34, on down the divisor passes 2^126:
// its reciprocal would be subnormal, and is 0.
__device__ __forceinline__ float sigmoid(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(x, -1.44269504f)));
  return reciprocal(__fadd_rn(1.0f, e));
}

// kBlocks: 128-value blocks per half warp; with fewer than 4 a row is one half warp's.
// (Rows of 128 values by half warps of 4 blocks: three in four loads less under way.)
template <int DT, int kBlocks>
__global__ void __launch_bounds__(kThreads)
swiglu_f8_kernel(const SwigluF8Args p) {
  wait_for_stream();
  let_next_start();
  const int lane = threadIdx.x % 16;
  const int nb = code_blocks(p.I), spans = (nb + kBlocks - 1) / kBlocks;   // per row
  const int64_t unit = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / 16;
  const int64_t row = unit <= UINT32_MAX ? uint32_t(unit) / uint32_t(spans) : unit / spans;
  const int b0 = static_cast<int>(unit - row * spans) * kBlocks;
  int64_t rows = p.M;
  if (p.group_off) {
    const int64_t there = p.group_off[p.G];
    if (there > rows && unit == 0) set_status(p.dev_status, MOE_ERR_CAPACITY);
    rows = min(rows, there);
  }
  // (both half warps stay for the shuffles)
  const bool live = row < rows;
  const char* h = static_cast<const char*>(p.h) +
                  (live ? row : 0) * p.h_stride * (DT == MOE_FP32 ? 4 : 2);
  Raw8<DT> g[kBlocks], u[kBlocks];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    const int c = (b0 + i) * kCodeBlock + 8 * lane;
    g[i] = {};
    u[i] = {};
    if (live && c < p.I) {
      g[i].load(h, c);
      u[i].load(h, p.I + c);
    }
  }
  uint8_t* codes = static_cast<uint8_t*>(p.codes) + (live ? row : 0) * f8_row_bytes(p.I);
  const int padded = static_cast<int>(f8_scales_at(p.I));
  float scales[kBlocks];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    const int c = (b0 + i) * kCodeBlock + 8 * lane;
    float a[8], b[8];
    g[i].get(a);
    u[i].get(b);
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = __fmul_rn(__fmul_rn(a[j], sigmoid(a[j])), b[j]);
    const F8Scale sc = f8_scale(block_max_bits(c < p.I ? abs_max_bits(a) : 0u));
    scales[i] = b0 + i < nb ? sc.scale : 0.0f;
    if (live && c < padded)
      *reinterpret_cast<uint2*>(codes + c) = c < p.I ? f8_codes(a, sc.inv) : make_uint2(0u, 0u);
  }
  if constexpr (kBlocks < 4) {            // all of the row's scales, and zeros up to 8
    float mine = 0.0f;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) mine = lane == i ? scales[i] : mine;
    if (live && lane < 8) reinterpret_cast<float*>(codes + padded)[lane] = mine;
  } else {
    float4* to = reinterpret_cast<float4*>(codes + padded + 4 * b0);
    if (live && lane == 0) to[0] = make_float4(scales[0], scales[1], scales[2], scales[3]);
    // the zeros up to the next multiple of 8 scales
    if (live && lane == 0 && b0 + kBlocks >= nb && (b0 + kBlocks) % 8 != 0)
      to[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
}

template <int DT, int kBlocks>
cudaError_t launch(const SwigluF8Args& p, cudaStream_t st) {
  const int64_t spans = (code_blocks(p.I) + kBlocks - 1) / kBlocks;
  const int64_t grid = (p.M * spans * 16 + kThreads - 1) / kThreads;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_early(swiglu_f8_kernel<DT, kBlocks>, grid, kThreads, 0, st, p);
}

template <int DT>
cudaError_t launch_type(const SwigluF8Args& p, cudaStream_t st) {
  const int nb = code_blocks(p.I);
  return nb == 1 ? launch<DT, 1>(p, st) : nb == 2 ? launch<DT, 2>(p, st) : launch<DT, 4>(p, st);
}

}  // namespace

cudaError_t launch_swiglu_f8(const SwigluF8Args& p, cudaStream_t st) {
  switch (p.dtype) {
    case MOE_BF16: return launch_type<MOE_BF16>(p, st);
    case MOE_FP16: return launch_type<MOE_FP16>(p, st);
    default: return launch_type<MOE_FP32>(p, st);
  }
}

}  // namespace moe_ep

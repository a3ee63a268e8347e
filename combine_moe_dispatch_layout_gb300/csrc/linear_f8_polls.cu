// linear_f8_polls.cu -- the e4m3 product's tile kernel with short waits, and the plan it runs
// by: entry points for tests (exported, not in the public header).
//
// A role that runs out of polls gives up as it does after kGemmSpin of them; the
// closing waits (for copies and commits in flight) keep the full bound.
#include <cuda_runtime.h>
#include <stdint.h>

#include "tcgen05.cuh"

namespace moe_ep {
namespace {
__constant__ uint32_t c_first;     // kGemmSpin less the polls

__device__ __forceinline__ bool look(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// As warp_bar_wait and warp_bar_wait4, with fewer polls (one at the least), which look and do
// not wait.
__device__ __forceinline__ bool warp_role_wait(uint32_t bar, uint32_t parity) {
  uint32_t i = c_first;
  do {
    if (__all_sync(0xffffffffu, look(bar, parity))) return true;
  } while (++i < kGemmSpin);
  return false;
}
__device__ __forceinline__ bool warp_role_wait2(uint32_t a, uint32_t b, uint32_t parity) {
  return warp_role_wait(a, parity) && warp_role_wait(b, parity);
}
__device__ __forceinline__ bool warp_role_wait4(uint32_t a, uint32_t b, uint32_t c,
                                                uint32_t parity, uint32_t d, uint32_t pd) {
  return warp_role_wait(a, parity) && warp_role_wait(b, parity) && warp_role_wait(c, parity) &&
         warp_role_wait(d, pd);
}
}  // namespace
}  // namespace moe_ep

#define MOE_LINEAR_F8_POLLS
#include "linear_f8.cu"

// What moe_linear_f8 does with a problem on a GPU of `sms` SMs: plan[0] = channels per tile of
// the kernel it takes (0: the kernel for few rows), plan[1] = clusters, plan[2] = CTAs of a
// cluster.  Host only.
extern "C" void moe_test_linear_f8_plan_of(int64_t a_rows, int32_t G, int32_t N, int32_t K,
                                           int32_t c_dtype, int32_t sms, int32_t* plan) {
  moe_ep::LinearArgs p{};
  p.a_rows = a_rows;
  p.G = G;
  p.N = N;
  p.K = K;
  p.c_dtype = c_dtype;
  plan[0] = plan[1] = plan[2] = 0;
  if (moe_ep::use_few(p, sms)) return;
  const moe_ep::Plan best = moe_ep::make_plan(p, sms);
  plan[0] = best.nt;
  plan[1] = best.clusters;
  plan[2] = best.form == moe_ep::kSingle ? 1 : best.form == moe_ep::kPair ? 2 : 4;
}
// The same with fp32 results.
extern "C" void moe_test_linear_f8_plan(int64_t a_rows, int32_t G, int32_t N, int32_t K,
                                        int32_t sms, int32_t* plan) {
  moe_test_linear_f8_plan_of(a_rows, G, N, K, MOE_FP32, sms, plan);
}

// moe_linear_f8's tile kernel with fp32 results and roles that wait for at most `polls`
// looks at a barrier (arguments as there; the caller keeps the limits).
extern "C" moe_status moe_test_linear_f8_polls(const void* a, int64_t a_rows, int64_t a_stride,
                                               const void* w, int64_t w_stride, int32_t G,
                                               int32_t N, int32_t K, const int32_t* group_rows,
                                               const float* w_scale, const void* a_scale,
                                               int64_t a_scale_stride, float* c,
                                               uint32_t polls, int32_t* dev_status,
                                               void* stream) {
  using namespace moe_ep;
  const LinearArgs p{a, a_rows, a_stride, w, w_stride, G, N, K, group_rows, w_scale,
                     static_cast<const unsigned char*>(a_scale), a_scale_stride, nullptr, c,
                     MOE_FP32};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int dev = 0, sms = 0, optin = 0;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  const uint32_t from = kGemmSpin - std::max(1u, std::min(polls, kGemmSpin));
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(c_first, &from, sizeof(from), 0, cudaMemcpyHostToDevice, st);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  Plan plan = make_plan(p, sms);
  Maps maps;
  e = make_maps(p, &plan, &maps);
  if (e == cudaSuccess)
    e = plan.form == kSingle
            ? launch_kernel<256, MOE_FP32, kSingle>(maps, p, plan, dev_status, optin, st)
        : plan.form == kHalves && plan.nt == 64
            ? launch_kernel<64, MOE_FP32, kHalves>(maps, p, plan, dev_status, optin, st)
        : plan.form == kHalves
            ? launch_kernel<128, MOE_FP32, kHalves>(maps, p, plan, dev_status, optin, st)
        : plan.nt == 64
            ? launch_kernel<64, MOE_FP32, kPair>(maps, p, plan, dev_status, optin, st)
        : plan.nt == 128
            ? launch_kernel<128, MOE_FP32, kPair>(maps, p, plan, dev_status, optin, st)
            : launch_kernel<256, MOE_FP32, kPair>(maps, p, plan, dev_status, optin, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

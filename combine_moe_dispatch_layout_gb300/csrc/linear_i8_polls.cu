// linear_i8_polls.cu -- the INT8 product's tile kernel with short waits, and the plan it
// runs by: entry points for tests (exported, not in the public header).
//
// A role that runs out of polls gives up as it does after kGemmSpin of them; the
// closing waits (for copies and commits in flight) keep the full bound.
#include <cuda_runtime.h>
#include <stdint.h>

#include "tcgen05.cuh"

namespace moe_ep {
namespace {
__constant__ uint32_t c_first;     // kGemmSpin less the polls

// As bar_wait, with fewer polls (one at the least), which look and do not wait.
__device__ __forceinline__ bool role_wait(uint32_t bar, uint32_t parity) {
  uint32_t i = c_first;
  do {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
  } while (++i < kGemmSpin);
  return false;
}
}  // namespace
}  // namespace moe_ep

#define MOE_LINEAR_I8_POLLS
#include "linear_i8.cu"

namespace moe_ep {
namespace {

LinearArgs sums_of(const void* a, int64_t a_rows, int64_t a_stride, const void* w,
                   int64_t w_stride, int32_t G, int32_t N, int32_t K, const int32_t* group_rows,
                   int32_t* c) {
  return LinearArgs{a, a_rows, a_stride, w, w_stride, G, N, K, group_rows, nullptr, nullptr, 4,
                    nullptr, c, MOE_INT32};
}

}  // namespace
}  // namespace moe_ep

// What moe_linear_i8 does with a problem on a GPU of `sms` SMs: plan[0] = tokens per tile
// of the kernel it takes (0: the kernel for few rows), plan[1] = pairs that share a
// tile's K, plan[2] = clusters.  Host only.
extern "C" void moe_test_linear_i8_plan(int64_t a_rows, int32_t G, int32_t N, int32_t K,
                                        int32_t sms, int32_t* plan) {
  const moe_ep::LinearArgs p =
      moe_ep::sums_of(nullptr, a_rows, K, nullptr, K, G, N, K, nullptr, nullptr);
  plan[0] = plan[1] = plan[2] = 0;
  if (moe_ep::use_few(p)) return;
  const moe_ep::Plan best = moe_ep::make_plan(p, sms);
  plan[0] = best.nt;
  plan[1] = best.split;
  plan[2] = best.clusters;
}

// moe_linear_i8's tile kernel with int32 results and roles that wait for at most `polls`
// looks at a barrier (arguments as there; the caller keeps the limits).
extern "C" moe_status moe_test_linear_i8_polls(const void* a, int64_t a_rows, int64_t a_stride,
                                               const void* w, int64_t w_stride, int32_t G,
                                               int32_t N, int32_t K, const int32_t* group_rows,
                                               int32_t* c, uint32_t polls, int32_t* dev_status,
                                               void* stream) {
  using namespace moe_ep;
  const LinearArgs p = sums_of(a, a_rows, a_stride, w, w_stride, G, N, K, group_rows, c);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int dev = 0, sms = 0, optin = 0;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  const uint32_t from = kGemmSpin - std::max(1u, std::min(polls, kGemmSpin));
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(c_first, &from, sizeof(from), 0, cudaMemcpyHostToDevice, st);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  const Plan plan = make_plan(p, sms);
  CUtensorMap mw, ma;
  e = encode_bytes_2d(&mw, p.w, int64_t(G) * N, K, w_stride, BM);
  if (e == cudaSuccess) e = encode_bytes_2d(&ma, p.a, a_rows, K, a_stride, plan.box_rows);
  if (e == cudaSuccess)
    e = plan.nt == 256
            ? launch_out<256, MOE_INT32>(mw, ma, p, plan, dev_status, optin, st)
            : launch_out<128, MOE_INT32>(mw, ma, p, plan, dev_status, optin, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

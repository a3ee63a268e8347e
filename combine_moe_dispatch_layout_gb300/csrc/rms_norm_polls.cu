// rms_norm_polls.cu -- the gradient of the norm with waits that run out: an entry point for
// tests (exported, not in the public header).
//
// Of a thread's waits for rows one in `odds` gives up at once, whichever the clock picks; the
// others, and the closing waits for copies in flight, keep their bound.
#include "moe_ep_internal.cuh"

namespace moe_ep {
namespace {
__constant__ uint32_t c_odds;

__device__ __forceinline__ bool row_wait(uint64_t* bar, uint32_t parity) {
  uint32_t x = static_cast<uint32_t>(clock()) * 2654435761u + threadIdx.x * 40503u;
  x ^= x >> 15;
  return x % c_odds != 0 && mbar_wait_bounded(bar, parity, kGemmSpin);
}
}  // namespace
}  // namespace moe_ep

#define MOE_RMS_NORM_POLLS
#include "rms_norm.cu"

// moe_rms_norm_backward of bf16 rows of at most 16,384 values, without d_gamma's sum over
// the CTAs (arguments as there; the caller keeps the limits).
extern "C" moe_status moe_test_rms_norm_backward_odds(
    const void* d_out, int64_t T, int32_t H, int64_t d_out_stride, const void* x,
    int64_t x_stride, const float* gamma, const float* rstd, const void* d_sum,
    int64_t d_sum_stride, void* d_x, int64_t d_x_stride, void* workspace, uint32_t odds,
    int32_t* dev_status, void* stream) {
  using namespace moe_ep;
  if (H > kMaxWidth) return MOE_ERR_INVALID_ARG;
  const NormBackwardArgs p{d_out, x, d_sum, gamma, rstd, d_x, static_cast<float*>(workspace),
                           dev_status, T, d_out_stride, x_stride, d_sum_stride, d_x_stride, H,
                           MOE_BF16};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const uint32_t of = std::max(1u, odds);
  cudaError_t e = cudaMemcpyToSymbolAsync(c_odds, &of, sizeof(of), 0, cudaMemcpyHostToDevice, st);
  if (e == cudaSuccess) e = launch_backward<MOE_BF16>(p, backward_parts(T, H), st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

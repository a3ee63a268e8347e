// route.cu -- routing: logits -> the k expert ids and gate weights of every
// token (include/moe_ep.h, moe_route).
//
// Mathematics.  Every expert e gets a ranked value: without a bias the logit
// itself (sigmoid and softmax are increasing, so it orders experts as their
// scores do), with a bias the choice s[e] + b[e]; -inf means "not available".
// The k largest are taken one after another; weights are then recomputed for the
// k chosen logits alone, in full precision, one per lane.  Softmax weights that
// are renormalised are exp(l - max of the chosen) over their sum: the sum over
// all experts cancels, so it is not computed.  Sigmoid weights that are renormalised
// take their common factor out first (sigmoid_scaled): small scores have quotients too.
//
// Warp kernel (E <= 1024): one warp per token, a lane holding VPT neighbouring
// experts, so the lowest lane and the lowest position inside it are the lowest
// id; a group has a power of two of lanes.  The cost is instructions, so the k
// rounds are kept short: a lane keeps only its three largest values (eight
// half-rate instructions per two experts) and their order-preserving integer
// keys, a round is one integer warp maximum, one ballot and a pop in the winning
// lane, and positions are looked up once at the end, in the lanes that won.  A
// lane that wins three times looks through its values again (rare: winners
// spread over the lanes; with two values kept it was not).
//
// Measured (in a graph, inputs as warm as they stay): 32,768 tokens x 256 fp32 logits,
// sigmoid with bias, 4 of 8 groups, k = 8: 21.2 us, of which 9.4 are the read, the scan
// and the write, 2.3 the sigmoid and the bias, 5.5 the seven further rounds, 3.8 the
// groups; 49,152 x 768 bf16, plain softmax: 42 us.  Memory would allow 5.3 and 11.6: the
// schedulers issue in 74% of their cycles and wait for the chain of a round in most
// others.  32 tokens: 3.4 us, a launch.  Tried and not faster: 8 or 16 lanes per token (half the instructions, but
// maxima run at half rate and the registers leave few warps: 28-34 us where this
// took 28.7, and 6.8 instead of 3.4 at 1024 tokens); a persistent grid (24 and 49).
#include <algorithm>
#include <type_traits>

#include "moe_ep_internal.cuh"
#include "route_math.cuh"

namespace moe_ep {
namespace {

// The sigmoid that ranks with a bias: the rounded product in the exponent costs s(1-s)|x|
// 2^-24 <= 2^-26, less than the rounding of s itself; 0 and 1 at the infinities.
__device__ __forceinline__ float sigmoid_rank(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;"
      : "=f"(r) : "f"(__fadd_rn(1.0f, exp2_approx(__fmul_rn(x, -kLog2e)))));
  return r;
}
// The same of two numbers.  nz: -0 (see mul2_rn).
__device__ __forceinline__ float2 sigmoid_rank2(float2 x, float nz) {
  const float2 t = mul2_rn(x, bcast2(-kLog2e), nz);
  const float2 d = add2_rn(make_float2(exp2_approx(t.x), exp2_approx(t.y)), bcast2(1.0f));
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  return r;
}

// Rank of a group without a bias, from its two highest logits x1 >= x2 (-inf: none); m:
// the row's maximum (softmax).  The sum of the scores (a softmax's without the common
// divisor) by the full-precision exponential, or, below 2^-100, where the scores leave
// fp32, its logarithm: a negative number, so below every sum, and as increasing.
__device__ __forceinline__ float group_rank(const RouteArgs& r, float x1, float x2, float m) {
  if (!(x1 > kNegInf)) return kNegInf;
  const bool two = r.group_top == 2 && x2 > kNegInf;
  float g, rest;
  if (r.score == MOE_SOFTMAX) {
    x1 = __fsub_rn(x1, m);
    x2 = __fsub_rn(x2, m);
    g = expf(x1);
    if (two) g = __fadd_rn(g, expf(x2));
  } else {
    g = sigmoid_scaled(x1, 0.0f, &rest);
    if (two) g = __fadd_rn(g, sigmoid_scaled(x2, 0.0f, &rest));
  }
  if (g >= 0x1p-100f) return g;
  // (a difference of infinities, from logits 3e38 apart, is a NaN, which fmaxf drops)
  return fmaxf(two ? __fadd_rn(x1, log1pf(expf(__fsub_rn(x2, x1)))) : x1, -kMaxF);
}

// Ids and weights of token t (there: it exists) by W lanes: slots j0 (of this lane)
// and, with H = 2 (k > 32), j0 + 32, from the chosen experts (sel = -1: none).
// m and sum: the softmax's maximum and sum (plain softmax only).
template <int DT, int H, int W>
__device__ __forceinline__ void write_token(const RouteArgs& r, int64_t t, bool there,
                                            const int (&sel)[H], float m, float sum, int j0,
                                            int32_t* idx, float* weights) {
  const auto* row = static_cast<const typename Elem<DT>::T*>(r.logits) + t * r.stride;
  float l[H], s[H];
#pragma unroll
  for (int h = 0; h < H; ++h)
    l[h] = sel[h] >= 0 ? fminf(load_logit<DT>(row + sel[h]), kMaxF) : kNegInf;
  if (r.renormalise) m = lanes_max<W>(H > 1 ? fmaxf(l[0], l[H - 1]) : l[0]);
  if (r.score == MOE_SOFTMAX) {
#pragma unroll
    for (int h = 0; h < H; ++h) s[h] = sel[h] >= 0 ? expf(__fsub_rn(l[h], m)) : 0.0f;
  } else {
    m = r.renormalise ? fminf(m, 0.0f) : 0.0f;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      float rest;
      s[h] = sel[h] >= 0 ? sigmoid_scaled(l[h], m, &rest) : 0.0f;
    }
  }
  float d = 1.0f;
  if (r.renormalise) {
    d = lanes_sum<W>(H > 1 ? __fadd_rn(s[0], s[H - 1]) : s[0]);
    if (d == 0.0f) d = 1.0f;
  } else if (r.score == MOE_SOFTMAX) {
    d = sum;
  }
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int j = j0 + 32 * h;
    if (there && j < r.k) {
      idx[t * r.k + j] = sel[h];
      weights[t * r.k + j] = sel[h] >= 0 ? __fmul_rn(__fdiv_rn(s[h], d), r.scale) : 0.0f;
    }
  }
}

// Tokens per CTA of the warp kernel: as many as write their weights together at
// k <= 8 (8 a CTA: 43 -> 47 us at 768 experts, one writing for itself: 21.9 instead of
// 21.3 at 256).
constexpr int kWarps = 4;

// CTAs that an SM should hold: as many as leave the registers for a lane's logits,
// its biases and about 32 more (a CTA is a warp for each of an SM's four schedulers).
// Occupancy hides the latency of the k rounds, each a
// chain of reduction, ballot and pop: 768 experts a token took 59 us at the 20
// warps the compiler's own choice left, 49 at 32.
constexpr int warp_ctas(int vpt, bool bias) {
  const int ctas = 512 / ((bias ? vpt * 9 / 4 : vpt) + 32);
  return ctas < 12 ? ctas : 12;
}

// vec, vec_bias: rows, and the bias, start at 16-byte boundaries, and so do groups.
template <int DT, int VPT, bool BIAS>
__global__ void __launch_bounds__(kWarps * 32, warp_ctas(VPT, BIAS))
route_warp_kernel(const RouteArgs r, bool vec, bool vec_bias, int group_shift, int per,
                  int32_t* __restrict__ idx, float* __restrict__ weights, float nz,
                  int32_t* dev_status) {
  using T = typename Elem<DT>::T;
  constexpr int kPer16 = 16 / sizeof(T);
  __shared__ int s_sel[kWarps][MOE_EP_MAX_TOPK], s_n[kWarps];
  __shared__ float s_m[kWarps], s_sum[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* chosen = s_sel[warp];
  const bool grouped = r.topk_group < r.n_group;
  // the lane's experts: e0 .. e0 + mine - 1, all of one group of `per` (ungrouped: E)
  const int lanes_per_group = 1 << group_shift;
  const int skip = (lane & (lanes_per_group - 1)) * VPT;
  const int e0 = (lane >> group_shift) * per + skip;
  const int mine = e0 < r.E ? min(per - skip, VPT) : 0;
  const bool want_sum = r.score == MOE_SOFTMAX && (!r.renormalise || BIAS || grouped);

  const int64_t t = int64_t(blockIdx.x) * kWarps + warp;
  wait_for_stream();
  let_next_start();
  if (t >= r.T) return;
  const T* row = static_cast<const T*>(r.logits) + t * r.stride;

  // ---- logits -----------------------------------------------------------------
  float l[VPT];
  if (VPT % kPer16 == 0 && vec && mine == VPT) {
#pragma unroll
    for (int c = 0; c < VPT / kPer16; ++c) {
      const uint4 v = reinterpret_cast<const uint4*>(row + e0)[c];
      unpack_logits<DT>(v, l + c * kPer16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) l[i] = i < mine ? load_logit<DT>(row + e0 + i) : 0.0f;
  }
  float bias[BIAS ? VPT : 1];
  bool odd_bias = false;                // an infinite or NaN bias
  if (BIAS) {
    if (VPT % 4 == 0 && vec_bias && mine == VPT) {
#pragma unroll
      for (int c = 0; c < VPT / 4; ++c) {
        const float4 v = reinterpret_cast<const float4*>(r.bias + e0)[c];
        bias[4 * c] = v.x;
        bias[4 * c + 1] = v.y;
        bias[4 * c + 2] = v.z;
        bias[4 * c + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) bias[i] = i < mine ? r.bias[e0 + i] : 0.0f;
    }
    float2 all = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < VPT; i += 2) all = add2_rn(all, make_float2(bias[i], bias[i + 1]));
    odd_bias = __any_sync(kAll, !(fabsf(__fadd_rn(all.x, all.y)) <= kMaxF));
  }
  // The sum shows what is special: NaN or +inf in it if there is one among the
  // logits, -inf if only that (or an overflow, which does no harm).  NaN is -inf
  // and reported, +inf the largest finite number.
  float2 all = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < VPT; i += 2) all = add2_rn(all, make_float2(l[i], l[i + 1]));
  const float probe = __fadd_rn(all.x, all.y);
  const bool odd = __any_sync(kAll, !(probe <= kMaxF));
  if (odd) {
    bool nan = false;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      nan |= l[i] != l[i];
      l[i] = l[i] != l[i] ? kNegInf : fminf(l[i], kMaxF);
    }
    if (nan) set_status(dev_status, MOE_ERR_INVALID_ARG);
  }
  if (VPT * 32 > r.E) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (i >= mine) l[i] = kNegInf;
  }

  // the lane's three largest: the largest, second and third of two ordered lists
  float v1, v2, v3;
  auto scan = [&]() {
    v1 = v2 = v3 = kNegInf;
#pragma unroll
    for (int i = 0; i < VPT; i += 2) {
      const float hi = fmaxf(l[i], l[i + 1]), lo = fminf(l[i], l[i + 1]);
      if (VPT > 2) v3 = fmaxf(fmaxf(v3, fminf(v2, hi)), fminf(v1, lo));
      v2 = fmaxf(fmaxf(v2, fminf(v1, hi)), lo);
      v1 = fmaxf(v1, hi);
    }
  };
  if (!BIAS) scan();                     // the logits rank themselves

  // ---- the softmax's maximum and sum, where a weight or a choice needs them -----
  float m = 0.0f, sum = 1.0f;
  if (want_sum) {
    if (!BIAS) {
      m = v1;
    } else {
      m = l[0];
#pragma unroll
      for (int i = 1; i < VPT; ++i) m = fmaxf(m, l[i]);
    }
    m = fmaxf(warp_max(m), -kMaxF);
    float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < VPT; i += 2)
      part = add2_rn(part, exp_neg2(add2_rn(make_float2(l[i], l[i + 1]), bcast2(-m)), nz));
    sum = warp_sum(__fadd_rn(part.x, part.y));
    if (sum == 0.0f) sum = 1.0f;
  }

  // ---- ranked values with a bias --------------------------------------------------
  if (BIAS) {
    const float inv_sum = want_sum ? __fdiv_rn(1.0f, sum) : 1.0f;
    // every: every value is an expert's finite logit, the usual case
    auto rank = [&](auto every, auto&& f) {
#pragma unroll
      for (int i = 0; i < VPT; i += 2) {
        const float2 c = add2_rn(f(make_float2(l[i], l[i + 1])), make_float2(bias[i], bias[i + 1]));
        l[i] = decltype(every)::value || l[i] > kNegInf ? c.x : kNegInf;
        l[i + 1] = decltype(every)::value || l[i + 1] > kNegInf ? c.y : kNegInf;
      }
    };
    auto soft = [&](float2 x) {
      return mul2_rn(exp_neg2(add2_rn(x, bcast2(-m)), nz), bcast2(inv_sum), nz);
    };
    auto sigmoid = [&](float2 x) { return sigmoid_rank2(x, nz); };
    const std::true_type yes;
    const std::false_type no;
    if (r.score == MOE_SOFTMAX) rank(no, soft);
    else if (VPT * 32 > r.E || __any_sync(kAll, !(fabsf(probe) <= kMaxF))) rank(no, sigmoid);
    else rank(yes, sigmoid);
    if (odd_bias) {                      // a NaN choice is no choice
#pragma unroll
      for (int i = 0; i < VPT; ++i) l[i] = l[i] > kNegInf ? l[i] : kNegInf;
    }
    scan();
  }

  // ---- groups: a power of two of lanes each ----------------------------------------
  if (grouped) {
    float a1 = v1, a2 = v2;
    for (int d = 1; d < lanes_per_group; d <<= 1) {
      const float b1 = __shfl_xor_sync(kAll, a1, d), b2 = __shfl_xor_sync(kAll, a2, d);
      a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
      a1 = fmaxf(a1, b1);
    }
    const float gs = !BIAS                               ? group_rank(r, a1, a2, m)
                     : r.group_top == 2 && a2 > kNegInf ? __fadd_rn(a1, a2)
                                                        : a1;
    uint32_t key = gs > kNegInf ? order_key(gs) : 0u;
    const int head = lane & -lanes_per_group;        // the group's first lane
    bool keep = false;
    for (int i = 0; i < r.topk_group; ++i) {
      const uint32_t best = __reduce_max_sync(kAll, key);
      if (best == 0) break;
      if (__ffs(__ballot_sync(kAll, key == best)) - 1 == head) {
        keep = true;
        key = 0u;
      }
    }
    if (!keep) v1 = v2 = v3 = kNegInf;
  }

  // ---- the k largest ---------------------------------------------------------------
  // keys of the values still to win; kAgain: the lane must look for more
  constexpr uint32_t kAgain = 0xffffffffu;
  uint32_t q1, q2, q3, wins = 0;       // wins: slot + 1 of the lane's 1st, 2nd, 3rd value
  int won = 0;                         // 8 * wins so far
  auto keys = [&]() {
    q1 = v1 > kNegInf ? order_key(v1) : 0u;
    q2 = v2 > kNegInf ? order_key(v2) : 0u;
    q3 = v3 > kNegInf ? order_key(v3) : 0u;
  };
  keys();
  // writes down the lane's wins; the positions of v1, v2, v3 where they won
  auto settle = [&]() {
    int i1 = -1, i2 = -1, i3 = -1;
#pragma unroll
    for (int i = VPT - 1; i >= 0; --i)
      if (l[i] == v1) i1 = i;
    if (__any_sync(kAll, won > 8)) {
#pragma unroll
      for (int i = VPT - 1; i >= 0; --i)
        if (l[i] == v2 && i != i1) i2 = i;
      if (__any_sync(kAll, won > 16)) {
#pragma unroll
        for (int i = VPT - 1; i >= 0; --i)
          if (l[i] == v3 && i != i1 && i != i2) i3 = i;
      }
    }
    if (won > 0) chosen[(wins & 255u) - 1] = e0 + i1;
    if (won > 8) chosen[((wins >> 8) & 255u) - 1] = e0 + i2;
    if (won > 16) chosen[((wins >> 16) & 255u) - 1] = e0 + i3;
    return make_int3(i1, i2, i3);
  };
  int n = 0;
  while (n < r.k) {
    const uint32_t best = __reduce_max_sync(kAll, q1);
    if (best - 1u >= kAgain - 1u) {    // rare: nothing left, or a lane must look again
      if (best == 0) break;
      const int3 at = settle();
      if (q1 == kAgain) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
          if (i == at.x || i == at.y || i == at.z) l[i] = kNegInf;
        scan();
        keys();
        wins = 0;
        won = 0;
      }
      continue;
    }
    const int win = __ffs(__ballot_sync(kAll, q1 == best)) - 1;
    ++n;
    if (lane == win) {
      wins |= static_cast<uint32_t>(n) << won;
      won += 8;
      q1 = q2;
      q2 = q3;
      q3 = VPT > 3 ? kAgain : 0u;
    }
  }
  settle();

  // ---- ids and weights: 8, 16 or 32 lanes per token, one warp for several tokens --------
  if (lane == 0) {
    s_n[warp] = n;
    s_m[warp] = m;
    s_sum[warp] = sum;
  }
  __syncthreads();
  auto write = [&](auto h, auto w) {
    constexpr int H = decltype(h)::value, W = decltype(w)::value;
    if (warp % (32 / W) != 0) return;
    const int from = warp + lane / W, j0 = lane % W;   // the token's warp
    const int64_t t = int64_t(blockIdx.x) * kWarps + from;
    const bool there = t < r.T;
    const int n = there ? s_n[from] : 0;
    int sel[H];
#pragma unroll
    for (int i = 0; i < H; ++i) sel[i] = j0 + 32 * i < n ? s_sel[from][j0 + 32 * i] : -1;
    write_token<DT, H, W>(r, t, there, sel, s_m[from], s_sum[from], j0, idx, weights);
  };
  const std::integral_constant<int, 1> one;
  if (r.k <= 8) write(one, std::integral_constant<int, 8>());
  else if (r.k <= 16) write(one, std::integral_constant<int, 16>());
  else if (r.k <= 32) write(one, std::integral_constant<int, 32>());
  else write(std::integral_constant<int, 2>(), std::integral_constant<int, 32>());
}

// Any E up to MOE_EP_MAX_EXPERTS and any groups: one CTA per token (persistent
// grid), ranking keys and choices in shared memory, a block-wide maximum of
// (key, lowest id) per chosen expert.  4096 tokens x 2048 fp32, sigmoid: 42 us (5.0 of
// reads), in 64 groups of which 8 stay 106; x 4096 bf16, softmax 95; 32,768 x 320 in 40
// groups 209 (6.5): every token pays the CTA's barriers, two per chosen expert, and a
// thread scores a whole group by itself.
constexpr int kWideThreads = 128;

template <int DT>
__global__ void __launch_bounds__(kWideThreads)
route_wide_kernel(const RouteArgs r, int32_t* __restrict__ idx, float* __restrict__ weights,
                  int32_t* dev_status) {
  using T = typename Elem<DT>::T;
  extern __shared__ uint32_t s_dyn[];
  uint32_t* key = s_dyn;                                       // [E]
  float* choice = reinterpret_cast<float*>(s_dyn + r.E);       // [E], logits without a bias
  float* gscore = choice + r.E;                                // [n_group]
  __shared__ float s_red[kWideThreads / 32];
  __shared__ uint64_t s_best[2][kWideThreads / 32];
  __shared__ int s_sel[MOE_EP_MAX_TOPK];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool grouped = r.topk_group < r.n_group;
  const int per = r.E / r.n_group;

  wait_for_stream();
  let_next_start();
  for (int64_t t = blockIdx.x; t < r.T; t += gridDim.x) {
    const T* row = static_cast<const T*>(r.logits) + t * r.stride;
    auto logit = [&](int e) {
      const float l = load_logit<DT>(row + e);
      return l != l ? kNegInf : fminf(l, kMaxF);
    };
    float m = kNegInf, sum = 0.0f;
    bool nan = false;
    for (int e = tid; e < r.E; e += kWideThreads) {
      const float l = load_logit<DT>(row + e);
      nan |= l != l;
      m = fmaxf(m, logit(e));
    }
    if (nan) set_status(dev_status, MOE_ERR_INVALID_ARG);
    if (r.score == MOE_SOFTMAX) {
      m = warp_max(m);
      if (lane == 0) s_red[warp] = m;
      __syncthreads();
      m = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
      m = fmaxf(m, -kMaxF);
      __syncthreads();
      for (int e = tid; e < r.E; e += kWideThreads) {
        const float l = logit(e);
        sum = __fadd_rn(sum, exp_neg(__fsub_rn(l, m)));
      }
      sum = warp_sum(sum);
      if (lane == 0) s_red[warp] = sum;
      __syncthreads();
      sum = __fadd_rn(__fadd_rn(s_red[0], s_red[1]), __fadd_rn(s_red[2], s_red[3]));
    }
    if (sum == 0.0f) sum = 1.0f;
    const float inv_sum = __fdiv_rn(1.0f, sum);
    for (int e = tid; e < r.E; e += kWideThreads) {
      const float l = logit(e);
      float c = l;
      if (r.bias) {
        c = r.score == MOE_SOFTMAX ? __fmul_rn(exp_neg(__fsub_rn(l, m)), inv_sum)
                                   : sigmoid_rank(l);
        c = __fadd_rn(c, r.bias[e]);
      }
      const bool on = l > kNegInf && c > kNegInf;
      key[e] = on ? order_key(c) : 0u;
      choice[e] = on ? c : kNegInf;
    }
    __syncthreads();
    if (grouped) {
      for (int g = tid; g < r.n_group; g += kWideThreads) {
        float a1 = kNegInf, a2 = kNegInf;
        for (int i = 0; i < per; ++i) {
          const float c = choice[g * per + i];
          a2 = fmaxf(fminf(a1, c), a2);
          a1 = fmaxf(a1, c);
        }
        gscore[g] = !r.bias                            ? group_rank(r, a1, a2, m)
                    : r.group_top == 2 && a2 > kNegInf ? __fadd_rn(a1, a2)
                                                       : a1;
      }
      __syncthreads();
      for (int g = tid; g < r.n_group; g += kWideThreads) {
        const float gs = gscore[g];
        int better = 0;
        for (int o = 0; o < r.n_group; ++o)
          better += gscore[o] > gs || (gscore[o] == gs && o < g);
        if (better >= r.topk_group)
          for (int i = 0; i < per; ++i) key[g * per + i] = 0u;
      }
      __syncthreads();
    }
    // (key, ~id): the larger key, then the lower id.  Every thread keeps the
    // best of its experts and looks again when it loses it.
    auto own_best = [&]() {
      uint64_t b = 0;
      for (int e = tid; e < r.E; e += kWideThreads) {
        const uint64_t v = uint64_t(key[e]) << 32 | uint32_t(~e);
        if (key[e] != 0 && v > b) b = v;
      }
      return b;
    };
    uint64_t own = own_best();
    int n = 0;
    for (; n < r.k; ++n) {
      uint64_t b = own;
#pragma unroll
      for (int d = 16; d; d >>= 1) {
        const uint64_t o = __shfl_xor_sync(kAll, b, d);
        b = o > b ? o : b;
      }
      if (lane == 0) s_best[n & 1][warp] = b;
      __syncthreads();
      b = s_best[n & 1][0];
      for (int i = 1; i < kWideThreads / 32; ++i)
        b = s_best[n & 1][i] > b ? s_best[n & 1][i] : b;
      if (b == 0) break;
      const int e = static_cast<int>(~uint32_t(b));
      if (tid == 0) s_sel[n] = e;
      if (b == own) {
        key[e] = 0u;
        own = own_best();
      }
    }
    __syncthreads();
    if (warp == 0) {
      const int sel[2] = {lane < n ? s_sel[lane] : -1, lane + 32 < n ? s_sel[lane + 32] : -1};
      write_token<DT, 2, 32>(r, t, true, sel, m, sum, lane, idx, weights);
    }
    __syncthreads();
  }
}

template <int DT, int VPT, bool BIAS>
cudaError_t launch_bias(const RouteArgs& r, int group_shift, int32_t* idx, float* weights,
                        int32_t* dev_status, cudaStream_t st) {
  const size_t el = DT == MOE_FP32 ? 4 : 2;
  const bool grouped = r.topk_group < r.n_group;
  const int per = grouped ? r.E / r.n_group : r.E;
  const bool vec = reinterpret_cast<uintptr_t>(r.logits) % 16 == 0 && r.stride * el % 16 == 0 &&
                   (!grouped || per * el % 16 == 0);
  const bool vec_bias =
      reinterpret_cast<uintptr_t>(r.bias) % 16 == 0 && (!grouped || per % 4 == 0);
  return launch_early(route_warp_kernel<DT, VPT, BIAS>, (r.T + kWarps - 1) / kWarps, kWarps * 32,
                      0, st, r, vec, vec_bias, group_shift, per, idx, weights, -0.0f, dev_status);
}

template <int DT, int VPT>
cudaError_t launch_warp(const RouteArgs& r, int group_shift, int32_t* idx, float* weights,
                        int32_t* dev_status, cudaStream_t st) {
  return r.bias ? launch_bias<DT, VPT, true>(r, group_shift, idx, weights, dev_status, st)
                : launch_bias<DT, VPT, false>(r, group_shift, idx, weights, dev_status, st);
}

// The warp kernel's experts per lane: the smallest of its sizes that holds E or,
// with groups in play, a group in its power of two of lanes (for the butterfly
// that joins their best choices); 0 where there is none.
int experts_per_lane(const RouteArgs& r, int* group_shift) {
  const bool grouped = r.topk_group < r.n_group;
  const int groups = grouped ? r.n_group : 1, per = r.E / groups;
  *group_shift = 5;
  while (*group_shift >= 0 && (groups << *group_shift) > 32) --*group_shift;
  if (*group_shift < 0) return 0;
  for (const int v : {2, 4, 8, 16, 24, 32})
    if ((v << *group_shift) >= per) return v;
  return 0;
}

template <int DT>
cudaError_t launch_t(const RouteArgs& r, int32_t* idx, float* weights, int32_t* dev_status,
                     cudaStream_t st) {
  int shift = 5;
  switch (experts_per_lane(r, &shift)) {
    case 2: return launch_warp<DT, 2>(r, shift, idx, weights, dev_status, st);
    case 4: return launch_warp<DT, 4>(r, shift, idx, weights, dev_status, st);
    case 8: return launch_warp<DT, 8>(r, shift, idx, weights, dev_status, st);
    case 16: return launch_warp<DT, 16>(r, shift, idx, weights, dev_status, st);
    case 24: return launch_warp<DT, 24>(r, shift, idx, weights, dev_status, st);
    case 32: return launch_warp<DT, 32>(r, shift, idx, weights, dev_status, st);
    default: break;
  }
  const size_t smem = (2 * size_t(r.E) + r.n_group) * 4;
  const void* fn = reinterpret_cast<const void*>(route_wide_kernel<DT>);
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e == cudaSuccess) e = kernel_blocks_per_sm(fn, kWideThreads, smem, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t grid = std::min<int64_t>(r.T, int64_t(std::max(1, per_sm)) * sms);
  return launch_early(route_wide_kernel<DT>, grid, kWideThreads, smem, st, r, idx, weights,
                      dev_status);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& r, int32_t* topk_idx, float* topk_weights,
                         int32_t* dev_status, cudaStream_t st) {
  switch (r.dtype) {
    case MOE_BF16: return launch_t<MOE_BF16>(r, topk_idx, topk_weights, dev_status, st);
    case MOE_FP16: return launch_t<MOE_FP16>(r, topk_idx, topk_weights, dev_status, st);
    default: return launch_t<MOE_FP32>(r, topk_idx, topk_weights, dev_status, st);
  }
}

}  // namespace moe_ep

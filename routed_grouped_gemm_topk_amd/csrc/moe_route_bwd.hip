// Gradient of the router producer (moe_route): d_weights [T, K] -> d_logits [T, E].
//
// With p = softmax(logits[t, :]) and c_j = topk_ids[t, j], moe_route's weights are
//   w_j = p[c_j]                    d w_j / d l_e = w_j (delta(e, c_j) - p_e)
//   w_j = p[c_j] / sum_i p[c_i]     the softmax over the chosen logits alone
// so with G = sum_j w_j dw_j the gradient is
//   d_l[e] = sum_{j: c_j = e} w_j dw_j - p_e G            (not renormalised)
//   d_l[e] = sum_{j: c_j = e} w_j (dw_j - G)              (renormalised; 0 if not chosen).
// The selection itself is piecewise constant and adds nothing.
#include "moe_route.h"

namespace moe {

constexpr int kRouteBwdThreads = 256;
constexpr int kRouteBwdTokens = kRouteBwdThreads / kWave;

// One wavefront per token.  Lane l holds p of experts l, l+64, ...; lane j < K holds slot j.
// Every sum is a wavefront all-reduction in fp32; a slot's term reaches the lane that holds its
// expert by a lane broadcast, slots in ascending j, so the result does not depend on timing.
// Bounded by latency: 2048 tokens of 256 experts, top 8, take 4.3 us (4.3 MB, 0.9 us at the rate
// of a copy), 4096 of 8 experts, top 2, 3.1 us.
template <int LPL>
__global__ __launch_bounds__(kRouteBwdThreads) void route_bwd_kernel(
    const float* __restrict__ logits, int T, int E, int K, int renorm,
    const int32_t* __restrict__ topk_ids, const float* __restrict__ d_w,
    float* __restrict__ d_logits) {
  const int lane = threadIdx.x & (kWave - 1);
  const int t = blockIdx.x * kRouteBwdTokens + threadIdx.x / kWave;
  if (t >= T) return;
  const float* lg = logits + (size_t)t * E;
  int id = -1;
  float dw = 0.0f, l = -INFINITY;
  if (lane < K) {
    id = topk_ids[(size_t)t * K + lane];
    dw = d_w[(size_t)t * K + lane];
  }
  const bool chosen = (uint32_t)id < (uint32_t)E;   // an id outside [0,E) names no logit
  if (chosen) l = lg[id];
  const auto add = [](float a, float b) { return a + b; };
  const auto larger = [](float a, float b) { return fmaxf(a, b); };

  float p[LPL];
  float w;
  if (renorm) {
    const float m = wave_allreduce(l, larger);
    w = chosen ? expf(l - m) : 0.0f;
    const float s = wave_allreduce(w, add);
    w = chosen ? w / s : 0.0f;
    #pragma unroll
    for (int i = 0; i < LPL; ++i) p[i] = 0.0f;
  } else {
    float m = -INFINITY;
    #pragma unroll
    for (int i = 0; i < LPL; ++i) {
      const int e = lane + kWave * i;
      p[i] = (e < E) ? lg[e] : -INFINITY;
      m = fmaxf(m, p[i]);
    }
    m = wave_allreduce(m, larger);
    float s = 0.0f;
    #pragma unroll
    for (int i = 0; i < LPL; ++i) {
      p[i] = (lane + kWave * i < E) ? expf(p[i] - m) : 0.0f;
      s += p[i];
    }
    s = wave_allreduce(s, add);
    #pragma unroll
    for (int i = 0; i < LPL; ++i) p[i] /= s;
    w = chosen ? expf(l - m) / s : 0.0f;
  }
  const float term = chosen ? w * dw : 0.0f;
  const float G = wave_allreduce(term, add);
  float d[LPL];
  #pragma unroll
  for (int i = 0; i < LPL; ++i) d[i] = renorm ? 0.0f : -p[i] * G;
  const float mine = renorm ? (chosen ? w * (dw - G) : 0.0f) : term;
  for (int j = 0; j < K; ++j) {
    const int e = __builtin_amdgcn_readlane(chosen ? id : -1, j);
    const float v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(
                        __builtin_bit_cast(int, mine), j));
    #pragma unroll
    for (int i = 0; i < LPL; ++i)
      if (lane + kWave * i == e) d[i] += v;
  }
  float* o = d_logits + (size_t)t * E;
  #pragma unroll
  for (int i = 0; i < LPL; ++i) {
    const int e = lane + kWave * i;
    if (e < E) o[e] = d[i];
  }
}

hipError_t launch_route_bwd(const Resolved& r, const float* logits, int renorm,
                            const int32_t* topk_ids, const float* d_w, float* d_logits,
                            hipStream_t s) {
  const unsigned blocks = (unsigned)((r.T + kRouteBwdTokens - 1) / kRouteBwdTokens);
  switch (route_lpl(r.E)) {
#define MOE_ROUTE_BWD_CASE(L)                                                                   \
  case L:                                                                                      \
    hipLaunchKernelGGL(route_bwd_kernel<L>, dim3(blocks), dim3(kRouteBwdThreads), 0, s, logits, \
                       r.T, r.E, r.K, renorm, topk_ids, d_w, d_logits);                        \
    break;
    MOE_ROUTE_BWD_CASE(1)
    MOE_ROUTE_BWD_CASE(2)
    MOE_ROUTE_BWD_CASE(4)
    MOE_ROUTE_BWD_CASE(8)
    MOE_ROUTE_BWD_CASE(16)
#undef MOE_ROUTE_BWD_CASE
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace moe

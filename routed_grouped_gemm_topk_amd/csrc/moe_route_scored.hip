// Router producer with scores, a bias for balance and groups of experts, and its gradient.
//
//   s_e = softmax(l)_e | 1 / (1 + exp(-l_e)),   c_e = s_e + bias_e
//   the topk_groups groups of the largest sum of their group_top largest c are kept; the top_k
//   experts of the largest c among them; w_j = scale * s_j (/ sum_i s_i of the chosen)
//
// One wavefront per token, four tokens per workgroup.  A group's experts lie on LG = 64 / (n_groups
// rounded up to a power of two) neighbouring lanes: expert g * GS + sub + LG * i (GS = E / n_groups)
// is item i of lane g * LG + sub, so that a group's value is a butterfly over its lanes, and without
// groups item i of lane l is expert l + 64 i.
#include <type_traits>

#include "moe_route.h"

namespace moe {

namespace rs {

constexpr int kThreads = 256;
constexpr int kTokens = kThreads / kWave;

struct Args {
  const void* logits;           // [T, E] fp32 or bf16
  const float* bias;            // [E] or null
  int32_t* ids;                 // [T, K]
  float* w;
  int T, E, K;
  int bf16, sigmoid, renorm;
  int groups, kept, top;        // groups, groups kept, scores that make a group's value
  int gs, lg;                   // experts of a group, log2 of the lanes of a group
  float scale;
};

// -inf and NaN take the expert out, +inf counts as the largest finite logit.
__device__ __forceinline__ float clean(float l) {
  return l > -INFINITY ? fminf(l, 3.40282347e38f) : -INFINITY;
}

__device__ __forceinline__ float load_logit(const void* p, int64_t at, bool bf16) {
  return clean(bf16 ? bf16_bits_to_f32(((const uint16_t*)p)[at]) : ((const float*)p)[at]);
}

__device__ __forceinline__ float bcast(float v, int lane) {
  return __builtin_bit_cast(float,
                            __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
__device__ __forceinline__ double bcast(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ double wave_sum(double v) {
  #pragma unroll
  for (int d = 1; d < kWave; d *= 2) v += __shfl_xor(v, d, kWave);
  return v;
}

__device__ __forceinline__ float wave_max(float v) {
  return wave_allreduce(v, [](float a, float b) { return fmaxf(a, b); });
}

// exp(l - m) in fp32 for l <= m: what the subtraction rounds off is put back (relative error 3 u,
// u = 2^-24, whatever l - m is).
__device__ __forceinline__ float exp_diff(float l, float m) {
  const float d = l - m, back = d - l;
  const float rest = (l - (d - back)) - (m + back);
  const float e = expf(d);
  return d > -104.0f ? __builtin_fmaf(e, rest, e) : 0.0f;      // below it e is 0, and rest may be NaN
}

struct Token {
  int64_t t;
  int lane, grp, sub, e0;       // lane, its group, its place in it, its first expert
};

// The choice and the weights in fp32; returns false, having stored nothing, where fp32 does not tell
// two experts or groups apart that the choice depends on.  Every lane of the wave must be active.
//
// Errors (u = 2^-24): a sigmoid score is at most 1 and 5 u of itself off; a softmax score p is 3 u
// of itself off for its exponential, 3 u and an addition's u for each of LPL + 6 for the sum, 1 u for
// the quotient, and at most 1 / total; a choice score c another u |c| for the addition of the bias, a
// sum of two the errors of both and its own.  Two that differ by more than both errors are in the
// right order.  Where the logits themselves are compared, only equal ones are uncertain.
template <int LPL, bool SCORES>
__device__ __forceinline__ bool route_fast(const Args& g, const Token& at, const float (&l)[LPL]) {
  constexpr float U = 0x1p-24f;
  float m = 0.0f, total = 1.0f, sure = 0.0f;   // sure: error of the scores of two experts
  float s[LPL], c[LPL];
  if (!g.sigmoid) {
    m = -INFINITY;
    #pragma unroll
    for (int i = 0; i < LPL; ++i) m = fmaxf(m, l[i]);
    m = wave_max(m);
    if (m == -INFINITY) m = 0.0f;
    float sum = 0.0f;
    #pragma unroll
    for (int i = 0; i < LPL; ++i) {
      s[i] = exp_diff(l[i], m);
      sum += s[i];
    }
    if (SCORES || !g.renorm) total = wave_allreduce(sum, [](float a, float b) { return a + b; });
    if (SCORES) sure = 2 * (LPL + 13) * U / total;
  } else {
    #pragma unroll
    for (int i = 0; i < LPL; ++i) s[i] = 1.0f / (1.0f + expf(-l[i]));
    sure = 2 * 5 * U;
  }
  #pragma unroll
  for (int i = 0; i < LPL; ++i) {
    c[i] = l[i];
    if (SCORES && l[i] > -INFINITY) {
      const float b = g.bias ? g.bias[at.e0 + (i << g.lg)] : 0.0f;
      c[i] = b > -INFINITY ? (g.sigmoid ? s[i] : s[i] / total) + b : -INFINITY;
    }
  }
  auto apart = [&](float hi, float lo, float err) {
    return hi - lo > (SCORES ? err + 4 * U * (fabsf(hi) + fabsf(lo)) : 0.0f);
  };
  bool ok = true;
  if (g.kept < g.groups) {
    float v1 = -INFINITY, v2 = -INFINITY;
    #pragma unroll
    for (int i = 0; i < LPL; ++i) {
      v2 = fmaxf(v2, fminf(v1, c[i]));
      v1 = fmaxf(v1, c[i]);
    }
    for (int d = 1; d < (1 << g.lg); d *= 2) {
      const float o1 = __shfl_xor(v1, d, kWave), o2 = __shfl_xor(v2, d, kWave);
      v2 = fmaxf(fminf(v1, o1), fmaxf(v2, o2));
      v1 = fmaxf(v1, o1);
    }
    const float value = g.top == 2 && v2 > -INFINITY ? v1 + v2 : v1;
    // a sum's error is at most that of its two scores, each off by u |c|, |c| <= |v1| + |v2|
    const float size = fabsf(v1) + (v2 > -INFINITY ? fabsf(v2) : 0.0f);
    int before = 0;             // groups that come before this lane's
    bool close = false;
    for (int o = 0; o < g.groups; ++o) {
      const float ov = bcast(value, o << g.lg), os = bcast(size, o << g.lg);
      before += ov > value;
      close |= o != at.grp && !(fabsf(ov - value) > (SCORES ? 2 * sure + 4 * U * (os + size) : 0.0f));
    }
    ok = __ballot(close && at.grp < g.groups) == 0;
    if (before >= g.kept) {
      #pragma unroll
      for (int i = 0; i < LPL; ++i) c[i] = -INFINITY;
    }
  }
  int round[LPL];               // the round in which the item was chosen
  #pragma unroll
  for (int i = 0; i < LPL; ++i) round[i] = -1;
  float prev = INFINITY;
  int found = 0;
  for (int j = 0; j <= g.K; ++j) {       // one more than are chosen, for the last one's margin
    float best = c[0];
    #pragma unroll
    for (int i = 1; i < LPL; ++i) best = fmaxf(best, c[i]);
    best = wave_max(best);
    if (best == -INFINITY) break;
    ok = ok && (j == 0 || apart(prev, best, sure));
    if (j == g.K) break;
    int n = 0;
    #pragma unroll
    for (int i = 0; i < LPL; ++i) {
      const bool is = c[i] == best;
      n += __popcll(__ballot(is));
      round[i] = is ? j : round[i];
      c[i] = is ? -INFINITY : c[i];
    }
    ok = ok && n == 1;
    prev = best;
    found = j + 1;
  }
  if (!ok) return false;
  if (g.renorm) {
    float sum = 0.0f;
    if (!g.sigmoid) {           // relative to the largest chosen, which may be far below m
      float top = -INFINITY;
      #pragma unroll
      for (int i = 0; i < LPL; ++i) top = fmaxf(top, round[i] >= 0 ? l[i] : -INFINITY);
      top = fmaxf(wave_max(top), -3.40282347e38f);
      if (top != m) {
        #pragma unroll
        for (int i = 0; i < LPL; ++i) s[i] = exp_diff(l[i], fmaxf(top, l[i]));
      }
    }
    #pragma unroll
    for (int i = 0; i < LPL; ++i) sum += round[i] >= 0 ? s[i] : 0.0f;
    total = wave_allreduce(sum, [](float a, float b) { return a + b; });
    if (g.sigmoid && total < 0x1p-100f) return false;    // their ratios need 64 bits
  }
  const bool divide = g.renorm || !g.sigmoid;
  #pragma unroll
  for (int i = 0; i < LPL; ++i) {
    if (round[i] < 0) continue;
    const float w = divide ? (total > 0.0f ? s[i] / total : 0.0f) : s[i];
    g.ids[at.t * g.K + round[i]] = at.e0 + (i << g.lg);
    g.w[at.t * g.K + round[i]] = w * g.scale;
  }
  if (at.lane >= found && at.lane < g.K) {
    g.ids[at.t * g.K + at.lane] = -1;
    g.w[at.t * g.K + at.lane] = 0.0f;
  }
  return true;
}

// The same with scores, group values and weights in 64 bits (SCORES) and ties to the lowest ids.
template <int LPL, bool SCORES>
__device__ __forceinline__ void route_exact(const Args& g, const Token& at_, const float (&l)[LPL]) {
  using C = typename std::conditional<SCORES, double, float>::type;
  constexpr C NONE = -INFINITY;
  const int lane = at_.lane, grp = at_.grp, e0 = at_.e0;
  const int64_t t = at_.t;
  float m = 0.0f;               // softmax: the largest logit, 0 without any
  double total = 0.0;           // softmax: the sum of exp(l - m)
  if (!g.sigmoid && (SCORES || !g.renorm)) {
    m = -INFINITY;
    #pragma unroll
    for (int i = 0; i < LPL; ++i) m = fmaxf(m, l[i]);
    m = wave_max(m);
    if (m == -INFINITY) m = 0.0f;
  }
  C c[LPL];                     // choice scores
  if constexpr (SCORES) {
    #pragma unroll
    for (int i = 0; i < LPL; ++i) {
      c[i] = g.sigmoid ? 1.0 / (1.0 + exp(-(double)l[i])) : exp((double)l[i] - (double)m);
      total += c[i];
    }
    if (!g.sigmoid) {
      total = wave_sum(total);
      #pragma unroll
      for (int i = 0; i < LPL; ++i) c[i] /= total;
    }
    #pragma unroll
    for (int i = 0; i < LPL; ++i) {
      if (l[i] == -INFINITY) {
        c[i] = NONE;
      } else if (g.bias) {
        const float b = g.bias[e0 + (i << g.lg)];
        c[i] = b > -INFINITY ? c[i] + (double)b : NONE;
      }
    }
  } else {
    #pragma unroll
    for (int i = 0; i < LPL; ++i) c[i] = l[i];
    if (!g.sigmoid && !g.renorm) {
      float sum = 0.0f;
      #pragma unroll
      for (int i = 0; i < LPL; ++i) sum += expf(l[i] - m);      // 0 for a lane without the item
      total = wave_allreduce(sum, [](float a, float b) { return a + b; });
    }
  }

  if (g.kept < g.groups) {
    C v1 = NONE, v2 = NONE;     // the lane's two largest, then the group's
    #pragma unroll
    for (int i = 0; i < LPL; ++i) {
      v2 = c[i] > v1 ? v1 : (c[i] > v2 ? c[i] : v2);
      v1 = c[i] > v1 ? c[i] : v1;
    }
    for (int d = 1; d < (1 << g.lg); d *= 2) {
      const C o1 = __shfl_xor(v1, d, kWave), o2 = __shfl_xor(v2, d, kWave);
      const C low = o1 > v1 ? v1 : o1, high = o2 > v2 ? o2 : v2;
      v1 = o1 > v1 ? o1 : v1;
      v2 = low > high ? low : high;
    }
    const C value = g.top == 2 && v2 > NONE ? v1 + v2 : v1;
    int before = 0;             // groups that come before this lane's
    for (int o = 0; o < g.groups; ++o) {
      const C ov = bcast(value, o << g.lg);
      before += ov > value || (ov == value && o < grp);
    }
    if (before >= g.kept) {
      #pragma unroll
      for (int i = 0; i < LPL; ++i) c[i] = NONE;
    }
  }

  // top_k rounds.  Rounding the scores to fp32 keeps their order, so the largest fp32 value names
  // the winner unless several lanes hold it; then their full scores and ids decide.
  int my_id = -1, my_lane = 0, my_item = 0;
  for (int j = 0; j < g.K; ++j) {
    C best = NONE;
    int item = 0;
    #pragma unroll
    for (int i = 0; i < LPL; ++i) {
      if (c[i] > best) {        // items ascend in id: the first of equals
        best = c[i];
        item = i;
      }
    }
    const float a = (float)best;
    const float top = wave_max(a);
    if (top == -INFINITY) break;                       // no expert is left
    uint64_t at = __ballot(a == top);
    int win = __builtin_ctzll(at);
    const int id = e0 + (item << g.lg);
    int win_id = __builtin_amdgcn_readlane(id, win);
    if (at & (at - 1)) {
      C win_v = bcast(best, win);
      for (at &= at - 1; at; at &= at - 1) {
        const int o = __builtin_ctzll(at);
        const C ov = bcast(best, o);
        const int oid = __builtin_amdgcn_readlane(id, o);
        if (ov > win_v || (ov == win_v && oid < win_id)) {
          win = o;
          win_v = ov;
          win_id = oid;
        }
      }
    }
    const int win_item = __builtin_amdgcn_readlane(item, win);
    #pragma unroll
    for (int i = 0; i < LPL; ++i)
      if (lane == win && i == win_item) c[i] = NONE;
    if (lane == j) {
      my_id = win_id;
      my_lane = win;
      my_item = win_item;
    }
  }

  // lane j: the weight of slot j, in 64 bits
  float lj = -INFINITY;
  #pragma unroll
  for (int i = 0; i < LPL; ++i) {
    const float v = __shfl(l[i], my_lane, kWave);
    if (my_id >= 0 && i == my_item) lj = v;
  }
  double s;
  if (g.sigmoid) {
    s = 1.0 / (1.0 + exp(-(double)lj));
  } else {
    if (g.renorm) m = fmaxf(wave_max(lj), -3.40282347e38f);     // the largest chosen
    s = exp((double)lj - (double)m);
  }
  if (my_id < 0) s = 0.0;
  if (g.renorm) total = wave_sum(s);
  if (g.renorm || !g.sigmoid) s = total > 0.0 ? s / total : 0.0;
  if (lane < g.K) {
    g.ids[t * g.K + lane] = my_id;
    g.w[t * g.K + lane] = (float)(s * (double)g.scale);
  }
}

// LPL: items per lane.  SCORES: scores and their sums are compared, not the logits.
template <int LPL, bool SCORES>
__global__ __launch_bounds__(kThreads) void route_scored_kernel(Args g) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t t = (int64_t)blockIdx.x * kTokens + threadIdx.x / kWave;
  if (t >= g.T) return;
  const int grp = lane >> g.lg, sub = lane & ((1 << g.lg) - 1);
  const Token at{t, lane, grp, sub, grp * g.gs + sub};
  float l[LPL];
  #pragma unroll
  for (int i = 0; i < LPL; ++i) {
    const int in = sub + (i << g.lg);
    l[i] = grp < g.groups && in < g.gs
               ? load_logit(g.logits, t * g.E + at.e0 + (i << g.lg), g.bf16) : -INFINITY;
  }
  if (!route_fast<LPL, SCORES>(g, at, l)) route_exact<LPL, SCORES>(g, at, l);
}

struct BwdArgs {
  const void* logits;
  const int32_t* ids;
  const float* d_w;
  void* d_logits;
  int T, E, K;
  int bf16, sigmoid, renorm;
  float scale;
};

// One wavefront per token.  Lane l holds experts l, l+64, ...; lane j < K slot j, whose terms are
// computed in 64 bits and reach the lane that holds the expert by a lane broadcast, slots in
// ascending j, so the result does not depend on timing.
template <int LPL>
__global__ __launch_bounds__(kThreads) void route_scored_bwd_kernel(BwdArgs g) {
  const int lane = threadIdx.x & (kWave - 1);
  const int t = blockIdx.x * kTokens + threadIdx.x / kWave;
  if (t >= g.T) return;
  const int64_t row = (int64_t)t * g.E;
  int id = -1;
  float dw = 0.0f, lj = -INFINITY;
  if (lane < g.K) {
    id = g.ids[(int64_t)t * g.K + lane];
    dw = g.d_w[(int64_t)t * g.K + lane];
    if ((uint32_t)id < (uint32_t)g.E) lj = load_logit(g.logits, row + id, g.bf16);
  }
  const bool chosen = lj > -INFINITY;   // an id outside [0,E) names no logit
  float d[LPL];
  #pragma unroll
  for (int i = 0; i < LPL; ++i) d[i] = 0.0f;
  float m = 0.0f, total = 1.0f;
  if (!g.sigmoid && !g.renorm) {        // every expert has a share
    m = -INFINITY;
    #pragma unroll
    for (int i = 0; i < LPL; ++i) {
      const int e = lane + kWave * i;
      d[i] = e < g.E ? load_logit(g.logits, row + e, g.bf16) : -INFINITY;
      m = fmaxf(m, d[i]);
    }
    m = wave_max(m);
    if (m == -INFINITY) m = 0.0f;
    total = 0.0f;
    #pragma unroll
    for (int i = 0; i < LPL; ++i) {
      d[i] = expf(d[i] - m);
      total += d[i];
    }
    total = wave_allreduce(total, [](float a, float b) { return a + b; });
  } else if (!g.sigmoid) {
    m = fmaxf(wave_max(lj), -3.40282347e38f);
  }
  double s, rest = 1.0;                 // the score, and 1 - s for the sigmoid
  if (g.sigmoid) {
    const double u = exp(-fabs((double)lj)), v = 1.0 / (1.0 + u);
    s = lj >= 0.0f ? v : u * v;
    rest = lj >= 0.0f ? u * v : v;
  } else {
    s = exp((double)lj - (double)m) / (double)total;
  }
  if (!chosen) s = 0.0;
  double mean = 0.0;                    // sum of the weights times their gradients
  double term = (double)dw;
  if (g.renorm) {
    const double sum = wave_sum(s);
    s = sum > 0.0 ? s / sum : 0.0;
    mean = wave_sum(chosen ? s * (double)dw : 0.0);
    term -= mean;
  } else if (!g.sigmoid) {
    mean = wave_sum(chosen ? s * (double)dw : 0.0);
    const float share = -(float)(mean * (double)g.scale) / (total > 0.0f ? total : 1.0f);
    #pragma unroll
    for (int i = 0; i < LPL; ++i) d[i] *= share;
  }
  const float mine = chosen ? (float)(s * (double)g.scale * rest * term) : 0.0f;
  for (int j = 0; j < g.K; ++j) {
    const int e = __builtin_amdgcn_readlane(chosen ? id : -1, j);
    const float v = bcast(mine, j);
    #pragma unroll
    for (int i = 0; i < LPL; ++i)
      if (lane + kWave * i == e) d[i] += v;
  }
  #pragma unroll
  for (int i = 0; i < LPL; ++i) {
    const int e = lane + kWave * i;
    if (e >= g.E) continue;
    if (g.bf16)
      ((uint16_t*)g.d_logits)[row + e] = (uint16_t)f32_to_bf16(d[i]);
    else
      ((float*)g.d_logits)[row + e] = d[i];
  }
}

template <bool SCORES>
hipError_t run_route(const Args& a, hipStream_t s) {
  const dim3 grid((unsigned)(((int64_t)a.T + kTokens - 1) / kTokens)), block(kThreads);
  const int items = (a.gs + (1 << a.lg) - 1) >> a.lg;    // at most 32 (E <= 1024)
  if (items <= 1) hipLaunchKernelGGL((route_scored_kernel<1, SCORES>), grid, block, 0, s, a);
  else if (items <= 2) hipLaunchKernelGGL((route_scored_kernel<2, SCORES>), grid, block, 0, s, a);
  else if (items <= 4) hipLaunchKernelGGL((route_scored_kernel<4, SCORES>), grid, block, 0, s, a);
  else if (items <= 8) hipLaunchKernelGGL((route_scored_kernel<8, SCORES>), grid, block, 0, s, a);
  else if (items <= 16) hipLaunchKernelGGL((route_scored_kernel<16, SCORES>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((route_scored_kernel<32, SCORES>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace rs

hipError_t launch_route_scored(const Resolved& r, const moe_router& q, const void* logits,
                               bool bf16, const float* bias, int32_t* topk_ids, float* topk_w,
                               hipStream_t s) {
  rs::Args a{};
  a.logits = logits; a.bias = bias; a.ids = topk_ids; a.w = topk_w;
  a.T = r.T; a.E = r.E; a.K = r.K;
  a.bf16 = bf16; a.sigmoid = q.score == MOE_SCORE_SIGMOID; a.renorm = q.renormalize != 0;
  a.groups = q.n_groups; a.kept = q.topk_groups; a.top = q.group_top;
  a.gs = r.E / q.n_groups;
  a.scale = q.scale;
  a.lg = 6;
  while ((kWave >> a.lg) < q.n_groups) --a.lg;
  const bool sums = bias || (q.topk_groups < q.n_groups && q.group_top == 2);
  return sums ? rs::run_route<true>(a, s) : rs::run_route<false>(a, s);
}

hipError_t launch_route_scored_bwd(const Resolved& r, const moe_router& q, const void* logits,
                                   bool bf16, const int32_t* topk_ids, const float* d_w,
                                   void* d_logits, hipStream_t s) {
  rs::BwdArgs a{};
  a.logits = logits; a.ids = topk_ids; a.d_w = d_w; a.d_logits = d_logits;
  a.T = r.T; a.E = r.E; a.K = r.K;
  a.bf16 = bf16; a.sigmoid = q.score == MOE_SCORE_SIGMOID; a.renorm = q.renormalize != 0;
  a.scale = q.scale;
  const dim3 grid((unsigned)(((int64_t)r.T + rs::kTokens - 1) / rs::kTokens)), block(rs::kThreads);
  switch (route_lpl(r.E)) {
#define MOE_CASE(L)                                                                   \
  case L:                                                                            \
    hipLaunchKernelGGL(rs::route_scored_bwd_kernel<L>, grid, block, 0, s, a);         \
    break;
    MOE_CASE(1)
    MOE_CASE(2)
    MOE_CASE(4)
    MOE_CASE(8)
    MOE_CASE(16)
#undef MOE_CASE
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace moe

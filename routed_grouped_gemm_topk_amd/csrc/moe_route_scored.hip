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
//
// Instructions bound it, not memory: one round of the choice after another, each a maximum over the wave
// and what takes its expert out (sigmoid, bias, 8 of 256 out of 4 of 8 groups: some 620 vector
// instructions a token, 85 more than with weights in fp32).  8192 such tokens take 14.5 us, 69 us
// where all of them need the choice in 64 bits too; 64 of them 5.7 us, one launch's time and one wave's
// chain; 8192 tokens of softmax, 6 of 64, bf16 7.1 us.  Backward: 4001 x 256 5.5 us (the bytes: 1.6 us).
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

// -inf and NaN take the expert out, +inf counts as the largest finite logit, -0 is 0 (their bits are
// compared).
__device__ __forceinline__ float clean(float l) {
  return l > -INFINITY ? fminf(l, 3.40282347e38f) + 0.0f : -INFINITY;
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

// A lane exchange after which groups of 2d lanes agree, if groups of d lanes did before.
template <class F>
__device__ __forceinline__ void exchange(int lg, F step) {
  if (lg > 0) step([](int v) { return dpp_xchg<0xB1>(v); });      // quad_perm 1,0,3,2
  if (lg > 1) step([](int v) { return dpp_xchg<0x4E>(v); });      // quad_perm 2,3,0,1
  if (lg > 2) step([](int v) { return dpp_xchg<0x141>(v); });     // row_half_mirror
  if (lg > 3) step([](int v) { return dpp_xchg<0x140>(v); });     // row_mirror
  if (lg > 4) step([](int v) { return __shfl_xor(v, 16, kWave); });
  if (lg > 5) step([](int v) { return __shfl_xor(v, 32, kWave); });
}

__device__ __forceinline__ double wave_sum(double v) {
  exchange(6, [&](auto from) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = from((int)(uint32_t)u), hi = from((int)(uint32_t)(u >> 32));
    v += __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
  });
  return v;
}

__device__ __forceinline__ float wave_max(float v) {
  return wave_allreduce(v, [](float a, float b) { return fmaxf(a, b); });
}

// 1 / (1 + exp(-l)): 6 u off (3 u, 1 u for the addition, 2 u for the reciprocal), and 0 below 2^-126.
__device__ __forceinline__ float sigmoid_of(float l) {
  return __builtin_amdgcn_rcpf(1.0f + exp_of(__builtin_amdgcn_fmed3f(-l, -88.0f, 88.0f)));
}

// exp(l - m) for l <= m: what the subtraction rounds off is put back too.  4 u off.
__device__ __forceinline__ float exp_diff(float l, float m) {
  const float d = l - m, back = d - l;
  const float rest = (l - (d - back)) - (m + back);
  const float e = exp_of(fmaxf(d, -100.0f));
  return d > -100.0f ? __builtin_fmaf(e, rest, e) : 0.0f;      // below it rest may be NaN
}

struct Token {
  int64_t t;
  int lane, grp, sub, e0;       // lane, its group, its place in it, its first expert
};

// Floats as integers of the same order (the function is its own inverse): their maxima need no
// quieting of NaN and take a lane exchange as an operand.  kNoKey is below all of them.
constexpr int kNoKey = INT32_MIN;
__device__ __forceinline__ int ordered(int b) { return b ^ ((b >> 31) & 0x7fffffff); }
__device__ __forceinline__ int key_of(float f) { return ordered(__builtin_bit_cast(int, f)); }
__device__ __forceinline__ float of_key(int k) { return __builtin_bit_cast(float, ordered(k)); }

// The largest of a wave's values, as a scalar: within rows of 16 lanes, then row 0 to 1 and 2 to 3, then
// rows 0-1 to 2-3, whose last lane has it.  Each step's exchange is an operand of its maximum.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int max_step(int v) {
  return max(v, __builtin_amdgcn_update_dpp(kNoKey, v, CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ int wave_top(int v) {
  v = max_step<0xB1>(v);          // quad_perm 1,0,3,2
  v = max_step<0x4E>(v);          // quad_perm 2,3,0,1
  v = max_step<0x141>(v);         // row_half_mirror
  v = max_step<0x140>(v);         // row_mirror
  v = max_step<0x142, 0xa>(v);    // row_bcast 15 into rows 1 and 3
  v = max_step<0x143, 0xc>(v);    // row_bcast 31 into rows 2 and 3
  return __builtin_amdgcn_readlane(v, 63);
}

// Stores slot j of lane j < K: its id (-1: none) and its weight, from the id's logit lj.  In 64 bits, so
// that the weight is rounded once: one evaluation a lane, but for softmax's sum over all experts.
template <int LPL>
__device__ __forceinline__ void store_slots(const Args& g, const Token& at, const float (&l)[LPL],
                                            int id, float lj) {
  double s, total = 1.0;
  if (g.sigmoid) {
    s = 1.0 / (1.0 + exp(-(double)lj));
  } else {
    float m = lj;               // the largest chosen; without renormalising the largest of all
    if (!g.renorm) {
      #pragma unroll
      for (int i = 0; i < LPL; ++i) m = fmaxf(m, l[i]);
    }
    m = fmaxf(wave_max(m), -3.40282347e38f);
    s = exp((double)lj - (double)m);
    if (!g.renorm) {
      total = 0.0;
      #pragma unroll
      for (int i = 0; i < LPL; ++i) total += exp((double)l[i] - (double)m);
      total = wave_sum(total);
    }
  }
  if (id < 0) s = 0.0;
  if (g.renorm) total = wave_sum(s);
  if (at.lane < g.K) {
    g.ids[at.t * g.K + at.lane] = id;
    g.w[at.t * g.K + at.lane] = total > 0.0 ? (float)(s / total * (double)g.scale) : 0.0f;
  }
}

// The choice in fp32; returns false, having stored nothing, where fp32 does not tell two experts or
// groups apart that the choice depends on.  Every lane of the wave must be active.
//
// An expert's key is its choice score's (its logit's) ordered integer, whose last bits hold the item's
// place in the lane, so that a lane's keys differ and the largest one names its item.  A bf16 logit
// leaves 16 bits, which hold the whole id, the lowest largest: its order, ties included, is exact.
//
// Errors otherwise (u = 2^-24): a sigmoid score is at most 1 and 6 u of itself off; a softmax score p is
// 4 u of itself off for its exponential, 4 u and an addition's u for each of LPL + 6 for the sum, 3 u
// for the product with its reciprocal, and at most 1 / total (2^-126 where it is smaller); a choice
// score c another u |c| for the addition of the bias and 2 LPL u |c| for the bits given up; a sum of
// two the errors of both and its own.  Two that differ by more than both errors are in the right
// order.  An expert's error grows with its own value alone, so neighbours in the order speak for all
// below them; a sum's does not (large scores may cancel), so every group is held to its own error, away
// from the middle between the last one kept and the first one that is not.
template <int LPL, bool SCORES>
__device__ __forceinline__ bool route_fast(const Args& g, const Token& at, const float (&l)[LPL],
                                           const float (&bias)[LPL]) {
  constexpr float U = 0x1p-24f;
  const bool whole_ids = !SCORES && g.bf16;
  float sure = 0.0f;            // error of the scores of two experts
  int key[LPL], group1 = kNoKey, group2 = kNoKey;      // the group's two largest
  if constexpr (SCORES) {
    float s[LPL], inv = 1.0f;
    if (!g.sigmoid) {
      float m = -INFINITY, sum = 0.0f;
      #pragma unroll
      for (int i = 0; i < LPL; ++i) m = fmaxf(m, l[i]);
      m = wave_max(m);
      if (m == -INFINITY) m = 0.0f;
      #pragma unroll
      for (int i = 0; i < LPL; ++i) {
        s[i] = exp_diff(l[i], m);
        sum += s[i];
      }
      sum = wave_allreduce(sum, [](float a, float b) { return a + b; });
      inv = sum > 0.0f ? __builtin_amdgcn_rcpf(sum) : 0.0f;
      sure = 2 * (LPL + 18) * U * inv;
    } else {
      #pragma unroll
      for (int i = 0; i < LPL; ++i) s[i] = sigmoid_of(l[i]);
      sure = 2 * 6 * U;
    }
    #pragma unroll
    for (int i = 0; i < LPL; ++i) {
      const float c = s[i] * inv + bias[i];
      key[i] = l[i] > -INFINITY && bias[i] > -INFINITY ? key_of(c) : kNoKey;
    }
  } else {
    #pragma unroll
    for (int i = 0; i < LPL; ++i) {
      const int k = key_of(l[i]);
      key[i] = l[i] == -INFINITY ? kNoKey
               : whole_ids ? (k & ~0xffff) | (0xffff - (at.e0 + (i << g.lg))) : k;
    }
  }
  // two values of the same kind that are further apart than their errors
  auto apart = [&](float hi, float lo, float err, float parts) {
    return hi - lo > (SCORES ? err : 0.0f) + parts * U * (fabsf(hi) + fabsf(lo));
  };
  bool ok = true;
  if (g.kept < g.groups) {
    #pragma unroll
    for (int i = 0; i < LPL; ++i) {
      group2 = max(group2, min(group1, key[i]));
      group1 = max(group1, key[i]);
    }
    exchange(g.lg, [&](auto from) {
      const int o1 = from(group1), o2 = from(group2);
      group2 = max(min(group1, o1), max(group2, o2));
      group1 = max(group1, o1);
    });
    const bool two = SCORES && g.top == 2 && group2 != kNoKey;
    const float v1 = of_key(group1), v2 = of_key(group2);
    const int value = two ? key_of(v1 + v2) : group1;
    int before = 0;             // groups that come before this lane's
    for (int o = 0; o < g.groups; ++o)
      before += __builtin_amdgcn_readlane(value, o << g.lg) > value;
    // the last group kept and the first that is not: one each unless two values are the same
    const bool first = at.sub == 0 && at.grp < g.groups;
    const uint64_t in = __ballot(first && before == g.kept - 1);
    const uint64_t out = __ballot(first && before == g.kept);
    if (__popcll(in) != 1 || __popcll(out) != 1) return false;
    const int a = __builtin_ctzll(in), b = __builtin_ctzll(out);
    const int va = __builtin_amdgcn_readlane(value, a), vb = __builtin_amdgcn_readlane(value, b);
    if (SCORES && vb != kNoKey) {
      const float border = 0.5f * of_key(va) + 0.5f * of_key(vb), v = of_key(value);
      const float err = sure + 4 * U * (fabsf(v1) + (two ? fabsf(v2) : 0.0f));
      const bool clear = value == kNoKey || (before < g.kept ? v - err > border : v + err < border);
      ok = __ballot(first && !clear) == 0;
    }
    if (before >= g.kept) {
      #pragma unroll
      for (int i = 0; i < LPL; ++i) key[i] = kNoKey;
    }
  }
  if (!whole_ids) {
    #pragma unroll
    for (int i = 0; i < LPL; ++i)
      key[i] = key[i] == kNoKey ? kNoKey : (key[i] & ~(LPL - 1)) | (LPL - 1 - i);
  }
  // lane j: the key and the lane of the j-th choice; one more than are chosen, for its margin
  int my_key = kNoKey, my_lane = 0, after = kNoKey, found = 0, same = 0;
  for (int j = 0; j <= g.K; ++j) {
    int best = key[0];
    #pragma unroll
    for (int i = 1; i < LPL; ++i) best = max(best, key[i]);
    const int mine = best;
    best = wave_top(best);
    after = best;
    if (best == kNoKey || j == g.K) break;
    const uint64_t who = __ballot(mine == best);
    same |= (who & (who - 1)) != 0;
    my_key = at.lane == j ? best : my_key;
    my_lane = at.lane == j ? __builtin_ctzll(who) : my_lane;
    #pragma unroll
    for (int i = 0; i < LPL; ++i) key[i] = key[i] == best ? kNoKey : key[i];
    found = j + 1;
  }
  const bool here = at.lane < found;
  if (!whole_ids) {
    int next = __shfl_down(my_key, 1, kWave);
    if (at.lane + 1 >= found) next = after;
    const bool sure_of = next == kNoKey || apart(of_key(my_key & ~(LPL - 1)),
                                                 of_key(next & ~(LPL - 1)), sure,
                                                 SCORES ? 2 * LPL + 4 : 2 * LPL);
    if (same || !ok || __ballot(here && !sure_of)) return false;
  }
  const int grp = my_lane >> g.lg, sub = my_lane & ((1 << g.lg) - 1);
  const int e0 = grp * g.gs + sub;
  int item, id;
  if (whole_ids) {
    id = 0xffff - (my_key & 0xffff);
    item = (id - e0) >> g.lg;
  } else {
    item = LPL - 1 - (my_key & (LPL - 1));
    id = e0 + (item << g.lg);
  }
  float lj = -INFINITY;
  #pragma unroll
  for (int i = 0; i < LPL; ++i) {
    const float v = __shfl(l[i], my_lane, kWave);
    if (i == item) lj = v;
  }
  store_slots(g, at, l, here ? id : -1, here ? lj : -INFINITY);
  return true;
}

// The same with scores and group values in 64 bits (SCORES) and ties to the lowest ids.
template <int LPL, bool SCORES>
__device__ __forceinline__ void route_exact(const Args& g, const Token& at_, const float (&l)[LPL]) {
  using C = typename std::conditional<SCORES, double, float>::type;
  constexpr C NONE = -INFINITY;
  const int lane = at_.lane, grp = at_.grp, e0 = at_.e0;
  C c[LPL];                     // choice scores
  if constexpr (SCORES) {
    float m = 0.0f;             // softmax: the largest logit, 0 without any
    double total = 0.0;         // softmax: the sum of exp(l - m)
    if (!g.sigmoid) {
      m = -INFINITY;
      #pragma unroll
      for (int i = 0; i < LPL; ++i) m = fmaxf(m, l[i]);
      m = wave_max(m);
      if (m == -INFINITY) m = 0.0f;
    }
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

  float lj = -INFINITY;         // lane j: the logit of slot j
  #pragma unroll
  for (int i = 0; i < LPL; ++i) {
    const float v = __shfl(l[i], my_lane, kWave);
    if (my_id >= 0 && i == my_item) lj = v;
  }
  store_slots(g, at_, l, my_id, lj);
}

// LPL: items per lane.  SCORES: scores and their sums are compared, not the logits.
template <int LPL, bool SCORES>
__global__ __launch_bounds__(kThreads) void route_scored_kernel(Args g) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t t = (int64_t)blockIdx.x * kTokens + threadIdx.x / kWave;
  if (t >= g.T) return;
  const int grp = lane >> g.lg, sub = lane & ((1 << g.lg) - 1);
  const Token at{t, lane, grp, sub, grp * g.gs + sub};
  // all loads first, from places that are there; lanes without the item drop it
  float l[LPL], bias[LPL];
  int e[LPL];
  #pragma unroll
  for (int i = 0; i < LPL; ++i) {
    const int in = sub + (i << g.lg);
    e[i] = grp < g.groups && in < g.gs ? at.e0 + (i << g.lg) : 0;
  }
  if (g.bf16) {
    uint16_t raw[LPL];
    #pragma unroll
    for (int i = 0; i < LPL; ++i) raw[i] = ((const uint16_t*)g.logits)[t * g.E + e[i]];
    #pragma unroll
    for (int i = 0; i < LPL; ++i) l[i] = bf16_bits_to_f32(raw[i]);
  } else {
    #pragma unroll
    for (int i = 0; i < LPL; ++i) l[i] = ((const float*)g.logits)[t * g.E + e[i]];
  }
  if (SCORES && g.bias) {
    #pragma unroll
    for (int i = 0; i < LPL; ++i) bias[i] = g.bias[e[i]];
  } else {
    #pragma unroll
    for (int i = 0; i < LPL; ++i) bias[i] = 0.0f;
  }
  #pragma unroll
  for (int i = 0; i < LPL; ++i) {
    const int in = sub + (i << g.lg);
    l[i] = grp < g.groups && in < g.gs ? clean(l[i]) : -INFINITY;
  }
  if (!route_fast<LPL, SCORES>(g, at, l, bias)) route_exact<LPL, SCORES>(g, at, l);
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

// One wavefront per token.  Lane l holds experts l, l+64, ...; lane j < K slot j, whose terms reach the
// lane that holds the expert by a lane broadcast, slots in ascending j, so the result does not depend on
// timing.  All in 64 bits until the end: an expert's share and a slot's term may cancel, and an expert
// may be named twice.
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
  double d[LPL];
  #pragma unroll
  for (int i = 0; i < LPL; ++i) d[i] = 0.0;
  float m = 0.0f;
  double total = 1.0;
  if (!g.sigmoid && !g.renorm) {        // every expert has a share
    m = -INFINITY;
    float l[LPL];
    #pragma unroll
    for (int i = 0; i < LPL; ++i) {
      const int e = lane + kWave * i;
      l[i] = e < g.E ? load_logit(g.logits, row + e, g.bf16) : -INFINITY;
      m = fmaxf(m, l[i]);
    }
    m = wave_max(m);
    if (m == -INFINITY) m = 0.0f;
    total = 0.0;
    #pragma unroll
    for (int i = 0; i < LPL; ++i) {
      d[i] = exp((double)l[i] - (double)m);
      total += d[i];
    }
    total = wave_sum(total);
  } else if (!g.sigmoid) {
    m = fmaxf(wave_max(lj), -3.40282347e38f);
  }
  double s, rest = 1.0;                 // the score, and 1 - s for the sigmoid
  if (g.sigmoid) {
    const double u = exp(-fabs((double)lj)), v = 1.0 / (1.0 + u);
    s = lj >= 0.0f ? v : u * v;
    rest = lj >= 0.0f ? u * v : v;
  } else {
    s = exp((double)lj - (double)m) / total;
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
    const double share = total > 0.0 ? -mean * (double)g.scale / total : 0.0;
    #pragma unroll
    for (int i = 0; i < LPL; ++i) d[i] *= share;
  }
  const double mine = chosen ? s * (double)g.scale * rest * term : 0.0;
  for (int j = 0; j < g.K; ++j) {
    const int e = __builtin_amdgcn_readlane(chosen ? id : -1, j);
    const double v = bcast(mine, j);
    #pragma unroll
    for (int i = 0; i < LPL; ++i)
      if (lane + kWave * i == e) d[i] += v;
  }
  #pragma unroll
  for (int i = 0; i < LPL; ++i) {
    const int e = lane + kWave * i;
    if (e >= g.E) continue;
    if (g.bf16)
      ((uint16_t*)g.d_logits)[row + e] = (uint16_t)f32_to_bf16((float)d[i]);
    else
      ((float*)g.d_logits)[row + e] = (float)d[i];
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

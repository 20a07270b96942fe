// Root-mean-square norm of token rows, with the residual's addition before it and rows and e4m3
// codes as its outputs, and its gradient.
//
//   s = round(x + residual),  r = 1 / sqrt(mean s^2 + eps),  n = s r w
//   y = round(n);  codes = e4m3(n / scale), scale = amax |n| / 448 over 128 columns, at least 2^-126
//   d_x = r (g - n' mean(g n')) + d_sum,  d_w = sum over rows of d_y n',   n' = s r, g = d_y w
//
// HBM bounds both: every row is read once and stays in registers.  TPR threads share a row, each
// with NV chunks of 8 columns.  Where rows are whole 16-byte blocks (VEC), chunk v of thread i begins
// at column (v TPR + i) 8, so that 16 neighbouring lanes hold one scale group; elsewhere its k-th
// column is (8 v + k) TPR + i, so that a wave's loads still are neighbours.
//
// Measured, operands from memory: forward, residual to rows and codes, bf16, 2048 x 7168 29.6 us (4.5
// TB/s) and 16384 x 7168 190 us (5.6 TB/s, more than a copy's 5.0, since reads outweigh writes); 2001
// x 2880 fp32 20.9 us (4.4 TB/s); one row of 7168 4.3 us, a launch's own time and one round trip to
// memory.  Backward with the weight's gradient, bf16, 4096 x 4096 34.4 us (3.9 TB/s); 1000 x 12288 43 us
// (2.3 TB/s; the bytes at a copy's rate: 19.5), whose registers leave two waves a SIMD.
#include <algorithm>
#include <type_traits>

#include "moe_internal.h"
#include "moe_route.h"

namespace moe {

namespace nm {

constexpr int kThreads = 256;     // of a workgroup, at least
constexpr int kMaxGrid = 1 << 21;  // workgroups of a launch; more rows are run by striding

struct Args {
  const void *x, *residual, *weight;
  void *sum, *y;
  uint8_t* codes;
  float *scales, *rstd;
  int T, H;
  float eps;
};

// Eight values of a row as they lie in memory, and as fp32; thread i's chunk v of a row that begins at
// `row`.
template <int TPR, bool BF16, bool VEC>
struct Chunk {
  static constexpr int W = BF16 ? 4 : 8;
  uint32_t w[W];

  __device__ static __forceinline__ int first(int v, int i) {
    return VEC ? (v * TPR + i) * 8 : v * 8 * TPR + i;
  }
  // column of value k, if the row has it
  template <class F>
  __device__ static __forceinline__ void each(int H, int v, int i, F f) {
    const int c = first(v, i);
    #pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c + (VEC ? k : k * TPR) < H) f(k, c + (VEC ? k : k * TPR));
  }

  __device__ __forceinline__ void load(const void* base, int64_t row, int H, int v, int i) {
    #pragma unroll
    for (int q = 0; q < W; ++q) w[q] = 0;
    if constexpr (VEC) {
      if (first(v, i) >= H) return;
      const i32x4* p = (const i32x4*)((const char*)base + (row + first(v, i)) * (BF16 ? 2 : 4));
      #pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        const i32x4 x = p[q];
        #pragma unroll
        for (int k = 0; k < 4; ++k) w[4 * q + k] = (uint32_t)x[k];
      }
    } else {
      each(H, v, i, [&](int k, int c) {
        if constexpr (BF16) w[k / 2] |= (uint32_t)((const uint16_t*)base)[row + c] << (16 * (k & 1));
        else w[k] = ((const uint32_t*)base)[row + c];
      });
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t row, int H, int v, int i) const {
    if constexpr (VEC) {
      if (first(v, i) >= H) return;
      i32x4* p = (i32x4*)((char*)base + (row + first(v, i)) * (BF16 ? 2 : 4));
      #pragma unroll
      for (int q = 0; q < W / 4; ++q)
        p[q] = i32x4{(int)w[4 * q], (int)w[4 * q + 1], (int)w[4 * q + 2], (int)w[4 * q + 3]};
    } else {
      each(H, v, i, [&](int k, int c) {
        if constexpr (BF16) ((uint16_t*)base)[row + c] = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
        else ((uint32_t*)base)[row + c] = w[k];
      });
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (BF16)
      return i & 1 ? __uint_as_float(w[i / 2] & 0xFFFF0000u) : __uint_as_float(w[i / 2] << 16);
    else
      return __uint_as_float(w[i]);
  }
  __device__ __forceinline__ void set(const float* v) {
    #pragma unroll
    for (int i = 0; i < W; ++i)
      w[i] = BF16 ? f32_to_bf16x2(v[BF16 ? 2 * i : i], v[BF16 ? 2 * i + 1 : i])
                  : __float_as_uint(v[i]);
  }
};

// Sum over the TPR threads of a row, the same on each: lanes first, then waves in their order.
// Every wave of the workgroup calls it as often; `turn` picks one of two sets of LDS words, so that
// one barrier per call is enough.
template <int TPR, class V>
__device__ __forceinline__ V row_sum(V v, V (*words)[TPR / kWave], int turn) {
  #pragma unroll
  for (int d = 1; d < kWave; d *= 2) v += __shfl_xor(v, d, kWave);
  if constexpr (TPR > kWave) {
    const int wave = threadIdx.x / kWave;
    if ((threadIdx.x & (kWave - 1)) == 0) words[turn][wave] = v;
    __syncthreads();
    v = words[turn][0];
    #pragma unroll
    for (int i = 1; i < TPR / kWave; ++i) v += words[turn][i];
  }
  return v;
}

template <int TPR, int NV, bool BF16, bool VEC>
__global__ __launch_bounds__(TPR < kThreads ? kThreads : TPR) void rms_norm_kernel(Args g) {
  constexpr int ROWS = TPR < kThreads ? kThreads / TPR : 1;      // of a workgroup
  using Part = Chunk<TPR, BF16, VEC>;
  __shared__ double words[2][TPR / kWave];
  const int i = ROWS > 1 ? threadIdx.x % TPR : threadIdx.x;
  const int in_row = ROWS > 1 ? threadIdx.x / TPR : 0;
  Part w[NV];
  #pragma unroll
  for (int v = 0; v < NV; ++v)
    if (g.weight) w[v].load(g.weight, 0, g.H, v, i);
  int turn = 0;
  for (int64_t set = blockIdx.x; set * ROWS < g.T; set += gridDim.x) {
    const int64_t t = set * ROWS + in_row, row = t * g.H;
    const bool live = t < g.T;                         // the same for a whole wave
    Part x[NV] = {};
    if (live) {
      #pragma unroll
      for (int v = 0; v < NV; ++v) x[v].load(g.x, row, g.H, v, i);
      if (g.residual) {
        Part r[NV];
        #pragma unroll
        for (int v = 0; v < NV; ++v) r[v].load(g.residual, row, g.H, v, i);
        #pragma unroll
        for (int v = 0; v < NV; ++v) {
          float s[8];
          #pragma unroll
          for (int k = 0; k < 8; ++k) s[k] = x[v].get(k) + r[v].get(k);
          x[v].set(s);
          x[v].store(g.sum, row, g.H, v, i);
        }
      }
    }
    // squares of fp32 values neither overflow nor vanish in 64 bits
    double sq = 0.0;
    #pragma unroll
    for (int v = 0; v < NV; ++v)
      #pragma unroll
      for (int k = 0; k < 8; ++k) {
        const double s = x[v].get(k);
        sq = __builtin_fma(s, s, sq);
      }
    sq = row_sum<TPR>(sq, words, turn);
    turn ^= 1;
    if (!live) continue;
    const double r64 = rsqrt(sq / (double)g.H + (double)g.eps);
    const float rstd = (float)r64;
    if (g.rstd && i == 0) g.rstd[t] = rstd;
    // n = (s p) w r with rstd = p r, p a power of two: s p is exact, and so is its product with w in
    // bf16, which leaves r's rounding and one more (s r w by itself rounds three times)
    const int exponent = min(max((int)(__float_as_uint(rstd) >> 23), 1), 254);
    const float p = __uint_as_float((uint32_t)exponent << 23);
    const double r_p = ldexp(r64, 127 - exponent);
    #pragma unroll
    for (int v = 0; v < NV; ++v) {
      float n[8], y[8];
      #pragma unroll
      for (int k = 0; k < 8; ++k) {
        n[k] = x[v].get(k) * p;
        if (g.weight) n[k] *= w[v].get(k);
        y[k] = n[k] * (float)r_p;
      }
      if (g.y) {
        Part o;
        o.set(y);
        o.store(g.y, row, g.H, v, i);
      }
      if (VEC && g.codes) {
        float m = 0.0f;
        #pragma unroll
        for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(n[k]));
        // 16 lanes hold a group
        m = fmaxf(m, dpp_xchg<0xB1>(m));
        m = fmaxf(m, dpp_xchg<0x4E>(m));
        m = fmaxf(m, dpp_xchg<0x141>(m));
        m = fmaxf(m, dpp_xchg<0x140>(m));
        // A scale below 2^-126 would lose bits, and its quotients pass 448.  A quotient is n times
        // r / scale: that factor's rounding and its own.
        const float amax = (float)(m * r_p);
        const float s = amax > 0.0f ? fmaxf(amax, kE4M3Max * 0x1p-126f) / kE4M3Max : 1.0f;
        const double inv = __builtin_amdgcn_rcpf(s);
        const float f = (float)(r_p * (inv * (2.0 - (double)s * inv)));
        const int c = Part::first(v, i);
        if (c < g.H) {
          // quotients are at most 448 up to their rounding, below the 464 from which e4m3 would
          // overflow, so the convert (nearest even, NaN kept) needs no clamp
          uint32_t q[2];
          #pragma unroll
          for (int h = 0; h < 2; ++h)
            q[h] = __builtin_amdgcn_cvt_pk_fp8_f32(
                n[4 * h + 2] * f, n[4 * h + 3] * f,
                __builtin_amdgcn_cvt_pk_fp8_f32(n[4 * h] * f, n[4 * h + 1] * f, 0, false), true);
          *(uint2*)(g.codes + row + c) = make_uint2(q[0], q[1]);
          if ((i & 15) == 0) g.scales[t * (g.H / kGroup) + c / kGroup] = s;
        }
      }
    }
  }
}

struct BwdArgs {
  const void *d_y, *d_sum, *sum, *weight;
  const float* rstd;
  void* d_x;
  float* partials;              // [gridDim.x, H], or null: no gradient of the weight
  int T, H;
};

// A workgroup takes every gridDim.x-th set of rows and keeps its part of d_w in registers; its rows
// (one per wave where TPR is a wave) are added through LDS at the end, then one row of partials.
// Up to 16 words of a row a thread (32 values of bf16), rows stay in registers and the next ones are on
// their way while a row's sum goes round (4096 x 4096: 42.5 -> 34.5 us).  Longer ones, and those of 1024
// threads, are loaded again, from the caches, once the sum is known.
template <int TPR, int NV, bool BF16, bool VEC>
__global__ __launch_bounds__(TPR < kThreads ? kThreads : TPR) void rms_norm_bwd_kernel(BwdArgs g) {
  constexpr int ROWS = TPR < kThreads ? kThreads / TPR : 1;
  using Part = Chunk<TPR, BF16, VEC>;
  constexpr bool HELD = NV * Part::W <= 16 && TPR < 1024;
  __shared__ float words[2][TPR / kWave];
  __shared__ float part[ROWS > 1 ? ROWS * TPR * 8 : 1];
  const int i = ROWS > 1 ? threadIdx.x % TPR : threadIdx.x;
  const int in_row = ROWS > 1 ? threadIdx.x / TPR : 0;
  float dw[NV][8];
  #pragma unroll
  for (int v = 0; v < NV; ++v)
    #pragma unroll
    for (int k = 0; k < 8; ++k) dw[v][k] = 0.0f;
  // one chunk's part of the sum of g n, and of d_w
  auto gather = [&](const Part& dy, const Part& s, const Part& w, float r, float (&d_w)[8],
                    float& dot) {
    #pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = dy.get(k), norm = s.get(k) * r;
      d_w[k] = __builtin_fmaf(d, norm, d_w[k]);
      dot = __builtin_fmaf(g.weight ? d * w.get(k) : d, norm, dot);
    }
  };
  auto finish = [&](const Part& dy, const Part& s, const Part& w, const Part& ds, float r, float dot,
                    int64_t row, int v) {
    float d[8];
    #pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float gk = g.weight ? dy.get(k) * w.get(k) : dy.get(k);
      d[k] = r * (gk - s.get(k) * r * dot);
      if (g.d_sum) d[k] += ds.get(k);
    }
    Part o;
    o.set(d);
    o.store(g.d_x, row, g.H, v, i);
  };
  int turn = 0;
  if constexpr (HELD) {
    Part w[NV];
    #pragma unroll
    for (int v = 0; v < NV; ++v)
      if (g.weight) w[v].load(g.weight, 0, g.H, v, i);
    struct Row {
      Part dy[NV], s[NV], ds[NV];
      float r;
    };
    auto load = [&](Row& o, int64_t set) {
      const int64_t t = set * ROWS + in_row, row = t * g.H;
      if (t >= g.T) {
        o.r = 0.0f;
        #pragma unroll
        for (int v = 0; v < NV; ++v) o.dy[v] = o.s[v] = Part{};
        return;
      }
      o.r = g.rstd[t];
      #pragma unroll
      for (int v = 0; v < NV; ++v) {
        o.dy[v].load(g.d_y, row, g.H, v, i);
        o.s[v].load(g.sum, row, g.H, v, i);
      }
      if (g.d_sum) {
        #pragma unroll
        for (int v = 0; v < NV; ++v) o.ds[v].load(g.d_sum, row, g.H, v, i);
      }
    };
    Row cur, nxt;
    load(cur, blockIdx.x);
    for (int64_t set = blockIdx.x; set * ROWS < g.T; set += gridDim.x) {
      load(nxt, set + gridDim.x);
      float dot = 0.0f;
      #pragma unroll
      for (int v = 0; v < NV; ++v) gather(cur.dy[v], cur.s[v], w[v], cur.r, dw[v], dot);
      dot = row_sum<TPR>(dot, words, turn) / (float)g.H;
      turn ^= 1;
      const int64_t t = set * ROWS + in_row;
      if (t < g.T) {
        #pragma unroll
        for (int v = 0; v < NV; ++v)
          finish(cur.dy[v], cur.s[v], w[v], cur.ds[v], cur.r, dot, t * g.H, v);
      }
      cur = nxt;
    }
  } else {
    static_assert(HELD || ROWS == 1, "every thread has a row");
    for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x) {
      const int64_t row = t * g.H;
      const float r = g.rstd[t];
      float dot = 0.0f;
      #pragma unroll
      for (int v = 0; v < NV; ++v) {
        Part dy, s, w = {};
        dy.load(g.d_y, row, g.H, v, i);
        s.load(g.sum, row, g.H, v, i);
        if (g.weight) w.load(g.weight, 0, g.H, v, i);
        gather(dy, s, w, r, dw[v], dot);
      }
      dot = row_sum<TPR>(dot, words, turn) / (float)g.H;
      turn ^= 1;
      #pragma unroll
      for (int v = 0; v < NV; ++v) {
        Part dy, s, w = {}, ds = {};
        dy.load(g.d_y, row, g.H, v, i);
        s.load(g.sum, row, g.H, v, i);
        if (g.weight) w.load(g.weight, 0, g.H, v, i);
        if (g.d_sum) ds.load(g.d_sum, row, g.H, v, i);
        finish(dy, s, w, ds, r, dot, row, v);
      }
    }
  }
  if (!g.partials) return;
  float* out = g.partials + (int64_t)blockIdx.x * g.H;
  #pragma unroll
  for (int v = 0; v < NV; ++v) {
    if constexpr (ROWS > 1) {
      __syncthreads();
      #pragma unroll
      for (int k = 0; k < 8; ++k) part[(in_row * TPR + i) * 8 + k] = dw[v][k];
      __syncthreads();
      if (in_row > 0) continue;
      #pragma unroll
      for (int q = 1; q < ROWS; ++q)
        #pragma unroll
        for (int k = 0; k < 8; ++k) dw[v][k] += part[(q * TPR + i) * 8 + k];
    }
    Part::each(g.H, v, i, [&](int k, int c) { out[c] = dw[v][k]; });
  }
}

// 64 columns a workgroup; its 16 waves take 16 neighbouring stretches of the rows, eight loads on their
// way at a time: latency bounds it (512 x 4096 partial sums, which lie in the last-level cache: 4 us).
constexpr int kSumWaves = 16;

__global__ __launch_bounds__(kSumWaves * kWave) void sum_rows_kernel(
    const float* __restrict__ partials, float* __restrict__ out, int rows, int cols) {
  __shared__ float part[kSumWaves][kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int64_t c = (int64_t)blockIdx.x * kWave + lane;
  const int per = (rows + kSumWaves - 1) / kSumWaves;
  const int end = min(rows, (wave + 1) * per);
  float t = 0.0f;
  if (c < cols) {
    const float* p = partials + c;
    int r = wave * per;
    for (; r + 8 <= end; r += 8) {
      float v[8];
      #pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = p[(int64_t)(r + k) * cols];
      #pragma unroll
      for (int k = 0; k < 8; ++k) t += v[k];
    }
    float v[8];
    #pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = r + k < end ? p[(int64_t)(r + k) * cols] : 0.0f;
    #pragma unroll
    for (int k = 0; k < 8; ++k) t += v[k];
  }
  part[wave][lane] = t;
  __syncthreads();
  if (wave > 0 || c >= cols) return;
  #pragma unroll
  for (int w = 1; w < kSumWaves; ++w) t += part[w][lane];
  out[c] = t;
}

// Calls f(TPR, NV, VEC) as compile-time constants for rows of H values.
template <class F>
hipError_t by_width(int H, F f) {
  using std::integral_constant;
  const bool vec = H % 8 == 0;
  auto with = [&](auto tpr, auto nv) {
    return vec ? f(tpr, nv, std::true_type{}) : f(tpr, nv, std::false_type{});
  };
  const integral_constant<int, 1> one{};
  const integral_constant<int, 2> two{};
  const integral_constant<int, 4> four{};
  const integral_constant<int, 64> wave{};
  const integral_constant<int, 256> four_waves{};
  const integral_constant<int, 512> eight_waves{};
  const integral_constant<int, 1024> all{};
  if (H <= 512) return with(wave, one);
  if (H <= 1024) return with(wave, two);
  if (H <= 2048) return with(four_waves, one);
  if (H <= 4096) return with(four_waves, two);
  if (H <= 8192) return with(eight_waves, two);
  if (H <= 16384) return with(eight_waves, four);
  return with(all, four);
}

}  // namespace nm

hipError_t launch_rms_norm(int T, int H, bool bf16, const void* x, const void* residual,
                           const void* weight, float eps, void* sum, void* y, uint8_t* codes,
                           float* scales, float* rstd, hipStream_t s) {
  nm::Args a{x, residual, weight, sum, y, codes, scales, rstd, T, H, eps};
  return nm::by_width(H, [&](auto tpr, auto nv, auto vec) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    constexpr bool VEC = decltype(vec)::value;
    constexpr int TH = std::max(TPR, nm::kThreads), ROWS = TH / TPR;
    const int64_t sets = ((int64_t)T + ROWS - 1) / ROWS;
    const unsigned grid = (unsigned)std::min<int64_t>(sets, nm::kMaxGrid);
    if (bf16)
      hipLaunchKernelGGL((nm::rms_norm_kernel<TPR, NV, true, VEC>), dim3(grid), dim3(TH), 0, s, a);
    else
      hipLaunchKernelGGL((nm::rms_norm_kernel<TPR, NV, false, VEC>), dim3(grid), dim3(TH), 0, s, a);
    return hipGetLastError();
  });
}

hipError_t launch_sum_rows(int rows, int cols, const float* partials, float* out, hipStream_t s) {
  hipLaunchKernelGGL(nm::sum_rows_kernel, dim3((unsigned)((cols + kWave - 1) / kWave)),
                     dim3(nm::kSumWaves * kWave), 0, s, partials, out, rows, cols);
  return hipGetLastError();
}

hipError_t launch_rms_norm_bwd(int T, int H, bool bf16, const void* d_y, const void* d_sum,
                               const void* sum, const void* weight, const float* rstd, void* d_x,
                               float* d_weight, float* partials, hipStream_t s) {
  nm::BwdArgs a{d_y, d_sum, sum, weight, rstd, d_x, d_weight ? partials : nullptr, T, H};
  const int cus = std::max(device_cu_count(), 8);
  unsigned grid = 0;
  const hipError_t e = nm::by_width(H, [&](auto tpr, auto nv, auto vec) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    constexpr bool VEC = decltype(vec)::value;
    constexpr int TH = std::max(TPR, nm::kThreads), ROWS = TH / TPR;
    const int64_t sets = ((int64_t)T + ROWS - 1) / ROWS;
    grid = (unsigned)std::min<int64_t>(std::min<int64_t>(sets, 2 * cus), kPartialRows);
    if (bf16)
      hipLaunchKernelGGL((nm::rms_norm_bwd_kernel<TPR, NV, true, VEC>), dim3(grid), dim3(TH), 0, s,
                         a);
    else
      hipLaunchKernelGGL((nm::rms_norm_bwd_kernel<TPR, NV, false, VEC>), dim3(grid), dim3(TH), 0, s,
                         a);
    return hipGetLastError();
  });
  if (e != hipSuccess || !d_weight) return e;
  return launch_sum_rows((int)grid, H, partials, d_weight, s);
}

}  // namespace moe

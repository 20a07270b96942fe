// Products of bf16 matrices with bias, activation and residual in their epilogue, and the gradient
// of that epilogue:
//
//   z = a b^T | a b | a^T b  (+ bias),   pre = round(z),   c = round(act(z) + residual)
//   d_z = round(d_c act'(pre)),  d_bias = sum over rows of d_c act'(pre)
//
// Accumulated in fp32 by the bf16 matrix instructions.  The operand order puts b on a result's rows
// and a on its columns, so a lane holds 4 neighbouring columns of ONE row of c.
#include <algorithm>

#include "moe_internal.h"

namespace moe {

namespace gb {

struct Args {
  const uint16_t *a, *b;
  const float* bias;
  const void* residual;
  uint16_t* pre;
  void* c;
  int M, N, K, act;
  int c_f32;
};

__device__ __forceinline__ float gelu_tanh_arg(float z) {       // 2 sqrt(2/pi) (z + 0.044715 z^3)
  return 1.59576912f * z * __builtin_fmaf(0.044715f * z, z, 1.0f);
}

__device__ __forceinline__ float activate(float z, int act) {
  if (act == MOE_ACT_SILU) return z / (1.0f + expf(-z));
  if (act == MOE_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.707106781f));
  // (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
  if (act == MOE_ACT_GELU_TANH) return z / (1.0f + expf(-gelu_tanh_arg(z)));
  return z;
}

// NC neighbouring values of row m of c from column n on, of which the first `left` exist.
template <int NC>
__device__ __forceinline__ void finish(const Args& g, const float* acc, int64_t m, int n, int left) {
  #pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (i >= left) break;
    const int64_t at = m * g.N + n + i;
    float z = acc[i];
    if (g.bias) z += g.bias[n + i];
    if (g.pre) g.pre[at] = (uint16_t)f32_to_bf16(z);
    z = activate(z, g.act);
    if (g.residual)
      z += g.c_f32 ? ((const float*)g.residual)[at]
                   : bf16_bits_to_f32(((const uint16_t*)g.residual)[at]);
    if (g.c_f32) ((float*)g.c)[at] = z;
    else ((uint16_t*)g.c)[at] = (uint16_t)f32_to_bf16(z);
  }
}

// Any sizes and any alignment of the rows: 64x64 tiles, 32 values of k a step, elements loaded one
// by one, zeros past the ends.
constexpr int kAnyThreads = 256;
constexpr int kAnyTile = 64, kAnyK = 32;
constexpr int64_t kAnyGrid = 1 << 22;    // workgroups of a launch; more tiles are run by striding

// KA, KB: k is the contiguous dimension of a, of b.
template <bool KA, bool KB>
__global__ __launch_bounds__(kAnyThreads) void any_kernel(Args g) {
  constexpr int PITCH = kAnyK + 8;                     // values
  __shared__ __attribute__((aligned(16))) uint16_t lds[2][kAnyTile * PITCH];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int wm = wave / 2 * 32, wn = wave % 2 * 32;
  const int fr = lane & 15, fq = lane >> 4;
  const int64_t nblk = ((int64_t)g.N + kAnyTile - 1) / kAnyTile;
  const int64_t tiles = ((int64_t)g.M + kAnyTile - 1) / kAnyTile * nblk;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t m0 = tile / nblk * kAnyTile;
    const int n0 = (int)(tile % nblk * kAnyTile);
    f32x4 acc[2][2] = {};
    for (int k0 = 0; k0 < g.K; k0 += kAnyK) {
      auto fill = [&](uint16_t* to, const uint16_t* p, bool kc, int64_t r0, int64_t rows) {
        #pragma unroll
        for (int i = 0; i < kAnyTile * kAnyK / kAnyThreads; ++i) {
          const int q = i * kAnyThreads + threadIdx.x;
          const int k = kc ? q % kAnyK : q / kAnyTile, r = kc ? q / kAnyK : q % kAnyTile;
          const bool in = r0 + r < rows && k0 + k < g.K;
          to[r * PITCH + k] =
              in ? p[kc ? (r0 + r) * g.K + k0 + k : (int64_t)(k0 + k) * rows + r0 + r] : 0;
        }
      };
      fill(lds[0], g.a, KA, m0, g.M);
      fill(lds[1], g.b, KB, n0, g.N);
      __syncthreads();
      #pragma unroll
      for (int i = 0; i < 2; ++i)
        #pragma unroll
        for (int j = 0; j < 2; ++j) {
          const bf16x8 a = OpBf16::load((const char*)&lds[0][(wm + i * 16 + fr) * PITCH + fq * 8]);
          const bf16x8 b = OpBf16::load((const char*)&lds[1][(wn + j * 16 + fr) * PITCH + fq * 8]);
          acc[i][j] = OpBf16::mma(b, a, acc[i][j]);
        }
      __syncthreads();
    }
    #pragma unroll
    for (int i = 0; i < 2; ++i)
      #pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t m = m0 + wm + i * 16 + fr;
        const int n = n0 + wn + j * 16 + fq * 4;
        const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        if (m < g.M) finish<4>(g, v, m, n, g.N - n);
      }
  }
}

hipError_t run_any(const Args& g, int layout, hipStream_t s) {
  const int64_t tiles = ((int64_t)g.M + kAnyTile - 1) / kAnyTile *
                        (((int64_t)g.N + kAnyTile - 1) / kAnyTile);
  const dim3 grid((unsigned)std::min(tiles, kAnyGrid)), block(kAnyThreads);
  if (layout == MOE_NT) hipLaunchKernelGGL((any_kernel<true, true>), grid, block, 0, s, g);
  else if (layout == MOE_NN) hipLaunchKernelGGL((any_kernel<true, false>), grid, block, 0, s, g);
  else hipLaunchKernelGGL((any_kernel<false, false>), grid, block, 0, s, g);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------------------------
// Gradient of the epilogue
// ---------------------------------------------------------------------------------------------
// Beyond 200 every slope is 0 or 1 in fp32, and its formula would multiply 0 by infinity.
__device__ __forceinline__ float slope(float z, int act) {
  if (z == z) z = fminf(fmaxf(z, -200.0f), 200.0f);
  if (act == MOE_ACT_SILU) {
    const float s = 1.0f / (1.0f + expf(-z));
    return s * (1.0f + z * (1.0f - s));
  }
  if (act == MOE_ACT_GELU)
    return 0.5f * (1.0f + erff(z * 0.707106781f)) + z * 0.398942280f * expf(-0.5f * z * z);
  if (act == MOE_ACT_GELU_TANH) {
    // with s = (1 + tanh u) / 2: s + z s (1 - s) 2 u'
    const float s = 1.0f / (1.0f + expf(-gelu_tanh_arg(z)));
    const float du = 1.59576912f * __builtin_fmaf(3.0f * 0.044715f * z, z, 1.0f);
    return s + z * s * (1.0f - s) * du;
  }
  return 1.0f;
}

struct ActArgs {
  const uint16_t *d_c, *pre;
  uint16_t* d_z;
  float* partials;              // [gridDim.y, N] or null
  int M, N, act;
};

// A workgroup takes 256 columns and every gridDim.y-th set of 4 rows, a wave of them each, 4
// neighbouring columns a lane.
constexpr int kActThreads = 256;

__global__ __launch_bounds__(kActThreads) void act_bwd_kernel(ActArgs g) {
  __shared__ float part[kActThreads / kWave][kActCols];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int64_t n0 = (int64_t)blockIdx.x * kActCols + lane * 4;
  const int left = (int)min((int64_t)4, g.N - n0);
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t m = (int64_t)blockIdx.y * 4 + wave; m < g.M; m += (int64_t)gridDim.y * 4) {
    const int64_t at = m * g.N + n0;
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= left) break;
      float d = bf16_bits_to_f32(g.d_c[at + i]);
      if (g.act != MOE_ACT_NONE) {
        d *= slope(bf16_bits_to_f32(g.pre[at + i]), g.act);
        g.d_z[at + i] = (uint16_t)f32_to_bf16(d);
      }
      sum[i] += d;
    }
  }
  if (!g.partials) return;
  #pragma unroll
  for (int i = 0; i < 4; ++i) part[wave][lane * 4 + i] = sum[i];
  __syncthreads();
  const int64_t n = (int64_t)blockIdx.x * kActCols + threadIdx.x;
  if (n >= g.N) return;
  float t = part[0][threadIdx.x];
  #pragma unroll
  for (int w = 1; w < kActThreads / kWave; ++w) t += part[w][threadIdx.x];
  g.partials[(int64_t)blockIdx.y * g.N + n] = t;
}

}  // namespace gb

hipError_t launch_gemm_bf16(const GemmBf16& p, hipStream_t s) {
  gb::Args g{(const uint16_t*)p.a, (const uint16_t*)p.b, p.bias, p.residual, (uint16_t*)p.pre, p.c,
             p.M, p.N, p.K, p.act, p.c_f32};
  return gb::run_any(g, p.layout, s);
}

hipError_t launch_act_bwd(int M, int N, int act, const void* d_c, const void* pre, void* d_z,
                          float* d_bias, float* partials, hipStream_t s) {
  gb::ActArgs g{(const uint16_t*)d_c, (const uint16_t*)pre, (uint16_t*)d_z,
                d_bias ? partials : nullptr, M, N, act};
  const int cus = std::max(device_cu_count(), 8);
  const int cols = (N + kActCols - 1) / kActCols;
  const int rows = act_partial_rows(M, N, cus);
  hipLaunchKernelGGL(gb::act_bwd_kernel, dim3((unsigned)cols, (unsigned)rows),
                     dim3(gb::kActThreads), 0, s, g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !d_bias) return e;
  return launch_sum_rows(rows, N, partials, d_bias, s);
}

}  // namespace moe

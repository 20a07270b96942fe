// HBM-streaming kernels: the per-(row, 128-group) e4m3 quantisation of X and the
// deterministic per-token combine.
#include "moe_internal.h"

namespace moe {

// ---------------------------------------------------------------------------------------------
// X quantisation ("MOE Bmm1 Fused Gather", pack_e4m3x2: round to nearest even with
// saturation to the largest finite e4m3 value).  16 lanes per 128-column group, 8 bf16
// values (16 bytes) per lane, 4 groups per wavefront: the group amax is a 16-lane max
// reduction, s = amax/448 (IEEE division), codes = e4m3(x/s) (IEEE division).
// ---------------------------------------------------------------------------------------------
constexpr int kQuantThreads = 256;
constexpr int kQuantLanes = kGroup / 8;                            // lanes per group
constexpr int kQuantGroupsPerBlock = kQuantThreads / kQuantLanes;  // 16

__global__ __launch_bounds__(kQuantThreads) void quant_rows_e4m3_kernel(
    const i32x4* __restrict__ x8, uint2* __restrict__ xq8, float* __restrict__ scales,
    int64_t n_groups) {
  const int sub = threadIdx.x & (kQuantLanes - 1);
  const int64_t grp = (int64_t)blockIdx.x * kQuantGroupsPerBlock + threadIdx.x / kQuantLanes;
  const bool live = grp < n_groups;
  float v[8];
  float m = 0.0f;
  if (live) {
    const i32x4 w = x8[grp * kQuantLanes + sub];
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_bits_to_f32((uint32_t)w[i] & 0xFFFFu);
      v[2 * i + 1] = bf16_bits_to_f32((uint32_t)w[i] >> 16);
    }
    #pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  }
  // the 16 lanes of a group are aligned within the wavefront: xor offsets below 16 stay in it
  #pragma unroll
  for (int d = kQuantLanes / 2; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, kWave));
  if (!live) return;
  const float s = (m == 0.0f) ? 1.0f : m / kE4M3Max;
  uint32_t lo = 0, hi = 0;
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo |= f32_to_e4m3(v[i] / s) << (8 * i);
    hi |= f32_to_e4m3(v[4 + i] / s) << (8 * i);
  }
  xq8[grp * kQuantLanes + sub] = make_uint2(lo, hi);
  if (sub == 0) scales[grp] = s;
}

hipError_t launch_quant_rows(const Resolved& r, const void* x, uint8_t* xq, float* scales,
                             hipStream_t s) {
  const int64_t groups = (int64_t)r.T * (r.H / kGroup);
  const int64_t blocks = (groups + kQuantGroupsPerBlock - 1) / kQuantGroupsPerBlock;
  hipLaunchKernelGGL(quant_rows_e4m3_kernel, dim3((unsigned)blocks), dim3(kQuantThreads), 0, s,
                     (const i32x4*)x, (uint2*)xq, scales, groups);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------------------------
// The same quantisation along the rows, transposed: x [M, C] -> codes [C, Mp], scales
// [C, Mp/128], Mp = M rounded up to 128.  Operand of a weight gradient, whose sum runs over the
// tokens.  One workgroup takes 128 rows x 64 columns: the tile goes through LDS, a thread takes
// 16 rows of two neighbouring columns (pitch 33 words: the 8 threads of a column pair and the 8
// pairs of a wave read different banks but for a two-way conflict) and stores 16 bytes of each;
// a column's 8 threads write its 128 bytes together.  Rows past M are zeros.  HBM bounds it:
// 4001 x 7168 in 22.8 us (89 MB, 3.9 TB/s), 4001 x 2048 in 10.5 us.
//
// Quotients: IEEE fp32, x / s for one s and 16 values of x: with r = v_rcp_f32(s), q = x r, then
// q += r (x - s q) by two fma, 4 operations a value with its sign instead of 11.  x and the
// amax / 448 behind s have 8 significant bits each, so there are 128 x 128 pairs up to powers of
// two, and every one of them gives the quotient of the division (tests go through them all;
// without the correction 3 of 1000 codes near a midpoint differ).  s outside [2^-96, 2^96] takes
// the division itself.  Quotients are at most 448 up to their rounding (up to 450 where s is
// subnormal), below the 464 from which e4m3 would overflow, so the gfx950 convert (nearest even,
// NaN kept) needs no clamp.
// ---------------------------------------------------------------------------------------------
constexpr int kQuantCols = 64;

__global__ __launch_bounds__(kQuantThreads) void quant_cols_e4m3_kernel(
    const uint16_t* __restrict__ x, uint8_t* __restrict__ xq, float* __restrict__ scales, int M,
    int C, int groups) {
  constexpr int PITCH = kQuantCols / 2 + 1;              // words
  constexpr int ROWS = 16;                               // of a thread
  constexpr int PARTS = kGroup / ROWS;
  __shared__ uint32_t tile[kGroup * PITCH];
  const int g = blockIdx.x % groups;
  const int c0 = (blockIdx.x / groups) * kQuantCols;
  const int64_t m0 = (int64_t)g * kGroup;
  #pragma unroll
  for (int i = 0; i < kGroup * kQuantCols / 8 / kQuantThreads; ++i) {
    const int q = i * kQuantThreads + threadIdx.x;
    const int r = q / (kQuantCols / 8), c = (q % (kQuantCols / 8)) * 8;
    i32x4 v{0, 0, 0, 0};
    if (m0 + r < M && c0 + c < C)                        // C is a multiple of 8
      v = *reinterpret_cast<const i32x4*>(x + (m0 + r) * C + c0 + c);
    #pragma unroll
    for (int k = 0; k < 4; ++k) tile[r * PITCH + c / 2 + k] = (uint32_t)v[k];
  }
  __syncthreads();
  const int part = threadIdx.x % PARTS, pair = threadIdx.x / PARTS;
  float v[2][ROWS];
  float m[2] = {0.0f, 0.0f};
  #pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const uint32_t w = tile[(part * ROWS + i) * PITCH + pair];
    v[0][i] = bf16_bits_to_f32(w & 0xFFFFu);
    v[1][i] = __uint_as_float(w & 0xFFFF0000u);
    m[0] = fmaxf(m[0], fabsf(v[0][i]));
    m[1] = fmaxf(m[1], fabsf(v[1][i]));
  }
  #pragma unroll
  for (int h = 0; h < 2; ++h) {
    #pragma unroll
    for (int d = 1; d < PARTS; d *= 2) m[h] = fmaxf(m[h], __shfl_xor(m[h], d, kWave));
    const int c = c0 + 2 * pair + h;
    if (c >= C) continue;
    const float s = (m[h] == 0.0f) ? 1.0f : m[h] / kE4M3Max;
    if (s >= 0x1p-96f && s <= 0x1p96f) {
      const float r = __builtin_amdgcn_rcpf(s);
      #pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        float q = v[h][i] * r;
        q = __builtin_fmaf(__builtin_fmaf(-s, q, v[h][i]), r, q);
        v[h][i] = __builtin_copysignf(q, v[h][i]);       // -0 stays -0
      }
    } else {
      #pragma unroll
      for (int i = 0; i < ROWS; ++i) v[h][i] = v[h][i] / s;
    }
    i32x4 o;
    #pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = __builtin_amdgcn_cvt_pk_fp8_f32(
          v[h][4 * i + 2], v[h][4 * i + 3],
          __builtin_amdgcn_cvt_pk_fp8_f32(v[h][4 * i], v[h][4 * i + 1], 0, false), true);
    *reinterpret_cast<i32x4*>(xq + (size_t)c * groups * kGroup + m0 + part * ROWS) = o;
    if (part == 0) scales[(size_t)c * groups + g] = s;
  }
}

hipError_t launch_quant_cols(int M, int C, const void* x, uint8_t* xq, float* scales,
                             hipStream_t s) {
  const int groups = (M + kGroup - 1) / kGroup;
  const int64_t blocks = (int64_t)groups * ((C + kQuantCols - 1) / kQuantCols);
  hipLaunchKernelGGL(quant_cols_e4m3_kernel, dim3((unsigned)blocks), dim3(kQuantThreads), 0, s,
                     (const uint16_t*)x, xq, scales, M, C, groups);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------------------------
// Combine ("factor_moe_fused_gemm.cu": index_add_ in the slow path and
// weighted_scatter_add_kernel, which there adds with float atomics).  Here each thread
// owns 16 bytes of one token's output row and adds that token's top_k slot rows in
// ascending j in fp32, then rounds once: no atomics, same bits on every run.
// ---------------------------------------------------------------------------------------------
constexpr int kCombineThreads = 256;

template <bool BF16>
__global__ __launch_bounds__(kCombineThreads) void combine_kernel(
    const i32x4* __restrict__ slot_out, const int32_t* __restrict__ slot_row,
    i32x4* __restrict__ out, int T, int top_k, int vec_per_row) {
  const int64_t idx = (int64_t)blockIdx.x * kCombineThreads + threadIdx.x;
  if (idx >= (int64_t)T * vec_per_row) return;
  const int t = (int)(idx / vec_per_row);
  const int c = (int)(idx - (int64_t)t * vec_per_row);
  constexpr int L = BF16 ? 8 : 4;
  float acc[L];
  #pragma unroll
  for (int i = 0; i < L; ++i) acc[i] = 0.0f;
  // slots in batches of 4: every row load of a batch is issued before the first add.  A slot
  // with an excluded id (another shard's expert) was never written and is not read: on an
  // expert-parallel shard most slots are such.
  constexpr int U = 4;
  for (int j0 = 0; j0 < top_k; j0 += U) {
    int ok[U];
    i32x4 v[U];
    #pragma unroll
    for (int u = 0; u < U; ++u)
      ok[u] = (j0 + u < top_k) ? slot_row[(int64_t)t * top_k + j0 + u] >= 0 : 0;
    #pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t s = (int64_t)t * top_k + j0 + u;
      v[u] = ok[u] ? slot_out[s * vec_per_row + c] : i32x4{0, 0, 0, 0};
    }
    #pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!ok[u]) continue;
      if (BF16) {
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[2 * i] += bf16_bits_to_f32((uint32_t)v[u][i] & 0xFFFFu);
          acc[2 * i + 1] += bf16_bits_to_f32((uint32_t)v[u][i] >> 16);
        }
      } else {
        #pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += __int_as_float(v[u][i]);
      }
    }
  }
  i32x4 o;
  if (BF16) {
    #pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (int)pack_bf16x2(acc[2 * i], acc[2 * i + 1]);
  } else {
    #pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __float_as_int(acc[i]);
  }
  out[idx] = o;
}

hipError_t launch_combine(const Resolved& r, const void* slot_out, const int32_t* slot_row,
                          void* out, hipStream_t s) {
  const bool bf16 = (r.dtype == MOE_BF16);
  const int vec_per_row = r.H * (bf16 ? 2 : 4) / 16;
  const int64_t total = (int64_t)r.T * vec_per_row;
  const unsigned blocks = (unsigned)((total + kCombineThreads - 1) / kCombineThreads);
  if (bf16)
    hipLaunchKernelGGL(combine_kernel<true>, dim3(blocks), dim3(kCombineThreads), 0, s,
                       (const i32x4*)slot_out, slot_row, (i32x4*)out, r.T, r.K, vec_per_row);
  else
    hipLaunchKernelGGL(combine_kernel<false>, dim3(blocks), dim3(kCombineThreads), 0, s,
                       (const i32x4*)slot_out, slot_row, (i32x4*)out, r.T, r.K, vec_per_row);
  return hipGetLastError();
}

}  // namespace moe

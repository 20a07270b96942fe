// Token rows into expert-sorted order and back, and the gradient of the way back.
//
//   permute       : rows[r] = x[sorted_slots[r] / top_k]       padding rows 0
//   unpermute     : out[t]  = sum_j w[t,j] * rows[slot_row[t*top_k+j]]
//   unpermute_bwd : d_rows[r] = w[s] * d_out[t],  d_w[s] = d_out[t] . rows[r],  s = t*top_k+j
//
// (The gather and the weighted scatter that the expert GEMMs fuse, as passes of their own:
// "MOE Bmm1 Fused Gather" load_activations, gather index = slot // top_k;
// "factor_moe_fused_gemm.cu" weighted_scatter_add_kernel, which there adds with atomics.)
//
// All three move rows and compute next to nothing: HBM bounds them.  They walk the tokens, not
// the sorted rows, so each token row (x, d_out) is read once for its top_k slots, and a token's
// slots are added by one thread in ascending j: no atomics, same bits on every run.  Walking the
// sorted rows instead, each gathering its token's, permute takes 64 us of the 53 that it takes for
// 8192 tokens, top 6, 2048 bf16 columns (235 MB: 4.4 TB/s; a fill of as many bytes runs at 6.6, a
// copy at 6.0); one workgroup per slot of a token 59 us.
#include <algorithm>
#include <type_traits>

#include "moe_internal.h"

namespace moe {

namespace pm {

constexpr int kThreads = 256;
constexpr int kPadRows = 8;      // sorted rows whose padding one workgroup clears, at most

struct Args {
  const i32x4* x;               // permute: x; unpermute(_bwd): rows
  const float* x_scales;
  const i32x4* d_out;
  const int32_t* slot_row;
  const int32_t* sorted_slots;
  const int32_t* num_tiles;
  const float* w;               // [N] or null (all 1)
  i32x4* rows;                  // permute: rows; unpermute: out; unpermute_bwd: d_rows
  float* row_scales;
  float* d_w;
  int T, K, vpr;                // tokens, slots per token, 16-byte vectors per row
  int BM, rows_max, tiles_max, groups;   // groups: scales per row (0: none)
  int64_t n_slots;
  int pad_rows;                 // sorted rows whose padding one workgroup clears
  int token_blocks;             // blocks [0, token_blocks) walk tokens, the rest clear padding
  int blocks;                   // all of them; a launch runs at most kMaxGrid and strides
};

// Cap of one launch (threads of a launch are counted in 32 bits); workgroups past it are run by
// striding.
constexpr int kMaxGrid = 1 << 22;

// Rows of valid tiles that hold no slot: zeros (and scales 1, what a row of zeros quantises
// to).  One workgroup looks at pad_rows rows; rows past the last valid tile are left alone.
__device__ __forceinline__ void clear_padding(const Args& g, int block) {
  const int64_t used = (int64_t)min(max(*g.num_tiles, 0), g.tiles_max) * g.BM;
  const int64_t r0 = (int64_t)block * g.pad_rows;
  if (r0 >= used) return;
  int slot[kPadRows];
  #pragma unroll
  for (int i = 0; i < kPadRows; ++i)
    slot[i] = (i < g.pad_rows && r0 + i < used) ? g.sorted_slots[r0 + i] : 0;
  #pragma unroll
  for (int i = 0; i < kPadRows; ++i) {
    if ((uint32_t)slot[i] < (uint32_t)g.n_slots) continue;
    i32x4* row = g.rows + (r0 + i) * g.vpr;
    for (int c = threadIdx.x; c < g.vpr; c += kThreads) row[c] = i32x4{0, 0, 0, 0};
    if (g.row_scales)
      for (int c = threadIdx.x; c < g.groups; c += kThreads)
        g.row_scales[(r0 + i) * g.groups + c] = 1.0f;
  }
}

// A thread owns 16 bytes of one token's row and stores them to each of its slots' rows.
__device__ __forceinline__ void permute_block(const Args& g, int block) {
  if (block >= g.token_blocks) {
    clear_padding(g, block - g.token_blocks);
    return;
  }
  const uint32_t idx = (uint32_t)block * kThreads + threadIdx.x;
  if (idx >= (uint32_t)g.T * (uint32_t)g.vpr) return;    // T * H < 2^31, so T * vpr < 2^29 + 1
  const int t = (int)(idx / (uint32_t)g.vpr);
  const int c = (int)(idx - (uint32_t)t * (uint32_t)g.vpr);
  const i32x4 v = g.x[idx];
  const bool scale = g.row_scales && (c & 7) == 0;   // e4m3: 8 vectors per 128 columns
  const float sc = scale ? g.x_scales[(int64_t)t * g.groups + (c >> 3)] : 0.0f;
  const int32_t* sr = g.slot_row + (int64_t)t * g.K;
  for (int j = 0; j < g.K; ++j) {
    const int r = sr[j];
    if ((uint32_t)r >= (uint32_t)g.rows_max) continue;   // excluded id
    g.rows[(int64_t)r * g.vpr + c] = v;
    if (scale) g.row_scales[(int64_t)r * g.groups + (c >> 3)] = sc;
  }
}

__global__ __launch_bounds__(kThreads) void permute_kernel(Args g) {
  for (int b = blockIdx.x; b < g.blocks; b += gridDim.x) permute_block(g, b);
}

template <bool BF16>
__device__ __forceinline__ void unpack(const i32x4& v, float* f) {
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      f[2 * i] = bf16_bits_to_f32((uint32_t)v[i] & 0xFFFFu);
      f[2 * i + 1] = __uint_as_float((uint32_t)v[i] & 0xFFFF0000u);
    } else {
      f[i] = __int_as_float(v[i]);
    }
  }
}

// One rounding to the row type, to nearest even; the integer rounding of bf16 would carry a NaN
// payload into the exponent's neighbour, so NaN is kept as it is.
template <bool BF16>
__device__ __forceinline__ i32x4 pack(const float* f) {
  i32x4 o;
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      const auto bits = [](float x) {
        return x == x ? f32_to_bf16_bits(x) : (__float_as_uint(x) >> 16) | 0x40u;
      };
      o[i] = (int)(bits(f[2 * i]) | (bits(f[2 * i + 1]) << 16));
    } else {
      o[i] = __float_as_int(f[i]);
    }
  }
  return o;
}

template <bool LARGE>
__device__ __forceinline__ i32x4 load_row(const i32x4* p) {
  if constexpr (LARGE) return __builtin_nontemporal_load(p);
  else return *p;
}

// A thread owns 16 bytes of one token's output row; slots in batches of 4, every row load of a
// batch issued before the first product.  The sum is carried in fp32 and rounded once.
// LARGE (rows of more than 128 MB, half of the last-level cache): every row is read once and loaded
// past the caches, 8192 tokens, top 6, 2048 columns (201 MB) from memory 48.7 -> 42.3 us
// (5.6 TB/s), behind the permute that wrote them 93.6 -> 83.7 us together, before the gradient
// that reads them again 144.7 -> 139.5 us; with 67 MB that last pair takes 58.6 us against 54.4.
template <bool BF16, bool LARGE>
__global__ __launch_bounds__(kThreads) void unpermute_kernel(Args g) {
  const uint32_t idx = (uint32_t)blockIdx.x * kThreads + threadIdx.x;
  if (idx >= (uint32_t)g.T * (uint32_t)g.vpr) return;
  const int t = (int)(idx / (uint32_t)g.vpr);
  const int c = (int)(idx - (uint32_t)t * (uint32_t)g.vpr);
  constexpr int L = BF16 ? 8 : 4;
  float acc[L];
  #pragma unroll
  for (int i = 0; i < L; ++i) acc[i] = 0.0f;
  constexpr int U = 4;
  for (int j0 = 0; j0 < g.K; j0 += U) {
    int r[U];
    float w[U];
    i32x4 v[U];
    #pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t s = (int64_t)t * g.K + min(j0 + u, g.K - 1);
      r[u] = g.slot_row[s];
      w[u] = g.w ? g.w[s] : 1.0f;
    }
    #pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j0 + u >= g.K || (uint32_t)r[u] >= (uint32_t)g.rows_max) r[u] = -1;
      v[u] = i32x4{0, 0, 0, 0};
      if (r[u] >= 0) v[u] = load_row<LARGE>(g.x + (int64_t)r[u] * g.vpr + c);
    }
    #pragma unroll
    for (int u = 0; u < U; ++u) {
      if (r[u] < 0) continue;
      float f[L];
      unpack<BF16>(v[u], f);
      #pragma unroll
      for (int i = 0; i < L; ++i) acc[i] = __builtin_fmaf(w[u], f[i], acc[i]);
    }
  }
  g.rows[idx] = pack<BF16>(acc);
}

// WPS wavefronts per slot: the token's d_out row and the slot's row are walked once, giving the
// slot's d_rows row and (sums in a fixed order) its d_w.  With one wavefront the waves of a
// workgroup belong to neighbouring slots, most of them of one token, whose d_out row then comes
// from L1/L2.  With few slots a workgroup's four share one (one token, top 8, 7168 columns: 8.1 us
// with one).  LARGE as above (97.8 -> 93.3 us from memory); stores past the caches as well, 86 us,
// cost whoever reads d_rows next more than they gain (with a reader behind it 119 -> 137 us).
template <bool BF16, int WPS, bool LARGE>
__device__ __forceinline__ void unpermute_bwd_block(const Args& g, int block, float* sums) {
  if (block >= g.token_blocks) {
    clear_padding(g, block - g.token_blocks);
    return;
  }
  constexpr int L = BF16 ? 8 : 4;
  constexpr int SPB = kThreads / kWave / WPS;            // slots per workgroup
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t s = (int64_t)block * SPB + wave / WPS;
  if (s >= g.n_slots) return;                            // SPB > 1 only: whole wavefronts
  const int r = g.slot_row[s];
  const bool there = (uint32_t)r < (uint32_t)g.rows_max;   // else an excluded id: no gradient
  float dot = 0.0f;
  if (there) {
    const float w = g.w ? g.w[s] : 1.0f;
    const i32x4* d = g.d_out + (s / g.K) * g.vpr;
    const i32x4* x = g.x + (int64_t)r * g.vpr;
    i32x4* o = g.rows + (int64_t)r * g.vpr;
    constexpr int U = 4;
    for (int c0 = wave % WPS * kWave + lane; c0 < g.vpr; c0 += U * WPS * kWave) {
      i32x4 dv[U], xv[U];
      #pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = min(c0 + u * WPS * kWave, g.vpr - 1);
        dv[u] = d[c];
        if (g.d_w) xv[u] = load_row<LARGE>(&x[c]);
      }
      #pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * WPS * kWave;
        if (c >= g.vpr) continue;
        float df[L];
        unpack<BF16>(dv[u], df);
        if (g.d_w) {
          float xf[L];
          unpack<BF16>(xv[u], xf);
          #pragma unroll
          for (int i = 0; i < L; ++i) dot = __builtin_fmaf(df[i], xf[i], dot);
        }
        if (g.rows) {
          #pragma unroll
          for (int i = 0; i < L; ++i) df[i] *= w;
          o[c] = pack<BF16>(df);
        }
      }
    }
  }
  if (!g.d_w) return;
  #pragma unroll
  for (int m = kWave / 2; m >= 1; m >>= 1) dot += __shfl_xor(dot, m, kWave);
  if constexpr (WPS > 1) {
    if (lane == 0) sums[wave] = dot;
    __syncthreads();
    dot = 0.0f;
    #pragma unroll
    for (int i = 0; i < WPS; ++i) dot += sums[i];
    __syncthreads();                                     // before the next block's sums
    if (wave > 0) return;
  }
  if (lane == 0) g.d_w[s] = dot;
}

template <bool BF16, int WPS, bool LARGE>
__global__ __launch_bounds__(kThreads) void unpermute_bwd_kernel(Args g) {
  static_assert(WPS == 1 || WPS == kThreads / kWave, "one slot per workgroup, or one per wave");
  __shared__ float sums[kThreads / kWave];
  for (int b = blockIdx.x; b < g.blocks; b += gridDim.x)
    unpermute_bwd_block<BF16, WPS, LARGE>(g, b, sums);
}

Args args(const Resolved& r, int row_dtype) {
  Args a{};
  a.T = r.T;
  a.K = r.K;
  a.vpr = r.H * (row_dtype == MOE_F32 ? 4 : row_dtype == MOE_BF16 ? 2 : 1) / 16;
  a.BM = r.BM;
  a.rows_max = (int)r.rows_max;
  a.tiles_max = (int)r.tiles_max;
  a.groups = r.H / kGroup;
  a.n_slots = r.N;
  // A workgroup's rows are cleared one after the other, and one that finds none to clear costs its
  // launch.  8 rows, but 4 where the padding may be as many rows as the slots and a row takes a
  // workgroup more than one store.  Top 8 of 256 in blocks of 128, 4 rows against 8: 7168 codes 53.1
  // against 55.0 us (2048 tokens), 53.1 against 57.6 (1500), 51.1 against 53.1 (1024), 2048 fp32
  // columns 50.9 against 54.6 (1024 tokens); with rows of one store 32.0 against 28.1 (2048 tokens,
  // 2048 bf16 columns; 26.3 against 27.8 at 512), with less padding 59.4 against 57.8 (3000 tokens,
  // 4096 bf16 columns).
  const bool much = r.rows_max - r.N >= r.N && a.vpr > kThreads;
  a.pad_rows = much ? kPadRows / 2 : kPadRows;
  return a;
}

bool large(const Resolved& r, const Args& a) { return r.N * a.vpr * 16 > (128LL << 20); }

template <class F>
void by_type(bool bf16, bool large, F f) {
  if (bf16 && large) f(std::true_type{}, std::true_type{});
  else if (bf16) f(std::true_type{}, std::false_type{});
  else if (large) f(std::false_type{}, std::true_type{});
  else f(std::false_type{}, std::false_type{});
}

int pad_blocks(const Args& a) {
  return (int)(((int64_t)a.rows_max + a.pad_rows - 1) / a.pad_rows);
}

}  // namespace pm

hipError_t launch_permute(const Resolved& r, int row_dtype, const void* x, const float* x_scales,
                          const int32_t* slot_row, const int32_t* sorted_slots,
                          const int32_t* num_tiles, void* rows, float* row_scales, hipStream_t s) {
  pm::Args a = pm::args(r, row_dtype);
  a.x = (const i32x4*)x;
  a.x_scales = x_scales;
  a.slot_row = slot_row;
  a.sorted_slots = sorted_slots;
  a.num_tiles = num_tiles;
  a.rows = (i32x4*)rows;
  a.row_scales = row_scales;
  a.token_blocks = (int)(((int64_t)r.T * a.vpr + pm::kThreads - 1) / pm::kThreads);
  a.blocks = a.token_blocks + pm::pad_blocks(a);
  hipLaunchKernelGGL(pm::permute_kernel, dim3((unsigned)std::min(a.blocks, pm::kMaxGrid)),
                     dim3(pm::kThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_unpermute(const Resolved& r, int row_dtype, const void* rows,
                            const int32_t* slot_row, const float* topk_w, void* out,
                            hipStream_t s) {
  pm::Args a = pm::args(r, row_dtype);
  a.x = (const i32x4*)rows;
  a.slot_row = slot_row;
  a.w = topk_w;
  a.rows = (i32x4*)out;
  const dim3 grid((unsigned)(((int64_t)r.T * a.vpr + pm::kThreads - 1) / pm::kThreads));
  pm::by_type(row_dtype == MOE_BF16, pm::large(r, a), [&](auto bf16, auto large) {
    hipLaunchKernelGGL((pm::unpermute_kernel<bf16.value, large.value>), grid, dim3(pm::kThreads), 0,
                       s, a);
  });
  return hipGetLastError();
}

hipError_t launch_unpermute_bwd(const Resolved& r, int row_dtype, const void* d_out,
                                const void* rows, const int32_t* slot_row,
                                const int32_t* sorted_slots, const int32_t* num_tiles,
                                const float* topk_w, void* d_rows, float* d_w, hipStream_t s) {
  pm::Args a = pm::args(r, row_dtype);
  a.x = (const i32x4*)rows;
  a.d_out = (const i32x4*)d_out;
  a.slot_row = slot_row;
  a.sorted_slots = sorted_slots;
  a.num_tiles = num_tiles;
  a.w = topk_w;
  a.rows = (i32x4*)d_rows;
  a.d_w = d_w;
  constexpr int kWaves = pm::kThreads / kWave;
  const bool few = r.N < 2048;          // fewer waves than 8 per compute unit of 256
  a.token_blocks = (int)(few ? r.N : (r.N + kWaves - 1) / kWaves);
  a.blocks = a.token_blocks + (d_rows ? pm::pad_blocks(a) : 0);
  const dim3 grid((unsigned)std::min(a.blocks, pm::kMaxGrid)), block(pm::kThreads);
  pm::by_type(row_dtype == MOE_BF16, pm::large(r, a), [&](auto bf16, auto large) {
    if (few)
      hipLaunchKernelGGL((pm::unpermute_bwd_kernel<bf16.value, kWaves, false>), grid, block, 0, s,
                         a);
    else
      hipLaunchKernelGGL((pm::unpermute_bwd_kernel<bf16.value, 1, large.value>), grid, block, 0, s,
                         a);
  });
  return hipGetLastError();
}

}  // namespace moe

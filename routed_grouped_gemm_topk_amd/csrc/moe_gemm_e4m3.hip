// Products of e4m3 codes with one fp32 scale per 128 values along K:
//
//   c[m, n] = sum over 128-wide groups g of  sa[m, g] * sb[., g] * ( a[m, g] . b[n, g] )
//
// dense (a [M, K] times b [N, K]^T) or over expert-sorted rows (every m-block of the alignment's
// tile table times its expert's b).  b's scales are per 128x128 block (weights) or per row (the
// weight gradient, whose two operands are quantised along the tokens).
//
// gfx950 v_mfma_f32_16x16x128_f8f6f4 takes exactly one group per instruction: its fp32 result is
// the group's unscaled product, scaled by one fma per value into the fp32 accumulators.  The
// operand order puts b's rows on the result's rows and a's rows on its columns, so a lane holds
// ONE row of a and its scale is one register, and 4 neighbouring n, which it stores together.
#include "moe_internal.h"

namespace moe {

namespace q8 {

constexpr int ROWB = 128;      // bytes per row per k-slice: one scale group
constexpr int kChunk = 32;     // logical tiles per chunk dealt to one XCD (xcd_chunked)
constexpr int kGroupM = 8;     // m-blocks that sweep the n-blocks together

struct Args {
  const uint8_t* a;
  const float* sa;              // [M, K/128]
  const uint8_t* b;
  const float* sb;              // [ceil(N/128), K/128] or [N, K/128]
  void* c;
  const int32_t* offsets;       // grouped: outputs of the alignment
  const int32_t* tiles;
  const int32_t* num_tiles;
  int tiles_max, E;
  int M, N, K;
};

__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// Raw buffer descriptor of [base, base + bytes): a lane whose offset is past `bytes` reads zeros
// without touching memory.
__device__ __forceinline__ i32x4 buf_rsrc(const void* base, uint32_t bytes) {
  const unsigned long long a = (unsigned long long)base;
  i32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));   // stride 0
  r[2] = __builtin_amdgcn_readfirstlane((int)bytes);                 // num_records (bytes)
  r[3] = 0x00020000;                                                 // raw 32-bit data
  return r;
}

// 64 lanes x 16 (4) bytes from the buffer at voff + soff straight to LDS at M0.
__device__ __forceinline__ void buf_dma16(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               ::"v"(voff), "s"(rsrc), "s"(soff), "s"(lds) : "memory");
}
__device__ __forceinline__ void buf_dma4(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\tbuffer_load_dword %0, %1, %2 offen lds"
               ::"v"(voff), "s"(rsrc), "s"(soff), "s"(lds) : "memory");
}

constexpr uint32_t kPastEnd = 0x80000000u;   // past every descriptor below (all < 2^31 bytes)

// Four neighbouring n of one row of c.
template <bool F32>
__device__ __forceinline__ void store4(void* c, int64_t at, const f32x4& v, int n_left, bool vec) {
  if constexpr (F32) {
    float* p = (float*)c + at;
    if (vec && n_left >= 4) {
      *(f32x4*)p = v;
    } else {
      #pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n_left) p[i] = v[i];
    }
  } else {
    uint16_t* p = (uint16_t*)c + at;
    uint32_t h[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i)       // to nearest even; NaN stays NaN
      h[i] = v[i] == v[i] ? f32_to_bf16_bits(v[i]) : 0x7FC0u;
    if (vec && n_left >= 4) {
      *(uint2*)p = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    } else {
      #pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n_left) p[i] = (uint16_t)h[i];
    }
  }
}

// One BM x BN tile of c per workgroup of WM x WN waves; 128-byte k-slices of both operands in a
// ring of NS LDS stages, copied by direct-to-LDS loads NS-1 slices ahead.
template <int BM, int BN, int WM, int WN, int NS, bool BROW, bool F32, bool GROUPED>
__global__ __launch_bounds__(WM * WN * kWave) void tile_kernel(Args g) {
  constexpr int NW = WM * WN;
  constexpr int WTM = BM / WM, WTN = BN / WN;        // a wave's rows of a and of b
  constexpr int FM = WTM / 16, FN = WTN / 16;
  constexpr int NQ_REAL = (BM + BN) * ROWB / 1024;   // 1 KB copies (8 rows) per slice
  constexpr int NQ = (NQ_REAL + NW - 1) / NW * NW;   // padded to whole waves
  constexpr int NQW = NQ / NW;
  constexpr int SA = (BM + 63) / 64;                 // 64-row copies of a's scales ...
  constexpr int SB = BROW ? (BN + 63) / 64 : 1;      // ... and of b's
  constexpr int NSW = (SA + SB + NW - 1) / NW;       // scale copies per wave
  constexpr int SC_OFF = NQ * 1024;
  constexpr int STAGE = SC_OFF + NSW * NW * 256;
  constexpr int OPS = NQW + NSW;
  static_assert(BM % 8 == 0 && WTM % 16 == 0 && WTN % 16 == 0, "whole copies and MFMA tiles");
  static_assert(BROW || kGroup % WTN == 0, "one scale block per wave");
  static_assert(NS >= 2 && (NS - 1) * OPS <= 63, "vmcnt range");
  static_assert(NS * STAGE <= 160 * 1024, "LDS");

  __shared__ __attribute__((aligned(1024))) char lds[NS * STAGE];

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wn = wave % WN, wm = wave / WN;
  const int K = g.K, KT = K / ROWB;
  const int nblk = (g.N + BN - 1) / BN;

  // ---- tile ----------------------------------------------------------------------------------
  const uint8_t* a;
  const float* sa;
  const uint8_t* b = g.b;
  const float* sb = g.sb;
  int64_t row0;
  int rows, n0;                                      // rows of a in this tile
  if constexpr (GROUPED) {
    const int nt = min(max(*g.num_tiles, 0), g.tiles_max);
    const int logical = xcd_chunked<kChunk>(blockIdx.x, nt * nblk);
    if (logical < 0) return;
    const TileRef t = grouped_tile<BM, kGroupM>(logical, nblk, g.tiles, g.offsets);
    row0 = t.row0;
    rows = BM;
    n0 = t.nt * BN;
    const int sb_rows = BROW ? g.N : (g.N + kGroup - 1) / kGroup;
    b += (size_t)t.e * g.N * K;
    sb += (size_t)t.e * sb_rows * KT;
  } else {
    const int mblk = (g.M + BM - 1) / BM;
    const int logical = xcd_chunked<kChunk>(blockIdx.x, mblk * nblk);
    if (logical < 0) return;
    // groups of kGroupM m-blocks sweep the n-blocks
    const int grp = logical / (kGroupM * nblk);
    const int gm = min(kGroupM, mblk - grp * kGroupM);
    const int w = logical - grp * kGroupM * nblk;
    row0 = (int64_t)(grp * kGroupM + w % gm) * BM;
    rows = (int)min((int64_t)BM, (int64_t)g.M - row0);
    n0 = w / gm * BN;
  }
  const int cols = min(BN, g.N - n0);                // rows of b in this tile
  a = g.a + (size_t)row0 * K;
  sa = g.sa + (size_t)row0 * KT;
  b += (size_t)n0 * K;
  sb += (size_t)(BROW ? n0 : n0 / kGroup) * KT;

  // ---- this wave's copies: rows past the operand's end read as zeros ---------------------------
  const i32x4 ra = buf_rsrc(a, (uint32_t)rows * (uint32_t)K);
  const i32x4 rb = buf_rsrc(b, (uint32_t)cols * (uint32_t)K);
  const i32x4 rsa = buf_rsrc(sa, (uint32_t)rows * KT * 4);
  const int sbn = BROW ? cols : (cols + kGroup - 1) / kGroup;
  const i32x4 rsb = buf_rsrc(sb, (uint32_t)sbn * KT * 4);
  uint32_t voff[NQW];
  #pragma unroll
  for (int i = 0; i < NQW; ++i) {
    const int q = wave * NQW + i;
    int r = q * 8 + (lane >> 3);
    const int cc = (lane & 7) ^ swz(r);
    const bool is_a = q < BM / 8;
    if (!is_a) r -= BM;
    voff[i] = r < (is_a ? rows : cols) && q < NQ_REAL ? (uint32_t)r * (uint32_t)K + cc * 16 : kPastEnd;
  }
  uint32_t soff[NSW];
  #pragma unroll
  for (int i = 0; i < NSW; ++i) {
    const int q = wave * NSW + i;
    const bool is_a = q < SA;
    const int r = (is_a ? q : q - SA) * 64 + lane;
    soff[i] = r < (is_a ? rows : sbn) ? (uint32_t)r * KT * 4 : kPastEnd;
  }
  const uint32_t lds_base = lds_u32(lds);
  auto issue = [&](int buf, int kt) {
    const uint32_t st = __builtin_amdgcn_readfirstlane(lds_base + buf * STAGE);
    #pragma unroll
    for (int i = 0; i < NQW; ++i) {
      const int q = wave * NQW + i;
      buf_dma16(q < BM / 8 ? ra : rb, voff[i], (uint32_t)kt * ROWB, st + q * 1024);
    }
    #pragma unroll
    for (int i = 0; i < NSW; ++i) {
      const int q = wave * NSW + i;
      buf_dma4(q < SA ? rsa : rsb, soff[i], (uint32_t)kt * 4, st + SC_OFF + q * 256);
    }
  };

  // ---- fragments: lane holds row lane & 15, bytes [(lane >> 4) * 32, +32) of the slice ---------
  const int fr = lane & 15, fq = lane >> 4;
  const int off0 = fr * ROWB + (((2 * fq) ^ swz(fr)) << 4);
  const int off1 = fr * ROWB + (((2 * fq + 1) ^ swz(fr)) << 4);
  auto frag = [&](const char* p) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(p + off0);
    const i32x4 hi = *reinterpret_cast<const i32x4*>(p + off1);
    i32x8 f;
    f[0] = lo[0]; f[1] = lo[1]; f[2] = lo[2]; f[3] = lo[3];
    f[4] = hi[0]; f[5] = hi[1]; f[6] = hi[2]; f[7] = hi[3];
    return f;
  };

  f32x4 acc[FM][FN];
  #pragma unroll
  for (int i = 0; i < FM; ++i)
    #pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  #pragma unroll
  for (int s = 0; s < NS - 1; ++s) issue(s, min(s, KT - 1));
  int buf = 0;
  for (int kt = 0; kt < KT; ++kt) {
    wait_vmcnt<(NS - 2) * OPS>();                    // this wave's copies of slice kt
    __syncthreads();
    // past the last slice: repeat it, never read
    issue(buf == 0 ? NS - 1 : buf - 1, min(kt + NS - 1, KT - 1));
    const char* st = lds + buf * STAGE;
    const float* sca = reinterpret_cast<const float*>(st + SC_OFF) + wm * WTM;
    const float* scb = reinterpret_cast<const float*>(st + SC_OFF + SA * 256);
    i32x8 bf[FN];
    #pragma unroll
    for (int j = 0; j < FN; ++j) bf[j] = frag(st + (BM + wn * WTN + j * 16) * ROWB);
    f32x4 s4[BROW ? FN : 1];
    float s1 = 0.0f;
    if constexpr (BROW) {
      #pragma unroll
      for (int j = 0; j < FN; ++j)
        s4[j] = *reinterpret_cast<const f32x4*>(scb + wn * WTN + j * 16 + fq * 4);
    } else {
      s1 = scb[wn * WTN / kGroup];
    }
    #pragma unroll
    for (int i = 0; i < FM; ++i) {
      const i32x8 af = frag(st + (wm * WTM + i * 16) * ROWB);
      const float s = sca[i * 16 + fr];
      f32x4 part[FN];
      #pragma unroll
      for (int j = 0; j < FN; ++j) part[j] = OpE4M3::mma(bf[j], af, f32x4{0.f, 0.f, 0.f, 0.f});
      #pragma unroll
      for (int j = 0; j < FN; ++j)
        #pragma unroll
        for (int v = 0; v < 4; ++v)
          acc[i][j][v] = __builtin_fmaf(part[j][v], BROW ? s * s4[BROW ? j : 0][v] : s * s1,
                                        acc[i][j][v]);
    }
    buf = (buf + 1 == NS) ? 0 : buf + 1;
  }
  wait_vmcnt<0>();

  // ---- c: lane holds row lane & 15 of a, b's rows (lane >> 4) * 4 + v ---------------------------
  const bool vec = (g.N & 3) == 0;
  #pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m = wm * WTM + i * 16 + fr;
    if (m >= rows) continue;
    #pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int n = wn * WTN + j * 16 + fq * 4;
      if (n < cols)
        store4<F32>(g.c, (row0 + m) * (int64_t)g.N + n0 + n, acc[i][j], cols - n, vec);
    }
  }
}

template <int BM, int BN, int WM, int WN, int NS, bool BROW, bool GROUPED>
hipError_t run_tile(const Args& a, bool f32, hipStream_t s) {
  const int64_t mblk = GROUPED ? a.tiles_max : ((int64_t)a.M + BM - 1) / BM;
  const int64_t grid = xcd_chunked_grid<kChunk>(mblk * ((a.N + BN - 1) / BN));
  if (f32)
    hipLaunchKernelGGL((tile_kernel<BM, BN, WM, WN, NS, BROW, true, GROUPED>),
                       dim3((unsigned)grid), dim3(WM * WN * kWave), 0, s, a);
  else
    hipLaunchKernelGGL((tile_kernel<BM, BN, WM, WN, NS, BROW, false, GROUPED>),
                       dim3((unsigned)grid), dim3(WM * WN * kWave), 0, s, a);
  return hipGetLastError();
}

}  // namespace q8

int64_t gemm_e4m3_split_bytes(int, int, int) { return 0; }

hipError_t launch_gemm_e4m3(int M, int N, int K, const uint8_t* a, const float* sa,
                            const uint8_t* b, const float* sb, bool b_rows, void* c, bool c_f32,
                            void*, hipStream_t s) {
  q8::Args g{};
  g.a = a; g.sa = sa; g.b = b; g.sb = sb; g.c = c;
  g.M = M; g.N = N; g.K = K;
  if (b_rows) return q8::run_tile<128, 128, 2, 2, 3, true, false>(g, c_f32, s);
  return q8::run_tile<128, 128, 2, 2, 3, false, false>(g, c_f32, s);
}

hipError_t launch_grouped_gemm_e4m3(const Resolved& r, int N, int K, const uint8_t* rows,
                                    const float* row_scales, const uint8_t* w,
                                    const float* w_scales, const int32_t* offsets,
                                    const int32_t* tiles, const int32_t* num_tiles, void* out,
                                    bool out_f32, hipStream_t s) {
  q8::Args g{};
  g.a = rows; g.sa = row_scales; g.b = w; g.sb = w_scales; g.c = out;
  g.offsets = offsets; g.tiles = tiles; g.num_tiles = num_tiles;
  g.tiles_max = (int)r.tiles_max;
  g.E = r.E;
  g.M = (int)r.rows_max; g.N = N; g.K = K;
  switch (r.BM) {
    case 16: return q8::run_tile<16, 128, 1, 4, 3, false, true>(g, out_f32, s);
    case 32: return q8::run_tile<32, 128, 1, 4, 3, false, true>(g, out_f32, s);
    case 64: return q8::run_tile<64, 128, 1, 4, 3, false, true>(g, out_f32, s);
    case 128: return q8::run_tile<128, 128, 2, 2, 3, false, true>(g, out_f32, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace moe

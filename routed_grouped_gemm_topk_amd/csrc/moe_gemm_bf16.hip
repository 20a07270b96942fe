// Products of bf16 matrices with bias, activation and residual in their epilogue, and the gradient
// of that epilogue:
//
//   z = a b^T | a b | a^T b  (+ bias),   pre = round(z),   c = round(act(z) + residual)
//   d_z = round(d_c act'(pre)),  d_bias = sum over rows of d_c act'(pre)
//
// Accumulated in fp32 by the bf16 matrix instructions.  The operand order puts b on a result's rows
// and a on its columns, so a lane holds 4 neighbouring columns of ONE row of c.
//
// Measured, kernels alone, operands from memory (a large library product reaches 1390 TFLOP/s here):
//   4096 x 14336 x 4096 367 us, 8192^3 753 us (1460 TFLOP/s); 4096 x 4096 x 14336 with residual 341 us
//   (1410): matrix cores busy 70% at 1.87 GHz
//   4096^3 a b^T, a b, a^T b 108, 112, 114 us (1210-1270 TFLOP/s)
//   64 x 256 x 7168 8.2 us, 1 x 256 x 7168 6.7 us: the chain of slices of one tile; 1 x 4096 x 7168
//   11.9 us, 4.9 TB/s of the weights
//   rows of any alignment, 2047^3: 48, 49, 52 us (2048^3: 21, 22, 23); 3 x 5 x 14001 a b^T 14.5 us
#include <algorithm>
#include <type_traits>

#include "moe_gemm_bf16_choice.h"
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

// 1 / (1 + exp(-z)): 6 u off (u = 2^-24); exactly 0 below -88, where z may be anything.
__device__ __forceinline__ float sigmoid_of(float z) {
  const float s = __builtin_amdgcn_rcpf(1.0f + exp_of(__builtin_amdgcn_fmed3f(-z, -88.0f, 88.0f)));
  return z < -88.0f ? 0.0f : s;
}

// The part of a normal distribution below -a is exp(-a^2 / 2) times this, 10 u off for 0 <= a <= 14, so
// that GELU does not cancel below 0 as 1 + erf does (z = -5: one digit left).  (a + 4.75) times it is a
// polynomial in (a - 4.75) / (a + 4.75), the variable of Shepherd and Laframboise (1981), fitted to the
// least relative error (0.24 u); beyond 14 the exponential is 0.
__device__ __forceinline__ float tail_ratio(float a) {
  const float w = __builtin_amdgcn_rcpf(a + 4.75f), q = __builtin_fmaf(w, -9.5f, 1.0f);
  float p = -1.304180477745831e-3f;
  p = __builtin_fmaf(p, q, 2.3066371795721352e-4f);
  p = __builtin_fmaf(p, q, 1.1544439941644669e-2f);
  p = __builtin_fmaf(p, q, -5.0630372017621994e-2f);
  p = __builtin_fmaf(p, q, 0.13810624182224274f);
  p = __builtin_fmaf(p, q, -0.28418365120887756f);
  p = __builtin_fmaf(p, q, 0.4720644950866699f);
  p = __builtin_fmaf(p, q, -0.6535893678665161f);
  return w * __builtin_fmaf(p, q, 0.7664163112640381f);
}
__device__ __forceinline__ float bell(float z) { return exp_of(fmaxf(-0.5f * z * z, -88.0f)); }

__device__ __forceinline__ float activate(float z, int act) {
  if (act == MOE_ACT_SILU) return z * sigmoid_of(z);
  if (act == MOE_ACT_GELU) {
    const float a = fminf(fabsf(z), 14.0f), tail = bell(z) * tail_ratio(a);
    return z < 0.0f ? z * tail : z - a * tail;
  }
  // (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
  if (act == MOE_ACT_GELU_TANH) return z * sigmoid_of(gelu_tanh_arg(z));
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

// ---------------------------------------------------------------------------------------------
// Tiles of c through LDS
// ---------------------------------------------------------------------------------------------
constexpr int ROWB = 128;       // bytes of a row of LDS
constexpr int kGroupM = 8;      // m-blocks that sweep the n-blocks together

// One tile of c: rows [m0, m0 + rows) x columns [n0, n0 + cols).
struct Tile {
  int64_t m0;
  int n0, rows, cols;
};

// Tile `logical` of the product: groups of kGroupM m-blocks sweep the n-blocks.
template <int BM, int BN>
__device__ __forceinline__ Tile tile_at(const Args& g, int logical) {
  const int mblk = (g.M + BM - 1) / BM, nblk = (g.N + BN - 1) / BN;
  const int grp = logical / (kGroupM * nblk);
  const int gm = min(kGroupM, mblk - grp * kGroupM);
  const int w = logical - grp * kGroupM * nblk;
  Tile t;
  t.m0 = (int64_t)(grp * kGroupM + w % gm) * BM;
  t.n0 = w / gm * BN;
  t.rows = (int)min((int64_t)BM, (int64_t)g.M - t.m0);
  t.cols = min(BN, g.N - t.n0);
  return t;
}

// Eight values of a row of c, rows being whole 16-byte blocks.
struct Eight {
  i32x4 lo, hi;                 // hi: fp32 only
  __device__ __forceinline__ float get(int i, bool f32) const {
    if (f32) return __int_as_float(i < 4 ? lo[i] : hi[i - 4]);
    const uint32_t w = (uint32_t)lo[i / 2];
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  }
};
__device__ __forceinline__ Eight load8(const void* p, int64_t at, bool f32) {
  Eight e;
  if (f32) {
    e.lo = *(const i32x4*)((const float*)p + at);
    e.hi = *(const i32x4*)((const float*)p + at + 4);
  } else {
    e.lo = *(const i32x4*)((const uint16_t*)p + at);
    e.hi = i32x4{0, 0, 0, 0};
  }
  return e;
}
__device__ __forceinline__ i32x4 pack8(const float* v) {
  return i32x4{(int)f32_to_bf16x2(v[0], v[1]), (int)f32_to_bf16x2(v[2], v[3]),
               (int)f32_to_bf16x2(v[4], v[5]), (int)f32_to_bf16x2(v[6], v[7])};
}
__device__ __forceinline__ void finish8(const Args& g, const f32x4& z0, const f32x4& z1, int64_t at,
                                        int n, const Eight& res) {
  float z[8] = {z0[0], z0[1], z0[2], z0[3], z1[0], z1[1], z1[2], z1[3]};
  if (g.bias) {
    #pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += g.bias[n + i];
  }
  if (g.pre) *(i32x4*)(g.pre + at) = pack8(z);
  if (g.act != MOE_ACT_NONE) {
    #pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = activate(z[i], g.act);
  }
  if (g.residual) {
    #pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += res.get(i, g.c_f32);
  }
  if (g.c_f32) {
    f32x4* to = (f32x4*)((float*)g.c + at);
    to[0] = f32x4{z[0], z[1], z[2], z[3]};
    to[1] = f32x4{z[4], z[5], z[6], z[7]};
  } else {
    *(i32x4*)((uint16_t*)g.c + at) = pack8(z);
  }
}

// Eight values from place `at` of an operand of `total`, of any alignment, of which the first `left` are
// wanted; `get` leaves zeros for the others.  They are loaded whole where they reach past the wanted
// ones, and at the operand's end from where they still lie in it.
struct Piece {
  i32x4 v;                      // not loaded where fix is 0
  int fix;                      // wanted values, from value fix / 16 of v on
  __device__ __forceinline__ void load(const uint16_t* p, int64_t at, int64_t total, int left) {
    fix = 0;
    if (left <= 0) return;
    if (total >= kChunk) {
      const int64_t start = min(at, total - kChunk);
      __builtin_memcpy(&v, p + start, 16);             // of 2-byte alignment
      fix = min(left, kChunk) | (int)(at - start) << 4;
    } else {
      v = i32x4{0, 0, 0, 0};
      fix = kChunk;
      #pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (i < left) v[i / 2] |= (int)((uint32_t)p[at + i] << (16 * (i & 1)));
    }
  }
  __device__ __forceinline__ i32x4 get() const {
    i32x4 o = v;
    if (fix != kChunk) {
      const int left = fix & 15, off = fix >> 4;
      if (off & 4) o = i32x4{o[2], o[3], 0, 0};
      if (off & 2) o = i32x4{o[1], o[2], o[3], 0};
      if (off & 1) {
        #pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = (int)((uint32_t)o[i] >> 16 | (uint32_t)(i < 3 ? o[i + 1] : 0) << 16);
      }
      #pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = left >= 2 * i + 2 ? o[i] : left == 2 * i + 1 ? o[i] & 0xffff : 0;
    }
    return o;
  }
};

// BM x BN tile by WM x WN waves; slices of 64 values of k of both operands in rings of LDS stages,
// NSA of a and NSB of b, copied by direct-to-LDS loads.  KG groups of WM x WN waves take every KG-th
// slice each and their sums are added at the end in the order of the groups.
//
// KA, KB: k is the contiguous dimension of the operand.  Then a stage holds its rows, 128 bytes of k
// each, chunk c of row r at c ^ swz(r).  Otherwise it holds panels of 64 columns, each 64 rows of k
// of 128 bytes, and the fragments are read with the transposing LDS load: 16 lanes name 4 rows of
// k times 16 columns, and each receives one column's 4 values.  Half a wave reads rows k of
// {0-3, 16-19} (+ 4, 8, 12, 32 ...), whose pairs of chunks lie at c ^ 2 f with f = bit 1 of k and twice
// bit 4 of k: all on different banks.  A lane's values of k are those of the other form: matrix
// instruction t of a slice takes k = 16 (lane / 16) + 8 t + 0..7 of every lane.
template <int BM, int BN, int WM, int WN, int KG, int NSA, int NSB, bool KA, bool KB>
struct TileGemm {
  static constexpr int NW = WM * WN;
  static constexpr int WTM = BM / WM, WTN = BN / WN;        // a wave's part of the tile
  static constexpr int FM = WTM / 16, FN = WTN / 16;
  static constexpr int CA = BM / 8 / NW, CB = BN / 8 / NW;  // a wave's 1 KB copies per slice
  static constexpr int STAGE_A = BM * ROWB, STAGE_B = BN * ROWB;
  static constexpr int RING_B = NSA * KG * STAGE_A;         // where b's ring begins
  static constexpr int RING = RING_B + NSB * KG * STAGE_B;
  static constexpr int SUMS = (KG - 1) * NW * FM * FN * kWave * 16;
  static constexpr int PITCH = WTN * 4 + 16;
  static constexpr int OUTF = FM <= 4 ? FM : FM % 4 ? 3 : 4;   // fragments turned around at a time
  static constexpr int OUT_OFF = KG > 1 ? SUMS : 0;
  static constexpr int OUT = OUT_OFF + NW * OUTF * 16 * PITCH;
  static constexpr int LDS = RING > OUT ? RING : OUT;
  // A slice is multiplied in STEPS: both matrix instructions' halves of k, one after the other, and
  // in each the fragments of a.  A fragment of a is read AHEAD steps before its products.
  static constexpr int STEPS = 2 * FM, AHEAD = 3;
  static constexpr int LAST = STEPS - 1 - AHEAD;            // the step that reads the slice's last
  static constexpr int BSTEPS = std::min({LAST + 1, FM, FN});           // that read b's second half
  static constexpr int BNEXT = LAST + 1 > FM ? LAST + 1 : FM;          // where its first half is free
  // The fragments of b of a slice are in registers before half of its steps are done, those of a
  // only towards its end.  With SOON a barrier of its own after step BFREE gives b's stage up there,
  // so that two stages of b reach as far ahead as three of a.
  static constexpr bool SOON = NSA != NSB;
  static constexpr int BFREE = BSTEPS + 1;
  // Copies go out one a step, b's (SOON) two a step from step BFREE + 1 on, the others from step
  // LAST + 1 on into the next slice's first steps.
  static constexpr int TAIL = SOON ? CA : CA + CB;
  static constexpr int EARLY = AHEAD < TAIL ? AHEAD : TAIL;   // of them before the next slice begins
  // copies that may still be on their way when the next slice has to have landed: those that went out
  // after its own
  static constexpr int PENDING = !SOON ? (NSA - 2) * (CA + CB)
                                 : NSB < NSA ? (NSB - 1) * (CA + CB)
                                             : (NSA - 2) * CA + (NSA - 1) * CB;
  static_assert(WTM % 16 == 0 && WTN % 16 == 0 && FM % OUTF == 0, "whole fragments");
  static_assert((KA || BM % 64 == 0) && (KB || BN % 64 == 0), "whole panels");
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "whole copies");
  static_assert(NSA >= 2 && NSB >= 2 && PENDING + TAIL <= 63, "vmcnt range");
  static_assert(LDS <= 160 * 1024, "LDS");
  static_assert(STEPS % (AHEAD + 1) == 0, "a fragment's registers are known");
  static_assert(BNEXT + 2 <= STEPS, "b is read by then");
  static_assert(TAIL - EARLY <= (SOON ? BFREE : LAST) + 1, "every copy goes out within its slice");
  static_assert(!SOON || BFREE + (CB + 1) / 2 <= LAST, "every copy goes out within its slice");

  // Where a lane finds a wave's fragments of an operand in a stage.
  template <bool KC, int WT, int F>
  struct Where {
    static constexpr int NADDR = KC ? 2 : (F < 4 ? F : 4);
    uint32_t at[NADDR];
    __device__ __forceinline__ void init(uint32_t base, int w, int lane) {
      const int fr = lane & 15, fq = lane >> 4;
      if constexpr (KC) {
        #pragma unroll
        for (int t = 0; t < 2; ++t)
          at[t] = base + (w * WT + fr) * ROWB + (((2 * fq + t) ^ swz(fr)) << 4);
      } else {
        const int k = fq * 16 + (fr >> 2);
        const int f = ((k >> 1) & 1) | ((k >> 4) & 1) << 1;
        #pragma unroll
        for (int v = 0; v < NADDR; ++v) {
          const int c = w * WT / 16 + v;               // 16 columns of the operand
          const int pair = (c & 3) ^ f;
          at[v] = base + (c / 4) * 64 * ROWB + k * ROWB +
                  ((2 * pair + ((fr >> 1) & 1)) << 4) + (fr & 1) * 8;
        }
      }
    }
    __device__ __forceinline__ void step(uint32_t d) {
      #pragma unroll
      for (int v = 0; v < NADDR; ++v) at[v] += d;
    }
    __device__ __forceinline__ bf16x8 read(const char* lds, int i, int t) const {
      if constexpr (KC) {
        return *reinterpret_cast<const bf16x8*>(lds + at[t] + i * 16 * ROWB);
      } else {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        using Shared = __attribute__((address_space(3))) bf16x4;
        const char* p = lds + at[i % NADDR] + (i / 4) * 64 * ROWB + t * 8 * ROWB;
        const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((Shared*)p);
        const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((Shared*)(p + 4 * ROWB));
        return bf16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      }
    }
  };

  __device__ static __forceinline__ void run(const Args& g, const Tile& t, char* lds) {
    const int lane = threadIdx.x & (kWave - 1);
    const int all = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int kg = all / NW, wave = all % NW;                // group, and wave of the group
    const int wn = wave % WN, wm = wave / WN;
    const int K = g.K, KT = (K + kSlice - 1) / kSlice, steps = (KT + KG - 1) / KG;

    // ---- this wave's copies.  Offsets past a descriptor's end read as zeros: rows past the
    // operand's last, k past K (in the last slice, and in slices past it, which the ring and the
    // k-groups run into) ------------------------------------------------------------------------
    const i32x4 ra = buf_rsrc(g.a + (size_t)t.m0 * K, (uint32_t)t.rows * (uint32_t)K * 2);
    const i32x4 rb = buf_rsrc(g.b + (size_t)t.n0 * K, (uint32_t)t.cols * (uint32_t)K * 2);
    // the descriptor of 64 rows of k of an operand whose rows are k
    auto rows_of_k = [&](auto ends, const uint16_t* p, int ld, int64_t first, int kt) {
      constexpr bool ENDS = decltype(ends)::value;
      const int left = ENDS ? min(max(K - kt * kSlice, 0), kSlice) : kSlice;
      const uint32_t bytes = (uint32_t)max((int64_t)left * ld - first, (int64_t)0) * 2;
      return buf_rsrc(p + (size_t)(ENDS ? min(kt, KT) : kt) * kSlice * ld + first, bytes);
    };
    const int kc = ((lane & 7) ^ (lane >> 3)) * 8;           // k of the lane's chunk, even copies
    // where copy q of an operand's slice (8 of its rows, or 8 rows of k of a panel) lies
    auto offset = [&](auto contiguous, int q, int ld) {
      if constexpr (decltype(contiguous)::value)
        return (uint32_t)(q * 8 + (lane >> 3)) * (uint32_t)K * 2 +
               (uint32_t)(kc ^ ((q & 1) * 8)) * 2;
      const int k = (q & 7) * 8 + (lane >> 3);
      const int f = ((k >> 1) & 1) | ((k >> 4) & 1) << 1;
      return (uint32_t)k * (uint32_t)ld * 2 + (uint32_t)((q >> 3) * ROWB) +
             (uint32_t)(((lane & 7) ^ (2 * f)) << 4);
    };
    using ContA = std::bool_constant<KA>;
    using ContB = std::bool_constant<KB>;
    uint32_t va[CA], vb[CB];
    #pragma unroll
    for (int i = 0; i < CA; ++i) va[i] = offset(ContA{}, wave * CA + i, g.M);
    #pragma unroll
    for (int i = 0; i < CB; ++i) vb[i] = offset(ContB{}, wave * CB + i, g.N);
    const uint32_t lds_base = __builtin_amdgcn_readfirstlane(lds_u32(lds));
    // copy q (the wave's) of an operand's slice of `step` into its stage; `ends`: k may pass K in it
    auto copy = [&](auto ends, auto contiguous, i32x4 r, uint32_t v, int q, int step, uint32_t stage) {
      const int kt = step * KG + kg;
      constexpr bool C = decltype(contiguous)::value;
      if (decltype(ends)::value && C && (kc ^ ((q & 1) * 8)) >= K - kt * kSlice) v = kPastEnd;
      buf_dma16(r, v, C ? (uint32_t)kt * ROWB : 0u, lds_base + stage + (uint32_t)q * 1024);
    };
    auto copy_a = [&](auto ends, int buf, int step, int i) {
      i32x4 r = ra;
      if constexpr (!KA) r = rows_of_k(ends, g.a, g.M, t.m0, step * KG + kg);
      copy(ends, ContA{}, r, va[i], wave * CA + i, step, (uint32_t)((buf * KG + kg) * STAGE_A));
    };
    auto copy_b = [&](auto ends, int buf, int step, int i) {
      i32x4 r = rb;
      if constexpr (!KB) r = rows_of_k(ends, g.b, g.N, t.n0, step * KG + kg);
      copy(ends, ContB{}, r, vb[i], wave * CB + i, step,
           (uint32_t)(RING_B + (buf * KG + kg) * STAGE_B));
    };
    // copy i of the tail's: b's first, where they are in it
    auto copy_tail = [&](auto ends, int buf_a, int buf_b, int step_a, int step_b, int i) {
      if (i < 0 || i >= TAIL) return;
      if (SOON) copy_a(ends, buf_a, step_a, i);
      else if (i < CB) copy_b(ends, buf_b, step_b, i);
      else copy_a(ends, buf_a, step_a, i - CB);
    };

    Where<KA, WTM, FM> wa;
    Where<KB, WTN, FN> wb;
    wa.init(kg * STAGE_A, wm, lane);
    wb.init(RING_B + kg * STAGE_B, wn, lane);

    f32x4 acc[FM][FN];
    #pragma unroll
    for (int i = 0; i < FM; ++i)
      #pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // Software pipeline.  The barrier of a slice sits AHEAD steps before its end: every wave has read
    // all of the slice by then, so its stages are refilled, and the steps left cover the first reads
    // of the next slice.  Fragments of b are read half a slice ahead, a few a step.
    bf16x8 bf[2][FN], af[AHEAD + 1];
    auto read_b = [&](int h, int step, int steps_for_it) {
      const int per = (FN + steps_for_it - 1) / steps_for_it;
      #pragma unroll
      for (int j = 0; j < FN; ++j)
        if (j / per == step) bf[h][j] = wb.read(lds, j, h);
    };
    int ba = 0, bb = 0;           // the slice's stages
    auto after = [](int buf, int n) { return buf + 1 == n ? 0 : buf + 1; };
    auto slice = [&](auto ends, int step) {
      const int na = after(ba, NSA), nb = after(bb, NSB);
      const int pa = ba == 0 ? NSA - 1 : ba - 1, pb = bb == 0 ? NSB - 1 : bb - 1;
      #pragma unroll
      for (int u = 0; u < STEPS; ++u) {
        const int next = (u + AHEAD) % STEPS;
        af[next % (AHEAD + 1)] = wa.read(lds, next % FM, next / FM);
        if (u <= LAST) read_b(1, u, BSTEPS);
        if (u >= BNEXT) read_b(0, u - BNEXT, 2);       // the next slice's
        if (u <= LAST) copy_tail(ends, pa, pb, step - 1 + NSA, step - 1 + NSB, EARLY + u);
        else copy_tail(ends, ba, bb, step + NSA, step + NSB, u - LAST - 1);
        #pragma unroll
        for (int i = 0; i < CB; ++i)
          if (SOON && u > BFREE && i / 2 == u - BFREE - 1) copy_b(ends, bb, step + NSB, i);
        #pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[u % FM][j] = OpBf16::mma(bf[u / FM][j], af[u % (AHEAD + 1)], acc[u % FM][j]);
        if (SOON && u == BFREE) {
          __builtin_amdgcn_sched_barrier(0);           // the waits come after these products
          // b was read two steps before and earlier; since then only a, once a step
          asm volatile("s_waitcnt lgkmcnt(2)" ::: "memory");
          __builtin_amdgcn_s_barrier();
        }
        if (u == LAST) {
          __builtin_amdgcn_sched_barrier(0);
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          wait_vmcnt<PENDING>();                       // this wave's copies of the next slice
          __builtin_amdgcn_s_barrier();
          wa.step((uint32_t)((na - ba) * KG * STAGE_A));
          wb.step((uint32_t)((nb - bb) * KG * STAGE_B));
        }
        // the scheduler would move the reads down to their products
        __builtin_amdgcn_sched_barrier(0);
      }
      ba = na;
      bb = nb;
    };
    // what the slices before the first would have copied, in their order
    #pragma unroll
    for (int e = -(NSA > NSB ? NSA : NSB); e < 0; ++e) {
      const std::true_type ends{};
      if (SOON && e + NSB >= 0)
        #pragma unroll
        for (int i = 0; i < CB; ++i) copy_b(ends, e + NSB, e + NSB, i);
      if (e + NSA < 0) continue;
      #pragma unroll
      for (int i = 0; i < (e == -1 ? EARLY : TAIL); ++i)
        copy_tail(ends, e + NSA, e + NSB, e + NSA, e + NSB, i);
    }
    // slice 0 has to have landed
    wait_vmcnt<!SOON ? (NSA - 2) * TAIL + EARLY : 0>();
    __syncthreads();
    #pragma unroll
    for (int u = 0; u < AHEAD; ++u) af[u] = wa.read(lds, u % FM, u / FM);
    read_b(0, 0, 1);
    // steps that copy whole slices only, and those that come to the end of k
    const int whole = min(steps, max(K / kSlice / KG - std::max(NSA, NSB), 0));
    int step = 0;
    for (; step < whole; ++step) slice(std::false_type{}, step);
    for (; step < steps; ++step) slice(std::true_type{}, step);
    wait_vmcnt<0>();
    __syncthreads();
    finish_tile(g, t, lds, acc, kg, wave, lane);
  }

  // The same tile from rows of any alignment: a thread loads its chunks of 16 bytes into registers a step
  // before it stores them to one of two stages of LDS.  With loads of single values at the rows' ends,
  // which hold up every step of the last column of tiles, 2047^3 a b takes 96 us, so 50.  Loads two steps
  // ahead gain nothing (their registers cost a workgroup per unit or are spilled), nor do those of whole
  // words that any_stream_kernel makes (a b^T 57 us against 47).
  __device__ static __forceinline__ void run_any(const Args& g, const Tile& t, char* lds) {
    const int lane = threadIdx.x & (kWave - 1);
    const int all = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int kg = all / NW, wave = all % NW;
    const int wn = wave % WN, wm = wave / WN;
    const int K = g.K, steps = ((K + kSlice - 1) / kSlice + KG - 1) / KG;
    constexpr int PA = BM * 8 / (NW * kWave), PB = BN * 8 / (NW * kWave);    // a thread's chunks
    static_assert(BM * 8 % (NW * kWave) == 0 && BN * 8 % (NW * kWave) == 0, "whole chunks");
    const int me = wave * kWave + lane;
    // chunk q of an operand: its place in a stage
    auto place = [](bool contiguous, int q) {
      const int c = q & 7;
      if (contiguous) return (q >> 3) * ROWB + ((c ^ swz(q >> 3)) << 4);
      const int k = (q >> 3) & 63;
      const int f = ((k >> 1) & 1) | ((k >> 4) & 1) << 1;
      return (q >> 9) * 64 * ROWB + k * ROWB + ((c ^ (2 * f)) << 4);
    };
    // chunk q of the slice that begins at k0 of an operand of `rows` rows (columns, if k is not its
    // contiguous dimension), whose part in the tile begins at `first`
    auto load = [&](bool contiguous, const uint16_t* p, int64_t first, int64_t rows, int q, int k0) {
      Piece o;
      const int c = q & 7;
      int64_t at;
      int left;
      if (contiguous) {
        const int64_t r = first + (q >> 3);
        at = r * K + c * 8 + k0;
        left = r < rows ? K - k0 - c * 8 : 0;
      } else {
        const int k = (q >> 3) & 63;
        const int64_t n = first + (q >> 9) * 64 + c * 8;
        at = k * rows + n + k0 * rows;
        left = k0 + k < K ? (int)min(rows - n, (int64_t)8) : 0;
      }
      o.load(p, at, rows * K, left);
      return o;
    };
    Piece a[PA], b[PB];
    auto load_step = [&](int step) {
      const int k0 = min(step * KG + kg, 1 << 24) * kSlice;
      #pragma unroll
      for (int i = 0; i < PA; ++i) a[i] = load(KA, g.a, t.m0, g.M, i * NW * kWave + me, k0);
      #pragma unroll
      for (int i = 0; i < PB; ++i) b[i] = load(KB, g.b, t.n0, g.N, i * NW * kWave + me, k0);
    };
    constexpr int STAGE = STAGE_A + STAGE_B;
    auto store_step = [&](int buf) {
      char* st = lds + (buf * KG + kg) * STAGE;
      #pragma unroll
      for (int i = 0; i < PA; ++i)
        *reinterpret_cast<i32x4*>(st + place(KA, i * NW * kWave + me)) = a[i].get();
      #pragma unroll
      for (int i = 0; i < PB; ++i)
        *reinterpret_cast<i32x4*>(st + STAGE_A + place(KB, i * NW * kWave + me)) = b[i].get();
    };
    Where<KA, WTM, FM> wa;
    Where<KB, WTN, FN> wb;
    wa.init(kg * STAGE, wm, lane);
    wb.init(kg * STAGE + STAGE_A, wn, lane);
    f32x4 acc[FM][FN];
    #pragma unroll
    for (int i = 0; i < FM; ++i)
      #pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    load_step(0);
    store_step(0);
    load_step(1);
    __syncthreads();
    for (int step = 0; step < steps; ++step) {
      store_step((step + 1) & 1);                      // read last in the step before
      load_step(step + 2);
      #pragma unroll
      for (int h = 0; h < 2; ++h) {
        bf16x8 bf[FN];
        #pragma unroll
        for (int j = 0; j < FN; ++j) bf[j] = wb.read(lds, j, h);
        #pragma unroll
        for (int i = 0; i < FM; ++i) {
          const bf16x8 af = wa.read(lds, i, h);
          #pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = OpBf16::mma(bf[j], af, acc[i][j]);
        }
      }
      __syncthreads();
      const uint32_t d = (uint32_t)(step & 1 ? -KG * STAGE : KG * STAGE);
      wa.step(d);
      wb.step(d);
    }
    finish_tile(g, t, lds, acc, kg, wave, lane);
  }

  // The sums of the k-groups, the epilogue, and c.  The stages are done with.
  __device__ static __forceinline__ void finish_tile(const Args& g, const Tile& t, char* lds,
                                                     f32x4 (&acc)[FM][FN], int kg, int wave,
                                                     int lane) {
    const int wn = wave % WN, wm = wave / WN;
    if constexpr (KG > 1) {
      f32x4* sums = reinterpret_cast<f32x4*>(lds);
      auto at = [&](int g_, int i, int j) {
        return (((g_ - 1) * NW + wave) * FM * FN + i * FN + j) * kWave + lane;
      };
      if (kg > 0) {
        #pragma unroll
        for (int i = 0; i < FM; ++i)
          #pragma unroll
          for (int j = 0; j < FN; ++j) sums[at(kg, i, j)] = acc[i][j];
      }
      __syncthreads();
      if (kg > 0) return;
      #pragma unroll
      for (int g_ = 1; g_ < KG; ++g_)
        #pragma unroll
        for (int i = 0; i < FM; ++i)
          #pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] += sums[at(g_, i, j)];
    }

    // ---- c: lane holds row lane & 15 of a, columns (lane >> 4) * 4 + v.  Each wave turns its
    // fragments around in its part of LDS, OUTF of them at a time, in fp32, and finishes 8
    // neighbouring columns of a row a lane, or, where rows of c are no whole 16-byte blocks, one
    // column a lane -----------------------------------------------------------------------------
    const int fr = lane & 15, fq = lane >> 4;
    char* mine = lds + OUT_OFF + wave * OUTF * 16 * PITCH;
    const int m_w = wm * WTM, n_w = wn * WTN;
    #pragma unroll
    for (int i0 = 0; i0 < FM; i0 += OUTF) {
      #pragma unroll
      for (int i = 0; i < OUTF; ++i)
        #pragma unroll
        for (int j = 0; j < FN; ++j)
          *reinterpret_cast<f32x4*>(mine + (i * 16 + fr) * PITCH + (j * 16 + fq * 4) * 4) =
              acc[i0 + i][j];
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (g.N % 8 == 0) {
        constexpr int VPR = WTN / 8, RPP = VPR <= 4 ? 16 : 8;    // lanes of a row, rows a turn
        static_assert(VPR <= 8 && OUTF * 16 % RPP == 0, "whole turns");
        constexpr int TURNS = OUTF * 16 / RPP;
        const int c = lane % VPR * 8, n = n_w + c;
        const bool in_n = lane < RPP * VPR && n < t.cols;
        #pragma unroll 2
        for (int u = 0; u < TURNS; ++u) {
          const int r = u * RPP + lane / VPR, m = m_w + i0 * 16 + r;
          if (!in_n || m >= t.rows) continue;
          const int64_t at = (t.m0 + m) * (int64_t)g.N + t.n0 + n;
          Eight res{};
          if (g.residual) res = load8(g.residual, at, g.c_f32);
          const f32x4* z = reinterpret_cast<const f32x4*>(mine + r * PITCH + c * 4);
          finish8(g, z[0], z[1], at, t.n0 + n, res);
        }
      } else {
        constexpr int VPR = WTN, RPP = kWave / VPR;
        static_assert(VPR <= kWave, "a column a lane");
        #pragma unroll 2
        for (int u = 0; u < OUTF * 16 / RPP; ++u) {        // OUTF * 16 is a multiple of 4
          if (lane >= RPP * VPR) break;
          const int r = u * RPP + lane / VPR, m = m_w + i0 * 16 + r;
          const int c = lane % VPR, n = n_w + c;
          if (m >= t.rows || n >= t.cols) continue;
          const float z = *reinterpret_cast<const float*>(mine + r * PITCH + c * 4);
          finish<1>(g, &z, t.m0 + m, t.n0 + n, 1);
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  }
};

template <int BM, int BN, int WM, int WN, int KG, int NSA, int NSB, int WPS, bool KA, bool KB>
__global__ __launch_bounds__(WM * WN * KG * kWave, WPS) void tile_kernel(Args g) {
  using G = TileGemm<BM, BN, WM, WN, KG, NSA, NSB, KA, KB>;
  __shared__ __attribute__((aligned(1024))) char lds[G::LDS];
  const int mblk = (g.M + BM - 1) / BM, nblk = (g.N + BN - 1) / BN;
  const int logical = xcd_logical(blockIdx.x, mblk * nblk);
  if (logical < 0) return;
  G::run(g, tile_at<BM, BN>(g, logical), lds);
}

// Rows of any alignment and sizes past the other kernels' offsets.  Four waves a SIMD: two workgroups of
// 128x128 a unit (1500 x 6000 x 4095 a b^T 157 us, with one 170).
constexpr int64_t kAnyGrid = 1 << 21;    // workgroups of a launch; more tiles are run by striding

template <int BM, int BN, int WM, int WN, int KG, bool KA, bool KB>
__global__ __launch_bounds__(WM * WN * KG * kWave, 4) void any_kernel(Args g) {
  using G = TileGemm<BM, BN, WM, WN, KG, 2, 2, KA, KB>;
  __shared__ __attribute__((aligned(1024))) char lds[G::LDS];
  const int64_t nblk = ((int64_t)g.N + BN - 1) / BN;
  const int64_t tiles = ((int64_t)g.M + BM - 1) / BM * nblk;
  for (int64_t i = blockIdx.x; i < tiles; i += gridDim.x) {
    Tile t;
    t.m0 = i / nblk * BM;
    t.n0 = (int)(i % nblk * BN);
    t.rows = (int)min((int64_t)BM, (int64_t)g.M - t.m0);
    t.cols = min(BN, g.N - t.n0);
    __syncthreads();
    G::run_any(g, t, lds);
  }
}

// 256x256 tiles in rounds of one workgroup per compute unit, the first `whole` of them whole, the others
// as two halves (whole_tiles).
template <bool KA, bool KB>
__global__ __launch_bounds__(512, 2) void large_kernel(Args g, int whole, int whole_grid) {
  using G = TileGemm<256, 256, 2, 4, 1, 3, 2, KA, KB>;
  using H = TileGemm<128, 256, 2, 4, 1, 3, 3, KA, KB>;
  __shared__ __attribute__((aligned(1024))) char lds[G::LDS > H::LDS ? G::LDS : H::LDS];
  if ((int)blockIdx.x < whole_grid) {
    const int logical = xcd_logical(blockIdx.x, whole);
    if (logical >= 0) G::run(g, tile_at<256, 256>(g, logical), lds);
    return;
  }
  const int tiles = ((g.M + 255) / 256) * ((g.N + 255) / 256);
  const int h = xcd_logical((int)blockIdx.x - whole_grid, (tiles - whole) * 2);
  if (h < 0) return;
  Tile t = tile_at<256, 256>(g, whole + h / 2);
  t.m0 += (h & 1) * 128;
  t.rows = min(128, t.rows - (h & 1) * 128);
  if (t.rows > 0) H::run(g, t, lds);
}

// Few rows, a b^T: what counts is how fast the operands stream into the compute units that there are
// tiles for, 64 bytes a cycle each at most.  A workgroup takes 16 * FM rows of a and 16 * FN of b, and
// its NW waves every NW-th slice, each through a ring of its own in LDS, NS stages deep: whole lines
// of memory in every copy, and no barrier until the waves' sums are added, in the order of the waves.
template <int FM, int FN, int NW, int NS>
__global__ __launch_bounds__(NW * kWave) void stream_kernel(Args g) {
  constexpr int BM = 16 * FM, BN = 16 * FN;
  constexpr int CA = BM / 8, CB = BN / 8;              // 1 KB copies of a slice
  constexpr int STAGE = (CA + CB) * 1024;
  constexpr int RING = NW * NS * STAGE, SUMS = NW * FM * FN * kWave * 16;
  static_assert(RING <= 160 * 1024 && SUMS <= RING && (NS - 1) * (CA + CB) <= 63, "LDS, vmcnt");
  __shared__ __attribute__((aligned(1024))) char lds[RING];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int K = g.K, KT = (K + kSlice - 1) / kSlice;
  const int fr = lane & 15, fq = lane >> 4;
  const int nblk = (g.N + BN - 1) / BN;
  const int m0 = (int)blockIdx.x / nblk * BM, n0 = (int)blockIdx.x % nblk * BN;
  // rows and values of k past the operands' ends read as zeros
  const i32x4 ra = buf_rsrc(g.a + (size_t)m0 * K, (uint32_t)min(BM, g.M - m0) * (uint32_t)K * 2);
  const i32x4 rb = buf_rsrc(g.b + (size_t)n0 * K, (uint32_t)min(BN, g.N - n0) * (uint32_t)K * 2);
  const int kc = ((lane & 7) ^ (lane >> 3)) * 8;       // k of the lane's chunk, even copies
  uint32_t v[2];                                       // copies 2 i and 2 i + 1 of an operand
  #pragma unroll
  for (int o = 0; o < 2; ++o)
    v[o] = (uint32_t)(o * 8 + (lane >> 3)) * (uint32_t)K * 2 + (uint32_t)(kc ^ (o * 8)) * 2;
  const uint32_t mine = __builtin_amdgcn_readfirstlane(lds_u32(lds) + wave * NS * STAGE);
  auto copy = [&](int slot, int i) {                   // the wave's i-th slice
    const int kt = i * NW + wave, left = K - kt * kSlice;
    #pragma unroll
    for (int q = 0; q < CA + CB; ++q) {
      const bool is_a = q < CA;
      const int o = q & 1, row16 = (is_a ? q : q - CA) / 2;
      uint32_t at = v[o] + (uint32_t)row16 * 32u * (uint32_t)K;
      if ((kc ^ (o * 8)) >= left) at = kPastEnd;
      buf_dma16(is_a ? ra : rb, at, (uint32_t)kt * ROWB, mine + slot * STAGE + q * 1024);
    }
  };
  f32x4 acc[FM][FN] = {};
  const int slices = (KT + NW - 1) / NW;               // the same for every wave
  #pragma unroll
  for (int i = 0; i < NS - 1; ++i) copy(i, i);
  const char* stages = lds + wave * NS * STAGE;
  int slot = 0;
  for (int i = 0; i < slices; ++i) {
    // the slice before has been read: its stage takes the one NS - 1 further on
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    copy(slot == 0 ? NS - 1 : slot - 1, i + NS - 1);
    wait_vmcnt<(NS - 1) * (CA + CB)>();
    const char* st = stages + slot * STAGE;
    #pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int chunk = ((2 * fq + h) ^ swz(fr)) << 4;
      bf16x8 a[FM], b[FN];
      #pragma unroll
      for (int r = 0; r < FM; ++r)
        a[r] = *reinterpret_cast<const bf16x8*>(st + (r * 16 + fr) * ROWB + chunk);
      #pragma unroll
      for (int c = 0; c < FN; ++c)
        b[c] = *reinterpret_cast<const bf16x8*>(st + (BM + c * 16 + fr) * ROWB + chunk);
      #pragma unroll
      for (int r = 0; r < FM; ++r)
        #pragma unroll
        for (int c = 0; c < FN; ++c) acc[r][c] = OpBf16::mma(b[c], a[r], acc[r][c]);
    }
    slot = slot + 1 == NS ? 0 : slot + 1;
  }
  wait_vmcnt<0>();
  __syncthreads();
  f32x4* sums = reinterpret_cast<f32x4*>(lds);
  #pragma unroll
  for (int r = 0; r < FM; ++r)
    #pragma unroll
    for (int c = 0; c < FN; ++c) sums[(wave * FM * FN + r * FN + c) * kWave + lane] = acc[r][c];
  __syncthreads();
  for (int f = wave; f < FM * FN; f += NW) {
    f32x4 c = sums[f * kWave + lane];
    #pragma unroll
    for (int w = 1; w < NW; ++w) c += sums[(w * FM * FN + f) * kWave + lane];
    const int m = m0 + f / FN * 16 + fr, n = n0 + f % FN * 16 + fq * 4;
    const float z[4] = {c[0], c[1], c[2], c[3]};
    if (m < g.M && n < g.N) finish<4>(g, z, m, n, g.N - n);
  }
}

// The same few rows where they are no whole 16-byte blocks: every wave loads its fragments straight into
// registers, AT_ONCE slices at a time, in aligned words, one more where a row begins in the middle of
// one (loads of 16 bytes that begin there take several times as long: 64 x 255 x 7167 46 us, 20 so).
// Lanes of rows that a or b has not take its last row, whose products are not stored.  k past the last
// whole slice is one wave's.
template <int NW>
__global__ __launch_bounds__(NW * kWave) void any_stream_kernel(Args g) {
  constexpr int AT_ONCE = 4;
  __shared__ f32x4 sums[NW * kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int K = g.K, whole = K / kSlice;
  const int fr = lane & 15, fq = lane >> 4;
  const int nblk = (g.N + 15) / 16;
  const int m0 = (int)blockIdx.x / nblk * 16, n0 = (int)blockIdx.x % nblk * 16;
  const int64_t at_a = (int64_t)min(m0 + fr, g.M - 1) * K + fq * 16;
  const int64_t at_b = (int64_t)min(n0 + fr, g.N - 1) * K + fq * 16;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  // a row's 16 values of a whole slice; they begin in the middle of a word only where rows are of an odd
  // length, and then one more follows them
  struct Sixteen {
    i32x4 v[2];
    int more, odd;
    __device__ __forceinline__ void load(const uint16_t* p, int64_t at) {
      odd = (int)(at & 1);
      const int* w = (const int*)p + (at >> 1);
      __builtin_memcpy(v, w, 32);                      // of 4-byte alignment
      more = w[7 + odd];
    }
    __device__ __forceinline__ i32x4 get(int h) const {
      const int next = h == 0 ? v[1][0] : more;
      i32x4 o;
      #pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = __builtin_amdgcn_alignbit(i < 3 ? v[h][i + 1] : next, v[h][i], odd * 16);
      return o;
    }
  };
  auto mul = [&](const i32x4& a, const i32x4& b) {
    acc = OpBf16::mma(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), acc);
  };
  for (int kt = wave; kt < whole; kt += AT_ONCE * NW) {
    Sixteen a[AT_ONCE], b[AT_ONCE];
    #pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const int64_t k = (int64_t)min(kt + u * NW, whole - 1) * kSlice;
      a[u].load(g.a, at_a + k);
      b[u].load(g.b, at_b + k);
    }
    #pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      if (kt + u * NW >= whole) break;
      #pragma unroll
      for (int h = 0; h < 2; ++h) mul(a[u].get(h), b[u].get(h));
    }
  }
  if (K % kSlice != 0 && wave == whole % NW) {
    #pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = whole * kSlice + h * kChunk, left = K - k - fq * 16;
      Piece a, b;
      a.load(g.a, at_a + k, (int64_t)g.M * K, left);
      b.load(g.b, at_b + k, (int64_t)g.N * K, left);
      mul(a.get(), b.get());
    }
  }
  sums[wave * kWave + lane] = acc;
  __syncthreads();
  if (wave > 0) return;
  #pragma unroll
  for (int w = 1; w < NW; ++w) acc += sums[w * kWave + lane];
  const int m = m0 + fr, n = n0 + fq * 4;
  const float z[4] = {acc[0], acc[1], acc[2], acc[3]};
  if (m < g.M && n < g.N) finish<4>(g, z, m, n, g.N - n);
}

// The kernels of these tiles, as moe_gemm_bf16_choice.h knows them.
template <int BM, int BN, int THREADS>
constexpr bool listed() {
  for (const TileSize& d : kTileSize)
    if (d.bm == BM && d.bn == BN && d.threads == THREADS) return true;
  return false;
}

template <int FM, int FN, int NW, int NS>
hipError_t run_stream(const Args& a, hipStream_t s) {
  static_assert(listed<16 * FM, 16 * FN, NW * kWave>(), "the choice counts these tiles and threads");
  const int64_t tiles = (((int64_t)a.M + 16 * FM - 1) / (16 * FM)) *
                        (((int64_t)a.N + 16 * FN - 1) / (16 * FN));
  hipLaunchKernelGGL((stream_kernel<FM, FN, NW, NS>), dim3((unsigned)tiles), dim3(NW * kWave), 0, s,
                     a);
  return hipGetLastError();
}

template <bool KA, bool KB>
struct Run {
  template <int BM, int BN, int WM, int WN, int KG, int NSA, int NSB, int WPS>
  static hipError_t tile(const Args& a, hipStream_t s) {
    static_assert(listed<BM, BN, WM * WN * KG * kWave>(), "the choice counts these tiles and threads");
    const int64_t tiles = (((int64_t)a.M + BM - 1) / BM) * (((int64_t)a.N + BN - 1) / BN);
    hipLaunchKernelGGL((tile_kernel<BM, BN, WM, WN, KG, NSA, NSB, WPS, KA, KB>),
                       dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(WM * WN * KG * kWave), 0, s, a);
    return hipGetLastError();
  }
  template <int BM, int BN, int WM, int WN, int KG>
  static hipError_t any(const Args& a, hipStream_t s) {
    const int64_t tiles = (((int64_t)a.M + BM - 1) / BM) * (((int64_t)a.N + BN - 1) / BN);
    hipLaunchKernelGGL((any_kernel<BM, BN, WM, WN, KG, KA, KB>),
                       dim3((unsigned)std::min(tiles, kAnyGrid)), dim3(WM * WN * KG * kWave), 0, s,
                       a);
    return hipGetLastError();
  }
  static hipError_t large(const Args& a, int cus, hipStream_t s) {
    const int64_t tiles = tiles_of(kTile256x256, a.M, a.N), whole = whole_tiles(tiles, cus);
    const int64_t whole_grid = (whole + 7) / 8 * 8, halves = ((tiles - whole) * 2 + 7) / 8 * 8;
    hipLaunchKernelGGL((large_kernel<KA, KB>), dim3((unsigned)(whole_grid + halves)), dim3(512), 0,
                       s, a, (int)whole, (int)whole_grid);
    return hipGetLastError();
  }
  static hipError_t dense(const Args& a, int cus, hipStream_t s) {
    switch (choose(a.M, a.N, a.K, KA, KB, cus)) {
      case kAny64x64: return any<64, 64, 2, 2, 4>(a, s);
      case kAny128x128: return any<128, 128, 2, 4, 1>(a, s);
      case kAnyStream16x16:
        if constexpr (KA && KB) {
          static_assert(listed<16, 16, 16 * kWave>(), "the choice counts these tiles and threads");
          const int64_t tiles = tiles_of(kAnyStream16x16, a.M, a.N);
          hipLaunchKernelGGL(any_stream_kernel<16>, dim3((unsigned)tiles), dim3(16 * kWave), 0, s, a);
          return hipGetLastError();
        }
        break;
      case kStream16x16:
        if constexpr (KA && KB) return run_stream<1, 1, 8, 4>(a, s);
        break;
      case kStream16x32:
        if constexpr (KA && KB) return run_stream<1, 2, 8, 3>(a, s);
        break;
      case kTile32x64:
        if constexpr (KA) return tile<32, 64, 1, 4, 2, 4, 4, 2>(a, s);
        break;
      case kTile64x64: return tile<64, 64, 2, 2, 2, 3, 3, 2>(a, s);
      case kTile64x128: return tile<64, 128, 2, 4, 1, 3, 3, 2>(a, s);
      case kTile128x128: return tile<128, 128, 2, 4, 1, 3, 3, 2>(a, s);
      case kTile128x256: return tile<128, 256, 2, 4, 1, 3, 3, 2>(a, s);
      case kTile192x192: return tile<192, 192, 2, 4, 1, 3, 3, 2>(a, s);
      case kTile192x256: return tile<192, 256, 2, 4, 1, 4, 2, 2>(a, s);
      case kTile256x256: return large(a, cus, s);
      case kKernels: break;
    }
    return hipErrorInvalidValue;
  }
};

// ---------------------------------------------------------------------------------------------
// Gradient of the epilogue
// ---------------------------------------------------------------------------------------------
// Beyond 200 every slope is 0 or 1 in fp32, and its formula would multiply 0 by infinity.
__device__ __forceinline__ float slope(float z, int act) {
  if (z == z) z = fminf(fmaxf(z, -200.0f), 200.0f);
  if (act == MOE_ACT_SILU) {
    const float s = sigmoid_of(z);
    return s * (1.0f + z * (1.0f - s));
  }
  if (act == MOE_ACT_GELU) {            // cdf + z phi
    const float a = fabsf(z), below = bell(z) * __builtin_fmaf(a, -0.398942280f, tail_ratio(a));
    return z < 0.0f ? below : 1.0f - below;
  }
  if (act == MOE_ACT_GELU_TANH) {
    // with s = (1 + tanh u) / 2: s + z s (1 - s) 2 u'
    const float s = sigmoid_of(gelu_tanh_arg(z));
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

// HBM bounds it: 4096 x 14336, tanh form, with the bias 74 us, 4.8 TB/s (GELU 75 to 84).  A workgroup
// takes kActCols columns, 8 a lane, and every gridDim.y-th set of rows, one of its waves each, two sets at
// a time.  VEC: rows are whole 16-byte blocks and a lane's columns neighbours; elsewhere a lane has every
// 64th column.
constexpr int kActThreads = 256, kActWaves = kActThreads / kWave;

template <bool VEC>
__global__ __launch_bounds__(kActThreads) void act_bwd_kernel(ActArgs g) {
  static_assert(kActCols == 8 * kWave, "8 columns a lane");
  __shared__ float part[kActWaves][kActCols];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int c0 = blockIdx.x * kActCols;
  auto col = [&](int i) { return VEC ? lane * 8 + i : lane + i * kWave; };
  struct Eight {
    uint32_t w[4];
    __device__ __forceinline__ float get(int i) const {
      return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
  };
  auto load = [&](const uint16_t* p, int64_t m) {
    Eight e = {};
    if (m >= g.M) return e;
    p += m * g.N + c0;
    if constexpr (VEC) {
      if (c0 + lane * 8 >= g.N) return e;
      const i32x4 v = *(const i32x4*)(p + lane * 8);
      #pragma unroll
      for (int i = 0; i < 4; ++i) e.w[i] = (uint32_t)v[i];
    } else {
      #pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c0 + col(i) < g.N) e.w[i / 2] |= (uint32_t)p[col(i)] << (16 * (i & 1));
    }
    return e;
  };
  float sum[8] = {};
  const int64_t stride = (int64_t)gridDim.y * kActWaves;
  for (int64_t m0 = (int64_t)blockIdx.y * kActWaves + wave; m0 < g.M; m0 += 2 * stride) {
    Eight d[2], z[2];
    #pragma unroll
    for (int u = 0; u < 2; ++u) {
      d[u] = load(g.d_c, m0 + u * stride);
      if (g.act != MOE_ACT_NONE) z[u] = load(g.pre, m0 + u * stride);
    }
    #pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t m = m0 + u * stride;
      if (m >= g.M) break;
      float v[8];
      #pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = d[u].get(i);
        if (g.act != MOE_ACT_NONE) v[i] *= slope(z[u].get(i), g.act);
        sum[i] += v[i];
      }
      if (g.act == MOE_ACT_NONE) continue;
      uint16_t* to = g.d_z + m * g.N + c0;
      if constexpr (VEC) {
        if (c0 + lane * 8 < g.N) *(i32x4*)(to + lane * 8) = pack8(v);
      } else {
        #pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c0 + col(i) < g.N) to[col(i)] = (uint16_t)f32_to_bf16(v[i]);
      }
    }
  }
  if (!g.partials) return;
  #pragma unroll
  for (int i = 0; i < 8; ++i) part[wave][col(i)] = sum[i];
  __syncthreads();
  for (int c = threadIdx.x; c < kActCols; c += kActThreads) {
    if (c0 + c >= g.N) continue;
    float t = part[0][c];
    #pragma unroll
    for (int w = 1; w < kActWaves; ++w) t += part[w][c];
    g.partials[(int64_t)blockIdx.y * g.N + c0 + c] = t;
  }
}

}  // namespace gb

hipError_t launch_gemm_bf16(const GemmBf16& p, hipStream_t s) {
  gb::Args g{(const uint16_t*)p.a, (const uint16_t*)p.b, p.bias, p.residual, (uint16_t*)p.pre, p.c,
             p.M, p.N, p.K, p.act, p.c_f32};
  const int cus = std::max(device_cu_count(), 8);
  if (p.layout == MOE_NT) return gb::Run<true, true>::dense(g, cus, s);
  if (p.layout == MOE_NN) return gb::Run<true, false>::dense(g, cus, s);
  return gb::Run<false, false>::dense(g, cus, s);
}

hipError_t launch_act_bwd(int M, int N, int act, const void* d_c, const void* pre, void* d_z,
                          float* d_bias, float* partials, hipStream_t s) {
  gb::ActArgs g{(const uint16_t*)d_c, (const uint16_t*)pre, (uint16_t*)d_z,
                d_bias ? partials : nullptr, M, N, act};
  const int cus = std::max(device_cu_count(), 8);
  const int cols = (N + kActCols - 1) / kActCols;
  const int rows = act_partial_rows(M, N, cus);
  const dim3 grid((unsigned)cols, (unsigned)rows), block(gb::kActThreads);
  if (N % 8 == 0) hipLaunchKernelGGL(gb::act_bwd_kernel<true>, grid, block, 0, s, g);
  else hipLaunchKernelGGL(gb::act_bwd_kernel<false>, grid, block, 0, s, g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !d_bias) return e;
  return launch_sum_rows(rows, N, partials, d_bias, s);
}

}  // namespace moe

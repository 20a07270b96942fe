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
#include <algorithm>
#include <type_traits>

#include "moe_gemm_e4m3_choice.h"
#include "moe_internal.h"

namespace moe {

namespace q8 {

constexpr int ROWB = 128;      // bytes per row per k-slice: one scale group
constexpr int kGroupM = 8;     // m-blocks that sweep the n-blocks together

struct Args {
  const uint8_t* a;
  const float* sa;              // [M, K/128]
  const uint8_t* b;
  const float* sb;              // [ceil(N/128), K/128] or [N, K/128]
  void* c;
  const int32_t* sorted_slots;  // grouped: outputs of the alignment
  const int32_t* offsets;
  const int32_t* tiles;
  const int32_t* num_tiles;
  int tiles_max, n_slots;
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

// 64 lanes x 16 (4) bytes from the buffer at voff + soff straight to LDS at M0 (s_nop: lds_dma16).
__device__ __forceinline__ void buf_dma16(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               ::"v"(voff), "s"(rsrc), "s"(soff), "s"(lds) : "memory");
}
// The same for memory that is read once: it does not push others out of the caches.
__device__ __forceinline__ void buf_dma16_once(i32x4 rsrc, uint32_t voff, uint32_t soff,
                                               uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen nt lds"
               ::"v"(voff), "s"(rsrc), "s"(soff), "s"(lds) : "memory");
}
__device__ __forceinline__ void buf_dma4(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds"
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

// One tile of c: rows [row0, row0 + rows) x columns [n0, n0 + cols), b and sb those of the rows'
// expert.
struct Tile {
  const uint8_t* b;
  const float* sb;
  int64_t row0;
  int rows, n0, cols;
  int zero_rows;                // rows [rows, zero_rows) of c are written as zeros
};

// v_mfma_f32_16x16x128_f8f6f4 adds 8 products at a time after dropping what lies more than 13
// bits below the largest of them (measured; 1.4e-5 of the result, root mean square, on products
// of quantised normals), and the sums in fp32.  Far below the rounding of a bf16 result (1.7e-3),
// which therefore uses it.  An fp32 result converts the codes to bf16, exactly, and multiplies
// with v_mfma_f32_16x16x32_bf16 (9e-9), at half the matrix rate.
struct Bf16Codes {
  bf16x8 q[4];                  // a lane's 32 codes; any order of K that both operands share
};
__device__ __forceinline__ Bf16Codes to_bf16(const i32x8& f) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  Bf16Codes o;
  #pragma unroll
  for (int w = 0; w < 8; ++w) {
    const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[w], 1.0f, false);
    const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[w], 1.0f, true);
    o.q[w >> 1][(w & 1) * 4 + 0] = lo[0];
    o.q[w >> 1][(w & 1) * 4 + 1] = lo[1];
    o.q[w >> 1][(w & 1) * 4 + 2] = hi[0];
    o.q[w >> 1][(w & 1) * 4 + 3] = hi[1];
  }
  return o;
}

// Products of one group: scale operands of 0 select the instruction without the MX scales, which
// issues in fewer words (3-4% on power-limited large products).
__device__ __forceinline__ f32x4 mma_codes(const i32x8& b, const i32x8& a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0,
                                                          0, 0, 0);
}
__device__ __forceinline__ f32x4 mma_codes(const Bf16Codes& b, const Bf16Codes& a) {
  f32x4 c = {0.f, 0.f, 0.f, 0.f};
  #pragma unroll
  for (int q = 0; q < 4; ++q) c = OpBf16::mma(b.q[q], a.q[q], c);
  return c;
}

// BM x BN tile by WM x WN waves; 128-byte k-slices of both operands in a ring of NS LDS stages,
// copied by direct-to-LDS loads NS-1 steps ahead.  KG groups of WM x WN waves take every KG-th
// slice each, side by side, and their sums are added at the end in the order of the groups: a
// small tile's step costs the latency of its barrier and reads (0.25-0.35 us) whatever it
// multiplies, so KG slices a step run it nearly KG times as fast.
template <int BM, int BN, int WM, int WN, int KG, int NS, bool BROW, bool F32>
struct TileGemm {
  static constexpr int NW = WM * WN;                        // waves of one group
  static constexpr int WTM = BM / WM, WTN = BN / WN;        // a wave's rows of a and of b
  static constexpr int FM = WTM / 16, FN = WTN / 16;
  static constexpr int NQ_REAL = (BM + BN) * ROWB / 1024;   // 1 KB copies (8 rows) per slice
  static constexpr int NQ = (NQ_REAL + NW - 1) / NW * NW;   // padded to whole waves
  static constexpr int NQW = NQ / NW;
  static constexpr int SA = (BM + 63) / 64;                 // 64-row copies of a's scales ...
  static constexpr int SB = BROW ? (BN + 63) / 64 : 1;      // ... and of b's
  static constexpr int NSW = (SA + SB + NW - 1) / NW;       // scale copies per wave
  static constexpr int STAGE = NQ * 1024;                   // ring of NS stages of codes ...
  static constexpr int SSTAGE = NSW * NW * 256;             // ... and then one of scales
  static constexpr int SC_OFF = NS * KG * STAGE;
  static constexpr int OPS = NQW + NSW;
  static constexpr int RING = NS * KG * (STAGE + SSTAGE);
  static constexpr int SUMS = (KG - 1) * NW * FM * FN * kWave * 16;
  static constexpr int ES = F32 ? 4 : 2;                    // bytes per value of c
  static constexpr int PITCH = WTN * ES + 16;
  static constexpr int OUT_OFF = KG > 1 ? SUMS : 0;         // waves' parts of c on their way out
  static constexpr int OUT = OUT_OFF + NW * 16 * PITCH;
  static constexpr int LDS = RING > OUT ? RING : OUT;
  // A slice's copies go out in parts: PART of each wave (and the scales) right after the barrier
  // that frees the stage, PART more before each of the next slice's fragments.  All at once they
  // held up the waves' matrix instructions behind the load unit (16 cycles per copy, 72 copies
  // per 256x256 slice): 3270 -> 2680 cycles per slice of 2048 cycles of matrix work.
  static constexpr int PART = NS == 2 && FM >= 4 ? std::max(2, (NQW + FM - 1) / FM) : NQW;
  static_assert(BM % 8 == 0 && WTM % 16 == 0 && WTN % 16 == 0, "whole copies and MFMA tiles");
  static_assert(BROW || kGroup % WTN == 0, "one scale block per wave");
  static_assert(NS >= 2 && (NS - 1) * OPS <= 63, "vmcnt range");
  static_assert(LDS <= 160 * 1024, "LDS");
  static_assert((NQW + PART - 1) / PART <= FM, "every part goes out within its slice");

  // PARTIAL: tiles may hold few rows (a loop of its own for waves that have fragments without any)
  // ONCE: nothing else reads this tile's part of b
  // PAST: c is larger than the last-level cache
  template <bool PARTIAL, bool ONCE = false, bool PAST = false>
  __device__ static __forceinline__ void run(const Args& g, const Tile& t, char* lds) {
    const int lane = threadIdx.x & (kWave - 1);
    const int all = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int kg = all / NW, wave = all % NW;                // group, and wave of the group
    const int wn = wave % WN, wm = wave / WN;
    const int K = g.K, KT = K / ROWB, steps = (KT + KG - 1) / KG;

    // ---- this wave's copies: rows past the operand's end (an offset past the descriptor's) read
    // as zeros --------------------------------------------------------------------------------
    const i32x4 ra = buf_rsrc(g.a + (size_t)t.row0 * K, (uint32_t)t.rows * (uint32_t)K);
    const i32x4 rsa = buf_rsrc(g.sa + (size_t)t.row0 * KT, (uint32_t)t.rows * KT * 4);
    const i32x4 rb = buf_rsrc(t.b + (size_t)t.n0 * K, (uint32_t)t.cols * (uint32_t)K);
    const int sb0 = BROW ? t.n0 : t.n0 / kGroup;
    const int sbn = BROW ? t.cols : (t.n0 % kGroup + t.cols + kGroup - 1) / kGroup;
    const i32x4 rsb = buf_rsrc(t.sb + (size_t)sb0 * KT, (uint32_t)sbn * KT * 4);
    uint32_t voff[NQW];
    #pragma unroll
    for (int i = 0; i < NQW; ++i) {
      const int q = wave * NQW + i;
      int r = q * 8 + (lane >> 3);
      const int cc = (lane & 7) ^ swz(r);
      const bool is_a = q < BM / 8;
      if (!is_a) r -= BM;
      voff[i] = q < NQ_REAL ? (uint32_t)r * (uint32_t)K + cc * 16 : kPastEnd;
    }
    uint32_t soff[NSW];
    #pragma unroll
    for (int i = 0; i < NSW; ++i) {
      const int q = wave * NSW + i;
      const bool is_a = q < SA;
      const int r = (is_a ? q : q - SA) * 64 + lane;
      soff[i] = q < SA + SB ? (uint32_t)r * KT * 4 : kPastEnd;
    }
    const uint32_t lds_base = lds_u32(lds);
    // part p of the group's slice of `step` into stage buf; past the last slice that one is
    // repeated (not read, or added with a scale of 0), so that every step leaves the same number
    // of copies outstanding
    auto issue = [&](int buf, int step, int p) {
      const int kt = min(step * KG + kg, KT - 1);
      const uint32_t st = __builtin_amdgcn_readfirstlane(lds_base + (buf * KG + kg) * STAGE);
      #pragma unroll
      for (int i = 0; i < NQW; ++i) {
        if (i / PART != p) continue;
        const int q = wave * NQW + i;
        if constexpr (ONCE) {
          if (q < BM / 8) buf_dma16(ra, voff[i], (uint32_t)kt * ROWB, st + q * 1024);
          else buf_dma16_once(rb, voff[i], (uint32_t)kt * ROWB, st + q * 1024);
        } else {
          buf_dma16(q < BM / 8 ? ra : rb, voff[i], (uint32_t)kt * ROWB, st + q * 1024);
        }
      }
      if (p == 0) {
        #pragma unroll
        for (int i = 0; i < NSW; ++i) {
          const int q = wave * NSW + i;
          buf_dma4(q < SA ? rsa : rsb, soff[i], (uint32_t)kt * 4,
                   __builtin_amdgcn_readfirstlane(lds_base + SC_OFF + (buf * KG + kg) * SSTAGE) +
                       q * 256);
        }
      }
    };

    // ---- fragments (fragment i of wave row wm: rows [(i * WM + wm) * 16, +16), so that a tile
    // whose rows end early leaves every wave its share): lane holds row lane & 15, bytes
    // [(lane >> 4) * 32, +32) of the slice.  The lane's addresses (of the two 16-byte chunks and
    // of the scales) step from stage to stage in place; everything else about an address is an
    // immediate offset. -------------------------------------------------------------------------
    const int fr = lane & 15, fq = lane >> 4;
    const uint32_t o0 = fr * ROWB + (((2 * fq) ^ swz(fr)) << 4);
    const uint32_t o1 = fr * ROWB + (((2 * fq + 1) ^ swz(fr)) << 4);
    const uint32_t wa = wm * 16 * ROWB, wb = (BM + wn * WTN) * ROWB;
    const uint32_t gd = kg * STAGE, gs = SC_OFF + kg * SSTAGE;
    uint32_t a0 = gd + o0 + wa, a1 = gd + o1 + wa, b0 = gd + o0 + wb, b1 = gd + o1 + wb;
    uint32_t oa = gs + (wm * 16 + fr) * 4;
    uint32_t ob = gs + SA * 256 +
                  (BROW ? (wn * WTN + fq * 4) * 4 : (t.n0 % kGroup + wn * WTN) / kGroup * 4);
    auto frag = [&](uint32_t p0, uint32_t p1, int at) {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(lds + p0 + at);
      const i32x4 hi = *reinterpret_cast<const i32x4*>(lds + p1 + at);
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

    // Software pipeline over a's fragments: while the products of fragment i run, fragment i+1 is
    // read and the scaled sums of fragment i-1 are taken.  The barrier of a slice sits before its
    // last fragment's products: every wave has read all of the slice by then, so its stage is
    // refilled (slice kt + NS) and those products cover the first reads of slice kt+1.
    using BFrag = typename std::conditional<F32, Bf16Codes, i32x8>::type;
    BFrag bf[FN];
    i32x8 af[2];
    f32x4 part[2][FN];
    f32x4 s4[BROW ? FN : 1], s4p[BROW ? FN : 1];
    float s1 = 0.0f, sa_cur = 0.0f, sa_nxt = 0.0f, sp = 0.0f;
    #pragma unroll
    for (int j = 0; j < FN; ++j) part[1][j] = f32x4{0.f, 0.f, 0.f, 0.f};   // before fragment 0
    #pragma unroll
    for (int j = 0; j < (BROW ? FN : 1); ++j) s4p[j] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto read_a = [&](int i, i32x8& f, float& sc) {
      f = frag(a0, a1, i * WM * 16 * ROWB);
      sc = *reinterpret_cast<const float*>(lds + oa + i * WM * 64);
    };
    auto read_b = [&](int j) {
      const i32x8 f = frag(b0, b1, j * 16 * ROWB);
      if constexpr (F32) bf[j] = to_bf16(f);
      else bf[j] = f;
    };
    auto read_sb = [&]() {
      if constexpr (BROW) {
        #pragma unroll
        for (int j = 0; j < FN; ++j) s4[j] = *reinterpret_cast<const f32x4*>(lds + ob + j * 64);
      } else {
        s1 = *reinterpret_cast<const float*>(lds + ob);
      }
    };
    // acc[i][j] += the products in `p`, whose scales are sp (times s4p)
    auto add = [&](int i, int j, const f32x4& p) {
      #pragma unroll
      for (int v = 0; v < 4; ++v)
        acc[i][j][v] = __builtin_fmaf(p[v], BROW ? sp * s4p[BROW ? j : 0][v] : sp, acc[i][j][v]);
    };
    int buf = 0;
    auto slice = [&](auto par, int kt) {        // kt: the step
      constexpr int P = decltype(par)::value * FM;     // fragments of the slices before, mod 2
      const int nbuf = (buf + 1 == NS) ? 0 : buf + 1;
      const int pbuf = (buf == 0) ? NS - 1 : buf - 1;
      #pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int c = (P + i) & 1;                     // this fragment's set
        const int before = i == 0 ? FM - 1 : i - 1;    // the fragment before it
        if (i + 1 < FM) {
          read_a(i + 1, af[c ^ 1], sa_nxt);
          if ((i + 1) * PART < NQW) issue(pbuf, kt - 1 + NS, i + 1);
        } else {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          wait_vmcnt<(NS - 2) * OPS>();                // this wave's copies of slice kt+1
          __builtin_amdgcn_s_barrier();
          issue(buf, kt + NS, 0);
          const int d = (nbuf - buf) * KG * STAGE, ds = (nbuf - buf) * KG * SSTAGE;
          a0 += d; a1 += d; b0 += d; b1 += d; oa += ds; ob += ds;
          read_a(0, af[c ^ 1], sa_nxt);
        }
        if constexpr (F32) {
          const Bf16Codes a16 = to_bf16(af[c]);
          #pragma unroll
          for (int q = 0; q < 4; ++q)
            #pragma unroll
            for (int j = 0; j < FN; ++j)
              part[c][j] = OpBf16::mma(bf[j].q[q], a16.q[q],
                                       q ? part[c][j] : f32x4{0.f, 0.f, 0.f, 0.f});
          if (i + 1 == FM)
            #pragma unroll
            for (int j = 0; j < FN; ++j) read_b(j);
          #pragma unroll
          for (int j = 0; j < FN; ++j) add(before, j, part[c ^ 1][j]);
        } else {
          #pragma unroll
          for (int j = 0; j < FN; ++j) {
            part[c][j] = mma_codes(bf[j], af[c]);
            if (i + 1 == FM) read_b(j);
            add(before, j, part[c ^ 1][j]);
          }
        }
        sp = BROW ? sa_cur : sa_cur * s1;
        const bool repeated = KG > 1 && kt * KG + kg >= KT;   // adds 0, also under infinite scales
        if (repeated) sp = 0.0f;
        if constexpr (BROW) {
          if (i == 0)
            #pragma unroll
            for (int j = 0; j < FN; ++j) s4p[j] = repeated ? f32x4{0.f, 0.f, 0.f, 0.f} : s4[j];
        }
        sa_cur = sa_nxt;
        if (i + 1 == FM) read_sb();
      }
      buf = nbuf;
    };
    // fragments of this wave that hold rows; the others are neither read nor multiplied
    const int fmv = !PARTIAL ? FM : __builtin_amdgcn_readfirstlane(
        min(FM, max(0, (t.rows - wm * 16 + WM * 16 - 1) / (WM * 16))));
    // slices 0..NS-2 whole and the first part of slice NS-1; slice 0 has to have landed
    #pragma unroll
    for (int s = 0; s < NS - 1; ++s)
      #pragma unroll
      for (int p = 0; p * PART < NQW; ++p) issue(s, s, p);
    issue(NS - 1, NS - 1, 0);
    wait_vmcnt<(NS - 2) * OPS + (PART < NQW ? PART : NQW) + NSW>();
    __syncthreads();
    if (fmv == FM) {
      read_a(0, af[0], sa_cur);
      #pragma unroll
      for (int j = 0; j < FN; ++j) read_b(j);
      read_sb();
      using Even = std::integral_constant<int, 0>;
      using Odd = std::integral_constant<int, 1>;
      int kt = 0;
      for (; kt + 1 < steps; kt += 2) {
        slice(Even{}, kt);
        slice(Odd{}, kt + 1);
      }
      const bool odd = kt < steps;
      if (odd) slice(Even{}, kt);
      #pragma unroll
      for (int j = 0; j < FN; ++j)
        add(FM - 1, j, odd ? part[(FM - 1) & 1][j] : part[(2 * FM - 1) & 1][j]);
    } else {
      // a partly filled tile: the same steps and barriers, one fragment after the other
      for (int kt = 0; kt < steps; ++kt) {
        #pragma unroll
        for (int p = 1; p * PART < NQW; ++p) issue(buf == 0 ? NS - 1 : buf - 1, kt - 1 + NS, p);
        if (fmv > 0) {
          #pragma unroll
          for (int j = 0; j < FN; ++j) read_b(j);
          read_sb();
          const bool in = KG == 1 || kt * KG + kg < KT;
          #pragma unroll
          for (int j = 0; j < (BROW ? FN : 1); ++j) s4p[j] = s4[j];
          #pragma unroll
          for (int i = 0; i < FM; ++i) {
            if (i >= fmv) break;
            read_a(i, af[0], sa_cur);
            sp = !in ? 0.0f : BROW ? sa_cur : sa_cur * s1;
            BFrag a;
            if constexpr (F32) a = to_bf16(af[0]);
            else a = af[0];
            #pragma unroll
            for (int j = 0; j < FN; ++j) part[0][j] = mma_codes(bf[j], a);
            #pragma unroll
            for (int j = 0; j < FN; ++j) add(i, j, part[0][j]);
          }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wait_vmcnt<(NS - 2) * OPS>();
        __builtin_amdgcn_s_barrier();
        issue(buf, kt + NS, 0);
        const int nbuf = (buf + 1 == NS) ? 0 : buf + 1;
        const int d = (nbuf - buf) * KG * STAGE, ds = (nbuf - buf) * KG * SSTAGE;
        a0 += d; a1 += d; b0 += d; b1 += d; oa += ds; ob += ds;
        buf = nbuf;
      }
    }
    wait_vmcnt<0>();

    if constexpr (KG > 1) {
      // the ring is done with: every copy has landed, every wave has read its last slice
      f32x4* sums = reinterpret_cast<f32x4*>(lds);
      auto at = [&](int g_, int i, int j) {
        return (((g_ - 1) * NW + wave) * FM * FN + i * FN + j) * kWave + lane;
      };
      __syncthreads();
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

    // ---- c: lane holds row lane & 15 of a, b's rows (lane >> 4) * 4 + v.  Stored from there, a
    // row's line would be written in pieces of 32 bytes (bf16): each wave turns its fragments
    // around in LDS, 16 rows at a time, and stores WTN neighbouring values a row: 16 bytes a lane
    // where every row of c begins on such a bound (grouped 7168 x 2048 over 256 experts: 889 ->
    // 863 us), else 4 bytes, or the 2 of a bf16 value where N is odd (6418 x 666 x 896: to fp32
    // 35.3 -> 27.0 us, to bf16 22.6 -> 14.4; 346 x 8243 x 256: to bf16 12.3 -> 8.7). ------------
    auto value = [&](int i, int j) {
      return (i * WM + wm) * 16 + fr < t.rows ? acc[i][j] : f32x4{0.f, 0.f, 0.f, 0.f};
    };
    if (KG == 1) __syncthreads();                      // the ring is done with (KG > 1: above)
    char* mine = lds + OUT_OFF + wave * 16 * PITCH;
    auto store = [&](auto type) {
      using V = decltype(type);
      constexpr int VPR = WTN * ES / sizeof(V);        // stores per row
      constexpr int RPP = kWave / VPR < 16 ? kWave / VPR : 16;   // rows per instruction
      static_assert(VPR <= kWave, "a row per instruction");
      const int c = lane % VPR, n = wn * WTN + c * (int)sizeof(V) / ES;
      #pragma unroll
      for (int i = 0; i < FM; ++i) {
        #pragma unroll
        for (int j = 0; j < FN; ++j)
          store4<F32>(mine, (fr * PITCH + (j * 16 + fq * 4) * ES) / ES, value(i, j), 4, true);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        #pragma unroll
        for (int r0 = 0; r0 < 16; r0 += RPP) {
          const int r = r0 + lane / VPR, m = (i * WM + wm) * 16 + r;
          if (lane < RPP * VPR && m < t.zero_rows && n < t.cols) {
            const V v = *reinterpret_cast<const V*>(mine + r * PITCH + c * sizeof(V));
            V* to = reinterpret_cast<V*>((char*)g.c +
                                         ((t.row0 + m) * (int64_t)g.N + t.n0 + n) * ES);
            if constexpr (PAST && sizeof(V) == 16) __builtin_nontemporal_store(v, to);
            else *to = v;
          }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
    };
    if (g.N % (16 / ES) == 0) return store(i32x4{});
    if constexpr (!F32) {
      if (g.N & 1) return store(uint16_t{});
    }
    store(uint32_t{});
  }
};

// Few rows of a (up to 16 * FM): what counts is how fast b streams from HBM.  A workgroup takes
// 16 * FN rows of b and its NW waves take every NW-th k-slice, straight from memory into the
// matrix instructions' registers: no value of b is used twice, so LDS would only add a stop, and
// cutting K over the waves keeps the workgroups as many as N / (16 * FN) with the bytes in flight
// of NW waves each.  a's rows come from L2.  The waves' sums are added through LDS in the order of
// the waves.  One row, 4096 x 7168: 8.0 us (29 MB, 3.7 TB/s; 3 us of it are what any launch takes).
template <int FM, int FN, int NW, int U, bool BROW, bool F32>
struct StreamGemm {
  static constexpr int BM = 16 * FM, BN = 16 * FN;
  static constexpr int LDS = NW * FM * FN * kWave * 16;

  struct Slice {                 // one k-slice in registers
    i32x8 a[FM], b[FN];
    float sa[FM], sb[BROW ? 4 * FN : 1];
  };

  __device__ static __forceinline__ void run(const Args& g, const Tile& t, char* lds) {
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int K = g.K, KT = K / ROWB;
    const int fr = lane & 15, fq = lane >> 4;
    // rows past the operands' ends read the last row, their products are not stored
    const uint8_t *pa[FM], *pb[FN];
    const float *psa[FM], *psb[BROW ? 4 * FN : 1];
    #pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int64_t m = t.row0 + min(i * 16 + fr, t.rows - 1);
      pa[i] = g.a + (size_t)m * K + fq * 16;
      psa[i] = g.sa + (size_t)m * KT;
    }
    #pragma unroll
    for (int j = 0; j < FN; ++j)
      pb[j] = t.b + (size_t)(t.n0 + min(j * 16 + fr, t.cols - 1)) * K + fq * 16;
    #pragma unroll
    for (int j = 0; j < (BROW ? 4 * FN : 1); ++j)
      psb[j] = t.sb + (size_t)(BROW ? t.n0 + min((j / 4) * 16 + fq * 4 + j % 4, t.cols - 1)
                                    : t.n0 / kGroup) * KT;
    // any order of K that both operands share: lane takes chunks fq and fq + 4 of the slice, so
    // that one load instruction reads 64 contiguous bytes of each row
    auto load = [&](Slice& s, int kt) {
      const size_t at = (size_t)kt * ROWB;
      auto chunk = [&](const uint8_t* p) {
        const i32x4 lo = *reinterpret_cast<const i32x4*>(p + at);
        const i32x4 hi = *reinterpret_cast<const i32x4*>(p + at + 64);
        i32x8 f;
        f[0] = lo[0]; f[1] = lo[1]; f[2] = lo[2]; f[3] = lo[3];
        f[4] = hi[0]; f[5] = hi[1]; f[6] = hi[2]; f[7] = hi[3];
        return f;
      };
      #pragma unroll
      for (int j = 0; j < FN; ++j) s.b[j] = chunk(pb[j]);
      #pragma unroll
      for (int i = 0; i < FM; ++i) {
        s.a[i] = chunk(pa[i]);
        s.sa[i] = psa[i][kt];
      }
      #pragma unroll
      for (int j = 0; j < (BROW ? 4 * FN : 1); ++j) s.sb[j] = psb[j][kt];
    };
    f32x4 acc[FM][FN];
    #pragma unroll
    for (int i = 0; i < FM; ++i)
      #pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const Slice& s) {
      using Codes = typename std::conditional<F32, Bf16Codes, i32x8>::type;
      auto codes = [](const i32x8& f) -> Codes {
        if constexpr (F32) return to_bf16(f);
        else return f;
      };
      Codes b[FN];
      #pragma unroll
      for (int j = 0; j < FN; ++j) b[j] = codes(s.b[j]);
      #pragma unroll
      for (int i = 0; i < FM; ++i) {
        const Codes a = codes(s.a[i]);
        #pragma unroll
        for (int j = 0; j < FN; ++j) {
          const f32x4 p = mma_codes(b[j], a);
          #pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[i][j][v] = __builtin_fmaf(p[v], s.sa[i] * s.sb[BROW ? 4 * j + v : 0], acc[i][j][v]);
        }
      }
    };
    // U slices are in flight while the U before them are multiplied
    Slice cur[U], nxt[U];
    int kt = wave;
    #pragma unroll
    for (int u = 0; u < U; ++u)
      if (kt + u * NW < KT) load(cur[u], kt + u * NW);
    for (; kt < KT; kt += U * NW) {
      #pragma unroll
      for (int u = 0; u < U; ++u)
        if (kt + (U + u) * NW < KT) load(nxt[u], kt + (U + u) * NW);
      #pragma unroll
      for (int u = 0; u < U; ++u)
        if (kt + u * NW < KT) multiply(cur[u]);
      #pragma unroll
      for (int u = 0; u < U; ++u) cur[u] = nxt[u];
    }

    f32x4* sums = reinterpret_cast<f32x4*>(lds);
    #pragma unroll
    for (int i = 0; i < FM; ++i)
      #pragma unroll
      for (int j = 0; j < FN; ++j) sums[(wave * FM * FN + i * FN + j) * kWave + lane] = acc[i][j];
    __syncthreads();
    const bool vec = (g.N & 3) == 0;
    for (int f = wave; f < FM * FN; f += NW) {
      f32x4 c = sums[f * kWave + lane];
      #pragma unroll
      for (int w = 1; w < NW; ++w) c += sums[(w * FM * FN + f) * kWave + lane];
      const int m = (f / FN) * 16 + fr, n = (f % FN) * 16 + fq * 4;
      if (m < t.rows && n < t.cols)
        store4<F32>(g.c, (t.row0 + m) * (int64_t)g.N + t.n0 + n, c, t.cols - n, vec);
    }
  }
};

// Tile `logical` of the dense product: groups of kGroupM m-blocks sweep the n-blocks.
template <int BM, int BN>
__device__ __forceinline__ Tile dense_tile(const Args& g, int logical) {
  const int mblk = (g.M + BM - 1) / BM, nblk = (g.N + BN - 1) / BN;
  const int grp = logical / (kGroupM * nblk);
  const int gm = min(kGroupM, mblk - grp * kGroupM);
  const int w = logical - grp * kGroupM * nblk;
  Tile t;
  t.b = g.b;
  t.sb = g.sb;
  t.row0 = (int64_t)(grp * kGroupM + w % gm) * BM;
  t.rows = (int)min((int64_t)BM, (int64_t)g.M - t.row0);
  t.n0 = w / gm * BN;
  t.cols = min(BN, g.N - t.n0);
  t.zero_rows = t.rows;
  return t;
}

template <int BM, int BN, int WM, int WN, int KG, int NS, bool BROW, bool F32>
__global__ __launch_bounds__(WM * WN * KG * kWave) void tile_kernel(Args g) {
  using G = TileGemm<BM, BN, WM, WN, KG, NS, BROW, F32>;
  __shared__ __attribute__((aligned(1024))) char lds[G::LDS];
  const int mblk = (g.M + BM - 1) / BM, nblk = (g.N + BN - 1) / BN;
  const int logical = xcd_chunked<kChunk>(blockIdx.x, mblk * nblk);
  if (logical < 0) return;
  G::template run<false>(g, dense_tile<BM, BN>(g, logical), lds);
}

// Large products (4096 x 14336 x 4096 in 218-232 us, 2.2-2.07 PFLOP/s; the library's product with
// one scale per tensor takes 214): a tile of 32 slices takes 101500 cycles, 65% of them matrix work,
// and the clock is held at 1.8-1.9 GHz while it runs (all codes 0: the same cycles at 2.38 GHz, 177
// us).  5 of the 256 registers spill, 24 bytes a lane.  256x256 tiles in
// rounds of one workgroup per compute unit, `full` of them whole; where the last round would fill
// at most half of the units, its tiles run as two halves of 128 x 256 each, so that the round takes
// about half as long.  Every element's sum is the same either way.
__global__ __launch_bounds__(512) void large_kernel(Args g, int full, int full_grid) {
  using G = TileGemm<256, 256, 2, 4, 1, 2, false, false>;
  using H = TileGemm<128, 256, 2, 4, 1, 2, false, false>;
  __shared__ __attribute__((aligned(1024))) char lds[G::LDS];
  if ((int)blockIdx.x < full_grid) {
    const int logical = xcd_chunked<kChunk>(blockIdx.x, full);
    if (logical >= 0) G::template run<false>(g, dense_tile<256, 256>(g, logical), lds);
    return;
  }
  const int total = ((g.M + 255) / 256) * ((g.N + 255) / 256);
  const int h = xcd_logical((int)blockIdx.x - full_grid, (total - full) * 2);
  if (h < 0) return;
  Tile t = dense_tile<256, 256>(g, full + h / 2);
  t.row0 += (h & 1) * 128;
  t.rows = min(128, t.rows - (h & 1) * 128);
  t.zero_rows = t.rows;
  if (t.rows > 0) H::template run<false>(g, t, lds);
}

template <int FM, int FN, int NW, int U, bool BROW, bool F32>
__global__ __launch_bounds__(NW * kWave) void stream_kernel(Args g) {
  using G = StreamGemm<FM, FN, NW, U, BROW, F32>;
  __shared__ __attribute__((aligned(1024))) char lds[G::LDS];
  G::run(g, dense_tile<G::BM, G::BN>(g, blockIdx.x), lds);
}

// The alignment's tiles, expert by expert, m-blocks of one expert side by side (grouped_tile).
// WPS: waves per SIMD to fit in registers, so that workgroups overlap on a compute unit.
// Reading the weights bounds it at the sizes of experts: 64 tokens, top 2 of 8 experts, 4096 x
// 14336 71 us (6.6 TB/s); 2048 tokens, top 8 of 256, 7168 x 2048 750 us (3.8 GB of weights and 0.5 GB of
// output, half of it the zeros of padding rows: 5.6 TB/s).
template <int BM, int BN, int WM, int WN, int KG, int NS, int WPS, bool PAST, bool F32>
__global__ __launch_bounds__(WM * WN * KG * kWave, WPS) void grouped_kernel(Args g) {
  using G = TileGemm<BM, BN, WM, WN, KG, NS, false, F32>;
  __shared__ __attribute__((aligned(1024))) char lds[G::LDS];
  const int nblk = (g.N + BN - 1) / BN;
  const int nt = min(max(*g.num_tiles, 0), g.tiles_max);
  const int logical = xcd_chunked<kChunk>(blockIdx.x, nt * nblk);
  if (logical < 0) return;
  const TileRef r = grouped_tile<BM, kGroupM>(logical, nblk, g.tiles, g.offsets);
  // an m-block holds its expert's rows first and padding after
  const int lane = threadIdx.x & (kWave - 1);
  int rows = 0;
  #pragma unroll
  for (int i = 0; i < BM; i += kWave) {
    const int slot = g.sorted_slots[r.row0 + min(i + lane, BM - 1)];
    rows += __popcll(__ballot(i + lane < BM && (uint32_t)slot < (uint32_t)g.n_slots));
  }
  Tile t;
  t.b = g.b + (size_t)r.e * g.N * g.K;
  t.sb = g.sb + (size_t)r.e * ((g.N + kGroup - 1) / kGroup) * (g.K / ROWB);
  t.row0 = r.row0;
  t.rows = __builtin_amdgcn_readfirstlane(rows);
  t.n0 = r.nt * BN;
  t.cols = min(BN, g.N - t.n0);
  t.zero_rows = BM;
  // An expert with one m-block reads its weights once: past 64 rows a block the plain loads are
  // the faster ones all the same (128 x 256: 822 against 1772 us), up to 64 rows the others
  // (32 rows, 8 experts of 4096 x 14336: 75 against 85 us; 16 rows, 256 experts of 4096 x 7168:
  // 957 against 1059 us; equal at K = 2048).  With several m-blocks they would read the weights
  // from memory again for each.
  if constexpr (BM <= 64) {
    if (g.offsets[r.e + 1] - g.offsets[r.e] == BM)
      return G::template run<true, true, PAST>(g, t, lds);
  }
  G::template run<true, false, PAST>(g, t, lds);
}

// The dense kernels of these tiles, as moe_gemm_e4m3_choice.h knows them.
template <int BM, int BN, int THREADS>
constexpr bool listed() {
  for (const DenseSize& d : kDenseSize)
    if (d.bm == BM && d.bn == BN && d.threads == THREADS) return true;
  return false;
}

template <int BM, int BN, int WM, int WN, int KG, int NS, bool BROW, bool F32>
hipError_t run_tile(const Args& a, hipStream_t s) {
  static_assert(listed<BM, BN, WM * WN * KG * kWave>(), "the choice counts these tiles and threads");
  const int64_t tiles = (((int64_t)a.M + BM - 1) / BM) * (((int64_t)a.N + BN - 1) / BN);
  hipLaunchKernelGGL((tile_kernel<BM, BN, WM, WN, KG, NS, BROW, F32>),
                     dim3((unsigned)xcd_chunked_grid<kChunk>(tiles)), dim3(WM * WN * KG * kWave), 0,
                     s, a);
  return hipGetLastError();
}

template <int FM, int FN, int NW, int U, bool BROW, bool F32>
hipError_t run_stream(const Args& a, hipStream_t s) {
  static_assert(listed<16 * FM, 16 * FN, NW * kWave>(), "the choice counts these tiles and threads");
  const int64_t tiles = (((int64_t)a.M + 16 * FM - 1) / (16 * FM)) *
                        (((int64_t)a.N + 16 * FN - 1) / (16 * FN));
  hipLaunchKernelGGL((stream_kernel<FM, FN, NW, U, BROW, F32>), dim3((unsigned)tiles),
                     dim3(NW * kWave), 0, s, a);
  return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int KG, int NS, int WPS = 2, bool PAST = false>
hipError_t run_grouped(const Args& a, bool f32, hipStream_t s) {
  const int64_t tiles = (int64_t)a.tiles_max * ((a.N + BN - 1) / BN);
  const dim3 grid((unsigned)xcd_chunked_grid<kChunk>(tiles)), block(WM * WN * KG * kWave);
  if (f32)
    hipLaunchKernelGGL((grouped_kernel<BM, BN, WM, WN, KG, NS, WPS, PAST, true>), grid, block, 0, s,
                       a);
  else
    hipLaunchKernelGGL((grouped_kernel<BM, BN, WM, WN, KG, NS, WPS, PAST, false>), grid, block, 0,
                       s, a);
  return hipGetLastError();
}

hipError_t run_large(const Args& a, int cus, hipStream_t s) {
  const int total = (int)(((int64_t)a.M + 255) / 256 * (((int64_t)a.N + 255) / 256));
  const int rem = total % cus;
  const int full = total > cus && rem * 2 <= cus ? total - rem : total;
  const int full_grid = (int)xcd_chunked_grid<kChunk>(full);
  const int halves = ((total - full) * 2 + 7) / 8 * 8;
  hipLaunchKernelGGL(large_kernel, dim3((unsigned)(full_grid + halves)), dim3(512), 0, s, a,
                     full, full_grid);
  return hipGetLastError();
}

template <bool BROW, bool F32>
hipError_t run_dense(const Args& a, int cus, hipStream_t s) {
  switch (choose_dense(a.M, a.N, a.K, BROW, F32, cus)) {
    case kStream16x16: return run_stream<1, 1, 8, 2, BROW, F32>(a, s);
    case kStream16x32: return run_stream<1, 2, 8, 2, BROW, F32>(a, s);
    case kTile16x64: return run_tile<16, 64, 1, 2, 4, 3, BROW, F32>(a, s);
    case kTile32x64: return run_tile<32, 64, 1, 4, 2, 3, BROW, F32>(a, s);
    case kTile64x64: return run_tile<64, 64, 2, 2, 2, 3, BROW, F32>(a, s);
    case kTile64x128: return run_tile<64, 128, 2, 4, 1, 3, BROW, F32>(a, s);
    case kTile128x128: return run_tile<128, 128, 2, 4, 1, 2, BROW, F32>(a, s);
    case kTile128x256: return run_tile<128, 256, 2, 4, 1, BROW || F32 ? 2 : 3, BROW, F32>(a, s);
    case kTile128x128Ring3:
      if constexpr (!F32) return run_tile<128, 128, 2, 4, 1, 3, BROW, false>(a, s);
      break;
    case kTile192x256:
      if constexpr (!F32) return run_tile<192, 256, 2, 4, 1, 2, BROW, false>(a, s);
      break;
    case kLarge256x256:
      if constexpr (!F32 && !BROW) return run_large(a, cus, s);
      break;
    case kDenseKernels: break;
  }
  return hipErrorInvalidValue;
}

}  // namespace q8

hipError_t launch_gemm_e4m3(int M, int N, int K, const uint8_t* a, const float* sa,
                            const uint8_t* b, const float* sb, bool b_rows, void* c, bool c_f32,
                            hipStream_t s) {
  q8::Args g{};
  g.a = a; g.sa = sa; g.b = b; g.sb = sb; g.c = c;
  g.M = M; g.N = N; g.K = K;
  const int cus = std::max(device_cu_count(), 8);
  if (b_rows)
    return c_f32 ? q8::run_dense<true, true>(g, cus, s) : q8::run_dense<true, false>(g, cus, s);
  return c_f32 ? q8::run_dense<false, true>(g, cus, s) : q8::run_dense<false, false>(g, cus, s);
}

hipError_t launch_grouped_gemm_e4m3(const Resolved& r, int N, int K, const uint8_t* rows,
                                    const float* row_scales, const uint8_t* w,
                                    const float* w_scales, const int32_t* sorted_slots,
                                    const int32_t* offsets, const int32_t* tiles,
                                    const int32_t* num_tiles, void* out, bool out_f32,
                                    hipStream_t s) {
  q8::Args g{};
  g.a = rows; g.sa = row_scales; g.b = w; g.sb = w_scales; g.c = out;
  g.sorted_slots = sorted_slots; g.offsets = offsets; g.tiles = tiles; g.num_tiles = num_tiles;
  g.tiles_max = (int)r.tiles_max;
  g.n_slots = (int)r.N;
  g.M = (int)r.rows_max; g.N = N; g.K = K;
  const int cus = std::max(device_cu_count(), 8);
  switch (q8::choose_grouped(r.BM, r.rows_max, r.tiles_max, N, out_f32, cus)) {
    case q8::kGrouped16x64: return q8::run_grouped<16, 64, 1, 2, 4, 3>(g, out_f32, s);
    case q8::kGrouped16x128: return q8::run_grouped<16, 128, 1, 4, 1, 3>(g, out_f32, s);
    case q8::kGrouped32x64: return q8::run_grouped<32, 64, 1, 4, 2, 3>(g, out_f32, s);
    case q8::kGrouped32x128: return q8::run_grouped<32, 128, 1, 4, 1, 3>(g, out_f32, s);
    case q8::kGrouped64x64: return q8::run_grouped<64, 64, 2, 2, 2, 3>(g, out_f32, s);
    case q8::kGrouped64x128: return q8::run_grouped<64, 128, 2, 4, 1, 3>(g, out_f32, s);
    case q8::kGrouped64x256: return q8::run_grouped<64, 256, 2, 4, 1, 3>(g, out_f32, s);
    case q8::kGrouped64x256Past:
      return q8::run_grouped<64, 256, 2, 4, 1, 3, 2, true>(g, out_f32, s);
    case q8::kGrouped128x128: return q8::run_grouped<128, 128, 2, 4, 1, 2, 4>(g, out_f32, s);
    case q8::kGrouped128x256: return q8::run_grouped<128, 256, 2, 4, 1, 3>(g, out_f32, s);
    case q8::kGrouped128x256Past:
      return q8::run_grouped<128, 256, 2, 4, 1, 3, 2, true>(g, out_f32, s);
    case q8::kGroupedKernels: break;
  }
  return hipErrorInvalidValue;
}

}  // namespace moe

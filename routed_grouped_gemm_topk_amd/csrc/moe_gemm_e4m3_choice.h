// Which kernel a product of e4m3 codes runs on, from its sizes and the device's number of compute
// units alone.  Host code without HIP, so that it is compiled and tested by itself.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace moe {
namespace q8 {

enum DenseKernel {
  kStream16x16, kStream16x32, kTile16x64, kTile32x64, kTile64x64, kTile64x128, kTile128x128,
  kTile128x128Ring3, kTile128x256, kTile192x256, kLarge256x256, kDenseKernels
};

struct DenseSize {
  int bm, bn, threads;          // a tile's rows of a and of b, threads of its workgroup
};
constexpr DenseSize kDenseSize[kDenseKernels] = {
    {16, 16, 512},   {16, 32, 512},   {16, 64, 512},   {32, 64, 512},   {64, 64, 512},
    {64, 128, 512},  {128, 128, 512}, {128, 128, 512}, {128, 256, 512}, {192, 256, 512},
    {256, 256, 512}};

constexpr int kChunk = 32;      // logical tiles per chunk dealt to one XCD (xcd_chunked)
constexpr int kSlice = 128;     // values of k per slice

inline int64_t dense_tiles(DenseKernel kernel, int M, int N) {
  const DenseSize& s = kDenseSize[kernel];
  return ((int64_t)M + s.bm - 1) / s.bm * (((int64_t)N + s.bn - 1) / s.bn);
}

// A launch counts its threads in 32 bits; its workgroups are whole chunks for each of the 8 XCDs.
inline bool dense_launchable(DenseKernel kernel, int M, int N) {
  const int64_t groups = (dense_tiles(kernel, M, N) + 8 * kChunk - 1) / (8 * kChunk) * (8 * kChunk);
  return groups * kDenseSize[kernel].threads < (1LL << 32);
}

// For few tiles: the largest kernel whose tiles still are at most as many as the compute units,
// since a product that leaves units idle takes the time of one tile, and a small tile's time is
// that of its steps along K.  Measured with K of 512, 2048 and 7168, M and N from 1 to 7168
// (us, K = 2048; the tile chosen against the next larger and smaller ones):
//   M = 1,    N = 7168: 16-row stream 4.9-5.1, 16x64 5.7
//   M = 64,   N = 2048: 16x64 5.9,  32x64 6.5
//   M = 64,   N = 7168: 32x64 6.4,  16x64 8.3,  64x64 8.2
//   M = 128,  N = 7168: 64x64 8.1,  32x64 9.3,  64x128 10.9
//   M = 256,  N = 7168: 64x128 10.7, 64x64 14.4, 128x128 15.2
inline DenseKernel choose_dense(int M, int N, int K, bool brow, bool f32, int cus) {
  auto tiles = [&](DenseKernel kernel) { return dense_tiles(kernel, M, N); };
  if (M <= 16) {
    // two fragments of b per workgroup once that still fills the units (7168 x 7168: 11.1 against
    // 11.7; 4096 x 7168, which it does not fill: 10.3 against 7.4)
    return tiles(kStream16x32) * 8 >= cus * 7 ? kStream16x32 : kStream16x16;
  }
  if (tiles(kTile16x64) <= cus) return kTile16x64;
  if (tiles(kTile32x64) <= cus) return kTile32x64;
  if (tiles(kTile64x64) <= cus) return kTile64x64;
  // two to a unit, before larger ones that leave units idle (92 x 9544, K = 4096: to bf16 15.0
  // against 17.0 us with 64x128, to fp32 18.9 against 25.5)
  if (tiles(kTile32x64) <= 2 * cus) return kTile32x64;
  if (tiles(kTile64x128) <= cus) return kTile64x128;
  // More tiles than that: the size whose rounds over the units take least.  `whole` is the time of
  // a round per slice (1/100 us), `half` that of a last round which fills at most half of its
  // places (two per unit for 128x128 tiles; 256x256 tiles run as halves then), `ends` the slices
  // that a round's start and end are worth; all fitted to 80 shapes of 300 to 8192 rows (rms 4-7%).
  // On 42 shapes of the same range that they were not fitted to, the size chosen takes 1.1-2.2%
  // more than the best one of each shape, on average (at worst 15%: 1641 x 2650 x 1408 to bf16 18.3
  // against 15.9 us); the best single one, 128x128 (bf16) and 64x128 (fp32), 3-6%.  A size whose
  // launch would count past 32 bits has no price: tiles of 128x256 and more stay far below it.
  auto price = [&](DenseKernel kernel, int places, int whole, int half, int ends) {
    if (!dense_launchable(kernel, M, N)) return INT64_MAX;
    const int64_t n = tiles(kernel), per = (int64_t)cus * places, rem = n % per;
    return (n / per * whole + (rem == 0 ? 0 : rem * 2 <= per ? half : whole)) *
           (int64_t)(K / kSlice + ends);
  };
  if (f32) {
    // the bf16 multiplication does not fit larger tiles in registers
    const int64_t p64 = brow ? price(kTile64x128, 1, 73, 61, 2) : price(kTile64x128, 1, 62, 51, 3);
    const int64_t p128 =
        brow ? price(kTile128x128, 2, 258, 132, 3) : price(kTile128x128, 2, 230, 117, 3);
    const int64_t p256 =
        brow ? price(kTile128x256, 1, 201, 201, 3) : price(kTile128x256, 1, 185, 185, 3);
    if (p64 < std::min(p128, p256)) return kTile64x128;
    return p256 < p128 ? kTile128x256 : kTile128x128;
  }
  const int64_t p128 =
      brow ? price(kTile128x128, 2, 140, 86, 2) : price(kTile128x128, 2, 114, 72, 3);
  const int64_t p256 =
      brow ? price(kTile128x256, 1, 130, 130, 4) : price(kTile128x256, 1, 99, 99, 5);
  const int64_t p192 =
      brow ? price(kTile192x256, 1, 159, 159, 4) : price(kTile192x256, 1, 128, 128, 5);
  const int64_t least = std::min({p128, p256, p192});
  // scales per row of b do not fit 256x256 tiles in registers (2.8 us per slice)
  if (!brow && price(kLarge256x256, 1, 153, 99, 5) < least) return kLarge256x256;
  if (p128 > least) return p192 < p256 ? kTile192x256 : kTile128x256;
  // One tile on a unit has no other's work to wait behind: a third stage, once K is long enough for
  // its longer start (2048 x 2048, K = 4096: 30.5 -> 27.6 us; 1024 x 4096, K = 2048: 15.2 -> 17.0).
  return tiles(kTile128x128) <= cus && K >= 26 * kSlice ? kTile128x128Ring3 : kTile128x128;
}

enum GroupedKernel {            // rows of an m-block, columns of a tile
  kGrouped16x64, kGrouped16x128, kGrouped32x64, kGrouped32x128, kGrouped64x64, kGrouped64x128,
  kGrouped64x256, kGrouped64x256Past, kGrouped128x128, kGrouped128x256, kGrouped128x256Past,
  kGroupedKernels               // none: m-blocks of other sizes
};

inline GroupedKernel choose_grouped(int block_m, int64_t rows_max, int64_t tiles_max, int N,
                                    bool f32, int cus) {
  // Stores past the last-level cache (256 MB) for an output that does not fit it (slots of 256
  // experts to 7168 columns: 16384 in 128-row blocks 851 -> 814 us, 8192 in 64-row blocks 783 ->
  // 704 us); a smaller output stays in reach of whoever reads it next.
  const bool past = rows_max * N * (f32 ? 4 : 2) > (256LL << 20);
  // 256 columns a tile while its last n-block wastes little (N = 7168: 857 us against 882 with 128;
  // N = 2880, 7% past the end: 788 against 807; N = 1408, 9%: 152 against 128).
  const bool wide = ((int64_t)N + 255) / 256 * 256 * 100 <= (int64_t)N * 108;
  // Few tiles: the k-groups of the dense product.
  const bool few = tiles_max * ((N + 63) / 64) <= cus;
  switch (block_m) {
    case 16: return few ? kGrouped16x64 : kGrouped16x128;
    case 32: return few ? kGrouped32x64 : kGrouped32x128;
    case 64:
      if (few) return kGrouped64x64;
      return !wide ? kGrouped64x128 : past ? kGrouped64x256Past : kGrouped64x256;
    case 128: return !wide ? kGrouped128x128 : past ? kGrouped128x256Past : kGrouped128x256;
    default: return kGroupedKernels;
  }
}

}  // namespace q8
}  // namespace moe

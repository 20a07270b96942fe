// Which kernel a bf16 product runs on, from its sizes, its layout and the device's number of compute
// units alone.  Host code without HIP, so that it is compiled and tested by itself.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace moe {
namespace gb {

enum Kernel {
  kAny64x64, kAny128x128, kAnyStream16x16, kStream16x16, kStream16x32, kTile32x64, kTile64x64,
  kTile64x128, kTile128x128, kTile128x256, kTile192x192, kTile192x256, kTile256x256, kKernels
};

struct TileSize {
  int bm, bn, threads;          // a tile's rows and columns of c, threads of its workgroup
};
constexpr TileSize kTileSize[kKernels] = {
    {64, 64, 1024},  {128, 128, 512}, {16, 16, 1024},  {16, 16, 512},   {16, 32, 512},
    {32, 64, 512},   {64, 64, 512},   {64, 128, 512},  {128, 128, 512}, {128, 256, 512},
    {192, 192, 512}, {192, 256, 512}, {256, 256, 512}};

constexpr int kSlice = 64;      // values of k per slice
constexpr int kChunk = 8;       // values of a load, of rows of any alignment

inline int64_t tiles_of(Kernel kernel, int M, int N) {
  const TileSize& s = kTileSize[kernel];
  return ((int64_t)M + s.bm - 1) / s.bm * (((int64_t)N + s.bn - 1) / s.bn);
}

// A launch counts its threads in 32 bits; its workgroups are as many for each of the 8 XCDs.
inline bool launchable(Kernel kernel, int M, int N) {
  const int64_t groups = (tiles_of(kernel, M, N) + 7) / 8 * 8;
  return groups * kTileSize[kernel].threads < (1LL << 32);
}

// Of 256x256 tiles in rounds of one per unit, those that run whole: where a last round would fill at
// most half of the units, its tiles run as two halves of 128x256 each.
inline int64_t whole_tiles(int64_t tiles, int cus) {
  const int64_t rem = tiles % cus;
  return tiles > cus && rem * 2 <= cus ? tiles - rem : tiles;
}

// ka, kb: k is the contiguous dimension of a, of b.  The kernels of 16-byte loads need rows of whole
// 16-byte blocks; 256 rows of up to 2^21 values of k, and 64 rows of up to 2^23 values of m or n,
// stay within the 31-bit offsets of one buffer descriptor.
inline bool fits_blocks(int M, int N, int K, bool ka, bool kb) {
  constexpr int kMaxK = 1 << 21, kMaxLd = 1 << 23;
  const bool a = ka ? K % 8 == 0 && K <= kMaxK : M % 8 == 0 && M <= kMaxLd;
  const bool b = kb ? K % 8 == 0 && K <= kMaxK : N % 8 == 0 && N <= kMaxLd;
  return a && b;
}

// Time of a product in ns: `fixed`, and for every round of one workgroup per unit `round` and per
// slice of k `slice`.  Fitted to 1500 shapes of 1 to 9000 rows, 16 to 16000 columns and k of 128 to
// 9600 (rms 7-17%, the most where the launch is most of it).  On 700 shapes of the same range that
// they were not fitted to, the kernel chosen takes 0.7% more than the best of each on average, at
// most 4% in 19 of 20, at worst 42% (105 x 64 x 296: 7.5 against 5.3 us).  Without any one of the
// kernels that is 0.8% to 6.6%.
struct Price {
  int fixed, round, slice;      // round 0: the kernel does not take the layout
};
struct Prices {
  Price of[kKernels];
  Price last64x128;             // a last round of 64x128 tiles, two to a unit, with one each
  Price last256x256;            // a last round of 256x256 tiles as halves
};
constexpr Prices kPrices[3] = {
    // a b^T
    {{{0, 0, 0}, {0, 0, 0}, {0, 0, 0}, {2310, 2231, 42}, {1888, 2692, 61},
      {1701, 3000, 112}, {1155, 3556, 140},
      {2656, 2315, 790}, {-325, 5585, 429}, {-3099, 9981, 640}, {-3528, 11839, 680},
      {-5239, 14066, 878}, {-7190, 18056, 1047}},
     {0, 1802, 235}, {0, 7500, 1000}},
    // a b
    {{{0, 0, 0}, {0, 0, 0}, {0, 0, 0}, {0, 0, 0}, {0, 0, 0}, {1611, 3405, 128},
      {1466, 3583, 158}, {2106, 3511, 735},
      {132, 5949, 420}, {-1141, 9202, 616}, {-1777, 10684, 682}, {-2593, 12172, 833},
      {-6485, 17865, 1066}},
     {0, 2921, 255}, {0, 7500, 1000}},
    // a^T b
    {{{0, 0, 0}, {0, 0, 0}, {0, 0, 0}, {0, 0, 0}, {0, 0, 0}, {0, 0, 0},
      {1023, 4165, 180}, {3263, 3131, 748},
      {-213, 6474, 436}, {-2273, 10140, 658}, {-3576, 12594, 686}, {-4274, 13851, 888},
      {-6245, 17291, 1147}},
     {0, 1759, 292}, {0, 7500, 1000}}};

// Rows of any alignment, in us:
//   a b^T in up to two 16x16 tiles a unit, a stream, against 64x64: 3 x 5 x 14001 14.5 and 94, 33 x 501 x
//   1003 5.5 and 13.0, 16 x 8001 x 4097 (501 tiles) 23 and 32; beyond, 16 x 11001 x 4097 40 and 32,
//   500 x 1001 x 2001 37 and 20
//   128x128 from half a tile per unit on, against 64x64 with four groups of waves along k: 1400 x 1501 x
//   1001 25.7 and 40.1, 2047 x 2047 x 1001 27.9 and 54.1; below, 700 x 1001 x 1001 26.6 and 15.7, 300
//   x 3001 x 2001 44.9 and 23.4 (a b^T; the other layouts are within 10% of that)
inline Kernel choose(int M, int N, int K, bool ka, bool kb, int cus) {
  if (!fits_blocks(M, N, K, ka, kb)) {
    if (ka && kb && tiles_of(kAnyStream16x16, M, N) <= 2LL * cus) return kAnyStream16x16;
    return tiles_of(kAny128x128, M, N) * 2 >= cus ? kAny128x128 : kAny64x64;
  }
  const Prices& prices = kPrices[ka ? kb ? 0 : 1 : 2];
  const int64_t slices = ((int64_t)K + kSlice - 1) / kSlice;
  Kernel best = kAny128x128;
  int64_t least = INT64_MAX;
  for (int i = kStream16x16; i < kKernels; ++i) {
    const Kernel kernel = (Kernel)i;
    const Price& p = prices.of[i];
    if (!p.round || !launchable(kernel, M, N)) continue;
    const int64_t tiles = tiles_of(kernel, M, N);
    const int64_t places = (int64_t)cus * (kernel == kTile64x128 ? 2 : 1), rem = tiles % places;
    int64_t price = p.fixed + tiles / places * (p.round + p.slice * slices);
    const Price& last = kernel == kTile64x128 && rem <= cus ? prices.last64x128
                        : kernel == kTile256x256 && whole_tiles(tiles, cus) < tiles
                            ? prices.last256x256 : p;
    if (rem) price += last.round + last.slice * slices;
    if (price < least) {
      least = price;
      best = kernel;
    }
  }
  return best;
}

}  // namespace gb
}  // namespace moe

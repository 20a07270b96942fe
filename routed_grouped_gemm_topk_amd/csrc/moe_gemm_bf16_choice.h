// Which kernel a bf16 product runs on, from its sizes, its layout and the device's number of compute
// units alone.  Host code without HIP, so that it is compiled and tested by itself.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace moe {
namespace gb {

enum Kernel {
  kAny, kStream16x16, kStream16x32, kTile32x64, kTile64x64, kTile64x128, kTile128x128,
  kTile128x256, kTile256x256, kKernels
};

struct TileSize {
  int bm, bn, threads;          // a tile's rows and columns of c, threads of its workgroup
};
constexpr TileSize kTileSize[kKernels] = {{64, 64, 256},   {16, 16, 512},   {16, 32, 512},
                                          {32, 64, 512},   {64, 64, 512},   {64, 128, 512},
                                          {128, 128, 512}, {128, 256, 512}, {256, 256, 512}};

constexpr int kChunk = 32;      // logical tiles per chunk dealt to one XCD (xcd_chunked)
constexpr int kSlice = 64;      // values of k per slice

inline int64_t tiles_of(Kernel kernel, int M, int N) {
  const TileSize& s = kTileSize[kernel];
  return ((int64_t)M + s.bm - 1) / s.bm * (((int64_t)N + s.bn - 1) / s.bn);
}

// A launch counts its threads in 32 bits; its workgroups are whole chunks for each of the 8 XCDs.
inline bool launchable(Kernel kernel, int M, int N) {
  const int64_t groups = (tiles_of(kernel, M, N) + 8 * kChunk - 1) / (8 * kChunk) * (8 * kChunk);
  return groups * kTileSize[kernel].threads < (1LL << 32);
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

inline Kernel choose(int M, int N, int K, bool ka, bool kb, int cus) {
  if (!fits_blocks(M, N, K, ka, kb)) return kAny;
  auto tiles = [&](Kernel kernel) { return tiles_of(kernel, M, N); };
  if (M <= 16 && ka && kb && launchable(kStream16x32, M, N))
    return tiles(kStream16x32) * 8 >= cus * 7 ? kStream16x32 : kStream16x16;
  if (ka && tiles(kTile32x64) <= cus) return kTile32x64;
  if (tiles(kTile64x64) <= cus) return kTile64x64;
  if (tiles(kTile64x128) <= cus) return kTile64x128;
  if (tiles(kTile128x128) <= 2 * cus) return kTile128x128;
  if (tiles(kTile128x256) <= cus) return kTile128x256;
  return kTile256x256;
}

}  // namespace gb
}  // namespace moe

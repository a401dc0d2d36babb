// row_tiles.h -- how the 4-bit product (mxfp4.cu) cuts an expert's rows into tiles.
// Host and device arithmetic without CUDA types, so that any compiler can check it.
#pragma once

#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

constexpr int kMaxTok = 192;  // rows of a tile at most: three blocks of 64

// Tiles of an expert's c rows: as few as kMaxTok allows, starting on multiples of
// 64 (so a tile's scales lie in at most two 128-row tiles, from column 0 or 2 of
// the first).
MOE_HD int tok_tiles(int c) { return (c + kMaxTok - 1) / kMaxTok; }
// First row of tile t of `tiles` = tok_tiles(c).  The blocks of 64 rows are at most two
// short of three a tile: so many tiles at the front have two, all others three.
// (t * blocks / tiles would be as even, but passes 32 bits from 5.1 million rows of
// one expert on.)
MOE_HD int tok_start(int c, int tiles, int t) {
  const int two = 3 * tiles - (c + 63) / 64;
  return (3 * t - (t < two ? t : two)) * 64;
}
// Rows of the largest tile (kMaxTok where there are many).
MOE_HD int tok_most(int c) {
  const int tt = tok_tiles(c);
  if (tt > 4) return kMaxTok;
  int most = 0;
  for (int t = 0; t < tt; ++t) {
    const int n = (t + 1 < tt ? tok_start(c, tt, t + 1) : c) - tok_start(c, tt, t);
    most = most > n ? most : n;
  }
  return most;
}

}  // namespace moe

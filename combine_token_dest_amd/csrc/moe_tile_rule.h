// Which tiles a dense product is made of, and in how many parts of k: host
// code without a device or HIP (tests go through it).
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>

namespace moe_ep_detail {

constexpr int tiles(int64_t rows, int tile) { return (int)((rows + tile - 1) / tile); }

// The tiles for P x Q results of k products.  Larger ones move less for each
// product, but the card's 256 CUs, one tile each at a time, go through them in
// rounds.  A round takes, for 64 k: 1.6 us with tiles of 256 x 256, 1.0 of
// 256 x 128 (1.15 where several rounds crowd the caches), 0.57 of 128 x 128,
// 0.28 of 64 x 64, 0.15 of 32 x 32; and some us to begin and to store.  A last
// round that is not full leaves power to those of the largest tiles that work.
// Measured, gated products of rows x 4096 (k 7168), us with each:
//   rows        128   256   512  1024  2048  4096  8192
//   256 x 256   149   154   153   153   154   189   385
//   256 x 128    99    99    98    98   113   276   518
//   128 x 128    58    58    58    64   127   309   576
//    64 x 64     30    31    61   121   240   515  1056
//    32 x 32    22.8    44    85   168   332   690
// All times are of that product, whose operands have k side by side; those with
// rows side by side take 12 to 14% more (8192 x 4096 x 7168), and parts of k
// (product_parts) are not weighed against larger tiles.
// k32x32 is only there for two operands with k side by side (`narrow`).
enum TileSize { k256x256, k256x128, k128x128, k64x64, k32x32 };
inline TileSize tile_size(int64_t P, int64_t Q, int64_t k, bool direct, bool narrow) {
  constexpr struct {
    TileSize size;
    int p, q;
    double one, more;         // us of a round for 64 k: the only one, or one of several
    double ends;              // us of a round beside
  } kinds[] = {{k256x256, 256, 256, 1.6, 1.6, 8},
               {k256x128, 256, 128, 1.0, 1.15, 6},
               {k128x128, 128, 128, 0.57, 0.57, 4},
               {k64x64, 64, 64, 0.28, 0.28, 3},
               {k32x32, 32, 32, 0.15, 0.12, 3}};
  TileSize best = k64x64;
  double least = 1e300;
  for (const auto& t : kinds) {
    if (t.p == 256 && !direct) continue;                  // through registers there are only smaller ones
    if (t.p == 32 && !narrow) continue;
    const double r = (double)((P + t.p - 1) / t.p) * (double)((Q + t.q - 1) / t.q) / 256;
    const double rounds = t.size == k256x256 ? (r + std::ceil(r)) / 2 : std::ceil(r);
    const double time = r <= 1 ? t.one * k / 64 + t.ends : (t.more * k / 64 + t.ends) * rounds;
    if (time < least) {
      least = time;
      best = t.size;
    }
  }
  return best;
}

// Floats of the sums over parts of k.
constexpr int64_t kPartialFloats = 512 * 64 * 64;

// A few results of many k (weights' gradients of small layers, a few rows'
// gradients), which are tiles of 64 x 64: parts of k, two tiles of 256 k at
// least, for all CUs.  (1: no parts.)
inline int product_parts(int64_t P, int64_t Q, int64_t k) {
  const int64_t count = (int64_t)tiles(P, 64) * tiles(Q, 64);
  return (int)std::max<int64_t>(1, std::min<int64_t>({8, 256 / count, k / 512, kPartialFloats / (P * Q)}));
}

// Up to how many rows a gated product with `inter` results a row takes the kernel
// that streams the weights: up to 64 that still wins, while its workgroups,
// each reading all of x, go through the card twice at most (48 rows, us, this
// and tiles: 7168 x 2048 14.6 and 21.6, 4096 x 1024 8.9 and 12.4, 2048 x 5632
// 17.2 and 12.7).
inline int gated_few_rows(int64_t inter) { return tiles(inter, 8) <= 512 ? 64 : 32; }

}  // namespace moe_ep_detail

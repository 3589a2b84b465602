// nm_tiles.h -- which kernel a 4-bit product takes, which tile a dense product of the cross entropy or
// of the orthogonalised update takes, and how the cross entropy's gradient is cut.  Plain C++ with no
// HIP types, so that a host-only test can compile it and say which kernels a size runs.
#ifndef NM_TILES_H
#define NM_TILES_H

#include <algorithm>
#include <cstdint>

namespace nm {

inline int64_t pad64(int64_t n) { return (n + 63) / 64 * 64; }

// ---- 4-bit products ------------------------------------------------------------------------------

// Bytes of LDS that X's columns take in matvec_kernel, 0 where slices of them are better.  Every
// workgroup lays out all of X, at a cost of K T for each that a unit gets (two at a time where they
// fit), so rows and columns are bounded together; eight columns, of which the slices lay out whole
// 16-byte pieces, at less.  Measured with weights out of cache, us, whole / slices: 4096 x 4096, 2
// columns 5.4 / 11.2, 5 6.2 / 10.8; 2:4 4096 x 11008, 5 columns 11.2 / 14.6; 2:4 11008 x 4096, 7 columns
// 14.4 / 16.2; 16384 x 8192, 2 columns 22.8 / 29.6, 3 24.3 / 25.9, 5 40.5 / 26.1; 5003 x 11007, 2
// columns 16.7 / 18.4, 3 17.6 / 16.2, 4 24.4 / 17.9.  Eight columns, one round: 4096 x 4096 7.1 / 8.8,
// 4096 x 6144 9.3 / 12.0, 64 x 6144 7.8 / 7.1, 1024 x 7168 9.5 / 7.6, 4096 x 7168 10.4 / 11.5; more: 2:4
// 8192 x 2048 7.0 / 7.8, 12288 x 2048 9.4 / 9.2, 2:4 4608 x 4096 10.8 / 9.4, 2:4 8192 x 4096 11.1 / 9.6,
// 2:4 11008 x 4096 15.2 / 12.8, 24576 x 1024 9.4 / 8.0.
constexpr int kColumnPad = 64;  // bytes: four columns of X apart are on all banks of LDS
constexpr int kFewColumns = 8;
constexpr int64_t kFewLds = 128 << 10;
inline int64_t column_lds(int64_t R, int64_t K, int64_t T) {
  const int64_t column = std::max<int64_t>(1, (K + 255) / 256) * 512;
  if (T == 1) return column <= 64 << 10 ? column : 0;
  const int64_t groups = (R + 15) / 16, all = T * (column + kColumnPad);
  if (T > kFewColumns || all > kFewLds) return 0;
  const double rounds = all <= 80 << 10 ? std::max(1.0, groups / 256.0) : (double)((groups + 255) / 256);
  const int most = T % 8 != 0 ? 80 << 10 : rounds > 1 ? 32 << 10 : 48 << 10;
  return rounds * (double)(K * T) <= most ? all : 0;
}

// ---- cross entropy ---------------------------------------------------------------------------

constexpr int64_t kPieceBytes = 64 << 20;  // of P
constexpr int kMaxSplit = 32;

// The products' tiles.  256 x 256 is the fastest on many large tiles; of 128 x 128 two fit a unit,
// so that one's epilogue runs under the other's steps, and short or few sums are faster in them;
// 128 x 64 suits few tokens.
enum XentTile { kTile256, kTile128, kTileNarrow, kXentTiles };
constexpr int kTileM[kXentTiles] = {256, 128, 128}, kTileN[kXentTiles] = {256, 128, 64};

inline int64_t tiles_of(int tile, int64_t m, int64_t n) {
  return ((m + kTileM[tile] - 1) / kTileM[tile]) * ((n + kTileN[tile] - 1) / kTileN[tile]);
}

// Estimated time (us) of `count` tiles of `steps` steps: whole rounds of 256 for the large tile,
// and 512 at a time in a steady flow for the small ones, but never less than one tile alone.
// Measured, 256 / 128 / narrow: loss 32768 x 4096, 2048 tokens 522 / 611 / 731 us; 20000 x 1024,
// 1000 tokens 74 / 58 / 71; 12000 x 2048, 128 tokens 54 / 25 / 17; 30000 x 4096, 32 tokens
// 99 / 62 / 41; dW of 12000 x 2048, 128 tokens 21 / 17 / 23.
inline double tile_us(int tile, int64_t count, int64_t steps) {
  if (tile == kTile256) return (double)((count + 255) / 256) * (2.0 * steps + 8.0);
  const bool mid = tile == kTile128;
  const double alone = mid ? 0.65 * steps + 4.0 : 0.45 * steps + 3.0;
  const double flow = (double)count / 512 * (mid ? 1.19 * steps + 4.6 : 0.71 * steps + 3.5);
  return alone > flow ? alone : flow;
}

inline int pick_tile(int64_t m, int64_t n, int64_t steps) {
  int best = 0;
  for (int t = 1; t < kXentTiles; ++t)
    if (tile_us(t, tiles_of(t, m, n), steps) < tile_us(best, tiles_of(best, m, n), steps)) best = t;
  return best;
}

// How the gradient is cut: the vocabulary into pieces whose P fits a bounded workspace, and dX's sums
// over a piece into splits.
struct XentGradCut {
  int64_t piece;  // rows of W at a time
  int tile_x = kTile256, splits = 1;
  XentGradCut(int64_t V, int64_t K, int64_t T) {
    const int64_t Tp = pad64(T);
    piece = kPieceBytes / (2 * Tp) / 256 * 256;
    if (piece < 256) piece = 256;
    if (piece > V) piece = V;
    // dX's sums over the piece are split where its tiles are too few; each split costs a write
    // and a read of its sums (5 GB a ms)
    const int64_t steps = (piece + 63) / 64;
    double least = 1e30;
    for (int t = 0; t < kXentTiles; ++t)
      for (int z = 1; z <= kMaxSplit && (z == 1 || steps / z >= 4); z = z < 4 ? z + 1 : z + 2) {
        const double us = tile_us(t, tiles_of(t, K, Tp) * z, (steps + z - 1) / z) +
                          (double)z * K * Tp * 8 / 5e6;
        if (us < least) {
          least = us;
          tile_x = t;
          splits = z;
        }
      }
  }
};

// ---- orthogonalised update ---------------------------------------------------------------------

// Square tiles of four sizes; a launch takes the one with the smallest estimated time: rounds of
// tiles over the 256 units, times the steps of 64 k at the time a step takes on a full device, plus
// a fixed time (fill of the pipeline, epilogue).  Large tiles read less per product, small ones
// fill the device, and the smallest fits on a unit twice; symmetric results have only the tiles on
// and below the diagonal, whose number is what matters: 4096 x 4096 in 256s is 136 tiles for 256
// units, in 192s 253.  Measured (us for five steps with the symmetric products in 256 / 192 / 128
// / 64, the update in its pick): 4096 x 11008 3566 / 3324 / 4002 / 4944, 2048 x 8192 1456 / 1106 /
// 874 / 955, 1536 x 6144 1020 / 750 / 556 / 480, 1024 x 4096 680 / 482 / 345 / 241.  With the
// update in each, the symmetric ones in their pick: 3315 / 3556 / 3818 / 4488, 868 / 931 / 1004 /
// 1094, 583 / 552 / 656 / 638, 337 / 276 / 244 / 262.
struct OrthTile {
  int size, per_unit;
  float step_us, fixed_us;
};
constexpr OrthTile kOrthTiles[] = {
    {256, 1, 1.85f, 11.f}, {192, 1, 1.15f, 8.f}, {128, 1, 0.5f, 4.5f}, {64, 2, 0.25f, 3.5f}};
constexpr OrthTile kOrthSplitTiles[] = {{128, 1, 1.1f, 5.f}, {64, 1, 0.45f, 4.f}};

template <int N>
inline int pick_orth_tile(const OrthTile (&tiles)[N], int64_t rows, int64_t cols, int steps, bool lower) {
  int best = tiles[0].size;
  double least = 1e30;
  for (const OrthTile& t : tiles) {
    const int64_t m = (rows + t.size - 1) / t.size, n = (cols + t.size - 1) / t.size;
    const int64_t count = lower ? m * (m + 1) / 2 : m * n;
    const double rounds = (double)((count * t.per_unit + 255) / 256) / t.per_unit;
    const double us = (rounds < 1 ? 1 : rounds) * (steps * (double)t.step_us + t.fixed_us);
    if (us < least) {
      least = us;
      best = t.size;
    }
  }
  return best;
}

}  // namespace nm

#endif  // NM_TILES_H

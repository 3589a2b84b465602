// nm_tiles.h -- which kernel a 4-bit product or a compressed one with an epilogue takes, which tile a dense
// product takes, and how the gradients and the logits are cut.  Plain C++ with no
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

// ---- compressed products of few tokens ------------------------------------------------------------

// The thin product's workgroup: 16 rg rows, 16 nt columns, a step of 64 K to each of eight waves at a
// time; Tp: padded columns; direct: X's numbers are loaded one by one where they lie, without a copy
// (T = 1: in whole pieces).  Estimated time (us): one launch or two and the first loads, then rounds of
// workgroups over 256 units times eight steps at `step`, which a unit's loads set.  Measured for 64
// steps: one round of 16 x 16 8.3, 32 x 32 10.3, 32 x 64 13.0; 16 rounds of 32 x 64 145; in fp32, whose
// expanded products set it, 13.2 and 29.  Through the copy / direct, bf16: 300 x 512, 8 columns 6.0 / 4.1,
// 1000 x 1024, 128 columns 7.4 / 5.2, 517 columns 11.8 / 14.2; 4096 x 4096, 8 columns 9.4 / 8.7, 32
// columns 11.0 / 11.5 (int8 10.3 / 12.9); 128 x 4096, 256 columns 11.2 / 7.6.  4:8 is expanded in
// registers: 4096 x 4096 with 8, 32 and 256 columns 11.8, 17.3 and 36 where 2:4 takes 8.7, 11.1 and 24.
struct ThinPlan {
  int rg = 1, nt = 1;
  int64_t Tp = 0;
  bool direct = false;
  double us = 1e30;
  ThinPlan(int64_t R, int64_t K, int64_t T, int m, bool f32) {
    constexpr int kShapes[3][2] = {{1, 1}, {2, 2}, {2, 4}};
    constexpr double kStep[3] = {0.41, 0.65, 1.0}, kStep32[2] = {1.0, 3.0};
    constexpr double kOnes[2] = {0.22, 0.6};  // more for X's numbers one by one
    for (int i = 0; i < (f32 ? 2 : 3); ++i) {
      const int64_t rows = 16 * kShapes[i][0], cols = 16 * kShapes[i][1], tp = (T + cols - 1) / cols;
      const int64_t groups = (R + rows - 1) / rows * tp, eights = ((K + 63) / 64 + 7) / 8;
      const double each = (double)((groups + 255) / 256) * (double)eights, more = m != 8 ? 1 : f32 ? 1.2 : 1.7;
      const double step = more * (f32 ? kStep32[i] : kStep[i]);
      for (int d = 0; d < (K % 64 == 0 && i < 2 ? 2 : 1); ++d) {
        const double t = d == 0 ? 5 + each * step : 3 + each * (step + (T == 1 ? 0 : kOnes[i]));
        if (t >= us) continue;
        us = t;
        direct = d == 1;
        rg = kShapes[i][0];
        nt = kShapes[i][1];
        Tp = tp * cols;
      }
    }
  }
};

// Estimated time (us) of the tiled kernels on the same product: a tile's steps alone where there are few
// tiles, a flow of tiles over the units where there are many.  Measured: 2:4 and 1:2 in 16 bits 4096 x
// 1024, 8 columns 15.5, 4096 x 4096 38.9, with 1024 columns 41, 8192 x 4096 40.7, 262144 x 256, 8
// columns 39; in 8 bits 4096 x 4096 24, 8192 x 4096, 1024 columns 32; expanded in 16 bits 100 and 128,
// in fp32 342 and 594; 4:8 in 16 bits 300 x 512 13.9, 2358 x 1856 40, 4096 x 4096 65, 8192 x 512, 1024
// columns 18.5.
inline double tiled_us(int64_t R, int64_t K, int n, int m, int64_t T, int elem) {
  const double S = (double)((K + 63) / 64);
  const bool sparse = ((n == 2 && m == 4) || (n == 1 && m == 2)) && K % 64 == 0;
  const double tiles = (double)((R + 127) / 128) * (double)((T + 127) / 128);
  if (elem == 4) return std::max(5.3 + 5.25 * S, tiles / 512 * (5 + 9.2 * S));
  if (n == 4 && m == 8 && elem == 2 && K % 64 == 0)
    return std::max(7 + 0.9 * S, tiles / 256 * (4.5 + 0.41 * S));
  if (!sparse || (elem == 1 && K % 128 != 0)) return std::max(7 + 1.45 * S, tiles / 512 * (5 + 1.9 * S));
  if (elem == 1) return std::max(9.7 + 0.22 * S, tiles / 512 * (6 + 0.2 * S));
  return std::max(7.2 + 0.49 * S, tiles / 256 * (3.9 + 0.25 * S));
}

// Whether nm_spmm_act's product goes to the thin kernel (elem: bytes of an element).  Its 512 work-items for
// 16 rows at least have to stay below the 2^32 of a launch's dimension.
inline bool thin_preferred(int64_t R, int64_t K, int n, int m, int64_t T, int elem) {
  const bool pattern = (n == 2 && m == 4) || (n == 1 && (m == 2 || m == 4)) || (n == 4 && m == 8);
  if (!pattern || K == 0 || T > 4096 || (R + 15) / 16 * 512 >= (int64_t)1 << 32) return false;
  const ThinPlan plan(R, K, T, m, elem == 4);
  if (!plan.direct && (K + 63) / 64 * 256 >= (int64_t)1 << 32) return false;  // (X turned, 256 for 64 K)
  return plan.us < tiled_us(R, K, n, m, T, elem);
}

// ---- gradient of the compressed product ---------------------------------------------------------

// Both products of nm_spmm_act_grad in one launch: a tile size for both, and the splits of their sums
// (dX's over R, dW's over T).  Estimated time: all tiles' work in a steady flow over the units, but no
// less than the longest tile, plus the splits' sums written and read (5 GB a ms) and a launch to join
// them.
struct SpmmGradCut {
  int tile = kTile256, splits_x = 1, splits_w = 1;
  SpmmGradCut(int64_t R, int64_t K, int64_t T, bool want_w, bool want_x) {
    const int64_t sx = pad64(R) / 64, sw = pad64(T) / 64;
    const auto next = [](int z) { return z < 4 ? z + 1 : z + 2; };
    const auto alone = [](int t, int64_t s) {
      return t == kTile256 ? 2.0 * s + 8 : t == kTile128 ? 0.65 * s + 4 : 0.45 * s + 3;
    };
    const auto flow = [](int t, int64_t count, int64_t s) {
      return t == kTile256 ? count * (2.0 * s + 8) / 256
                           : count * (t == kTile128 ? 1.19 * s + 4.6 : 0.71 * s + 3.5) / 512;
    };
    const auto join = [](int z, int64_t numbers) { return z == 1 ? 0.0 : 4.5 + z * numbers * 8 / 5e6; };
    double least = 1e30;
    for (int t = 0; t < kXentTiles; ++t)
      for (int zx = 1; zx <= kMaxSplit && (zx == 1 || (want_x && sx / zx >= 4)); zx = next(zx))
        for (int zw = 1; zw <= kMaxSplit && (zw == 1 || (want_w && sw / zw >= 4)); zw = next(zw)) {
          const int64_t lx = (sx + zx - 1) / zx, lw = (sw + zw - 1) / zw;
          double us = 0, longest = 0;
          if (want_x) {
            us += flow(t, tiles_of(t, K, T) * zx, lx);
            longest = alone(t, lx);
          }
          if (want_w) {
            us += flow(t, tiles_of(t, R, K) * zw, lw);
            longest = std::max(longest, alone(t, lw));
          }
          us = std::max(us, longest) + (want_x ? join(zx, K * T) : 0) + (want_w ? join(zw, R * K) : 0);
          if (us < least) {
            least = us;
            tile = t;
            splits_x = zx;
            splits_w = zw;
          }
        }
  }
};

// ---- logits ------------------------------------------------------------------------------------

constexpr int kLogitsCells = 8192;  // words x columns of a workgroup
constexpr int kLogitsEach = 8;      // of them to a work-item, at most
constexpr int kLogitsThreads = 1024;

// A workgroup's tile: 2^log_cols columns, 2^log_cells entries, `threads` work-items.
struct LogitsPlan {
  int log_cols, log_cells, threads;
  int copies;        // of a workgroup's counts
  int64_t blocks_v, blocks_t;
  int64_t grid_v, grid_z;  // blocks_v in two dimensions of the launch, the last ones empty
  bool table;        // the counts go through the workspace
  LogitsPlan(int64_t V, int64_t T, int64_t count);
};

// Columns: 32, whose 128 bytes (fp32) of a row are a whole line, or what there are, to a power of two;
// 16 where tokens are counted in LDS, whose readers are then half as many (50257 x 64, 96,000 tokens
// 20.7 -> 18.0 us, 128000 x 32, 64,000 tokens 25.7 -> 19.6; through the table 28.5 -> 32.7).
// Entries: as many as fit, since every workgroup reads its columns' tokens (50257 x 64 by 32 columns:
// 8192 a workgroup 18 us, 4096 25, 1024 80), but few enough that most of the 256 units have a workgroup.
// Work-items: eight entries each, but all 1024 where there are tokens for them (5000 x 8, 32,000
// tokens 15.2 -> 8.6).
inline LogitsPlan::LogitsPlan(int64_t V, int64_t T, int64_t count) {
  const auto cut = [&](int most) {
    log_cols = 0;
    while (log_cols < most && ((int64_t)1 << log_cols) < T) ++log_cols;
    const int64_t cols = (int64_t)1 << log_cols;
    blocks_t = (T + cols - 1) / cols;
    const int least = std::max(8, 5 + log_cols);  // whole words of the mask
    for (log_cells = 13; log_cells > least; --log_cells) {
      const int64_t words = ((int64_t)1 << log_cells) / cols;
      if ((V + words - 1) / words * blocks_t >= 224) break;
    }
    const int64_t words = ((int64_t)1 << log_cells) / cols;
    blocks_v = (V + words - 1) / words;
  };
  cut(T < (int64_t)1 << 19 ? 4 : 5);  // (a grid has 65535 columns at most)
  // In LDS each of blocks_v workgroups reads a column's tokens, as fast as the caches give them to the
  // units that work; through the table they are read once, and the table is written and read, with two
  // more launches.  `count` is the room for tokens, of which a part is in use.  Measured, us in LDS /
  // through the table: 32000 words, one column of 2000 tokens 5.4 / 10.1, of 100,000 19.8 / 12.3; 32000
  // x 8, 16,000 tokens 7.2 / 10.8, 160,000 25 / 14.5; 50257 x 64, 96,000 tokens 15.7 / 22, 512,000 34 /
  // 29, 2,000,000 99 / 41; 128000 x 256, 256,000 tokens 88 / 98, 1,000,000 124 / 108.
  const double share = std::min(1.0, (double)(blocks_v * blocks_t) / 256), cells = (double)V * (double)T;
  const double in_lds = 3 + 0.45e-6 * cells + (double)blocks_v * (double)count * 8 / (24e6 * share);
  table = count > 0 && in_lds > 8 + 1.1e-6 * cells;
  if (table || count == 0) cut(5);
  copies = std::min(16, kLogitsCells >> log_cells);
  const int64_t each = count / std::max<int64_t>(1, T);  // tokens of a column
  if (each <= 512) copies = 1;
  threads = each > 512 ? kLogitsThreads : std::max(256, (1 << log_cells) / kLogitsEach);
  // a dimension of a launch has fewer than 2^32 work-items
  grid_v = std::min<int64_t>(blocks_v, 1 << 20);
  grid_z = (blocks_v + grid_v - 1) / std::max<int64_t>(1, grid_v);
}

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

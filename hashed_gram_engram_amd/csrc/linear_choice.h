// Which tile and how many parts of K an engram_linear call takes (host side, plain C++).
#pragma once

#include <math.h>
#include <stdint.h>

#include <initializer_list>

namespace engram {

constexpr int kBK = 64;                   // features of a stage
constexpr int kRowB = kBK * 2;            // bytes of a row of a stage
constexpr int kBig = 256;                 // k_linear_big: tokens and weight rows of a tile,
constexpr int kBigLds = 5 * kBig * kRowB; // its ring (three stages of weight rows, two of tokens)

// Tiles: tokens x weight rows, waves, ring slots (0: k_linear_big).
struct TileShape {
  int bm, bn, waves, slots;
};
constexpr TileShape kTiles[15] = {{256, 256, 8, 0}, {128, 256, 8, 3}, {256, 128, 8, 3}, {160, 160, 4, 4}, {128, 160, 4, 4},
                                  {192, 128, 4, 4}, {128, 128, 4, 4}, {128, 128, 4, 2}, {64, 256, 8, 4},  {64, 128, 8, 6},
                                  {64, 64, 4, 4},   {32, 128, 4, 6},  {32, 64, 4, 8},   {32, 32, 2, 8},   {16, 16, 1, 12}};
constexpr int kFew8 = 15, kFew16 = 16;  // k_linear_few for up to 8 and 16 tokens

// Microseconds that a tile shape and a split take, as a model: per stage and compute unit the copies into its
// LDS (66 KB per us) or the MFMAs (8 TFLOP/s); per round of workgroups a prologue and an epilogue; over all, the
// bytes (at 7.3 TB/s, of which 43% of the shorter of the two times does not overlap); the parts written and read at
// 5.5 TB/s and a second launch.  The rates are fitted numbers, not the card's (a copy reaches 4.8 TB/s): fitted to
// 90 plain shapes, 10..8192 tokens, K 128..10240, N 72..25600, without the tiles of fewer than 64 tokens where there
// are more than 64.  Timed since with every tile and split, on those and 40 gated shapes: the choice takes 1.8% longer
// than the best one on average, more than 10% for 9 of the 130, and 23% at worst (2012 x 128 x 1032: 8.5 us, 6.9 with
// 64 x 256).  Where the 256 x 256 tile runs it takes 0.91-1.23 times what the model says, 1.11 on average.
inline double model_us(const TileShape& t, int parts, int64_t M, int K, int64_t rows, int64_t N, int cus) {
  const double tiles = double((M + t.bm - 1) / t.bm) * double((rows + t.bn - 1) / t.bn);
  const int lds = t.slots == 0 ? kBigLds : t.slots * (t.bm + t.bn) * kRowB;
  int fit = 160 * 1024 / lds;  // workgroups of a compute unit
  const int by_waves = t.waves >= 4 ? 8 / t.waves : 8;
  fit = fit < by_waves ? fit : by_waves;
  const double work = tiles * parts, stages = K / 64.0 / parts;
  double n = ceil(work / cus);
  n = n < fit ? n : fit;
  double rounds = work / (cus * n);
  rounds = rounds < 4 ? ceil(rounds) : rounds + 0.5;
  const double copies = n * (t.bm + t.bn) * kRowB / 1024 / 66.0, mfma = n * t.bm * t.bn * 128 / 8.0e6;
  double stage = copies > mfma ? copies : mfma;
  stage = stage > 0.1 ? stage : 0.1;
  const double tile_us = 0.9 + rounds * (stages * stage + 2.9 + t.bm * t.bn * 1.24e-4);
  const double mem_us = 0.9 + 2.0 * (double(M) * K + double(rows) * K + double(M) * N) / 7.3e6;
  double us = tile_us > mem_us ? tile_us + 0.43 * mem_us : mem_us + 0.43 * tile_us;
  if (parts > 1) us += 2.2 + parts * tiles * t.bm * t.bn * 8 / 5.5e6;
  return us;
}

constexpr int64_t kMostPartBytes = int64_t(512) << 20;

// The tile, the parts and the bytes of their workspace.
struct LinearChoice {
  int tile = 0, parts = 1;
  int64_t bytes = 0;
};
inline LinearChoice choose(int64_t M, int K, int N, bool glu, int cus) {
  LinearChoice best;
  const int64_t rows = glu ? 2 * int64_t(N) : N;
  // Up to 16 tokens: the shared-K kernel (one token x 5120 x 5120: 11.0 us, the best tile and split of the
  // others 12.8; x 4096 x 1024: 4.4 and 7.9; 16 tokens x 2048 x 8192: 7.7 and 8.3).  From 9 tokens on only
  // while its tiles are at most two to a compute unit: it reads x once per 16 rows (16 tokens x 6144 x
  // 25,600: 65.7 us, and 55.4 with tiles of 128 rows).
  const int64_t few = (rows + 15) / 16;
  if (M <= 8 || (M <= 16 && few <= 2 * cus)) {
    best.tile = M <= 8 ? kFew8 : kFew16;
    return best;
  }
  double least = 1e30;
  for (int i = 0; i < 15; ++i) {
    const TileShape& t = kTiles[i];
    const int64_t tiles = (M + t.bm - 1) / t.bm * ((rows + t.bn - 1) / t.bn);
    if (tiles > (int64_t(1) << 24)) continue;  // far below what a launch takes
    for (int parts : {1, 2, 3, 4, 6, 8}) {
      const int64_t bytes = parts > 1 ? tiles * parts * t.bm * t.bn * 4 : 0;
      // split only while the parts fill the device at most about three times and are not too short
      if (parts > 1 && (tiles * parts > 3 * cus || K / 64 / parts < 4 || bytes > kMostPartBytes)) break;
      const double us = model_us(t, parts, M, K, rows, N, cus);
      if (us < least) {
        least = us;
        best.tile = i;
        best.parts = parts;
        best.bytes = bytes;
      }
    }
  }
  return best;
}

// The most workspace bytes of any call of at most M rows.  (Fewer rows may need more than M: they have fewer tiles
// and are split.)  Row counts with more tiles than the split's limit above need none, so at most 384 x 256 are
// looked at, 0.5 us each.
inline int64_t most_bytes_up_to(int64_t M, int K, int N, bool glu, int cus) {
  const int64_t rows = glu ? 2 * int64_t(N) : N;
  int64_t last = 0, most = 0;
  if (K / 64 >= 8)
    for (const TileShape& t : kTiles) {
      const int64_t split = 3 * cus / 2 / ((rows + t.bn - 1) / t.bn) * t.bm;
      last = split > last ? split : last;
    }
  last = M < last ? M : last;
  for (int64_t m = 1; m <= last; ++m) {
    const int64_t bytes = choose(m, K, N, glu, cus).bytes;
    most = bytes > most ? bytes : most;
  }
  return most;
}

}  // namespace engram

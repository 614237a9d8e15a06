// Which schedule a call of the FP4 linear takes: whole numbers of the host only, so that a test can ask for it.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace mtp {

constexpr int kLM = 128;          // weight rows per tile
constexpr int kLK = 256;          // codes per stage: four MMAs of 64
constexpr int kMaxSplits = 8;
constexpr int kGroup = 16;        // activation tiles that share a pass over long weights

struct LinearSched {
  int nt;       // activation rows per tile
  int mt;       // weight tiles
  int tiles;    // all tiles: mt times the activation tiles
  int nkb;      // stages per tile
  int splits;   // CTAs per tile (a cluster along k); 1: persistent
  bool group;   // persistent, activation tiles in groups
};

// Few rows (up to one tile of them): the smallest N tile, and k split over clusters until the weight
// tiles fill the SMs. More: the N tile whose waves cost the least (a wave's time goes with N).
inline LinearSched make_sched(int R, int N, int kp, int sm_count) {
  LinearSched c{};
  c.mt = N / kLM + (N % kLM != 0 ? 1 : 0);  // (N + kLM may pass 2^31)
  c.nkb = kp / kLK;
  c.splits = 1;
  static const int kTiles[] = {16, 32, 64, 128, 192, 224};
  double best = 1e30;
  for (int nt : kTiles) {
    if (R > 128 && nt < 64) continue;  // (the workspace holds the scale blocks of no smaller tiles)
    const int64_t tiles = static_cast<int64_t>(c.mt) * ((R + nt - 1) / nt);
    int splits = 1;
    while (splits < kMaxSplits && splits < c.nkb && tiles * (splits + 1) <= sm_count &&
           static_cast<size_t>(splits) * nt * kLM * 4 <= 160 * 1024)
      ++splits;
    const int64_t waves = (tiles * splits + sm_count - 1) / sm_count;
    const int kbs = (c.nkb + splits - 1) / splits;
    // per stage: the MMAs (N 16 columns at a time), or the copy of 128 + nt rows of codes
    const double cost = static_cast<double>(waves) * (kbs * (nt > 96 ? nt : 96 + nt / 16) + 400.0) + nt;
    if (cost < best) {
      best = cost;
      c.nt = nt;
      c.tiles = static_cast<int>(tiles);
      c.splits = splits;
    }
  }
  // Weights beyond half of L2 are passed over once for kGroup activation tiles (154880 x 6144, 256 rows: 139 us, with
  // a pass for each tile 180; 2048 rows 944 and 1033); shorter ones stay there while the activations go by (2048 rows
  // of 6144 -> 12288: 77 us, in groups 108; 4096 rows of 12288 -> 6144: 141 and 147).
  c.group = c.splits == 1 && c.nt >= 128 && c.tiles >= sm_count && static_cast<int64_t>(N) * kp * 9 / 16 > (64 << 20);
  return c;
}

}  // namespace mtp

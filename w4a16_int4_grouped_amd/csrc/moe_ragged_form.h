// The forms of a grouped product's tiles and the rule that chooses one, host
// arithmetic on a call's sizes.
#pragma once

#include <stdint.h>

namespace moe {

// The forms of tiles, and which a call takes: the one whose estimate is the
// least. An estimate is rounds of workgroups times the us of one, and no less
// than the bytes at 5.5 TB/s; ties (the bytes) go to the first.
//   LARGE  256 x 256, 8 waves, a workgroup per CU: a step (64 values, 256 in FP4) 1.0 alone to 1.75 on all CUs, less
//          where a group's last tile has fewer rows, 10 besides
//   TWO    128 x 128, 4 waves, two a CU: 0.65 to 1.0 a step, 5 besides
//   FOUR   the same in one LDS stage, four a CU that cover for each other: 0.95 to 2.0, 6 besides
//   SPLIT  64 x 64, the contraction split over 4 waves: 0.75 for four steps, 4 besides
//   THIN   32 x 64 over 6 waves (FP4: 5): 0.75 for six steps (0.5 on few CUs), 4 besides
// Measured in us (rows in all, N, K):       LARGE   TWO  FOUR SPLIT  THIN
//   48 experts, 24576, 4096, 7168            1467          2327
//   384 experts, 32768, 7168, 256             517   514   409  2070
//   16 experts, 8192, 2048, 1024               52    47    48   107
//   1 expert, 1024, 4096, 4096                 74    47    68    59
//   1 expert, 250, 4872, 7168                               46    55
//   1 expert, 512, 512, 7168                  113    76   110    25    20
//   1 expert, 64, 1024, 7168                                20    14
//   wgrad, 64 experts, 4000, 2048, 2048       134   130   107   717
enum Form : int { LARGE = 0, TWO = 1, FOUR = 2, SPLIT = 3, THIN = 4 };

// Waves that share a tile's contraction (SPLIT, THIN).
constexpr int split_waves(bool mx, int BI) { return BI == 64 ? 4 : mx ? 5 : 6; }

// A call: E experts, M rows in all, I output columns, contraction C; wgrad: J
// output rows of an expert, the contraction is its rows.
struct FormCall {
  bool mx, wgrad;
  int E, M, I, J, C;
  int out_size;   // bytes of an output value
};

inline Form form_of(const FormCall& p) {
  if (p.M == 0) return LARGE;
  const double live = p.E < p.M ? p.E : p.M, rows = p.M / live;
  const double C = p.wgrad ? rows : p.C;
  const double steps = __builtin_ceil(C / (p.mx ? 256 : 64));
  auto tiles = [&](int B, int BI) {
    return (p.wgrad ? p.E * __builtin_ceil((double)p.J / B) : live * __builtin_ceil(rows / B)) *
           __builtin_ceil((double)p.I / BI);
  };
  auto busy = [](double n, double full) { return n < full ? n / full : 1.0; };
  const double j = p.wgrad ? p.J : rows;   // rows of an expert's tiles
  const double part = j <= 64 ? 0.5 : j <= 128 ? 0.65 : j <= 192 ? 0.83 : 1.0, few = j <= 64 ? 0.75 : 1.0;
  const double size = p.mx ? 17.0 / 32 : 2, osize = p.out_size;
  const double bytes = p.wgrad ? (double)p.M * (p.I + p.J) * 2 + (double)p.E * p.I * p.J * osize
                               : live * p.I * p.C * size + (double)p.M * (p.C * size + p.I * osize);
  const double n0 = tiles(256, 256), n1 = tiles(128, 128), n2 = tiles(64, 64), n3 = tiles(64, 32);
  const double us[5] = {
      __builtin_ceil(n0 / 256) * (steps * (1.0 + 0.75 * busy(n0, 256)) * part + 10),
      __builtin_ceil(n1 / 512) * (steps * (0.65 + 0.35 * busy(n1, 512)) * few + 5),
      __builtin_ceil(n1 / 1024) * (steps * (0.95 + 1.05 * busy(n1, 1024)) * few + 6),
      __builtin_ceil(n2 / 256) * (__builtin_ceil(steps / 4) * 0.75 + 4),
      __builtin_ceil(n3 / 256) * (__builtin_ceil(steps / split_waves(p.mx, 32)) * 0.75 + 4)};
  int best = LARGE;
  double least = 0;
  for (int f = LARGE; f <= THIN; ++f) {
    const double t = us[f] > bytes / 5.5e6 ? us[f] : bytes / 5.5e6;
    if (f == LARGE || t < least) best = f, least = t;
  }
  return (Form)best;
}

}  // namespace moe

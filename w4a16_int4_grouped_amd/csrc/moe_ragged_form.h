// The forms of a grouped product's tiles and the rule that chooses one, host
// arithmetic on a call's sizes.
#pragma once

namespace moe {

// The forms of tiles, and which a call takes: the one whose estimate is the
// least. An estimate is rounds of workgroups times the us of one, and no less
// than the bytes at 5.5 TB/s; ties (the bytes) go to the first.
//   LARGE  256 x 256, 8 waves, a workgroup per CU: a step (64 values, 256 in FP4) 1.0 alone to 1.75 on all CUs, less
//          where a group's last tile has fewer rows, 10 besides
//   TWO    128 x 128, 4 waves, two a CU: 0.65 to 1.0 a step, 5 besides
//   FOUR   the same in one LDS stage, four a CU that cover for each other: 0.95 to 2.0, 6 besides
//   SPLIT  64 x 64, the contraction split over 4 waves: 0.75 for four steps, 4 besides
//   THIN   32 x 64 over 6 waves (FP4: 5): 0.75 for six steps, 4 besides
// The constants were fitted to the forward product; the gradients and FP4 use
// them too. Measured in us, each form in turn on one GPU (rows in all, N, K; the
// form taken is marked):
//                                            LARGE    TWO   FOUR  SPLIT   THIN
//   forward   48 experts, 24576, 4096, 7168  1412*   1696   2295   2832   4134
//            384 experts, 32768, 7168, 256    483     448    363*  1684   2746
//             16 experts,  8192, 2048, 1024    52*     47     49    106    154
//             16 experts,  8192, 2048, 2048    92*     84     90    154    223
//              1 expert,   1024, 4096, 4096    69      45*    63     57     90
//              1 expert,    250, 4872, 7168   114      76    107     46*    55
//              1 expert,    512,  512, 7168   114      76    108     24     19*
//              1 expert,     64, 1024, 7168    50      42     52     20     14*
//   input     48 experts, 24576, 4096, 7168  1440*   1684   2048   3119   5093
//            384 experts, 32768, 256, 7168    490     474    380*  1711   2850
//             16 experts,  8192, 2048, 1024    47      55*    50     80    124
//             16 experts,  8192, 2048, 2048    94*     84     89    155    243
//              1 expert,   1024, 4096, 4096    73      46*    63     58    104
//              1 expert,    512, 7168, 512    120      74    103     28     26*
//   weights    8 experts, 16384, 4096, 7168   884*   1002    971   1983   3246
//             64 experts,  4000, 2048, 2048   150     128    107*   764   1133
//             16 experts,  8192, 2048, 1024    48      50     45*   141    213
//             16 experts,  2048,  512,  512    10       8.6*   9.3   14     20
//              1 expert,   2000,  512,  512    42      17     24      9.4    8.9*
//              1 expert,  24576,  256,  256   440     244    336     68     62*
//   FP4       48 experts, 24576, 4096, 7168   487*    563    541   1193   1725
//            384 experts, 32768, 7168, 256    288     284    201*  1462   2482
//             16 experts,  8192, 2048, 2048    38      34     32*    89    129
//              1 expert,   1024, 4096, 4096    27      16*    21     28     44
//              1 expert,    250, 4872, 7168    39      24     33     20*    24
//              1 expert,    512,  512, 7168    38      17     25     10      8.6*
// Where the form taken is not the fastest (16 experts of 512 rows), estimates lie
// within a few us of each other and the call loses 9 to 18 %.
// The rule knows the rows in all, not the groups, which are on the device: it
// takes a call as even over min(E, M) experts. A call whose rows lie with a few
// of its experts gets the form of an even one.
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

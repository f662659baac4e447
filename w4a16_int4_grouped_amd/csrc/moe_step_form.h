// The rules that choose forms of the kernels of a training step, host arithmetic
// on a call's sizes.
#pragma once

namespace moe {

// ---- combine's gradient ----

// Threads of a team, and whether it takes a token's rows one by one. Measured in
// us (BF16, top-8, 384 experts with groups padded to 16 rows; 64 and 256 threads,
// all rows / one row a team; the form taken is marked):
//   columns, tokens     64: all    one   256: all    one
//    7168      16           54     12         18    6.1*
//    7168     128           78     28         32     28*
//    7168     512           84     39*        39     41
//    7168    1024          101     75         64*    76
//    7168    4096          234    229        216*   267
//    2880      16           23    6.2         12    4.8*
//    2880     512           38     18*        24     20
//    2880    1024           45     31         30*    34
//    2880    4096           96     91         91*   109
//    2048     512           22     12*        18     16
//    2048    2048           35     36*        39     46
//    1536    4096           49*    48         54     76
// 48 experts:
//    1024    8192           68*    64         86    132
//    2048   16384          234*   241        229    316
// 48 experts, 16 and 64 threads:   16: all    one    64: all    one
//      64    2048                     7.2    4.2*       7.9    7.7
//      64   16384                      22*    25         40     55
//     256    2048                      11    6.7*        14     11
//     512    2048                      16    9.7*        17     13
//     512   16384                      65     59*        66     80
struct Team {
  int threads;
  bool one;
};
inline Team team_of(int T, int H) {
  if (H > 2048) return T <= 128 ? Team{256, true} : T < 1024 ? Team{64, true} : Team{256, false};
  return H > 512 ? Team{64, T < 4096} : Team{16, T < 8192 || H > 256};
}

}  // namespace moe

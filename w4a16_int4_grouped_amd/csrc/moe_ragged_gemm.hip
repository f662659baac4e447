// Grouped products over ragged groups of rows on tiles of the matrix cores:
// out[j][i] = sum over c of Q(j, c) P(i, c) per expert (moe_ragged.h).
//
// A tile's operands pass through LDS in steps of 128 bytes a row, brought by
// copies straight from global memory; each 16-byte fragment feeds a 32x32
// matrix instruction, BF16 / FP16 (16 values of the contraction) and FP4 (64)
// alike, so one kernel serves all. What bounds it:
//   prefill (48 experts, 24576 rows, 4096 x 7168): 1409 us, 1.0 PFLOP/s where
//     the library's plain product of 16384 rows reaches 1.5 and this kernel 1.3
//     on one expert; the same loop on operands that stay in LDS takes 960 (at
//     the higher clock of operands that do not change): the rest is waiting for
//     operands, which miss the L2 (7.0 GB for 3.2 GB of them), a tile's fill and
//     store, with nothing beside it on its CU, and groups that end inside a tile
//     and a round (5 and 7 %); FP4 474 us, 3.0 PFLOP/s
//   decode (448 rows): the weights' bytes, 6.2 TB/s; FP4 5.6 TB/s
//   short contractions (TP8 down, 256): the bytes, 5.1 TB/s
#include "moe_ragged_tile.h"

namespace moe {

hipError_t launch_ragged_gemm(const RaggedParams& p, int way, int type, hipStream_t s) {
  if (way == WAY_MX) return launch<FMT_MX, false, false>(p, s);
  if (type == TYPE_BF16) {
    if (way == WAY_FWD) return launch<FMT_BF16, false, false>(p, s);
    if (way == WAY_DGRAD) return launch<FMT_BF16, true, false>(p, s);
    return launch<FMT_BF16, true, true>(p, s);
  }
  if (way == WAY_FWD) return launch<FMT_F16, false, false>(p, s);
  if (way == WAY_DGRAD) return launch<FMT_F16, true, false>(p, s);
  return launch<FMT_F16, true, true>(p, s);
}

}  // namespace moe

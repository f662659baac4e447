// The experts' forward product with an epilogue on its FP32 sums: a bias per
// expert, SwiGLU of gate | up weights, a residual, one rounding.
//
// The tiles are those of the plain product (moe_ragged_tile.h). For SwiGLU a
// tile's rows of weights alternate, 32 gate rows and the 32 up rows that belong
// to them (16 and 16 where the tile has 32), so that a lane holds both values of
// a pair.
//
// What bounds it is what bounds the plain product; the epilogue adds (us, plain
// / bias and SwiGLU, with half the output / bias and residual, BF16):
//   48 experts, 24576 rows, 4096 x 7168       1146 / 1151 / 1178
//   48 experts, 448 rows, 4096 x 7168          458 / 450 / 451 (64 x 64 tiles)
//   384 experts, 32768 rows, 7168 x 256        352 / 390 / 475 (470 MB more to read)
//   1 expert, 250 rows, 4864 x 7168             45 / 55 / 49
//   8 experts, 64 rows, 1024 x 256             3.8 / 4.1 / 4.1
// form_of_linear chooses the form of tiles: the fastest of the five or one within
// 6 % of it at 14 such sizes.
// Measured and left out: bias and residual read before the products where the
// contraction is split (none, and 16 -> 23 us for one row of 4096 x 7168); the
// residual of the first 32 rows read with the first operands of 128-row tiles
// (registers spill: TP8 down 526 -> 555 us); tiles of few rows dealt last (1435 ->
// 1460 us for uneven groups: their weights are read again).
#include "moe_ragged_tile.h"

namespace moe {

template <int FMT>
static hipError_t linear_for(const RaggedParams& p, hipStream_t s) {
  if (p.epi.swiglu) return launch<FMT, false, false, EPI_GLU>(p, s);
  return launch<FMT, false, false, EPI_ADD>(p, s);
}

hipError_t launch_ragged_linear(const RaggedParams& p, int type, hipStream_t s) {
  return type == TYPE_BF16 ? linear_for<FMT_BF16>(p, s) : linear_for<FMT_F16>(p, s);
}

}  // namespace moe

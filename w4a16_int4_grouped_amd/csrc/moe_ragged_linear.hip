// The experts' forward product with an epilogue on its FP32 sums: a bias per
// expert, SwiGLU of gate | up weights, a residual, one rounding.
//
// The tiles are those of the plain product (moe_ragged_tile.h). For SwiGLU a
// tile's rows of weights alternate, 32 gate rows and the 32 up rows that belong
// to them (16 and 16 where the tile has 32), so that a lane holds both values of
// a pair.
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

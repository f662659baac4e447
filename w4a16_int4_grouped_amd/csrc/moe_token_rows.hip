// The sum of a token's rows and its gradients:
//   out[t] = sum_j w[t, j] y[slots[t, j]]
//   d_y[slots[t, j]] = w[t, j] d_out[t],  d_w[t, j] = <d_out[t], y[slots[t, j]]>
// with sums in FP32, j ascending, rounded once. A slot outside [0, R) names no
// row and adds nothing. Without weights (w = 1) the sum is the gradient of a
// permutation, and d_y a permutation itself.
//
// Both go by tokens: a token's row of d_out is read once for its topk rows, and
// no two tokens meet in a row (a routing's slots are distinct), so nothing is
// added in memory. HBM bounds the large calls, the chain slot -> row -> sum the
// small (one token of 7168, top-8: 2.8 us). 8192 tokens of 7168, top-8, BF16: the
// sum 188 us, 5.6 TB/s; the gradients, with the rows of 384 groups padded to 128,
// 520 us for 1.06 GB read and 1.41 GB written, 4.8 TB/s where a copy runs at 4.95.
// The gradients of rows pass the caches by: nothing here reads them again (561
// us through them, padding behind the tokens).
#include "moe_grid.h"
#include "moe_rows.h"
#include "moe_step.h"
#include "moe_step_form.h"

namespace moe {
namespace {

constexpr int kRowsAhead = 8;   // rows whose loads are in flight together

// A thread sums 8 columns of a token. 1 << lg threads (a power of two, at most
// 256) lie along a row, `parts` workgroups where it is longer.
//   NARROW  less than a wave on a row
//   ROW     a wave's lanes have one token, whose slots and weights are scalars
//   FLAT    where several workgroups a row would leave more than a quarter of
//           their threads idle: adjacent threads on adjacent columns, a division
//           for each (32640 tokens of 2056, four rows each, BF16: 119 against 141 us,
//           half as many in FP32 135 against 203; 131072 of 136, one workgroup for
//           eight tokens, 43 against 44)
// (One workgroup that goes through the parts of its row measured 2.8 -> 6.3 us for
// a token of 7168, 24 -> 25 for 1024 tokens and 96 -> 98 for 4096.)
enum Mode : int { NARROW = 0, ROW = 1, FLAT = 2 };

template <int TYPE, int MODE>
__global__ __launch_bounds__(256) void combine_sum(CombineParams p, int out_type, int lg, int parts,
                                                   uint32_t first) {
  const uint32_t wg = first + blockIdx.x;   // of the call's
  int64_t t;
  int col;
  if constexpr (MODE == FLAT) {
    const uint32_t i = wg * 256 + threadIdx.x, n = (uint32_t)p.H / 8;
    t = i / n;
    col = 8 * (int)(i - (uint32_t)t * n);
  } else {
    const int blk = parts == 1 ? wg : wg / parts, part = wg - blk * parts;
    const int row = threadIdx.x >> lg;
    t = (int64_t)blk * (256 >> lg) + (MODE == ROW ? __builtin_amdgcn_readfirstlane(row) : row);
    col = 8 * (part * 256 + (threadIdx.x & ((1 << lg) - 1)));
  }
  if (t >= p.T || col >= p.H) return;
  const int32_t* slots = p.slots + t * p.topk;
  float acc[8] = {};
  for (int j0 = 0; j0 < p.topk; j0 += kRowsAhead) {
    int slot[kRowsAhead];
    float w[kRowsAhead];
    Raw8<TYPE> raw[kRowsAhead];
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
      const bool in = j0 + j < p.topk;
      slot[j] = in ? slots[j0 + j] : -1;
      w[j] = in && p.w ? p.w[t * p.topk + j0 + j] : 1.f;
    }
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
      raw[j].zero();
      if (slot[j] >= 0 && slot[j] < p.R) raw[j].load(p.y, slot[j] * p.y_ld + col);
    }
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
      if (slot[j] < 0 || slot[j] >= p.R) continue;
      float v[8];
      raw[j].get(v);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = __builtin_fmaf(w[j], v[k], acc[k]);
    }
  }
  const int64_t at = t * p.out_ld + col;
  if (out_type == TYPE_BF16) store8<TYPE_BF16>(p.out, at, acc);
  else if (out_type == TYPE_F16) store8<TYPE_F16>(p.out, at, acc);
  else store8<TYPE_F32>(p.out, at, acc);
}

constexpr int kHeld = 4;        // pieces of 8 values of d_out that a thread holds
constexpr int kPadRows = 16;

// The sum over a team's lanes, 16 (a row of lanes: rotations by 1, 2, 4 and 8) or 64.
template <int TEAM>
__device__ __forceinline__ float team_sum(float v) {
  if constexpr (TEAM == 16) {
    v += dpp_or_0<0x121>(v);
    v += dpp_or_0<0x122>(v);
    v += dpp_or_0<0x124>(v);
    return v + dpp_or_0<0x128>(v);
  }
  return wave_sum_of(v);
}

// TEAM threads (16, 64 or 256) take `each` of a token's rows, 16 threads only of
// up to 512 columns. The call's first workgroups (this launch's begin with
// `first`) look through kPadRows rows each for such as no token names and write
// 0 there.
template <int TYPE, int TEAM>
__global__ __launch_bounds__(256) void combine_grad(CombineParams p, int parts, int each, int pad_blocks,
                                                    uint32_t first) {
  __shared__ float sums[4][64];   // TEAM 256: of a wave, per row
  const int blk = (int)(first + blockIdx.x);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (blk < pad_blocks) {
    const int lo = p.offsets ? max(p.offsets[0], 0) : 0, hi = p.offsets ? min(p.offsets[p.E], p.R) : p.R;
    const float zero[8] = {};
    int src[kPadRows / 4];
    const int64_t r0 = (int64_t)blk * kPadRows + wave * (kPadRows / 4);
#pragma unroll
    for (int i = 0; i < kPadRows / 4; ++i) src[i] = r0 + i >= lo && r0 + i < hi ? p.row_src[r0 + i] : 0;
    for (int i = 0; i < kPadRows / 4; ++i) {
      if (r0 + i < lo || r0 + i >= hi || (src[i] >= 0 && (int64_t)src[i] < (int64_t)p.T * p.topk)) continue;
      for (int c = 8 * lane; c < p.H; c += 512) store8<TYPE, true>(p.d_y, (r0 + i) * p.dy_ld + c, zero);
    }
    return;
  }
  const int64_t block = blk - pad_blocks;
  const int64_t team = TEAM == 16 ? (block * 4 + wave) * 4 + lane / 16 : TEAM == 64 ? block * 4 + wave : block;
  const int64_t t = parts == 1 ? team : (uint32_t)team / (uint32_t)parts;
  const int id = TEAM == 16 ? lane % 16 : TEAM == 64 ? lane : threadIdx.x;
  const int j0 = (int)(team - t * parts) * each, j1 = min(j0 + each, p.topk);
  if (t < p.T) {
    float mine = 0.f;             // lane j: of row j0 + j, in this wave's columns
    for (int base = 0; base < p.H; base += TEAM * 8 * kHeld) {
      float d[kHeld][8];
      int cols[kHeld];
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        cols[i] = base + 8 * (i * TEAM + id);
        Raw8<TYPE> raw;
        raw.zero();
        if (cols[i] < p.H) raw.load(p.d_out, t * p.d_ld + cols[i]);
        raw.get(d[i]);
      }
      for (int j = j0; j < j1; ++j) {
        const int slot = p.slots[t * p.topk + j];
        const bool has = slot >= 0 && slot < p.R;
        const float w = p.w ? p.w[t * p.topk + j] : 1.f;
        float dot = 0.f;
        if (has && p.y) {
          Raw8<TYPE> raw[kHeld];
#pragma unroll
          for (int i = 0; i < kHeld; ++i) {
            raw[i].zero();
            if (cols[i] < p.H) raw[i].load(p.y, slot * p.y_ld + cols[i]);
          }
#pragma unroll
          for (int i = 0; i < kHeld; ++i) {
            float v[8];
            raw[i].get(v);
#pragma unroll
            for (int k = 0; k < 8; ++k) dot = __builtin_fmaf(d[i][k], v[k], dot);
          }
        }
        if (has) {
#pragma unroll
          for (int i = 0; i < kHeld; ++i) {
            if (cols[i] >= p.H) continue;
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = w * d[i][k];
            store8<TYPE, true>(p.d_y, slot * p.dy_ld + cols[i], v);
          }
        }
        if (p.d_w) {
          const float sum = team_sum<TEAM>(dot);
          if (TEAM == 16) {
            if (id == 0) p.d_w[t * p.topk + j] = sum;
          } else if (lane == j - j0) {
            mine += sum;
          }
        }
      }
    }
    if (TEAM == 64 && p.d_w && lane < j1 - j0) p.d_w[t * p.topk + j0 + lane] = mine;
    if (TEAM == 256) sums[wave][lane] = mine;
  }
  if (TEAM == 256) {              // t < T for all of the workgroup, or for none
    __syncthreads();
    if (t < p.T && p.d_w && threadIdx.x < (unsigned)(j1 - j0))
      p.d_w[t * p.topk + j0 + threadIdx.x] =
          sums[0][threadIdx.x] + sums[1][threadIdx.x] + sums[2][threadIdx.x] + sums[3][threadIdx.x];
  }
}

}  // namespace

hipError_t launch_combine_out(const CombineParams& p, int type, int out_type, hipStream_t s) {
  const int H8 = p.H / 8;
  int lg = 0;
  while (lg < 8 && (1 << lg) < H8) ++lg;
  const int parts = (H8 + 255) / 256;
  const int64_t all = (int64_t)p.T * H8;
  const bool flat = parts > 1 && 4 * H8 < 3 * 256 * parts && all < ((int64_t)1 << 31) - 256;
  const int64_t g = flat ? (all + 255) / 256 : ((int64_t)p.T + (256 >> lg) - 1) / (256 >> lg) * parts;
  if (g > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  auto go = [&](auto ty) {
    constexpr int TYPE = decltype(ty)::value;
    return in_slices(g, 256, [&](uint32_t first, uint32_t n) {
      if (flat) combine_sum<TYPE, FLAT><<<n, 256, 0, s>>>(p, out_type, lg, parts, first);
      else if (lg >= 6) combine_sum<TYPE, ROW><<<n, 256, 0, s>>>(p, out_type, lg, parts, first);
      else combine_sum<TYPE, NARROW><<<n, 256, 0, s>>>(p, out_type, lg, parts, first);
      return hipGetLastError();
    });
  };
  if (type == TYPE_BF16) return go(std::integral_constant<int, TYPE_BF16>{});
  if (type == TYPE_F16) return go(std::integral_constant<int, TYPE_F16>{});
  return go(std::integral_constant<int, TYPE_F32>{});
}

hipError_t launch_combine_grad(const CombineParams& p, int type, hipStream_t s) {
  const Team m = team_of(p.T, p.H);
  const int parts = m.one ? p.topk : 1, each = m.one ? 1 : p.topk;
  const int64_t teams = (int64_t)p.T * parts, blocks = (teams * m.threads + 255) / 256;
  const int pads = p.row_src ? (p.R + kPadRows - 1) / kPadRows : 0;
  const int64_t g = blocks + pads;
  if (g > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  auto go = [&](auto ty) {
    constexpr int TYPE = decltype(ty)::value;
    return in_slices(g, 256, [&](uint32_t first, uint32_t n) {
      if (m.threads == 256) combine_grad<TYPE, 256><<<n, 256, 0, s>>>(p, parts, each, pads, first);
      else if (m.threads == 64) combine_grad<TYPE, 64><<<n, 256, 0, s>>>(p, parts, each, pads, first);
      else combine_grad<TYPE, 16><<<n, 256, 0, s>>>(p, parts, each, pads, first);
      return hipGetLastError();
    });
  };
  if (type == TYPE_BF16) return go(std::integral_constant<int, TYPE_BF16>{});
  if (type == TYPE_F16) return go(std::integral_constant<int, TYPE_F16>{});
  return go(std::integral_constant<int, TYPE_F32>{});
}

}  // namespace moe

// Gradient of the experts' biases: the sum of each group's rows, in FP32.
//
// A workgroup sums LANES * 8 columns of one group: LANES lanes lie along a row
// (16 bytes each), the others and the waves along the rows, whose sums meet in a
// fixed order. A group's rows are one workgroup's, whatever their number.
#include "moe_rows.h"
#include "moe_step.h"

namespace moe {
namespace {

constexpr int kWaves = 8;
constexpr int kAhead = 4;   // rows of a lane whose loads are in flight together

template <int TYPE, int LANES>
__global__ __launch_bounds__(64 * kWaves) void bias_grad(BiasGradParams p, int out_type, int blocks) {
  __shared__ float part[kWaves][LANES * 8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x / blocks, c0 = (blockIdx.x - e * blocks) * LANES * 8;
  const int col = c0 + 8 * (lane % LANES);
  const int lo = min(max(p.offsets[e], 0), p.M), hi = min(p.offsets[e + 1], p.M);
  float sum[8] = {};
  if (col < p.N) {
    constexpr int kStep = 64 / LANES * kWaves;   // rows of a round
    for (int64_t r = lo + wave * (64 / LANES) + lane / LANES; r < hi; r += kStep * kAhead) {
      Raw8<TYPE> raw[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        raw[i].zero();
        if (r + i * kStep < hi) raw[i].load(p.dy, (r + i * kStep) * p.ld + col);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        float v[8];
        raw[i].get(v);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] += v[k];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
#pragma unroll
    for (int o = LANES; o < 64; o <<= 1) sum[k] += __shfl_xor(sum[k], o, 64);
  }
  if (lane < LANES) {
#pragma unroll
    for (int k = 0; k < 8; ++k) part[wave][8 * lane + k] = sum[k];
  }
  __syncthreads();
  const int c = threadIdx.x;
  if (c >= LANES * 8 || c0 + c >= p.N) return;
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) v += part[w][c];
  const int64_t at = (int64_t)e * p.db_ld + c0 + c;
  if (out_type == TYPE_BF16) store1<TYPE_BF16>(p.db, at, v);
  else if (out_type == TYPE_F16) store1<TYPE_F16>(p.db, at, v);
  else store1<TYPE_F32>(p.db, at, v);
}

template <int TYPE, int LANES>
hipError_t go(const BiasGradParams& p, int out_type, hipStream_t s) {
  const int blocks = (p.N + LANES * 8 - 1) / (LANES * 8);
  const int64_t g = (int64_t)p.E * blocks;
  if (g > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  bias_grad<TYPE, LANES><<<(unsigned)g, 64 * kWaves, 0, s>>>(p, out_type, blocks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_bias_grad(const BiasGradParams& p, int type, int out_type, hipStream_t s) {
  const bool wide = (int64_t)p.E * ((p.N + 63) / 64) >= 256;   // workgroups for every CU
  if (type == TYPE_BF16) return wide ? go<TYPE_BF16, 8>(p, out_type, s) : go<TYPE_BF16, 1>(p, out_type, s);
  return wide ? go<TYPE_F16, 8>(p, out_type, s) : go<TYPE_F16, 1>(p, out_type, s);
}

}  // namespace moe

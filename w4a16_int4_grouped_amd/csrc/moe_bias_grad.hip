// Gradient of the experts' biases: the sum of each group's rows, in FP32.
//
// A workgroup sums 64 columns of one group: 8 lanes lie along a row (16 bytes
// each, a line), the others and the waves along the rows, whose sums meet in a
// fixed order. HBM bounds it where there are enough groups and columns: 24576
// rows of 4096 in 48 even groups 34 to 37 us (5.4 to 5.9 TB/s), uneven ones on
// other rows at each call 39. A workgroup alone reads some 60 to 90 GB/s:
// where groups are few and long, the rows are cut into chunks, a workgroup sums
// 64 columns of a chunk for each group in it, and a second kernel adds the
// chunks' sums up. Part c + e of the workspace belongs to chunk c and group e; no
// two such pairs have the same sum, because both only grow along the rows.
#include "moe_grid.h"
#include "moe_rows.h"
#include "moe_step.h"

namespace moe {
namespace {

constexpr int kWaves = 8;
constexpr int kAhead = 4;    // rows of a lane whose loads are in flight together
constexpr int kChunk = 256;  // rows: a round of loads
constexpr int kStep = 8 * kWaves;   // rows that a workgroup's lanes take at a time
// Values that FP32 adds up one after another; such sums are added in FP64 (4
// million equal rows in one chain a lane were off by 2^-11). A group's rows go
// through the whole workgroup's sum that many a lane at a time, because a second
// set of sums in registers costs short groups more: 384 groups of 170 rows of
// 2048 43 -> 45 us.
constexpr int kFold = 256;

struct Rows {
  int lo, hi;
};
__device__ __forceinline__ Rows group(const BiasGradParams& p, int e) {
  const int lo = min(max(p.offsets[e], 0), p.M);
  return Rows{lo, max(min(p.offsets[e + 1], p.M), lo)};
}

// The sum of column c0 + threadIdx.x over rows [lo, hi), in threads below 64.
template <int TYPE>
__device__ __forceinline__ float column_sum(const BiasGradParams& p, int c0, int lo, int hi, float (&part)[kWaves][64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = c0 + 8 * (lane & 7);
  float sum[8] = {};
  if (col < p.N) {
    for (int64_t r = lo + wave * 8 + (lane >> 3); r < hi; r += kStep * kAhead) {
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
    for (int o = 8; o < 64; o <<= 1) sum[k] += __shfl_xor(sum[k], o, 64);
  }
  if (lane < 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) part[wave][8 * lane + k] = sum[k];
  }
  __syncthreads();
  float v = 0.f;
  if (threadIdx.x < 64) {
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += part[w][threadIdx.x];
  }
  return v;
}

__device__ __forceinline__ void store_any(void* x, int64_t at, int type, float v) {
  if (type == TYPE_BF16) store1<TYPE_BF16>(x, at, v);
  else if (type == TYPE_F16) store1<TYPE_F16>(x, at, v);
  else store1<TYPE_F32>(x, at, v);
}

template <int TYPE>
__global__ __launch_bounds__(64 * kWaves) void bias_grad(BiasGradParams p, int out_type, int blocks, uint32_t first) {
  __shared__ float part[kWaves][64];
  const int wg = (int)(first + blockIdx.x), e = wg / blocks, c0 = (wg - e * blocks) * 64;
  const Rows g = group(p, e);
  float v = column_sum<TYPE>(p, c0, g.lo, min((int64_t)g.lo + kStep * kFold, (int64_t)g.hi), part);
  if (g.hi - g.lo > kStep * kFold) {
    double far = v;
    for (int64_t r = (int64_t)g.lo + kStep * kFold; r < g.hi; r += kStep * kFold) {
      __syncthreads();   // part is read
      far += column_sum<TYPE>(p, c0, (int)r, min(r + kStep * kFold, (int64_t)g.hi), part);
    }
    v = (float)far;
  }
  if (threadIdx.x < 64 && c0 + (int)threadIdx.x < p.N)
    store_any(p.db, (int64_t)e * p.db_ld + c0 + threadIdx.x, out_type, v);
}

// A chunk of rows by 64 columns; the groups in it, the first found by halves.
template <int TYPE>
__global__ __launch_bounds__(64 * kWaves) void bias_grad_parts(BiasGradParams p, int blocks, uint32_t first) {
  __shared__ float part[kWaves][64];
  const int wg = (int)(first + blockIdx.x), c = wg / blocks, c0 = (wg - c * blocks) * 64;
  const int r0 = c * kChunk, r1 = min((int64_t)r0 + kChunk, (int64_t)p.M);
  int a = 0, b = p.E;
  while (a < b) {
    const int m = (a + b) / 2;
    if (p.offsets[m + 1] > r0) b = m;
    else a = m + 1;
  }
  for (int e = a; e < p.E; ++e) {
    const Rows g = group(p, e);
    if (g.lo >= r1) break;
    const int lo = max(g.lo, r0), hi = min(g.hi, r1);
    if (lo >= hi) continue;
    const float v = column_sum<TYPE>(p, c0, lo, hi, part);
    if (threadIdx.x < 64 && c0 + (int)threadIdx.x < p.N)
      static_cast<float*>(p.ws)[((int64_t)c + e) * p.N + c0 + threadIdx.x] = v;
    __syncthreads();
  }
}

__global__ __launch_bounds__(64 * kWaves) void bias_grad_finish(BiasGradParams p, int out_type, int blocks,
                                                               uint32_t first) {
  __shared__ float part[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wg = (int)(first + blockIdx.x), e = wg / blocks, col = (wg - e * blocks) * 64 + lane;
  const Rows g = group(p, e);
  float v = 0.f;
  if (g.lo < g.hi && col < p.N) {
    const float* from = static_cast<const float*>(p.ws) + (int64_t)e * p.N + col;
    auto add_up = [&](int c, int last) {
#pragma unroll 8
      for (; c <= last; c += kWaves) v += from[(int64_t)c * p.N];
    };
    const int first = g.lo / kChunk, last = (g.hi - 1) / kChunk;
    if (last - first < kWaves * kFold) {
      add_up(first + wave, last);
    } else {
      double far = 0.0;
      for (int c = first; c <= last; c += kWaves * kFold) {
        add_up(c + wave, min(c + kWaves * kFold - 1, last));
        far += v, v = 0.f;
      }
      v = (float)far;
    }
  }
  part[wave][lane] = v;
  __syncthreads();
  if (wave || col >= p.N) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v += part[w][lane];
  store_any(p.db, (int64_t)e * p.db_ld + col, out_type, v);
}

int64_t chunks_of(int M) { return ((int64_t)M + kChunk - 1) / kChunk; }

// Whether the rows are cut: where an even group's rows take one workgroup longer
// (at 60 GB/s) than all bytes at 5.5 TB/s and a second kernel's 3.5 us. In us,
// whole / cut (groups, rows in all, columns; the one taken is marked):
//   1, 2048, 512     5.1 / 4.9*      1, 24576, 64     34 / 5.8*       4, 8192, 1024    8.3* / 6.7
//   1, 4096, 512     7.8 / 4.9*      1, 24576, 512    73 / 7.8*       8, 24576, 64     9.2 / 5.6*
//   2, 4096, 7168    12* / 13        1, 24576, 4096   93 / 36*        8, 16384, 4096   25* / 25
//   16, 8192, 1024   4.2* / 6.7      48, 24576, 4096  37* / 37        8, 448, 4096     3.4* / 9.7
// (4 groups of 2048 rows of 1024 take the slower side.) The rule takes the rows as
// even over the groups: where one of many has most of them, it alone takes as long
// as a single group: nine tenths of 24576 rows of 4096 with one of 48 86 us.
bool cut(int E, int M, int N) {
  const double bytes = (double)M * N * 2 / 5.5e6, waves = (double)E * ((N + 63) / 64) / 512;
  const double alone = (double)M / E * 128 / 60e3 * (waves > 1 ? waves : 1);
  return alone > bytes + 3.5;
}

}  // namespace

size_t bias_grad_ws_bytes(int E, int M, int N) { return cut(E, M, N) ? (size_t)(chunks_of(M) + E) * N * 4 : 0; }

hipError_t launch_bias_grad(const BiasGradParams& p, int type, int out_type, hipStream_t s) {
  const int blocks = (p.N + 63) / 64;
  const int64_t groups = (int64_t)p.E * blocks, parts = chunks_of(p.M) * blocks;
  if (groups > 0x7FFFFFFF || parts > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  constexpr int kThreads = 64 * kWaves;
  if (!cut(p.E, p.M, p.N)) {
    return in_slices(groups, kThreads, [&](uint32_t first, uint32_t n) {
      if (type == TYPE_BF16) bias_grad<TYPE_BF16><<<n, kThreads, 0, s>>>(p, out_type, blocks, first);
      else bias_grad<TYPE_F16><<<n, kThreads, 0, s>>>(p, out_type, blocks, first);
      return hipGetLastError();
    });
  }
  const hipError_t e = in_slices(parts, kThreads, [&](uint32_t first, uint32_t n) {
    if (type == TYPE_BF16) bias_grad_parts<TYPE_BF16><<<n, kThreads, 0, s>>>(p, blocks, first);
    else bias_grad_parts<TYPE_F16><<<n, kThreads, 0, s>>>(p, blocks, first);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  return in_slices(groups, kThreads, [&](uint32_t first, uint32_t n) {
    bias_grad_finish<<<n, kThreads, 0, s>>>(p, out_type, blocks, first);
    return hipGetLastError();
  });
}

}  // namespace moe

// MXFP4: rows of FP4 (e2m1) codes with one power-of-two scale (E8M0, a biased
// exponent byte) per 32 values.
//
// For a block of 32 with largest magnitude m the scale is 2^(floor(log2 m) -
// 2), 2 being the exponent of e2m1's largest value 6; its byte is m's FP32
// exponent field less 2, at least 0 (2^-127, for m below 2^-124). Each value
// over the scale is rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, to
// the even code of two as near, and what lies above 6 becomes 6. A block with
// a NaN or an infinity gets byte 255: all of it reads back as NaN.
//
// Four lanes share a block, eight values each: 16-byte loads of 2-byte
// values, 4-byte stores of codes, one byte of scale from the first. A
// workgroup takes 1024 adjacent groups of 8, four a thread, so that the grid
// passes through memory once (98304 x 7168 BF16: 310 us, 5.8 TB/s read and
// written; a fixed grid striding through memory took 410 us). HBM bounds it, as
// it does the way back (328 us). A thread's four loads do not cover for each
// other where 16-bit values are unpacked under the load's condition: each is
// waited for there, and the other waves of the CU are the cover; FP32 loads, and
// the codes on the way back, are in flight together.
#include "moe_device.h"
#include "moe_ragged.h"

namespace moe {
namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

// Values are read once: past the caches (310 against 315 us for 1.4 GB).
template <int TYPE>
__device__ __forceinline__ void load8(const void* x, int64_t at, float (&v)[8]) {
  if constexpr (TYPE == TYPE_F32) {
    const f32x4_t* p = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(x) + at);
    const f32x4_t a = __builtin_nontemporal_load(p), b = __builtin_nontemporal_load(p + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  } else {
    const u32x4_t w =
        __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(x) + at));
    if constexpr (TYPE == TYPE_BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
    } else {
      const f16x8_t h = __builtin_bit_cast(f16x8_t, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
    }
  }
}

template <int TYPE>
__device__ __forceinline__ void store8(void* x, int64_t at, const float (&v)[8]) {
  if constexpr (TYPE == TYPE_F32) {
    f32x4_t* p = reinterpret_cast<f32x4_t*>(static_cast<float*>(x) + at);
    p[0] = f32x4_t{v[0], v[1], v[2], v[3]};
    p[1] = f32x4_t{v[4], v[5], v[6], v[7]};
  } else if constexpr (TYPE == TYPE_BF16) {
    *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(x) + at) =
        u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  } else {
    f16x8_t h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (_Float16)v[i];
    *reinterpret_cast<f16x8_t*>(static_cast<_Float16*>(x) + at) = h;
  }
}

// A thread's places among rows of n8 groups of 8 values: its first by one
// division, the next ones a workgroup's 256 groups on by additions.
struct Place {
  int64_t r;
  int c;
};
__device__ __forceinline__ Place place_of(int64_t i, int n8) {
  const int64_t r = i / n8;
  return Place{r, (int)(i - r * n8)};
}
__device__ __forceinline__ void advance(Place& p, const Place& step, int n8) {
  p.r += step.r;
  p.c += step.c;
  if (p.c >= n8) p.c -= n8, ++p.r;
}

constexpr int kBatch = 4;   // groups per thread

template <int TYPE>
__global__ __launch_bounds__(256) void mx_quant(const void* __restrict__ x, int64_t rows, int K8, int64_t ld,
                                                uint32_t* __restrict__ q, uint8_t* __restrict__ scales, int s_ld) {
  const Place step{256 / K8, 256 % K8};
  Place p = place_of((int64_t)blockIdx.x * (256 * kBatch) + threadIdx.x, K8);
  // K8 is a multiple of 4, so the four lanes of a block are all in or all out
  float v[kBatch][8];
  Place at[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    at[b] = p;
    if (p.r < rows) load8<TYPE>(x, p.r * ld + 8 * p.c, v[b]);
    advance(p, step, K8);
  }
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    if (at[b].r >= rows) break;
    uint32_t m = 0;   // magnitudes order as their bits do, NaN above infinity
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(v[b][k]) & 0x7FFFFFFFu);
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, 0xB1, 0xF, 0xF, false));   // lane ^ 1
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, 0x4E, 0xF, 0xF, false));   // lane ^ 2
    const bool bad = m >= 0x7F800000u;
    const int e = max((int)(m >> 23) - 2, 0);
    const float s = __uint_as_float(e > 0 ? (uint32_t)e << 23 : 0x00400000u);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[b][0], v[b][1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[b][2], v[b][3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[b][4], v[b][5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[b][6], v[b][7], s, 3);
    const int64_t r = at[b].r;
    const int c = at[b].c;
    q[r * K8 + c] = bad ? 0u : w;
    if ((c & 3) == 0) {
      scales[r * s_ld + (c >> 2)] = (uint8_t)(bad ? 255 : e);
      // and, with a row's last scale, the bytes behind it
      if (c + 4 == K8)
        for (int z = K8 / 4; z < s_ld; ++z) scales[r * s_ld + z] = 0;
    }
  }
}

template <int TYPE>
__global__ __launch_bounds__(256) void mx_dequant(const uint32_t* __restrict__ q, const uint8_t* __restrict__ scales,
                                                  int64_t rows, int K8, int s_ld, void* __restrict__ out, int64_t ld) {
  const Place step{256 / K8, 256 % K8};
  Place p = place_of((int64_t)blockIdx.x * (256 * kBatch) + threadIdx.x, K8);
  uint32_t w[kBatch], e[kBatch];
  Place at[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    at[b] = p;
    if (p.r < rows) w[b] = q[p.r * K8 + p.c], e[b] = scales[p.r * s_ld + (p.c >> 2)];
    advance(p, step, K8);
  }
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    if (at[b].r >= rows) break;
    const float s = __uint_as_float(e[b] == 255 ? 0x7FC00000u : e[b] > 0 ? e[b] << 23 : 0x00400000u);
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t code = (w[b] >> (4 * k)) & 15u, m = code & 7u;
      // e2m1: exponent m / 2, one mantissa bit; 0 and 0.5 have exponent field 0
      const float f = m < 2 ? 0.5f * (float)m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
      v[k] = (code & 8u ? -f : f) * s;
    }
    store8<TYPE>(out, at[b].r * ld + 8 * at[b].c, v);
  }
}

int64_t grid_for(int64_t groups) { return (groups + 256 * kBatch - 1) / (256 * kBatch); }

}  // namespace

hipError_t launch_mx_quant(const void* x, int type, int64_t rows, int K, int64_t x_ld, uint8_t* q, uint8_t* scales,
                           int s_ld, hipStream_t s) {
  const int K8 = K / 8;
  const int64_t g = grid_for(rows * K8);
  if (g > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  uint32_t* qw = reinterpret_cast<uint32_t*>(q);
  if (type == TYPE_BF16) mx_quant<TYPE_BF16><<<(unsigned)g, 256, 0, s>>>(x, rows, K8, x_ld, qw, scales, s_ld);
  else if (type == TYPE_F16) mx_quant<TYPE_F16><<<(unsigned)g, 256, 0, s>>>(x, rows, K8, x_ld, qw, scales, s_ld);
  else mx_quant<TYPE_F32><<<(unsigned)g, 256, 0, s>>>(x, rows, K8, x_ld, qw, scales, s_ld);
  return hipGetLastError();
}

hipError_t launch_mx_dequant(const uint8_t* q, const uint8_t* scales, int64_t rows, int K, int s_ld, void* out,
                             int type, int64_t out_ld, hipStream_t s) {
  const int K8 = K / 8;
  const int64_t g = grid_for(rows * K8);
  if (g > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const uint32_t* qw = reinterpret_cast<const uint32_t*>(q);
  if (type == TYPE_BF16) mx_dequant<TYPE_BF16><<<(unsigned)g, 256, 0, s>>>(qw, scales, rows, K8, s_ld, out, out_ld);
  else if (type == TYPE_F16) mx_dequant<TYPE_F16><<<(unsigned)g, 256, 0, s>>>(qw, scales, rows, K8, s_ld, out, out_ld);
  else mx_dequant<TYPE_F32><<<(unsigned)g, 256, 0, s>>>(qw, scales, rows, K8, s_ld, out, out_ld);
  return hipGetLastError();
}

}  // namespace moe

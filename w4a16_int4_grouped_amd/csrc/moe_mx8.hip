// Rows in 8 bits and SwiGLU with such a checkpoint of its input.
//
// For a block of 32 values along a row (the row's last may be shorter) with
// largest magnitude m the scale is 2^e, e = floor(log2 m), its byte m's FP32
// exponent field (0: 2^-127); a value is the integer q = x / 2^(e - 6) rounded
// to the nearest (even of two as near), at most 127 in magnitude, so m itself
// may lose half a step more than the others. q 2^(e - 6) has 7 significant
// bits: exact in BF16, so that a product of rows read back multiplies the
// checkpoint's own values. A block with a NaN or an infinity gets byte 255:
// all of it reads back as NaN.
//
// Four lanes share a block, eight values each, as in the MXFP4 kernels; a row is
// a whole number of such quads of lanes, the last of which may have lanes
// without values.
#include "moe_rows.h"
#include "moe_step.h"

namespace moe {
namespace {

struct Range {
  int64_t lo, hi;
};
__device__ __forceinline__ Range live_rows(const LiveRows& l, int64_t rows) {
  if (!l.offsets) return Range{0, rows};
  const int64_t lo = min((int64_t)max(l.offsets[0], 0), rows);
  return Range{lo, max(min((int64_t)l.offsets[l.E], rows), lo)};
}

// Group i among rows of n: by 32-bit division where the call's groups allow it.
__device__ __forceinline__ Place group_place(int64_t i, int n, bool small) {
  if (small) {
    const uint32_t r = (uint32_t)i / (uint32_t)n;
    return Place{(int64_t)r, (int)((uint32_t)i - r * (uint32_t)n)};
  }
  return place_of(i, n);
}

// Scale byte of the quad's block, in its four lanes (255: not finite).
__device__ __forceinline__ uint32_t block_scale(const float (&v)[8]) {
  uint32_t m = 0;   // magnitudes order as their bits do, NaN above infinity
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(v[k]) & 0x7FFFFFFFu);
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, 0xB1, 0xF, 0xF, false));   // lane ^ 1
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, 0x4E, 0xF, 0xF, false));   // lane ^ 2
  return m >> 23;
}

// The codes of eight values under scale byte b. x + 1.5 * 2^23 rounds x to an
// integer (nearest, even of two) and holds it in its low bits.
__device__ __forceinline__ u32x2_t encode(const float (&v)[8], uint32_t b) {
  uint32_t x[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float s = __builtin_amdgcn_ldexpf(v[k], 133 - (int)b);
    x[k] = __float_as_uint(__builtin_amdgcn_fmed3f(s, -127.f, 127.f) + kRoundMagic);
  }
  u32x2_t r;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t lo = __builtin_amdgcn_perm(x[4 * k + 1], x[4 * k], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(x[4 * k + 3], x[4 * k + 2], 0x04000C0Cu);
    r[k] = b == 255 ? 0u : lo | hi;
  }
  return r;
}

__device__ __forceinline__ void decode(u32x2_t w, uint32_t b, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int q = (int)(w[k >> 2] << (24 - 8 * (k & 3))) >> 24;
    v[k] = b == 255 ? __uint_as_float(0x7FC00000u) : __builtin_amdgcn_ldexpf((float)q, (int)b - 133);
  }
}

// Codes and scale of group c of a row of K8, and behind a row's last scale the
// bytes up to s_ld.
__device__ __forceinline__ void store_codes(int8_t* q, uint8_t* scales, int c, int K8, int s_ld, u32x2_t codes,
                                            uint32_t b) {
  *reinterpret_cast<u32x2_t*>(q + 8 * c) = codes;
  if ((c & 3) == 0) {
    scales[c >> 2] = (uint8_t)b;
    if (c + 4 >= K8)
      for (int z = (c >> 2) + 1; z < s_ld; ++z) scales[z] = 0;
  }
}

constexpr int kBatch = 4;   // groups per thread

template <int TYPE>
__global__ __launch_bounds__(256) void mx8_quant(const void* __restrict__ x, int64_t rows, int K8, int64_t ld,
                                                 int8_t* __restrict__ q, uint8_t* __restrict__ scales, int s_ld,
                                                 bool small) {
  const int n = (K8 + 3) & ~3;   // a row's lanes
  const Place step{256 / n, 256 % n};
  Place p = group_place((int64_t)blockIdx.x * (256 * kBatch) + threadIdx.x, n, small);
  Raw8<TYPE> raw[kBatch];
  Place at[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    at[b] = p;
    raw[b].zero();
    if (p.r < rows && p.c < K8) raw[b].load(x, p.r * ld + 8 * p.c);
    advance(p, step, n);
  }
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    float v[8];
    raw[b].get(v);
    const uint32_t sc = block_scale(v);
    const u32x2_t codes = encode(v, sc);
    const int64_t r = at[b].r;
    if (r < rows && at[b].c < K8) store_codes(q + r * 8 * K8, scales + r * s_ld, at[b].c, K8, s_ld, codes, sc);
  }
}

template <int TYPE>
__global__ __launch_bounds__(256) void mx8_dequant(Mx8Rows m, bool small) {
  const int K8 = m.K / 8;
  const Range live = live_rows(m.live, m.out_rows);
  const Place step{256 / K8, 256 % K8};
  const int64_t first = (int64_t)blockIdx.x * (256 * kBatch);
  Place p = group_place(first + threadIdx.x, K8, small);
  u32x2_t w[kBatch];
  uint32_t e[kBatch];
  Place at[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    at[b] = p;
    int64_t r = p.r;
    bool has = r >= live.lo && r < live.hi;
    if (has && m.row_src) {
      const int id = m.row_src[r];
      r = (uint32_t)id / (uint32_t)m.topk;
      has = id >= 0 && r < m.rows;
    }
    w[b] = u32x2_t{}, e[b] = 0;
    if (has) {
      w[b] = *reinterpret_cast<const u32x2_t*>(m.q + r * m.K + 8 * p.c);
      e[b] = m.scales[r * m.s_ld + (p.c >> 2)];
    }
    advance(p, step, K8);
  }
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    if (at[b].r < live.lo || at[b].r >= live.hi) continue;
    float v[8];
    decode(w[b], e[b], v);
    store8<TYPE>(m.out, at[b].r * m.ld + 8 * at[b].c, v);
  }
}

// sigmoid(g): for 16-bit rows by v_exp_f32 and v_rcp_f32, off by a few 2^-24
// times |g|, far less than the outputs' rounding; for FP32 rows as expf and a
// division give it.
template <int TYPE>
__device__ __forceinline__ float sigma(float g) {
  if constexpr (TYPE == TYPE_F32) return 1.0f / (1.0f + expf(-g));
  else return __builtin_amdgcn_rcpf(1.0f + __expf(-g));
}

constexpr int kPairs = 2;   // groups per thread, of both halves

// a = g s(g) u, and g | u in 8 bits, each half of a row in blocks of its own.
template <int TYPE>
__global__ __launch_bounds__(256) void swiglu_save(SwigluParams s, bool small) {
  const int I8 = s.I / 8, n = (I8 + 3) & ~3;
  const Range live = live_rows(s.live, s.rows);
  const Place step{256 / n, 256 % n};
  Place p = group_place((int64_t)blockIdx.x * (256 * kPairs) + threadIdx.x, n, small);
  Raw8<TYPE> rg[kPairs], ru[kPairs];
  Place at[kPairs];
#pragma unroll
  for (int b = 0; b < kPairs; ++b) {
    at[b] = p;
    rg[b].zero(), ru[b].zero();
    if (p.r >= live.lo && p.r < live.hi && p.c < I8) {
      rg[b].load(s.h, p.r * s.h_ld + 8 * p.c);
      ru[b].load(s.h, p.r * s.h_ld + s.I + 8 * p.c);
    }
    advance(p, step, n);
  }
#pragma unroll
  for (int b = 0; b < kPairs; ++b) {
    float g[8], u[8], a[8];
    rg[b].get(g), ru[b].get(u);
    const uint32_t bg = block_scale(g), bu = block_scale(u);
    const u32x2_t cg = encode(g, bg), cu = encode(u, bu);
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] = g[k] * sigma<TYPE>(g[k]) * u[k];
    const int64_t r = at[b].r;
    if (r < live.lo || r >= live.hi || at[b].c >= I8) continue;
    store8<TYPE>(s.a, r * s.a_ld + 8 * at[b].c, a);
    store_codes(s.q + 2 * r * s.I, s.scales + 2 * r * s.s_ld, at[b].c, I8, s.s_ld, cg, bg);
    store_codes(s.q + (2 * r + 1) * s.I, s.scales + (2 * r + 1) * s.s_ld, at[b].c, I8, s.s_ld, cu, bu);
  }
}

// dg = da u s (1 + g (1 - s)), du = da g s, and a = g s u again.
template <int TYPE, bool PACKED>
__global__ __launch_bounds__(256) void swiglu_grad(SwigluParams s, bool small) {
  const int I8 = s.I / 8;
  const Range live = live_rows(s.live, s.rows);
  const Place step{256 / I8, 256 % I8};
  Place p = group_place((int64_t)blockIdx.x * (256 * kPairs) + threadIdx.x, I8, small);
  Raw8<TYPE> rg[kPairs], ru[kPairs], rd[kPairs];
  u32x2_t cg[kPairs], cu[kPairs];
  uint32_t bg[kPairs], bu[kPairs];
  Place at[kPairs];
#pragma unroll
  for (int b = 0; b < kPairs; ++b) {
    at[b] = p;
    const int64_t r = p.r;
    if (r >= live.lo && r < live.hi) {
      if constexpr (PACKED) {
        const int8_t* q = s.q_in + 2 * r * s.I + 8 * p.c;
        const uint8_t* sc = s.scales_in + 2 * r * s.s_ld + (p.c >> 2);
        cg[b] = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(q));
        cu[b] = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(q + s.I));
        bg[b] = sc[0], bu[b] = sc[s.s_ld];
      } else {
        rg[b].load(s.h, r * s.h_ld + 8 * p.c);
        ru[b].load(s.h, r * s.h_ld + s.I + 8 * p.c);
      }
      rd[b].load(s.d_a, r * s.da_ld + 8 * p.c);
    }
    advance(p, step, I8);
  }
#pragma unroll
  for (int b = 0; b < kPairs; ++b) {
    const int64_t r = at[b].r;
    if (r < live.lo || r >= live.hi) continue;
    float g[8], u[8], d[8], dg[8], a[8];
    if constexpr (PACKED) decode(cg[b], bg[b], g), decode(cu[b], bu[b], u);
    else rg[b].get(g), ru[b].get(u);
    rd[b].get(d);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float sg = sigma<TYPE>(g[k]), silu = g[k] * sg;
      a[k] = silu * u[k];
      dg[k] = d[k] * u[k] * sg * (1.0f + g[k] * (1.0f - sg));
      d[k] *= silu;
    }
    const int64_t h = r * s.dh_ld + 8 * at[b].c;
    store8<TYPE>(s.d_h, h, dg);
    store8<TYPE>(s.d_h, h + s.I, d);
    if (s.a) store8<TYPE>(s.a, r * s.a_ld + 8 * at[b].c, a);
  }
}

// Workgroups for `groups` groups of 8, or 0 where they are too many for a grid.
unsigned blocks_for(int64_t groups, int each) {
  const int64_t g = (groups + 256 * each - 1) / (256 * each);
  return g > 0x7FFFFFFF ? 0u : (unsigned)g;
}
bool is_small(int64_t groups) { return groups < 0x7FFFFFFF - 4096; }

}  // namespace

hipError_t launch_mx8_quant(const void* x, int type, int64_t rows, int K, int64_t ld, int8_t* q, uint8_t* scales,
                            int s_ld, hipStream_t s) {
  const int K8 = K / 8;
  const int64_t n = rows * ((K8 + 3) & ~3);
  const unsigned g = blocks_for(n, kBatch);
  const bool small = is_small(n);
  if (!g) return hipErrorInvalidConfiguration;
  if (type == TYPE_BF16) mx8_quant<TYPE_BF16><<<g, 256, 0, s>>>(x, rows, K8, ld, q, scales, s_ld, small);
  else if (type == TYPE_F16) mx8_quant<TYPE_F16><<<g, 256, 0, s>>>(x, rows, K8, ld, q, scales, s_ld, small);
  else mx8_quant<TYPE_F32><<<g, 256, 0, s>>>(x, rows, K8, ld, q, scales, s_ld, small);
  return hipGetLastError();
}

hipError_t launch_mx8_dequant(const Mx8Rows& p, int type, hipStream_t s) {
  const int64_t n = p.out_rows * (p.K / 8);
  const unsigned g = blocks_for(n, kBatch);
  const bool small = is_small(n);
  if (!g) return hipErrorInvalidConfiguration;
  if (type == TYPE_BF16) mx8_dequant<TYPE_BF16><<<g, 256, 0, s>>>(p, small);
  else if (type == TYPE_F16) mx8_dequant<TYPE_F16><<<g, 256, 0, s>>>(p, small);
  else mx8_dequant<TYPE_F32><<<g, 256, 0, s>>>(p, small);
  return hipGetLastError();
}

hipError_t launch_swiglu_save(const SwigluParams& p, int type, hipStream_t s) {
  const int64_t n = (int64_t)p.rows * ((p.I / 8 + 3) & ~3);
  const unsigned g = blocks_for(n, kPairs);
  const bool small = is_small(n);
  if (!g) return hipErrorInvalidConfiguration;
  if (type == TYPE_BF16) swiglu_save<TYPE_BF16><<<g, 256, 0, s>>>(p, small);
  else if (type == TYPE_F16) swiglu_save<TYPE_F16><<<g, 256, 0, s>>>(p, small);
  else swiglu_save<TYPE_F32><<<g, 256, 0, s>>>(p, small);
  return hipGetLastError();
}

template <bool PACKED>
static hipError_t grad_for(const SwigluParams& p, int type, hipStream_t s) {
  const int64_t n = (int64_t)p.rows * (p.I / 8);
  const unsigned g = blocks_for(n, kPairs);
  const bool small = is_small(n);
  if (!g) return hipErrorInvalidConfiguration;
  if (type == TYPE_BF16) swiglu_grad<TYPE_BF16, PACKED><<<g, 256, 0, s>>>(p, small);
  else if (type == TYPE_F16) swiglu_grad<TYPE_F16, PACKED><<<g, 256, 0, s>>>(p, small);
  else swiglu_grad<TYPE_F32, PACKED><<<g, 256, 0, s>>>(p, small);
  return hipGetLastError();
}

hipError_t launch_swiglu_grad(const SwigluParams& p, int type, hipStream_t s) {
  return p.h ? grad_for<false>(p, type, s) : grad_for<true>(p, type, s);
}

}  // namespace moe

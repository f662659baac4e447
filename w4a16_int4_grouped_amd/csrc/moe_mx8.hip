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
// without values. All four kernels pass once over their data and are bound by it
// (a large copy runs at 4.95 TB/s here, a fill at 6.8), BF16:
//   mx8_quant    8192 rows of 7168: 31 us, 5.7 TB/s
//   mx8_dequant  as 68288 rows of a routing: 212 to 222 us, 6.6 to 6.9 TB/s, a
//                third of it codes that a token's eight rows read in eight XCDs
//   swiglu_save  65536 rows of 2 x 2048: 180 us, 6.0 TB/s
//   swiglu_grad  the same, from 8 bits: 232 us, 5.9 TB/s
// A thread's loads all stand before its first conversion, so that they are in
// flight together.
#include "moe_grid.h"
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

// A workgroup's threads along rows of n groups of 8 values, `each` groups a
// thread. One division at most, and the same row for a wave's lanes wherever a
// row has more than 32 groups, so that rows, their sources and addresses are
// scalars.
//   NARROW  up to 32 groups: 1 << lg threads on a row (a power of two)
//   ROWS    up to 256 groups: the same, at least a wave on a row
//   WIDE    longer rows: a workgroup on 256 * each groups of one row
//   FLAT    where those would leave more than a quarter of their threads idle:
//           adjacent threads on adjacent groups, a division for each (in us for
//           2^28 values in BF16, to 8 bits / back: rows of 264 148 / 147 against 191 /
//           231, of 520 152 / 147 against 173 / 234, of 2056 133 / 146 against 173 /
//           208; where rows fill their threads, of 512, 122 / 147 without it)
enum Mode : int { NARROW = 0, ROWS = 1, WIDE = 2, FLAT = 3 };

struct Shape {
  int mode, lg, chunks;   // WIDE: chunks of a row; FLAT: a row's groups
  unsigned blocks;        // workgroups, 0: more than 2^31 - 1
  uint32_t first;         // of a launch, among the call's
};

Shape shape_of(int64_t rows, int n, int each) {
  Shape s{n > 256 ? WIDE : n > 32 ? ROWS : NARROW, 0, 1, 0, 0};
  while (s.lg < 8 && (1 << s.lg) < n) ++s.lg;
  int64_t g;
  const int span = s.mode == WIDE ? (n + 255) / 256 * 256 : 1 << s.lg;
  if (4 * n < 3 * span && rows * n < ((int64_t)1 << 31) - 256 * each) {
    s.mode = FLAT, s.chunks = n;
    s.blocks = (unsigned)((rows * n + 256 * each - 1) / (256 * each));
    return s;
  }
  if (s.mode == WIDE) {
    s.chunks = (n + 256 * each - 1) / (256 * each);
    g = rows * s.chunks;
  } else {
    const int64_t per = (int64_t)each * (256 >> s.lg);
    g = (rows + per - 1) / per;
  }
  s.blocks = g > 0x7FFFFFFF ? 0u : (unsigned)g;
  return s;
}

// Row and group of a thread's b-th place.
template <int MODE, int EACH>
__device__ __forceinline__ Place place(const Shape& s, int b) {
  const uint32_t blk = s.first + blockIdx.x;
  const int tid = threadIdx.x;
  if constexpr (MODE == WIDE) {
    const uint32_t r = s.chunks == 1 ? blk : blk / (uint32_t)s.chunks;
    return Place{(int64_t)r, (int)(blk - r * (uint32_t)s.chunks) * (256 * EACH) + 256 * b + tid};
  }
  if constexpr (MODE == FLAT) {
    const uint32_t i = (blk * EACH + b) * 256 + tid, r = i / (uint32_t)s.chunks;
    return Place{(int64_t)r, (int)(i - r * (uint32_t)s.chunks)};
  }
  const int row = MODE == ROWS ? __builtin_amdgcn_readfirstlane(tid >> s.lg) : tid >> s.lg;
  return Place{((int64_t)blk * EACH + b) * (256 >> s.lg) + row, tid & ((1 << s.lg) - 1)};
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

// 2^(b - 133), which is subnormal below b = 7; NaN for 255.
__device__ __forceinline__ float step_of(uint32_t b) {
  return __uint_as_float(b == 255 ? 0x7FC00000u : b > 6 ? (b - 6) << 23 : 1u << (b + 16));
}

// Eight codes times s, exactly.
__device__ __forceinline__ void decode(u32x2_t w, float s, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = (float)(int8_t)(w[k >> 2] >> (8 * (k & 3))) * s;
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

// store8, FP32 in pieces of 64 adjacent bytes where every four lanes hold 32
// adjacent values (quad): first the values of the quad's lower two lanes, then of
// the upper two, rather than 16 bytes of each 32 (2^27 values in rows of 512:
// 136 against 153 us; SwiGLU's kernels, with more to read, gain nothing).
__device__ __forceinline__ float quad_lane(float v, bool upper) {   // of lane q / 2 of the quad, or 2 + q / 2
  const int i = __float_as_int(v);
  return __int_as_float(upper ? __builtin_amdgcn_update_dpp(i, i, 0xFA, 0xF, 0xF, false)
                              : __builtin_amdgcn_update_dpp(i, i, 0x50, 0xF, 0xF, false));
}
template <int TYPE>
__device__ __forceinline__ void store8_of_quad(void* x, int64_t at, const float (&v)[8], bool quad) {
  if constexpr (TYPE == TYPE_F32) {
    if (quad) {
      const int q = threadIdx.x & 3;
      f32x4_t lo, hi;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = quad_lane(v[k], false), b = quad_lane(v[4 + k], false);
        const float c = quad_lane(v[k], true), d = quad_lane(v[4 + k], true);
        lo[k] = q & 1 ? b : a, hi[k] = q & 1 ? d : c;
      }
      float* to = static_cast<float*>(x) + at - 4 * q;   // the quad's first value is at - 8 q
      *reinterpret_cast<f32x4_t*>(to) = lo;
      *reinterpret_cast<f32x4_t*>(to + 16) = hi;
      return;
    }
  }
  store8<TYPE>(x, at, v);
}

// Groups per thread (pairs: of both halves). In us for 1 / 2 / 4 pairs, 65536 rows
// of 2 x 2048: kept 180 / 185 / 190, gradient 232 / 237 / 244; for 2 / 4 / 8 groups
// 8192 rows of 7168 to 8 bits 32 / 31 / 33, back as a routing's 303 / 222 / 319.
constexpr int kQuant = 4, kDequant = 4, kPairs = 1;
// WIDE rows of a workgroup, where they are the many rows of a routing. In us for
// 1 / 4 rows: 11536 rows of 7168 39 / 37, 35808 112 / 112, 68288 281 / 209, 134064
// 639 / 518; of 4096 11552 29 / 31, 35664 80 / 79, 68512 160 / 146.
constexpr int kRoutedRows = 4, kManyRows = 32768;

template <int TYPE, int MODE>
__global__ __launch_bounds__(256) void mx8_quant(const void* __restrict__ x, int64_t rows, int K8, int64_t ld,
                                                 int8_t* __restrict__ q, uint8_t* __restrict__ scales, int s_ld,
                                                 Shape sh) {
  Raw8<TYPE> raw[kQuant];
#pragma unroll
  for (int b = 0; b < kQuant; ++b) {
    const Place p = place<MODE, kQuant>(sh, b);
    raw[b].zero();
    if (p.r < rows && p.c < K8) raw[b].load(x, p.r * ld + 8 * p.c);
  }
#pragma unroll
  for (int b = 0; b < kQuant; ++b) {
    const Place p = place<MODE, kQuant>(sh, b);
    float v[8];
    raw[b].get(v);
    const uint32_t sc = block_scale(v);
    const u32x2_t codes = encode(v, sc);
    if (p.r < rows && p.c < K8) store_codes(q + p.r * 8 * K8, scales + p.r * s_ld, p.c, K8, s_ld, codes, sc);
  }
}

// NR rows at a time (WIDE), so that the chain from a row's source to its codes
// is waited for once for all of them.
template <int TYPE, int MODE, int NR>
__global__ __launch_bounds__(256) void mx8_dequant(Mx8Rows m, Shape sh) {
  const int K8 = m.K / 8;
  const Range live = live_rows(m.live, m.out_rows);
  int64_t src[NR][kDequant];
  u32x2_t w[NR][kDequant];
  uint32_t e[NR][kDequant];
  auto at = [&](int n, int b) {
    Place p = place<MODE, kDequant>(sh, b);
    if (MODE == WIDE) p.r = p.r * NR + n;
    return p;
  };
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int b = 0; b < kDequant; ++b) {
      const int64_t r = at(n, b).r;
      src[n][b] = -1;
      if (r < live.lo || r >= live.hi) continue;
      src[n][b] = r;
      if (!m.row_src) continue;
      const int id = m.row_src[r];
      const uint32_t from = m.topk == 1 ? (uint32_t)id : (uint32_t)id / (uint32_t)m.topk;
      src[n][b] = id >= 0 && from < m.rows ? (int64_t)from : -1;
    }
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int b = 0; b < kDequant; ++b) {
      const int c = at(n, b).c;
      w[n][b] = u32x2_t{}, e[n][b] = 0;
      if (src[n][b] < 0 || c >= K8) continue;
      w[n][b] = *reinterpret_cast<const u32x2_t*>(m.q + src[n][b] * m.K + 8 * c);
      e[n][b] = m.scales[src[n][b] * m.s_ld + (c >> 2)];
    }
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int b = 0; b < kDequant; ++b) {
      const Place p = at(n, b);
      if (p.r < live.lo || p.r >= live.hi || p.c >= K8) continue;
      float v[8];
      decode(w[n][b], step_of(e[n][b]), v);
      store8_of_quad<TYPE>(m.out, p.r * m.ld + 8 * p.c, v, K8 % 4 == 0);
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

// a = g s(g) u, and g | u in 8 bits, each half of a row in blocks of its own.
template <int TYPE, int MODE>
__global__ __launch_bounds__(256) void swiglu_save(SwigluParams s, Shape sh) {
  const int I8 = s.I / 8;
  const Range live = live_rows(s.live, s.rows);
  Raw8<TYPE> rg[kPairs], ru[kPairs];
#pragma unroll
  for (int b = 0; b < kPairs; ++b) {
    const Place p = place<MODE, kPairs>(sh, b);
    rg[b].zero(), ru[b].zero();
    if (p.r >= live.lo && p.r < live.hi && p.c < I8) {
      rg[b].load(s.h, p.r * s.h_ld + 8 * p.c);
      ru[b].load(s.h, p.r * s.h_ld + s.I + 8 * p.c);
    }
  }
#pragma unroll
  for (int b = 0; b < kPairs; ++b) {
    const Place p = place<MODE, kPairs>(sh, b);
    float g[8], u[8], a[8];
    rg[b].get(g), ru[b].get(u);
    const uint32_t bg = block_scale(g), bu = block_scale(u);
    const u32x2_t cg = encode(g, bg), cu = encode(u, bu);
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] = g[k] * sigma<TYPE>(g[k]) * u[k];
    if (p.r < live.lo || p.r >= live.hi || p.c >= I8) continue;
    store8<TYPE>(s.a, p.r * s.a_ld + 8 * p.c, a);
    store_codes(s.q + 2 * p.r * s.I, s.scales + 2 * p.r * s.s_ld, p.c, I8, s.s_ld, cg, bg);
    store_codes(s.q + (2 * p.r + 1) * s.I, s.scales + (2 * p.r + 1) * s.s_ld, p.c, I8, s.s_ld, cu, bu);
  }
}

// dg = da u s (1 + g (1 - s)), du = da g s, and a = g s u again.
template <int TYPE, int MODE, bool PACKED>
__global__ __launch_bounds__(256) void swiglu_grad(SwigluParams s, Shape sh) {
  const int I8 = s.I / 8;
  const Range live = live_rows(s.live, s.rows);
  Raw8<TYPE> rg[kPairs], ru[kPairs], rd[kPairs];
  u32x2_t cg[kPairs], cu[kPairs];
  uint32_t bg[kPairs], bu[kPairs];
#pragma unroll
  for (int b = 0; b < kPairs; ++b) {
    const Place p = place<MODE, kPairs>(sh, b);
    if (p.r < live.lo || p.r >= live.hi || p.c >= I8) continue;
    if constexpr (PACKED) {
      const int8_t* q = s.q_in + 2 * p.r * s.I + 8 * p.c;
      const uint8_t* sc = s.scales_in + 2 * p.r * s.s_ld + (p.c >> 2);
      cg[b] = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(q));
      cu[b] = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(q + s.I));
      bg[b] = sc[0], bu[b] = sc[s.s_ld];
    } else {
      rg[b].load(s.h, p.r * s.h_ld + 8 * p.c);
      ru[b].load(s.h, p.r * s.h_ld + s.I + 8 * p.c);
    }
    rd[b].load(s.d_a, p.r * s.da_ld + 8 * p.c);
  }
#pragma unroll
  for (int b = 0; b < kPairs; ++b) {
    const Place p = place<MODE, kPairs>(sh, b);
    if (p.r < live.lo || p.r >= live.hi || p.c >= I8) continue;
    float g[8], u[8], d[8], dg[8], a[8];
    if constexpr (PACKED) decode(cg[b], step_of(bg[b]), g), decode(cu[b], step_of(bu[b]), u);
    else rg[b].get(g), ru[b].get(u);
    rd[b].get(d);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float sg = sigma<TYPE>(g[k]), silu = g[k] * sg;
      a[k] = silu * u[k];
      dg[k] = d[k] * u[k] * sg * (1.0f + g[k] * (1.0f - sg));
      d[k] *= silu;
    }
    const int64_t h = p.r * s.dh_ld + 8 * p.c;
    store8<TYPE>(s.d_h, h, dg);
    store8<TYPE>(s.d_h, h + s.I, d);
    if (s.a) store8<TYPE>(s.a, p.r * s.a_ld + 8 * p.c, a);
  }
}

// f(TYPE, MODE, shape) for a call's type and shape, once for each launch that it
// takes, whose workgroups the shape passed on has.
template <class F>
hipError_t choose(int type, Shape s, F&& f) {
  using std::integral_constant;
  if (!s.blocks) return hipErrorInvalidConfiguration;
  auto by_mode = [&](auto ty) {
    if (s.mode == NARROW) f(ty, integral_constant<int, NARROW>{}, s);
    else if (s.mode == ROWS) f(ty, integral_constant<int, ROWS>{}, s);
    else if (s.mode == WIDE) f(ty, integral_constant<int, WIDE>{}, s);
    else f(ty, integral_constant<int, FLAT>{}, s);
  };
  return in_slices(s.blocks, 256, [&](uint32_t first, uint32_t n) {
    s.first = first, s.blocks = n;
    if (type == TYPE_BF16) by_mode(integral_constant<int, TYPE_BF16>{});
    else if (type == TYPE_F16) by_mode(integral_constant<int, TYPE_F16>{});
    else by_mode(integral_constant<int, TYPE_F32>{});
    return hipGetLastError();
  });
}
// Lanes of a row whose blocks of 32 are found by four lanes each.
int quads(int n8) { return (n8 + 3) & ~3; }

}  // namespace

hipError_t launch_mx8_quant(const void* x, int type, int64_t rows, int K, int64_t ld, int8_t* q, uint8_t* scales,
                            int s_ld, hipStream_t s) {
  const Shape shape = shape_of(rows, quads(K / 8), kQuant);
  return choose(type, shape, [&](auto ty, auto mode, const Shape& sh) {
    mx8_quant<decltype(ty)::value, decltype(mode)::value><<<sh.blocks, 256, 0, s>>>(x, rows, K / 8, ld, q, scales, s_ld,
                                                                                    sh);
  });
}

hipError_t launch_mx8_dequant(const Mx8Rows& p, int type, hipStream_t s) {
  Shape shape = shape_of(p.out_rows, p.K / 8, kDequant);
  const bool many = shape.mode == WIDE && p.row_src && p.out_rows >= kManyRows;
  if (many) {
    const int64_t g = (p.out_rows + kRoutedRows - 1) / kRoutedRows * shape.chunks;
    shape.blocks = g > 0x7FFFFFFF ? 0u : (unsigned)g;
  }
  return choose(type, shape, [&](auto ty, auto mode, const Shape& sh) {
    constexpr int TYPE = decltype(ty)::value, MODE = decltype(mode)::value;
    if constexpr (MODE == WIDE)
      if (many) return mx8_dequant<TYPE, MODE, kRoutedRows><<<sh.blocks, 256, 0, s>>>(p, sh);
    mx8_dequant<TYPE, MODE, 1><<<sh.blocks, 256, 0, s>>>(p, sh);
  });
}

hipError_t launch_swiglu_save(const SwigluParams& p, int type, hipStream_t s) {
  const Shape shape = shape_of(p.rows, quads(p.I / 8), kPairs);
  return choose(type, shape, [&](auto ty, auto mode, const Shape& sh) {
    swiglu_save<decltype(ty)::value, decltype(mode)::value><<<sh.blocks, 256, 0, s>>>(p, sh);
  });
}

hipError_t launch_swiglu_grad(const SwigluParams& p, int type, hipStream_t s) {
  const Shape shape = shape_of(p.rows, p.I / 8, kPairs);
  return choose(type, shape, [&](auto ty, auto mode, const Shape& sh) {
    constexpr int TYPE = decltype(ty)::value, MODE = decltype(mode)::value;
    if (p.h) swiglu_grad<TYPE, MODE, false><<<sh.blocks, 256, 0, s>>>(p, sh);
    else swiglu_grad<TYPE, MODE, true><<<sh.blocks, 256, 0, s>>>(p, sh);
  });
}

}  // namespace moe

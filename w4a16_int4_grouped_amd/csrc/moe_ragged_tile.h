// The tiles of grouped products over ragged groups of rows, on the matrix
// cores: out[j][i] = sum over c of Q(j, c) P(i, c) per expert (moe_ragged.h).
// What bounds them stands where they are launched.
#pragma once

#include <type_traits>

#include "moe_device.h"
#include "moe_grid.h"
#include "moe_ragged.h"
#include "moe_ragged_form.h"
#include "moe_tile.h"

namespace moe {
namespace {

typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(3))) char lds_char_t;
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

enum Fmt : int { FMT_BF16 = 0, FMT_F16 = 1, FMT_MX = 2 };

constexpr int kStageBytes = 128;          // contraction bytes of a row per step: 64 values, or 256 FP4 codes
constexpr uint32_t kPastEnd = 0x80000000u; // an offset past every operand tile: the load gives 0

// D += A . B on one 32x32 tile (FP32 accumulate), 32 contraction bytes: 16
// BF16 or FP16 values, or 64 FP4 codes. Lane l feeds row l%32 of A and column
// l%32 of B with the 16 bytes of its half l/32; component 4k + i of D is row
// 8k + 4 (l/32) + i, column l%32. FP4: times 2^(scale - 127) of byte SB of the
// lane's scale words, one per 32 codes.
template <int FMT, int SB>
__device__ __forceinline__ f32x16_t mma(u32x4_t a, u32x4_t b, f32x16_t c, int sa, int sb) {
  if constexpr (FMT == FMT_MX) {
    const i32x8_t A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8_t B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, 4, SB, sa, SB, sb);
  } else if constexpr (FMT == FMT_F16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  }
}

// First row and row count of expert e, whatever the offsets hold: within [0, M].
struct Group {
  int lo, n;
};
__device__ __forceinline__ Group group_of(const RaggedParams& p, int e) {
  const int lo = min(max(p.offsets[e], 0), p.M);
  return Group{lo, min(max(p.offsets[e + 1], lo), p.M) - lo};
}

// Workgroup b's item of `total`: runs of G consecutive items (tiles that share
// operands, and one XCD's L2) dealt round-robin to the XCDs, so that each gets
// its part of large and small experts; -1 past the last. A run is 16 items (8,
// 32 and 64 measured within 3 %), less where that would leave XCDs without
// one, but `least`. The grid needs total + 8 * 16 workgroups.
__device__ __forceinline__ int deal(int b, int total, int least) {
  const int G = min(max(total / 64, least), 16);
  const int idx = b >> 3, run = (idx / G) * 8 + (b & 7);
  const int t = run * G + idx % G;
  return t < total ? t : -1;
}
constexpr int kDealSlack = 8 * 16;

struct Tile {
  int e, it, jt;
};

// Tile t of an expert's nj x NI: bands of up to 8 rows, column by column, so
// that tiles which share weights start side by side and 32 tiles in a row (an
// XCD's CUs) have few operand panels (8 x 4: 12).
__device__ __forceinline__ Tile tile_of(int e, int t, int nj, int NI) {
  const int band = t / (8 * NI), r = t - band * 8 * NI, h = min(8, nj - band * 8);
  return Tile{e, r / h, band * 8 + r % h};
}

__device__ __forceinline__ int wave_scan(int v) {   // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o, 64);
    v += lane >= o ? u : 0;
  }
  return v;
}

// The tile of workgroup b among all experts' tiles of BJ rows x NI columns,
// experts in order, and its expert's rows. e < 0: none left. A lane adds up the
// tiles of ceil(E / 64) neighbouring experts, a scan finds the lane that holds
// the tile, and with an expert of that lane's per lane a second scan the
// expert: one load after another only for more than 64 experts, whatever E.
struct Found {
  Tile t;
  Group g;
};
__device__ __forceinline__ Found find_tile(const RaggedParams& p, int b, int BJ, int NI, int least) {
  const int lane = threadIdx.x & 63, each = (p.E + 63) / 64;
  const int32_t* off = p.offsets;
  const Found none = {{-1, 0, 0}, {0, 0}};
  int mine = 0;
  Group g = {0, 0};
  {
    int e = lane * each;
    const int end = min(e + each, p.E);
    int lo = e < end ? off[e] : 0;
#pragma unroll 8
    for (; e < end; ++e) {
      const int hi = off[e + 1];
      g.lo = min(max(lo, 0), p.M);
      g.n = min(max(hi, g.lo), p.M) - g.lo;
      mine += (g.n + BJ - 1) / BJ;
      lo = hi;
    }
  }
  int sum = wave_scan(mine);
  const int t = deal(b, __builtin_amdgcn_readlane(sum, 63) * NI, least);
  if (t < 0) return none;
  uint64_t past = __ballot(sum * NI > t);
  if (!past) return none;
  int at = __builtin_ctzll(past), e0 = 0, before = 0;
  if (each > 1) {
    before = __builtin_amdgcn_readlane(sum - mine, at), e0 = at * each;
    g = lane < each && e0 + lane < p.E ? group_of(p, e0 + lane) : Group{0, 0};
    mine = (g.n + BJ - 1) / BJ;
    sum = wave_scan(mine);
    past = __ballot((before + sum) * NI > t);
    if (!past) return none;
    at = __builtin_ctzll(past);
  }
  const int nj = __builtin_amdgcn_readlane(mine, at);
  const int local = t - (before + __builtin_amdgcn_readlane(sum, at) - nj) * NI;
  const Tile tl = tile_of(e0 + at, local, nj, NI);
  return Found{{__builtin_amdgcn_readfirstlane(tl.e), __builtin_amdgcn_readfirstlane(tl.it),
                __builtin_amdgcn_readfirstlane(tl.jt)},
               {__builtin_amdgcn_readlane(g.lo, at), __builtin_amdgcn_readlane(g.n, at)}};
}

// The same where every expert has J output rows (wgrad), tiles of BJ x BI.
__device__ __forceinline__ Found even_tile(const RaggedParams& p, int b, int BJ, int BI, int least) {
  const int nj = (p.J + BJ - 1) / BJ, NI = (p.I + BI - 1) / BI;
  const int t = deal(b, p.E * nj * NI, least);
  if (t < 0) return Found{{-1, 0, 0}, {0, 0}};
  const int e = t / (nj * NI);
  return Found{tile_of(e, t - e * nj * NI, nj, NI), group_of(p, e)};
}

// Buffer descriptor of `bytes` bytes from p: loads past the last read 0.
__device__ __forceinline__ u32x4_t rsrc(const void* p, uint32_t bytes) {
  const uint64_t a = (uint64_t)p;
  return u32x4_t{(uint32_t)a, (uint32_t)(a >> 32) & 0xFFFFu, bytes, 0x00020000u};
}

// 16 bytes per lane straight from global memory (r + voff + soff) to LDS
// (dst + 16 * lane), in assembly: the compiler would hold every LDS read back
// until all such copies have landed. fence() waits for them. One wait state
// after the write of m0; a scalar operand from a vector instruction (a lane
// read) would need five: settle() stands between those and the first copy, the
// later ones' operands come from scalar instructions.
__device__ __forceinline__ void copy16(char* dst, u32x4_t r, uint32_t voff, uint32_t soff) {
  const uint32_t at = (uint32_t)(uintptr_t)(lds_void_t*)dst;
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "{m0}"(at), "v"(voff), "s"(r), "s"(soff)
               : "memory");
}

__device__ __forceinline__ void settle() { asm volatile("s_nop 4" ::: "memory"); }

// All but this wave's last N copies have landed and its LDS reads are done;
// and so it is with every wave of the workgroup.
template <int N>
__device__ __forceinline__ void fence() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// One operand's tile of B output rows/columns: copies to LDS and fragment
// reads. A copy moves 1 KB per wave; offsets past the operand's last byte read
// as 0 and take part in nothing.
//
// COL false (contiguous along the contraction): B rows of 128 bytes, 16-byte
// piece c of row r at position c ^ spread(r). A 16-byte LDS read serves lanes
// 0-3, 12-15, 20-27 at a time, then the others of a half: either way rows of
// one parity (half of the banks) get eight different positions (no conflict
// counted).
// COL true: 64 contraction rows of B values, 32-byte chunk c of row r at
// c ^ chunk_swizzle(r); a fragment is two transposing reads of 4 rows x 16
// values per 16 lanes. 32 lanes are served at a time: two neighbouring chunks
// of 4 rows in a row, whose 8 places must fall on all banks (c ^ r%4 counted a
// conflict in every second cycle).
__device__ __forceinline__ int spread(int r) { return ((r >> 1) & 3) | (((r >> 4) & 1) << 2); }

// GLU (not COL): of 64 rows (32 where the tile has no more) the first half are
// gate rows of the weights, the others the up rows that belong to them, `far`
// bytes behind.
template <int FMT, bool COL, int B, int NW, bool GLU = false>
struct Operand {
  static constexpr int kBytes = B * kStageBytes;
  static constexpr int kCopies = B / 8 / NW;       // per wave and step
  static constexpr int kRowB = B * 2;              // COL: bytes of a contraction row
  static constexpr int kLanes = COL ? (kRowB / 16) : 8;   // lanes on one row of a copy
  static constexpr int kRows = 64 / kLanes;        // rows of a copy
  __device__ __forceinline__ static int chunk_swizzle(int r) { return B >= 128 ? 2 * (r & 3) : B == 64 ? r & 2 : 0; }
  static constexpr int kTiles = 4;                 // fragments a wave may hold
  static_assert(B / 8 % NW == 0 && kRowB <= 1024, "whole copies");
  static_assert(!GLU || (!COL && (B % 64 == 0 ? NW == 1 || NW == 4 || NW == 8 : B == 32 && NW == 1)),
                "pairs of 32 or 16 rows in whole copies");
  // not COL: spread() of a copy's rows changes with 16 rows, so with the copy where fewer than 4 waves share them
  static constexpr int kVar = COL || NW >= 4 ? 1 : 2;
  static constexpr int variant(int i) { return kVar == 1 ? 0 : NW == 2 ? i & 1 : (i >> 1) & 1; }

  const char* base;
  int64_t ld;
  uint32_t bytes;      // from base to the operand's last byte (COL: of `rows` rows, see copy())
  int rows;            // COL: contraction rows; else: contraction bytes of a row
  int width;           // COL: bytes to the last needed column
  int64_t far;         // GLU
  uint32_t voff[kVar];
  int piece[kVar];     // not COL: where in a step the lane's piece lies
  int rd[4];

  // w0: the wave's first row/column of the tile.
  __device__ __forceinline__ void init(const void* b, int64_t row_bytes, int n, int c_bytes, int wave, int lane,
                                       int w0) {
    base = static_cast<const char*>(b);
    ld = row_bytes;
    const int row = wave * kRows + lane / kLanes, pos = lane % kLanes;
    if constexpr (COL) {
      rows = n;
      width = c_bytes;
      const int g = chunk_swizzle(row);
      voff[0] = (uint32_t)(row * (int)ld + (((pos >> 1) ^ g) * 2 + (pos & 1)) * 16);
      // 16 lanes read values 16 (l/16%2).. of contraction rows 8 (l/32) + l%16/4
      const int j = (lane & 15) >> 2, h = lane >> 5, gr = chunk_swizzle(j);
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
        rd[t] = (8 * h + j) * kRowB + (((w0 / 16 + 2 * t + ((lane >> 4) & 1)) ^ gr) * 32) + (lane & 3) * 8;
    } else {
      bytes = n > 0 ? (uint32_t)((n - 1) * (int)ld + c_bytes) : 0u;
      rows = c_bytes;
#pragma unroll
      for (int v = 0; v < kVar; ++v) {
        piece[v] = (pos ^ spread((row + 16 * v) & 31)) * 16;
        voff[v] = (uint32_t)((GLU ? lane / kLanes : row) * (int)ld + piece[v]);
      }
      // quarter k of a step: pieces 2k and 2k + 1 of the lane's row; MX: k and k + 4, so that the scales of a lane's
      // four pieces are one word
      const int r = lane & 31, h = lane >> 5;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        rd[k] = (w0 + r) * kStageBytes + (((FMT == FMT_MX ? 4 * h + k : 2 * k + h) ^ spread(r)) * 16);
    }
  }

  // Copies [from, to) of this wave's share of step s into `stage`.
  __device__ __forceinline__ void copy(char* stage, int s, int wave, int from, int to) const {
    u32x4_t r, up;
    uint32_t v[kVar], at = 0;
    if constexpr (COL) {
      const int left = min(rows - 64 * s, 64);
      r = rsrc(base + (int64_t)s * 64 * ld, left > 0 ? (uint32_t)((left - 1) * (int)ld + width) : 0u);
      v[0] = voff[0];
    } else {
      r = rsrc(base, bytes);
      if constexpr (GLU) up = rsrc(base + far, bytes);
      at = s * kStageBytes;
#pragma unroll
      for (int k = 0; k < kVar; ++k)   // or the row's contraction ends before this piece
        v[k] = (int)at + piece[k] < rows ? voff[k] : kPastEnd;
    }
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      if (i < from || i >= to) continue;
      if constexpr (GLU) {   // rows 8 (i NW + wave) .. + 7 of the tile
        const int r8 = i * NW + wave;
        const int half = B == 32 ? i >> 1 : NW == 4 ? i & 1 : NW == 8 ? wave >> 2 : (i >> 2) & 1;
        const int row = B == 32 ? (i & 1) * 8 : (r8 >> 3) * 32 + (r8 & 3) * 8;
        copy16(stage + r8 * 1024, half ? up : r, v[variant(i)], row * (int)ld + at);
      } else {
        copy16(stage + (i * NW + wave) * 1024, r, v[variant(i)], i * NW * kRows * (int)ld + at);
      }
    }
  }

  // Fragment t (32 rows/columns from w0 + 32 t) of quarter k of a step.
  __device__ __forceinline__ u32x4_t frag(const char* stage, int t, int k) const {
    if constexpr (COL) {
      const lds_char_t* at = (const lds_char_t*)(stage + rd[t] + k * 16 * kRowB);
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)at);
      const s16x4_t hi =
          __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(at + 4 * kRowB));
      const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, hi);
      return u32x4_t{a[0], a[1], b[0], b[1]};
    } else {
      return *reinterpret_cast<const u32x4_t*>(stage + rd[k] + t * 32 * kStageBytes);
    }
  }
};

// The operands of the tile at (i0, j0) of expert e; wi0, wj0: the wave's part of it.
template <int FMT, bool PC, bool QC, class OpP, class OpQ>
__device__ __forceinline__ void init_operands(OpP& P, OpQ& Q, const RaggedParams& p, int e, const Group& g, int i0,
                                              int j0, int ni, int nj, int C, int wave, int lane, int wi0, int wj0) {
  const char* pb = static_cast<const char*>(p.p);
  const char* qb = static_cast<const char*>(p.q);
  const int cb = C / 8 * (FMT == FMT_MX ? 4 : 16);   // contraction bytes of a row (C a multiple of 8 there)
  if constexpr (QC) {
    P.init(pb + (int64_t)g.lo * p.p_ld + (int64_t)i0 * 2, p.p_ld, C, ni * 2, wave, lane, wi0);
    Q.init(qb + (int64_t)g.lo * p.q_ld + (int64_t)j0 * 2, p.q_ld, C, nj * 2, wave, lane, wj0);
  } else {
    const char* we = pb + (int64_t)e * p.p_stride;
    if constexpr (PC) P.init(we + (int64_t)i0 * 2, p.p_ld, C, ni * 2, wave, lane, wi0);
    else P.init(we + (int64_t)i0 * p.p_ld, p.p_ld, ni, cb, wave, lane, wi0);
    Q.init(qb + (int64_t)(g.lo + j0) * p.q_ld, p.q_ld, nj, cb, wave, lane, wj0);
  }
}

// Four values rounded to TYPE.
template <int TYPE>
__device__ __forceinline__ auto pack4(float a, float b, float c, float d) {
  if constexpr (TYPE == TYPE_F32) {
    return f32x4_t{a, b, c, d};
  } else if constexpr (TYPE == TYPE_F16) {
    const f16x4_t h = {(_Float16)a, (_Float16)b, (_Float16)c, (_Float16)d};
    return __builtin_bit_cast(u32x2_t, h);
  } else {
    return u32x2_t{pack_bf16x2(a, b), pack_bf16x2(c, d)};
  }
}

__device__ __forceinline__ void store4(void* out, int64_t at, int type, f32x4_t v) {
  if (type == TYPE_BF16)
    *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(out) + at) = pack4<TYPE_BF16>(v[0], v[1], v[2], v[3]);
  else if (type == TYPE_F16)
    *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(out) + at) = pack4<TYPE_F16>(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(out) + at) = v;
}

// What happens to a product's sums: nothing, a bias and a residual, or with GLU
// a bias, SwiGLU of the pairs of columns that a tile's rows of weights make, and
// a residual.
enum Epi : int { EPI_NONE = 0, EPI_ADD = 1, EPI_GLU = 2 };

__device__ __forceinline__ f32x4_t load4(const void* x, int64_t at, int type) {
  if (type == TYPE_F32) return *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(x) + at);
  const u32x2_t w = *reinterpret_cast<const u32x2_t*>(static_cast<const uint16_t*>(x) + at);
  if (type == TYPE_BF16) return f32x4_t{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
  const f16x4_t h = __builtin_bit_cast(f16x4_t, w);
  return f32x4_t{(float)h[0], (float)h[1], (float)h[2], (float)h[3]};
}

// Four biases of expert e.
__device__ __forceinline__ f32x4_t bias4(const Epilogue& x, int e, int col) {
  return load4(x.bias, (int64_t)e * x.bias_ld + col, x.bias_type);
}

// 16 bytes of a row of the residual, added to v.
template <int TYPE>
__device__ __forceinline__ void add_residual(const u32x4_t& w, float* v) {
  if constexpr (TYPE == TYPE_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += __uint_as_float(w[i]);
  } else {
    const f16x8_t h = __builtin_bit_cast(f16x8_t, w);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] += TYPE == TYPE_F16 ? (float)h[i] : i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
  }
}

// Everything of one output tile. BJ may be less than the workgroup's largest
// tile: a group's last rows.
// ONE: a single LDS stage, no overlap within a workgroup (four of them share a
// CU): for contractions of about a step.
template <int FMT, bool PC, bool QC, int BI, int BJ, int WI, int WJ, bool ONE, int EPI = EPI_NONE>
struct TileBody {
  static constexpr int NW = WI * WJ, TI = BI / WI / 32, TJ = BJ / WJ / 32;
  static constexpr bool MX = FMT == FMT_MX, GLU = EPI == EPI_GLU;
  static constexpr int kVal = MX ? 256 : 64;     // contraction values per step
  static constexpr int BO = GLU ? BI / 2 : BI;   // output columns
  static constexpr int TO = GLU ? TI / 2 : TI;   // tiles of 32 of them that a wave holds, after the epilogue
  static_assert(!GLU || TI == 2, "a wave holds 32 gate rows and the 32 up rows that belong to them");
  using OpP = Operand<FMT, PC, BI, NW, GLU>;
  using OpQ = Operand<FMT, QC, BJ, NW>;
  OpP P;
  OpQ Q;
  f32x16_t acc[TI][TJ];
  int wave, lane, wi, wj;
  int blocks;                       // MX: scale blocks of a row
  u32x4_t prs, qrs;                 // MX scales
  int s_ld;

  // LDS stages of P and of Q: for 8 waves what fits in 160 KB (MX: with two of scales), for 4 two of each, so that two
  // workgroups share a CU
  static constexpr int kPS = ONE ? 1 : NW == 4 ? 2 : MX ? (BJ > 192 ? 2 : 3) : BJ > 64 ? 3 : 4;
  static constexpr int kQS = ONE ? 1 : NW == 4 || BJ > 128 ? 2 : MX || BJ > 64 ? 3 : 4;
  // a pair of steps' scales, 16 bytes a row of P and of Q: copied 64 rows at a time, so Q's 32 rows have room for 64
  static constexpr int kScaleQ = (BJ + 63) / 64;   // copies
  static constexpr int kPB = BI * kStageBytes, kQB = BJ * kStageBytes, kSB = MX ? BI * 16 + kScaleQ * 1024 : 0;
  static_assert(!MX || BI % 64 == 0, "whole copies of P's scales");
  static constexpr int kPC = OpP::kCopies, kQC = OpQ::kCopies;
  static constexpr int kTurn = NW * 32 * (BI / WI * 4 + 16);   // what store() needs for FP32
  static constexpr int kRings = kPS * kPB + kQS * kQB + 2 * kSB, kLds = kRings > kTurn ? kRings : kTurn;
  static_assert(kLds <= 160 * 1024 && kPS >= kQS, "LDS");

  char* lds;
  __device__ __forceinline__ char* p_stage(int s) const { return lds + s % kPS * kPB; }
  __device__ __forceinline__ char* q_stage(int s) const { return lds + kPS * kPB + s % kQS * kQB; }
  __device__ __forceinline__ char* scales(int s) const {
    return lds + kPS * kPB + kQS * kQB + ((s >> 1) & 1) * kSB;
  }

  // MX: the scales of steps s and s + 1, s even.
  __device__ __forceinline__ void issue_scales(int s) const {
    char* ss = scales(s);
#pragma unroll
    for (int n = 0; n < BI / 64; n += NW)
      if (n + wave < BI / 64) copy16(ss + (n + wave) * 1024, prs, ((n + wave) * 64 + lane) * s_ld, s * 8);
#pragma unroll
    for (int n = 0; n < kScaleQ; n += NW)
      if (n + wave < kScaleQ)
        copy16(ss + BI * 16 + (n + wave) * 1024, qrs, ((n + wave) * 64 + lane) * s_ld, s * 8);
  }

  // MX: a lane's four scale bytes of step s (its blocks 4h .. 4h + 3) in tile t of P, u of Q.
  __device__ __forceinline__ int scale(int s, int row) const {
    return *reinterpret_cast<const int*>(scales(s) + (row + (lane & 31)) * 16 + (s & 1) * 8 + (lane >> 5) * 4);
  }
  __device__ __forceinline__ int scale_p(int s, int t) const { return scale(s, wi * (BI / WI) + 32 * t); }
  __device__ __forceinline__ int scale_q(int s, int u) const { return scale(s, BI + wj * (BJ / WJ) + 32 * u); }

  struct Frags {
    u32x4_t p[TI], q[TJ];
  };
  struct Scales {
    int p[TI], q[TJ];
  };

  // Quarter k of a step (stages ps, qs).
  __device__ __forceinline__ void load(Frags& f, const char* ps, const char* qs, int k) const {
#pragma unroll
    for (int t = 0; t < TI; ++t) f.p[t] = P.frag(ps, t, k);
#pragma unroll
    for (int u = 0; u < TJ; ++u) f.q[u] = Q.frag(qs, u, k);
  }
  __device__ __forceinline__ void load_scales(Scales& c, int s) const {
#pragma unroll
    for (int t = 0; t < TI; ++t) c.p[t] = scale_p(s, t);
#pragma unroll
    for (int u = 0; u < TJ; ++u) c.q[u] = scale_q(s, u);
  }

  // Scales past the row's last block may hold anything: 2^0 there.
  __device__ __forceinline__ void cut_scales(Scales& c, int s) const {
    const int left = blocks - 8 * s - 4 * (lane >> 5);
    const uint32_t keep = left >= 4 ? 0xFFFFFFFFu : left > 0 ? (1u << (8 * left)) - 1u : 0u;
#pragma unroll
    for (int t = 0; t < TI; ++t) c.p[t] = (c.p[t] & keep) | (0x7F7F7F7Fu & ~keep);
#pragma unroll
    for (int u = 0; u < TJ; ++u) c.q[u] = (c.q[u] & keep) | (0x7F7F7F7Fu & ~keep);
  }

  // Column u of quarter K.
  template <int K>
  __device__ __forceinline__ void mul(const Frags& f, const Scales& c, int u) {
#pragma unroll
    for (int t = 0; t < TI; ++t) {
      acc[t][u] = mma<FMT, K>(f.p[t], f.q[u], acc[t][u], c.p[t], c.q[u]);
      // the compiler would move the scaled products past the branches behind them, and spill their operands
      if constexpr (MX) asm volatile("" : "+v"(acc[t][u]));
    }
  }

  __device__ __forceinline__ void init(const RaggedParams& p, int e, const Group& g, int i0, int j0, int ni, int nj,
                                       int C) {
    lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wi = wave / WJ, wj = wave % WJ;
    init_operands<FMT, PC, QC>(P, Q, p, e, g, i0, j0, ni, nj, C, wave, lane, wi * (BI / WI), wj * (BJ / WJ));
    if constexpr (GLU) P.far = (int64_t)p.I * p.p_ld;
    if constexpr (MX) {
      s_ld = (int)p.s_ld;
      blocks = C / 32;
      prs = rsrc(p.ps + (int64_t)e * p.ps_stride + (int64_t)i0 * s_ld, (uint32_t)(ni * s_ld));
      qrs = rsrc(p.qs + (int64_t)(g.lo + j0) * s_ld, (uint32_t)(nj * s_ld));
    }
#pragma unroll
    for (int t = 0; t < TI; ++t)
#pragma unroll
      for (int u = 0; u < TJ; ++u) acc[t][u] = f32x16_t{};
  }

  // The refills of step s's stages behind its barrier, Q of step s + kQS, then
  // P of step s + kPS: copy number c of them.
  template <bool ALL>
  __device__ __forceinline__ void refill(int s, int c, int steps) const {
    if (c < kQC) {
      if (ALL || s + kQS < steps) Q.copy(q_stage(s), s + kQS, wave, c, c + 1);
    } else if (c < kQC + kPC) {
      if (ALL || s + kPS < steps) P.copy(p_stage(s), s + kPS, wave, c - kQC, c - kQC + 1);
    }
  }

  // The contraction. P and Q pass through rings of LDS stages of one step
  // each; the fragments of a quarter step are read while the quarter before it
  // is multiplied. In quarter 3, behind its first columns, comes the one
  // barrier of a step: every wave's reads of the step's stages are done, and
  // step s + 1 has landed. The copies that refill the stages follow one by one
  // between the columns, up to the next step's quarter 2: side by side they
  // would hold up the products behind them.
  // The scheduling barriers keep the order as written.
  //   MODE 0: all refills are within the contraction, 1: some may not be (or s
  //   is 0), 2: the last step
  template <int MODE>
  __device__ __forceinline__ void step(Frags& f, Frags& g, Scales& c, Scales& n, int s, int steps) {
    constexpr int kHead = 1;                                                // columns ahead of the barrier
    constexpr int kGap = (kQC + kPC + 4 * TJ - kHead - 1) / (4 * TJ - kHead);   // copies per column
    const char* ph = p_stage(s);
    const char* qh = q_stage(s);
    if constexpr (MX && MODE == 2) cut_scales(c, s);
    auto column = [&](auto k, Frags& x, int u) {
      constexpr int K = decltype(k)::value;
      mul<K>(x, c, u);
      if constexpr (MODE != 2) {
        const int at = (K == 3 ? u - kHead : TJ - kHead + K * TJ + u) * kGap;   // the column's place behind a barrier
#pragma unroll
        for (int i = 0; i < kGap; ++i) {
          if (K == 3) refill<MODE == 0>(s, at + i, steps);
          else if (MODE == 0 || s > 0) refill<MODE == 0>(s - 1, at + i, steps);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    load(g, ph, qh, 1);
#pragma unroll
    for (int u = 0; u < TJ; ++u) column(std::integral_constant<int, 0>{}, f, u);
    load(f, ph, qh, 2);
#pragma unroll
    for (int u = 0; u < TJ; ++u) column(std::integral_constant<int, 1>{}, g, u);
    load(g, ph, qh, 3);
#pragma unroll
    for (int u = 0; u < TJ; ++u) column(std::integral_constant<int, 2>{}, f, u);
#pragma unroll
    for (int u = 0; u < kHead; ++u) {
      mul<3>(g, c, u);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (MODE != 2) {
      // the copies behind those of step s + 1 may still be on their way
      if (MODE == 0 || s - 1 + kPS < steps) fence<(kQS - 2) * (kPC + kQC) + (kPS > kQS ? kPC : 0)>();
      else fence<0>();
      if constexpr (MX) {
        load_scales(n, s + 1);
        if (((s + kQS) & 1) == 0 && s + kQS < steps) issue_scales(s + kQS);
      }
      load(f, p_stage(s + 1), q_stage(s + 1), 0);
    }
#pragma unroll
    for (int u = kHead; u < TJ; ++u) column(std::integral_constant<int, 3>{}, g, u);
    if constexpr (MX && MODE != 2) c = n;
  }

  __device__ __forceinline__ void contract_one(int steps) {
    Frags f, g;
    Scales c;
    settle();
    for (int s = 0; s < steps; ++s) {
      if (s > 0) fence<0>();   // every wave's reads of step s - 1 are done
      if constexpr (MX)
        if ((s & 1) == 0) issue_scales(s);
      P.copy(p_stage(s), s, wave, 0, kPC);
      Q.copy(q_stage(s), s, wave, 0, kQC);
      fence<0>();
      load(f, p_stage(s), q_stage(s), 0);
      if constexpr (MX) {
        load_scales(c, s);
        if (s + 1 == steps) cut_scales(c, s);
      }
      load(g, p_stage(s), q_stage(s), 1);
#pragma unroll
      for (int u = 0; u < TJ; ++u) mul<0>(f, c, u);
      load(f, p_stage(s), q_stage(s), 2);
#pragma unroll
      for (int u = 0; u < TJ; ++u) mul<1>(g, c, u);
      load(g, p_stage(s), q_stage(s), 3);
#pragma unroll
      for (int u = 0; u < TJ; ++u) mul<2>(f, c, u);
#pragma unroll
      for (int u = 0; u < TJ; ++u) mul<3>(g, c, u);
    }
  }

  __device__ __forceinline__ void contract(int steps) {
    if (steps <= 0) return;
    Frags f, g;
    Scales c, n;   // MX: of this step and the next
    settle();
#pragma unroll
    for (int s = 0; s < kPS; ++s) {
      if constexpr (MX)
        if ((s & 1) == 0 && s < kQS && s < steps) issue_scales(s);
      if (s < steps) P.copy(p_stage(s), s, wave, 0, kPC);
      if (s < kQS && s < steps) Q.copy(q_stage(s), s, wave, 0, kQC);
    }
    if (!MX && steps >= kPS) fence<(kPS - 1) * kPC + (kQS - 1) * kQC>();
    else fence<0>();
    load(f, p_stage(0), q_stage(0), 0);
    if constexpr (MX) load_scales(c, 0);
    int s = 0;
    if (steps > 1) step<1>(f, g, c, n, s++, steps);
    for (; s + kPS < steps; ++s) step<0>(f, g, c, n, s, steps);
    for (; s + 1 < steps; ++s) step<1>(f, g, c, n, s, steps);
    step<2>(f, g, c, n, s, steps);
  }

  // The tile's rows to global memory, turned in LDS: a lane holds 4 adjacent
  // values of a row, whole 128-byte lines (16 bytes a lane) go out. In pieces
  // of 8 bytes the same stores cost 2.4 times as long (weight gradients of 48
  // experts, 2.8 GB: 885 us of the call).
  // Each wave turns 32 rows at a time in LDS of its own.
  // PAST: past the caches (see launch()).
  template <int TYPE, bool PAST>
  __device__ __forceinline__ void store_as(const RaggedParams& p, int64_t base, int64_t row0, int i0, int ni, int nj) {
    constexpr int kW = BO / WI, kSize = TYPE == TYPE_F32 ? 4 : 2;   // columns of a wave
    constexpr int kRow = kW * kSize, kPitch = kRow + 16;            // 16 bytes more: rows on other banks
    constexpr int kLanes = kRow / 16, kRows = 64 / kLanes;          // lanes on a row, rows of a store
    static_assert(NW * 32 * kPitch <= kLds, "LDS");
    char* buf = lds + wave * 32 * kPitch;
    const int col = wi * kW + (lane % kLanes) * (16 / kSize);
#pragma unroll
    for (int u = 0; u < TJ; ++u) {
#pragma unroll
      for (int t = 0; t < TO; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f32x16_t& v = acc[t][u];
          const auto w = pack4<TYPE>(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          __builtin_memcpy(__builtin_assume_aligned(
                               buf + (lane & 31) * kPitch + (32 * t + 8 * k + 4 * (lane >> 5)) * kSize, 4 * kSize),
                           &w, sizeof w);
        }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int r = 0; r < 32; r += kRows) {
        const int j = r + lane / kLanes, jj = wj * (BJ / WJ) + 32 * u + j;
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(buf + j * kPitch + (lane % kLanes) * 16);
        if (jj < nj && col < ni) {
          u32x4_t* at = reinterpret_cast<u32x4_t*>(static_cast<char*>(p.out) +
                                                   (base + (row0 + jj) * p.out_ld + i0 + col) * kSize);
          if constexpr (PAST) __builtin_nontemporal_store(w, at);
          else *at = w;
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  }

  // The same with a residual: turned in FP32, 16 bytes of the output a lane. The
  // residual of 32 rows is read before they are turned.
  template <int TYPE, bool PAST>
  __device__ __forceinline__ void store_onto(const RaggedParams& p, int64_t row0, int i0, int ni, int nj) {
    constexpr int kW = BO / WI, kSize = TYPE == TYPE_F32 ? 4 : 2, kV = 16 / kSize;
    constexpr int kPitch = kW * 4 + 16;
    constexpr int kLanes = kW / kV, kRows = 64 / kLanes;
    static_assert(NW * 32 * kPitch <= kLds, "LDS");
    char* buf = lds + wave * 32 * kPitch;
    const int col = wi * kW + (lane % kLanes) * kV;
#pragma unroll
    for (int u = 0; u < TJ; ++u) {
      u32x4_t res[32 / kRows];
#pragma unroll
      for (int r = 0; r < 32; r += kRows) {
        const int jj = wj * (BJ / WJ) + 32 * u + r + lane / kLanes;
        const u32x4_t* at = reinterpret_cast<const u32x4_t*>(static_cast<const char*>(p.epi.res) +
                                                             ((row0 + jj) * p.epi.res_ld + i0 + col) * kSize);
        res[r / kRows] = u32x4_t{};
        if (jj < nj && col < ni) res[r / kRows] = PAST ? __builtin_nontemporal_load(at) : *at;
      }
#pragma unroll
      for (int t = 0; t < TO; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f32x16_t& v = acc[t][u];
          *reinterpret_cast<f32x4_t*>(buf + (lane & 31) * kPitch + (32 * t + 8 * k + 4 * (lane >> 5)) * 4) =
              f32x4_t{v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]};
        }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int r = 0; r < 32; r += kRows) {
        const int j = r + lane / kLanes, jj = wj * (BJ / WJ) + 32 * u + j;
        float v[kV];
        const f32x4_t* from = reinterpret_cast<const f32x4_t*>(buf + j * kPitch + (lane % kLanes) * kV * 4);
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = from[i / 4][i % 4];
        add_residual<TYPE>(res[r / kRows], v);
        u32x4_t w;
        if constexpr (TYPE == TYPE_F32) {
          w = __builtin_bit_cast(u32x4_t, f32x4_t{v[0], v[1], v[2], v[3]});
        } else {
          const u32x2_t lo = pack4<TYPE>(v[0], v[1], v[2], v[3]), hi = pack4<TYPE>(v[4], v[5], v[6], v[7]);
          w = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
        }
        if (jj < nj && col < ni) {
          u32x4_t* at = reinterpret_cast<u32x4_t*>(static_cast<char*>(p.out) +
                                                   ((row0 + jj) * p.out_ld + i0 + col) * kSize);
          if constexpr (PAST) __builtin_nontemporal_store(w, at);
          else *at = w;
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  }

  // The bias, and with GLU silu(gate) * up in the gate's place.
  __device__ __forceinline__ void epilogue(const Epilogue& x, int e, int i0, int ni, int I) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = wi * (BO / WI) + 8 * k + 4 * (lane >> 5);
      f32x4_t b[TI];
#pragma unroll
      for (int t = 0; t < TI; ++t) {
        const int col = GLU ? c : c + 32 * t;
        b[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if (x.bias && col < ni) b[t] = bias4(x, e, i0 + col + (GLU ? t * I : 0));
      }
#pragma unroll
      for (int u = 0; u < TJ; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int t = 0; t < TI; ++t) acc[t][u][4 * k + i] += b[t][i];
          if constexpr (GLU) acc[0][u][4 * k + i] = swiglu(acc[0][u][4 * k + i], acc[TI - 1][u][4 * k + i]);
        }
    }
  }

  __device__ __forceinline__ void store(const RaggedParams& p, int64_t base, int64_t row0, int i0, int ni, int nj) {
    fence<0>();   // every wave is past its last fragments
    if constexpr (EPI != EPI_NONE) {
      if (p.epi.res) {
        if (p.stream_out) onto_any<true>(p, row0, i0, ni, nj);
        else onto_any<false>(p, row0, i0, ni, nj);
        return;
      }
    }
    if (p.stream_out) store_any<true>(p, base, row0, i0, ni, nj);
    else store_any<false>(p, base, row0, i0, ni, nj);
  }

  template <bool PAST>
  __device__ __forceinline__ void onto_any(const RaggedParams& p, int64_t row0, int i0, int ni, int nj) {
    if (p.out_type == TYPE_BF16) store_onto<TYPE_BF16, PAST>(p, row0, i0, ni, nj);
    else if (p.out_type == TYPE_F16) store_onto<TYPE_F16, PAST>(p, row0, i0, ni, nj);
    else store_onto<TYPE_F32, PAST>(p, row0, i0, ni, nj);
  }

  template <bool PAST>
  __device__ __forceinline__ void store_any(const RaggedParams& p, int64_t base, int64_t row0, int i0, int ni, int nj) {
    if (p.out_type == TYPE_BF16) store_as<TYPE_BF16, PAST>(p, base, row0, i0, ni, nj);
    else if (p.out_type == TYPE_F16) store_as<TYPE_F16, PAST>(p, base, row0, i0, ni, nj);
    else store_as<TYPE_F32, PAST>(p, base, row0, i0, ni, nj);
  }

  __device__ __forceinline__ static void run(const RaggedParams& p, int e, const Group& g, int i0, int j0, int ni,
                                             int nj, char* lds) {
    TileBody b;
    b.lds = lds;
    const int C = QC ? g.n : p.C;
    b.init(p, e, g, i0, j0, ni, nj, C);
    if constexpr (ONE) b.contract_one((C + kVal - 1) / kVal);
    else b.contract((C + kVal - 1) / kVal);
    if constexpr (EPI != EPI_NONE) b.epilogue(p.epi, e, i0, ni, p.I);
    b.store(p, QC ? (int64_t)e * p.out_stride : 0, QC ? (int64_t)j0 : (int64_t)(g.lo + j0), i0, ni, nj);
  }
};

// One BI x BJ output tile per workgroup of WI x WJ waves.
template <int FMT, bool PC, bool QC, int BI, int BJ, int WI, int WJ, bool ONE, int EPI = EPI_NONE>
__global__ __launch_bounds__(64 * WI * WJ)
__attribute__((amdgpu_waves_per_eu(ONE ? 4 : 2, ONE ? 4 : 2))) void ragged_gemm(RaggedParams p) {
  constexpr bool kLarge = BJ == 256, kThree = kLarge && !QC;   // (otherwise no whole copies, or no whole fragments)
  using B4 = TileBody<FMT, PC, QC, BI, BJ, WI, WJ, ONE, EPI>;
  using B3 = TileBody<FMT, PC, QC, BI, kThree ? BJ / 4 * 3 : BJ, WI, WJ, ONE, EPI>;
  using B2 = TileBody<FMT, PC, QC, BI, BJ / 2, WI, WJ, ONE, EPI>;
  // (a quarter of 128 rows would leave a wave 32 columns, which are no gate | up pairs)
  using B1 = std::conditional_t<EPI == EPI_GLU && !kLarge, B2,
                                TileBody<FMT, PC, QC, BI, BJ / 4, kLarge ? WI : WI * 2, kLarge ? WJ : WJ / 2, ONE, EPI>>;
  constexpr int BO = B4::BO;
  constexpr auto most = [](int a, int b) { return a > b ? a : b; };
  __shared__ __align__(1024) char lds[most(most(B4::kLds, B3::kLds), most(B2::kLds, B1::kLds))];
  const int b = (int)(p.first + blockIdx.x);
  const Found f = QC ? even_tile(p, b, BJ, BO, 1) : find_tile(p, b, BJ, (p.I + BO - 1) / BO, 1);
  const Tile t = f.t;
  const Group g = f.g;
  if (t.e < 0) return;
  const int e = t.e;
  const int i0 = t.it * BO, j0 = t.jt * BJ;
  const int ni = min(p.I - i0, BO), nj = min((QC ? p.J : g.n) - j0, BJ);
  if (i0 < 0 || j0 < 0 || ni <= 0 || nj <= 0) return;   // sums of offsets that decrease may wrap
  // a group's last rows take a tile of fewer rows: less to multiply, more stages in flight
  if (nj > (kThree ? BJ / 4 * 3 : BJ / 2)) B4::run(p, e, g, i0, j0, ni, nj, lds);
  else if (kThree && nj > BJ / 2) B3::run(p, e, g, i0, j0, ni, nj, lds);
  else if (nj > BJ / 4) B2::run(p, e, g, i0, j0, ni, nj, lds);
  else B1::run(p, e, g, i0, j0, ni, nj, lds);
}

// One BI x BJ tile of W waves that share its contraction: wave w takes steps w,
// w + W, .. on stages of its own, without a barrier, and the W FP32 sums are
// added in wave order through LDS. For calls of few tiles, where a tile's chain
// of steps is the time: BI = 64 with 4 waves, or 32 with 6 (FP4 5), which LDS
// has room for.
template <int FMT, int BI>
constexpr int kSplitWaves = split_waves(FMT == FMT_MX, BI);

template <int FMT, bool PC, bool QC, int BI, int BJ, int EPI = EPI_NONE>
struct SplitBody {
  static constexpr int W = kSplitWaves<FMT, BI>, TI = BI / 32, TJ = BJ / 32;
  static constexpr bool MX = FMT == FMT_MX, GLU = EPI == EPI_GLU;
  static constexpr int kVal = MX ? 256 : 64;
  static constexpr int BO = GLU ? BI / 2 : BI;                     // output columns
  using OpP = Operand<FMT, PC, BI, 1, GLU>;
  using OpQ = Operand<FMT, QC, BJ, 1>;
  static constexpr int kSB = MX ? 2048 : 0;                        // 16 scales of up to 64 rows of each operand
  static constexpr int kStage = (BI + BJ) * kStageBytes + kSB;
  static constexpr int kCopies = OpP::kCopies + OpQ::kCopies + (MX ? 2 : 0);
  static constexpr int kPitch = BI * 4 + 16, kSum = BJ * kPitch;   // a wave's sums
  static constexpr int kLds = W * (2 * kStage > kSum ? 2 * kStage : kSum);
  static_assert(kLds <= 160 * 1024, "LDS");
  static_assert(BI <= 64 && BJ <= 64, "one copy of scales of each operand");

  __device__ __forceinline__ static void run(const RaggedParams& p, int e, const Group& g, int i0, int j0, int ni,
                                             int nj, char* all) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    char* lds = all + wave * (kLds / W);
    const int C = QC ? g.n : p.C, steps = (C + kVal - 1) / kVal, blocks = C / 32;
    const int mine = steps > wave ? (steps - wave + W - 1) / W : 0;
    OpP P;
    OpQ Q;
    init_operands<FMT, PC, QC>(P, Q, p, e, g, i0, j0, ni, nj, C, 0, lane, 0, 0);
    if constexpr (GLU) P.far = (int64_t)p.I * p.p_ld;
    u32x4_t prs, qrs;
    if constexpr (MX) {
      prs = rsrc(p.ps + (int64_t)e * p.ps_stride + (int64_t)i0 * p.s_ld, (uint32_t)(ni * (int)p.s_ld));
      qrs = rsrc(p.qs + (int64_t)(g.lo + j0) * p.s_ld, (uint32_t)(nj * (int)p.s_ld));
    }
    auto issue = [&](int k) {
      char* st = lds + (k & 1) * kStage;
      const int s = k * W + wave;
      P.copy(st, s, 0, 0, OpP::kCopies);
      Q.copy(st + OpP::kBytes, s, 0, 0, OpQ::kCopies);
      if constexpr (MX) {
        char* ss = st + OpP::kBytes + OpQ::kBytes;
        copy16(ss, prs, lane * (int)p.s_ld, (s & ~1) * 8);
        copy16(ss + 1024, qrs, lane * (int)p.s_ld, (s & ~1) * 8);
      }
    };
    f32x16_t acc[TI][TJ];
#pragma unroll
    for (int t = 0; t < TI; ++t)
#pragma unroll
      for (int u = 0; u < TJ; ++u) acc[t][u] = f32x16_t{};
    settle();
    if (mine > 0) issue(0);
    if (mine > 1) issue(1);
    for (int k = 0; k < mine; ++k) {
      if (k + 1 < mine) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kCopies) : "memory");
      else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      const char* st = lds + (k & 1) * kStage;
      const int s = k * W + wave;
      int sp[TI] = {}, sq[TJ] = {};
      if constexpr (MX) {
        const char* ss = st + OpP::kBytes + OpQ::kBytes + (lane & 31) * 16 + (s & 1) * 8 + (lane >> 5) * 4;
        // scales past the row's last block may hold anything: 2^0 there
        const int left = blocks - 8 * s - 4 * (lane >> 5);
        const uint32_t keep = left >= 4 ? 0xFFFFFFFFu : left > 0 ? (1u << (8 * left)) - 1u : 0u;
        auto get = [&](int row) {
          return (int)((*reinterpret_cast<const uint32_t*>(ss + row * 16) & keep) | (0x7F7F7F7Fu & ~keep));
        };
#pragma unroll
        for (int t = 0; t < TI; ++t) sp[t] = get(32 * t);
#pragma unroll
        for (int u = 0; u < TJ; ++u) sq[u] = get(64 + 32 * u);
      }
      auto quarter = [&](auto kk) {
        constexpr int K = decltype(kk)::value;
        u32x4_t pf[TI], qf[TJ];
#pragma unroll
        for (int t = 0; t < TI; ++t) pf[t] = P.frag(st, t, K);
#pragma unroll
        for (int u = 0; u < TJ; ++u) qf[u] = Q.frag(st + OpP::kBytes, u, K);
#pragma unroll
        for (int t = 0; t < TI; ++t)
#pragma unroll
          for (int u = 0; u < TJ; ++u) acc[t][u] = mma<FMT, K>(pf[t], qf[u], acc[t][u], sp[t], sq[u]);
      };
      quarter(std::integral_constant<int, 0>{});
      quarter(std::integral_constant<int, 1>{});
      quarter(std::integral_constant<int, 2>{});
      quarter(std::integral_constant<int, 3>{});
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the stage is read
      if (k + 2 < mine) issue(k + 2);
    }
    // the sums as rows j of BI values i
#pragma unroll
    for (int u = 0; u < TJ; ++u)
#pragma unroll
      for (int t = 0; t < TI; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f32x16_t& v = acc[t][u];
          *reinterpret_cast<f32x4_t*>(lds + (32 * u + (lane & 31)) * kPitch + (32 * t + 8 * k + 4 * (lane >> 5)) * 4) =
              f32x4_t{v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]};
        }
    __syncthreads();
    const int64_t at = QC ? (int64_t)e * p.out_stride + (int64_t)j0 * p.out_ld : (int64_t)(g.lo + j0) * p.out_ld;
    const int i = (int)threadIdx.x % (BO / 4) * 4;
    f32x4_t bias[GLU ? 2 : 1] = {};
    if constexpr (EPI != EPI_NONE) {
      if (p.epi.bias && i < ni) {
        bias[0] = bias4(p.epi, e, i0 + i);
        if constexpr (GLU) bias[1] = bias4(p.epi, e, p.I + i0 + i);
      }
    }
    for (int j = (int)threadIdx.x / (BO / 4); j < BJ; j += 64 * W / (BO / 4)) {
      f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < W; ++w) v += *reinterpret_cast<const f32x4_t*>(all + w * (kLds / W) + j * kPitch + i * 4);
      if constexpr (EPI != EPI_NONE) v += bias[0];
      if constexpr (GLU) {
        f32x4_t up = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < W; ++w)
          up += *reinterpret_cast<const f32x4_t*>(all + w * (kLds / W) + j * kPitch + (BI / 2 + i) * 4);
        up += bias[1];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = swiglu(v[k], up[k]);
      }
      if (j < nj && i < ni) {
        if constexpr (EPI != EPI_NONE)
          if (p.epi.res) v += load4(p.epi.res, (int64_t)(g.lo + j0 + j) * p.epi.res_ld + i0 + i, p.out_type);
        store4(p.out, at + (int64_t)j * p.out_ld + i0 + i, p.out_type, v);
      }
    }
  }
};

template <int FMT, bool PC, bool QC, int BI, int EPI = EPI_NONE>
__global__ __launch_bounds__((64 * kSplitWaves<FMT, BI>)) void ragged_split(RaggedParams p) {
  using Wide = SplitBody<FMT, PC, QC, BI, 64, EPI>;
  using Narrow = SplitBody<FMT, PC, QC, BI, 32, EPI>;
  constexpr int BO = Wide::BO;
  __shared__ __align__(1024) char lds[Wide::kLds > Narrow::kLds ? Wide::kLds : Narrow::kLds];
  // two tiles that read the halves of the same lines on one XCD (1 expert, 64 rows, 7168 by 1024: 14.7 against 25.7 us)
  constexpr int kLeast = PC && BI == 32 ? 2 : 1;
  const int b = (int)(p.first + blockIdx.x);
  const Found f = QC ? even_tile(p, b, 64, BO, kLeast) : find_tile(p, b, 64, (p.I + BO - 1) / BO, kLeast);
  const Tile t = f.t;
  const Group g = f.g;
  if (t.e < 0) return;
  const int i0 = t.it * BO, j0 = t.jt * 64;
  const int ni = min(p.I - i0, BO), nj = min((QC ? p.J : g.n) - j0, 64);
  if (i0 < 0 || j0 < 0 || ni <= 0 || nj <= 0) return;   // as above
  if (nj > 32) Wide::run(p, t.e, g, i0, j0, ni, nj, lds);
  else Narrow::run(p, t.e, g, i0, j0, ni, nj, lds);
}

// Tiles of BI x B: at most, where groups are ragged.
template <bool QC>
int64_t tile_bound(const RaggedParams& p, int BI, int B) {
  const int64_t NI = (p.I + BI - 1) / BI, live = p.E < p.M ? p.E : p.M;   // experts that can hold rows
  return QC ? p.E * NI * ((p.J + B - 1) / B) : NI * ((p.M + live * (B - 1)) / B);
}

template <int FMT, bool PC, bool QC, int EPI = EPI_NONE>
hipError_t launch(RaggedParams p, hipStream_t s) {
  constexpr bool GLU = EPI == EPI_GLU;
  if (!QC && p.M == 0) return hipSuccess;
  const int64_t size = p.out_type == TYPE_F32 ? 4 : 2;
  const FormCall call{FMT == FMT_MX, QC, p.E, p.M, GLU ? 2 * p.I : p.I, p.J, p.C, (int)size};
  const Form f = EPI != EPI_NONE ? form_of_linear(call) : form_of(call);
  const int64_t bytes = (QC ? (int64_t)p.E * p.J : p.M) * p.I * size;
  // Whole lines that the L2s (32 MB) cannot hold leave them to the operands when they pass them by: FP4, 8 experts of
  // 2048 rows 230 against 252 us. FOUR's calls are bound by such writes, and up to 256 MB the last-level cache takes
  // them sooner: 21 against 27 us for 141 MB. Rows that begin inside a line need the caches to put lines together
  // (24 against 70 us).
  p.stream_out = p.out_ld * size % 128 == 0 && (uintptr_t)p.out % 128 == 0 &&
                 bytes > ((int64_t)(f == FOUR ? 256 : 64) << 20);
  const int64_t grid = tile_bound<QC>(p, (f == LARGE ? 256 : f == SPLIT ? 64 : f == THIN ? 32 : 128) / (GLU ? 2 : 1),
                                      f == LARGE ? 256 : f >= SPLIT ? 64 : 128);
  if (grid > 0x7FFFFFFF - kDealSlack) return hipErrorInvalidConfiguration;
  const int threads = f == LARGE ? 512 : f == SPLIT ? 64 * kSplitWaves<FMT, 64> : f == THIN ? 64 * kSplitWaves<FMT, 32> : 256;
  return in_slices(grid + kDealSlack, threads, [&](uint32_t first, uint32_t n) {
    p.first = first;
    if (f == LARGE) ragged_gemm<FMT, PC, QC, 256, 256, 4, 2, false, EPI><<<n, threads, 0, s>>>(p);
    else if (f == TWO) ragged_gemm<FMT, PC, QC, 128, 128, 2, 2, false, EPI><<<n, threads, 0, s>>>(p);
    else if (f == FOUR) ragged_gemm<FMT, PC, QC, 128, 128, 2, 2, true, EPI><<<n, threads, 0, s>>>(p);
    else if (f == SPLIT) ragged_split<FMT, PC, QC, 64, EPI><<<n, threads, 0, s>>>(p);
    else ragged_split<FMT, PC, QC, 32, EPI><<<n, threads, 0, s>>>(p);
    return hipGetLastError();
  });
}

}  // namespace
}  // namespace moe

// Grouped products over ragged groups of rows on tiles of the matrix cores.
#include <type_traits>

#include "moe_device.h"
#include "moe_ragged.h"

namespace moe {
namespace {

typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(3))) char lds_char_t;
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

enum Fmt : int { FMT_BF16 = 0, FMT_F16 = 1, FMT_MX = 2 };

constexpr int kStageBytes = 128;          // contraction bytes of a row per step: 64 values, or 256 FP4 codes
constexpr uint32_t kPastEnd = 0x80000000u; // an offset past every operand tile: the load gives 0

template <int FMT>
__device__ __forceinline__ f32x4_t mma(u32x4_t a, u32x4_t b, f32x4_t c) {
  if constexpr (FMT == FMT_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                  0, 0, 0);
  else
    return mfma16(a, b, c);
}

// D += A . B on one 16x16x128 tile of FP4 codes, byte KK of each lane's scale
// word: lane l feeds 32 codes of row l%16 of A (column l%16 of B), its block
// l/16 of the four.
template <int KK>
__device__ __forceinline__ f32x4_t mma_mx(u32x4_t a, u32x4_t b, f32x4_t c, int sa, int sb) {
  const i32x8_t A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8_t B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, KK, sa, KK, sb);
}

// First row and row count of expert e, whatever the offsets hold: within [0, M].
struct Group {
  int lo, n;
};
__device__ __forceinline__ Group group_of(const RaggedParams& p, int e) {
  const int lo = min(max(p.offsets[e], 0), p.M);
  return Group{lo, min(max(p.offsets[e + 1], lo), p.M) - lo};
}

// The tile of workgroup b among all experts' tiles of BJ rows x NI columns,
// experts in order, a column's row tiles side by side, each XCD one
// contiguous share. e < 0: none left. Every lane of a wave looks at one of 64
// experts at a time.
struct Tile {
  int e, it, jt;
};
__device__ __forceinline__ Tile find_tile(const RaggedParams& p, int b, int BJ, int NI) {
  const int lane = threadIdx.x & 63;
  auto count = [&](int e) { return e < p.E ? (group_of(p, e).n + BJ - 1) / BJ : 0; };
  int total = 0;
  for (int base = 0; base < p.E; base += 64) total += count(base + lane);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o, 64);
  const int t = xcd_remap_active(b, __builtin_amdgcn_readfirstlane(total) * NI);
  if (t < 0) return Tile{-1, 0, 0};
  int before = 0;
  for (int base = 0; base < p.E; base += 64) {
    const int n = count(base + lane);
    int sum = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(sum, o, 64);
      sum += lane >= o ? v : 0;
    }
    const uint64_t past = __ballot((before + sum) * NI > t);
    if (past) {
      const int at = __builtin_ctzll(past);
      const int ne = __shfl(n, at, 64), local = t - (before + __shfl(sum, at, 64) - ne) * NI;
      const int it = local / ne;
      return Tile{__builtin_amdgcn_readfirstlane(base + at), __builtin_amdgcn_readfirstlane(it),
                  __builtin_amdgcn_readfirstlane(local - it * ne)};
    }
    before += __shfl(sum, 63, 64);
  }
  return Tile{-1, 0, 0};
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}

// One operand's tile of B output rows/columns: copies to LDS and fragment
// reads. A copy moves 1 KB per wave, straight from global memory to LDS;
// offsets past the operand's last byte read as 0 and take part in nothing.
//
// COL false (contiguous along the contraction): B rows of 128 bytes, 16-byte
// piece c of row r at position c ^ f(r), f = r%8 ^ r/8%2: the 16 rows a
// fragment read takes one piece from, and any 8 of them side by side, fall on
// distinct banks.
// COL true: 64 contraction rows of B values, 32-byte chunk c of row r at
// c ^ g(r), g = r%4 + 4 (r/8%2); a fragment is two transposing reads of 4
// rows x 16 values per 16 lanes.
template <int FMT, bool COL, int B, int NW>
struct Operand {
  static constexpr int kBytes = B * kStageBytes;
  static constexpr int kCopies = B / 8 / NW;       // per wave and step
  static constexpr int kRowB = B * 2;              // COL: bytes of a contraction row
  static constexpr int kLanes = COL ? (kRowB / 16) : 8;   // lanes on one row of a copy
  static constexpr int kRows = 64 / kLanes;        // rows of a copy
  static_assert(B / 8 % NW == 0 && kRowB <= 1024, "whole copies");

  const char* base;
  int64_t ld;
  uint32_t bytes;      // from base to the operand's last byte (COL: of `rows` rows, see at())
  int rows, width;     // COL: contraction rows, bytes to the last needed column
  uint32_t voff;
  int rd[COL ? 8 : 2];

  __device__ __forceinline__ void init(const void* b, int64_t row_bytes, int n, int c_bytes, int wave, int lane,
                                       int w0) {
    base = static_cast<const char*>(b);
    ld = row_bytes;
    const int row = wave * kRows + lane / kLanes, pos = lane % kLanes;
    if constexpr (COL) {
      rows = n;
      width = c_bytes;
      const int g = (row & 3) | (((row >> 3) & 1) << 2);
      voff = (uint32_t)(row * (int)ld + (((pos >> 1) ^ g) * 2 + (pos & 1)) * 16);
      const int j = (lane & 15) >> 2, q = lane >> 4, gr = j | ((q & 1) << 2);
#pragma unroll
      for (int t = 0; t < 8; ++t) rd[t] = (8 * q + j) * kRowB + (((w0 / 16 + t) ^ gr) * 32) + (lane & 3) * 8;
    } else {
      bytes = n > 0 ? (uint32_t)((n - 1) * (int)ld + c_bytes) : 0u;
      const int piece = pos ^ ((row & 7) ^ (wave & 1));
      voff = (uint32_t)(row * (int)ld + piece * 16);
      width = piece * 16;
      rows = c_bytes;
      const int r = lane & 15, q = lane >> 4, f = (r & 7) ^ (r >> 3);
      const int first = FMT == FMT_MX ? 2 * q : q, step = FMT == FMT_MX ? 16 : 64;
      rd[0] = (w0 + r) * kStageBytes + (first ^ f) * 16;
      rd[1] = rd[0] ^ step;
    }
  }

  // Step s into `stage`.
  __device__ __forceinline__ void copy(char* stage, int s, int wave) const {
    if constexpr (COL) {
      const int left = min(rows - 64 * s, 64);
      const __amdgpu_buffer_rsrc_t r =
          rsrc(base + (int64_t)s * 64 * ld, left > 0 ? (uint32_t)((left - 1) * (int)ld + width) : 0u);
#pragma unroll
      for (int i = 0; i < kCopies; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)(stage + (i * NW + wave) * 1024), 16, voff,
                                                 i * NW * kRows * (int)ld, 0, 0);
    } else {
      const __amdgpu_buffer_rsrc_t r = rsrc(base, bytes);
      const int at = s * kStageBytes;
      const uint32_t v = at + width < rows ? voff : kPastEnd;   // the row's contraction ends before this piece
#pragma unroll
      for (int i = 0; i < kCopies; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)(stage + (i * NW + wave) * 1024), 16, v,
                                                 i * NW * kRows * (int)ld + at, 0, 0);
    }
  }

  // Fragment t (16 rows/columns from w0 + 16 t) of half kk of a step.
  __device__ __forceinline__ u32x4_t frag(const char* stage, int t, int kk) const {
    if constexpr (COL) {
      const lds_char_t* at = (const lds_char_t*)(stage + rd[t] + kk * 32 * kRowB);
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)at);
      const s16x4_t hi =
          __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(at + 4 * kRowB));
      const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, hi);
      return u32x4_t{a[0], a[1], b[0], b[1]};
    } else {
      return *reinterpret_cast<const u32x4_t*>(stage + rd[kk] + t * 16 * kStageBytes);
    }
  }
};

__device__ __forceinline__ void store4(void* out, int64_t at, int type, f32x4_t v) {
  if (type == TYPE_BF16) {
    *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(out) + at) =
        u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  } else if (type == TYPE_F16) {
    const f16x4_t h = {(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
    *reinterpret_cast<f16x4_t*>(static_cast<_Float16*>(out) + at) = h;
  } else {
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(out) + at) = v;
  }
}

// One BI x BJ output tile per workgroup of WI x WJ waves. Two LDS stages:
// while the waves multiply step s, step s + 1 is on its way to the other.
template <int FMT, bool PC, bool QC, int BI, int BJ, int WI, int WJ>
__global__ __launch_bounds__(64 * WI * WJ) void ragged_gemm(RaggedParams p) {
  constexpr int NW = WI * WJ, TI = BI / WI / 16, TJ = BJ / WJ / 16;
  constexpr bool MX = FMT == FMT_MX;
  constexpr int kVal = MX ? 256 : 64;     // contraction values per step
  using OpP = Operand<FMT, PC, BI, NW>;
  using OpQ = Operand<FMT, QC, BJ, NW>;
  constexpr int kStage = OpP::kBytes + OpQ::kBytes;
  __shared__ __align__(1024) char lds[2 * kStage];
  __shared__ __align__(1024) char lds_s[MX ? 2 * (BI + BJ) * 16 : 16];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave / WJ, wj = wave % WJ;
  const int NI = (p.I + BI - 1) / BI;

  int e, it, jt;
  if constexpr (QC) {
    const int nj = (p.J + BJ - 1) / BJ;
    const int t = xcd_remap(blockIdx.x, gridDim.x);
    e = t / (nj * NI);
    it = (t - e * nj * NI) / nj;
    jt = t - e * nj * NI - it * nj;
  } else {
    const Tile t = find_tile(p, blockIdx.x, BJ, NI);
    if (t.e < 0) return;
    e = t.e, it = t.it, jt = t.jt;
  }
  const Group g = group_of(p, e);
  const int i0 = it * BI, j0 = jt * BJ;
  const int ni = min(p.I - i0, BI), nj = min((QC ? p.J : g.n) - j0, BJ);
  const int C = QC ? g.n : p.C;

  OpP P;
  OpQ Q;
  constexpr int kBits = MX ? 4 : 16;
  const char* pb = static_cast<const char*>(p.p);
  const char* qb = static_cast<const char*>(p.q);
  const int cb = C / 8 * kBits + C % 8 * kBits / 8;   // contraction bytes of a row
  if constexpr (QC) {
    P.init(pb + (int64_t)g.lo * p.p_ld + (int64_t)i0 * 2, p.p_ld, C, ni * 2, wave, lane, wi * (BI / WI));
    Q.init(qb + (int64_t)g.lo * p.q_ld + (int64_t)j0 * 2, p.q_ld, C, nj * 2, wave, lane, wj * (BJ / WJ));
  } else {
    const char* we = pb + (int64_t)e * p.p_stride;
    if constexpr (PC)
      P.init(we + (int64_t)i0 * 2, p.p_ld, C, ni * 2, wave, lane, wi * (BI / WI));
    else
      P.init(we + (int64_t)i0 * p.p_ld, p.p_ld, ni, cb, wave, lane, wi * (BI / WI));
    Q.init(qb + (int64_t)(g.lo + j0) * p.q_ld, p.q_ld, nj, cb, wave, lane, wj * (BJ / WJ));
  }

  const int steps = (C + kVal - 1) / kVal;
  const int blocks = C / 32;   // MX: scale blocks of a row
  auto issue = [&](int s) {
    char* st = lds + (s & 1) * kStage;
    P.copy(st, s, wave);
    Q.copy(st + OpP::kBytes, s, wave);
    if constexpr (MX) {
      if ((s & 1) == 0) {
        // 16 scales of every row: two steps' worth
        char* ss = lds_s + ((s >> 1) & 1) * (BI + BJ) * 16;
        const int ld = (int)p.s_ld;
        for (int n = wave; n < (BI + BJ) / 64; n += NW) {
          const bool isp = n < BI / 64;
          const int r0 = (isp ? n : n - BI / 64) * 64;
          const uint8_t* b = isp ? p.ps + (int64_t)e * p.ps_stride + (int64_t)i0 * ld
                                 : p.qs + (int64_t)(g.lo + j0) * ld;
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(b, (uint32_t)((isp ? ni : nj) * ld)),
                                                   (lds_void_t*)(ss + n * 1024), 16, (r0 + lane) * ld, s * 8, 0, 0);
        }
      }
    }
  };

  f32x4_t acc[TI][TJ];
#pragma unroll
  for (int t = 0; t < TI; ++t)
#pragma unroll
    for (int u = 0; u < TJ; ++u) acc[t][u] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  if (steps > 0) issue(0);
  for (int s = 0; s < steps; ++s) {
    __syncthreads();   // step s has landed, and every wave is past step s - 1
    if (s + 1 < steps) issue(s + 1);
    const char* st = lds + (s & 1) * kStage;
    int sp[TI], sq[TJ];
    if constexpr (MX) {
      const char* ss = lds_s + ((s >> 1) & 1) * (BI + BJ) * 16 + (lane & 15) * 16 + (s & 1) * 8 + (lane >> 4) * 2;
#pragma unroll
      for (int t = 0; t < TI; ++t)
        sp[t] = *reinterpret_cast<const uint16_t*>(ss + (wi * (BI / WI) + 16 * t) * 16);
#pragma unroll
      for (int u = 0; u < TJ; ++u)
        sq[u] = *reinterpret_cast<const uint16_t*>(ss + (BI + wj * (BJ / WJ) + 16 * u) * 16);
      if (8 * s + 8 > blocks) {
        // scales past the row's last block may hold anything: 2^0 there
        const int at = 8 * s + 2 * (lane >> 4);
        const int keep = at + 1 < blocks ? 0xFFFF : at < blocks ? 0xFF : 0;
#pragma unroll
        for (int t = 0; t < TI; ++t) sp[t] = (sp[t] & keep) | (0x7F7F & ~keep);
#pragma unroll
        for (int u = 0; u < TJ; ++u) sq[u] = (sq[u] & keep) | (0x7F7F & ~keep);
      }
    }
    auto half = [&](auto kk) {
      constexpr int KK = decltype(kk)::value;
      u32x4_t pf[TI], qf[TJ];
#pragma unroll
      for (int t = 0; t < TI; ++t) pf[t] = P.frag(st, t, KK);
#pragma unroll
      for (int u = 0; u < TJ; ++u) qf[u] = Q.frag(st + OpP::kBytes, u, KK);
#pragma unroll
      for (int u = 0; u < TJ; ++u)
#pragma unroll
        for (int t = 0; t < TI; ++t) {
          if constexpr (MX) acc[t][u] = mma_mx<KK>(pf[t], qf[u], acc[t][u], sp[t], sq[u]);
          else acc[t][u] = mma<FMT>(pf[t], qf[u], acc[t][u]);
        }
    };
    half(std::integral_constant<int, 0>{});
    half(std::integral_constant<int, 1>{});
  }

  const int64_t row0 = QC ? (int64_t)j0 : (int64_t)(g.lo + j0);
  const int64_t ob = QC ? (int64_t)e * p.out_stride : 0;
#pragma unroll
  for (int u = 0; u < TJ; ++u) {
    const int j = wj * (BJ / WJ) + 16 * u + (lane & 15);
    if (j >= nj) continue;
#pragma unroll
    for (int t = 0; t < TI; ++t) {
      const int i = wi * (BI / WI) + 16 * t + 4 * (lane >> 4);
      if (i < ni) store4(p.out, ob + (row0 + j) * p.out_ld + i0 + i, p.out_type, acc[t][u]);
    }
  }
}

template <int FMT, bool PC, bool QC>
hipError_t launch(const RaggedParams& p, hipStream_t s) {
  constexpr int BI = 128, BJ = 128;
  const int64_t NI = (p.I + BI - 1) / BI;
  const int64_t live = p.E < p.M ? p.E : p.M;   // experts that can hold rows
  const int64_t grid = QC ? p.E * NI * ((p.J + BJ - 1) / BJ) : NI * ((p.M + live * (BJ - 1)) / BJ);
  if (grid == 0) return hipSuccess;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  ragged_gemm<FMT, PC, QC, BI, BJ, 2, 2><<<(unsigned)grid, 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

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

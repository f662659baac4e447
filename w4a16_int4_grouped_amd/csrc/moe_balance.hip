// Balance loss of the router and the gradient of its logits.
//
// Scores p[t, e] of token t: softmax of its logits, or their sigmoids over the
// sigmoids' sum. For a sequence of n rows with counts[e] of their n k choices:
//   loss = E sum_e f_e P_e,  f_e = counts[e] / (n k),  P_e = sum_t p[t, e] / n
//   d l[t, e] = p[t, e] (c_e - sum_i c_i p[t, i]) (1 - sigmoid(l[t, e]) or, for softmax, 1)
//   with c_e = d_loss E counts[e] / (n^2 k)
// (counts have no gradient). A logit of -inf or NaN has score 0, +inf counts as
// the largest FP32 value, and a row without any other has no scores at all.
//
// One wave per row, a lane holding the experts of its places. The sums over rows
// keep a fixed order: a wave adds up its rows in registers, a workgroup its
// waves, and a second kernel the workgroups' parts in FP64 (one kernel does
// where one workgroup has all rows). A workgroup's rows are a chunk of all rows,
// whatever sequences meet in it: part c + s belongs to chunk c and sequence s,
// no two such pairs have the same sum, because both only grow along the rows.
//
// 16411 tokens of 384 experts in 13 sequences, sigmoid, BF16: 10.5 us for the
// sums, 5.2 for the second kernel, 13.2 for the gradient (added to another), where
// the bytes take 2.5 and 7.6. Latency bounds the first: its vector instructions
// take 3 us, but 257 workgroups are two waves a SIMD, which wait in half of their
// cycles, for a second round of loads behind the first's scores and for a row's
// sums (one row's loads at a time, expf and divisions: 15.1 us). Four dependent
// steps of memory bound the second, bytes and a row's chain of two sums the third
// (20.7 us).
#include "moe_rows.h"
#include "moe_step.h"

namespace moe {
namespace {

constexpr int kSumWaves = 8;       // of a workgroup that sums
// Rows of a chunk: those whose loads a workgroup has in flight together (more
// than 1024 experts: twice as many), more where there would be too many chunks.
// In us for both kernels (BF16), chunks of 8 / 16 / 32 / 64 rows:
//   experts, tokens    384, 512        8.6    7.9    8.1*   9.7
//                      384, 4096        12    9.2    8.5*    11
//                     1024, 512        9.1    8.7*    10     14
//                     1024, 4096        13     10*    11     16
//                     4096, 512         15*    18     26     43
//                     4096, 4096        22*    23     30     47
// and in chunks of 32 / 64 / 128 rows for 384 experts 16411 tokens 13.5 / 11.7* /
// 14.7, 65536 tokens 26.0 / 25.8 / 24.1*; for 64 experts 262144 tokens (FP32) in at
// most 512 / 1024 / 2048 chunks 38.1 / 35.2* / 37.4.
// One sequence of up to twice as many rows is one workgroup's: 384 experts, 64
// tokens 6.0 against 7.8 us; 1024, 32 tokens 6.2 against 8.1, 64 tokens 10.3 against
// 7.9; 4096, 16 tokens 12.8 against 12.6.
int least_rows(int E) { return E <= 512 ? 32 : E <= 1024 ? 16 : 8; }
bool is_solo(int T, int E, int S) { return S == 1 && T <= 2 * least_rows(E); }
int chunk_rows(int T, int E, int S) {
  const int least = least_rows(E), most = E > 64 ? 512 : 1024;
  if (is_solo(T, E, S)) return 2 * least;
  const int n = (T + most - 1) / most;
  return n > least ? (n + least - 1) / least * least : least;
}

// Workspace: parts [chunks + S][E] of P in FP32 and of the counts, the columns'
// shares of each loss [S][ceil(E / 64)] in FP64, tickets [S].
struct BalanceWs {
  int chunk, chunks, groups;
  int64_t p_at, n_at, loss_at, ticket_at, bytes;
};
__host__ __device__ __forceinline__ int64_t up256(int64_t n) { return (n + 255) & ~(int64_t)255; }

BalanceWs ws_of(int T, int E, int S) {
  BalanceWs w;
  w.chunk = chunk_rows(T, E, S);
  w.chunks = (int)(((int64_t)T + w.chunk - 1) / w.chunk);
  w.groups = (E + 63) / 64;
  const int64_t part = up256(((int64_t)w.chunks + S) * E * 4);
  w.p_at = 0;
  w.n_at = part;
  w.loss_at = 2 * part;
  w.ticket_at = w.loss_at + up256((int64_t)S * w.groups * 8);
  w.bytes = w.ticket_at + up256((int64_t)S * 4);
  return w;
}

// Rows [lo, hi) of sequence s within all T.
struct Rows {
  int lo, hi;
};
__device__ __forceinline__ Rows sequence(const BalanceParams& p, int s) {
  if (!p.offsets) return Rows{0, p.T};
  const int lo = min(max(p.offsets[s], 0), p.T);
  return Rows{lo, max(min(p.offsets[s + 1], p.T), lo)};
}

// The first sequence that ends behind row r, S if none does, for a whole wave:
// its lanes look at 64 of them at a time.
__device__ __forceinline__ int sequence_at(const BalanceParams& p, int r) {
  if (!p.offsets) return 0;
  const int lane = threadIdx.x & 63;
  int a = 0, n = p.S;                    // it is one of a .. a + n
  while (n > 0) {
    const int step = (n + 63) / 64, at = min((lane + 1) * step, n) - 1;
    const uint64_t past = __ballot(p.offsets[a + at + 1] > r);
    if (!past) return a + n;
    const int f = __builtin_ctzll(past);
    a += f * step;
    n = step == 1 ? 0 : min(step, n - f * step) - 1;   // (the last of them is one that does)
  }
  return a;
}

// A row's places: lane holds experts V lane + 64 V g + i at place V g + i.
template <int V>
__device__ __forceinline__ int expert_of(int lane, int place) {
  return V * lane + 64 * V * (place / V) + place % V;
}

// A row as loaded: the conversions stand behind the loads, so that those of
// several rows are in flight together. Places without an expert, and rows
// without `has`, hold -inf, or with ZERO 0.
template <int TYPE, int VPL, int V, bool ZERO = false>
struct RowRaw {
  static constexpr bool F32 = TYPE == TYPE_F32;
  static constexpr uint32_t kNone = ZERO ? 0u : F32 ? 0xFF800000u : TYPE == TYPE_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
  static constexpr int kWords = F32 ? VPL : (VPL + 1) / 2;
  uint32_t w[V == 1 ? VPL : kWords];
  __device__ __forceinline__ void load(const void* x, int64_t row, int E, int lane, bool has) {
#pragma unroll
    for (int g = 0; g < VPL; g += V) {
      const int e = expert_of<V>(lane, g);
      const bool in = has && e < E;
      if constexpr (V == 1) {
        w[g] = kNone;
        if (in) {
          if constexpr (F32) w[g] = static_cast<const uint32_t*>(x)[row + e];
          else w[g] = static_cast<const uint16_t*>(x)[row + e];
        }
      } else if constexpr (F32) {
        u32x2_t v = {kNone, kNone};
        if (in) v = *reinterpret_cast<const u32x2_t*>(static_cast<const float*>(x) + row + e);
        w[g] = v[0], w[g + 1] = v[1];
      } else {
        w[g / 2] = kNone;
        if (in) w[g / 2] = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(x) + row + e);
      }
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (F32) return __uint_as_float(w[i]);
    const uint32_t h = V == 1 ? w[i] : i & 1 ? w[i / 2] >> 16 : w[i / 2];
    if constexpr (TYPE == TYPE_BF16) return __uint_as_float(h << 16);
    else return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
  }
};

// e^x, x <= 0, by v_exp_f32; results below 2^-126 are 0. For 16-bit logits of x
// log2 e rounded, which moves it by up to |x| 2^-24 of itself. FINE (FP32 logits):
// what that left out, x - y ln 2, is multiplied in, so that scores are off by a
// few 2^-24 whatever x is, as by expf (2^21 tokens of 64 experts 215 -> 227 us,
// 12000 of 512 in 64 sequences 21.3 -> 22.0).
constexpr float kLog2e = 1.44269502f, kLn2 = 0.693147182f, kLn2Rest = -1.90465421e-9f;
template <bool FINE>
__device__ __forceinline__ float exp_of(float x) {
  if constexpr (!FINE) return __builtin_amdgcn_exp2f(x * kLog2e);
  x = fmaxf(x, -200.f);   // (-inf leaves nothing out)
  const float y = x * kLog2e, v = __builtin_amdgcn_exp2f(y);
  return __builtin_fmaf(v, __builtin_fmaf(-y, kLn2Rest, __builtin_fmaf(-y, kLn2, x)), v);
}
// l becomes the scores, `rest` what remains of 1 above the sigmoid (softmax: 1).
// Where the sigmoids' sum would lose them to FP32's small end, they are e^l to
// FP32 accuracy, and e^(l - top) does not vanish.
template <int VPL, bool FINE>
__device__ __forceinline__ void scores(float (&l)[VPL], int sigmoid_scores, float (&rest)[VPL]) {
  float v[VPL], total = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) l[i] = l[i] >= -kMax ? fminf(l[i], kMax) : -INFINITY, rest[i] = 1.f;
  if (sigmoid_scores) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const float x = exp_of<FINE>(-fabsf(l[i])), y = __builtin_amdgcn_rcpf(1.0f + x);   // sigmoid(|l|) = y, sigmoid(-|l|) = x y
      const float xy = x * y;
      v[i] = l[i] < 0.f ? xy : y;
      rest[i] = l[i] < 0.f ? y : xy;
      total += v[i];
    }
    total = wave_sum_of(total);
  }
  if (!sigmoid_scores || total < 0x1p-80f) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) top = fmaxf(top, l[i]);
    top = wave_max_of(top);
    if (top == -INFINITY) top = 0.f;
    total = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      v[i] = exp_of<FINE>(l[i] - top);
      rest[i] = 1.f;
      total += v[i];
    }
    total = wave_sum_of(total);
  }
  const float inv = total > 0.f ? __builtin_amdgcn_rcpf(total) : 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) l[i] = v[i] * inv;
}

// Rows of a wave whose loads are in flight together.
constexpr int rows_ahead(int VPL) { return VPL <= 8 ? 4 : VPL <= 16 ? 2 : 1; }

// Rows that a wave adds up in registers one after another; its sum of more is
// (LONG) one of such sums, in LDS. All terms have one sign: 2^24 tokens of even
// scores, 2048 a wave for 13 experts, were off by 434 2^-24 in one chain of FP32.
// LONG's branch in all kernels cost shorter chunks up to 4 % (512 tokens of 4096
// experts 14.5 -> 15.1 us).
constexpr int kFold = 128;

// W waves sum a chunk. SOLO: the one chunk of the one sequence: counts and loss at
// once. LONG: of more than kFold rows a wave.
template <int TYPE, int VPL, int V, int W, bool SOLO, bool LONG>
__global__ __launch_bounds__(64 * W) void balance_sums(BalanceParams p, BalanceWs ws) {
  constexpr int kE = 64 * VPL, NR = rows_ahead(VPL);
  __shared__ float part[W][kE];
  __shared__ int hist[kE];
  __shared__ double shares[W];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  char* const base = static_cast<char*>(p.ws);
  const int r0 = blockIdx.x * ws.chunk, r1 = min((int64_t)r0 + ws.chunk, (int64_t)p.T);
  if (!SOLO && blockIdx.x == 0) {
    int* ticket = reinterpret_cast<int*>(base + ws.ticket_at);
    for (int s = threadIdx.x; s < p.S; s += 64 * W) ticket[s] = 0;
  }
  // the first rows and ids of the chunk, whatever sequence they belong to
  RowRaw<TYPE, VPL, V> raw[NR];
  const int mine = r0 + wave * NR;
  int held = mine;             // the row that raw begins with
#pragma unroll
  for (int n = 0; n < NR; ++n) raw[n].load(p.logits, (int64_t)(mine + n) * p.ld, p.E, lane, mine + n < r1);
  const int64_t id_first = (int64_t)r0 * p.topk + threadIdx.x, id_end = (int64_t)r1 * p.topk;
  const int first_id = id_first < id_end ? p.ids[id_first] : -1;
  for (int s = SOLO ? 0 : sequence_at(p, r0); s < p.S; ++s) {
    Rows q = sequence(p, s);
    if (!SOLO && q.lo >= r1) break;
    q.lo = max(q.lo, r0), q.hi = min(q.hi, r1);
    if (!SOLO && q.lo >= q.hi) continue;
    for (int e = threadIdx.x; e < kE; e += 64 * W) hist[e] = 0;
    __syncthreads();
    float sum[VPL] = {};
    int added = 0;
    bool more = false;         // part holds sums of this wave's rows
    auto fold = [&] {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        float& at = part[wave][expert_of<V>(lane, i)];
        at = LONG && more ? at + sum[i] : sum[i];
        sum[i] = 0.f;
      }
      more = true, added = 0;
    };
    for (int r = mine; r < q.hi; r += W * NR) {
      if (r + NR <= q.lo) continue;
      if (LONG && added == kFold) fold();
      added += NR;
      if (r != held) {
        held = r;
#pragma unroll
        for (int n = 0; n < NR; ++n) raw[n].load(p.logits, (int64_t)(r + n) * p.ld, p.E, lane, r + n < r1);
      }
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        if (r + n < q.lo || r + n >= q.hi) continue;
        float l[VPL], rest[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) l[i] = raw[n].get(i);
        scores<VPL, TYPE == TYPE_F32>(l, p.sigmoid, rest);
#pragma unroll
        for (int i = 0; i < VPL; ++i) sum[i] += l[i];
      }
    }
    const int64_t id_lo = (int64_t)q.lo * p.topk, id_hi = (int64_t)q.hi * p.topk;
    for (int64_t i = id_first; i < id_hi; i += 64 * W) {
      if (i < id_lo) continue;
      const int e = i == id_first ? first_id : p.ids[i];
      if (e >= 0 && e < p.E) atomicAdd(&hist[e], 1);
    }
    fold();
    __syncthreads();
    if constexpr (SOLO) {
      double share = 0.0;
      for (int e = threadIdx.x; e < p.E; e += 64 * W) {
        double P = 0.0;
#pragma unroll
        for (int w = 0; w < W; ++w) P += part[w][e];
        p.counts[e] = hist[e];
        share += P * hist[e];
      }
      share = wave_sum_of(share);
      if (lane == 0) shares[wave] = share;
      __syncthreads();
      if (threadIdx.x == 0) {
        double loss = 0.0;
        for (int w = 0; w < W; ++w) loss += shares[w];
        const double n = q.hi - q.lo;
        p.loss[0] = n > 0 ? (float)(loss * p.E / (n * n * p.topk)) : 0.f;
      }
      return;
    } else {
      const int64_t at = ((int64_t)blockIdx.x + s) * p.E;
      float* P = reinterpret_cast<float*>(base + ws.p_at) + at;
      int* N = reinterpret_cast<int*>(base + ws.n_at) + at;
      for (int e = threadIdx.x; e < p.E; e += 64 * W) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += part[w][e];
        P[e] = v;
        N[e] = hist[e];
      }
      __syncthreads();
    }
  }
}

// Sequence blockIdx.x, 64 experts. The last workgroup of a sequence adds up the
// shares of its loss, in their order. (2^20 sequences of 4 groups in one dimension
// would be 2^32 threads, which a launch does not take.)
constexpr int kFinishWaves = 16;
__global__ __launch_bounds__(64 * kFinishWaves) void balance_finish(BalanceParams p, BalanceWs ws) {
  __shared__ double part[kFinishWaves][64];
  __shared__ int num[kFinishWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int s = blockIdx.x, g = blockIdx.y;
  const int e = 64 * g + lane;
  char* const base = static_cast<char*>(p.ws);
  const Rows q = sequence(p, s);
  double P = 0.0;
  int N = 0;
  if (q.lo < q.hi && e < p.E) {
    const int c0 = q.lo / ws.chunk, c1 = (q.hi - 1) / ws.chunk;
    const float* ps = reinterpret_cast<const float*>(base + ws.p_at) + (int64_t)s * p.E + e;
    const int* ns = reinterpret_cast<const int*>(base + ws.n_at) + (int64_t)s * p.E + e;
#pragma unroll 8
    for (int c = c0 + wave; c <= c1; c += kFinishWaves) {
      P += ps[(int64_t)c * p.E];
      N += ns[(int64_t)c * p.E];
    }
  }
  part[wave][lane] = P, num[wave][lane] = N;
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int w = 1; w < kFinishWaves; ++w) P += part[w][lane], N += num[w][lane];
  if (e < p.E) p.counts[(int64_t)s * p.E + e] = N;
  double share = wave_sum_of(P * N);
  const double n = q.hi - q.lo;
  const double scale = n > 0 ? p.E / (n * n * p.topk) : 0.0;
  double* shares = reinterpret_cast<double*>(base + ws.loss_at) + (int64_t)s * ws.groups;
  if (ws.groups > 1) {
    int* ticket = reinterpret_cast<int*>(base + ws.ticket_at) + s;
    int last = 0;
    if (lane == 0) {
      __hip_atomic_store(shares + g, share, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = __hip_atomic_fetch_add(ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == ws.groups - 1;
    }
    if (!__builtin_amdgcn_readfirstlane(last)) return;
    double v = lane < ws.groups ? __hip_atomic_load(shares + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
    share = wave_sum_of(v);   // at most 64 groups
  }
  if (lane == 0) p.loss[s] = (float)(share * scale);
}

template <int TYPE, int VPL, int V>
__global__ __launch_bounds__(256) void balance_grad(BalanceParams p) {
  constexpr int NR = rows_ahead(VPL);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t first = ((int64_t)blockIdx.x * 4 + wave) * NR;
  if (first >= p.T) return;
  const int r0 = (int)first;
  RowRaw<TYPE, VPL, V> raw[NR];
  RowRaw<TYPE, VPL, V, true> add[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    raw[n].load(p.logits, (first + n) * p.ld, p.E, lane, first + n < p.T);
    if (p.add) add[n].load(p.add, (first + n) * p.add_ld, p.E, lane, first + n < p.T);
  }
  int s = sequence_at(p, r0), has = -1;   // the row's sequence, and whose coefficients c holds
  Rows q = s < p.S ? sequence(p, s) : Rows{0, 0};
  float c[VPL] = {};
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int r = r0 + n;
    if (r >= p.T) return;
    while (s < p.S && r >= q.hi)
      if (++s < p.S) q = sequence(p, s);
    float l[VPL], rest[VPL];
    if (s < p.S && r >= q.lo) {
      if (s != has) {
        const double rows = q.hi - q.lo;
        const float scale = (float)((double)p.d_loss[s] * p.E / (rows * rows * p.topk));
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int e = expert_of<V>(lane, i);
          c[i] = e < p.E ? scale * (float)p.counts_in[(int64_t)s * p.E + e] : 0.f;
        }
        has = s;
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] = raw[n].get(i);
      scores<VPL, TYPE == TYPE_F32>(l, p.sigmoid, rest);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) dot = __builtin_fmaf(c[i], l[i], dot);
      dot = wave_sum_of(dot);
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] *= (c[i] - dot) * rest[i];
    } else {                   // of no sequence
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] = 0.f;
    }
    if (p.add) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] += add[n].get(i);
    }
    const int64_t row = (int64_t)r * p.d_ld;
#pragma unroll
    for (int g = 0; g < VPL; g += V) {
      const int e = expert_of<V>(lane, g);
      if (e >= p.E) continue;
      if constexpr (V == 1) {
        store1<TYPE>(p.d_logits, row + e, l[g]);
      } else if constexpr (TYPE == TYPE_F32) {
        *reinterpret_cast<float2*>(static_cast<float*>(p.d_logits) + row + e) = float2{l[g], l[g + 1]};
      } else {
        uint32_t w;
        if constexpr (TYPE == TYPE_BF16) {
          w = pack_bf16x2(l[g], l[g + 1]);
        } else {
          const f16x2_t h = {(_Float16)l[g], (_Float16)l[g + 1]};
          w = __builtin_bit_cast(uint32_t, h);
        }
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.d_logits) + row + e) = w;
      }
    }
  }
}

// Rows of `type` can be read and written two values at a time.
bool pairs(const void* x, int64_t ld, int type) {
  return !x || (ld % 2 == 0 && (uintptr_t)x % (type == TYPE_F32 ? 8 : 4) == 0);
}

template <int TYPE, int VPL, int V>
hipError_t sums_for(const BalanceParams& p, const BalanceWs& ws, bool solo, hipStream_t s) {
  constexpr int W = VPL > 16 ? 4 : kSumWaves;   // LDS holds each wave's sums
  const unsigned n = ws.chunks > 0 ? ws.chunks : 1;
  if (solo) balance_sums<TYPE, VPL, V, W, true, false><<<1, 64 * W, 0, s>>>(p, ws);
  else if (ws.chunk <= W * kFold) balance_sums<TYPE, VPL, V, W, false, false><<<n, 64 * W, 0, s>>>(p, ws);
  else balance_sums<TYPE, VPL, V, W, false, true><<<n, 64 * W, 0, s>>>(p, ws);
  return hipGetLastError();
}

// f(VPL, V) for E experts, two adjacent ones at a time where rows allow it.
template <class F>
hipError_t by_experts(int E, bool two, F&& f) {
  using std::integral_constant;
  two = two && E % 2 == 0;
  auto go = [&](auto vpl) {
    constexpr int N = decltype(vpl)::value;
    if constexpr (N > 1)
      if (two) return f(vpl, integral_constant<int, 2>{});
    return f(vpl, integral_constant<int, 1>{});
  };
  if (E <= 64) return go(integral_constant<int, 1>{});
  if (E <= 128) return go(integral_constant<int, 2>{});
  if (E <= 256) return go(integral_constant<int, 4>{});
  if (E <= 384) return go(integral_constant<int, 6>{});
  if (E <= 512) return go(integral_constant<int, 8>{});
  if (E <= 1024) return go(integral_constant<int, 16>{});
  return go(integral_constant<int, 64>{});
}

template <class F>
hipError_t by_type(int type, F&& f) {
  if (type == TYPE_BF16) return f(std::integral_constant<int, TYPE_BF16>{});
  if (type == TYPE_F16) return f(std::integral_constant<int, TYPE_F16>{});
  return f(std::integral_constant<int, TYPE_F32>{});
}

}  // namespace

size_t balance_ws_bytes(int T, int E, int S) { return is_solo(T, E, S) ? 0 : (size_t)ws_of(T, E, S).bytes; }

hipError_t launch_balance(const BalanceParams& p, int type, hipStream_t s) {
  const BalanceWs ws = ws_of(p.T, p.E, p.S);
  const bool solo = is_solo(p.T, p.E, p.S);
  const hipError_t e = by_type(type, [&](auto ty) {
    return by_experts(p.E, pairs(p.logits, p.ld, type), [&](auto vpl, auto v) {
      return sums_for<decltype(ty)::value, decltype(vpl)::value, decltype(v)::value>(p, ws, solo, s);
    });
  });
  if (e != hipSuccess || solo) return e;
  balance_finish<<<dim3((unsigned)p.S, (unsigned)ws.groups), 64 * kFinishWaves, 0, s>>>(p, ws);
  return hipGetLastError();
}

hipError_t launch_balance_grad(const BalanceParams& p, int type, hipStream_t s) {
  const bool two = pairs(p.logits, p.ld, type) && pairs(p.add, p.add_ld, type) && pairs(p.d_logits, p.d_ld, type);
  return by_type(type, [&](auto ty) {
    return by_experts(p.E, two, [&](auto vpl, auto v) {
      constexpr int rows = 4 * rows_ahead(decltype(vpl)::value);
      const unsigned n = (unsigned)((p.T + rows - 1) / rows);
      balance_grad<decltype(ty)::value, decltype(vpl)::value, decltype(v)::value><<<n, 256, 0, s>>>(p);
      return hipGetLastError();
    });
  });
}

}  // namespace moe

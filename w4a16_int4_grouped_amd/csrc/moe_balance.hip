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
#include "moe_rows.h"
#include "moe_step.h"

namespace moe {
namespace {

constexpr int kSumWaves = 8;       // of a workgroup that sums
constexpr int kMaxChunks = 1024;

// Rows of a chunk: at least 4 a wave, more where there would be too many chunks.
int chunk_rows(int T) {
  const int least = 4 * kSumWaves;
  const int n = (T + kMaxChunks - 1) / kMaxChunks;
  return (n + least - 1) / least * least > least ? (n + least - 1) / least * least : least;
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
  w.chunk = chunk_rows(T);
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

// The first sequence that ends behind row r, S if none does.
__device__ __forceinline__ int sequence_at(const BalanceParams& p, int r) {
  if (!p.offsets) return 0;
  int a = 0, b = p.S;
  while (a < b) {
    const int m = (a + b) / 2;
    if (p.offsets[m + 1] > r) b = m;
    else a = m + 1;
  }
  return a;
}

// A row's places: lane holds experts V lane + 64 V g + i at place V g + i.
template <int V>
__device__ __forceinline__ int expert_of(int lane, int place) {
  return V * lane + 64 * V * (place / V) + place % V;
}

template <int TYPE, int VPL, int V>
__device__ __forceinline__ void load_row(const void* x, int64_t row, int E, int lane, float (&l)[VPL], float none) {
#pragma unroll
  for (int g = 0; g < VPL; g += V) {
    const int e = expert_of<V>(lane, g);
#pragma unroll
    for (int i = 0; i < V; ++i) l[g + i] = none;
    if (e >= E) continue;
    if constexpr (V == 1) {
      l[g] = load1<TYPE>(x, row + e);
    } else if constexpr (TYPE == TYPE_F32) {
      const float2 v = *reinterpret_cast<const float2*>(static_cast<const float*>(x) + row + e);
      l[g] = v.x, l[g + 1] = v.y;
    } else {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(x) + row + e);
      if constexpr (TYPE == TYPE_BF16) {
        l[g] = bf16_lo(v), l[g + 1] = bf16_hi(v);
      } else {
        const f16x2_t h = __builtin_bit_cast(f16x2_t, v);
        l[g] = (float)h[0], l[g + 1] = (float)h[1];
      }
    }
  }
}

// l becomes the scores, `rest` what remains of 1 above the sigmoid (softmax: 1).
// Where every sigmoid is below e^-60 they are e^l to FP32 accuracy, and e^(l -
// top) does not vanish.
template <int VPL>
__device__ __forceinline__ void scores(float (&l)[VPL], int sigmoid_scores, float (&rest)[VPL]) {
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) l[i] = clean(l[i]), top = fmaxf(top, l[i]);
  top = wave_max_of(top);
  if (top == -INFINITY) top = 0.f;
  float total = 0.f;
  if (sigmoid_scores && top > -60.f) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const float x = expf(-fabsf(l[i])), y = 1.0f / (1.0f + x);   // sigmoid(|l|) = y, sigmoid(-|l|) = x y
      const float xy = l[i] == -INFINITY ? 0.f : x * y;
      rest[i] = l[i] < 0.f ? y : xy;
      l[i] = l[i] < 0.f ? xy : y;
      total += l[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      l[i] = expf(l[i] - top);
      rest[i] = 1.f;
      total += l[i];
    }
  }
  total = wave_sum_of(total);
  const float inv = total > 0.f ? 1.0f / total : 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) l[i] *= inv;
}

// W waves sum a chunk. SOLO: the one chunk of the one sequence: counts and loss at once.
template <int TYPE, int VPL, int V, int W, bool SOLO>
__global__ __launch_bounds__(64 * W) void balance_sums(BalanceParams p, BalanceWs ws) {
  constexpr int kE = 64 * VPL;
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
  for (int s = SOLO ? 0 : sequence_at(p, r0); s < p.S; ++s) {
    Rows q = sequence(p, s);
    if (!SOLO && q.lo >= r1) break;
    q.lo = max(q.lo, r0), q.hi = min(q.hi, r1);
    if (!SOLO && q.lo >= q.hi) continue;
    for (int e = threadIdx.x; e < kE; e += 64 * W) hist[e] = 0;
    __syncthreads();
    float sum[VPL] = {};
    for (int r = q.lo + wave; r < q.hi; r += W) {
      float l[VPL], rest[VPL];
      load_row<TYPE, VPL, V>(p.logits, (int64_t)r * p.ld, p.E, lane, l, -INFINITY);
      scores(l, p.sigmoid, rest);
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum[i] += l[i];
    }
    const int64_t end = (int64_t)q.hi * p.topk;
    for (int64_t i = (int64_t)q.lo * p.topk + threadIdx.x; i < end; i += 64 * W) {
      const int e = p.ids[i];
      if (e >= 0 && e < p.E) atomicAdd(&hist[e], 1);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) part[wave][expert_of<V>(lane, i)] = sum[i];
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
        const double n = p.T;
        p.loss[0] = p.T > 0 ? (float)(loss * p.E / (n * n * p.topk)) : 0.f;
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

// Sequence blockIdx.x / groups, 64 experts. The last workgroup of a sequence
// adds up the shares of its loss, in their order.
constexpr int kFinishWaves = 16;
__global__ __launch_bounds__(64 * kFinishWaves) void balance_finish(BalanceParams p, BalanceWs ws) {
  __shared__ double part[kFinishWaves][64];
  __shared__ int num[kFinishWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int s = blockIdx.x / ws.groups, g = blockIdx.x - s * ws.groups;
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

constexpr int kGradRows = 4;   // rows of a wave, one after another

template <int TYPE, int VPL, int V>
__global__ __launch_bounds__(256) void balance_grad(BalanceParams p) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t first = ((int64_t)blockIdx.x * 4 + wave) * kGradRows;
  const int r0 = (int)first, r1 = (int)min(first + kGradRows, (int64_t)p.T);
  if (first >= p.T) return;
  int s = sequence_at(p, r0), has = -1;   // the row's sequence, and whose coefficients c holds
  Rows q = s < p.S ? sequence(p, s) : Rows{0, 0};
  float c[VPL];
  for (int r = r0; r < r1; ++r) {
    while (s < p.S && r >= q.hi)
      if (++s < p.S) q = sequence(p, s);
    if (s < p.S && s != has) {
      const double n = q.hi - q.lo;
      const float scale = n > 0 ? (float)((double)p.d_loss[s] * p.E / (n * n * p.topk)) : 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = expert_of<V>(lane, i);
        c[i] = e < p.E ? scale * (float)p.counts_in[(int64_t)s * p.E + e] : 0.f;
      }
      has = s;
    }
    float l[VPL], rest[VPL], add[VPL];
    if (p.add) load_row<TYPE, VPL, V>(p.add, (int64_t)r * p.add_ld, p.E, lane, add, 0.f);
    if (s < p.S && r >= q.lo) {
      load_row<TYPE, VPL, V>(p.logits, (int64_t)r * p.ld, p.E, lane, l, -INFINITY);
      scores(l, p.sigmoid, rest);
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
      for (int i = 0; i < VPL; ++i) l[i] += add[i];
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
  if (solo) balance_sums<TYPE, VPL, V, W, true><<<1, 64 * W, 0, s>>>(p, ws);
  else balance_sums<TYPE, VPL, V, W, false><<<n, 64 * W, 0, s>>>(p, ws);
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

size_t balance_ws_bytes(int T, int E, int S) { return (size_t)ws_of(T, E, S).bytes; }

hipError_t launch_balance(const BalanceParams& p, int type, hipStream_t s) {
  const BalanceWs ws = ws_of(p.T, p.E, p.S);
  const bool solo = ws.chunks <= 1 && !p.offsets;
  const hipError_t e = by_type(type, [&](auto ty) {
    return by_experts(p.E, pairs(p.logits, p.ld, type), [&](auto vpl, auto v) {
      return sums_for<decltype(ty)::value, decltype(vpl)::value, decltype(v)::value>(p, ws, solo, s);
    });
  });
  if (e != hipSuccess || solo) return e;
  balance_finish<<<(unsigned)(p.S * ws.groups), 64 * kFinishWaves, 0, s>>>(p, ws);
  return hipGetLastError();
}

hipError_t launch_balance_grad(const BalanceParams& p, int type, hipStream_t s) {
  const bool two = pairs(p.logits, p.ld, type) && pairs(p.add, p.add_ld, type) && pairs(p.d_logits, p.d_ld, type);
  const unsigned n = (unsigned)((p.T + 4 * kGradRows - 1) / (4 * kGradRows));
  return by_type(type, [&](auto ty) {
    return by_experts(p.E, two, [&](auto vpl, auto v) {
      balance_grad<decltype(ty)::value, decltype(vpl)::value, decltype(v)::value><<<n, 256, 0, s>>>(p);
      return hipGetLastError();
    });
  });
}

}  // namespace moe

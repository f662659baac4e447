// Router: the top-k experts of each token and their weights, and the
// gradient of the logits.
//
// Score s_e = softmax(l)_e or sigmoid(l_e). The k experts of largest key are
// chosen, largest first, the lowest index of equal ones: the key is l_e
// itself (both scores grow with it), or with a bias s_e + b_e in FP64, where
// FP32 would merge or swap near ones. A logit of -inf or NaN and a bias of
// -inf or NaN take their expert out; +inf counts as the largest FP32.
// Weights: w_j = scale * s_j, or scale * s_j / (sum of the chosen s), the
// latter as a softmax over the chosen l_j (softmax) or log sigmoid(l_j)
// (sigmoid), which neither overflows nor divides by zero.
//
// One wave per token: each lane holds the keys of experts lane, lane + 64,
// ..; a round takes each lane's best, then the wave's. Latency bounds small T:
// the k rounds depend on each other, and before them a lane's loads do not
// overlap, because the conversion (and the bias) stands under the load's
// condition: 64 experts take 3.4 us, 384 take 6.0 (one token in FP32 with a
// bias, top-8). The wave's best comes by six DPP steps (lane exchanges through
// LDS: 10.4 us for the token of 384 experts). The rounds' instructions, which go
// over all of a lane's keys, bound large T (8192 tokens of 384 experts in BF16,
// top-8: 8.0 us; 65536: 46 us).
#include <type_traits>

#include "moe_device.h"
#include "moe_ragged.h"

namespace moe {
namespace {

template <int TYPE>
__device__ __forceinline__ float load1(const void* x, int64_t at) {
  if constexpr (TYPE == TYPE_F32) return static_cast<const float*>(x)[at];
  else if constexpr (TYPE == TYPE_BF16) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(x)[at] << 16);
  else return (float)static_cast<const _Float16*>(x)[at];
}

template <int TYPE>
__device__ __forceinline__ void store1(void* x, int64_t at, float v) {
  if constexpr (TYPE == TYPE_F32) static_cast<float*>(x)[at] = v;
  else if constexpr (TYPE == TYPE_BF16) static_cast<__bf16*>(x)[at] = (__bf16)v;
  else static_cast<_Float16*>(x)[at] = (_Float16)v;
}

constexpr float kMax = 3.4028234663852886e38f;

// -inf and NaN become -inf (not chosen), +inf the largest finite value, -0 the
// 0 that it is equal to.
__device__ __forceinline__ float clean(float l) { return l >= -kMax ? fminf(l, kMax) + 0.f : -INFINITY; }

// v of the lane that DPP control CTRL names; lanes without one keep theirs.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  const int i = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(i, i, CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const int lo = (int)u, hi = (int)(u >> 32);
  const uint32_t a = (uint32_t)__builtin_amdgcn_update_dpp(lo, lo, CTRL, 0xF, 0xF, false);
  const uint32_t b = (uint32_t)__builtin_amdgcn_update_dpp(hi, hi, CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)b << 32 | a);
}
__device__ __forceinline__ uint32_t last_lane(uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 63); }
__device__ __forceinline__ float last_lane(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ double last_lane(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)u, 63);
  const uint32_t b = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)b << 32 | a);
}
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }

// What the wave's lanes wrote to LDS before is seen by what its lanes read behind.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// v of the lane that DPP control CTRL names, in the rows of mask ROWS; 0 where there is none.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t dpp_or_0(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, true);
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp_or_0(float v) {
  return __uint_as_float(dpp_or_0<CTRL, ROWS>(__float_as_uint(v)));
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp_or_0(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp_or_0<CTRL, ROWS>((uint32_t)(u >> 32)) << 32 |
                                        dpp_or_0<CTRL, ROWS>((uint32_t)u));
}

// The largest v of the wave, in every lane (v is no NaN): rotations by 1, 2, 4
// and 8 lanes within rows of 16, then each row's lane 15 into the next, then
// lane 31 into rows 2 and 3; lane 63 has seen all. Where every lane has a
// source, or 0 stands for none, a step of an integer key is one instruction;
// with a lane's own value for none (the last two of others) it takes a copy.
template <class T>
__device__ __forceinline__ T wave_max_of(T v) {
  v = larger(v, dpp_or_0<0x121>(v));
  v = larger(v, dpp_or_0<0x122>(v));
  v = larger(v, dpp_or_0<0x124>(v));
  v = larger(v, dpp_or_0<0x128>(v));
  if constexpr (std::is_same_v<T, uint32_t>) {
    v = larger(v, dpp_or_0<0x142>(v));
    v = larger(v, dpp_or_0<0x143>(v));
  } else {
    v = larger(v, dpp<0x142>(v));
    v = larger(v, dpp<0x143>(v));
  }
  return last_lane(v);
}

// The sum of the wave's v, in every lane: shifts by 1, 2, 4 and 8 lanes within
// rows, so that a row's lane 15 has its sum, then as above.
template <class T>
__device__ __forceinline__ T wave_sum_of(T v) {
  v += dpp_or_0<0x111, 0xF>(v);
  v += dpp_or_0<0x112, 0xF>(v);
  v += dpp_or_0<0x114, 0xF>(v);
  v += dpp_or_0<0x118, 0xF>(v);
  v += dpp_or_0<0x142, 0xA>(v);
  v += dpp_or_0<0x143, 0xC>(v);
  return last_lane(v);
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }
// log sigmoid(l), exact in its small part for either sign
__device__ __forceinline__ float log_sigmoid(float l) { return fminf(l, 0.f) - log1pf(expf(-fabsf(l))); }

// Chosen experts' shares u_j of a renormalised weight, lane j < k holding
// logit l (-inf: none).
__device__ __forceinline__ float chosen_share(float l, int sig) {
  const float x = l == -INFINITY ? l : sig ? log_sigmoid(l) : l;
  const float m = wave_max_of(x);
  const float e = x == -INFINITY ? 0.f : expf(x - m);
  const float s = wave_sum_of(e);
  return s > 0.f ? e / s : 0.f;
}

// What a choice is made by.
//   KEY16  a 16-bit logit's ordered bits above 0xFFFF - expert: one integer
//          that no other expert has, so the largest names its expert
//   KEY32  an FP32 logit's ordered bits above 4095 - expert, 44 bits held in a
//          double (v_max_f64 compares them in one instruction)
//   KEYB   score + bias in FP64; equal ones are told apart by a ballot
enum KeyKind : int { KEY16 = 0, KEY32 = 1, KEYB = 2 };

// FP32 bits in the order of their values, and back.
__device__ __forceinline__ uint32_t ordered(uint32_t b) { return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u); }
__device__ __forceinline__ uint32_t unordered(uint32_t s) { return s ^ (s >> 31 ? 0x80000000u : 0xFFFFFFFFu); }

// VPL: places for experts per lane, kept in registers; those past E cost their
// instructions all the same.
template <int TYPE, int VPL, int KIND>
__global__ __launch_bounds__(256) void router_topk(RouterParams p) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= p.T) return;
  const int64_t row = (int64_t)t * p.ld;
  float l[VPL], b[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < p.E ? load1<TYPE>(p.logits, row + e) : -INFINITY;
    if constexpr (KIND == KEYB) b[i] = e < p.E ? p.bias[e] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) l[i] = clean(l[i]);
  float top = 0.f, total = 1.f;
  if (!p.sigmoid && (KIND == KEYB || !p.renorm)) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) top = fmaxf(top, l[i]);
    top = wave_max_of(top);
    if (top == -INFINITY) top = 0.f;
    total = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) total += expf(l[i] - top);
    total = wave_sum_of(total);
  }
  int mine = -1;            // lane j: the j-th choice and its logit
  float lj = -INFINITY;
  if constexpr (KIND == KEYB) {
    double key[VPL], sum = 1.0;
    if (!p.sigmoid) {
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (64 * i < p.E) sum += exp((double)l[i] - (double)top);
      sum = wave_sum_of(sum);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      key[i] = -INFINITY;
      if (64 * i < p.E) {
        const double s = p.sigmoid ? 1.0 / (1.0 + exp(-(double)l[i])) : exp((double)l[i] - (double)top) / sum;
        const double k = s + (double)b[i];
        if (l[i] != -INFINITY && k >= -1.7976931348623157e308) key[i] = k;
      }
    }
    for (int j = 0; j < p.topk; ++j) {
      double best = key[0];
      int at = 0;
#pragma unroll
      for (int i = 1; i < VPL; ++i)
        if (key[i] > best) best = key[i], at = i;
      const double most = wave_max_of(best);
      if (most == -INFINITY) break;   // the same in every lane: none left
      const uint64_t has = __ballot(best == most);
      int owner = __builtin_ctzll(has);
      if (has & (has - 1)) {
        // equal keys in several lanes: the lowest expert, so the lowest i, then the lowest lane
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i) {
          const uint64_t m = __ballot(best == most && at == i);
          if (m) owner = __builtin_ctzll(m);
        }
      }
      float v = l[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) v = at == i ? l[i] : v;
      const int id = owner + 64 * __builtin_amdgcn_readlane(at, owner);
      const float lv = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), owner));
      if (lane == j) mine = id, lj = lv;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (id == lane + 64 * i) key[i] = -INFINITY;
    }
  } else {
    using KEY = std::conditional_t<KIND == KEY16, uint32_t, double>;
    KEY key[VPL];           // 0: taken or not to be chosen
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const uint32_t e = (uint32_t)(lane + 64 * i);
      if constexpr (KIND == KEY16) {
        // the top half of a BF16 logit's FP32 bits, an FP16 logit's own; +inf, above either's largest, as itself
        const float x = l[i] == kMax ? INFINITY : l[i];
        uint32_t h;
        if constexpr (TYPE == TYPE_BF16) h = __float_as_uint(x) >> 16;
        else h = __builtin_bit_cast(uint16_t, (_Float16)x);
        h ^= h & 0x8000u ? 0xFFFFu : 0x8000u;
        key[i] = l[i] == -INFINITY ? 0u : h << 16 | (0xFFFFu - e);
      } else {
        const uint64_t k = (uint64_t)ordered(__float_as_uint(l[i])) << 12 | (4095u - e);
        key[i] = l[i] == -INFINITY ? 0.0 : (double)k;
      }
    }
    KEY pick = 0;           // lane j: the j-th choice's key
    for (int j = 0; j < p.topk; ++j) {
      KEY best = key[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) best = larger(best, key[i]);
      const KEY most = wave_max_of(best);
      if (most == 0) break;   // the same in every lane: none left
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = key[i] == most ? (KEY)0 : key[i];
      pick = lane == j ? most : pick;
    }
    if (pick != 0) {
      if constexpr (KIND == KEY16) {
        mine = (int)(0xFFFFu - (pick & 0xFFFFu));
        uint32_t h = pick >> 16;
        h ^= h & 0x8000u ? 0x8000u : 0xFFFFu;
        if constexpr (TYPE == TYPE_BF16) lj = clean(__uint_as_float(h << 16));
        else lj = clean((float)__builtin_bit_cast(_Float16, (uint16_t)h));
      } else {
        const uint64_t k = (uint64_t)pick;
        mine = (int)(4095u - (uint32_t)(k & 4095u));
        lj = __uint_as_float(unordered((uint32_t)(k >> 12)));
      }
    }
  }
  float w;
  if (p.renorm) w = chosen_share(lj, p.sigmoid);
  else if (mine < 0) w = 0.f;
  else w = p.sigmoid ? sigmoid(lj) : expf(lj - top) / total;
  if (lane < p.topk) {
    p.ids[(int64_t)t * p.topk + lane] = mine;
    p.w[(int64_t)t * p.topk + lane] = mine >= 0 ? w * p.scale : 0.f;
  }
}

// Gradient of the logits for the chosen ids and the gradient dw of their
// weights. With g_j = scale * dw_j, p the scores, u the renormalised shares:
//   softmax           dl_e = p_e (G_e - sum_j g_j p_j), G_e = g_j at e = id_j, else 0
//   softmax, renorm   dl_j = u_j (g_j - sum g u)
//   sigmoid           dl_j = g_j s_j (1 - s_j)
//   sigmoid, renorm   dl_j = u_j (1 - s_j) (g_j - sum g u)
// and 0 for experts not chosen in the last three. Ids outside [0, E) take no
// part; an id given twice adds up.
// One wave per token; a lane writes V adjacent experts at a time (V = 8, 16
// bytes and more, where rows allow it). The chosen experts' values are put in
// their places of 64 V zeros in LDS: side by side 5.1 us for 8192 tokens of 384
// experts, 7.1 for 2000 of 4096, top-32 (k comparisons for each of a lane's
// experts: 7.0 and 30). The bytes bound the large rows, the wave's instructions
// the small. The softmax's own gradient (no renorm) reads its row three times,
// twice a value a lane at a time: 12.3 us for 8192 tokens of 384, 87 for 8192 of
// 4096, top-32, where the bytes take 2.5 and 27.
template <int TYPE, int V>
__global__ __launch_bounds__(256) void router_topk_grad(RouterParams p) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= p.T) return;
  __shared__ __align__(32) float parts[4][64 * V];   // a wave's part of the row
  float* part = (float*)__builtin_assume_aligned(parts[threadIdx.x >> 6], 4 * V);
  const int64_t row = (int64_t)t * p.ld;
  int id = -1;
  float lj = -INFINITY, g = 0.f;
  if (lane < p.topk) {
    id = p.ids[(int64_t)t * p.topk + lane];
    g = p.dw[(int64_t)t * p.topk + lane] * p.scale;
    if (id < 0 || id >= p.E) id = -1;
    if (id >= 0) lj = clean(load1<TYPE>(p.logits, row + id));
    if (lj == -INFINITY) id = -1, g = 0.f;
  }
  float top = 0.f, total = 1.f, dot = 0.f, d = 0.f;
  const bool dense = !p.sigmoid && !p.renorm;
  if (p.renorm) {
    const float u = chosen_share(lj, p.sigmoid);
    dot = wave_sum_of(g * u);
    d = u * (g - dot);
    if (p.sigmoid && id >= 0) d *= sigmoid(-lj);
  } else if (p.sigmoid) {
    d = id >= 0 ? g * sigmoid(lj) * sigmoid(-lj) : 0.f;
  } else {
    d = g;
    top = -INFINITY;
    for (int e = lane; e < p.E; e += 64) top = fmaxf(top, clean(load1<TYPE>(p.logits, row + e)));
    top = wave_max_of(top);
    if (top == -INFINITY) top = 0.f;
    total = 0.f;
    for (int e = lane; e < p.E; e += 64) total += expf(clean(load1<TYPE>(p.logits, row + e)) - top);
    total = wave_sum_of(total);
    if (total == 0.f) total = 1.f;
    dot = wave_sum_of(id >= 0 ? g * (expf(lj - top) / total) : 0.f);
  }
  float own = 0.f;   // of every place that names the lane's id
  for (int j = 0; j < p.topk; ++j) {
    const float x = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(d), j));
    own += __builtin_amdgcn_readlane(id, j) == id ? x : 0.f;
  }
  for (int base = 0; base < p.E; base += 64 * V) {
    const int e0 = base + V * lane;
    float v[V] = {};
    float* at0 = part + V * lane;
    __builtin_memcpy(at0, v, sizeof v);
    wave_sync();
    if (id >= base && id < base + 64 * V) part[id - base] = own;
    wave_sync();
    __builtin_memcpy(v, at0, sizeof v);
    wave_sync();
    if (e0 >= p.E) continue;
    if (dense) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        v[i] = expf(clean(load1<TYPE>(p.logits, row + e0 + i)) - top) / total * (v[i] - dot);
    }
    const int64_t at = (int64_t)t * p.d_ld + e0;
    if constexpr (V == 1) {
      store1<TYPE>(p.dlogits, at, v[0]);
    } else if constexpr (TYPE == TYPE_F32) {
      f32x4_t* o = reinterpret_cast<f32x4_t*>(static_cast<float*>(p.dlogits) + at);
      o[0] = f32x4_t{v[0], v[1], v[2], v[3]};
      o[1] = f32x4_t{v[4], v[5], v[6], v[7]};
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (TYPE == TYPE_BF16) {
          w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        } else {
          const f16x2_t h = {(_Float16)v[2 * i], (_Float16)v[2 * i + 1]};
          w[i] = __builtin_bit_cast(uint32_t, h);
        }
      }
      *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p.dlogits) + at) = u32x4_t{w[0], w[1], w[2], w[3]};
    }
  }
}

// Places by E, in kernel us for 8192 tokens, top-8 (BF16 softmax / FP32 sigmoid
// with a bias), at both ends of each step:
//   1    up to 64      5.2 / 11
//   4    65 .. 256     6.6 / 14   ..  6.9 / 16
//   6    257 .. 384    7.8 / 19   ..  8.0 / 20
//   16   385 .. 1024    13 / 33   ..   14 / 44
//   64   1025 .. 4096   37 / 221  ..   69 / 381
// A step costs most just past its border: 385 experts take 16 places where 7
// would do, 1025 take 64 where 17 would.
template <int TYPE, int KIND>
hipError_t topk_for(const RouterParams& p, hipStream_t s) {
  const unsigned g = (unsigned)((p.T + 3) / 4);
  if (p.E <= 64) router_topk<TYPE, 1, KIND><<<g, 256, 0, s>>>(p);
  else if (p.E <= 256) router_topk<TYPE, 4, KIND><<<g, 256, 0, s>>>(p);
  else if (p.E <= 384) router_topk<TYPE, 6, KIND><<<g, 256, 0, s>>>(p);
  else if (p.E <= 1024) router_topk<TYPE, 16, KIND><<<g, 256, 0, s>>>(p);
  else router_topk<TYPE, 64, KIND><<<g, 256, 0, s>>>(p);
  return hipGetLastError();
}

template <int TYPE>
hipError_t grad_for(const RouterParams& p, hipStream_t s) {
  const unsigned g = (unsigned)((p.T + 3) / 4);
  if (p.E % 8 == 0 && p.d_ld % 8 == 0 && (uintptr_t)p.dlogits % 16 == 0) router_topk_grad<TYPE, 8><<<g, 256, 0, s>>>(p);
  else router_topk_grad<TYPE, 1><<<g, 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_router_topk(const RouterParams& p, int type, hipStream_t s) {
  if (type == TYPE_BF16) return p.bias ? topk_for<TYPE_BF16, KEYB>(p, s) : topk_for<TYPE_BF16, KEY16>(p, s);
  if (type == TYPE_F16) return p.bias ? topk_for<TYPE_F16, KEYB>(p, s) : topk_for<TYPE_F16, KEY16>(p, s);
  return p.bias ? topk_for<TYPE_F32, KEYB>(p, s) : topk_for<TYPE_F32, KEY32>(p, s);
}

hipError_t launch_router_topk_grad(const RouterParams& p, int type, hipStream_t s) {
  if (type == TYPE_BF16) return grad_for<TYPE_BF16>(p, s);
  if (type == TYPE_F16) return grad_for<TYPE_F16>(p, s);
  return grad_for<TYPE_F32>(p, s);
}

}  // namespace moe

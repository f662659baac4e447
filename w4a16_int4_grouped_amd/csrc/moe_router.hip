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
// ..; a round takes each lane's best, then the wave's. A wave's work is k
// rounds of dependent lane exchanges, so latency bounds small T.
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

// -inf and NaN become -inf (not chosen), +inf the largest finite value.
__device__ __forceinline__ float clean(float l) { return l >= -kMax ? fminf(l, kMax) : -INFINITY; }

template <class T>
__device__ __forceinline__ T wave_max_of(T v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const T u = __shfl_xor(v, o, 64);
    v = u > v ? u : v;
  }
  return v;
}
template <class T>
__device__ __forceinline__ T wave_sum_of(T v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
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

// VPL: experts per lane. KEY: float (the logits), double (score + bias).
template <int TYPE, int VPL, class KEY>
__global__ __launch_bounds__(256) void router_topk(RouterParams p) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= p.T) return;
  const int64_t row = (int64_t)t * p.ld;
  float l[VPL];
  KEY key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < p.E ? clean(load1<TYPE>(p.logits, row + e)) : -INFINITY;
  }
  float top = 0.f, total = 1.f;
  if (!p.sigmoid && (sizeof(KEY) == 8 || !p.renorm)) {
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
  if constexpr (sizeof(KEY) == 8) {
    double sum = 1.0;
    if (!p.sigmoid) {
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum += exp((double)l[i] - (double)top);
      sum = wave_sum_of(sum);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 64 * i;
      const double s = p.sigmoid ? 1.0 / (1.0 + exp(-(double)l[i])) : exp((double)l[i] - (double)top) / sum;
      const double k = e < p.E ? s + (double)p.bias[e] : 0.0;
      key[i] = e < p.E && l[i] != -INFINITY && k >= -1.7976931348623157e308 ? k : -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = l[i];
  }
  int mine = -1;   // lane j: the j-th choice
  for (int j = 0; j < p.topk; ++j) {
    KEY best = key[0];
    int at = lane;
#pragma unroll
    for (int i = 1; i < VPL; ++i)
      if (key[i] > best) best = key[i], at = lane + 64 * i;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const KEY k = __shfl_xor(best, o, 64);
      const int a = __shfl_xor(at, o, 64);
      if (k > best || (k == best && a < at)) best = k, at = a;
    }
    if (best == -INFINITY) break;   // the same in every lane: none left
    if (lane == j) mine = at;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (at == lane + 64 * i) key[i] = -INFINITY;
  }
  const float lj = mine >= 0 ? clean(load1<TYPE>(p.logits, row + mine)) : -INFINITY;
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
template <int TYPE>
__global__ __launch_bounds__(256) void router_topk_grad(RouterParams p) {
  extern __shared__ float rows[];   // [4][E]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * (blockDim.x >> 6) + wave;
  const bool live = t < p.T;
  float* G = rows + wave * p.E;
  for (int e = lane; e < p.E; e += 64) G[e] = 0.f;
  const int64_t row = (int64_t)t * p.ld;
  int id = -1;
  float lj = -INFINITY, g = 0.f;
  if (live && lane < p.topk) {
    id = p.ids[(int64_t)t * p.topk + lane];
    if (id < 0 || id >= p.E) id = -1;
    if (id >= 0) {
      lj = clean(load1<TYPE>(p.logits, row + id));
      g = p.dw[(int64_t)t * p.topk + lane] * p.scale;
      if (lj == -INFINITY) id = -1, g = 0.f;
    }
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
    if (live)
      for (int e = lane; e < p.E; e += 64) top = fmaxf(top, clean(load1<TYPE>(p.logits, row + e)));
    top = wave_max_of(top);
    if (top == -INFINITY) top = 0.f;
    total = 0.f;
    if (live)
      for (int e = lane; e < p.E; e += 64) total += expf(clean(load1<TYPE>(p.logits, row + e)) - top);
    total = wave_sum_of(total);
    if (total == 0.f) total = 1.f;
    dot = wave_sum_of(id >= 0 ? g * (expf(lj - top) / total) : 0.f);
  }
  // the lanes of one id add up in lane order, the first of them writes
  float sum = 0.f;
  bool first = id >= 0;
  for (int j = 0; j < p.topk; ++j) {
    const int other = __shfl(id, j, 64);
    const float v = __shfl(d, j, 64);
    if (other == id) {
      sum += v;
      if (j < lane) first = false;
    }
  }
  __syncthreads();   // zeros of every lane before the chosen entries
  if (first) G[id] = sum;
  __syncthreads();
  if (!live) return;
  for (int e = lane; e < p.E; e += 64) {
    float v = G[e];
    if (dense) v = expf(clean(load1<TYPE>(p.logits, row + e)) - top) / total * (v - dot);
    store1<TYPE>(p.dlogits, (int64_t)t * p.d_ld + e, v);
  }
}

template <int TYPE, class KEY>
hipError_t topk_for(const RouterParams& p, hipStream_t s) {
  const unsigned g = (unsigned)((p.T + 3) / 4);
  if (p.E <= 64) router_topk<TYPE, 1, KEY><<<g, 256, 0, s>>>(p);
  else if (p.E <= 256) router_topk<TYPE, 4, KEY><<<g, 256, 0, s>>>(p);
  else if (p.E <= 512) router_topk<TYPE, 8, KEY><<<g, 256, 0, s>>>(p);
  else if (p.E <= 1024) router_topk<TYPE, 16, KEY><<<g, 256, 0, s>>>(p);
  else router_topk<TYPE, 64, KEY><<<g, 256, 0, s>>>(p);
  return hipGetLastError();
}

template <int TYPE>
hipError_t grad_for(const RouterParams& p, hipStream_t s) {
  // a token's row of FP32 in LDS: 4 tokens a workgroup up to 1024 experts (16 KB), one above
  const int waves = p.E <= 1024 ? 4 : 1;
  router_topk_grad<TYPE><<<(unsigned)((p.T + waves - 1) / waves), 64 * waves, (size_t)waves * p.E * 4, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_router_topk(const RouterParams& p, int type, hipStream_t s) {
  if (type == TYPE_BF16) return p.bias ? topk_for<TYPE_BF16, double>(p, s) : topk_for<TYPE_BF16, float>(p, s);
  if (type == TYPE_F16) return p.bias ? topk_for<TYPE_F16, double>(p, s) : topk_for<TYPE_F16, float>(p, s);
  return p.bias ? topk_for<TYPE_F32, double>(p, s) : topk_for<TYPE_F32, float>(p, s);
}

hipError_t launch_router_topk_grad(const RouterParams& p, int type, hipStream_t s) {
  if (type == TYPE_BF16) return grad_for<TYPE_BF16>(p, s);
  if (type == TYPE_F16) return grad_for<TYPE_F16>(p, s);
  return grad_for<TYPE_F32>(p, s);
}

}  // namespace moe

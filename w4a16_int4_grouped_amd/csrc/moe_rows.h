// Helpers of the kernels that work on rows: 16-byte pieces of a row in its
// type, places among rows, single values, and what a wave's lanes have in
// common (largest, sum) by lane moves in registers.
#pragma once

#include <type_traits>

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

// Eight values as loaded; values are read once, past the caches.
template <int TYPE>
struct Raw8 {
  u32x4_t w[TYPE == TYPE_F32 ? 2 : 1];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (auto& x : w) x = u32x4_t{};
  }
  __device__ __forceinline__ void load(const void* x, int64_t at) {
    const u32x4_t* p =
        reinterpret_cast<const u32x4_t*>(static_cast<const char*>(x) + at * (TYPE == TYPE_F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (TYPE == TYPE_F32 ? 2 : 1); ++i) w[i] = __builtin_nontemporal_load(p + i);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (TYPE == TYPE_F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i >> 2][i & 3]);
    } else if constexpr (TYPE == TYPE_BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(w[0][i]), v[2 * i + 1] = bf16_hi(w[0][i]);
    } else {
      const f16x8_t h = __builtin_bit_cast(f16x8_t, w[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
    }
  }
};

// PAST: past the caches.
template <bool PAST, class V>
__device__ __forceinline__ void store_vec(void* p, V v) {
  if constexpr (PAST) __builtin_nontemporal_store(v, static_cast<V*>(p));
  else *static_cast<V*>(p) = v;
}
template <int TYPE, bool PAST = false>
__device__ __forceinline__ void store8(void* x, int64_t at, const float (&v)[8]) {
  if constexpr (TYPE == TYPE_F32) {
    f32x4_t* p = reinterpret_cast<f32x4_t*>(static_cast<float*>(x) + at);
    store_vec<PAST>(p, f32x4_t{v[0], v[1], v[2], v[3]});
    store_vec<PAST>(p + 1, f32x4_t{v[4], v[5], v[6], v[7]});
  } else if constexpr (TYPE == TYPE_BF16) {
    store_vec<PAST>(static_cast<uint16_t*>(x) + at,
                    u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                            pack_bf16x2(v[6], v[7])});
  } else {
    f16x8_t h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (_Float16)v[i];
    store_vec<PAST>(static_cast<_Float16*>(x) + at, h);
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

}  // namespace
}  // namespace moe

// FP32 steps of the selection kernels, and typed row loads and stores.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

namespace moe {

// A float as an unsigned integer in the same order (every key of a number is above 1;
// 0 is free for "none"), and back.  -inf .. +inf; not for NaN.
__device__ __forceinline__ uint32_t float_key(float f) {
  const uint32_t u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_float(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}

// 1 / (1 + exp(-l)) of two logits, the exponential in Cody & Waite's reduction and a Taylor
// polynomial of degree 7, every step one IEEE FP32 operation: the bits of the router
// kernels' sigmoid, two lanes to an instruction.  Their rint is here the sum with 1.5 * 2^23
// (whose low bits are then the integer), their ldexp an addition to the exponent: with -l
// held to [-80, 89] (below, exp(-l) vanishes in 1 + exp(-l)) the integer is in [-115, 128],
// so half the result is a normal number, and the factor 2 joins the final sum exactly.
// CLAMP: false where the caller has seen |l| <= 80.
template <bool CLAMP>
__device__ __forceinline__ float2 sigmoid_steps2(float l0, float l1) {
  float2 x = make_float2(-l0, -l1);
  if constexpr (CLAMP)
    x = make_float2(fminf(fmaxf(x.x, -80.0f), 89.0f), fminf(fmaxf(x.y, -80.0f), 89.0f));
  auto both = [](float c) { return make_float2(c, c); };
  const float2 t = __fmul2_rn(x, both(1.44269502162933349609375f));
  const float2 m = __fadd2_rn(t, both(12582912.0f));
  const float2 n = __fadd2_rn(m, both(-12582912.0f));
  float2 r = __ffma2_rn(n, both(-0.693145751953125f), x);
  r = __ffma2_rn(n, both(-1.428606765330187e-06f), r);
  float2 p = both(1.0f / 5040.0f);
  p = __ffma2_rn(p, r, both(1.0f / 720.0f));
  p = __ffma2_rn(p, r, both(1.0f / 120.0f));
  p = __ffma2_rn(p, r, both(1.0f / 24.0f));
  p = __ffma2_rn(p, r, both(1.0f / 6.0f));
  p = __ffma2_rn(p, r, both(0.5f));
  p = __ffma2_rn(p, r, both(1.0f));
  p = __ffma2_rn(p, r, both(1.0f));
  auto half_exp = [](float p, float m) {  // p 2^(n - 1)
    return __int_as_float(__float_as_int(p) + (int)((uint32_t)__float_as_int(m) << 23) - (1 << 23));
  };
  const float2 e = make_float2(half_exp(p.x, m.x), half_exp(p.y, m.y));
  const float2 d = __ffma2_rn(e, both(2.0f), both(1.0f));
  return make_float2(__frcp_rn(d.x), __frcp_rn(d.y));
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
  else return __float2bfloat16_rn(v);
}

// N consecutive values (16-byte accesses where they fill them; p aligned to N * sizeof(T),
// at most 16 bytes)
template <typename T, int N>
__device__ __forceinline__ void load_floats(const T* p, float (&v)[N]) {
  constexpr int B = N * (int)sizeof(T);
  union {
    T t[N];
    uint4 q[(B + 15) / 16];
    uint2 d;
    uint32_t w;
    uint16_t h;
  } u;
  if constexpr (B >= 16) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) u.q[i] = reinterpret_cast<const uint4*>(p)[i];
  } else if constexpr (B == 8) {
    u.d = *reinterpret_cast<const uint2*>(p);
  } else if constexpr (B == 4) {
    u.w = *reinterpret_cast<const uint32_t*>(p);
  } else {
    u.h = *reinterpret_cast<const uint16_t*>(p);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = to_float(u.t[i]);
}

template <typename T, int N>
__device__ __forceinline__ void store_floats(T* p, const float (&v)[N]) {
  constexpr int B = N * (int)sizeof(T);
  union {
    T t[N];
    uint4 q[(B + 15) / 16];
    uint2 d;
    uint32_t w;
    uint16_t h;
  } u;
#pragma unroll
  for (int i = 0; i < N; ++i) u.t[i] = from_float<T>(v[i]);
  if constexpr (B >= 16) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) reinterpret_cast<uint4*>(p)[i] = u.q[i];
  } else if constexpr (B == 8) {
    *reinterpret_cast<uint2*>(p) = u.d;
  } else if constexpr (B == 4) {
    *reinterpret_cast<uint32_t*>(p) = u.w;
  } else {
    *reinterpret_cast<uint16_t*>(p) = u.h;
  }
}

// every row start (base + t * ld) allows N-value accesses
template <typename T, int N>
__device__ __forceinline__ bool rows_aligned(const void* base, long long ld) {
  constexpr int B = N * (int)sizeof(T) < 16 ? N * (int)sizeof(T) : 16;
  return reinterpret_cast<uintptr_t>(base) % B == 0 && (ld * (long long)sizeof(T)) % B == 0;
}

}  // namespace moe

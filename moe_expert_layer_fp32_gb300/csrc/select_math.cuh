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

// 1 / (1 + exp(-l)) with the exponential in Cody & Waite's reduction and a Taylor
// polynomial of degree 7, every step one IEEE FP32 operation: the bits of the router
// kernels' sigmoid.  They scale by 2^n with ldexp; here 2^n is applied as two exact
// powers of two (n in [-150, 129]), which differs only where exp(-l) is below 2^-126
// and so vanishes in 1 + exp(-l).
__device__ __forceinline__ float sigmoid_steps(float l) {
  float x = fminf(fmaxf(-l, -104.0f), 89.0f);
  const float n = rintf(__fmul_rn(x, 1.44269502162933349609375f));
  float r = fmaf(-n, 0.693145751953125f, x);
  r = fmaf(-n, 1.428606765330187e-06f, r);
  float p = 1.0f / 5040.0f;
  p = fmaf(p, r, 1.0f / 720.0f);
  p = fmaf(p, r, 1.0f / 120.0f);
  p = fmaf(p, r, 1.0f / 24.0f);
  p = fmaf(p, r, 1.0f / 6.0f);
  p = fmaf(p, r, 0.5f);
  p = fmaf(p, r, 1.0f);
  p = fmaf(p, r, 1.0f);
  const int i = (int)n, h = i >> 1;
  const float e = p * __int_as_float((h + 127) << 23) * __int_as_float((i - h + 127) << 23);
  return __frcp_rn(__fadd_rn(1.0f, e));
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

// Device steps of the 4-bit row quantisation: pieces of eight values, their block maxima and
// codes, and where a row comes from.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "mx4.cuh"
#include "select_math.cuh"

namespace moe {

// Eight consecutive values as they were loaded, and the FP32 bits (sign cleared) of a
// magnitude that has the largest one's exponent, over the four lanes of a block.
template <typename Tin>
struct Piece {
  float v[8];
  __device__ __forceinline__ void load(const Tin* p) { load_floats<Tin, 8>(p, v); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  }
  __device__ __forceinline__ uint32_t block_max() const {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
    return max(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
  }
  __device__ __forceinline__ void scaled(float inv, float (&q)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v[i] * inv;
  }
};

// bf16: magnitudes order as 16-bit integers, two to an instruction (the widened form costs
// twice the integer instructions, which bound the row images' kernel)
template <>
struct Piece<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t block_max() const {
    constexpr uint32_t M = 0x7FFF7FFFu;
    uint32_t a = __vmaxu2(__vmaxu2(r.x & M, r.y & M), __vmaxu2(r.z & M, r.w & M));
    a = __vmaxu2(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
    a = __vmaxu2(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
    return max(a << 16, a & 0xFFFF0000u);
  }
  __device__ __forceinline__ void scaled(float inv, float (&q)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[2 * i] = bf16_lo(w[i]) * inv;
      q[2 * i + 1] = bf16_hi(w[i]) * inv;
    }
  }
};

// The lane's piece to codes; `byte`: the block's scale (the same in its four lanes).
template <typename Tin>
__device__ __forceinline__ uint32_t quantize8(const Piece<Tin>& p, uint32_t& byte) {
  byte = mx4_scale_byte(p.block_max());
  float q[8];
  p.scaled(mx4_inverse_scale(byte), q);
  const uint32_t c = mx4_encode8(q);
  return byte == 255u ? 0u : c;
}

// Four rows' pieces at once; returns the lane's four scale bytes, row i's in byte i.  (A NaN
// block's codes are left as they fall: its scale decides.)
template <typename Tin>
__device__ __forceinline__ uint32_t quantize4x8(const Piece<Tin> (&p)[4], uint32_t (&c)[4]) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t byte;
    c[i] = quantize8(p[i], byte);
    w |= byte << (8 * i);
  }
  return w;
}
// bf16: two rows' maxima and scale bytes ride in the halves of one register.  Integer
// instructions bound this step; so packed they are a third fewer.
__device__ __forceinline__ uint32_t quantize4x8(const Piece<__nv_bfloat16> (&p)[4],
                                                uint32_t (&c)[4]) {
  constexpr uint32_t M = 0x7FFF7FFFu;
  uint32_t m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m[i] = __vmaxu2(__vmaxu2(p[i].r.x & M, p[i].r.y & M), __vmaxu2(p[i].r.z & M, p[i].r.w & M));
  uint32_t b[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t a = __vmaxu2(__byte_perm(m[2 * h], m[2 * h + 1], 0x5410),
                          __byte_perm(m[2 * h], m[2 * h + 1], 0x7632));
    a = __vmaxu2(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
    a = __vmaxu2(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
    const uint32_t e = (a >> 7) & 0x00FF00FFu;  // exponents
    b[h] = __vmaxu2(e, 0x00020002u) - 0x00020002u;
    b[h] |= ((e + 0x00010001u) & 0x01000100u) >> 7;  // 255 - 2 -> 255
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t byte = (i & 1) ? b[i >> 1] >> 16 : b[i >> 1] & 0xFFFFu;
    float q[8];
    p[i].scaled(__uint_as_float(0x7F000000u - (byte << 23)), q);  // 2^(127 - byte)
    c[i] = mx4_encode8(q);
  }
  return __byte_perm(b[0], b[1], 0x6420);
}

// A lane's four bytes are four rows' scales of one block.  The first lane of each half
// k-block collects the words of the other three blocks and turns the 4 x 4 bytes: one word
// of four scales per row.
__device__ __forceinline__ void turn_scales(uint32_t b0, uint4& w) {
  const uint32_t b1 = __shfl_down_sync(0xFFFFFFFFu, b0, 4);
  const uint32_t b2 = __shfl_down_sync(0xFFFFFFFFu, b0, 8);
  const uint32_t b3 = __shfl_down_sync(0xFFFFFFFFu, b0, 12);
  const uint32_t lo01 = __byte_perm(b0, b1, 0x5140), hi01 = __byte_perm(b0, b1, 0x7362);
  const uint32_t lo23 = __byte_perm(b2, b3, 0x5140), hi23 = __byte_perm(b2, b3, 0x7362);
  w = make_uint4(__byte_perm(lo01, lo23, 0x5410), __byte_perm(lo01, lo23, 0x7632),
                 __byte_perm(hi01, hi23, 0x5410), __byte_perm(hi01, hi23, 0x7632));
}

// The piece of `col` (of K) of a source row, SwiGLU applied; zeros past K or where !in.
template <typename Tin, int SRC, typename P>
__device__ __forceinline__ void load_piece(P& p, const Tin* row, int col, int K, bool in) {
  if (!in) {
    p.zero();
  } else if constexpr (SRC == 2) {
    float up[8];
    load_floats<Tin, 8>(row + col, p.v);
    load_floats<Tin, 8>(row + K + col, up);
#pragma unroll
    for (int j = 0; j < 8; ++j) p.v[j] = __fmul_rn(silu_f32(p.v[j]), up[j]);
  } else {
    p.load(row + col);
  }
}

// First element of the source row of operand row r.
template <typename Tin, int SRC>
__device__ __forceinline__ const Tin* source_row(const Tin* x, const int32_t* row_of, int k, int T,
                                                 int K, int r, int32_t* status) {
  long long src = r;
  if constexpr (SRC == 1) {
    const int slot = row_of[r];
    src = slot >= 0 ? slot / k : T;
    if (src >= T) {
      flag_error(status, MOE_ERR_DEVICE_CHECK);
      src = 0;
    }
  }
  return x + (size_t)src * (SRC == 2 ? 2 * (size_t)K : (size_t)K);
}

}  // namespace moe

// Microscaled 4-bit floating point (MXFP4): the block format, and the layout in which
// the grouped product streams its operands.
//
// A block is 32 consecutive values of a row over K.  Its scale is 2^(byte - 127), one byte
// (255: NaN); each value is a 4-bit code, sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6.  Two
// codes share a byte, the even one in the low half.  (OCP Microscaling Formats v1.0:
// element E2M1, scale E8M0, block size 32.)
//
// Operand images.  The product reads shared-memory images that one bulk copy (or tensor load of
// 1024-byte lines) brings in:
// rows of 128 bytes (256 codes, a k-block) whose 16-byte chunk c sits at c ^ (row & 7)
// (the MMA's 128-byte swizzle), and the scales of 128 rows x 128 K as 512 bytes, row r's
// four scales at (r % 32) * 16 + (r / 32) * 4 (the order in which tensor memory takes
// them).
//   weights  per (expert, 128 output columns, k-block): 16384 bytes of codes, then 1024 of
//            scales (two halves of the k-block)
//   rows     the rows of an expert in tiles of at most tile_rows (by the form of the product),
//            evenly cut to a multiple of 16; a tile has a slot of tile_rows rows, in which its
//            k-blocks follow one another (the tile's own padded rows x 128 bytes each).  The
//            scales of a tile's k-block b are at slot (tile * KB + b) of 2048 bytes,
//            [128-row half][half k-block][512]
// Padding rows are never written; they only reach accumulator columns that are not stored.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "kernels.cuh"

namespace moe {

constexpr int kMx4KB = 256;           // values of a k-block: one 128-byte row of codes
constexpr int kMx4PairRows = 224;     // rows of the largest tile (accumulator columns) of a
                                      // pair of CTAs, which batches of many rows run on,
constexpr int kMx4SingleRows = 64;    // and of a single CTA
constexpr int kMx4WTile = 128;        // output columns of a weight tile (accumulator lanes)
constexpr int kMx4WBytes = kMx4WTile * 128 + 1024;  // image of a weight tile's k-block
constexpr int kMx4SfSlot = 2048;      // scales of a row tile's k-block

__host__ __device__ inline int mx4_kblocks(int K) { return (K + kMx4KB - 1) / kMx4KB; }

// How an expert's m rows are cut: n tiles of `step` rows (a multiple of 16), the last shorter.
struct Mx4Cut {
  int n, step;
};
__host__ __device__ inline Mx4Cut mx4_cut(int m, int tile_rows) {
  Mx4Cut c;
  c.n = m / tile_rows + (m % tile_rows != 0);
  c.step = c.n > 0 ? (m / c.n + (m % c.n != 0) + 15) / 16 * 16 : 16;
  return c;
}

// Tiles of R rows among E experts, at most.
inline long long mx4_max_tiles(long long R, int E, int tile_rows) {
  const long long with = R < E ? R : E;  // experts that can have rows
  return R / tile_rows + with;
}

// Bytes of a tile's slot of codes, and of its scales.
__host__ __device__ inline size_t mx4_slot(int K, int tile_rows) {
  return (size_t)mx4_kblocks(K) * tile_rows * 128;
}
__host__ __device__ inline size_t mx4_sf_slots(int K) { return (size_t)mx4_kblocks(K) * kMx4SfSlot; }

// Prefix tables of a grouped operand in shared memory, from offsets [E+1]; every thread of
// the block calls it (blockDim a multiple of 32, at least 32).  Returns false (and flags) if
// the offsets are not 0 = o_0 <= ... <= o_E = R.
struct Mx4Tables {
  int off[kMaxE + 1];    // first row of each expert
  int tile[kMaxE + 1];   // its first row tile
  int step[kMaxE];       // rows of its tiles (the last may have fewer)
  int ok;
};

__device__ __forceinline__ bool mx4_build_tables(Mx4Tables& s, const int32_t* __restrict__ offsets,
                                                 int E, int R, int32_t* status,
                                                 int tile_rows) {
  for (int e = threadIdx.x; e <= E; e += blockDim.x) s.off[e] = offsets[e];
  __syncthreads();
  if (threadIdx.x < 32) {  // one warp scans, 32 experts a step
    const int lane = threadIdx.x;
    int tile = 0;
    bool ok = s.off[0] == 0 && s.off[E] == R;
    for (int b = 0; b < E; b += 32) {
      const int e = b + lane;
      int m = 0;
      if (e < E) {
        const int lo = s.off[e], hi = s.off[e + 1];
        if (lo < 0 || hi < lo || hi > R) ok = false;
        else m = hi - lo;
      }
      const Mx4Cut cut = mx4_cut(m, tile_rows);
      int n = cut.n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int nu = __shfl_up_sync(0xFFFFFFFFu, n, o);
        if (lane >= o) n += nu;
      }
      if (e < E) {
        s.tile[e] = tile + n - cut.n;
        s.step[e] = cut.step;
      }
      tile += __shfl_sync(0xFFFFFFFFu, n, 31);
    }
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (lane == 0) {
      s.tile[E] = tile;
      s.ok = ok;
      if (!ok) flag_error(status, MOE_ERR_DEVICE_CHECK);
    }
  }
  __syncthreads();
  return s.ok != 0;
}

// largest e in [0, E) with table[e] <= v (experts without entries share the next value)
__device__ __forceinline__ int mx4_find(const int* table, int E, int v) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (table[mid] <= v) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// A row tile: its expert, first row and rows.  Walks keep the expert of the tile before (any
// but the first costs a step or two; a search and the cut's divisions for every tile, on the
// one thread that issues the MMAs, cost 1900 cycles a unit).
struct Mx4Tile {
  int e, row0, rows, rows16;
};
__device__ __forceinline__ Mx4Tile mx4_tile_in(int e, int tile, const Mx4Tables& tb) {
  Mx4Tile t;
  t.e = e;
  const int step = tb.step[e], first = (tile - tb.tile[e]) * step;
  t.row0 = tb.off[e] + first;
  t.rows = min(step, tb.off[e + 1] - t.row0);
  t.rows16 = (t.rows + 15) & ~15;
  return t;
}
// e: the expert of an earlier tile of the walk (up: of a tile not after this one), or any
// expert not after (up) or not before (down) the tile's
__device__ __forceinline__ Mx4Tile mx4_walk_up(int& e, int tile, const Mx4Tables& tb) {
  while (tb.tile[e + 1] <= tile) ++e;
  return mx4_tile_in(e, tile, tb);
}
__device__ __forceinline__ Mx4Tile mx4_walk_down(int& e, int tile, const Mx4Tables& tb) {
  while (tb.tile[e] > tile) --e;
  return mx4_tile_in(e, tile, tb);
}

// Scale byte of a block whose largest magnitude has the FP32 bits `amax` (sign cleared):
// the exponent of the block's largest value becomes the format's (4 = 2^2), clamped to the
// smallest scale; infinities and NaN give 255.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax) {
  const uint32_t e = amax >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^(127 - byte), which takes the block's values into the code's range (0 for a NaN block,
// whose codes are then 0 or, for its NaNs, whatever the conversion gives: its scale decides)
__device__ __forceinline__ float mx4_inverse_scale(uint32_t byte) {
  if (byte == 255u) return 0.0f;
  return __uint_as_float((254u - byte) << 23);
}
// 2^(byte - 127); 255: NaN
__device__ __forceinline__ float mx4_scale(uint32_t byte) {
  if (byte == 255u) return __uint_as_float(0x7FC00000u);
  return byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

// Eight values (already scaled) to eight codes, the first in the lowest four bits: to
// nearest, ties to even, at most 6.
__device__ __forceinline__ uint32_t mx4_encode8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The eight values of mx4_encode8's codes times the block's scale, as bf16 (exact).  A
// magnitude's bf16 bytes come from two eight-byte tables by byte permutes; the sign joins
// in FP32, where the scale multiplies.
__device__ __forceinline__ uint4 mx4_decode8_bf16(uint32_t codes, float scale) {
  const uint32_t mag = codes & 0x77777777u;
  uint32_t o[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // four codes a step
    const uint32_t sel = mag >> (16 * h);
    // 0 0.5 1 1.5 | 2 3 4 6 = 0000 3F00 3F80 3FC0 | 4000 4040 4080 40C0
    const uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, sel);
    const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, sel);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint32_t two = __byte_perm(lo, hi, p == 0 ? 0x5140 : 0x7362);  // two bf16
      const int b = 16 * h + 8 * p;                                        // first code's bit
      const float v0 = __uint_as_float((two << 16) | ((codes << (28 - b)) & 0x80000000u));
      const float v1 = __uint_as_float((two & 0xFFFF0000u) | ((codes << (24 - b)) & 0x80000000u));
      o[2 * h + p] = pack_bf16x2(v0 * scale, v1 * scale);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace moe

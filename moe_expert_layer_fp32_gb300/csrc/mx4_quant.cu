// Microscaled 4-bit quantisation: rows (moe_mx4_quantize), an expert operand's row tiles
// (the first half of moe_mx4_expert_product), and weight images (moe_mx4_pack,
// moe_mx4_prepack).  Format and layouts: mx4.cuh.
//
// Per block of 32 values v: a = max |v|, the scale 2^(floor(log2 a) - 2) (so that a lands
// in [4, 8)), the codes v / scale rounded to nearest even and cut at 6.  A power of two
// divides exactly, so the only rounding is the one to the code.
//
// Memory-bound: 8 values a lane (one or two 16-byte loads), four lanes a block whose
// maximum meets in two shuffles; a warp covers one row's 256-value k-block.  Measured on GB300:
// 32768 x 4096 bf16 rows with their values 90 us for 608 MB, the copy rate (four pieces in
// flight a thread and values by byte permutes: 127 us without); the row images of 131072 x
// 2048 117 us (ncu) for 537 MB read and 285 written, of which half is still in L2 when the
// product starts; integer instructions are next (ALU pipe two thirds busy).
#include <type_traits>

#include "common.cuh"
#include "kernels.cuh"
#include "mx4.cuh"
#include "mx4_rows.cuh"
#include "pdl.cuh"
#include "select_math.cuh"

namespace moe {
namespace {

constexpr int kQThreads = 256;
constexpr int kQWarps = kQThreads / 32;

// ------------------------------------------------------------ logical rows ---
// The pieces of 8 values are numbered row-major; a block of 32 is four neighbouring lanes'.
// Each thread keeps kQUnroll pieces in flight.  DENSE: ld == K.
constexpr int kQUnroll = 4;

template <typename Tin, bool DENSE>
__global__ void __launch_bounds__(kQThreads) quantize_kernel(const Tin* __restrict__ x, long long ld,
                                                             long long n, int per_row,
                                                             uint32_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scales,
                                                             uint4* __restrict__ values) {
  // n is a multiple of 4, so a block is whole or past the end
  const long long base = (long long)blockIdx.x * (kQThreads * kQUnroll) + threadIdx.x;
  Piece<Tin> v[kQUnroll];
#pragma unroll
  for (int q = 0; q < kQUnroll; ++q) {
    const long long i = base + q * kQThreads;
    if (i < n) {
      if constexpr (DENSE) {
        v[q].load(x + i * 8);
      } else {
        const long long row = i / per_row;
        v[q].load(x + row * ld + (i - row * per_row) * 8);
      }
    } else {
      v[q].zero();
    }
  }
#pragma unroll
  for (int q = 0; q < kQUnroll; ++q) {
    const long long i = base + q * kQThreads;
    uint32_t byte;
    const uint32_t c = quantize8(v[q], byte);
    if (i < n) {
      if (codes != nullptr) codes[i] = c;
      if (scales != nullptr && (i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
      if (values != nullptr) values[i] = mx4_decode8_bf16(c, mx4_scale(byte));
    }
  }
}

// ------------------------------------------------------------ operand rows ---
// SRC 0: rows of x.  SRC 1: row r of the operand is row row_of[r] / k of x (the gather of
// the dispatch).  SRC 2: x holds [R, 2K] (gate | up), the operand is silu(gate) * up.
//
// MANY rows: a warp takes the rows rr, rr + 32, rr + 64, rr + 96 of a tile's 128-row half
// over all of K: four loads in flight a lane, and the four rows' scales of a half k-block
// are one 16-byte store.
constexpr int kRowsBlocksPerSm = 4;
template <typename Tin, int SRC>
__global__ void __launch_bounds__(kQThreads, kRowsBlocksPerSm) quantize_rows_kernel(
    const Tin* __restrict__ x, const int32_t* __restrict__ row_of, int k, int T,
    const int32_t* __restrict__ offsets, int E, int R, int K, int tile_rows,
    uint8_t* __restrict__ codes, uint8_t* __restrict__ sf, int32_t* status) {
  __shared__ Mx4Tables tb;
  pdl_wait();               // x, the offsets and the images' last reader: the kernel before
  pdl_launch_dependents();  // the product reads this kernel's images only after its own wait
  if (!mx4_build_tables(tb, offsets, E, R, status, tile_rows)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KB = mx4_kblocks(K);
  const long long items = (long long)tb.tile[E] * 64;  // (tile, half, rr)
  int e = 0;
  for (long long it = (long long)blockIdx.x * kQWarps + warp; it < items;
       it += (long long)gridDim.x * kQWarps) {
    const int tile = (int)(it >> 6), half = (int)(it >> 5) & 1, rr = (int)it & 31;
    const Mx4Tile t = mx4_walk_up(e, tile, tb);
    const int r0 = half * 128 + rr;  // this warp's first row of the tile
    if (r0 >= t.rows) continue;
    const int rows16 = t.rows16;
    const int nr = min(4, (t.rows - r0 + 31) / 32);
    const int row0 = t.row0 + r0;
    // (rows 32 apart have the same row & 7)
    uint8_t* cdst = codes + tile * mx4_slot(K, tile_rows) + r0 * 128 + (((lane >> 2) ^ (rr & 7)) * 16) +
                    (lane & 3) * 4;
    uint8_t* sdst = sf + tile * mx4_sf_slots(K) + half * 1024 + rr * 16 + (lane >> 4) * 512;
    const Tin* src[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      src[i] = source_row<Tin, SRC>(x, row_of, k, T, K, row0 + (i < nr ? i * 32 : 0), status);
    using P = Piece<std::conditional_t<SRC == 2, float, Tin>>;
    for (int kb = 0; kb < KB; ++kb) {
      // (K is a multiple of 128: whole half-warps lie inside)
      const int col = kb * kMx4KB + lane * 8;
      const bool in = col < K;
      P v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) load_piece<Tin, SRC>(v[i], src[i], col, K, in && i < nr);
      uint32_t c[4];
      const uint32_t b0 = quantize4x8(v, c);
      uint8_t* ck = cdst + (size_t)kb * rows16 * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (in && i < nr) *reinterpret_cast<uint32_t*>(ck + i * 32 * 128) = c[i];
      // A lane's four bytes are four rows' scales of one block; the first lane of each half
      // k-block collects the words of the other three blocks and turns the 4 x 4 bytes.
      uint4 w;
      turn_scales(b0, w);
      if (in && (lane & 15) == 0) *reinterpret_cast<uint4*>(sdst + (size_t)kb * kMx4SfSlot) = w;
    }
  }
}

// FEW rows: a warp per (row, k-block).
template <typename Tin, int SRC>
__global__ void __launch_bounds__(kQThreads) quantize_few_rows_kernel(
    const Tin* __restrict__ x, const int32_t* __restrict__ row_of, int k, int T,
    const int32_t* __restrict__ offsets, int E, int R, int K, int tile_rows,
    uint8_t* __restrict__ codes, uint8_t* __restrict__ sf, int32_t* status) {
  __shared__ Mx4Tables tb;
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KB = mx4_kblocks(K);
  const int it = blockIdx.x * kQWarps + warp;  // < 2^31: R is small
  const int r = it / KB, kb = it - r * KB;
  const int col = kb * kMx4KB + lane * 8;
  const bool in = r < R && col < K;
  using P = Piece<std::conditional_t<SRC == 2, float, Tin>>;
  P v;
  const Tin* row = r < R ? source_row<Tin, SRC>(x, row_of, k, T, K, r, status) : x;
  load_piece<Tin, SRC>(v, row, col, K, in);
  if (!mx4_build_tables(tb, offsets, E, R, status, tile_rows) || r >= R) return;
  const int e = mx4_find(tb.off, E, r);
  const int local = r - tb.off[e], step = tb.step[e];
  const int ti = local / step, rt = local - ti * step;
  const int rows16 = min(step, (tb.off[e + 1] - tb.off[e] - ti * step + 15) & ~15);
  uint32_t byte;
  const uint32_t c = quantize8(v, byte);
  const uint32_t w = byte | (__shfl_down_sync(0xFFFFFFFFu, byte, 4) << 8) |
                     (__shfl_down_sync(0xFFFFFFFFu, byte, 8) << 16) |
                     (__shfl_down_sync(0xFFFFFFFFu, byte, 12) << 24);
  if (!in) return;
  uint8_t* cdst = codes + (tb.tile[e] + ti) * mx4_slot(K, tile_rows) + (size_t)kb * rows16 * 128 + rt * 128;
  *reinterpret_cast<uint32_t*>(cdst + (((lane >> 2) ^ (rt & 7)) * 16) + (lane & 3) * 4) = c;
  if ((lane & 15) == 0)
    *reinterpret_cast<uint32_t*>(sf + ((size_t)(tb.tile[e] + ti) * KB + kb) * kMx4SfSlot +
                                 (rt >> 7) * 1024 + (lane >> 4) * 512 + (rt & 31) * 16 +
                                 ((rt >> 5) & 3) * 4) = w;
}

// ---------------------------------------------------------- weight images ---
// codes [E, N, K/2], scales [E, N, K/32] -> images; one CTA per (k-block, weight tile)
__global__ void __launch_bounds__(kQThreads) pack_kernel(const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, int K,
                                                         int N, uint8_t* __restrict__ packed) {
  const int KB = mx4_kblocks(K);
  const int kb = blockIdx.x;
  const long long tile = blockIdx.y + (long long)blockIdx.z * (N / kMx4WTile);
  uint8_t* dst = packed + (tile * KB + kb) * (size_t)kMx4WBytes;
  const size_t row0 = (size_t)blockIdx.z * N + (size_t)blockIdx.y * kMx4WTile;
  for (int i = threadIdx.x; i < kMx4WTile * 8; i += kQThreads) {
    const int r = i >> 3, c = i & 7;
    const int col = kb * 128 + c * 16;  // bytes
    const uint4 v = col < K / 2 ? *reinterpret_cast<const uint4*>(codes + (row0 + r) * (K / 2) + col)
                                : make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(dst + r * 128 + ((c ^ (r & 7)) * 16)) = v;
  }
  for (int i = threadIdx.x; i < kMx4WTile * 2; i += kQThreads) {
    const int r = i >> 1, j = i & 1;
    const int s = kb * 8 + j * 4;
    const uint32_t w =
        s < K / 32 ? *reinterpret_cast<const uint32_t*>(scales + (row0 + r) * (K / 32) + s) : 0u;
    *reinterpret_cast<uint32_t*>(dst + kMx4WTile * 128 + j * 512 + (r & 31) * 16 + (r >> 5) * 4) = w;
  }
}

// w [E, K, N] bf16 (row-major over K) -> images, quantised along K.  One CTA per (k-block,
// weight tile, expert); the tile goes through shared memory 32 values of K at a time, a
// thread quantising one output column's block.
__global__ void __launch_bounds__(128) prepack_kernel(const __nv_bfloat16* __restrict__ w, int K,
                                                      int N, int tile0, int tiles,
                                                      uint8_t* __restrict__ packed) {
  __shared__ __nv_bfloat16 s[32][128];
  const int KB = mx4_kblocks(K);
  const int kb = blockIdx.x, e = blockIdx.z;
  const long long tile = tile0 + blockIdx.y + (long long)e * tiles;
  uint8_t* dst = packed + (tile * KB + kb) * (size_t)kMx4WBytes;
  const __nv_bfloat16* src = w + ((size_t)e * K + (size_t)kb * kMx4KB) * N + blockIdx.y * kMx4WTile;
  const int r = threadIdx.x;
  for (int c = 0; c < 8; ++c) {
    const bool in = kb * kMx4KB + c * 32 < K;
    __syncthreads();
    if (in) {
      for (int i = threadIdx.x; i < 32 * 16; i += 128) {
        const int kk = i >> 4, q = i & 15;
        *reinterpret_cast<uint4*>(&s[kk][q * 8]) =
            *reinterpret_cast<const uint4*>(src + (size_t)(c * 32 + kk) * N + q * 8);
      }
    }
    __syncthreads();
    uint32_t byte = 0;
    uint32_t out[4] = {0, 0, 0, 0};
    if (in) {
      uint32_t a = 0;
#pragma unroll
      for (int kk = 0; kk < 32; ++kk)
        a = max(a, __float_as_uint(__bfloat162float(s[kk][r])) & 0x7FFFFFFFu);
      byte = mx4_scale_byte(a);
      const float inv = mx4_inverse_scale(byte);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = byte == 255u ? 0.0f : __bfloat162float(s[q * 8 + i][r]) * inv;
        out[q] = mx4_encode8(v);
      }
    }
    *reinterpret_cast<uint4*>(dst + r * 128 + ((c ^ (r & 7)) * 16)) =
        make_uint4(out[0], out[1], out[2], out[3]);
    dst[kMx4WTile * 128 + (c >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (c & 3)] = (uint8_t)byte;
  }
}

}  // namespace

cudaError_t launch_mx4_quantize(const void* x, int dtype, long long ld, long long R, int K,
                                void* codes, void* scales, void* values, cudaStream_t s) {
  const int per_row = K / 8;
  const long long n = R * per_row;
  if (n == 0) return cudaSuccess;
  const long long grid = (n + kQThreads * kQUnroll - 1) / (kQThreads * kQUnroll);  // < 2^31
  uint32_t* c = static_cast<uint32_t*>(codes);
  uint8_t* sc = static_cast<uint8_t*>(scales);
  uint4* v = static_cast<uint4*>(values);
  auto go = [&](auto* p) {
    using Tin = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    if (ld == K || R == 1)
      quantize_kernel<Tin, true><<<(unsigned)grid, kQThreads, 0, s>>>(p, ld, n, per_row, c, sc, v);
    else
      quantize_kernel<Tin, false><<<(unsigned)grid, kQThreads, 0, s>>>(p, ld, n, per_row, c, sc, v);
    return cudaGetLastError();
  };
  if (dtype == MOE_DTYPE_F32) return go(static_cast<const float*>(x));
  if (dtype == MOE_DTYPE_BF16) return go(static_cast<const __nv_bfloat16*>(x));
  return go(static_cast<const __half*>(x));
}

cudaError_t launch_mx4_rows(const void* x, int dtype, int src, const int32_t* row_of, int k, int T,
                            const int32_t* offsets, int E, int R, int K, int tile_rows, void* codes,
                            void* sf, int32_t* status, cudaStream_t s) {
  if (R == 0) return cudaSuccess;
  uint8_t* c = static_cast<uint8_t*>(codes);
  uint8_t* f = static_cast<uint8_t*>(sf);
  // Few: less than 16 warps of four rows on every SM.  With the product, 64 experts, K = N = 2048,
  // few / many: 1024 rows 32.8 / 39.9 us, 4096 rows 44.4 / 43.6, 9728 rows 67.4 / 53.9.
  const bool few = R < device_sm_count() * 64;
  const long long warps = few ? (long long)R * mx4_kblocks(K) : mx4_max_tiles(R, E, tile_rows) * 64;
  const long long need = (warps + kQWarps - 1) / kQWarps;
  const long long most = few ? need : (long long)device_sm_count() * kRowsBlocksPerSm;
  const int grid = (int)(need < most ? need : most);
  // Few rows: a dependent launch hides the start behind the end of a product before it
  // (8 rows of 8 experts, K = N = 2048: 10.3 -> 8.2 us in a row of calls).  Many: blocks that wait beside a running
  // product's CTAs are spread unevenly when they start (131072 rows: 280 -> 317 us), so not there.
  auto go = [&](auto many, auto few_rows, auto* p) -> cudaError_t {
    if (few)
      return launch_pdl(few_rows, dim3(grid), dim3(kQThreads), 0, s, p, row_of, k, T, offsets, E, R,
                        K, tile_rows, c, f, status);
    many<<<grid, kQThreads, 0, s>>>(p, row_of, k, T, offsets, E, R, K, tile_rows, c, f, status);
    return cudaGetLastError();
  };
#define MOE_MX4_ROWS(Tin, SRC) \
  go(quantize_rows_kernel<Tin, SRC>, quantize_few_rows_kernel<Tin, SRC>, static_cast<const Tin*>(x))
  if (src == 1) return MOE_MX4_ROWS(__nv_bfloat16, 1);
  if (src == 2) return MOE_MX4_ROWS(__nv_bfloat16, 2);
  if (dtype == MOE_DTYPE_F32) return MOE_MX4_ROWS(float, 0);
  if (dtype == MOE_DTYPE_BF16) return MOE_MX4_ROWS(__nv_bfloat16, 0);
  return MOE_MX4_ROWS(__half, 0);
#undef MOE_MX4_ROWS
}

cudaError_t launch_mx4_pack(const void* codes, const void* scales, int E, int K, int N,
                            void* packed, cudaStream_t s) {
  pack_kernel<<<dim3(mx4_kblocks(K), N / kMx4WTile, E), kQThreads, 0, s>>>(
      static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), K, N,
      static_cast<uint8_t*>(packed));
  return cudaGetLastError();
}

cudaError_t launch_mx4_prepack(const void* w, int E, int K, int N, int col0, int N_total,
                               void* packed, cudaStream_t s) {
  prepack_kernel<<<dim3(mx4_kblocks(K), N / kMx4WTile, E), 128, 0, s>>>(
      static_cast<const __nv_bfloat16*>(w), K, N, col0 / kMx4WTile, N_total / kMx4WTile,
      static_cast<uint8_t*>(packed));
  return cudaGetLastError();
}

}  // namespace moe

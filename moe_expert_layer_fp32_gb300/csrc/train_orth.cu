// Orthogonalisation of small matrices (at most 128 x 256, either way round) in one kernel: a CTA
// holds one matrix from its load to its result.
//
//   X = M / (|M| + eps), then `steps` times  A = X X^T, B = b A + c A A, X = a X + B X
//
// X stays in registers in FP32 (a thread has half a row, 128 columns); what the tensor cores
// read (X, A, B) goes to shared memory in FP16 times 1024, in rows of 128 bytes with the
// 128-byte swizzle.  The same image of X serves both products: its rows as the K-major operands of
// X X^T, and as the MN-major operand of B X.  What the rounding of B's diagonal, its largest values,
// left joins a in FP32 (it is most of the error of these sizes).  The diagonal itself multiplies the
// rounded X as the rest of B does: what X's rounding leaves outside of X's span then stays of second order
// in B X, where one part of B on X unrounded brings it in at first order (the whole diagonal there: rank
// 8 of 128 x 256 was 0.1 off after eight steps, each of which lifts it a times).  Everything waits on everything in a step, so the
// time is that of 3 x steps dependent products with their barriers (about 1.4 us each) and of the
// way in and out (18 us), not of bytes or operations: 38.6 us for 8 matrices of 128 x 256, five steps
// (36 without the diagonal's rest).
// The chain of kernels for larger matrices (train_gemm.cu) takes 17 launches and 78 us for them.
// A CTA writes its result while others may not have read their matrices yet, so that an out which
// lies in other matrices' bytes goes to the chain.
#include "common.cuh"
#include "kernels.cuh"
#include "pdl.cuh"
#include "train.cuh"

namespace moe {
namespace {

constexpr int S = 128, L = 256;  // rows and columns held (zeros behind the matrix's own)
constexpr int OFF_X = 0, OFF_A = (L / 64) * S * 128, OFF_B = OFF_A + (S / 64) * S * 128;
constexpr int OFF_END = OFF_B + (S / 64) * S * 128;
constexpr int OFF_DIAG = OFF_END + 128, SMEM = OFF_DIAG + S * 4;
constexpr int G_COL = 0, Q_COL = 128, Y_COL = 256, TMEM_COLS = 512;
constexpr int HALF = L / 2;
constexpr float HELD = 1024.0f;

// Piece (16 bytes, 8 values) c of row r of a [S rows][64 columns] chunk.
__device__ __forceinline__ uint4* piece(uint8_t* base, int chunk, int r, int c) {
  return reinterpret_cast<uint4*>(base + chunk * (S * 128) + r * 128 + ((c ^ (r & 7)) << 4));
}
__device__ __forceinline__ uint32_t half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr) {  // (64 columns a chunk of S rows)
  return sdesc_k_major_sw128(saddr) & ~(uint64_t)(0x3FFFu << 16) | (uint64_t)((S * 128) >> 4) << 16;
}
template <int TYPE>
__device__ __forceinline__ float load(const void* p, long long i) {
  if constexpr (TYPE == MOE_DTYPE_F32) return __ldg(static_cast<const float*>(p) + i);
  else if constexpr (TYPE == MOE_DTYPE_BF16)
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else return __half2float(static_cast<const __half*>(p)[i]);
}

template <int TYPE>
__global__ void __launch_bounds__(256, 1)
    orth_small_kernel(const void* __restrict__ m, long long ld, long long es, int rows,
                      int cols, float a, float b, float c, int steps, float eps, float scale,
                      void* out, int out_type, long long out_ld, long long out_es, int32_t* status,
                      long long limit) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + OFF_END);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* sums = reinterpret_cast<float*>(tmem_slot + 2);  // 3 x 8 (and the largest)
  float* diagonal = reinterpret_cast<float*>(smem + OFF_DIAG);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = 32 * (warp & 3) + lane, h = warp >> 2;  // this thread's row of X, and half of it
  const bool turned = rows > cols;
  const int N = turned ? rows : cols;

  if (threadIdx.x == 0) {
    *abort_flag = (smem_u32(smem) & 1023u) != 0;  // (never: asked for above)
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  pdl_wait();
  if (warp == 0) tmem_alloc(tmem_slot, TMEM_COLS);
  pdl_launch_dependents();

  // in and out through shared memory in FP32 (all of it is free then), so that global accesses run
  // along the matrix's rows: element (row i, column j) at fp(i, j), conflict-free either way
  float* whole = reinterpret_cast<float*>(smem);
  auto fp = [&](int i, int j) -> float& {
    return whole[(j >> 6) * (S * 64) + i * 64 + ((j + i) & 63)];
  };
  const int shift = turned ? 7 : 8;  // the fast index: a column, or a row of X if it is turned
  float x[HALF];
  float largest = 0.0f;
  const long long base = blockIdx.x * es;
  constexpr int AHEAD = 32;  // loads of a thread in flight (in order, they take 60 us a matrix)
#pragma unroll 1
  for (int t0 = threadIdx.x; t0 < S * L; t0 += AHEAD * 256) {
    float w[AHEAD];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      const int t = t0 + q * 256, u = t & ((1 << shift) - 1), v = t >> shift;
      w[q] = load<TYPE>(m, base + (long long)min(v, rows - 1) * ld + min(u, cols - 1));
    }
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      const int t = t0 + q * 256, u = t & ((1 << shift) - 1), v = t >> shift;
      fp(turned ? u : v, turned ? v : u) = v < rows && u < cols ? w[q] : 0.0f;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < HALF; ++j) {
    x[j] = fp(r, h * HALF + j);
    // (an infinity or a NaN: the norm below is one too)
    largest = fmaxf(largest, fabsf(x[j]));
  }
  // |M| from values scaled by a power of two that brings the largest to [1, 2)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) largest = fmaxf(largest, __shfl_xor_sync(~0u, largest, o));
  if (lane == 0) sums[warp] = largest;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  for (int i = 0; i < 8; ++i) largest = fmaxf(largest, sums[i]);
  int k = 0;
  if (largest > 0.0f && largest <= 0x1.fffffep127f) {
    frexpf(largest, &k);
    k = 1 - k;  // largest 2^k in [1, 2)
  }
  const float s1 = ldexpf(1.0f, k / 2), s2 = ldexpf(1.0f, k - k / 2);
  float sq = 0.0f;
#pragma unroll
  for (int j = 0; j < HALF; ++j) {
    x[j] = x[j] * s1 * s2;
    sq = fmaf(x[j], x[j], sq);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(~0u, sq, o);
  if (lane == 0) sums[8 + warp] = sq;
  __syncthreads();
  sq = 0.0f;
  for (int i = 0; i < 8; ++i) sq += sums[8 + i];
  // X = M / (|M| + eps) = (x 2^-k) / (|x| 2^-k + eps) = x / (|x| + eps 2^k)
  const float norm = sqrtf(sq) + eps * s1 * s2;
  const float inv = !(norm <= 0x1.fffffep127f) && !(eps * s1 * s2 > 0x1.fffffep127f)
                        ? __int_as_float(0x7FC00000)  // NaN or an infinity in M
                        : (sq > 0.0f ? 1.0f / norm : 0.0f);  // (sq at least 1, or M is zero)
#pragma unroll
  for (int j = 0; j < HALF; ++j) x[j] *= inv;

  const uint32_t tmem = *tmem_slot;
  const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  const uint32_t sx = smem_u32(smem + OFF_X), sa = smem_u32(smem + OFF_A), sb = smem_u32(smem + OFF_B);
  constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(S >> 4) << 24);  // FP16, FP32 sums, M = 128
  constexpr uint32_t N128 = (128u >> 3) << 17, N256 = (256u >> 3) << 17;
  const int k16 = (N + 15) / 16;
  uint32_t phase = 0;
  bool ok = *abort_flag == 0;
  // operands are in place: thread 0 issues, all wait
  auto product = [&](auto issue) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0 && ok) {
      if (elect_one()) {
        issue();
        mma_commit(bar);
      }
      __syncwarp();
    }
    if (threadIdx.x == 0 && ok) ok = mbar_wait_bounded(bar, phase, abort_flag, status, limit);
    phase ^= 1;
    ok = __syncthreads_and(ok);  // (a wait that ran out ends all threads' work alike)
    tc_fence_after();
  };

  for (int step = 0; step < steps && ok; ++step) {
#pragma unroll
    for (int q = 0; q < HALF / 8; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = half2(x[8 * q + 2 * j] * HELD, x[8 * q + 2 * j + 1] * HELD);
      *piece(smem + OFF_X, 2 * h + q / 8, r, q % 8) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    product([&] {  // X X^T
      for (int i = 0; i < k16; ++i) {
        const uint64_t d = sdesc_k_major_sw128(sx + (i / 4) * (S * 128) + (i % 4) * 32);
        mma_bf16(tmem + G_COL, d, d, IDESC | N128, i > 0);
      }
    });
    if (!ok) break;
    float g[64];  // A of this row, half of its columns
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(lanes + G_COL + 64 * h + 32 * t, v);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; ++j) g[32 * t + j] = __uint_as_float(v[j]) * (1.0f / (HELD * HELD));
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = half2(g[8 * q + 2 * j] * HELD, g[8 * q + 2 * j + 1] * HELD);
      *piece(smem + OFF_A, h, r, q) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    product([&] {  // A A
      for (int i = 0; i < S / 16; ++i) {
        const uint64_t d = sdesc_k_major_sw128(sa + (i / 4) * (S * 128) + (i % 4) * 32);
        mma_bf16(tmem + Q_COL, d, d, IDESC | N128, i > 0);
      }
    });
    if (!ok) break;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(lanes + Q_COL + 64 * h + 32 * t, v);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; ++j)
        g[32 * t + j] = fmaf(c / (HELD * HELD), __uint_as_float(v[j]), b * g[32 * t + j]);
    }
#pragma unroll
    for (int j = 0; j < 64; ++j)
      if (64 * h + j == r) {
        diagonal[r] = g[j] - __half2float(__float2half_rn(g[j] * HELD)) * (1.0f / HELD);
      }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = half2(g[8 * q + 2 * j] * HELD, g[8 * q + 2 * j + 1] * HELD);
      *piece(smem + OFF_B, h, r, q) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    product([&] {  // B X: X [k][n] as it lies, n along the rows of 128 bytes
      for (int i = 0; i < S / 16; ++i) {
        const uint64_t da = sdesc_k_major_sw128(sb + (i / 4) * (S * 128) + (i % 4) * 32);
        mma_bf16(tmem + Y_COL, da, sdesc_mn(sx + i * (16 * 128)), IDESC | N256 | (1u << 16), i > 0);
      }
    });
    if (!ok) break;
    const float ad = a + diagonal[r];
#pragma unroll
    for (int t = 0; t < HALF / 32; ++t) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(lanes + Y_COL + HALF * h + 32 * t, v);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; ++j)
        x[32 * t + j] = fmaf(ad, x[32 * t + j], __uint_as_float(v[j]) * (1.0f / (HELD * HELD)));
    }
  }

  if (ok) {
    uint16_t* o = static_cast<uint16_t*>(out) + blockIdx.x * out_es;
#pragma unroll
    for (int j = 0; j < HALF; ++j) fp(r, h * HALF + j) = x[j] * scale;
    __syncthreads();
    const bool bf16 = out_type == MOE_DTYPE_BF16;
#pragma unroll 16
    for (int t = threadIdx.x; t < S * L; t += 256) {
      const int u = t & ((1 << shift) - 1), v = t >> shift;
      const float y = fp(turned ? u : v, turned ? v : u);
      const uint16_t lo = __bfloat16_as_ushort(__float2bfloat16_rn(y));
      const uint16_t hi = __half_as_ushort(__float2half_rn(y));
      if (v < rows && u < cols) o[(long long)v * out_ld + u] = bf16 ? lo : hi;
    }
  }
  if (!ok && threadIdx.x == 0 && smem_u32(smem) % 1024 == 0)
    wait_drain(bar, phase ^ 1, kSpinLimitCycles);  // the MMAs issued last
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

}  // namespace

bool orth_small(int rows, int cols) {
  return (rows < cols ? rows : cols) <= S && (rows < cols ? cols : rows) <= L;
}

cudaError_t launch_orth_small(const void* m, int type, long long ld, long long es, int E, int rows,
                              int cols, const float* coefficients, int steps, float eps, float scale,
                              void* out, int out_type, long long out_ld, long long out_es,
                              int32_t* status, long long limit, cudaStream_t s) {
  auto go = [&](auto kern) {
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (err != cudaSuccess) return err;
    return launch_pdl(kern, dim3(E), dim3(256), SMEM, s, m, ld, es, rows, cols, coefficients[0],
                      coefficients[1], coefficients[2], steps, eps, scale, out, out_type, out_ld,
                      out_es, status, limit);
  };
  if (type == MOE_DTYPE_F32) return go(orth_small_kernel<MOE_DTYPE_F32>);
  if (type == MOE_DTYPE_BF16) return go(orth_small_kernel<MOE_DTYPE_BF16>);
  return go(orth_small_kernel<MOE_DTYPE_F16>);
}

}  // namespace moe

// The grouped 4-bit product of few rows in one kernel, for K up to 2048: each CTA quantises a
// tile's rows into its own shared memory and multiplies them by the expert's weights, so a
// decode step is one launch and the rows' codes never go to memory.
//
//   y[r, n] = sum over k of q(x)[r, k] * q(W_e)[k, n]
//
// A tile is up to 48 rows of one expert (48 KB of codes for K = 2048, two buffers: a tile is
// quantised while the one before is multiplied).  The weights, which bound such a batch, stream
// through a ring of 17 KB k-block images, 128 output columns an MMA (mx4_gemm.cu).
// Roles of a CTA:
//   warp 0       weights: one bulk copy a k-block, the next weight tile moved into L2
//   warp 1       MMA issuer
//   warps 2-5    epilogue (32 lanes x 32 columns at a time; four accumulators)
//   warps 6-17   quantisation: four rows x 256 values an item, the next item's loads in flight
// The (row tile, weight tile) units lie in a row, and every CTA takes an equal run of them: the
// weights are read once, evenly, and a row tile is quantised by the few CTAs that share it.
//
// Every wait is bounded and drains as in expert_gemm.cu.
#include "common.cuh"
#include "kernels.cuh"
#include "mx4.cuh"
#include "mx4_mma.cuh"
#include "mx4_rows.cuh"

namespace moe {
namespace {

constexpr int kFTile = 48;                 // rows of the largest tile
constexpr int kFKB = kMx4FusedMaxK / kMx4KB;
constexpr int kFQuant = 12;                // quantising warps
constexpr int kFFirst = 6;                 // the first of them
constexpr int kFThreads = (kFFirst + kFQuant) * 32;
constexpr int kFAcc = 4;                   // accumulators
constexpr int kFAccCols = 64;              // columns of one (read 32 at a time)

struct FCfg {
  static constexpr int STAGES = 6;
  static constexpr int CODE_BYTES = kFKB * kFTile * 128;  // a buffer's codes
  static constexpr int SF_BYTES = kFKB * 1024;            // a buffer's scales
  static constexpr int CODE_OFF = STAGES * kMx4WBytes;
  static constexpr int SF_OFF = CODE_OFF + 2 * CODE_BYTES;
  static constexpr int BAR_OFF = SF_OFF + 2 * SF_BYTES;
  static constexpr int NBAR = 2 * STAGES + 2 * kFAcc + 4 + 1;
  static constexpr int TMEM_COLS = 512;
  static constexpr int SF_COL = kFAcc * kFAccCols;        // two sets of 16 scale columns
  static constexpr int SMEM_BYTES = 1024 + BAR_OFF + NBAR * 8 + 16 + (int)sizeof(Mx4Tables) + 16;
  static_assert(CODE_OFF % 1024 == 0 && CODE_BYTES % 1024 == 0, "swizzled images: 1024 bytes");
  static_assert(SF_COL + 32 <= TMEM_COLS, "scale columns");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of one CTA");
};

// A run of weight tiles [n0, n1) of one row tile.
struct Run {
  int tile, n0, n1;
};
// The runs of CTA c of C: its equal share of all (row tile, weight tile) units in order.
struct Runs {
  int NT;
  long long cur, end;
  __device__ __forceinline__ Runs(int tiles, int NT_, int C, int c) : NT(NT_) {
    const long long all = (long long)tiles * NT;
    cur = all * c / C;
    end = all * (c + 1) / C;
  }
  __device__ __forceinline__ bool next(Run& r) {
    if (cur >= end) return false;
    r.tile = (int)(cur / NT);
    r.n0 = (int)(cur - (long long)r.tile * NT);
    r.n1 = (int)min((long long)NT, r.n0 + (end - cur));
    cur += r.n1 - r.n0;
    return true;
  }
};

template <typename Tin, int SRC, typename Tout>
__global__ void __launch_bounds__(kFThreads, 1)
    mx4_fused_kernel(const Tin* __restrict__ x, const int32_t* __restrict__ row_of, int k, int T,
                     const uint8_t* __restrict__ wimg, const int32_t* __restrict__ offsets, int E,
                     int R, int K, int N, Tout* __restrict__ y, int32_t* status,
                     long long spin_limit) {
  using C = FCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(base + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint64_t* tempty = tfull + kFAcc;
  uint64_t* qfull = tempty + kFAcc;
  uint64_t* qempty = qfull + 2;
  uint64_t* mma_done = qempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Mx4Tables& tb = *reinterpret_cast<Mx4Tables*>(tmem_slot + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int NT = N / kMx4WTile;
  const int KB = mx4_kblocks(K);

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < kFAcc; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 4);           // the epilogue warps
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&qfull[b], kFQuant);      // the quantising warps
      mbar_init(&qempty[b], 1);
    }
    mbar_init(mma_done, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, C::TMEM_COLS);
  const bool ok_tables = mx4_build_tables(tb, offsets, E, R, status, kFTile);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  Runs runs(ok_tables ? tb.tile[E] : 0, NT, gridDim.x, blockIdx.x);
  Run run;
  int e = 0;  // the walk's expert (runs go up)

  if (warp == 0) {
    if (elect_one()) {
      // ------------------------------------------------------------ weights
      int it = 0;
      bool aborted = false;
      while (!aborted && runs.next(run)) {
        const Mx4Tile t = mx4_walk_up(e, run.tile, tb);
        for (int n = run.n0; n < run.n1 && !aborted; ++n) {
          const uint8_t* w = wimg + (size_t)(t.e * NT + n) * KB * kMx4WBytes;
          const bool ahead = n + 1 < run.n1;
          const uint8_t* next_w = w + (size_t)KB * kMx4WBytes;
          for (int kb = 0; kb < KB; ++kb, ++it) {
            const int s = it % C::STAGES;
            if (!mbar_wait_bounded(&empty[s], ((it / C::STAGES) & 1) ^ 1, abort_flag, status,
                                   spin_limit)) {
              aborted = true;
              break;
            }
            mbar_arrive_expect_tx(&full[s], kMx4WBytes);
            bulk_load(base + s * kMx4WBytes, w + (size_t)kb * kMx4WBytes, kMx4WBytes, &full[s]);
            if (ahead) prefetch_l2(next_w + (size_t)kb * kMx4WBytes, kMx4WBytes);
          }
        }
      }
      if (aborted) {
        // the copies issued into the last STAGES slots may still be in flight
        for (int i = (it > C::STAGES ? it - C::STAGES : 0); i < it; ++i)
          wait_drain(&full[i % C::STAGES], (i / C::STAGES) & 1, kSpinLimitCycles);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      // ---------------------------------------------------------- MMA issuer
      int it = 0, tcount = 0, q = 0;
      bool aborted = false;
      while (!aborted && runs.next(run)) {
        const Mx4Tile t = mx4_walk_up(e, run.tile, tb);
        const int b = q & 1;
        if (!mbar_wait_bounded(&qfull[b], (q >> 1) & 1, abort_flag, status, spin_limit)) break;
        ++q;
        const uint32_t codes = smem_u32(base + C::CODE_OFF + b * C::CODE_BYTES);
        const uint32_t scales = smem_u32(base + C::SF_OFF + b * C::SF_BYTES);
        const uint32_t kb_bytes = (uint32_t)t.rows16 * 128u;
        const uint32_t id0 = idesc_mx4(128, t.rows16, 0), id1 = idesc_mx4(128, t.rows16, 2);
        for (int n = run.n0; n < run.n1 && !aborted; ++n, ++tcount) {
          const int acc = tcount % kFAcc;
          if (!mbar_wait_bounded(&tempty[acc], ((tcount / kFAcc) & 1) ^ 1, abort_flag, status,
                                 spin_limit)) {
            aborted = true;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + acc * kFAccCols;
          for (int kb = 0; kb < KB; ++kb, ++it) {
            const int s = it % C::STAGES;
            if (!mbar_wait_bounded(&full[s], (it / C::STAGES) & 1, abort_flag, status, spin_limit)) {
              aborted = true;
              break;
            }
            tc_fence_after();
            const uint32_t st = smem_u32(base + s * kMx4WBytes);
            const uint64_t da = sdesc_k_major_sw128(st);
            const uint64_t db = sdesc_k_major_sw128(codes + kb * kb_bytes);
            const uint64_t fa = sdesc_scales(st + kMx4WTile * 128);
            const uint64_t fb = sdesc_scales(scales + kb * 1024);
            // scale columns, four per half k-block: weights, then rows
            const uint32_t sfa = tmem_base + C::SF_COL + (it & 1) * 16, sfb = sfa + 8;
            const bool whole = (kb + 1) * kMx4KB <= K;  // else the first half only
            copy_scales<false>(sfa, fa);
            copy_scales<false>(sfb, fb);
            if (whole) {
              copy_scales<false>(sfa + 4, fa + 32);
              copy_scales<false>(sfb + 4, fb + 32);
            }
            mma_mx4<false>(d, da, db, id0, sfa, sfb, kb > 0 ? 1u : 0u);
            mma_mx4<false>(d, da + 2, db + 2, id1, sfa, sfb, 1u);
            if (whole) {
              mma_mx4<false>(d, da + 4, db + 4, id0, sfa + 4, sfb + 4, 1u);
              mma_mx4<false>(d, da + 6, db + 6, id1, sfa + 4, sfb + 4, 1u);
            }
            mma_commit(&empty[s]);
          }
          if (!aborted) mma_commit(&tfull[acc]);
        }
        if (!aborted) mma_commit(&qempty[b]);
      }
      // every MMA this thread issued completes before tensor memory is released
      mma_commit(mma_done);
      wait_drain(mma_done, 0, kSpinLimitCycles);
    }
    __syncwarp();
  } else if (warp < kFFirst) {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3;  // lane quarter of tensor memory this warp may access
    int tcount = 0;
    bool aborted = false;
    while (!aborted && runs.next(run)) {
      const Mx4Tile t = mx4_walk_up(e, run.tile, tb);
      for (int n = run.n0; n < run.n1; ++n, ++tcount) {
        const int acc = tcount % kFAcc;
        int ok = 1;
        if (lane == 0)
          ok = mbar_wait_bounded(&tfull[acc], (tcount / kFAcc) & 1, abort_flag, status, spin_limit);
        if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) {
          aborted = true;
          break;
        }
        tc_fence_after();
        const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kFAccCols);
        Tout* dst = y + (size_t)t.row0 * N + n * kMx4WTile + q * 32 + lane;
        for (int c0 = 0; c0 < t.rows; c0 += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + c0, v);
          tmem_ld_wait();
          Tout* o = dst + (size_t)c0 * N;
          const int m = t.rows - c0;
#pragma unroll
          for (int i = 0; i < 32; ++i, o += N)
            if (i < m) store_one(o, __uint_as_float(v[i]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc]);
      }
    }
  } else {
    // ---------------------------------------------------------- quantisation
    using Pc = Piece<std::conditional_t<SRC == 2, float, Tin>>;
    const int qw = warp - kFFirst;
    int qc = 0;
    while (runs.next(run)) {
      const Mx4Tile t = mx4_walk_up(e, run.tile, tb);
      const int b = qc & 1;
      const int items = (t.rows + 3) / 4 * KB;  // four rows x one k-block
      uint8_t* codes = base + C::CODE_OFF + b * C::CODE_BYTES;
      uint8_t* scales = base + C::SF_OFF + b * C::SF_BYTES;
      auto load = [&](Pc (&v)[4], int item) {
        const int g = item / KB, col = (item - g * KB) * kMx4KB + lane * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = col < K && g * 4 + i < t.rows;
          const Tin* row =
              in ? source_row<Tin, SRC>(x, row_of, k, T, K, t.row0 + g * 4 + i, status) : x;
          load_piece<Tin, SRC>(v[i], row, col, K, in);
        }
      };
      Pc next[4];
      if (qw < items) load(next, qw);
      int ok = 1;
      if (lane == 0)
        ok = mbar_wait_bounded(&qempty[b], ((qc >> 1) & 1) ^ 1, abort_flag, status, spin_limit);
      if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) break;
      ++qc;
      for (int item = qw; item < items; item += kFQuant) {
        Pc v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = next[i];
        if (item + kFQuant < items) load(next, item + kFQuant);
        const int g = item / KB, kb = item - g * KB;
        uint32_t c[4];
        uint4 w;
        turn_scales(quantize4x8(v, c), w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = g * 4 + i;  // (a group's rows past the tile's lie inside its padding)
          *reinterpret_cast<uint32_t*>(codes + (kb * t.rows16 + r) * 128 +
                                       (((lane >> 2) ^ (r & 7)) * 16) + (lane & 3) * 4) = c[i];
        }
        if ((lane & 15) == 0) {
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = g * 4 + i;
            *reinterpret_cast<uint32_t*>(scales + kb * 1024 + (lane >> 4) * 512 + (n & 31) * 16 +
                                         (n >> 5) * 4) = ws[i];
          }
        }
      }
      // generic-proxy writes before the tensor core reads them
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&qfull[b]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

template <typename Tin, int SRC, typename Tout>
cudaError_t go(const void* x, const int32_t* row_of, int k, int T, const void* packed,
               const int32_t* offsets, int E, int R, int K, int N, void* y, int32_t* status,
               long long limit, cudaStream_t s) {
  auto kern = mx4_fused_kernel<Tin, SRC, Tout>;
  static bool attr[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64 || !attr[dev]) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, FCfg::SMEM_BYTES);
    if (err != cudaSuccess) return err;
    if (dev < 64) attr[dev] = true;
  }
  const long long units = mx4_max_tiles(R, E, kFTile) * (N / kMx4WTile);
  const int sms = device_sm_count();
  kern<<<(unsigned)(units < sms ? units : sms), kFThreads, FCfg::SMEM_BYTES, s>>>(
      static_cast<const Tin*>(x), row_of, k, T, static_cast<const uint8_t*>(packed), offsets, E, R, K,
      N, static_cast<Tout*>(y), status, limit);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx4_fused(const void* x, int dtype, int src, const int32_t* row_of, int k, int T,
                             const void* packed, const int32_t* offsets, int E, int R, int K, int N,
                             void* y, int y_dtype, int32_t* status, long long spin_limit,
                             cudaStream_t s) {
  if (R == 0) return cudaSuccess;
#define MOE_MX4_FUSED(Tin, SRC, Tout) \
  go<Tin, SRC, Tout>(x, row_of, k, T, packed, offsets, E, R, K, N, y, status, spin_limit, s)
  using bf16 = __nv_bfloat16;
  if (src == 1) return MOE_MX4_FUSED(bf16, 1, bf16);  // the layer's gate and up
  if (src == 2) return MOE_MX4_FUSED(bf16, 2, float);  // its down projection
  const bool f32 = y_dtype == MOE_DTYPE_F32;
  if (dtype == MOE_DTYPE_F32) return f32 ? MOE_MX4_FUSED(float, 0, float) : MOE_MX4_FUSED(float, 0, bf16);
  if (dtype == MOE_DTYPE_BF16) return f32 ? MOE_MX4_FUSED(bf16, 0, float) : MOE_MX4_FUSED(bf16, 0, bf16);
  return f32 ? MOE_MX4_FUSED(__half, 0, float) : MOE_MX4_FUSED(__half, 0, bf16);
#undef MOE_MX4_FUSED
}

}  // namespace moe

// The grouped 4-bit product in one kernel, for K up to 2048: each CTA pair quantises a tile's
// rows into its own shared memory and multiplies them by all of the expert's weights, so the
// rows' codes never go to memory.
//
//   y[r, n] = sum over k of q(x)[r, k] * q(W_e)[k, n]
//
// A pair (cta_group::2) takes a tile of up to 112 rows of one expert: 56 rows' codes in each
// CTA (57 KB for K = 2048, two buffers: a tile is quantised while the one before is
// multiplied), the tile's scales in both.  The weights stream through a ring of 17 KB k-block
// images, 128 output columns a CTA, 256 an MMA; per k-block an SM takes in 17 KB, which at 64
// bytes a clock bounds the main loop at 272 cycles (the MMA's own 224 + the scales).
// Roles of a CTA:
//   warp 0       weights: one bulk copy a k-block
//   warp 1       even CTA: MMA issuer; odd CTA: passes its full stages on to the even CTA
//   warps 2-9    epilogue (32 lanes x 32 columns at a time; four accumulators of 112 columns)
//   warps 10-21  quantisation: four rows x 256 values an item, the next item's loads in
//                flight; codes to this CTA's buffer, scales to both CTAs'
// Tiles go round the pairs while there is a whole round of them (neighbours then share an
// expert's weights in L2); what is left of the last round is cut into runs of weight tiles of
// equal length, so that a batch of few tiles still reaches every SM.
//
// Every wait is bounded and drains as in expert_gemm.cu.
#include "common.cuh"
#include "kernels.cuh"
#include "mx4.cuh"
#include "mx4_mma.cuh"
#include "mx4_rows.cuh"

namespace moe {
namespace {

constexpr int kFTile = 112;                // rows of the largest tile
constexpr int kFHalf = kFTile / 2;         // of which a CTA holds
constexpr int kFKB = kMx4FusedMaxK / kMx4KB;
constexpr int kFQuant = 12;                // quantising warps
constexpr int kFThreads = (10 + kFQuant) * 32;
constexpr int kFAcc = 4;                   // accumulators

struct FCfg {
  static constexpr int STAGES = 5;
  static constexpr int CODE_BYTES = kFKB * kFHalf * 128;  // a buffer's codes
  static constexpr int SF_BYTES = kFKB * 1024;            // a buffer's scales
  static constexpr int CODE_OFF = STAGES * kMx4WBytes;
  static constexpr int SF_OFF = CODE_OFF + 2 * CODE_BYTES;
  static constexpr int BAR_OFF = SF_OFF + 2 * SF_BYTES;
  static constexpr int NBAR = 2 * STAGES + 2 * kFAcc + 4 + 1;
  static constexpr int TMEM_COLS = 512;
  static constexpr int SF_COL = kFAcc * kFTile;           // two sets of 16 scale columns
  static constexpr int SMEM_BYTES = 1024 + BAR_OFF + NBAR * 8 + 16 + (int)sizeof(Mx4Tables) + 16;
  static_assert(CODE_OFF % 1024 == 0 && CODE_BYTES % 1024 == 0, "swizzled images: 1024 bytes");
  static_assert(SF_COL + 32 <= TMEM_COLS, "scale columns");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of one CTA");
};

// A run of weight-tile pairs [p0, p1) of one row tile.
struct Run {
  int tile, p0, p1;
};

// The runs of pair c of C: every C-th tile while whole rounds last, then its share of the
// remaining tiles' weight-tile pairs.
struct Runs {
  int C, c, P, round, full;
  long long cur, end;
  __device__ __forceinline__ Runs(int tiles, int P_, int C_, int c_) : C(C_), c(c_), P(P_), round(0) {
    full = tiles / C;
    const long long left = (long long)(tiles - full * C) * P;
    cur = left * c / C;
    end = left * (c + 1) / C;
  }
  __device__ __forceinline__ bool next(Run& r) {
    if (round < full) {
      r = Run{round * C + c, 0, P};
      ++round;
      return true;
    }
    if (cur >= end) return false;
    r.tile = full * C + (int)(cur / P);
    r.p0 = (int)(cur % P);
    r.p1 = (int)min((long long)P, r.p0 + (end - cur));
    cur += r.p1 - r.p0;
    return true;
  }
};

__device__ __forceinline__ void store_peer(uint32_t addr_cluster, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr_cluster), "r"(v) : "memory");
}
// Arrive with cluster-scope release (after a proxy fence: the writes before it are read by
// the tensor cores of both CTAs).
__device__ __forceinline__ void arrive_release_cluster(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster)
               : "memory");
}

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
  const int NT = N / kMx4WTile, P = (NT + 1) / 2;
  const int KB = mx4_kblocks(K);
  const int rank = (int)cluster_ctarank();

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], rank == 0 ? 2 : 1);  // its producer (and the odd CTA's relay)
      mbar_init(&empty[s], 1);                 // the MMA's commit
    }
    for (int a = 0; a < kFAcc; ++a) {
      mbar_init(&tfull[a], 1);                 // the MMA's commit
      mbar_init(&tempty[a], 16);               // the epilogue warps of both CTAs
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&qfull[b], 2 * kFQuant);       // the quantising warps of both CTAs
      mbar_init(&qempty[b], 1);                // the MMA's commit
    }
    mbar_init(mma_done, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
  const bool ok_tables = mx4_build_tables(tb, offsets, E, R, status, kFTile);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers and buffers exist before any remote use
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  Runs runs(ok_tables ? tb.tile[E] : 0, P, gridDim.x / 2, blockIdx.x / 2);
  Run run;
  int e = 0;  // the walk's expert (runs go up)

  if (warp == 0) {
    if (elect_one()) {
      // ------------------------------------------------------------ weights
      int it = 0;
      bool aborted = false;
      while (!aborted && runs.next(run)) {
        const Mx4Tile t = mx4_walk_up(e, run.tile, tb);
        for (int p = run.p0; p < run.p1 && !aborted; ++p) {
          // (an odd last tile has no partner: the odd CTA multiplies it again and stores nothing)
          const int nt = min(2 * p + rank, NT - 1);
          const uint8_t* w = wimg + ((size_t)t.e * NT + nt) * KB * kMx4WBytes;
          for (int kb = 0; kb < KB; ++kb, ++it) {
            const int s = it % C::STAGES;
            if (!mbar_wait_bounded(&empty[s], ((it / C::STAGES) & 1) ^ 1, abort_flag, status,
                                   spin_limit)) {
              aborted = true;
              break;
            }
            mbar_arrive_expect_tx(&full[s], kMx4WBytes);
            bulk_load(base + s * kMx4WBytes, w + (size_t)kb * kMx4WBytes, kMx4WBytes, &full[s]);
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
    if (rank == 1) {
      if (elect_one()) {
        // ------------------------------------------- relay of the odd CTA's full stages
        int it = 0;
        bool aborted = false;
        while (!aborted && runs.next(run)) {
          for (int i = (run.p1 - run.p0) * KB; i > 0; --i, ++it) {
            const int s = it % C::STAGES;
            if (!mbar_wait_bounded(&full[s], (it / C::STAGES) & 1, abort_flag, status, spin_limit)) {
              aborted = true;
              break;
            }
            // CTA-scope release: the bytes are in this SM's shared memory, which only its own
            // tensor core reads; a cluster-scope release took about 1500 cycles a stage
            mbar_arrive_remote(mapa_shared(smem_u32(&full[s]), 0));
          }
        }
      }
    } else if (elect_one()) {
      // ---------------------------------------------------------- MMA issuer
      int it = 0, tcount = 0, q = 0;
      bool aborted = false;
      while (!aborted && runs.next(run)) {
        const Mx4Tile t = mx4_walk_up(e, run.tile, tb);
        const int b = q & 1;
        if (!wait_full<true>(&qfull[b], (q >> 1) & 1, abort_flag, status, spin_limit)) break;
        ++q;
        const uint32_t codes = smem_u32(base + C::CODE_OFF + b * C::CODE_BYTES);
        const uint32_t scales = smem_u32(base + C::SF_OFF + b * C::SF_BYTES);
        const uint32_t half_bytes = (uint32_t)t.rows16 * 64u;  // a CTA's rows of a k-block
        const uint32_t id0 = idesc_mx4(256, t.rows16, 0), id1 = idesc_mx4(256, t.rows16, 2);
        for (int p = run.p0; p < run.p1 && !aborted; ++p, ++tcount) {
          const int acc = tcount % kFAcc;
          if (!mbar_wait_bounded(&tempty[acc], ((tcount / kFAcc) & 1) ^ 1, abort_flag, status,
                                 spin_limit)) {
            aborted = true;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + acc * kFTile;
          for (int kb = 0; kb < KB; ++kb, ++it) {
            const int s = it % C::STAGES;
            if (!mbar_wait_bounded(&full[s], (it / C::STAGES) & 1, abort_flag, status, spin_limit)) {
              aborted = true;
              break;
            }
            tc_fence_after();
            const uint32_t st = smem_u32(base + s * kMx4WBytes);
            const uint64_t da = sdesc_k_major_sw128(st);
            const uint64_t db = sdesc_k_major_sw128(codes + kb * half_bytes);
            const uint64_t fa = sdesc_scales(st + kMx4WTile * 128);
            const uint64_t fb = sdesc_scales(scales + kb * 1024);
            // scale columns, four per half k-block: weights, then rows
            const uint32_t sfa = tmem_base + C::SF_COL + (it & 1) * 16, sfb = sfa + 8;
            const bool whole = (kb + 1) * kMx4KB <= K;  // else the first half only
            copy_scales<true>(sfa, fa);
            copy_scales<true>(sfb, fb);
            if (whole) {
              copy_scales<true>(sfa + 4, fa + 32);
              copy_scales<true>(sfb + 4, fb + 32);
            }
            mma_mx4<true>(d, da, db, id0, sfa, sfb, kb > 0 ? 1u : 0u);
            mma_mx4<true>(d, da + 2, db + 2, id1, sfa, sfb, 1u);
            if (whole) {
              mma_mx4<true>(d, da + 4, db + 4, id0, sfa + 4, sfb + 4, 1u);
              mma_mx4<true>(d, da + 6, db + 6, id1, sfa + 4, sfb + 4, 1u);
            }
            mma_commit_pair(&empty[s], 0x3);
          }
          if (!aborted) mma_commit_pair(&tfull[acc], 0x3);
        }
        if (!aborted) mma_commit_pair(&qempty[b], 0x3);
      }
      // every MMA this thread issued completes before tensor memory is released
      mma_commit_pair(mma_done, 0x1);
      wait_drain(mma_done, 0, kSpinLimitCycles);
    }
    __syncwarp();
  } else if (warp < 10) {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3;            // lane quarter of tensor memory this warp may access
    const int half = (warp - 2) >> 2;  // of the quarter's two warps: every other 32 columns
    int tcount = 0;
    bool aborted = false;
    while (!aborted && runs.next(run)) {
      const Mx4Tile t = mx4_walk_up(e, run.tile, tb);
      for (int p = run.p0; p < run.p1; ++p, ++tcount) {
        const int acc = tcount % kFAcc;
        int ok = 1;
        if (lane == 0)
          ok = mbar_wait_bounded(&tfull[acc], (tcount / kFAcc) & 1, abort_flag, status, spin_limit);
        if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) {
          aborted = true;
          break;
        }
        tc_fence_after();
        const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kFTile);
        const int nt = 2 * p + rank;
        Tout* dst = y + (size_t)t.row0 * N + nt * kMx4WTile + q * 32 + lane;
        const int rows = nt < NT ? t.rows : 0;
        for (int c0 = half * 32; c0 < rows; c0 += 64) {
          // (the last 32 columns of an accumulator reach into the next: read, not stored)
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + c0, v);
          tmem_ld_wait();
          Tout* o = dst + (size_t)c0 * N;
          if (rows - c0 >= 32) {
#pragma unroll
            for (int i = 0; i < 32; ++i, o += N) store_one(o, __uint_as_float(v[i]));
          } else {
            const int n = rows - c0;
#pragma unroll
            for (int i = 0; i < 32; ++i, o += N)
              if (i < n) store_one(o, __uint_as_float(v[i]));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(&tempty[acc]), 0));
      }
    }
  } else {
    // ---------------------------------------------------------- quantisation
    using Pc = Piece<std::conditional_t<SRC == 2, float, Tin>>;
    const int qw = warp - 10;
    int qc = 0;
    while (runs.next(run)) {
      const Mx4Tile t = mx4_walk_up(e, run.tile, tb);
      const int b = qc & 1;
      int ok = 1;
      if (lane == 0)
        ok = mbar_wait_bounded(&qempty[b], ((qc >> 1) & 1) ^ 1, abort_flag, status, spin_limit);
      if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) break;
      ++qc;
      const int half = t.rows16 / 2;                        // rows of this CTA (a multiple of 8)
      const int n0 = rank * half;                           // the first one's place in the tile
      const int mine = min(half, max(0, t.rows - n0));      // of them real
      const int items = (mine + 3) / 4 * KB;                // four rows x one k-block
      uint8_t* codes = base + C::CODE_OFF + b * C::CODE_BYTES;
      uint8_t* scales = base + C::SF_OFF + b * C::SF_BYTES;
      const uint32_t peer = mapa_shared(smem_u32(scales), rank ^ 1);
      auto load = [&](Pc (&v)[4], int item) {
        const int g = item / KB, col = (item - g * KB) * kMx4KB + lane * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = col < K && g * 4 + i < mine;
          const Tin* row = in ? source_row<Tin, SRC>(x, row_of, k, T, K, t.row0 + n0 + g * 4 + i, status)
                              : x;
          load_piece<Tin, SRC>(v[i], row, col, K, in);
        }
      };
      Pc next[4];
      if (qw < items) load(next, qw);
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
          const int r = g * 4 + i;  // (rows past `mine` of a group lie inside the half: 8 | half)
          *reinterpret_cast<uint32_t*>(codes + (kb * half + r) * 128 +
                                       (((lane >> 2) ^ (r & 7)) * 16) + (lane & 3) * 4) = c[i];
        }
        if ((lane & 15) == 0) {
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = n0 + g * 4 + i;
            const int o = kb * 1024 + (lane >> 4) * 512 + (n & 31) * 16 + (n >> 5) * 4;
            *reinterpret_cast<uint32_t*>(scales + o) = ws[i];
            store_peer(peer + o, ws[i]);
          }
        }
      }
      // generic-proxy writes (this CTA's codes, both CTAs' scales) before the tensor cores read
      asm volatile("fence.proxy.async;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive_release_cluster(mapa_shared(smem_u32(&qfull[b]), 0));
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves or frees tensor memory while the pair may still use it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
  }
}

template <typename Tin, int SRC, typename Tout>
cudaError_t go(const void* x, const int32_t* row_of, int k, int T, const void* packed,
               const int32_t* offsets, int E, int R, int K, int N, void* y, int32_t* status,
               long long limit, cudaStream_t s) {
  auto kern = mx4_fused_kernel<Tin, SRC, Tout>;
  static int cache[64] = {};  // per device: pairs that fit
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kFThreads);
  cfg.dynamicSmemBytes = FCfg::SMEM_BYTES;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int fit = dev < 64 ? cache[dev] : 0;
  if (fit == 0) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, FCfg::SMEM_BYTES);
    if (err != cudaSuccess) return err;
    cfg.gridDim = dim3(2 * device_sm_count());
    err = cudaOccupancyMaxActiveClusters(&fit, kern, &cfg);
    if (err != cudaSuccess) return err;
    if (fit < 1) return cudaErrorInvalidConfiguration;
    if (dev < 64) cache[dev] = fit;
  }
  const long long units = mx4_max_tiles(R, E, kFTile) * ((N / kMx4WTile + 1) / 2);
  cfg.gridDim = dim3(2u * (unsigned)(units < fit ? units : fit));
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const Tin*>(x), row_of, k, T,
                            static_cast<const uint8_t*>(packed), offsets, E, R, K, N,
                            static_cast<Tout*>(y), status, limit);
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

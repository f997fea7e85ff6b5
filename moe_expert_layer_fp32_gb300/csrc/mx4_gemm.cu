// Grouped product of microscaled 4-bit operands on the 5th-generation tensor cores.
//
//   y[r, n] = sum over k of q(x)[r, k] * q(W_e)[k, n]     for the rows r of expert e,
//
// each operand a code times its block's power-of-two scale (mx4.cuh), products exact and
// accumulated in FP32 by tcgen05.mma kind::mxf4 (block scales from tensor memory).
//
// The weights take the MMA's M side: 128 output columns in the accumulator's lanes, a
// tile of up to 224 rows of the expert in its columns (N is the tile's own row count, so
// a short tile costs what it holds).  Persistent CTAs, one per SM, warp-specialised:
//   warp 0   producer: three copies a k-block of 256 (weights with their scales, rows, row
//            scales) into a ring of STAGES shared-memory images
//   warp 1   MMA issuer: the scales from shared into tensor memory, then four MMAs of
//            K = 64.  The role runs in one elected lane for its whole loop: issued from a
//            lane picked by its index instead, an MMA took 95 cycles of issue, the 224-row
//            MMA itself 112.
//   warps 2-9  epilogue: 32 lanes x 32 columns at a time from tensor memory, two warps a
//            lane quarter; a warp writes 32 consecutive output columns of one row per store
// Tensor memory: two accumulators of up to 224 columns (a unit's epilogue runs under the next
// one's main loop) and two sets of 24 scale columns, at most 496 of 512.
//
// What it has to do: read each row's codes and each active expert's weights (0.53 bytes a
// value) once, write y.  Measured on GB300 (ncu, alone): 131072 rows of 128 experts, K = 2048,
// N = 1536, bf16 out: 169 us for 825 GFLOP and 0.71 GB (107 us at the copy rate), 4.9 PFLOP/s,
// tensor pipe busy 55%; 512 rows of 64 experts, K = N = 2048: 29.6 us for 140 MB of weights
// (21 us).  Per k-block the pair's MMAs take 416 cycles at 208 rows (the K = 64 rate of 16384
// products a clock and SM) and the loads 528 (34 KB at 64 bytes a clock); the rest is waiting
// for rows and weights.  What the steps brought, packed case with its row images: single CTAs
// of 224 rows 346 us; pairs 323; units walked without searches and divisions on the issuing
// thread (1900 cycles a unit before, hidden now) 294 -> 280; what a unit touches first moved
// into L2 ahead 277; the odd CTA's bytes counted by the even one, three tensor loads a k-block in
// place of its own bulk copies and a relay without cluster scope, 288; rows before weights 282.5.
// Not kept: the rows' images made and multiplied chunk by chunk side by side (no gain: every
// product's start and drain cost what the overlap saved), every CTA prefetching its next unit
// (six CTAs ask for the same rows: 198 -> 240), quantising inside this kernel (457 us: too few
// warps for the loads beside the tensor core's share of memory), the odd CTA's loads from two
// threads (280.4 in a graph).
//
// Every wait is bounded.  A wait that runs out, in whichever role, raises the CTA's abort flag;
// once all roles of the CTA (or pair) are done, a raised flag makes the producers wait for the
// copies that no role waited for, so that none is in flight when shared memory is given up.
#include <type_traits>

#include "common.cuh"
#include "kernels.cuh"
#include "mx4.cuh"
#include "mx4_mma.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kThreads = 320;  // producer, MMA issuer, eight epilogue warps

// PAIR: two CTAs of a cluster run one MMA (cta_group::2) of 256 output columns.
template <bool PAIR>
struct MxCfg {
  static constexpr int TILE_ROWS = PAIR ? kMx4PairRows : kMx4SingleRows;
  static constexpr int STAGES = PAIR ? 6 : 7;
  static constexpr int STAGE_ROWS = PAIR ? TILE_ROWS / 2 : TILE_ROWS;
  static constexpr int SF_OFF = kMx4WBytes;                  // row scales
  static constexpr int ROW_OFF = SF_OFF + kMx4SfSlot;        // row codes (1024-byte aligned)
  static constexpr int STAGE_BYTES = ROW_OFF + STAGE_ROWS * 128;
  static constexpr int NBAR = 2 * STAGES + 2 + 2 + 1;
  static constexpr int TMEM_COLS = 512;
  static constexpr int ACC_COLS = TILE_ROWS;
  static constexpr int SF_COL = 2 * ACC_COLS;                // first scale column
  static constexpr int SMEM_BYTES =
      1024 + STAGES * STAGE_BYTES + NBAR * 8 + 32 + (int)sizeof(Mx4Tables) + 16;
  static_assert(ROW_OFF % 1024 == 0 && STAGE_BYTES % 1024 == 0, "swizzled images: 1024 bytes");
  static_assert(SF_COL + 48 <= TMEM_COLS, "scale columns");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of one CTA");
};

// One unit: a row tile of an expert times one weight tile (PAIR: two, one a CTA).
struct MxUnit {
  int row0;              // first output row
  int rows;              // rows of the tile
  int rows16;            // padded to 16: N of its MMAs
  int nt;                // this CTA's weight tile of the expert (NT or more: none to store)
  size_t w_img;          // byte offsets of k-block 0's images
  size_t row_img;        // (of the tile; a pair's CTAs load one half of its rows each)
  size_t sf_img;
};

// The units of one CTA (or pair): every `step`-th from the first, tiles from the last one down
// (the row images written last are still in L2), a tile's weight tiles in order.
template <bool PAIR>
struct MxUnits {
  int e, tile, j, nu, q, r, NT, KB, rank;
  __device__ __forceinline__ MxUnits(int first, int step, const Mx4Tables& tb, int E, int NT_, int KB_,
                                     int rank_, bool ok)
      : NT(NT_), KB(KB_), rank(rank_) {
    nu = PAIR ? (NT + 1) / 2 : NT;  // units of a row tile
    const int t = first / nu;
    j = first - t * nu;
    tile = (ok ? tb.tile[E] : 0) - 1 - t;
    q = step / nu;
    r = step - q * nu;
    e = E - 1;
  }
  __device__ __forceinline__ bool more() const { return tile >= 0; }
  __device__ __forceinline__ void advance() {
    tile -= q;
    j += r;
    if (j >= nu) {
      j -= nu;
      --tile;
    }
  }
  __device__ __forceinline__ MxUnit unit(const Mx4Tables& tb) {
    const Mx4Tile t = mx4_walk_down(e, tile, tb);
    MxUnit w;
    w.nt = PAIR ? 2 * j + rank : j;
    w.row0 = t.row0;
    w.rows = t.rows;
    w.rows16 = t.rows16;
    w.w_img = (size_t)(e * NT + min(w.nt, NT - 1)) * KB * kMx4WBytes;
    w.row_img = (size_t)tile * KB * (MxCfg<PAIR>::TILE_ROWS * 128);
    w.sf_img = (size_t)tile * KB * kMx4SfSlot;
    return w;
  }
};

// The images as matrices of 1024-byte lines (every image, tile and half tile is whole lines), for
// the odd CTA of a pair: boxes of a weight image, of one and of two lines of scales, and of each
// height that a half tile can have (16 n rows: n lines).  A map per height, so that a k-block
// is three loads: with heights of 8, 4, 2 and 1 lines (up to six loads) the packed case took 321 us
// against 288; the lines' width (128 to 1024 bytes) made no difference.
constexpr int kMxHeights = kMx4PairRows / 16;
struct MxPairMaps {
  CUtensorMap w, sf[2], rows[kMxHeights];
};
struct MxNoMaps {};
static_assert(kMx4WBytes % 1024 == 0 && kMx4SfSlot == 2048 && kMx4PairRows % 16 == 0 &&
                  sizeof(MxPairMaps) <= 3840,
              "whole lines; kernel parameters");

// Pair form: every CTA loads its own weight tile, its half of the rows' codes and all of
// their scales; the bytes of both count on the even CTA's `full` barrier (the only full
// barriers in use), whose MMA thread runs both tensor cores.  So the odd CTA's loads are
// cta_group::2 tensor loads, which may signal the pair's other CTA while they write their own
// (a plain bulk copy signals the CTA that it writes).  Commits free the stage in both CTAs.
// Not kept: the odd CTA's completions on a barrier of its own, handed on by a thread of it.
// Handing operand bytes on takes a cluster-scope release, about 1500 cycles a stage (packed
// case 372 us); a CTA-scope one is no ordering between two CTAs.
template <typename Tout, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    mx4_gemm_kernel(const __grid_constant__ std::conditional_t<PAIR, MxPairMaps, MxNoMaps> maps,
                    const uint8_t* __restrict__ wimg, const uint8_t* __restrict__ rimg,
                    const uint8_t* __restrict__ simg, const int32_t* __restrict__ offsets, int E,
                    int R, int K, int N, Tout* __restrict__ y, int32_t* status,
                    long long spin_limit) {
  using C = MxCfg<PAIR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::STAGES * C::STAGE_BYTES);
  uint64_t* full = bars;
  uint64_t* empty = bars + C::STAGES;
  uint64_t* tfull = bars + 2 * C::STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* peer_abort = abort_flag + 1;   // pair: the other CTA's flag and the k-blocks
  volatile int* peer_issued = abort_flag + 2;  // that it has issued, written by it at its end
  volatile int* committed = abort_flag + 3;    // k-blocks and accumulators that the issuer has committed
  Mx4Tables& tb = *reinterpret_cast<Mx4Tables*>(tmem_slot + 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int NT = N / kMx4WTile;
  const int KB = mx4_kblocks(K);
  const int rank = PAIR ? (int)cluster_ctarank() : 0;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    *peer_abort = 0;
    *peer_issued = 0;
    committed[0] = committed[1] = 0;
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);                            // the (even) producer; all bytes
      mbar_init(&empty[s], 1);                           // the MMA's commit
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);                           // the MMA's commit
      mbar_init(&tempty[a], PAIR ? 16 : 8);              // the epilogue warps (of both CTAs)
    }
    mbar_init(mma_done, 1);
    fence_mbar_init();
  }
  if constexpr (PAIR) {
    if (threadIdx.x == 0 && rank == 1) {
      prefetch_tensormap(&maps.w);
      prefetch_tensormap(&maps.sf[0]);
      prefetch_tensormap(&maps.sf[1]);
    }
  }
  if (warp == 1) {
    if constexpr (PAIR) tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
    else tmem_alloc(tmem_slot, C::TMEM_COLS);
  }
  mx4_build_tables(tb, offsets, E, R, status, C::TILE_ROWS);
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // both CTAs' barriers exist before any remote use
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  auto first_unit = [&]() {
    return MxUnits<PAIR>(PAIR ? blockIdx.x / 2 : blockIdx.x, PAIR ? gridDim.x / 2 : gridDim.x, tb, E,
                         NT, KB, rank, tb.ok != 0);
  };
  MxUnits<PAIR> units = first_unit();
  int issued = -1;  // the producer's thread: k-blocks issued

  // ---- the producer's steps
  // bytes of a k-block's rows and scales that this CTA loads
  auto row_bytes = [&](const MxUnit& w) { return (uint32_t)w.rows16 * (PAIR ? 64u : 128u); };
  auto sf_bytes = [&](const MxUnit& w) { return w.rows16 > 128 ? 2048u : 1024u; };
  // the bytes that stage s will get (of a pair: from both CTAs, counted by the even one)
  auto arm = [&](int s, const MxUnit& w) {
    if (!PAIR || rank == 0)
      mbar_arrive_expect_tx(&full[s], (PAIR ? 2 : 1) * (kMx4WBytes + row_bytes(w) + sf_bytes(w)));
  };
  auto load_weights = [&](int s, const MxUnit& w, int kb) {
    uint8_t* st = base + s * C::STAGE_BYTES;
    if constexpr (PAIR) {
      if (rank == 1) {
        tma_load_2d_pair(&maps.w, st, mapa_shared(smem_u32(&full[s]), 0), 0,
                         (int)(w.w_img / 1024) + kb * (kMx4WBytes / 1024));
        return;
      }
    }
    bulk_load(st, wimg + w.w_img + (size_t)kb * kMx4WBytes, kMx4WBytes, &full[s]);
  };
  auto load_rows = [&](int s, const MxUnit& w, int kb) {
    uint8_t* st = base + s * C::STAGE_BYTES;
    const uint32_t rb = row_bytes(w), sb = sf_bytes(w);
    const size_t rows = w.row_img + (size_t)rank * rb + (size_t)kb * w.rows16 * 128;
    const size_t scales = w.sf_img + (size_t)kb * kMx4SfSlot;
    if constexpr (PAIR) {
      if (rank == 1) {
        const uint32_t bar = mapa_shared(smem_u32(&full[s]), 0);
        tma_load_2d_pair(&maps.rows[w.rows16 / 16 - 1], st + C::ROW_OFF, bar, 0, (int)(rows / 1024));
        tma_load_2d_pair(&maps.sf[sb / 1024 - 1], st + C::SF_OFF, bar, 0, (int)(scales / 1024));
        return;
      }
    }
    bulk_load(st + C::ROW_OFF, rimg + rows, rb, &full[s]);
    bulk_load(st + C::SF_OFF, simg + scales, sb, &full[s]);
  };

  if (warp == 0) {
    if (elect_one()) {
      // ------------------------------------------------------------ producer
      // The weights are inputs: the first unit's first stages are on their way before the
      // rows' quantisation, the kernel before this one, has finished.
      int early = 0;
      if (units.more()) {
        const MxUnit w = units.unit(tb);
        for (; early < KB && early < C::STAGES; ++early) {
          arm(early, w);
          load_weights(early, w, early);
        }
      }
      pdl_wait();
      pdl_launch_dependents();  // (whatever comes next waits for this kernel itself)
      int it = 0;
      bool aborted = false;
      for (; units.more() && !aborted; units.advance()) {
        const MxUnit w = units.unit(tb);
        // What this CTA's next unit is the first to touch moves into L2 while this one is
        // multiplied: an expert's weights with its first tile, a tile's rows with its first
        // weight tile.  (Six stages cover a load from L2, not one from memory.)
        MxUnits<PAIR> ahead = units;
        ahead.advance();
        const bool more = ahead.more();
        const MxUnit nx = more ? ahead.unit(tb) : w;
        const bool fetch_w = more && ahead.tile == tb.tile[ahead.e + 1] - 1;
        const bool fetch_rows = more && ahead.j == 0 && rank == 0;
        for (int kb = 0; kb < KB; ++kb, ++it) {
          const int s = it % C::STAGES;
          const uint32_t ph = (it / C::STAGES) & 1;
          if (!mbar_wait_bounded(&empty[s], ph ^ 1, abort_flag, status, spin_limit)) {
            aborted = true;
            break;
          }
          // (rows before weights: packed case 282.8 us the other way round, 279.0 so, in a graph)
          if (it >= early) arm(s, w);
          load_rows(s, w, kb);
          if (it >= early) load_weights(s, w, kb);
          if (fetch_w) prefetch_l2(wimg + nx.w_img + (size_t)kb * kMx4WBytes, kMx4WBytes);
          if (fetch_rows)
            prefetch_l2(rimg + nx.row_img + (size_t)kb * nx.rows16 * 128, nx.rows16 * 128);
        }
      }
      // the last k-blocks' commits arrive in this CTA, the odd one too: it does not leave before
      // (the epilogue has waited for every accumulator's)
      for (int i = (it > C::STAGES ? it - C::STAGES : 0); i < it && !aborted; ++i)
        aborted = !mbar_wait_bounded(&empty[i % C::STAGES], (i / C::STAGES) & 1, abort_flag, status,
                                     spin_limit);
      issued = it;
      if constexpr (PAIR) st_shared_remote(mapa_shared(smem_u32((const void*)peer_issued), rank ^ 1), it);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      // ---------------------------------------------------------- MMA issuer
      int it = 0, tcount = 0;
      int rows16 = units.more() ? units.unit(tb).rows16 : 0;
      for (; rows16 != 0; ++tcount) {
        const int acc = tcount & 1;
        const uint32_t aph = (tcount >> 1) & 1;
        int next16 = 0;
        if (!mbar_wait_bounded(&tempty[acc], aph ^ 1, abort_flag, status, spin_limit)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + acc * C::ACC_COLS;
        constexpr int M = PAIR ? 256 : 128;
        const uint32_t id0 = idesc_mx4(M, rows16, 0), id1 = idesc_mx4(M, rows16, 2);
        const bool two = rows16 > 128;
        bool aborted = false;
        for (int kb = 0; kb < KB; ++kb, ++it) {
          if (kb == KB - 1) {  // the next unit, while MMAs are queued
            units.advance();
            if (units.more()) next16 = units.unit(tb).rows16;
          }
          const int s = it % C::STAGES;
          const uint32_t ph = (it / C::STAGES) & 1;
          if (!mbar_wait_bounded(&full[s], ph, abort_flag, status, spin_limit)) {
            aborted = true;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_u32(base + s * C::STAGE_BYTES);
          const uint64_t da = sdesc_k_major_sw128(st), db = sdesc_k_major_sw128(st + C::ROW_OFF);
          const uint64_t fa = sdesc_scales(st + kMx4WTile * 128), fb = sdesc_scales(st + C::SF_OFF);
          // scale columns: weights 4 per half k-block, rows 8 (two 128-row halves)
          const uint32_t sfa = tmem_base + C::SF_COL + (it & 1) * 24, sfb = sfa + 8;
          const bool whole = (kb + 1) * kMx4KB <= K;  // else the first half only
          copy_scales<PAIR>(sfa, fa);
          copy_scales<PAIR>(sfb, fb);
          if (two) copy_scales<PAIR>(sfb + 4, fb + 64);
          if (whole) {
            copy_scales<PAIR>(sfa + 4, fa + 32);
            copy_scales<PAIR>(sfb + 8, fb + 32);
            if (two) copy_scales<PAIR>(sfb + 12, fb + 96);
          }
          mma_mx4<PAIR>(d, da, db, id0, sfa, sfb, kb > 0 ? 1u : 0u);
          mma_mx4<PAIR>(d, da + 2, db + 2, id1, sfa, sfb, 1u);
          if (whole) {
            mma_mx4<PAIR>(d, da + 4, db + 4, id0, sfa + 4, sfb + 8, 1u);
            mma_mx4<PAIR>(d, da + 6, db + 6, id1, sfa + 4, sfb + 8, 1u);
          }
          if constexpr (PAIR) mma_commit_pair(&empty[s], 0x3);
          else mma_commit(&empty[s]);
        }
        if (aborted) break;
        if constexpr (PAIR) mma_commit_pair(&tfull[acc], 0x3);
        else mma_commit(&tfull[acc]);
        rows16 = next16;
      }
      // every MMA this thread issued completes before tensor memory is released
      if constexpr (PAIR) mma_commit_pair(mma_done, 0x1);
      else mma_commit(mma_done);
      wait_drain(mma_done, 0, kSpinLimitCycles);
      committed[0] = it;
      committed[1] = tcount;
      if constexpr (PAIR)
        for (int i = 0; i < 2; ++i)
          st_shared_remote(mapa_shared(smem_u32((const void*)(committed + i)), 1), i ? tcount : it);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3;  // lane quarter of tensor memory this warp may access
    const int half = (warp - 2) >> 2;  // of the quarter's two warps: every other 32 columns
    int tcount = 0;
    for (; units.more(); units.advance(), ++tcount) {
      const MxUnit w = units.unit(tb);
      const int acc = tcount & 1;
      const uint32_t aph = (tcount >> 1) & 1;
      int ok = 1;
      if (lane == 0) ok = mbar_wait_bounded(&tfull[acc], aph, abort_flag, status, spin_limit);
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * C::ACC_COLS);
      Tout* dst = y + (size_t)w.row0 * N + w.nt * kMx4WTile + q * 32 + lane;
      const int rows = (!PAIR || w.nt < NT) ? w.rows : 0;
      for (int c0 = half * 32; c0 < rows; c0 += 64) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(taddr + c0, v);
        tmem_ld_wait();
        Tout* p = dst + (size_t)c0 * N;
        if (rows - c0 >= 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i, p += N) store_one(p, __uint_as_float(v[i]));
        } else {
          const int n = rows - c0;
#pragma unroll
          for (int i = 0; i < 32; ++i, p += N)
            if (i < n) store_one(p, __uint_as_float(v[i]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_remote(mapa_shared(smem_u32(&tempty[acc]), 0));
        else mbar_arrive(&tempty[acc]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  bool aborted = *abort_flag != 0;
  if constexpr (PAIR) {
    if (threadIdx.x == 0 && aborted)
      st_shared_remote(mapa_shared(smem_u32((const void*)peer_abort), rank ^ 1), 1);
    cluster_sync();  // no CTA leaves while the pair may still use it
    aborted = aborted || *peer_abort != 0;  // (the same in both CTAs)
  }
  if (aborted) {
    // All MMAs are complete and no role waits any more.  Copies into the last STAGES slots may
    // still be in flight (of a unit that no MMA took: whoever gave up, the producer need not
    // have noticed).  A stage that only one CTA of a pair has issued gets the other's bytes now
    // (its slot's last MMAs are complete, or the one could not have issued it), so that its barrier
    // completes; the even CTA waits for the bytes of both.  A role that gave up did not wait for
    // the commits that arrive in its CTA: thread 0 does.
    if (threadIdx.x == 0) {
      const int blocks = committed[0], tiles = committed[1];
      for (int i = (blocks > C::STAGES ? blocks - C::STAGES : 0); i < blocks; ++i)
        wait_drain(&empty[i % C::STAGES], (i / C::STAGES) & 1, kSpinLimitCycles);
      for (int i = (tiles > 2 ? tiles - 2 : 0); i < tiles; ++i)
        wait_drain(&tfull[i & 1], (i >> 1) & 1, kSpinLimitCycles);
    }
    if (issued >= 0) {
      int n = issued;
      if constexpr (PAIR) {
        MxUnits<PAIR> u = first_unit();
        for (int i = n / KB; i > 0; --i) u.advance();
        for (; n < *peer_issued; ++n) {
          const MxUnit w = u.unit(tb);
          arm(n % C::STAGES, w);
          load_weights(n % C::STAGES, w, n % KB);
          load_rows(n % C::STAGES, w, n % KB);
          if (n % KB == KB - 1) u.advance();
        }
      }
      if (rank == 0)
        for (int i = n > C::STAGES ? n - C::STAGES : 0; i < n; ++i)
          wait_drain(&full[i % C::STAGES], (i / C::STAGES) & 1, kSpinLimitCycles);
    }
    if constexpr (PAIR) cluster_sync();  // the odd CTA's copies count on the even CTA's barriers
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// One CTA per SM (pairs: as many clusters of two as fit), at most one per unit.
template <typename Tout, bool PAIR>
cudaError_t go(const uint8_t* w, const uint8_t* r, const uint8_t* sf, const int32_t* offsets, int E,
               int R, int K, int N, void* y, int32_t* status, long long limit, cudaStream_t s) {
  using C = MxCfg<PAIR>;
  auto kern = mx4_gemm_kernel<Tout, PAIR>;
  static int cache[64] = {};  // per device: CTAs that fit
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  pdl_attr(attr[0]);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  int fit = dev < 64 ? cache[dev] : 0;
  if (fit == 0) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (err != cudaSuccess) return err;
    fit = device_sm_count();
    if (PAIR) {
      int clusters = 0;
      cfg.gridDim = dim3(2 * fit);
      cfg.attrs = attr + 1;
      cfg.numAttrs = 1;
      err = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
      if (err != cudaSuccess) return err;
      if (clusters < 1) return cudaErrorInvalidConfiguration;
      fit = 2 * clusters;
    }
    if (dev < 64) cache[dev] = fit;
  }
  const int NT = N / kMx4WTile;
  const long long units = mx4_max_tiles(R, E, C::TILE_ROWS) * (PAIR ? (NT + 1) / 2 * 2 : NT);
  cfg.gridDim = dim3((unsigned)(units < fit ? units : fit));
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  std::conditional_t<PAIR, MxPairMaps, MxNoMaps> maps;
  if constexpr (PAIR) {
    const uint64_t tiles = (uint64_t)mx4_max_tiles(R, E, C::TILE_ROWS);
    auto lines = [](CUtensorMap* m, const void* p, uint64_t n, uint32_t box) {
      return encode_rowmajor_2d(m, p, 256, n, true, 256, box);
    };
    bool ok = lines(&maps.w, w, (uint64_t)E * NT * mx4_kblocks(K) * (kMx4WBytes / 1024),
                    kMx4WBytes / 1024);
    for (uint32_t j = 0; j < 2; ++j)
      ok = ok && lines(&maps.sf[j], sf, tiles * (mx4_sf_slots(K) / 1024), j + 1);
    for (uint32_t j = 0; j < kMxHeights; ++j)
      ok = ok && lines(&maps.rows[j], r, tiles * (mx4_slot(K, C::TILE_ROWS) / 1024), j + 1);
    if (!ok) return cudaErrorInvalidValue;
  }
  return cudaLaunchKernelEx(&cfg, kern, maps, w, r, sf, offsets, E, R, K, N, static_cast<Tout*>(y), status,
                            limit);
}

}  // namespace

// Pairs share the rows' bytes that a single CTA takes in alone (64 bytes a clock bound the main
// loop of large tiles); a batch of few rows is bound by its weights, and single CTAs with a
// deeper ring stream them faster.  64 experts, K = N = 2048, pairs / single CTAs: 16 rows an
// expert 32.8 / 31.7 us, 32 rows 36.4 / 36.9, 64 rows 44.4 / 48.1, 256 rows 96.7 / 128.  Every
// output element is the same sequence of MMAs in both forms, so its bits do not depend on the
// choice.
static bool use_pair(int E, int R, int N) {
  return N >= 2 * kMx4WTile && (long long)R >= 64LL * (R < E ? R : E);
}
int mx4_tile_rows(int E, int R, int N) { return use_pair(E, R, N) ? kMx4PairRows : kMx4SingleRows; }

cudaError_t launch_mx4_gemm(const void* packed, const void* codes, const void* sf,
                            const int32_t* offsets, int E, int R, int K, int N, void* y,
                            int y_dtype, int32_t* status, long long spin_limit, cudaStream_t s) {
  if (R == 0) return cudaSuccess;
  const uint8_t* w = static_cast<const uint8_t*>(packed);
  const uint8_t* r = static_cast<const uint8_t*>(codes);
  const uint8_t* f = static_cast<const uint8_t*>(sf);
  auto run = [&](auto kind) {
    using T = decltype(kind);
    return use_pair(E, R, N)
               ? go<T, true>(w, r, f, offsets, E, R, K, N, y, status, spin_limit, s)
               : go<T, false>(w, r, f, offsets, E, R, K, N, y, status, spin_limit, s);
  };
  return y_dtype == MOE_DTYPE_F32 ? run(float{}) : run(__nv_bfloat16{});
}

}  // namespace moe

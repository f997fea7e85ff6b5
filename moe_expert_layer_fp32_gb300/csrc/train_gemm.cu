// Products that train the experts, on the 5th-generation tensor cores (tcgen05 + TMEM + TMA):
//
//   PRODUCT  y[r] = x[r] W_e (W [E, K, N]) or x[r] W_e^T (W [E, N, K]) for the rows r of expert e
//   WGRAD    dW_e = sum over the rows r of expert e of x[r]^T dy[r]
//   BATCH    out_e = alpha A_e B_e + beta C_e, one of each an expert (Newton-Schulz steps)
//   SYM      the same where the result is symmetric (X X^T, its square): only the tiles on and
//            above the diagonal are computed and stored
//
// All read the operands in the caller's layout.  An operand whose contraction index runs along
// its rows (x and W^T of a product) is staged K-major, the others (W, and both operands of a
// weight gradient) MN-major: tcgen05 takes either from 128-byte-swizzled shared memory, so
// nothing is transposed or packed beforehand.  A symmetric operand is read by its upper tiles: a
// k-block left of the diagonal comes MN-major from its mirror image.
//
// Roles of a CTA (352 threads): warp 0 loads A (TMA), warp 10 B, warp 1 issues the MMAs, warps 2..9
// are the epilogue (two a TMEM lane quarter, every other 128 bytes of a row), over a ring of
// k-blocks of 64 and two accumulators in TMEM.  Forms:
//   pair     two CTAs share one M = 256 MMA over 256 columns (cta_group::2): each SM stages
//            32 KB a k-block for 256 x 256 x 64 products
//   single   one CTA, 128 x 128, for few rows: of A only the 16-row boxes that hold rows of the
//            expert are loaded, so that the ring streams weights
//
// A weight gradient contracts over an expert's rows, which end anywhere.  The rows of an
// expert's last, partial k-block are copied beforehand (tails_kernel) and filled up with zeros, so
// another expert's rows (or infinities and NaN among them) never enter the sum.
//
// What bounds it.  Few rows: the weights' bytes (512 rows of 64 experts, 1024 x 2048: 44.3 us, 6.2 TB/s,
// 91% of the copy rate).  Many rows: the tensor pipe, 94% active at 131072 rows of 128 experts, 2048 x
// 1536 (532 us alone under the profiler, 608 among others under the power cap; full 256-row tiles
// would be 12% fewer).  Weight gradients: the FP32 output's way out beside the short contractions
// (512 rows an expert, 2048 x 2048: 273 us, 4.92 TB/s, tensor pipe 49%).  Chains of Newton-Schulz
// products: 70-83% of the tensor pipe at 64 x 1024 x 2048, the rest is each kernel's first and last
// tile.
//
// What it took: a k-block of the pair form is 512 cycles of MMA, so everything that a role's thread
// does for one has to stay under that.  Descriptors made anew for each MMA cost the issuing thread
// more (product of 64 x 512 rows 208 us, made once 192), and so did four copies of a weight
// gradient's stage from one thread (450 us, from two 351); the roles' threads are elected, so that
// copies and MMAs are issued without a loop over active lanes (128 x 1024 rows: 480 against 456).
//
// Bounded waits, and what happens when one runs out, as in expert_gemm.cu.
#include "common.cuh"
#include "kernels.cuh"
#include "pdl.cuh"
#include "train.cuh"

namespace moe {
namespace {

enum Kind { PRODUCT, WGRAD, BATCH, SYM };
enum Major { KM, MN, UPPER };  // UPPER: a symmetric matrix of which the upper tiles are there

constexpr int GM = 128, GK = 64, UK = 16;
constexpr int EPI_WARPS = 8, B_WARP = 2 + EPI_WARPS, THREADS = 32 * (B_WARP + 1);
constexpr int BOX_ROWS = 16;  // A boxes of the single form of a product
// k-blocks whose products one accumulator sums.  The tensor cores' addition drops up to 2^-23 of the
// running sum at each step of sixteen products, always towards zero, so that an error grows with the
// contraction (relative 2-norm, K = N = 256, random signs / one sign: 4096 rows 4.4e-6 / 1.4e-5, 131072
// 1.5e-4 / 8.2e-4).  Longer sums are taken apart, and the parts added in FP32 by the epilogue, while the
// MMAs wait (65536 rows, 2048 x 2048 FP32: 158 -> 162 us; parts half as long would double both).  (Not
// in BATCH and SYM: at their longest, 16384, the error is a third of the rounding to FP16 behind them.)
constexpr int SEG = 64;

template <int CTAS, int BN>
struct Shape {
  static constexpr int STAGES = 6;
  static constexpr int A_BYTES = GM * GK * 2;
  static constexpr int BROWS = BN / CTAS;  // of B in this CTA
  static constexpr int B_BYTES = BROWS * GK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int TMEM_COLS = 2 * BN;
  static constexpr int NBAR = 2 * STAGES + 2 + 2 + 1;
  static constexpr int EPI_BYTES = EPI_WARPS * 32 * 128;
  static constexpr int SMEM_BYTES =
      STAGES * STAGE_BYTES + EPI_BYTES + NBAR * 8 + 48 + 2 * (kMaxE + 1) * 4;
};

struct Args {
  CUtensorMap a, b;
  CUtensorMap o;       // the output, boxes of 128 bytes x 32 rows, if tma
  CUtensorMap o_lo;    // BATCH: what the output's rounding left, times 2048, if has_lo
  CUtensorMap at, bt;  // UPPER: the same matrix in MN-major boxes; WGRAD: the experts' tails
  const int32_t* offsets;
  int E, R, M, N, K;
  Div nt, per;  // column tiles, and tiles an expert (not PRODUCT)
  void* out;
  long long ld, es;
  int out_type, tma;  // (else: rows that start anywhere)
  int has_lo;
  int n_lim;          // columns that may be stored
  const void* c;      // BATCH, SYM: FP16 rows in 16-byte pieces; WGRAD: the FP32 output
  const void* c_lo;   // what c's rounding left, times 2048, or null
  long long c_ld, c_es;
  float alpha, beta;
  const float *alpha_e, *beta_e;  // per expert, or null
  uint32_t formats;
  int32_t* status;
  long long limit;
};

struct Tile {
  int e, row0, nrows, col0;  // output rows [row0, row0 + nrows) of this CTA, first column
  int a_mn, b_mn;            // this CTA's first A row and B row (or column) of the maps
  int k0, kb, last16;        // first k (WGRAD: row), k-blocks, and 16-deep steps of the last
  int segs;                  // parts of the sum, SEG k-blocks each
  bool tail;                 // WGRAD: the last k-block is the expert's tail
  int boxes;                 // A boxes of the single product form
};

__device__ __forceinline__ void tma_load_3d(const void* map, void* dst, uint32_t bar, int c0, int c1,
                                            int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(const void* map, void* dst, uint32_t bar_cluster,
                                                 int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar_cluster)
      : "memory");
}

// MN-major tile: 64 of the M (or N) index in a 128-byte row, one row a k, 64 rows a chunk of
// 8192 bytes; the eight-row groups of 1024 bytes follow each other along k.
__device__ __forceinline__ uint64_t sdesc_mn_major_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(8192u >> 4) << 16;  // next 64 of the M (N) index
  d |= (uint64_t)(1024u >> 4) << 32;  // next 8 of k
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}
template <int TYPE>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (TYPE == MOE_DTYPE_BF16) {
    return pack_bf16x2(lo, hi);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1,
                                             int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(src))
      : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// This thread's stores have read their shared memory (all: and are performed).
__device__ __forceinline__ void tma_stores_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void tma_stores_done() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// A warp's 32 rows x 128 bytes in shared memory: 16-byte piece c of row r at place c ^ (r & 7), the
// 128-byte swizzle of a TMA store; a lane writing its row and eight lanes reading one row both
// meet every bank once.
__device__ __forceinline__ uint4* piece(uint4* st, int r, int c) { return st + 8 * r + (c ^ (r & 7)); }

// Epilogue of one warp: its 32 rows (TMEM lanes at taddr) by every other 128-byte span of the
// tile's columns, from span `first`.  With a map the block leaves by TMA (clipped at the output's
// ends), else (an expert's last rows, sums added to the output, rows that start anywhere) through
// registers, four whole spans an instruction.  out and c point to the rows' first element at
// the tile's first column.
template <int TYPE, bool ADD16, bool ADD32>
__device__ __forceinline__ void store_tile(uint32_t taddr, uint4* st, int lane, int first,
                                           const CUtensorMap* map, int col0, int row0, int e,
                                           void* out, long long ld, bool vec, int nrows, int ncols,
                                           const void* c, long long c_ld, float alpha, float beta,
                                           const CUtensorMap* map_lo = nullptr,
                                           const void* c_lo = nullptr) {
  constexpr int COLS = TYPE == MOE_DTYPE_F32 ? 32 : 64, PER = COLS / 8;  // of a span, of a piece
  constexpr int BYTES = 128 / COLS;
#pragma unroll 1
  for (int c0 = first * COLS; c0 < ncols; c0 += 2 * COLS) {
    const int cp = lane & 7, r4 = lane >> 3;  // this lane's piece and row (of four) in memory order
    const bool in = c0 + cp * PER < ncols;
    uint4 add[8];
    auto fetch = [&](const void* from) {
      const uint8_t* src = static_cast<const uint8_t*>(from) + (size_t)(c0 + cp * PER) * BYTES;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + r4;
        add[i] = in && r < nrows ? *reinterpret_cast<const uint4*>(src + r * c_ld * BYTES)
                                 : make_uint4(0, 0, 0, 0);
      }
    };
    uint32_t w[32], v[TYPE == MOE_DTYPE_F32 ? 1 : 64];
    if constexpr (TYPE == MOE_DTYPE_F32) {
      tmem_ld_32x32b_x32(taddr + c0, w);
      tmem_ld_wait();
    } else {
      // v = a v + b add: what was fetched in memory order reaches this lane's row through st
      auto stage = [&]() {
#pragma unroll
        for (int i = 0; i < 8; ++i) *piece(st, 4 * i + r4, cp) = add[i];
        __syncwarp();
      };
      auto added = [&](float a, float b) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint4 x = *piece(st, lane, q);
          const uint32_t h[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
            uint32_t *lo = &v[8 * q + 2 * j], *hi = lo + 1;
            *lo = __float_as_uint(fmaf(a, __uint_as_float(*lo), b * f.x));
            *hi = __float_as_uint(fmaf(a, __uint_as_float(*hi), b * f.y));
          }
        }
      };
      if constexpr (ADD16) {
        if (c_lo != nullptr) fetch(c_lo);
        else fetch(c);
        if (lane == 0) tma_stores_read();
        __syncwarp();
        stage();
      }
      tmem_ld_32x32b_x32(taddr + c0, *reinterpret_cast<uint32_t(*)[32]>(v));
      tmem_ld_32x32b_x32(taddr + c0 + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
      tmem_ld_wait();
      if constexpr (ADD16) {
        if (c_lo != nullptr) {
          added(alpha, beta * (1.0f / 2048.0f));
          fetch(c);
          __syncwarp();
          stage();
          added(1.0f, beta);
        } else {
          added(alpha, beta);
        }
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        float lo = __uint_as_float(v[2 * j]), hi = __uint_as_float(v[2 * j + 1]);
        if constexpr (!ADD16) {
          lo *= alpha;
          hi *= alpha;
        }
        w[j] = pack16<TYPE>(lo, hi);
      }
    }
    if constexpr (!ADD16) {
      if (lane == 0) tma_stores_read();
      __syncwarp();
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
      *piece(st, lane, q) = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    if (map != nullptr) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) tma_store_3d(map, st, col0 + c0, row0, e);
      if constexpr (TYPE == MOE_DTYPE_F16 && ADD16) {
        if (map_lo != nullptr) {
          if (lane == 0) tma_stores_read();
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint32_t l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[4 * q + j]));
              l[j] = pack16<TYPE>((__uint_as_float(v[8 * q + 2 * j]) - f.x) * 2048.0f,
                                  (__uint_as_float(v[8 * q + 2 * j + 1]) - f.y) * 2048.0f);
            }
            *piece(st, lane, q) = make_uint4(l[0], l[1], l[2], l[3]);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) tma_store_3d(map_lo, st, col0 + c0, row0, e);
        }
      }
      continue;
    }
    __syncwarp();
    if (vec) {
      uint8_t* dst = static_cast<uint8_t*>(out) + (size_t)(c0 + cp * PER) * BYTES;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + r4;
        uint4 x = *piece(st, r, cp);
        if constexpr (ADD32) {
          if (in && r < nrows) {
            const float4 y = *reinterpret_cast<const float4*>(dst + r * ld * BYTES);
            x.x = __float_as_uint(__uint_as_float(x.x) + y.x);
            x.y = __float_as_uint(__uint_as_float(x.y) + y.y);
            x.z = __float_as_uint(__uint_as_float(x.z) + y.z);
            x.w = __float_as_uint(__uint_as_float(x.w) + y.w);
          }
        }
        if (in && r < nrows) *reinterpret_cast<uint4*>(dst + r * ld * BYTES) = x;
      }
    } else if constexpr (TYPE != MOE_DTYPE_F32) {  // rows that start anywhere: two columns a lane
      uint16_t* dst = static_cast<uint16_t*>(out) + c0 + 2 * lane;
      const int n = ncols - c0 - 2 * lane;
#pragma unroll 4
      for (int r = 0; r < 32; ++r) {
        const uint32_t x = reinterpret_cast<const uint32_t*>(piece(st, r, lane >> 2))[lane & 3];
        if (r < nrows && n > 0) dst[r * ld] = (uint16_t)x;
        if (r < nrows && n > 1) dst[r * ld + 1] = (uint16_t)(x >> 16);
      }
    }
    __syncwarp();
  }
}

// The same for an expert without rows: zeros.
__device__ __forceinline__ void zero_tile(uint4* st, int lane, int first, int cols, const CUtensorMap* map,
                                          int col0, int row0, int e, int ncols) {
  if (lane == 0) tma_stores_read();
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 8; ++q) *piece(st, lane, q) = make_uint4(0, 0, 0, 0);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0)
    for (int c0 = first * cols; c0 < ncols; c0 += 2 * cols) tma_store_3d(map, st, col0 + c0, row0, e);
}

// Adds the accumulator at `part` to the one at `sum`, the columns that store_tile() gives this warp.
template <int COLS>
__device__ __forceinline__ void add_part(uint32_t sum, uint32_t part, int first, int ncols) {
#pragma unroll 1
  for (int c0 = first * COLS; c0 < ncols; c0 += 2 * COLS) {
#pragma unroll 1
    for (int c = c0; c < c0 + COLS; c += 32) {
      uint32_t a[32], b[32];
      tmem_ld_32x32b_x32(sum + c, a);
      tmem_ld_32x32b_x32(part + c, b);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; ++j)
        a[j] = __float_as_uint(__uint_as_float(a[j]) + __uint_as_float(b[j]));
      tmem_st_32x32b_x32(sum + c, a);
    }
  }
  tmem_st_wait();
}

template <int CTAS, int BN, Kind KIND, Major A, Major B>
__global__ void __launch_bounds__(THREADS, 1) train_gemm_kernel(const __grid_constant__ Args p) {
  using C = Shape<CTAS, BN>;
  constexpr int TM = GM * CTAS;
  constexpr bool BOXED = KIND == PRODUCT && CTAS == 1;
  constexpr bool PARTS = KIND == PRODUCT || KIND == WGRAD;
  extern __shared__ __align__(1024) uint8_t smem[];  // (the swizzle's period; there is no other)
  uint8_t* sA = smem;
  uint8_t* sB = smem + C::STAGES * C::A_BYTES;
  uint4* s_epi = reinterpret_cast<uint4*>(sB + C::STAGES * C::B_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(s_epi) + C::EPI_BYTES);
  uint64_t* full = bars;
  uint64_t* empty = bars + C::STAGES;
  uint64_t* tfull = bars + 2 * C::STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* peer_abort = abort_flag + 1;  // the other CTA's flag, written by it at its end
  volatile int* issued = abort_flag + 2;  // k-blocks issued of A and B here, and by the other CTA
  int* s_total = reinterpret_cast<int*>(tmem_slot + 7);
  int* s_bad = s_total + 1;
  volatile int* committed = s_bad + 1;  // by the issuer: k-blocks, uses of either accumulator
  int* s_off = reinterpret_cast<int*>(tmem_slot + 12);
  int* s_prefix = s_off + (kMaxE + 1);  // PRODUCT: first unit of an expert
  int* s_exp = s_prefix;                // WGRAD: experts by falling number of rows

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CTAS == 2 ? (int)cluster_ctarank() : 0;
  const int P = gridDim.x / CTAS, unit0 = blockIdx.x / CTAS;
  const int NT = p.nt.d, MT = (p.M + TM - 1) / TM;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    *peer_abort = 0;
    for (int i = 0; i < 4; ++i) issued[i] = 0;
    for (int i = 0; i < 3; ++i) committed[i] = 0;
    *s_bad = (smem_u32(smem) & 1023u) != 0;  // (never: asked for above)
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], EPI_WARPS * CTAS);  // the epilogue warps
    }
    mbar_init(mma_done, 1);
    fence_mbar_init();
    prefetch_tensormap(&p.a);
    prefetch_tensormap(&p.b);
  }
  pdl_wait();
  if (warp == 1) {
    if constexpr (CTAS == 2) tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
    else tmem_alloc(tmem_slot, C::TMEM_COLS);
  }
  pdl_launch_dependents();
  if constexpr (KIND == PRODUCT || KIND == WGRAD) {
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) s_off[e] = __ldg(p.offsets + e);
    __syncthreads();
    // 0 = o_0 <= o_1 <= ... <= o_E = R
    for (int e = threadIdx.x; e < p.E; e += blockDim.x)
      if (s_off[e + 1] < s_off[e] || (e == 0 && s_off[0] != 0) ||
          (e == p.E - 1 && s_off[p.E] != p.R))
        *s_bad = 1;
    if constexpr (KIND == WGRAD) {
      for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        const int n = s_off[e + 1] - s_off[e];
        int r = 0;
        for (int f = 0; f < p.E; ++f) {
          const int m = s_off[f + 1] - s_off[f];
          r += m > n || (m == n && f < e);
        }
        s_exp[r] = e;
      }
      if (threadIdx.x == 0) *s_total = p.E * p.per.d;
    } else if (warp == 5) {
      int carry = 0;
      for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int e = e0 + lane;
        const int n = e < p.E ? max(0, s_off[e + 1] - s_off[e]) : 0;
        const int units = (n + TM - 1) / TM * NT;
        int v = units;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
          if (lane >= d) v += o;
        }
        if (e < p.E) s_prefix[e] = carry + v - units;
        carry += __shfl_sync(0xFFFFFFFFu, v, 31);
      }
      if (lane == 0) *s_total = carry;
    }
  } else if (threadIdx.x == 0) {
    *s_total = p.E * p.per.d;
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) cluster_sync();  // barriers and tensor memory exist before remote use
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if (*s_bad && threadIdx.x == 0) flag_error(p.status, MOE_ERR_DEVICE_CHECK);
  const int total = *s_bad ? 0 : *s_total;

  // Units in turn over the CTAs (pairs); a weight gradient's cost goes with the expert's rows,
  // so its units come in falling order and every other turn runs backwards.
  auto unit_of = [&](int i) {
    if (KIND == WGRAD && (i & 1)) return i * P + P - 1 - unit0;
    return i * P + unit0;
  };
  auto tile_of = [&](int u) {
    Tile t;
    t.boxes = 0;
    if constexpr (KIND == PRODUCT) {
      int lo = 0, hi = p.E - 1;  // largest e with s_prefix[e] <= u
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_prefix[mid] <= u) lo = mid;
        else hi = mid - 1;
      }
      const int local = u - s_prefix[lo], mt = local / p.nt;
      t.e = lo;
      t.row0 = s_off[lo] + mt * TM + rank * GM;
      t.nrows = min(GM, max(0, s_off[lo + 1] - t.row0));
      t.col0 = (local - mt * NT) * BN;
      t.a_mn = t.row0;
      if constexpr (BOXED) t.boxes = (t.nrows + BOX_ROWS - 1) / BOX_ROWS;
    } else {
      const int x = u / p.per;
      int local = u - x * p.per.d, mt, nt;
      if constexpr (KIND == SYM) {
        mt = 0;
        while (local >= MT - mt) local -= MT - mt++;
        nt = mt + local;
      } else {
        mt = local / p.nt;
        nt = local - mt * NT;
      }
      t.e = KIND == WGRAD ? s_exp[x] : x;
      t.row0 = mt * TM + rank * GM;
      t.nrows = min(GM, max(0, p.M - t.row0));
      t.col0 = nt * BN;
      t.a_mn = t.row0;
    }
    t.b_mn = t.col0 + rank * C::BROWS;
    const int k = KIND == WGRAD ? s_off[t.e + 1] - s_off[t.e] : p.K;
    t.k0 = KIND == WGRAD ? s_off[t.e] : 0;
    t.kb = (k + GK - 1) / GK;
    t.tail = KIND == WGRAD && k % GK != 0;
    t.last16 = (k - (t.kb - 1) * GK + UK - 1) / UK;
    t.segs = PARTS ? (t.kb + SEG - 1) / SEG : 1;
    return t;
  };
  // the k-blocks of this CTA's units, in order
  int it = 0, wi = 0, wkb = 0;  // k-blocks issued; next unit, next k-block of the present one
  Tile wt;
  wt.kb = 0;
  auto advance = [&]() {
    while (wkb >= wt.kb) {
      if (wi * P >= total) return false;
      const int u = unit_of(wi++);
      if (u >= total) return false;
      wt = tile_of(u);
      wkb = 0;
    }
    return true;
  };
  const bool second = warp == B_WARP;  // loads B
  const uint32_t full0 = CTAS == 2 ? mapa_shared(smem_u32(full), 0) : smem_u32(full);
  auto load = [&](int s) {
    const bool upper = (second ? B : A) == UPPER;
    const bool mn = (second ? B : A) == MN ||
                    (upper && wkb * GK / TM < (second ? wt.b_mn : wt.a_mn) / TM);
    const bool tail = KIND == WGRAD && wt.tail && wkb == wt.kb - 1;
    const bool other = tail || (upper && mn);
    const CUtensorMap* m = second ? (other ? &p.bt : &p.b) : (other ? &p.at : &p.a);
    const int k = tail ? 0 : wt.k0 + wkb * GK;
    const int e = KIND == WGRAD ? (tail ? wt.e : 0) : KIND == PRODUCT && !second ? 0 : wt.e;
    const int x = second ? wt.b_mn : wt.a_mn;
    uint8_t* d = second ? sB + s * C::B_BYTES : sA + s * C::A_BYTES;
    const uint32_t bar = full0 + 8 * s;
    if (!second) {  // the phase's one arrival, with the bytes of both operands (and CTAs)
      if (CTAS == 2) {
        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::STAGE_BYTES);
      } else {
        mbar_arrive_expect_tx(&full[s],
                              C::B_BYTES + (BOXED ? wt.boxes * BOX_ROWS * GK * 2 : C::A_BYTES));
      }
    }
    auto one = [&](uint8_t* dst, int c0, int c1) {
      if constexpr (CTAS == 2) tma_load_3d_pair(m, dst, bar, c0, c1, e);
      else tma_load_3d(m, dst, bar, c0, c1, e);
    };
    if (mn) {
      one(d, x, k);
      one(d + 8192, x + 64, k);
    } else if (BOXED && !second) {
      for (int j = 0; j < wt.boxes; ++j) one(d + j * BOX_ROWS * 128, k, x + j * BOX_ROWS);
    } else {
      one(d, k, x);
    }
    ++wkb;
    ++it;
  };

  bool loads = false;
  if (warp == 0 || second) {
    if (elect_one()) {
      // ----------------------------------------------------------- producers
      loads = true;
      int s = 0;
      uint32_t ph = 1;
      bool ok = true;
      while (advance()) {
        ok = mbar_wait_bounded(&empty[s], ph, abort_flag, p.status, p.limit);
        if (!ok) break;
        load(s);
        if (++s == C::STAGES) {
          s = 0;
          ph ^= 1;
        }
      }
      // the last k-blocks' commits arrive in this CTA, the odd one too: it does not leave before
      // (the epilogue has waited for every accumulator's)
      for (int i = it > C::STAGES ? it - C::STAGES : 0; i < it && ok; ++i)
        ok = mbar_wait_bounded(&empty[i % C::STAGES], (i / C::STAGES) & 1, abort_flag, p.status,
                               p.limit);
      issued[second] = it;
      if constexpr (CTAS == 2)
        st_shared_remote(mapa_shared(smem_u32((const void*)(issued + 2 + second)), rank ^ 1), it);
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t idesc0 = p.formats | (1u << 4) | ((uint32_t)(BN >> 3) << 17) |
                              ((uint32_t)(TM >> 4) << 24);
      // descriptors of stage 0, in both majors; a stage and a 16-deep step only add to the address
      const uint64_t a_km = sdesc_k_major_sw128(smem_u32(sA)), a_tm = sdesc_mn_major_sw128(smem_u32(sA));
      const uint64_t b_km = sdesc_k_major_sw128(smem_u32(sB)), b_tm = sdesc_mn_major_sw128(smem_u32(sB));
      constexpr uint32_t KM_STEP = UK * 2 / 16, MN_STEP = UK * 128 / 16;
      int s = 0, acc0 = 0, blocks = 0;
      int uses[2] = {0, 0};  // of either accumulator
      uint32_t ph = 0;
      bool aborted = false;
      for (int i = 0; i * P < total && !aborted; ++i) {
        const int u = unit_of(i);
        if (u >= total) break;
        const Tile t = tile_of(u);
        if (t.kb == 0) continue;
        // a sum's first part stays where it is, the others pass through the other accumulator
        for (int seg = 0; seg < t.segs && !aborted; ++seg) {
          const int acc = seg == 0 ? acc0 : acc0 ^ 1;
          const int used = acc ? uses[1] : uses[0];
          if (!mbar_wait_bounded(&tempty[acc], (used & 1) ^ 1, abort_flag, p.status, p.limit)) {
            aborted = true;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * BN;
          const int kb0 = PARTS ? seg * SEG : 0, kb1 = PARTS ? min(t.kb, kb0 + SEG) : t.kb;
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait_bounded(&full[s], ph, abort_flag, p.status, p.limit)) {
              aborted = true;
              break;
            }
            tc_fence_after();
            const bool a_mn = A == MN || (A == UPPER && kb * GK / TM < t.row0 / TM);
            const bool b_mn = B == MN || (B == UPPER && kb * GK / TM < t.col0 / TM);
            const uint32_t idesc = idesc0 | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16);
            const uint64_t da = (a_mn ? a_tm : a_km) + (uint32_t)(s * (C::A_BYTES / 16));
            const uint64_t db = (b_mn ? b_tm : b_km) + (uint32_t)(s * (C::B_BYTES / 16));
            const uint32_t ga = a_mn ? MN_STEP : KM_STEP, gb = b_mn ? MN_STEP : KM_STEP;
            auto mma = [&](int kk) {
              const uint32_t more = kk > 0 || kb > kb0 ? 1u : 0u;
              if constexpr (CTAS == 2)
                mma_bf16_pair(d_tmem, da + kk * ga, db + kk * gb, idesc, more);
              else
                mma_bf16(d_tmem, da + kk * ga, db + kk * gb, idesc, more);
            };
            if (kb + 1 < t.kb || t.last16 == GK / UK) {
#pragma unroll
              for (int kk = 0; kk < GK / UK; ++kk) mma(kk);
            } else {
              for (int kk = 0; kk < t.last16; ++kk) mma(kk);
            }
            if constexpr (CTAS == 2) mma_commit_pair(&empty[s], 0x3);
            else mma_commit(&empty[s]);
            ++blocks;
            if (++s == C::STAGES) {
              s = 0;
              ph ^= 1;
            }
          }
          if (aborted) break;
          if constexpr (CTAS == 2) mma_commit_pair(&tfull[acc], 0x3);
          else mma_commit(&tfull[acc]);
          if (acc) ++uses[1];
          else ++uses[0];
        }
        acc0 ^= 1;
      }
      // every MMA this thread issued completes before tensor memory is released
      if constexpr (CTAS == 2) mma_commit_pair(mma_done, 0x1);
      else mma_commit(mma_done);
      wait_drain(mma_done, 0, kSpinLimitCycles);
      const int done[3] = {blocks, uses[0], uses[1]};
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        committed[i] = done[i];
        if constexpr (CTAS == 2)
          st_shared_remote(mapa_shared(smem_u32((const void*)(committed + i)), 1), done[i]);
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    const int first = (warp - 2) >> 2;
    uint4* st = s_epi + (warp - 2) * (32 * 8);
    int tcount = 0, odd = 0;  // PARTS, bit a of odd: the next use of accumulator a is an odd one
    // the next use's products of accumulator a are there
    auto ready = [&](int a) {
      int ok = 1;
      if (lane == 0)
        ok = mbar_wait_bounded(&tfull[a], (PARTS ? odd >> a : tcount >> 1) & 1, abort_flag, p.status,
                               p.limit);
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (PARTS) odd ^= 1 << a;
      tc_fence_after();
      return ok != 0;
    };
    auto release = [&](int a) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CTAS == 2) mbar_arrive_remote(mapa_shared(smem_u32(&tempty[a]), 0));
        else mbar_arrive(&tempty[a]);
      }
    };
    for (int i = 0; i * P < total; ++i) {
      const int u = unit_of(i);
      if (u >= total) break;
      const Tile t = tile_of(u);
      if (KIND == WGRAD && t.kb == 0 && p.c != nullptr) continue;  // nothing to add
      const int acc = tcount & 1;
      const bool sums = KIND != WGRAD || t.kb > 0;
      if constexpr (KIND == BATCH) {  // this tile's rows of c move into L2 while it is multiplied
        const int row = t.row0 + q * 32 + lane;
        if (row < p.M) {
          const long long at = t.e * p.c_es + row * p.c_ld;
          for (int col = t.col0 + 64 * first; col < min(p.n_lim, t.col0 + BN); col += 128) {
            prefetch_l2(static_cast<const __half*>(p.c) + at + col);
            if (p.c_lo) prefetch_l2(static_cast<const __half*>(p.c_lo) + at + col);
          }
        }
      }
      if (sums) {
        if (!ready(acc)) break;
      }
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN);
      const int nrows = min(32, t.nrows - q * 32);
      const int ncols = min(BN, p.n_lim - t.col0);
      if constexpr (PARTS) {
        bool ok = true;
        for (int seg = 1; seg < t.segs && ok; ++seg) {
          ok = ready(acc ^ 1);
          if (ok && nrows > 0) {
            const uint32_t part = acc ? taddr - BN : taddr + BN;
            if (p.out_type == MOE_DTYPE_F32) add_part<32>(taddr, part, first, ncols);
            else add_part<64>(taddr, part, first, ncols);
          }
          if (ok) release(acc ^ 1);
        }
        if (!ok) break;
      }
      if (nrows > 0) {
        const int row0 = t.row0 + q * 32;
        const long long at = (KIND == PRODUCT ? 0 : t.e * p.es) + row0 * p.ld + t.col0;
        void* out = static_cast<uint8_t*>(p.out) + at * (p.out_type == MOE_DTYPE_F32 ? 4 : 2);
        const int oe = KIND == PRODUCT ? 0 : t.e;
        if constexpr (KIND == BATCH || KIND == SYM) {
          const CUtensorMap* map = p.tma ? &p.o : nullptr;
          const float alpha = p.alpha * (p.alpha_e ? __ldg(p.alpha_e + t.e) : 1.0f);
          const float beta = p.beta * (p.beta_e ? __ldg(p.beta_e + t.e) : 1.0f);
          const long long c_at = t.e * p.c_es + row0 * p.c_ld + t.col0;
          const __half* c = static_cast<const __half*>(p.c) + c_at;
          const __half* c_lo = p.c_lo ? static_cast<const __half*>(p.c_lo) + c_at : nullptr;
          if (KIND == BATCH && p.out_type == MOE_DTYPE_BF16)  // (the last step's result)
            store_tile<MOE_DTYPE_BF16, true, false>(taddr, st, lane, first, map, t.col0, row0,
                                                    oe, out, p.ld, false, nrows, ncols, c, p.c_ld,
                                                    alpha, beta, nullptr,
                                                    KIND == BATCH ? c_lo : nullptr);
          else if (p.c != nullptr)
            store_tile<MOE_DTYPE_F16, true, false>(taddr, st, lane, first, map, t.col0, row0, oe,
                                                   out, p.ld, false, nrows, ncols, c, p.c_ld, alpha,
                                                   beta, KIND == BATCH && p.has_lo ? &p.o_lo : nullptr,
                                                   KIND == BATCH ? c_lo : nullptr);
          else
            store_tile<MOE_DTYPE_F16, false, false>(taddr, st, lane, first, map, t.col0, row0,
                                                    oe, out, p.ld, false, nrows, ncols, nullptr, 0,
                                                    alpha, 0.0f);
        } else {
          // (a product's rows behind the expert's last belong to the next one)
          const CUtensorMap* map = KIND == WGRAD || nrows == 32 ? &p.o : nullptr;
          if (!sums) {
            zero_tile(st, lane, first, p.out_type == MOE_DTYPE_F32 ? 32 : 64, map, t.col0, row0, oe,
                      ncols);
          } else if (p.out_type == MOE_DTYPE_F32) {
            if (KIND == WGRAD && p.c != nullptr)
              store_tile<MOE_DTYPE_F32, false, true>(taddr, st, lane, first, nullptr, 0, 0, 0,
                                                     out, p.ld, true, nrows, ncols, nullptr, 0, 1.0f,
                                                     1.0f);
            else
              store_tile<MOE_DTYPE_F32, false, false>(taddr, st, lane, first, map, t.col0, row0,
                                                      oe, out, p.ld, true, nrows, ncols, nullptr, 0,
                                                      1.0f, 0.0f);
          } else if (p.out_type == MOE_DTYPE_BF16) {
            store_tile<MOE_DTYPE_BF16, false, false>(taddr, st, lane, first, map, t.col0, row0,
                                                     oe, out, p.ld, true, nrows, ncols, nullptr, 0,
                                                     1.0f, 0.0f);
          } else {
            store_tile<MOE_DTYPE_F16, false, false>(taddr, st, lane, first, map, t.col0, row0,
                                                    oe, out, p.ld, true, nrows, ncols, nullptr, 0,
                                                    1.0f, 0.0f);
          }
        }
      }
      if (sums) {
        release(acc);
        ++tcount;
      }
    }
    if (lane == 0) tma_stores_done();
  }

  tc_fence_before();
  __syncthreads();
  bool aborted = *abort_flag != 0;
  if constexpr (CTAS == 2) {
    if (threadIdx.x == 0 && aborted)
      st_shared_remote(mapa_shared(smem_u32((const void*)peer_abort), rank ^ 1), 1);
    cluster_sync();  // no CTA leaves or frees tensor memory while the pair may still use it
    aborted = aborted || *peer_abort != 0;  // (the same in both CTAs)
  }
  if (aborted) {
    // All MMAs are complete and no role waits any more.  Copies into the last STAGES slots may
    // still be in flight.  A stage that one producer has issued and another has not gets the
    // other's bytes now (its slot's last MMAs are complete, or the one could not have issued
    // it), so that its barrier completes; the even CTA waits for the bytes of both.
    // A role that gave up did not wait for the commits that arrive in its CTA: thread 0 does.
    const int most = max(max(issued[0], issued[1]), max(issued[2], issued[3]));
    if (threadIdx.x == 0) {
      const int blocks = committed[0];
      for (int i = (blocks > C::STAGES ? blocks - C::STAGES : 0); i < blocks; ++i)
        wait_drain(&empty[i % C::STAGES], (i / C::STAGES) & 1, kSpinLimitCycles);
      for (int a = 0; a < 2; ++a)
        if (committed[1 + a] > 0) wait_drain(&tfull[a], (committed[1 + a] - 1) & 1, kSpinLimitCycles);
    }
    if (loads)
      while (it < most && advance()) load(it % C::STAGES);
    if (threadIdx.x == 0 && rank == 0)
      for (int i = (most > C::STAGES ? most - C::STAGES : 0); i < most; ++i)
        wait_drain(&full[i % C::STAGES], (i / C::STAGES) & 1, kSpinLimitCycles);
    if constexpr (CTAS == 2) cluster_sync();  // the odd CTA's copies count on the even's barriers
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CTAS == 2) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// The rows of each expert's partial last k-block (fewer than 64) to tails [E][64][cols], filled up
// with zeros to the 16 rows that an MMA reads; x's and then dy's.  A block a row, so that all rows
// are under way at once (eight blocks an expert, a row after the other, took 13 us).
__global__ void __launch_bounds__(256)
    tails_kernel(const int32_t* __restrict__ offsets, int R, const uint8_t* x, long long x_bytes, int K,
                 const uint8_t* dy, long long dy_bytes, int N, uint4* tx, uint4* tdy) {
  pdl_wait();
  pdl_launch_dependents();
  const int r = blockIdx.x, e = blockIdx.y;
  const int lo = __ldg(offsets + e), hi = __ldg(offsets + e + 1);
  if (lo < 0 || hi <= lo || hi > R) return;  // (a bad sequence: the product reports it and reads nothing)
  const int rem = (hi - lo) % GK;
  if (r >= (rem + UK - 1) / UK * UK) return;
  const long long row = (long long)(hi - rem) + r, at = (long long)e * GK + r;
  const uint4* sx = reinterpret_cast<const uint4*>(x + row * x_bytes);
  const uint4* sd = reinterpret_cast<const uint4*>(dy + row * dy_bytes);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const bool in = r < rem;
  for (int c = threadIdx.x; c < max(K, N) / 8; c += blockDim.x) {
    const bool a = c < K / 8, b = c < N / 8;
    const uint4 u = in && a ? __ldg(sx + c) : zero, v = in && b ? __ldg(sd + c) : zero;
    if (a) tx[at * (K / 8) + c] = u;
    if (b) tdy[at * (N / 8) + c] = v;
  }
}

template <int CTAS, int BN, Kind KIND, Major A, Major B>
cudaError_t launch(Args& p, long long units, cudaStream_t s) {
  using C = Shape<CTAS, BN>;
  constexpr int TM = GM * CTAS;
  const int MT = (p.M + TM - 1) / TM;
  p.nt = make_div((p.N + BN - 1) / BN);
  if (KIND != PRODUCT) p.per = make_div(KIND == SYM ? MT * (MT + 1) / 2 : MT * p.nt.d);
  auto kern = train_gemm_kernel<CTAS, BN, KIND, A, B>;
  static int cache[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  pdl_attr(attr[0]);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CTAS;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  int most = dev < 64 ? cache[dev] : 0;  // CTAs resident at once
  if (most == 0) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (err != cudaSuccess) return err;
    most = device_sm_count();
    if (CTAS == 2) {
      cfg.gridDim = dim3(2 * most, 1, 1);
      cfg.attrs = attr + 1;
      cfg.numAttrs = 1;
      int clusters = 0;
      err = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
      if (err != cudaSuccess) return err;
      if (clusters < 1) return cudaErrorInvalidConfiguration;
      most = 2 * clusters;
    }
    if (dev < 64) cache[dev] = most;
  }
  const long long grid = units * CTAS < most ? units * CTAS : most;
  if (grid == 0) return cudaSuccess;
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = CTAS == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

bool encode_out(CUtensorMap* m, const void* out, int type, uint64_t cols, uint64_t rows, int E,
                long long ld, long long es) {
  return encode_out_3d(m, out, type == MOE_DTYPE_F32, cols, rows, E, ld, es);
}

uint32_t formats_of(int dtype) {  // A and B: BF16, or both FP16
  return dtype == MOE_DTYPE_BF16 ? (1u << 7) | (1u << 10) : 0u;
}

}  // namespace

// The pair form's 256-row tiles need rows to fill them; with fewer, the single form loads no more
// than the rows there are.  64 experts with unevenly spread rows, 2048 x 2048 BF16, pair
// against single, at 32, 64, 96, 128, 256 and 512 rows an expert on average: 89 against 84 us, 91
// against 86, 94 against 96, 95 against 110, 122 against 170, 200 against 298 (768 x 2048 crosses at
// the same place).  Nor does it pay where 128 x 128 tiles do not go round the SMs once: 8 experts of
// 256 rows, 512 x 512, 8.1 us against 6.6, 2 of 1000 rows, 1000 x 1000, 12.7 against 11.7.  Both
// forms give a row the same bits.
static bool product_pairs(int E, int R, int N) {
  return (long long)R >= 96LL * E && (long long)(R / 128) * ((N + 127) / 128) > device_sm_count();
}

// The pair form of the Newton-Schulz products halves the bytes that an SM reads a product, but
// makes tiles of twice the side.  A product takes as many turns of the SMs as its tiles need, a pair's
// twice as long as a single CTA's, and a single CTA's turn costs a quarter more for its bytes; a step
// is the Gram product over the long side, its square over the short one (both upper tiles only), and the
// product over the short side.  Of 48 stacks between 256 and 4096 this takes the slower form for seven, by
// 3% on average (13% at worst: 16 of 512 x 512, 152 us against 135).  Whole updates, pair against single:
// 8 of 512 x 512 143 against 101 us, 64 of 300 x 520 290 against 250, 8 of 1024 x 1024 264 against 238, 5 of
// 1439 x 1001 250 against 315, 64 of 768 x 2048 1429 against 1504, 64 of 1024 x 2048 2206 against 2525.  Both
// forms give the same bits.
bool batch_pairs(int E, int rows, int cols) {
  const long long S = rows < cols ? rows : cols, L = rows < cols ? cols : rows;
  if (S <= 256) return false;
  auto step = [&](int tile, int at_once) {
    const long long s = (S + tile - 1) / tile, l = (L + tile - 1) / tile;
    const long long half = (E * s * (s + 1) / 2 + at_once - 1) / at_once;
    const long long whole = (E * s * l + at_once - 1) / at_once;
    return (L + S) * half + S * whole;
  };
  const int sms = device_sm_count();
  return 4 * 2 * step(256, sms / 2) <= 5 * step(128, sms);
}

cudaError_t launch_product(const TrainProduct& q, cudaStream_t s) {
  if (q.R == 0) return cudaSuccess;
  const bool pair = product_pairs(q.E, q.R, q.N);
  Args p = {};
  if (!encode_16bit_3d(&p.a, q.x, q.K, q.R, 1, q.x_ld, 0, pair ? GM : BOX_ROWS))
    return cudaErrorInvalidValue;
  const bool okb = q.turned ? encode_16bit_3d(&p.b, q.w, q.K, q.N, q.E, q.w_ld, q.w_es, 128)
                            : encode_16bit_3d(&p.b, q.w, q.N, q.K, q.E, q.w_ld, q.w_es, GK);
  if (!okb) return cudaErrorInvalidValue;
  p.offsets = q.offsets;
  p.E = q.E;
  p.R = q.R;
  p.N = p.n_lim = q.N;
  p.K = q.K;
  p.out = q.y;
  p.ld = q.y_ld;
  p.out_type = q.y_type;
  if (!encode_out(&p.o, q.y, q.y_type, q.N, q.R, 1, q.y_ld, 0)) return cudaErrorInvalidValue;
  p.formats = formats_of(q.type);
  p.status = q.status;
  p.limit = q.limit;
  const int bn = pair ? 256 : 128, tm = pair ? 256 : 128;
  const long long tiles = (q.R + tm - 1) / tm + (q.E < q.R ? q.E : q.R);
  const long long units = tiles * ((q.N + bn - 1) / bn);
  if (pair)
    return q.turned ? launch<2, 256, PRODUCT, KM, KM>(p, units, s)
                    : launch<2, 256, PRODUCT, KM, MN>(p, units, s);
  return q.turned ? launch<1, 128, PRODUCT, KM, KM>(p, units, s)
                  : launch<1, 128, PRODUCT, KM, MN>(p, units, s);
}

static long long wgrad_units(const TrainWgrad& q, int t) {
  return (long long)q.E * ((q.K + t - 1) / t) * ((q.N + t - 1) / t);
}

// The pair form's 256 x 256 tiles need rows to multiply, three turns of the SMs to go round, and not much
// more than a quarter of them may be empty.  With few rows an expert the output's way out is the time:
// FP32 leaves single CTAs as fast, and 16 bits the pairs faster once there are many tiles.  64 unevenly
// loaded experts, BF16 in, pair against single, FP32 and BF16 out: 16 rows each, 768 x 2048 81.4 / 52.6
// against 81.1 / 60.7 us, 192 x 1024 19.1 / 17.9 against 17.1 / 17.3; 128 rows, 768 x 2048 93.2 / 56.4 against 87.4 /
// 66.1; 512 rows, 768 x 2048 112 / 88 against 144 / 112, 192 x 1024 32.2 / 28.1 against 34.0 / 29.9, 384 x 384 26.4 / 22.9
// against 21.9 / 18.6, 192 x 192 15.0 / 14.7 against 13.5 / 13.3; 8 experts of 2048 rows, 1024 x 1024 31.6 / 29.1 against
// 38.0 / 35.1, 512 x 512 22.5 / 22.3 against 17.2 / 17.1.  Both forms give the same bits.
static bool wgrad_pairs(const TrainWgrad& q) {
  const long long single = wgrad_units(q, 128), sms = device_sm_count();
  if (single <= 3 * sms || 5 * 4 * wgrad_units(q, 256) > 7 * single) return false;
  return (long long)q.R >= 256LL * q.E || (q.out_type != MOE_DTYPE_F32 && single > 24 * sms);
}

size_t wgrad_tail_bytes(int E, int cols) { return (size_t)E * GK * cols * 2; }

cudaError_t launch_wgrad(const TrainWgrad& q, cudaStream_t s) {
  Args p = {};
  if (!encode_16bit_3d(&p.a, q.x, q.K, q.R, 1, q.x_ld, 0, GK) ||
      !encode_16bit_3d(&p.b, q.dy, q.N, q.R, 1, q.dy_ld, 0, GK) ||
      !encode_16bit_3d(&p.at, q.tail_x, q.K, GK, q.E, q.K, (uint64_t)GK * q.K, GK) ||
      !encode_16bit_3d(&p.bt, q.tail_dy, q.N, GK, q.E, q.N, (uint64_t)GK * q.N, GK))
    return cudaErrorInvalidValue;
  cudaError_t err = launch_pdl(tails_kernel, dim3(GK, q.E), dim3(256), 0, s, q.offsets, q.R,
                               static_cast<const uint8_t*>(q.x), 2 * q.x_ld, q.K,
                               static_cast<const uint8_t*>(q.dy), 2 * q.dy_ld, q.N,
                               static_cast<uint4*>(q.tail_x), static_cast<uint4*>(q.tail_dy));
  if (err != cudaSuccess) return err;
  p.offsets = q.offsets;
  p.E = q.E;
  p.R = q.R;
  p.M = q.K;
  p.N = p.n_lim = q.N;
  p.out = q.out;
  p.ld = q.ld;
  p.es = q.es;
  p.out_type = q.out_type;
  if (q.accumulate) p.c = q.out;
  if (!encode_out(&p.o, q.out, q.out_type, q.N, q.K, q.E, q.ld, q.es)) return cudaErrorInvalidValue;
  p.formats = formats_of(q.type);
  p.status = q.status;
  p.limit = q.limit;
  const bool pair = wgrad_pairs(q);
  const int t = pair ? 256 : 128;
  const long long units = wgrad_units(q, t);
  return pair ? launch<2, 256, WGRAD, MN, MN>(p, units, s)
              : launch<1, 128, WGRAD, MN, MN>(p, units, s);
}

cudaError_t launch_batch(const TrainBatch& q, cudaStream_t s) {
  const bool pair = q.pair;
  Args p = {};
  auto encode = [&](CUtensorMap* m, const void* x, bool mn, int mn_size, long long ld, long long es) {
    return mn ? encode_16bit_3d(m, x, mn_size, q.K, q.E, ld, es, GK)
              : encode_16bit_3d(m, x, q.K, mn_size, q.E, ld, es, GM);
  };
  const bool a_mn = q.form == TrainBatch::GRAM_COLS;
  const bool b_mn = a_mn || q.form == TrainBatch::LEFT;
  const bool square = q.form == TrainBatch::SQUARE;
  if (!encode(&p.a, q.a, a_mn, q.M, q.a_ld, q.a_es) || !encode(&p.b, q.b, b_mn, q.N, q.b_ld, q.b_es))
    return cudaErrorInvalidValue;
  if ((square || q.form == TrainBatch::LEFT) && !encode(&p.at, q.a, true, q.M, q.a_ld, q.a_es))
    return cudaErrorInvalidValue;
  if ((square || q.form == TrainBatch::RIGHT) && !encode(&p.bt, q.b, true, q.N, q.b_ld, q.b_es))
    return cudaErrorInvalidValue;
  p.E = q.E;
  p.M = q.M;
  p.N = q.N;
  p.K = q.K;
  p.out = q.out;
  p.ld = q.ld;
  p.es = q.es;
  p.out_type = q.out_type;
  // columns of a padded buffer may be written up to its row length (they hold zeros)
  p.n_lim = q.padded ? (q.N + 7) / 8 * 8 : q.N;
  // (a TMA store ends a row with a whole 16-byte piece, whatever the map's extent)
  p.tma = q.padded || (q.N % 8 == 0 && q.ld % 8 == 0 && (q.E == 1 || q.es % q.ld == 0));
  if (p.tma && !encode_out(&p.o, q.out, q.out_type, p.n_lim, q.M, q.E, q.ld, q.es))
    return cudaErrorInvalidValue;
  if (q.out_lo != nullptr) {
    p.has_lo = 1;
    if (!encode_out(&p.o_lo, q.out_lo, q.out_type, p.n_lim, q.M, q.E, q.ld, q.es))
      return cudaErrorInvalidValue;
  }
  p.c_lo = q.c_lo;
  p.c = q.c;
  p.c_ld = q.c_ld;
  p.c_es = q.c_es;
  p.alpha = q.alpha;
  p.beta = q.beta;
  p.alpha_e = q.alpha_e;
  p.beta_e = q.beta_e;
  p.formats = formats_of(MOE_DTYPE_F16);
  p.status = q.status;
  p.limit = q.limit;
  const int t = pair ? 256 : 128;
  const long long mt = (q.M + t - 1) / t, nt = (q.N + t - 1) / t;
  const bool half = q.form != TrainBatch::LEFT && q.form != TrainBatch::RIGHT;
  const long long units = q.E * (half ? mt * (mt + 1) / 2 : mt * nt);
  switch (q.form) {
    case TrainBatch::GRAM_ROWS:
      return pair ? launch<2, 256, SYM, KM, KM>(p, units, s) : launch<1, 128, SYM, KM, KM>(p, units, s);
    case TrainBatch::GRAM_COLS:
      return pair ? launch<2, 256, SYM, MN, MN>(p, units, s) : launch<1, 128, SYM, MN, MN>(p, units, s);
    case TrainBatch::SQUARE:
      return pair ? launch<2, 256, SYM, UPPER, UPPER>(p, units, s)
                  : launch<1, 128, SYM, UPPER, UPPER>(p, units, s);
    case TrainBatch::LEFT:
      return pair ? launch<2, 256, BATCH, UPPER, MN>(p, units, s)
                  : launch<1, 128, BATCH, UPPER, MN>(p, units, s);
    default:
      return pair ? launch<2, 256, BATCH, KM, UPPER>(p, units, s)
                  : launch<1, 128, BATCH, KM, UPPER>(p, units, s);
  }
}

}  // namespace moe

// Products that train the experts, on the 5th-generation tensor cores (tcgen05 + TMEM + TMA):
//
//   PRODUCT  y[r] = x[r] W_e (W [E, K, N]) or x[r] W_e^T (W [E, N, K]) for the rows r of expert e
//   WGRAD    dW_e = sum over the rows r of expert e of x[r]^T dy[r]
//   BATCH    out_e = alpha A_e B_e + beta C_e, one of each an expert (Newton-Schulz steps)
//   SYM      the same where the result is symmetric (X X^T, its square): the tiles on and above
//            the diagonal are computed and stored twice
//
// All read the operands in the caller's layout.  An operand whose contraction index runs along
// its rows (x and W^T of a product) is staged K-major, the others (W, and both operands of a
// weight gradient) MN-major: tcgen05 takes either from 128-byte-swizzled shared memory, so
// nothing is transposed or packed beforehand.
//
// Roles of a CTA (192 threads): warp 0 the TMA producer, warp 1 the MMA issuer, warps 2..5
// the epilogue, over a ring of k-blocks of 64 and two accumulators in TMEM.  Forms:
//   pair     two CTAs share one M = 256 MMA over 256 columns (cta_group::2): each SM stages
//            32 KB a k-block for 256 x 256 x 64 products
//   single   one CTA, 128 x 128, for few rows: of A only the 16-row boxes that hold rows of the
//            expert are loaded, so that the ring streams weights
//
// A weight gradient contracts over an expert's rows, which end anywhere.  Its tensor maps are
// made on the device (wgrad_maps_kernel), one an expert and operand, that end with the expert's
// last row: TMA fills the rest of the last k-block with zeros, so another expert's rows (or
// infinities and NaN among them) never enter the sum.
//
// Bounded waits, and what happens when one runs out, as in expert_gemm.cu.
#include "common.cuh"
#include "kernels.cuh"
#include "pdl.cuh"
#include "train.cuh"

namespace moe {
namespace {

enum Kind { PRODUCT, WGRAD, BATCH, SYM };

constexpr int GM = 128, GK = 64, UK = 16;
constexpr int BOX_ROWS = 16;  // A boxes of the single form of a product

template <int CTAS, int BN>
struct Shape {
  static constexpr int STAGES = 6;
  static constexpr int A_BYTES = GM * GK * 2;
  static constexpr int BROWS = BN / CTAS;  // of B in this CTA
  static constexpr int B_BYTES = BROWS * GK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int TMEM_COLS = 2 * BN;
  static constexpr int NBAR = 2 * STAGES + 2 + 2 + 1;
  static constexpr int EPI_LD = 33;
  static constexpr int EPI_BYTES = 4 * 32 * EPI_LD * 4;
  static constexpr int SMEM_BYTES =
      1024 + STAGES * STAGE_BYTES + EPI_BYTES + NBAR * 8 + 32 + 3 * (kMaxE + 1) * 4;
};

struct Args {
  CUtensorMap a, b;
  const uint8_t* maps;  // WGRAD: kMapBytes each, the experts' A maps and then their B maps
  const int32_t* offsets;
  int E, R, M, N, K;
  void* out;
  long long ld, es;
  int out_type, turned, vec;  // turned: stored transposed; vec: rows in 16-byte pieces
  int m_lim, n_lim;           // rows and columns that may be stored
  const void* c;              // out += beta c, at the untransposed place; FP16, or FP32 as the output
  long long c_ld, c_es;
  int c_type;
  float alpha, beta;
  const float *alpha_e, *beta_e;  // per expert, or null
  uint32_t formats;
  int32_t* status;
  long long limit;
};

struct Tile {
  int e, row0, nrows, col0;  // output rows [row0, row0 + nrows) of this CTA, first column
  int a_mn, b_mn;            // this CTA's first A row and B row (or column) of the maps
  int kb, last16;            // k-blocks, and 16-deep steps of the last
  int boxes;                 // A boxes of the single product form
  bool mirror;
};

__device__ __forceinline__ void tma_load_3d(const void* map, void* dst, uint64_t* bar, int c0,
                                            int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
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
template <bool MN>
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, int k16) {
  if constexpr (MN) return sdesc_mn_major_sw128(saddr + k16 * (UK * 128));
  else return sdesc_k_major_sw128(saddr + k16 * (UK * 2));
}

__device__ __forceinline__ uint16_t to16(float v, int type) {
  return type == MOE_DTYPE_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v))
                                : __half_as_ushort(__float2half_rn(v));
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, int type) {
  return (uint32_t)to16(lo, type) | ((uint32_t)to16(hi, type) << 16);
}

// One 32 x 32 block of an accumulator that the warp has staged in shared memory (row i at
// i * 33: conflict-free by rows and by columns) goes to rows row0.. and columns col0.. of out,
// as far as nrows and ncols allow; `turned`: element (i, j) to row j, column i.
__device__ __forceinline__ void store_block(const float* st, int lane, void* out, long long ld,
                                            int type, bool vec, bool turned, long long row0,
                                            int col0, int nrows, int ncols) {
  // (i, j) of the output block; staged element (si, sj)
  const long long r0 = turned ? col0 : row0;
  const long long c0 = turned ? row0 : col0;
  const int nr = turned ? ncols : nrows, nc = turned ? nrows : ncols;
  const int di = turned ? 1 : 33, dj = turned ? 33 : 1;
  if (type == MOE_DTYPE_F32) {
    float* o = static_cast<float*>(out) + r0 * ld + c0;
    if (vec) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + (lane >> 3), c = 4 * (lane & 7);
        const float* s = st + r * di + c * dj;
        if (r < nr && c < nc)
          *reinterpret_cast<float4*>(o + r * ld + c) =
              make_float4(s[0], s[dj], s[2 * dj], s[3 * dj]);
      }
    } else {
#pragma unroll 8
      for (int r = 0; r < 32; ++r)
        if (r < nr && lane < nc) o[r * ld + lane] = st[r * di + lane * dj];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(out) + r0 * ld + c0;
    if (vec) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2), c = 8 * (lane & 3);
        const float* s = st + r * di + c * dj;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = pack16(s[2 * j * dj], s[(2 * j + 1) * dj], type);
        if (r < nr && c < nc)
          *reinterpret_cast<uint4*>(o + r * ld + c) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
#pragma unroll 8
      for (int r = 0; r < 32; ++r)
        if (r < nr && lane < nc) o[r * ld + lane] = to16(st[r * di + lane * dj], type);
    }
  }
}

// st = alpha st + beta c over the block (c FP16 in 16-byte pieces of a padded buffer, or FP32)
__device__ __forceinline__ void add_block(float* st, int lane, const void* c, long long ld,
                                          int type, bool vec, float beta, long long row0, int col0,
                                          int nrows, int ncols) {
  if (type == MOE_DTYPE_F16) {
    const uint16_t* p = static_cast<const uint16_t*>(c) + row0 * ld + col0;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2), cc = 8 * (lane & 3);
      v[i] = r < nrows && cc < ncols ? *reinterpret_cast<const uint4*>(p + r * ld + cc)
                                     : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float* s = st + (8 * i + (lane >> 2)) * 33 + 8 * (lane & 3);
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        s[2 * j] = fmaf(beta, f.x, s[2 * j]);
        s[2 * j + 1] = fmaf(beta, f.y, s[2 * j + 1]);
      }
    }
  } else {
    const float* p = static_cast<const float*>(c) + row0 * ld + col0;
#pragma unroll 8
    for (int r = 0; r < 32; ++r)
      if (r < nrows && lane < ncols) st[r * 33 + lane] = fmaf(beta, p[r * ld + lane], st[r * 33 + lane]);
  }
  __syncwarp();
}

template <int CTAS, int BN, Kind KIND, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(192, 1) train_gemm_kernel(const __grid_constant__ Args p) {
  using C = Shape<CTAS, BN>;
  constexpr int TM = GM * CTAS;
  constexpr bool BOXED = KIND == PRODUCT && CTAS == 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = base;
  uint8_t* sB = base + C::STAGES * C::A_BYTES;
  float* s_epi = reinterpret_cast<float*>(sB + C::STAGES * C::B_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(s_epi) + C::EPI_BYTES);
  uint64_t* full = bars;
  uint64_t* empty = bars + C::STAGES;
  uint64_t* tfull = bars + 2 * C::STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* peer_abort = abort_flag + 1;   // the other CTA's flag, and the k-blocks that it
  volatile int* peer_issued = abort_flag + 2;  // has issued: written by it at its end
  int* s_total = reinterpret_cast<int*>(tmem_slot + 4);
  int* s_bad = s_total + 1;
  int* s_off = reinterpret_cast<int*>(tmem_slot + 8);
  int* s_prefix = s_off + (kMaxE + 1);  // PRODUCT: first unit of an expert
  int* s_exp = s_prefix + (kMaxE + 1);  // WGRAD: experts by falling number of rows

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CTAS == 2 ? (int)cluster_ctarank() : 0;
  const int P = gridDim.x / CTAS, unit0 = blockIdx.x / CTAS;
  const int NT = (p.N + BN - 1) / BN;
  const int MT = (p.M + TM - 1) / TM;  // (not PRODUCT)

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    *peer_abort = 0;
    *peer_issued = 0;
    *s_bad = 0;
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 4 * CTAS);  // the epilogue warps
    }
    mbar_init(mma_done, 1);
    fence_mbar_init();
    if (KIND != WGRAD) prefetch_tensormap(&p.a);
    if (KIND != WGRAD) prefetch_tensormap(&p.b);
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
      if (threadIdx.x == 0) *s_total = p.E * MT * NT;
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
    *s_total = p.E * (KIND == SYM ? MT * (MT + 1) / 2 : MT * NT);
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
    t.mirror = false;
    if constexpr (KIND == PRODUCT) {
      int lo = 0, hi = p.E - 1;  // largest e with s_prefix[e] <= u
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_prefix[mid] <= u) lo = mid;
        else hi = mid - 1;
      }
      const int local = u - s_prefix[lo], mt = local / NT;
      t.e = lo;
      t.row0 = s_off[lo] + mt * TM + rank * GM;
      t.nrows = min(GM, max(0, s_off[lo + 1] - t.row0));
      t.col0 = (local - mt * NT) * BN;
      t.a_mn = t.row0;
      if constexpr (BOXED) t.boxes = (t.nrows + BOX_ROWS - 1) / BOX_ROWS;
    } else {
      const int per = KIND == SYM ? MT * (MT + 1) / 2 : MT * NT;
      const int x = u / per;
      int local = u - x * per, mt, nt;
      if constexpr (KIND == SYM) {
        mt = 0;
        while (local >= MT - mt) local -= MT - mt++;
        nt = mt + local;
        t.mirror = nt > mt;
      } else {
        mt = local / NT;
        nt = local - mt * NT;
      }
      t.e = KIND == WGRAD ? s_exp[x] : x;
      t.row0 = mt * TM + rank * GM;
      t.nrows = min(GM, max(0, p.m_lim - t.row0));
      t.col0 = nt * BN;
      t.a_mn = t.row0;
    }
    t.b_mn = t.col0 + rank * C::BROWS;
    const int k = KIND == WGRAD ? s_off[t.e + 1] - s_off[t.e] : p.K;
    t.kb = (k + GK - 1) / GK;
    t.last16 = (k - (t.kb - 1) * GK + UK - 1) / UK;
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
      if constexpr (KIND == WGRAD) {
        if (wt.kb > 0) {
          acquire_map(p.maps + (size_t)wt.e * kMapBytes);
          acquire_map(p.maps + (size_t)(p.E + wt.e) * kMapBytes);
        }
      }
    }
    return true;
  };
  auto load = [&](int s) {
    const void* ma = &p.a;
    const void* mb = &p.b;
    const int k = wkb * GK;
    int ea = KIND == PRODUCT ? 0 : wt.e, eb = wt.e;
    if constexpr (KIND == WGRAD) {
      ma = p.maps + (size_t)wt.e * kMapBytes;
      mb = p.maps + (size_t)(p.E + wt.e) * kMapBytes;
      ea = eb = 0;
    }
    uint8_t* da = sA + s * C::A_BYTES;
    uint8_t* db = sB + s * C::B_BYTES;
    uint32_t bar = 0;
    if constexpr (CTAS == 2) {
      if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::STAGE_BYTES);
      bar = mapa_shared(smem_u32(&full[s]), 0);
    } else {
      mbar_arrive_expect_tx(&full[s],
                            C::B_BYTES + (BOXED ? wt.boxes * BOX_ROWS * GK * 2 : C::A_BYTES));
    }
    auto one = [&](const void* m, uint8_t* d, int c0, int c1, int c2) {
      if constexpr (CTAS == 2) tma_load_3d_pair(m, d, bar, c0, c1, c2);
      else tma_load_3d(m, d, &full[s], c0, c1, c2);
    };
    if constexpr (A_MN) {
#pragma unroll
      for (int j = 0; j < GM / 64; ++j) one(ma, da + j * 8192, wt.a_mn + 64 * j, k, ea);
    } else if constexpr (BOXED) {
      for (int j = 0; j < wt.boxes; ++j)
        one(ma, da + j * BOX_ROWS * 128, k, wt.a_mn + j * BOX_ROWS, ea);
    } else {
      one(ma, da, k, wt.a_mn, ea);
    }
    if constexpr (B_MN) {
#pragma unroll
      for (int j = 0; j < C::BROWS / 64; ++j) one(mb, db + j * 8192, wt.b_mn + 64 * j, k, eb);
    } else {
      one(mb, db, k, wt.b_mn, eb);
    }
    ++wkb;
    ++it;
  };

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      while (advance()) {
        const int s = it % C::STAGES;
        if (!mbar_wait_bounded(&empty[s], ((it / C::STAGES) & 1) ^ 1, abort_flag, p.status,
                               p.limit))
          break;
        load(s);
      }
      if constexpr (CTAS == 2)
        st_shared_remote(mapa_shared(smem_u32((const void*)peer_issued), rank ^ 1), it);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t idesc = p.formats | (1u << 4) | ((uint32_t)A_MN << 15) |
                             ((uint32_t)B_MN << 16) | ((uint32_t)(BN >> 3) << 17) |
                             ((uint32_t)(TM >> 4) << 24);
      int jt = 0, tcount = 0;
      bool aborted = false;
      for (int i = 0; i * P < total && !aborted; ++i) {
        const int u = unit_of(i);
        if (u >= total) break;
        const Tile t = tile_of(u);
        if (t.kb == 0) continue;
        const int acc = tcount & 1;
        if (!mbar_wait_bounded(&tempty[acc], ((tcount >> 1) & 1) ^ 1, abort_flag, p.status,
                               p.limit))
          break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int kb = 0; kb < t.kb; ++kb, ++jt) {
          const int s = jt % C::STAGES;
          if (!mbar_wait_bounded(&full[s], (jt / C::STAGES) & 1, abort_flag, p.status, p.limit)) {
            aborted = true;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(sA + s * C::A_BYTES);
          const uint32_t b_addr = smem_u32(sB + s * C::B_BYTES);
          const int steps = kb + 1 < t.kb ? GK / UK : t.last16;
          for (int kk = 0; kk < steps; ++kk) {
            if constexpr (CTAS == 2)
              mma_bf16_pair(d_tmem, sdesc<A_MN>(a_addr, kk), sdesc<B_MN>(b_addr, kk), idesc,
                            (kb > 0 || kk > 0) ? 1u : 0u);
            else
              mma_bf16(d_tmem, sdesc<A_MN>(a_addr, kk), sdesc<B_MN>(b_addr, kk), idesc,
                       (kb > 0 || kk > 0) ? 1u : 0u);
          }
          if constexpr (CTAS == 2) mma_commit_pair(&empty[s], 0x3);
          else mma_commit(&empty[s]);
        }
        if (aborted) break;
        if constexpr (CTAS == 2) mma_commit_pair(&tfull[acc], 0x3);
        else mma_commit(&tfull[acc]);
        ++tcount;
      }
      // every MMA this thread issued completes before tensor memory is released
      if constexpr (CTAS == 2) mma_commit_pair(mma_done, 0x1);
      else mma_commit(mma_done);
      wait_drain(mma_done, 0, kSpinLimitCycles);
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    float* st = s_epi + q * 32 * C::EPI_LD;
    const int elt = p.out_type == MOE_DTYPE_F32 ? 4 : 2;
    const int c_elt = p.c_type == MOE_DTYPE_F32 ? 4 : 2;
    int tcount = 0;
    for (int i = 0; i * P < total; ++i) {
      const int u = unit_of(i);
      if (u >= total) break;
      const Tile t = tile_of(u);
      if (KIND == WGRAD && t.kb == 0 && p.c != nullptr) continue;  // nothing to add
      const int acc = tcount & 1;
      if (t.kb > 0) {
        int ok = 1;
        if (lane == 0)
          ok = mbar_wait_bounded(&tfull[acc], (tcount >> 1) & 1, abort_flag, p.status, p.limit);
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (!ok) break;
        tc_fence_after();
      }
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN);
      const int nrows = min(32, max(0, t.nrows - q * 32));
      const long long row0 = t.row0 + q * 32;
      const int ncols = min(BN, p.n_lim - t.col0);
      uint8_t* out = static_cast<uint8_t*>(p.out) + (KIND == PRODUCT ? 0 : t.e * p.es * elt);
      const float alpha = p.alpha * (p.alpha_e ? __ldg(p.alpha_e + t.e) : 1.0f);
      const float beta = p.beta * (p.beta_e ? __ldg(p.beta_e + t.e) : 1.0f);
      if (nrows > 0) {
#pragma unroll 1
        for (int c0 = 0; c0 < ncols; c0 += 32) {
          if (t.kb > 0) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(taddr + c0, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) st[lane * 33 + j] = alpha * __uint_as_float(v[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) st[lane * 33 + j] = 0.0f;
          }
          __syncwarp();
          const int nc = min(32, ncols - c0);
          if (KIND != PRODUCT && p.c != nullptr)
            add_block(st, lane, static_cast<const uint8_t*>(p.c) + t.e * p.c_es * c_elt, p.c_ld,
                      p.c_type, p.vec, beta, row0, t.col0 + c0, nrows, nc);
          store_block(st, lane, out, p.ld, p.out_type, p.vec, p.turned, row0, t.col0 + c0, nrows,
                      nc);
          if (KIND == SYM && t.mirror)  // (a padded row has more columns than there are rows)
            store_block(st, lane, out, p.ld, p.out_type, p.vec, true, row0, t.col0 + c0, nrows,
                        min(nc, p.N - t.col0 - c0));
          __syncwarp();
        }
      }
      if (t.kb > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CTAS == 2) mbar_arrive_remote(mapa_shared(smem_u32(&tempty[acc]), 0));
          else mbar_arrive(&tempty[acc]);
        }
        ++tcount;
      }
    }
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
    // still be in flight.  A stage that only one CTA of a pair has issued gets the other's
    // bytes now, so that its barrier completes; the even CTA waits for the bytes of both.
    if (threadIdx.x == 0) {
      if constexpr (CTAS == 2)
        while (it < *peer_issued && advance()) load(it % C::STAGES);
      if (rank == 0)
        for (int i = (it > C::STAGES ? it - C::STAGES : 0); i < it; ++i)
          wait_drain(&full[i % C::STAGES], (i / C::STAGES) & 1, kSpinLimitCycles);
    }
    if constexpr (CTAS == 2) cluster_sync();  // the odd CTA's copies count on the even's barriers
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CTAS == 2) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// One warp makes one expert's map of one operand: the caller's map of all rows with the base
// address and the number of rows of the expert.
struct BaseMaps {
  CUtensorMap a, b;
};
__global__ void __launch_bounds__(32)
    wgrad_maps_kernel(const __grid_constant__ BaseMaps base, const int32_t* __restrict__ offsets,
                      int E, int R, const uint8_t* x, long long x_bytes, const uint8_t* dy,
                      long long dy_bytes, uint8_t* maps) {
  __shared__ alignas(128) uint32_t m[32];
  const bool second = blockIdx.x >= E;
  const int e = blockIdx.x - (second ? E : 0), lane = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int lo = __ldg(offsets + e), hi = __ldg(offsets + e + 1);
  if (lo < 0 || hi <= lo || hi > R) return;  // (a bad sequence: the product reports it and reads no map)
  m[lane] = reinterpret_cast<const uint32_t*>(second ? &base.b : &base.a)[lane];
  __syncwarp();
  if (lane == 0) {
    const uint64_t addr = reinterpret_cast<uint64_t>(
        second ? dy + (long long)lo * dy_bytes : x + (long long)lo * x_bytes);
    asm volatile("tensormap.replace.tile.global_address.shared::cta.b1024.b64 [%0], %1;" ::"r"(
                     smem_u32(m)),
                 "l"(addr)
                 : "memory");
    asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(
                     smem_u32(m)),
                 "r"(hi - lo)
                 : "memory");
  }
  __syncwarp();
  asm volatile(
      "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned "
      "[%0], [%1], 128;" ::"l"(maps + (size_t)blockIdx.x * kMapBytes),
      "r"(smem_u32(m))
      : "memory");
}

template <int CTAS, int BN, Kind KIND, bool A_MN, bool B_MN>
cudaError_t launch(const Args& p, long long units, cudaStream_t s) {
  using C = Shape<CTAS, BN>;
  auto kern = train_gemm_kernel<CTAS, BN, KIND, A_MN, B_MN>;
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
  cfg.blockDim = dim3(192, 1, 1);
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

uint32_t formats_of(int dtype) {  // A and B: BF16, or both FP16
  return dtype == MOE_DTYPE_BF16 ? (1u << 7) | (1u << 10) : 0u;
}

bool vec_ok(const void* out, int type, long long ld, long long es, long long n) {
  const int per = type == MOE_DTYPE_F32 ? 4 : 8;
  return (reinterpret_cast<uintptr_t>(out) & 15) == 0 && ld % per == 0 && es % per == 0 &&
         n % per == 0;
}

}  // namespace

// The pair form needs many rows an expert to fill its 256-row tiles; with fewer the single form
// loads no more than the rows there are and spreads an expert's columns over twice the CTAs.
bool product_pair_form(int E, int R) { return (long long)R >= 128LL * E; }

cudaError_t launch_product(const TrainProduct& q, cudaStream_t s) {
  if (q.R == 0) return cudaSuccess;
  const bool pair = product_pair_form(q.E, q.R);
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
  p.vec = vec_ok(q.y, q.y_type, q.y_ld, 0, q.N);
  p.alpha = 1.0f;
  p.formats = formats_of(q.type);
  p.status = q.status;
  p.limit = q.limit;
  const int bn = pair ? 256 : 128, tm = pair ? 256 : 128;
  const long long tiles = (q.R + tm - 1) / tm + (q.E < q.R ? q.E : q.R);
  const long long units = tiles * ((q.N + bn - 1) / bn);
  if (pair)
    return q.turned ? launch<2, 256, PRODUCT, false, false>(p, units, s)
                    : launch<2, 256, PRODUCT, false, true>(p, units, s);
  return q.turned ? launch<1, 128, PRODUCT, false, false>(p, units, s)
                  : launch<1, 128, PRODUCT, false, true>(p, units, s);
}

cudaError_t launch_wgrad(const TrainWgrad& q, cudaStream_t s) {
  BaseMaps base;
  if (!encode_16bit_3d(&base.a, q.x, q.K, q.R, 1, q.x_ld, 0, GK) ||
      !encode_16bit_3d(&base.b, q.dy, q.N, q.R, 1, q.dy_ld, 0, GK))
    return cudaErrorInvalidValue;
  cudaError_t err = launch_pdl(wgrad_maps_kernel, dim3(2 * q.E), dim3(32), 0, s, base, q.offsets,
                               q.E, q.R, static_cast<const uint8_t*>(q.x), 2 * q.x_ld,
                               static_cast<const uint8_t*>(q.dy), 2 * q.dy_ld, q.maps);
  if (err != cudaSuccess) return err;
  Args p = {};
  p.maps = q.maps;
  p.offsets = q.offsets;
  p.E = q.E;
  p.R = q.R;
  p.M = p.m_lim = q.K;
  p.N = p.n_lim = q.N;
  p.out = q.out;
  p.ld = q.ld;
  p.es = q.es;
  p.out_type = q.out_type;
  p.vec = vec_ok(q.out, q.out_type, q.ld, q.es, q.N);
  p.alpha = 1.0f;
  if (q.accumulate) {
    p.c = q.out;
    p.c_ld = q.ld;
    p.c_es = q.es;
    p.c_type = MOE_DTYPE_F32;
    p.beta = 1.0f;
  }
  p.formats = formats_of(q.type);
  p.status = q.status;
  p.limit = q.limit;
  const bool pair = q.K > 128 && q.N > 128;
  const int t = pair ? 256 : 128;
  const long long units = (long long)q.E * ((q.K + t - 1) / t) * ((q.N + t - 1) / t);
  return pair ? launch<2, 256, WGRAD, true, true>(p, units, s)
              : launch<1, 128, WGRAD, true, true>(p, units, s);
}

cudaError_t launch_batch(const TrainBatch& q, cudaStream_t s) {
  const int least = q.M < q.N ? q.M : q.N;
  const bool pair = least > 128;
  const uint32_t rows = 128;
  Args p = {};
  if (!encode_16bit_3d(&p.a, q.a, q.K, q.M, q.E, q.a_ld, q.a_es, GM)) return cudaErrorInvalidValue;
  const bool okb = q.sym ? encode_16bit_3d(&p.b, q.b, q.K, q.N, q.E, q.b_ld, q.b_es, rows)
                         : encode_16bit_3d(&p.b, q.b, q.N, q.K, q.E, q.b_ld, q.b_es, GK);
  if (!okb) return cudaErrorInvalidValue;
  p.E = q.E;
  p.M = p.m_lim = q.M;
  p.N = q.N;
  p.K = q.K;
  p.out = q.out;
  p.ld = q.ld;
  p.es = q.es;
  p.out_type = q.out_type;
  p.turned = q.turned;
  // columns of a padded buffer may be written up to its row length (they hold zeros)
  p.n_lim = q.padded ? (q.N + 7) / 8 * 8 : q.N;
  p.vec = q.padded || vec_ok(q.out, q.out_type, q.ld, q.es, q.turned ? q.M : q.N);
  p.c = q.c;
  p.c_ld = q.c_ld;
  p.c_es = q.c_es;
  p.c_type = MOE_DTYPE_F16;
  p.alpha = q.alpha;
  p.beta = q.beta;
  p.alpha_e = q.alpha_e;
  p.beta_e = q.beta_e;
  p.formats = formats_of(MOE_DTYPE_F16);
  p.status = q.status;
  p.limit = q.limit;
  const int t = pair ? 256 : 128;
  const long long mt = (q.M + t - 1) / t, nt = (q.N + t - 1) / t;
  const long long units = q.E * (q.sym ? mt * (mt + 1) / 2 : mt * nt);
  if (pair)
    return q.sym ? launch<2, 256, SYM, false, false>(p, units, s)
                 : launch<2, 256, BATCH, false, true>(p, units, s);
  return q.sym ? launch<1, 128, SYM, false, false>(p, units, s)
               : launch<1, 128, BATCH, false, true>(p, units, s);
}

}  // namespace moe

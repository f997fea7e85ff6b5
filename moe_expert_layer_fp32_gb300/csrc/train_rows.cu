// Row-wise operators that train the experts: SwiGLU and its gradient, and the first step of an
// orthogonalisation (norm and scaling).
#include "common.cuh"
#include "kernels.cuh"
#include "pdl.cuh"
#include "train.cuh"

namespace moe {
namespace {

template <int TYPE>
__device__ __forceinline__ float2 two(uint32_t v) {
  if constexpr (TYPE == MOE_DTYPE_BF16) return make_float2(bf16_lo(v), bf16_hi(v));
  else return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <int TYPE>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  if constexpr (TYPE == MOE_DTYPE_BF16) {
    return pack_bf16x2(lo, hi);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// s = sigmoid(g), act = g s, h = act u:
//   d_gate = w d u s (1 + g (1 - s)), d_up = w d act, d_w = sum d h, and w h once more for the
// down projection's gradient.  One rounding each; the row's sum in FP32.  The sigmoid is the special-function
// unit's, within 2^-23 (8 + 2 |g|): the roundings to 16 bits that follow are 2^-8 and 2^-11, and the row's
// sum, which alone is FP32, keeps that.
template <int TYPE>
__device__ __forceinline__ void swiglu_bwd_pair(uint32_t g, uint32_t u, uint32_t d, float w,
                                                uint32_t& dg, uint32_t& du, uint32_t& h,
                                                float& dw) {
  const float2 gf = two<TYPE>(g), uf = two<TYPE>(u), df = two<TYPE>(d);
  float2 rg, ru, rh;
  auto one = [&](float a, float b, float c, float& x, float& y, float& z) {
    const float s = __fdividef(1.0f, 1.0f + __expf(-a));
    const float act = a * s, hh = act * b, wd = w * c;
    x = wd * b * s * fmaf(a, 1.0f - s, 1.0f);
    y = wd * act;
    z = w * hh;
    dw = fmaf(c, hh, dw);
  };
  one(gf.x, uf.x, df.x, rg.x, ru.x, rh.x);
  one(gf.y, uf.y, df.y, rg.y, ru.y, rh.y);
  dg = pack<TYPE>(rg.x, rg.y);
  du = pack<TYPE>(ru.x, ru.y);
  h = pack<TYPE>(rh.x, rh.y);
}

// A warp a row, 16-byte pieces; PIECES of a lane's are loaded before the first is used.  Bound by its
// bytes: three values in and three out, 131072 x 768 BF16 in 181.3 us, 6.67 TB/s, 98% of the copy rate
// (513 x 1024: 5.4 us, the host's launch and two allocations).  One piece where a row has few, whose
// lanes would else wait with the rest of a group empty, four in long rows, whose warps have little else
// under way; gradient / forward of 2^20 x 100 BF16 values, by 1, 2, 3 and 4 pieces: rows of 256 196/99,
// 232/123, 267/120, 271/123 us; of 768 191/97, 199/112, 192/101, 194/96; of 1408 191/97, 197/119, 196/98, 198/98; of
// 2048 202/102, 195/113, 191/104, 195/100; of 8192 198/120, 193/97, 197/101, 193/97.
constexpr int ROW_WARPS = 8, LONG_ROW = 2048;

// Whether offsets [E + 1] are a non-decreasing sequence from 0 to R: the same answer in every thread of
// the block.
__device__ __forceinline__ bool block_sequence(const int32_t* __restrict__ offsets, int E, int R) {
  int bad = 0;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    const int a = __ldg(offsets + e), b = __ldg(offsets + e + 1);
    bad |= b < a || (e == 0 && a != 0) || (e == E - 1 && b != R);
  }
  return !__syncthreads_or(bad);
}

template <int TYPE, bool BWD, int PIECES>
__global__ void __launch_bounds__(32 * ROW_WARPS)
    swiglu_kernel(const uint8_t* __restrict__ gu, long long gu_ld, const uint8_t* __restrict__ d,
                  long long d_ld, const float* __restrict__ w, int R, int I, uint8_t* dgu,
                  long long dgu_ld, uint8_t* h, long long h_ld, float* d_w,
                  const int32_t* __restrict__ offsets, int E) {
  pdl_wait();
  pdl_launch_dependents();
  // (bad offsets: the product that d comes from wrote nothing)
  if (BWD && offsets && !block_sequence(offsets, E, R)) return;
  const int lane = threadIdx.x & 31;
  for (long long r = blockIdx.x * ROW_WARPS + (threadIdx.x >> 5); r < R;
       r += (long long)gridDim.x * ROW_WARPS) {
    const uint4* pg = reinterpret_cast<const uint4*>(gu + 2 * r * gu_ld);
    const uint4* pu = reinterpret_cast<const uint4*>(gu + 2 * (r * gu_ld + I));
    const uint4* pd = BWD ? reinterpret_cast<const uint4*>(d + 2 * r * d_ld) : nullptr;
    uint4* og = BWD ? reinterpret_cast<uint4*>(dgu + 2 * r * dgu_ld) : nullptr;
    uint4* ou = BWD ? reinterpret_cast<uint4*>(dgu + 2 * (r * dgu_ld + I)) : nullptr;
    uint4* oh = h ? reinterpret_cast<uint4*>(h + 2 * r * h_ld) : nullptr;
    const float wr = w ? __ldg(w + r) : 1.0f;
    float dw = 0.0f;
    const int n = I / 8;
    for (int c0 = lane; c0 < n; c0 += 32 * PIECES) {
      uint4 vg[PIECES], vu[PIECES], vd[PIECES];
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int c = c0 + 32 * i;
        if (c < n) {
          vg[i] = __ldcs(pg + c);
          vu[i] = __ldcs(pu + c);
          if constexpr (BWD) vd[i] = __ldcs(pd + c);
        }
      }
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int c = c0 + 32 * i;
        if (c < n) {
          const uint32_t* a = reinterpret_cast<const uint32_t*>(&vg[i]);
          const uint32_t* b = reinterpret_cast<const uint32_t*>(&vu[i]);
          uint4 rg, ru, rh;
          uint32_t *xg = reinterpret_cast<uint32_t*>(&rg), *xu = reinterpret_cast<uint32_t*>(&ru),
                   *xh = reinterpret_cast<uint32_t*>(&rh);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (BWD) {
              const uint32_t* e = reinterpret_cast<const uint32_t*>(&vd[i]);
              swiglu_bwd_pair<TYPE>(a[j], b[j], e[j], wr, xg[j], xu[j], xh[j], dw);
            } else {
              const float2 gf = two<TYPE>(a[j]), uf = two<TYPE>(b[j]);
              xh[j] = pack<TYPE>(wr * (silu_f32(gf.x) * uf.x), wr * (silu_f32(gf.y) * uf.y));
            }
          }
          if constexpr (BWD) {
            __stcs(og + c, rg);
            __stcs(ou + c, ru);
          }
          if (oh) __stcs(oh + c, rh);
        }
      }
    }
    if (BWD && d_w) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dw += __shfl_xor_sync(0xFFFFFFFFu, dw, o);
      if (lane == 0) d_w[r] = dw;
    }
  }
}

template <bool BWD>
cudaError_t launch_rows(const void* gu, long long gu_ld, const void* d, long long d_ld,
                        const float* w, int type, int R, int I, void* dgu, long long dgu_ld,
                        void* h, long long h_ld, float* d_w, const int32_t* offsets, int E,
                        cudaStream_t s) {
  if (R == 0) return cudaSuccess;
  const long long need = ((long long)R + ROW_WARPS - 1) / ROW_WARPS;
  const long long most = 8LL * device_sm_count();
  const dim3 grid((unsigned)(need < most ? need : most));
  const bool bf16 = type == MOE_DTYPE_BF16;
  auto kern = I < LONG_ROW ? (bf16 ? swiglu_kernel<MOE_DTYPE_BF16, BWD, 1> : swiglu_kernel<MOE_DTYPE_F16, BWD, 1>)
                           : (bf16 ? swiglu_kernel<MOE_DTYPE_BF16, BWD, 4> : swiglu_kernel<MOE_DTYPE_F16, BWD, 4>);
  return launch_pdl(kern, grid, dim3(32 * ROW_WARPS), 0, s, static_cast<const uint8_t*>(gu), gu_ld,
                    static_cast<const uint8_t*>(d), d_ld, w, R, I, static_cast<uint8_t*>(dgu),
                    dgu_ld, static_cast<uint8_t*>(h), h_ld, d_w, offsets, E);
}

__global__ void __launch_bounds__(256)
    no_rows_kernel(const int32_t* __restrict__ offsets, int E, int32_t* status, uint8_t* out, int elt,
                   int rows, int pieces, long long ld, long long es) {
  pdl_wait();
  pdl_launch_dependents();
  if (!block_sequence(offsets, E, 0)) {
    if (threadIdx.x == 0) flag_error(status, MOE_ERR_DEVICE_CHECK);
    return;
  }
  if (out == nullptr) return;
  for (long long i = blockIdx.x; i < (long long)E * rows; i += gridDim.x) {
    const long long e = i / rows, r = i - e * rows;
    uint4* row = reinterpret_cast<uint4*>(out + (e * es + r * ld) * elt);
    for (int c = threadIdx.x; c < pieces; c += blockDim.x) row[c] = make_uint4(0, 0, 0, 0);
  }
}

// ------------------------------------------------ start of an orthogonalisation ---
// Eight elements of a row as they lie in memory, and as FP32; VEC: whole 16-byte pieces, else element
// by element with zeros behind the row's end.
template <int TYPE, bool VEC>
struct Eight {
  static constexpr int ELT = TYPE == MOE_DTYPE_F32 ? 4 : 2;
  uint4 w[VEC ? ELT / 2 : 1];
  float f[VEC ? 1 : 8];
  __device__ __forceinline__ void load(const uint8_t* row, int c, int n) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < ELT / 2; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(row + ELT * c) + i);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = min(c + i, n - 1);
        float v;
        if constexpr (TYPE == MOE_DTYPE_F32) v = __ldg(reinterpret_cast<const float*>(row) + j);
        else if constexpr (TYPE == MOE_DTYPE_BF16)
          v = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[j]);
        else v = __half2float(reinterpret_cast<const __half*>(row)[j]);
        f[i] = c + i < n ? v : 0.0f;
      }
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    if constexpr (!VEC) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = f[i];
    } else {
      const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (TYPE == MOE_DTYPE_F32) {
          v[2 * i] = __uint_as_float(u[2 * i]), v[2 * i + 1] = __uint_as_float(u[2 * i + 1]);
        } else {
          const float2 t = two<TYPE>(u[i]);
          v[2 * i] = t.x, v[2 * i + 1] = t.y;
        }
      }
    }
  }
};

// f(piece, its elements) for the 8-element pieces of `rows` rows of n pieces, AHEAD of a thread's
// loaded before the first is used.
constexpr int AHEAD = 4;
template <int TYPE, bool VEC, typename F>
__device__ __forceinline__ void pieces(const uint8_t* m, long long row_bytes, int rows, const Div& n,
                                       int cols, F f) {
  const int total = rows * n.d;
  for (int i0 = threadIdx.x; i0 < total; i0 += AHEAD * blockDim.x) {
    Eight<TYPE, VEC> e[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int i = min(i0 + j * (int)blockDim.x, total - 1), r = i / n;
      e[j].load(m + r * row_bytes, 8 * (i - r * n.d), cols);
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int i = i0 + j * (int)blockDim.x;
      if (i < total) {
        float v[8];
        e[j].values(v);
        f(i, v);
      }
    }
  }
}

// Sums of squares: pieces whose sum leaves [2^-80, 2^100] are summed from values times 2^-80 (big) or
// 2^88 (small) instead, so that no finite matrix of up to 2^28 elements overflows (mid at most 2^125, big
// 2^(2 (128 - 80) + 28), small 2^(-80 + 2 * 88 + 25)) and the smallest value's square, 2^(2 (88 - 149)), is no
// subnormal number.
constexpr int kBig = -80, kSmall = 88;
struct Squares {
  float mid, big, small;
  __device__ void add(const float (&v)[8]) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(v[j], v[j], s);
    if (s >= 0x1p-80f && s <= 0x1p100f) {
      mid += s;
      return;
    }
    const bool tiny = s < 0x1p-80f;
    const float by = tiny ? 0x1p88f : 0x1p-80f;
    float t = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) t = fmaf(v[j] * by, v[j] * by, t);
    if (tiny) small += t;
    else big += t;  // (infinities and NaN too)
  }
};

__device__ __forceinline__ float block_sum(float v, float* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
  for (int i = 0; i < (int)blockDim.x / 32; ++i) t += sh[i];
  return t;
}

// parts [E][3][nb]: the sums of squares of nb groups of rows.  (64 x 1024 x 2048 BF16: 46 us, 5.8 TB/s;
// scale_kernel 78 us, 6.9 TB/s.)
template <int TYPE, bool VEC>
__global__ void __launch_bounds__(256)
    squares_kernel(const uint8_t* __restrict__ m, long long ld, long long es, int rows, int cols,
                   int per, Div n, float* __restrict__ parts) {
  __shared__ float sh[8];
  pdl_wait();
  pdl_launch_dependents();
  const int e = blockIdx.y, nb = gridDim.x;
  const int r0 = blockIdx.x * per, r1 = min(rows, r0 + per);
  Squares q = {0.0f, 0.0f, 0.0f};
  constexpr int ELT = TYPE == MOE_DTYPE_F32 ? 4 : 2;
  pieces<TYPE, VEC>(m + (e * es + r0 * ld) * ELT, ld * ELT, r1 - r0, n, cols,
                    [&](int, const float(&v)[8]) { q.add(v); });
  const float a = block_sum(q.mid, sh), b = block_sum(q.big, sh), c = block_sum(q.small, sh);
  if (threadIdx.x == 0) {
    float* o = parts + ((long long)e * 3) * nb + blockIdx.x;
    o[0] = a;
    o[nb] = b;
    o[2 * nb] = c;
  }
}

// x [E][rows][ldx] (ldx = cols padded to 8, the padding zero) = M 2^k in FP16, `per` rows a block.
// 2^k brings the norm to [512, 1024): elements of a BF16 matrix stay exact down to 2^-24 of the norm
// (below they are rounded to a multiple of 2^-33 of it at most), and neither a product of rows nor (with
// eps) 1 / norm comes near FP32's ends.
template <int TYPE, bool VEC>
__global__ void __launch_bounds__(256)
    scale_kernel(const uint8_t* __restrict__ m, long long ld, long long es, int rows, int cols,
                 int per, Div n, int ldx, float eps, const float* __restrict__ parts,
                 __half* __restrict__ x, __half* __restrict__ x_lo, float* __restrict__ f, int E) {
  __shared__ float sh[8];
  pdl_wait();
  pdl_launch_dependents();
  const int e = blockIdx.y, nb = gridDim.x;
  float s[3];
  for (int j = 0; j < 3; ++j) {
    float v = 0.0f;
    for (int i = threadIdx.x; i < nb; i += blockDim.x) v += parts[((long long)e * 3 + j) * nb + i];
    s[j] = block_sum(v, sh);
  }
  float root;  // |M| 2^by, which FP32 holds whatever |M| is
  int by = 0;
  if (!(s[1] <= 0.0f)) {  // (NaN too)
    root = sqrtf(ldexpf(s[0], 2 * kBig) + s[1]);
    by = kBig;
  } else if (!(s[0] <= 0.0f)) {
    root = sqrtf(s[0] + ldexpf(s[2], -2 * kSmall));
  } else {
    root = sqrtf(s[2]);
    by = kSmall;
  }
  int k = 0, ex = 0;
  const bool finite = root <= 0x1.fffffep127f;
  if (finite && root > 0.0f) {
    frexpf(root, &ex);  // root = r 2^ex, r in [0.5, 1)
    k = 10 - ex + by;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    // 2^-k / (|M| + eps), as 1 / (|M| 2^k + eps 2^k)
    const float norm = ldexpf(root, 10 - ex);
    float v = !finite ? __int_as_float(0x7FC00000) : root > 0.0f ? 1.0f / (norm + ldexpf(eps, k)) : 0.0f;
    f[e] = v;
    f[E + e] = v * v;
  }
  const float s1 = ldexpf(1.0f, k / 2), s2 = ldexpf(1.0f, k - k / 2);
  const int r0 = blockIdx.x * per, r1 = min(rows, r0 + per);
  constexpr int ELT = TYPE == MOE_DTYPE_F32 ? 4 : 2;
  const long long at = ((long long)e * rows + r0) * ldx;
  uint4* o = reinterpret_cast<uint4*>(x + at);
  uint4* o_lo = x_lo ? reinterpret_cast<uint4*>(x_lo + at) : nullptr;
  pieces<TYPE, VEC>(m + (e * es + r0 * ld) * ELT, ld * ELT, r1 - r0, n, cols,
                    [&](int i, const float(&v)[8]) {
                      uint32_t w[4], l[4];
#pragma unroll
                      for (int j = 0; j < 4; ++j) {
                        const float a = v[2 * j] * s1 * s2, b = v[2 * j + 1] * s1 * s2;
                        w[j] = pack<MOE_DTYPE_F16>(a, b);
                        const float2 h = two<MOE_DTYPE_F16>(w[j]);
                        l[j] = pack<MOE_DTYPE_F16>((a - h.x) * 2048.0f, (b - h.y) * 2048.0f);
                      }
                      o[i] = make_uint4(w[0], w[1], w[2], w[3]);
                      if (o_lo) o_lo[i] = make_uint4(l[0], l[1], l[2], l[3]);
                    });
}

template <int TYPE, bool VEC>
cudaError_t start(const uint8_t* m, long long ld, long long es, int E, int rows, int cols, float eps,
                  float* parts, __half* x, __half* x_lo, float* f, cudaStream_t s) {
  // rows a block: 32768 elements of large stacks (four rounds of loads a thread), fewer where that
  // would leave SMs with fewer than eight blocks
  const long long most = (long long)E * rows * cols / (8LL * device_sm_count());
  const int elements = most < 2048 ? 2048 : most > 32768 ? 32768 : (int)most;
  int per = (elements + cols - 1) / cols;
  if ((rows + per - 1) / per > kNormParts) per = (rows + kNormParts - 1) / kNormParts;
  const dim3 grid((rows + per - 1) / per, E);
  cudaError_t err = launch_pdl(squares_kernel<TYPE, VEC>, grid, dim3(256), 0, s, m, ld, es, rows, cols,
                               per, make_div((cols + 7) / 8), parts);
  if (err != cudaSuccess) return err;
  return launch_pdl(scale_kernel<TYPE, VEC>, grid, dim3(256), 0, s, m, ld, es, rows, cols, per,
                    make_div((cols + 7) / 8), (cols + 7) / 8 * 8, eps,
                    static_cast<const float*>(parts), x, x_lo, f, E);
}

}  // namespace

cudaError_t launch_swiglu(const void* gate_up, long long gu_ld, const float* w, int type, int R,
                          int I, void* h, long long h_ld, cudaStream_t s) {
  return launch_rows<false>(gate_up, gu_ld, nullptr, 0, w, type, R, I, nullptr, 0, h, h_ld, nullptr,
                            nullptr, 0, s);
}

cudaError_t launch_swiglu_bwd(const void* gate_up, long long gu_ld, const void* d, long long d_ld,
                              const float* w, int type, int R, int I, void* d_gate_up,
                              long long dgu_ld, void* h, long long h_ld, float* d_w,
                              const int32_t* offsets, int E, cudaStream_t s) {
  return launch_rows<true>(gate_up, gu_ld, d, d_ld, w, type, R, I, d_gate_up, dgu_ld, h, h_ld, d_w,
                           offsets, E, s);
}

cudaError_t launch_no_rows(const int32_t* offsets, int E, int32_t* status, void* out, int elt, int rows,
                           int cols, long long ld, long long es, cudaStream_t s) {
  const long long need = out ? (long long)E * rows : 1, most = 8LL * device_sm_count();
  return launch_pdl(no_rows_kernel, dim3((unsigned)(need < most ? need : most)), dim3(256), 0, s, offsets,
                    E, status, static_cast<uint8_t*>(out), elt, rows, cols * elt / 16, ld, es);
}

cudaError_t launch_orth_start(const void* m, int type, long long ld_m, long long es_m, int E,
                              int rows, int cols, float eps, float* parts, void* x, void* x_lo,
                              float* f, cudaStream_t s) {
  const uint8_t* src = static_cast<const uint8_t*>(m);
  __half *o = static_cast<__half*>(x), *l = static_cast<__half*>(x_lo);
  const int elt = type == MOE_DTYPE_F32 ? 4 : 2;
  const bool vec = cols % 8 == 0 && ld_m * elt % 16 == 0 && (E == 1 || es_m * elt % 16 == 0);
#define MOE_START(T)                                                                          \
  return vec ? start<T, true>(src, ld_m, es_m, E, rows, cols, eps, parts, o, l, f, s)            \
             : start<T, false>(src, ld_m, es_m, E, rows, cols, eps, parts, o, l, f, s)
  if (type == MOE_DTYPE_F32) MOE_START(MOE_DTYPE_F32);
  if (type == MOE_DTYPE_BF16) MOE_START(MOE_DTYPE_BF16);
  MOE_START(MOE_DTYPE_F16);
#undef MOE_START
}

}  // namespace moe

// Launchers of the operators that train the experts (train_gemm.cu, train_rows.cu).
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

// n / d for n < 2^31 by a multiplication: m = 2^32 (2^s - d) / d + 1, s = ceil(log2 d).
struct Div {
  uint32_t m;
  int s, d;
};
inline Div make_div(int d) {
  Div v = {0, 0, d};
  while ((1LL << v.s) < d) ++v.s;
  v.m = (uint32_t)(((1ULL << 32) * ((1ULL << v.s) - d)) / d + 1);
  return v;
}
__device__ __forceinline__ int operator/(int n, const Div& v) {
  return (int)((__umulhi((uint32_t)n, v.m) + (uint32_t)n) >> v.s);
}

// A map of 16-bit elements [d2][d1][d0], rows ld and slices es elements apart, boxes of
// 64 x box1 x 1 with 128-byte swizzle, zeros outside (moe_api.cu).
bool encode_16bit_3d(CUtensorMap* m, const void* ptr, uint64_t d0, uint64_t d1, uint64_t d2,
                     uint64_t ld, uint64_t es, uint32_t box1);

// The same for an output of FP32 or 16-bit elements, boxes of 128 bytes x 32 rows.
bool encode_out_3d(CUtensorMap* m, const void* ptr, bool fp32, uint64_t d0, uint64_t d1, uint64_t d2,
                   uint64_t ld, uint64_t es);

// y [R, N] of y_type = the rows of x [R, K] times their expert's matrix, [K, N] or (turned) [N, K].
struct TrainProduct {
  const void* x;
  const int32_t* offsets;
  const void* w;
  void* y;
  int E, R, K, N, type, y_type;
  bool turned;
  long long x_ld, w_ld, w_es, y_ld;
  int32_t* status;
  long long limit;
};
cudaError_t launch_product(const TrainProduct& q, cudaStream_t s);

// out [E, K, N] = (or, FP32, +=) the sums over each expert's rows of x [R, K]^T dy [R, N]; R > 0.
// tail_x, tail_dy: wgrad_tail_bytes(E, K) and (E, N) bytes of scratch.
struct TrainWgrad {
  const void *x, *dy;
  const int32_t* offsets;
  void* out;
  int E, R, K, N, type, out_type;
  bool accumulate;
  long long x_ld, dy_ld, ld, es;
  void *tail_x, *tail_dy;
  int32_t* status;
  long long limit;
};
size_t wgrad_tail_bytes(int E, int cols);
cudaError_t launch_wgrad(const TrainWgrad& q, cudaStream_t s);

// out_e = alpha A_e B_e + beta C_e (C null: without), out [M, N] over K, FP16 operands with padded
// rows.  Symmetric matrices (marked ~) hold the tiles on and above the diagonal: 256 wide if pair, else
// 128, the same choice in every call on them.
//   GRAM_ROWS  ~out = A A^T         A [M, K], b = a
//   GRAM_COLS  ~out = A^T A         A [K, M], b = a
//   SQUARE     ~out = A A           ~A [M, M], b = a
//   LEFT       out = A B            ~A [M, M], B [M, N]
//   RIGHT      out = A B            A [M, N], ~B [N, N]
// padded: out is a padded buffer too; else (LEFT, RIGHT) rows of any length.
// c_lo, out_lo (null: without): what the rounding of c and of a padded out left, times 2048, in
// FP16 and the same layouts; c then counts with both.
struct TrainBatch {
  enum Form { GRAM_ROWS, GRAM_COLS, SQUARE, LEFT, RIGHT } form;
  const void *a, *b, *c, *c_lo;
  void *out, *out_lo;
  int E, M, N, K, out_type;
  bool pair, padded;
  long long a_ld, a_es, b_ld, b_es, c_ld, c_es, ld, es;
  float alpha, beta;
  const float *alpha_e, *beta_e;
  int32_t* status;
  long long limit;
};
// The choice of `pair` for matrices of this size.
bool batch_pairs(int E, int rows, int cols);
cudaError_t launch_batch(const TrainBatch& q, cudaStream_t s);

// h [R, I] = w silu(gate) up of gate_up [R, 2 I] (w: [R] FP32 or null)
cudaError_t launch_swiglu(const void* gate_up, long long gu_ld, const float* w, int type, int R,
                          int I, void* h, long long h_ld, cudaStream_t s);
// its gradient for d [R, I]; h (w silu(gate) up) and d_w [R] may be null.  offsets [E + 1] (null:
// not looked at): nothing is written if they are not a sequence from 0 to R.
cudaError_t launch_swiglu_bwd(const void* gate_up, long long gu_ld, const void* d, long long d_ld,
                              const float* w, int type, int R, int I, void* d_gate_up,
                              long long dgu_ld, void* h, long long h_ld, float* d_w,
                              const int32_t* offsets, int E, cudaStream_t s);

// A grouped call without rows: offsets [E + 1] other than zeros are flagged, else (out not null) the E
// slices of rows x cols elements of elt bytes become zeros (rows of whole 16-byte pieces).
cudaError_t launch_no_rows(const int32_t* offsets, int E, int32_t* status, void* out, int elt, int rows,
                           int cols, long long ld, long long es, cudaStream_t s);

// First step of an orthogonalisation: x [E][rows][ld] FP16 (ld = cols padded to 8) = M 2^k, x_lo what its rounding left, times 2048 (null: without),
// f[e] = 2^-k / (|M| + eps), f[E + e] = f[e]^2.
constexpr int kNormParts = 512;  // at most, partial sums of squares an expert
cudaError_t launch_orth_start(const void* m, int type, long long ld_m, long long es_m, int E,
                              int rows, int cols, float eps, float* parts, void* x, void* x_lo, float* f,
                              cudaStream_t s);

// The whole orthogonalisation in one kernel, a CTA a matrix (train_orth.cu): at most 128 x 256 or
// 256 x 128.  coefficients: host.
bool orth_small(int rows, int cols);
cudaError_t launch_orth_small(const void* m, int type, long long ld, long long es, int E, int rows,
                              int cols, const float* coefficients, int steps, float eps, float scale,
                              void* out, int out_type, long long out_ld, long long out_es,
                              int32_t* status, long long limit, cudaStream_t s);

}  // namespace moe

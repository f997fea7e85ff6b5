// C ABI of the calls that train the experts (declared in include/moe.h): argument checks,
// workspace layouts and launch sequences.  As in moe_api.cu, no call allocates device memory or
// synchronises.
#include <math.h>

#include "common.cuh"
#include "kernels.cuh"
#include "train.cuh"

namespace moe {
namespace {

constexpr size_t kAlign = 256;
inline size_t up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

#define MOE_TRY(expr)            \
  do {                           \
    moe_status _s = (expr);      \
    if (_s != MOE_OK) return _s; \
  } while (0)

#define MOE_CUDA(expr)                              \
  do {                                              \
    if ((expr) != cudaSuccess) return MOE_ERR_CUDA; \
  } while (0)

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

template <typename T>
inline T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

bool is16(int dtype) { return dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_F16; }
bool known(int dtype) { return dtype == MOE_DTYPE_F32 || is16(dtype); }
int bytes_of(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

moe_status check_workspace(const void* ws, size_t have, size_t want) {
  if (ws == nullptr) return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) != 0) return MOE_ERR_MISALIGNED;
  return have < want ? MOE_ERR_WORKSPACE : MOE_OK;
}

moe_status check_grouped(int E, int K, int N) {
  if (E <= 0 || K <= 0 || N <= 0) return MOE_ERR_INVALID_ARG;
  if (E > kMaxE || K % 8 != 0 || N % 8 != 0 || K > 32768 || N > 32768) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
// Rows of a product: a tile may end 256 rows behind them, and tiles are numbered in 32 bits.
moe_status check_rows(long long R, int E, int N) {
  if (R < 0) return MOE_ERR_INVALID_ARG;
  if (R > (1LL << 31) - 512) return MOE_ERR_UNSUPPORTED;
  return (R / 128 + E + 1) * ((N + 127) / 128) >= (1LL << 30) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Rows of `cols` elements, ld apart, that start on 16-byte boundaries; ptr may be null if there
// is nothing to read.
moe_status check_matrix(const void* ptr, long long rows, long long cols, long long ld, int dtype) {
  if (ld < cols) return MOE_ERR_INVALID_ARG;
  if (ld >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
  if (ld * bytes_of(dtype) % 16 != 0) return MOE_ERR_MISALIGNED;
  return rows > 0 ? validate_ptr(ptr) : MOE_OK;
}
// E slices of rows x cols, es elements apart (a whole number of rows).
moe_status check_stack(const void* ptr, int E, long long rows, long long cols, long long ld,
                       long long es, int dtype) {
  MOE_TRY(check_matrix(ptr, 1, cols, ld, dtype));
  if (E > 1 && (es < rows * ld || es % ld != 0)) return MOE_ERR_INVALID_ARG;
  return es >= (1LL << 38) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// status word, then the weight gradient's tails of x and dy
struct GroupedLayout {
  size_t status, tail_x, tail_dy, total;
};
GroupedLayout grouped_layout(int E, int K, int N) {
  GroupedLayout L;
  L.status = 0;
  L.tail_x = up(kAlign);
  L.tail_dy = L.tail_x + up(wgrad_tail_bytes(E, K));
  L.total = L.tail_dy + up(wgrad_tail_bytes(E, N));
  return L;
}

moe_status do_product(const void* x, long long x_ld, int type, const int32_t* offsets,
                      const void* w, long long w_ld, long long w_es, bool turned, int R, int K,
                      int N, int E, void* y, long long y_ld, int y_type, void* ws,
                      cudaStream_t s) {
  if (R == 0) {
    MOE_CUDA(launch_no_rows(offsets, E, static_cast<int32_t*>(ws), nullptr, 0, 0, 0, 0, 0, s));
    return MOE_OK;
  }
  TrainProduct q;
  q.x = x;
  q.offsets = offsets;
  q.w = w;
  q.y = y;
  q.E = E;
  q.R = R;
  q.K = K;
  q.N = N;
  q.type = type;
  q.y_type = y_type;
  q.turned = turned;
  q.x_ld = x_ld;
  q.w_ld = w_ld;
  q.w_es = w_es;
  q.y_ld = y_ld;
  q.status = static_cast<int32_t*>(ws);
  q.limit = wait_limit();
  MOE_CUDA(launch_product(q, s));
  return MOE_OK;
}

moe_status do_wgrad(const void* x, long long x_ld, const void* dy, long long dy_ld, int type,
                    const int32_t* offsets, int R, int K, int N, int E, void* out, long long ld,
                    long long es, int out_type, bool accumulate, void* ws, cudaStream_t s) {
  if (R == 0) {
    MOE_CUDA(launch_no_rows(offsets, E, static_cast<int32_t*>(ws), accumulate ? nullptr : out,
                            bytes_of(out_type), K, N, ld, es, s));
    return MOE_OK;
  }
  TrainWgrad q;
  q.x = x;
  q.dy = dy;
  q.offsets = offsets;
  q.out = out;
  q.E = E;
  q.R = R;
  q.K = K;
  q.N = N;
  q.type = type;
  q.out_type = out_type;
  q.accumulate = accumulate;
  q.x_ld = x_ld;
  q.dy_ld = dy_ld;
  q.ld = ld;
  q.es = es;
  const GroupedLayout L = grouped_layout(E, K, N);
  q.tail_x = at<void>(ws, L.tail_x);
  q.tail_dy = at<void>(ws, L.tail_dy);
  q.status = static_cast<int32_t*>(ws);
  q.limit = wait_limit();
  MOE_CUDA(launch_wgrad(q, s));
  return MOE_OK;
}

// -------------------------------------------------------- orthogonalisation ---
struct OrthLayout {
  size_t status, parts, f, x0, x1, lo0, lo1, a, b, total;
};
OrthLayout orth_layout(int E, int rows, int cols) {
  const size_t m = rows < cols ? rows : cols;
  const size_t x = up((size_t)E * rows * ((cols + 7) / 8 * 8) * 2), a = up(E * m * ((m + 7) / 8 * 8) * 2);
  OrthLayout L;
  size_t o = 0;
  L.status = o;  o += up(kAlign);
  L.parts = o;   o += up((size_t)E * 3 * kNormParts * 4);
  L.f = o;       o += up((size_t)E * 2 * 4);
  L.x0 = o;      o += x;
  L.x1 = o;      o += x;
  L.lo0 = o;     o += x;
  L.lo1 = o;     o += x;
  L.a = o;       o += a;
  L.b = o;       o += a;
  L.total = o;
  return L;
}
constexpr float kHeld = 1024.0f;  // X, A and B are held in FP16 times this
constexpr int kMaxSteps = 64;
// The iterates (M itself, if FP32, and the next ones) also keep what their rounding to FP16 left,
// which counts in a X only: later steps lift a rounding there up to a times each, and B X does not
// lift it (B vanishes where the singular values do).  The last two need not (a rounding of
// theirs is lifted twice at most).  Without: an error of 0.041 for rank 8 of 500 x 720,
// 0.0021 for full-rank momenta; three kept 0.0024 and 0.0008, all five 0.0003 and 0.0009, at a read
// and a write of X more each (64 x 1024 x 2048 BF16: 2183 us without, 2250 with).  Three kept of ten
// steps: 1.8 for rank 8 of 300 x 500, eight 0.022 (FP32 throughout 0.021).
inline int keep_low(int steps) { return steps > 5 ? steps - 2 : 3; }

// Whether result e may lie in bytes of another matrix than e, whose CTA of the one-kernel form may not
// have read it yet.  (The chain of kernels writes out in its last launch.)
bool orth_crosses(const void* m, int dtype, long long ld, long long es, const void* out, long long out_ld,
                  long long out_es, int E, int rows, int cols) {
  const int b = bytes_of(dtype);
  if (E == 1 || (m == out && b == 2 && ld == out_ld && es == out_es)) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(m), o = reinterpret_cast<uintptr_t>(out);
  const uintptr_t a_end = a + ((E - 1) * es + (rows - 1) * ld + cols) * b;
  const uintptr_t o_end = o + ((E - 1) * out_es + (rows - 1) * out_ld + cols) * 2;
  return a < o_end && o < a_end;
}

bool orth_sizes(int E, int rows, int cols) {
  return E > 0 && rows > 0 && cols > 0 && E <= kMaxE && rows <= 16384 && cols <= 16384;
}

// ----------------------------------------------------- the experts' backward ---
struct BwdLayout {
  size_t grouped, gate_up, d_gate_up, d_h, h, total;
};
BwdLayout bwd_layout(int R, int H, int I, int E) {
  const size_t n = up((size_t)R * I * 2);
  BwdLayout L;
  size_t o = 0;
  L.grouped = o;    o += grouped_layout(E, H, 2 * I).total;
  L.gate_up = o;    o += 2 * n;
  L.d_gate_up = o;  o += 2 * n;
  L.d_h = o;        o += n;
  L.h = o;          o += n;
  L.total = o;
  return L;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grouped_workspace_bytes(int32_t E, int32_t K, int32_t N) {
  return check_grouped(E, K, N) == MOE_OK ? grouped_layout(E, K, N).total : 0;
}

moe_status moe_grouped_product(const void* x, int64_t x_ld, int32_t dtype, const int32_t* offsets,
                               const void* w, int64_t w_ld, int64_t w_es, int32_t transposed,
                               int32_t R, int32_t K, int32_t N, int32_t E, void* y, int64_t y_ld,
                               int32_t y_dtype, void* workspace, size_t ws_bytes, void* stream) {
  MOE_TRY(check_grouped(E, K, N));
  if (!is16(dtype) || !known(y_dtype)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_rows(R, E, N));
  MOE_TRY(check_matrix(x, R, K, x_ld, dtype));
  MOE_TRY(transposed ? check_stack(w, E, N, K, w_ld, w_es, dtype)
                     : check_stack(w, E, K, N, w_ld, w_es, dtype));
  MOE_TRY(check_matrix(y, R, N, y_ld, y_dtype));
  MOE_TRY(validate_ptr(offsets));
  MOE_TRY(check_workspace(workspace, ws_bytes, grouped_layout(E, K, N).total));
  MOE_TRY(validate_device());
  return do_product(x, x_ld, dtype, offsets, w, w_ld, w_es, transposed != 0, R, K, N, E, y, y_ld,
                    y_dtype, workspace, as_stream(stream));
}

moe_status moe_grouped_weight_grad(const void* x, int64_t x_ld, const void* dy, int64_t dy_ld,
                                   int32_t dtype, const int32_t* offsets, int32_t R, int32_t K,
                                   int32_t N, int32_t E, void* d_w, int64_t w_ld, int64_t w_es,
                                   int32_t w_dtype, int32_t accumulate, void* workspace,
                                   size_t ws_bytes, void* stream) {
  MOE_TRY(check_grouped(E, K, N));
  if (!is16(dtype) || !known(w_dtype) || (accumulate && w_dtype != MOE_DTYPE_F32))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_rows(R, E, N));
  MOE_TRY(check_matrix(x, R, K, x_ld, dtype));
  MOE_TRY(check_matrix(dy, R, N, dy_ld, dtype));
  MOE_TRY(check_stack(d_w, E, K, N, w_ld, w_es, w_dtype));
  MOE_TRY(validate_ptr(offsets));
  MOE_TRY(check_workspace(workspace, ws_bytes, grouped_layout(E, K, N).total));
  MOE_TRY(validate_device());
  return do_wgrad(x, x_ld, dy, dy_ld, dtype, offsets, R, K, N, E, d_w, w_ld, w_es, w_dtype,
                  accumulate != 0, workspace, as_stream(stream));
}

moe_status moe_swiglu(const void* gate_up, int64_t gate_up_ld, const float* row_w, int32_t dtype,
                      int32_t R, int32_t I, void* h, int64_t h_ld, void* stream) {
  if (!is16(dtype) || R < 0 || I <= 0) return MOE_ERR_INVALID_ARG;
  if (I % 8 != 0 || I > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  MOE_TRY(check_matrix(gate_up, R, 2LL * I, gate_up_ld, dtype));
  MOE_TRY(check_matrix(h, R, I, h_ld, dtype));
  if (row_w != nullptr) MOE_TRY(validate_ptr(row_w));
  MOE_TRY(validate_device());
  MOE_CUDA(launch_swiglu(gate_up, gate_up_ld, row_w, dtype, R, I, h, h_ld, as_stream(stream)));
  return MOE_OK;
}

moe_status moe_swiglu_bwd(const void* gate_up, int64_t gate_up_ld, const void* d_h, int64_t d_ld,
                          const float* row_w, int32_t dtype, int32_t R, int32_t I,
                          void* d_gate_up, int64_t d_gate_up_ld, void* h, int64_t h_ld,
                          float* d_row_w, void* stream) {
  if (!is16(dtype) || R < 0 || I <= 0) return MOE_ERR_INVALID_ARG;
  if (I % 8 != 0 || I > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  MOE_TRY(check_matrix(gate_up, R, 2LL * I, gate_up_ld, dtype));
  MOE_TRY(check_matrix(d_h, R, I, d_ld, dtype));
  MOE_TRY(check_matrix(d_gate_up, R, 2LL * I, d_gate_up_ld, dtype));
  if (h != nullptr) MOE_TRY(check_matrix(h, R, I, h_ld, dtype));
  if (row_w != nullptr) MOE_TRY(validate_ptr(row_w));
  if (d_row_w != nullptr) MOE_TRY(validate_ptr(d_row_w));
  MOE_TRY(validate_device());
  MOE_CUDA(launch_swiglu_bwd(gate_up, gate_up_ld, d_h, d_ld, row_w, dtype, R, I, d_gate_up,
                             d_gate_up_ld, h, h_ld, d_row_w, nullptr, 0, as_stream(stream)));
  return MOE_OK;
}

size_t moe_expert_ffn_bwd_workspace_bytes(int32_t R, int32_t H, int32_t I, int32_t E) {
  if (R < 0 || I > 16384 || check_grouped(E, H, I) != MOE_OK) return 0;
  return bwd_layout(R, H, I, E).total;
}

moe_status moe_expert_ffn_bwd(const void* x_perm, const int32_t* offsets, const void* w_gate_up,
                              const void* w_down, const void* gate_up, const float* row_w,
                              const void* d_y, int32_t dtype, int32_t R, int32_t H, int32_t I,
                              int32_t E, void* d_x_perm, int32_t d_x_dtype, void* d_w_gate_up,
                              void* d_w_down, int32_t d_w_dtype, int32_t accumulate,
                              float* d_row_w, void* workspace, size_t ws_bytes, void* stream) {
  MOE_TRY(check_grouped(E, H, I));
  if (I > 16384) return MOE_ERR_UNSUPPORTED;
  if (!is16(dtype) || !known(d_x_dtype) || !known(d_w_dtype) ||
      (accumulate && d_w_dtype != MOE_DTYPE_F32))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_rows(R, E, H > 2 * I ? H : 2 * I));
  MOE_TRY(check_matrix(x_perm, R, H, H, dtype));
  MOE_TRY(check_matrix(d_y, R, H, H, dtype));
  MOE_TRY(validate_ptr(offsets));
  MOE_TRY(validate_ptr(w_gate_up));
  MOE_TRY(validate_ptr(w_down));
  for (const void* p : {gate_up, static_cast<const void*>(row_w), static_cast<const void*>(d_x_perm),
                        static_cast<const void*>(d_w_gate_up), static_cast<const void*>(d_w_down),
                        static_cast<const void*>(d_row_w)})
    if (p != nullptr) MOE_TRY(validate_ptr(p));
  const BwdLayout L = bwd_layout(R, H, I, E);
  MOE_TRY(check_workspace(workspace, ws_bytes, L.total));
  MOE_TRY(validate_device());
  cudaStream_t s = as_stream(stream);
  void* ws = workspace;
  if (gate_up == nullptr) {
    MOE_TRY(do_product(x_perm, H, dtype, offsets, w_gate_up, 2 * I, 2LL * H * I, false, R, H, 2 * I,
                       E, at<void>(ws, L.gate_up), 2 * I, dtype, ws, s));
    gate_up = at<void>(ws, L.gate_up);
  }
  void *d_h = at<void>(ws, L.d_h), *dgu = at<void>(ws, L.d_gate_up), *h = at<void>(ws, L.h);
  MOE_TRY(do_product(d_y, H, dtype, offsets, w_down, H, (long long)H * I, true, R, H, I, E, d_h, I,
                     dtype, ws, s));
  MOE_CUDA(launch_swiglu_bwd(gate_up, 2 * I, d_h, I, row_w, dtype, R, I, dgu, 2 * I,
                             d_w_down ? h : nullptr, I, d_row_w, offsets, E, s));
  if (d_w_down != nullptr)
    MOE_TRY(do_wgrad(h, I, d_y, H, dtype, offsets, R, I, H, E, d_w_down, H, (long long)H * I,
                     d_w_dtype, accumulate != 0, ws, s));
  if (d_x_perm != nullptr)
    MOE_TRY(do_product(dgu, 2 * I, dtype, offsets, w_gate_up, 2 * I, 2LL * H * I, true, R, 2 * I, H,
                       E, d_x_perm, H, d_x_dtype, ws, s));
  if (d_w_gate_up != nullptr)
    MOE_TRY(do_wgrad(x_perm, H, dgu, 2 * I, dtype, offsets, R, H, 2 * I, E, d_w_gate_up, 2 * I,
                     2LL * H * I, d_w_dtype, accumulate != 0, ws, s));
  return MOE_OK;
}

size_t moe_orthogonalize_workspace_bytes(int32_t E, int32_t rows, int32_t cols) {
  return orth_sizes(E, rows, cols) ? orth_layout(E, rows, cols).total : 0;
}

moe_status moe_orthogonalize(const void* m, int32_t dtype, int64_t ld, int64_t es, int32_t E,
                             int32_t rows, int32_t cols, const float* coefficients, int32_t steps,
                             float eps, float scale, void* out, int32_t out_dtype, int64_t out_ld,
                             int64_t out_es, void* workspace, size_t ws_bytes, void* stream) {
  if (E <= 0 || rows <= 0 || cols <= 0 || steps <= 0 || coefficients == nullptr || !known(dtype) ||
      !is16(out_dtype))
    return MOE_ERR_INVALID_ARG;
  if (!orth_sizes(E, rows, cols) || steps > kMaxSteps) return MOE_ERR_UNSUPPORTED;
  const float a = coefficients[0], b = coefficients[1], c = coefficients[2];
  if (!isfinite(a) || !isfinite(b) || !isfinite(c) || !isfinite(scale) || !(eps >= 0.0f) ||
      !isfinite(eps))
    return MOE_ERR_INVALID_ARG;
  for (int j = 0; j < 2; ++j) {  // (any strides that keep elements apart)
    const long long l = j ? out_ld : ld, t = j ? out_es : es;
    if (l < cols || (E > 1 && t < rows * l)) return MOE_ERR_INVALID_ARG;
    if (l >= (1LL << 31) || t >= (1LL << 38)) return MOE_ERR_UNSUPPORTED;
  }
  MOE_TRY(validate_ptr(m));
  MOE_TRY(validate_ptr(out));
  const OrthLayout L = orth_layout(E, rows, cols);
  MOE_TRY(check_workspace(workspace, ws_bytes, L.total));
  MOE_TRY(validate_device());
  cudaStream_t s = as_stream(stream);
  if (orth_small(rows, cols) &&
      !orth_crosses(m, dtype, ld, es, out, out_ld, out_es, E, rows, cols)) {
    MOE_CUDA(launch_orth_small(m, dtype, ld, es, E, rows, cols, coefficients, steps, eps, scale, out,
                               out_dtype, out_ld, out_es, static_cast<int32_t*>(workspace),
                               wait_limit(), s));
    return MOE_OK;
  }
  // the shorter side's products: X X^T, or X^T X of a tall matrix, S x S
  const bool tall = rows > cols;
  const int S = tall ? cols : rows;
  const long long lx = (cols + 7) / 8 * 8, la = (S + 7) / 8 * 8;
  const long long xs = rows * lx, as = S * la;
  void *x = at<void>(workspace, L.x0), *x1 = at<void>(workspace, L.x1);
  void *lo = at<void>(workspace, L.lo0), *lo1 = at<void>(workspace, L.lo1);
  void *A = at<void>(workspace, L.a), *B = at<void>(workspace, L.b);
  float* f = at<float>(workspace, L.f);
  MOE_CUDA(launch_orth_start(m, dtype, ld, es, E, rows, cols, eps, at<float>(workspace, L.parts), x,
                             dtype == MOE_DTYPE_F32 ? lo : nullptr, f, s));
  TrainBatch q = {};
  q.E = E;
  q.pair = batch_pairs(E, rows, cols);
  q.status = static_cast<int32_t*>(workspace);
  q.limit = wait_limit();
  const int keep = keep_low(steps);
  for (int i = 0; i < steps; ++i) {
    const bool first = i == 0, last = i == steps - 1;
    const float held = first ? 1.0f : kHeld;  // x holds X times this (the first: X / f_e)
    // A = X X^T
    q.form = tall ? TrainBatch::GRAM_COLS : TrainBatch::GRAM_ROWS;
    q.a = q.b = x;
    q.a_ld = q.b_ld = lx;
    q.a_es = q.b_es = xs;
    q.M = q.N = S;
    q.K = tall ? rows : cols;
    q.padded = true;
    q.out = A;
    q.ld = la;
    q.es = as;
    q.out_type = MOE_DTYPE_F16;
    q.c = q.c_lo = nullptr;
    q.out_lo = nullptr;
    q.alpha = kHeld / (held * held);
    q.alpha_e = first ? f + E : nullptr;
    q.beta = 0.0f;
    q.beta_e = nullptr;
    MOE_CUDA(launch_batch(q, s));
    // B = b A + c A A
    q.form = TrainBatch::SQUARE;
    q.a = q.b = q.c = A;
    q.a_ld = q.b_ld = q.c_ld = la;
    q.a_es = q.b_es = q.c_es = as;
    q.K = S;
    q.out = B;
    q.alpha = c / kHeld;
    q.alpha_e = nullptr;
    q.beta = b;
    MOE_CUDA(launch_batch(q, s));
    // X = a X + B X (tall: X B)
    const float next = last ? scale : kHeld;
    q.form = tall ? TrainBatch::RIGHT : TrainBatch::LEFT;
    (tall ? q.b : q.a) = B;
    (tall ? q.a : q.b) = x;
    (tall ? q.a_ld : q.b_ld) = lx;
    (tall ? q.a_es : q.b_es) = xs;
    q.M = rows;
    q.N = cols;
    q.c = x;
    q.c_lo = i < keep && (i > 0 || dtype == MOE_DTYPE_F32) ? lo : nullptr;
    q.c_ld = lx;
    q.c_es = xs;
    q.alpha = next / (held * kHeld);
    q.beta = a * next / held;
    q.alpha_e = q.beta_e = first ? f : nullptr;
    q.padded = !last;
    q.out = last ? out : x1;
    q.out_lo = last || i + 1 >= keep ? nullptr : lo1;
    q.ld = last ? out_ld : lx;
    q.es = last ? out_es : xs;
    q.out_type = last ? out_dtype : MOE_DTYPE_F16;
    MOE_CUDA(launch_batch(q, s));
    void* t = x;
    x = x1;
    x1 = t;
    t = lo;
    lo = lo1;
    lo1 = t;
  }
  return MOE_OK;
}

}  // extern "C"

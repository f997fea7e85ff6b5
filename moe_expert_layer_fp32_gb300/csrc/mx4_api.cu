// C ABI of the selection and microscaled 4-bit calls (declared in include/moe.h):
// argument checks, workspace layouts and launch sequences.  As in moe_api.cu, no call
// allocates device memory or synchronises.
#include <math.h>

#include "common.cuh"
#include "kernels.cuh"
#include "mx4.cuh"

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

int dtype_bytes(int dtype) {
  switch (dtype) {
    case MOE_DTYPE_F32: return 4;
    case MOE_DTYPE_BF16:
    case MOE_DTYPE_F16: return 2;
  }
  return 0;
}

moe_status check_workspace(const void* ws, size_t have, size_t want) {
  if (ws == nullptr) return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) != 0) return MOE_ERR_MISALIGNED;
  return have < want ? MOE_ERR_WORKSPACE : MOE_OK;
}

// --------------------------------------------------------------- selection ---
moe_status check_select(const moe_select_opts* o, int T, int E, int k) {
  if (o == nullptr || T < 0 || E <= 0 || k <= 0 || k > E) return MOE_ERR_INVALID_ARG;
  if (E > kMaxE || k > kMaxK || (long long)T * k >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
  if (o->kind != MOE_ROUTER_SOFTMAX && o->kind != MOE_ROUTER_SIGMOID_BIAS_SELECT)
    return MOE_ERR_INVALID_ARG;
  if (o->n_group < 1 || o->topk_group < 1 || o->topk_group > o->n_group || E % o->n_group != 0)
    return MOE_ERR_INVALID_ARG;
  if (o->n_group > 32) return MOE_ERR_UNSUPPORTED;
  if (o->group_top != 1 && o->group_top != 2) return MOE_ERR_INVALID_ARG;
  if (k > o->topk_group * (E / o->n_group)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status check_logits(const void* p, int dtype, long long ld, int T, int E) {
  if (dtype_bytes(dtype) == 0 || ld < E) return MOE_ERR_INVALID_ARG;
  return T > 0 ? validate_ptr(p) : MOE_OK;
}

// ----------------------------------------------------------------- product ---
moe_status check_mx4(int E, int K, int N) {
  if (E <= 0 || K <= 0 || N <= 0) return MOE_ERR_INVALID_ARG;
  if (E > kMaxE || K % 128 != 0 || N % 128 != 0 || K > 16384 || N > 32768)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Row images of an operand of R rows over K among E experts: codes, then scales.
size_t rows_bytes(long long R, int K, int E, int tile_rows) {
  return up(mx4_max_tiles(R, E, tile_rows) * mx4_slot(K, tile_rows));
}
size_t images_bytes(long long R, int K, int E, int tile_rows) {
  return rows_bytes(R, K, E, tile_rows) + up(mx4_max_tiles(R, E, tile_rows) * mx4_sf_slots(K));
}

struct ProductLayout {
  size_t status, images, total;
};
ProductLayout product_layout(int R, int K, int E) {
  ProductLayout L;
  size_t o = 0;
  L.status = o;  o += up(kAlign);
  const size_t pair = images_bytes(R, K, E, kMx4PairRows);  // (the form goes by N too)
  const size_t single = images_bytes(R, K, E, kMx4SingleRows);
  L.images = o;  o += pair > single ? pair : single;
  L.total = o;
  return L;
}

// The grouped product of quantised rows (sources as launch_mx4_rows).
moe_status do_product(const void* x, int x_dtype, int src, const int32_t* row_of, int k, int T,
                      const int32_t* offsets, const void* packed, int E, int R, int K, int N,
                      void* y, int y_dtype, void* images, int32_t* status, cudaStream_t s) {
  const long long lim = wait_limit();
  const int tile_rows = mx4_tile_rows(E, R, N);
  void* sf = at<void>(images, rows_bytes(R, K, E, tile_rows));
  MOE_CUDA(launch_mx4_rows(x, x_dtype, src, row_of, k, T, offsets, E, R, K, tile_rows, images, sf,
                           status, s));
  MOE_CUDA(launch_mx4_gemm(packed, images, sf, offsets, E, R, K, N, y, y_dtype, status, lim, s));
  return MOE_OK;
}

struct LayerLayout {
  size_t status, logits, idx, w, counts, offsets, blk_counts, blk_base, row_of_slot, slot_of_row,
      images, gate_up, y, total;
};
LayerLayout layer_layout(const moe_dims& d) {
  const size_t T = (size_t)d.T, R = T * d.k, E = (size_t)d.E;
  const size_t nb = (T + kPermBlock - 1) / kPermBlock;
  LayerLayout L;
  size_t o = 0;
  L.status = o;       o += up(kAlign);
  L.logits = o;       o += up(T * E * 4);
  L.idx = o;          o += up(R * 4);
  L.w = o;            o += up(R * 4);
  L.counts = o;       o += up(E * 4);
  L.offsets = o;      o += up((E + 1) * 4);
  L.blk_counts = o;   o += up(nb * E * 4);
  L.blk_base = o;     o += up(nb * E * 4);
  L.row_of_slot = o;  o += up(R * 4);
  L.slot_of_row = o;  o += up(R * 4);
  const size_t up_img = product_layout((int)R, d.H, d.E).total;
  const size_t down_img = product_layout((int)R, d.I, d.E).total;
  L.images = o;       o += up_img > down_img ? up_img : down_img;
  L.gate_up = o;      o += up(R * 2 * (size_t)d.I * 2);
  L.y = o;            o += up(R * (size_t)d.H * 4);
  L.total = o;
  return L;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_router_logits(const void* x, const float* w_router, const float* bias, moe_dims d,
                             float* logits, void* stream) {
  MOE_TRY(validate_dims(d));
  if (d.T == 0) return MOE_OK;
  MOE_TRY(validate_ptr(x));
  MOE_TRY(validate_ptr(w_router));
  if (bias != nullptr) MOE_TRY(validate_ptr(bias));
  MOE_TRY(validate_ptr(logits));
  MOE_TRY(validate_device());
  MOE_CUDA(launch_router_logits(x, w_router, bias, d.T, d.H, d.E, logits, nullptr,
                                as_stream(stream)));
  return MOE_OK;
}

size_t moe_select_workspace_bytes(int32_t T, int32_t E) {
  if (T < 0 || E <= 0 || E > kMaxE) return 0;
  return up(select_partial_bytes(T, E)) + kAlign;
}

moe_status moe_route_select(const void* logits, int32_t dtype, int64_t ld, const float* bias,
                            const moe_select_opts* opts, int32_t T, int32_t E, int32_t k,
                            int32_t* topk_idx, float* topk_w, float* prob_sum, void* workspace,
                            size_t ws_bytes, void* stream) {
  MOE_TRY(check_select(opts, T, E, k));
  MOE_TRY(check_logits(logits, dtype, ld, T, E));
  if (bias != nullptr) MOE_TRY(validate_ptr(bias));
  if (T > 0) {
    MOE_TRY(validate_ptr(topk_idx));
    MOE_TRY(validate_ptr(topk_w));
  }
  if (prob_sum != nullptr) {
    MOE_TRY(validate_ptr(prob_sum));
    MOE_TRY(check_workspace(workspace, ws_bytes, moe_select_workspace_bytes(T, E)));
  }
  MOE_TRY(validate_device());
  cudaStream_t s = as_stream(stream);
  if (T == 0) {
    if (prob_sum != nullptr) MOE_CUDA(cudaMemsetAsync(prob_sum, 0, (size_t)E * 4, s));
    return MOE_OK;
  }
  MOE_CUDA(launch_select(logits, dtype, ld, bias, *opts, T, E, k, topk_idx, topk_w, prob_sum,
                         static_cast<float*>(workspace), s));
  return MOE_OK;
}

moe_status moe_route_select_bwd(const void* logits, int32_t dtype, int64_t ld, const float* bias,
                                const moe_select_opts* opts, int32_t T, int32_t E, int32_t k,
                                const int32_t* topk_idx, const float* d_topk_w,
                                const float* d_prob_sum, void* d_logits, int64_t ld_d,
                                float* d_bias, void* workspace, size_t ws_bytes, void* stream) {
  MOE_TRY(check_select(opts, T, E, k));
  MOE_TRY(check_logits(logits, dtype, ld, T, E));
  MOE_TRY(check_logits(d_logits, dtype, ld_d, T, E));
  if (bias != nullptr) MOE_TRY(validate_ptr(bias));
  if (d_prob_sum != nullptr) MOE_TRY(validate_ptr(d_prob_sum));
  if (T > 0) {
    MOE_TRY(validate_ptr(topk_idx));
    MOE_TRY(validate_ptr(d_topk_w));
  }
  if (d_bias != nullptr) {
    if (opts->kind != MOE_ROUTER_SOFTMAX) return MOE_ERR_INVALID_ARG;
    MOE_TRY(validate_ptr(d_bias));
    MOE_TRY(check_workspace(workspace, ws_bytes, moe_select_workspace_bytes(T, E)));
  }
  MOE_TRY(validate_device());
  cudaStream_t s = as_stream(stream);
  if (T == 0) {
    if (d_bias != nullptr) MOE_CUDA(cudaMemsetAsync(d_bias, 0, (size_t)E * 4, s));
    return MOE_OK;
  }
  MOE_CUDA(launch_select_bwd(logits, dtype, ld, bias, *opts, T, E, k, topk_idx, d_topk_w,
                             d_prob_sum, d_logits, ld_d, d_bias, static_cast<float*>(workspace),
                             s));
  return MOE_OK;
}

moe_status moe_mx4_quantize(const void* x, int32_t dtype, int64_t ld, int64_t R, int32_t K,
                            void* codes, void* scales, void* values, void* stream) {
  const int es = dtype_bytes(dtype);
  if (es == 0 || R < 0 || K <= 0 || ld < K) return MOE_ERR_INVALID_ARG;
  if (K % 32 != 0 || K > (1 << 24) || R >= (1LL << 40) / K) return MOE_ERR_UNSUPPORTED;
  if ((ld * es) % 16 != 0) return MOE_ERR_MISALIGNED;
  if (R == 0) return MOE_OK;
  MOE_TRY(validate_ptr(x));
  if (codes != nullptr) MOE_TRY(validate_ptr(codes));
  if (scales != nullptr) MOE_TRY(validate_ptr(scales));
  if (values != nullptr) MOE_TRY(validate_ptr(values));
  MOE_TRY(validate_device());
  MOE_CUDA(launch_mx4_quantize(x, dtype, ld, R, K, codes, scales, values, as_stream(stream)));
  return MOE_OK;
}

size_t moe_mx4_packed_bytes(int32_t E, int32_t K, int32_t N) {
  if (check_mx4(E, K, N) != MOE_OK) return 0;
  return (size_t)E * (N / kMx4WTile) * mx4_kblocks(K) * kMx4WBytes;
}

moe_status moe_mx4_pack(const void* codes, const void* scales, int32_t E, int32_t K, int32_t N,
                        void* packed, size_t packed_bytes, void* stream) {
  MOE_TRY(check_mx4(E, K, N));
  MOE_TRY(validate_ptr(codes));
  MOE_TRY(validate_ptr(scales));
  MOE_TRY(validate_ptr(packed));
  if (packed_bytes < moe_mx4_packed_bytes(E, K, N)) return MOE_ERR_WORKSPACE;
  MOE_TRY(validate_device());
  MOE_CUDA(launch_mx4_pack(codes, scales, E, K, N, packed, as_stream(stream)));
  return MOE_OK;
}

moe_status moe_mx4_prepack(const void* w, int32_t E, int32_t K, int32_t N, int32_t col0,
                           int32_t N_total, void* packed, size_t packed_bytes, void* stream) {
  MOE_TRY(check_mx4(E, K, N));
  MOE_TRY(check_mx4(E, K, N_total));
  if (col0 < 0 || col0 % 128 != 0 || (long long)col0 + N > N_total) return MOE_ERR_INVALID_ARG;
  MOE_TRY(validate_ptr(w));
  MOE_TRY(validate_ptr(packed));
  if (packed_bytes < moe_mx4_packed_bytes(E, K, N_total)) return MOE_ERR_WORKSPACE;
  MOE_TRY(validate_device());
  MOE_CUDA(launch_mx4_prepack(w, E, K, N, col0, N_total, packed, as_stream(stream)));
  return MOE_OK;
}

size_t moe_mx4_product_workspace_bytes(int32_t R, int32_t K, int32_t E) {
  if (R < 0 || check_mx4(E, K, 128) != MOE_OK) return 0;
  return product_layout(R, K, E).total;
}

moe_status moe_mx4_expert_product(const void* x, int32_t x_dtype, const int32_t* offsets,
                                  const void* packed, int32_t R, int32_t K, int32_t N, int32_t E,
                                  void* y, int32_t y_dtype, void* workspace, size_t ws_bytes,
                                  void* stream) {
  MOE_TRY(check_mx4(E, K, N));
  if (R < 0 || dtype_bytes(x_dtype) == 0) return MOE_ERR_INVALID_ARG;
  if (y_dtype != MOE_DTYPE_F32 && y_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  const ProductLayout L = product_layout(R, K, E);
  MOE_TRY(check_workspace(workspace, ws_bytes, L.total));
  if (R == 0) return MOE_OK;
  MOE_TRY(validate_ptr(x));
  MOE_TRY(validate_ptr(offsets));
  MOE_TRY(validate_ptr(packed));
  MOE_TRY(validate_ptr(y));
  MOE_TRY(validate_device());
  return do_product(x, x_dtype, 0, nullptr, 1, R, offsets, packed, E, R, K, N, y, y_dtype,
                    at<void>(workspace, L.images), at<int32_t>(workspace, L.status),
                    as_stream(stream));
}

size_t moe_mx4_layer_workspace_bytes(moe_dims d) {
  if (validate_dims(d) != MOE_OK) return 0;
  return layer_layout(d).total;
}

moe_status moe_mx4_layer_fwd(const void* x, const float* w_router, const float* bias,
                             const moe_select_opts* opts, float route_scale,
                             const void* packed_gate_up, const void* packed_down, moe_dims d,
                             void* out, int32_t* topk_idx_out, float* topk_w_out,
                             int32_t* counts_out, void* workspace, size_t ws_bytes, void* stream) {
  MOE_TRY(validate_dims(d));
  MOE_TRY(check_select(opts, d.T, d.E, d.k));
  if (!(route_scale > 0.0f) || !isfinite(route_scale)) return MOE_ERR_INVALID_ARG;
  const LayerLayout L = layer_layout(d);
  MOE_TRY(check_workspace(workspace, ws_bytes, L.total));
  MOE_TRY(validate_ptr(w_router));
  if (bias != nullptr) MOE_TRY(validate_ptr(bias));
  MOE_TRY(validate_ptr(packed_gate_up));
  MOE_TRY(validate_ptr(packed_down));
  if (topk_idx_out != nullptr) MOE_TRY(validate_ptr(topk_idx_out));
  if (topk_w_out != nullptr) MOE_TRY(validate_ptr(topk_w_out));
  if (counts_out != nullptr) MOE_TRY(validate_ptr(counts_out));
  if (d.T > 0) {
    MOE_TRY(validate_ptr(x));
    MOE_TRY(validate_ptr(out));
  }
  MOE_TRY(validate_device());
  cudaStream_t s = as_stream(stream);
  const int T = d.T, R = d.T * d.k, nb = (T + kPermBlock - 1) / kPermBlock;
  int32_t* status = at<int32_t>(workspace, L.status);
  float* logits = at<float>(workspace, L.logits);
  int32_t* idx = topk_idx_out ? topk_idx_out : at<int32_t>(workspace, L.idx);
  float* w = topk_w_out ? topk_w_out : at<float>(workspace, L.w);
  int32_t* counts = counts_out ? counts_out : at<int32_t>(workspace, L.counts);
  int32_t* offsets = at<int32_t>(workspace, L.offsets);
  int32_t* blk_counts = at<int32_t>(workspace, L.blk_counts);
  int32_t* blk_base = at<int32_t>(workspace, L.blk_base);
  int32_t* ros = at<int32_t>(workspace, L.row_of_slot);
  int32_t* sor = at<int32_t>(workspace, L.slot_of_row);
  void* images = at<void>(workspace, L.images);
  void* gu = at<void>(workspace, L.gate_up);
  float* y = at<float>(workspace, L.y);
  if (T > 0) {
    MOE_CUDA(launch_router_logits(x, w_router, nullptr, T, d.H, d.E, logits, status, s));
    MOE_CUDA(launch_select(logits, MOE_DTYPE_F32, d.E, bias, *opts, T, d.E, d.k, idx, w, nullptr,
                           nullptr, s));
  }
  MOE_CUDA(launch_block_counts(idx, T, d.k, d.E, blk_counts, status, s));
  MOE_CUDA(launch_scan(blk_counts, nb, d.E, R, counts, offsets, false, blk_base, status, s));
  if (T == 0) return MOE_OK;
  MOE_CUDA(launch_rank(idx, T, d.k, d.E, blk_base, ros, sor, status, s));
  MOE_TRY(do_product(x, MOE_DTYPE_BF16, 1, sor, d.k, T, offsets, packed_gate_up, d.E, R, d.H,
                     2 * d.I, gu, MOE_DTYPE_BF16, images, status, s));
  MOE_TRY(do_product(gu, MOE_DTYPE_BF16, 2, nullptr, 1, R, offsets, packed_down, d.E, R, d.I, d.H,
                     y, MOE_DTYPE_F32, images, status, s));
  MOE_CUDA(launch_combine(y, w, ros, T, d.H, d.k, route_scale, out, s));
  return MOE_OK;
}

}  // extern "C"

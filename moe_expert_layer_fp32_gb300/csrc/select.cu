// Selection from router logits, and its gradient.
//
// For a row of E logits l (one token), m_e = "masked": l_e, b_e or (for softmax) l_e + b_e
// is -inf or NaN.
//   softmax   key_e = l_e + b_e,            score_e = exp(key_e) / sum_E exp(key)
//   sigmoid   s_e = 1 / (1 + exp(-l_e)),    key_e = s_e + b_e,   score_e = s_e
// (the keys' arithmetic is the router kernels': one FP32 add, and for the sigmoid the
// Cody & Waite exponential whose every step is one IEEE operation, so that a choice does
// not depend on which kernel made it).  Groups are E / n_group consecutive experts; a
// group's score is the sum of its group_top (1 or 2) largest keys that are not masked (-inf
// if all are); the topk_group groups with the largest scores stay, then the k experts in them
// with the largest keys, both with ties to the lower index.  w_j = score_j, or score_j / sum of
// the chosen scores.  prob_sum[e] = sum over tokens of score_e / sum_E score (what a balance loss
// needs), like d_bias an FP32 sum over each warp's tokens, the block's warps and the blocks, with
// T / 4864 + 60 terms in a chain (608 blocks).
//
// Gradient, with c the chosen experts, S = sum of their scores, q = score / sum_E score,
// g = d_prob_sum:
//   d score_j += renorm ? (dw_j - sum_i dw_i w_i) / S : dw_j        (j chosen)
//   softmax: d l_e = q_e (D_e - sum_i D_i q_i),  D_e = g_e + [e chosen] dw'
//   sigmoid: d l_e = s_e (1 - s_e) (d score_e + (g_e - sum_i g_i q_i) / sum_E s), the factor
//            from exp(-|l_e|) without a difference
// For the renormalised softmax the factor 1/S cancels against q: d l_j = w_j (dw_j - sum
// dw_i w_i) for the chosen, formed from exponentials relative to the largest chosen key,
// so that chosen experts far below the row's largest logit keep their precision.
//
// One warp per token, EP/32 consecutive experts per lane; 32 warps an SM at 64 registers.
// What each has to move is one pass over the logits (T = 32768, E = 256 in FP32: 34 MB, 5 us).
// What bounds the selection is its instructions, some 900 a token and warp, issued in three of
// four cycles; comparisons, selections and integers issue at half the rate of the arithmetic.
// Measured on GB300 at that size, sigmoid scores, 8 of 256 experts from 4 of 8 groups, in a
// CUDA graph: 30.0 us, with prob_sum 34.5; of it the sigmoids take 5, the groups 4, the choice
// of eight instead of one 3.5.  The steps that brought it there from 81 us: candidates above a
// bound of the k-th key ranked side by side instead of k argmax rounds over all keys (45), two
// sigmoids an instruction and group maxima in registers (40), the next token's loads in flight
// (38.5), candidates by a lane mask (37.4), no limits and masks for plain rows (35.6), the bias
// by 16-byte loads (34.5).  Three heads a lane and k rounds of warp maxima instead of bound and
// ranks took 45.9.
// The gradient with every expert's share: 16.2-16.7 us in a graph for 67 MB (10 us), latency and
// issue; of the chosen alone (no d_prob_sum, renormalised) 13.5.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.cuh"
#include "pdl.cuh"
#include "select_math.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr float kLowest = -3.402823466e38f;  // FP32's
constexpr int kSelBlocksPerSm = 4;  // 32 warps of at most 64 registers a thread

struct SelectArgs {
  const void* logits;
  long long ld;
  const float* bias;
  int T, E, k;
  int n_group, topk_group, group_top, renorm;
  int per;         // experts of a group
  int per_magic;   // (e * per_magic) >> 16 = e / per for e < 256
  int lane_shift;  // log2 of the lanes that share a group in the group sums
};

// NV logits of one lane: experts e0 .. e0 + NV - 1 of the row, -inf past E.
template <typename Tin, int NV>
__device__ __forceinline__ void load_row(const Tin* row, int e0, int E, bool vec, float (&l)[NV]) {
  if (vec && e0 + NV <= E) {
    load_floats<Tin, NV>(row + e0, l);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = (e0 + i < E) ? to_float(row[e0 + i]) : -INFINITY;
  }
}

// key and score of the lane's experts.  KIND 0: score is left to the caller (it needs
// the row's maximum); masked experts and those past E (of the lane's NV, `inside` are within)
// have key -inf and score 0.  b is the bias as lane_bias made it, so a sum with it is never -0
// (which would order below +0); open: none of the lane's is -inf.
template <int KIND, int NV>
__device__ __forceinline__ void keys_of(const float (&l)[NV], const float (&b)[NV], bool open,
                                        int inside, float (&key)[NV], float (&sc)[NV]) {
  if constexpr (KIND == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      key[i] = fmaxf(__fadd_rn(l[i], b[i]), -INFINITY);  // (a maximum drops NaN)
      sc[i] = 0.0f;
    }
  } else {
    // A row whose logits are all numbers within +-80 (nearly every one) needs no limits and
    // no masks: comparisons and selections issue at half the rate of the arithmetic.  (0 l is
    // not 0 for an infinity or a NaN.)
    float zero = 0.0f, big = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      zero = fmaf(l[i], 0.0f, zero);
      big = fmaxf(big, fabsf(l[i]));
    }
    const bool plain = inside == 0 || (inside == NV && open && zero == 0.0f && big <= 80.0f);
    if (__all_sync(kFull, plain)) {
#pragma unroll
      for (int i = 0; i < NV; i += 2) {
        const float2 s = sigmoid_steps2<false>(l[i], l[NV > 1 ? i + 1 : i]);
        sc[i] = s.x;
        key[i] = __fadd_rn(s.x, b[i]);
        if (NV > 1) {
          sc[NV > 1 ? i + 1 : i] = s.y;
          key[NV > 1 ? i + 1 : i] = __fadd_rn(s.y, b[NV > 1 ? i + 1 : i]);
        }
      }
      if (inside == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          key[i] = -INFINITY;
          sc[i] = 0.0f;
        }
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < NV; i += 2) {
      const float2 s = sigmoid_steps2<true>(l[i], l[NV > 1 ? i + 1 : i]);
      sc[i] = s.x;
      if (NV > 1) sc[NV > 1 ? i + 1 : i] = s.y;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = l[i] > -INFINITY && b[i] > -INFINITY;
      key[i] = in ? __fadd_rn(sc[i], b[i]) : -INFINITY;
      sc[i] = in ? sc[i] : 0.0f;
    }
  }
}

// The lane's values of an FP32 vector over the experts (16-byte aligned), 0 where there is none.
template <int NV>
__device__ __forceinline__ void lane_vector(const float* p, int e0, int E, float (&v)[NV]) {
  if (p != nullptr && e0 + NV <= E) {
    load_floats<float, NV>(p + e0, v);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = (p != nullptr && e0 + i < E) ? __ldg(p + e0 + i) : 0.0f;
  }
}

// Biases as the keys take them: NaN masks its expert as -inf does, -0 becomes +0.
template <int NV>
__device__ __forceinline__ void lane_bias(const float* bias, int e0, int E, float (&b)[NV]) {
  lane_vector<NV>(bias, e0, E, b);
#pragma unroll
  for (int i = 0; i < NV; ++i) b[i] = (b[i] == b[i]) ? __fadd_rn(b[i], 0.0f) : -INFINITY;
}

// exp(key - m), 1 where key is the maximum (also +inf), 0 where masked
__device__ __forceinline__ float exp_rel(float key, float m) {
  if (key == -INFINITY) return 0.0f;
  return key == m ? 1.0f : expf(key - m);
}

// exp_rel on the special-function unit: within 2 FP32 steps plus |key - m| / 2 (the product
// with log2 e is rounded), for sums of many terms
__device__ __forceinline__ float exp_rel_fast(float key, float m) {
  return key == m ? (m > -INFINITY ? 1.0f : 0.0f) : __expf(key - m);
}

// The gradient's sigmoid s and its slope s (1 - s), both 0 where masked.  With t = exp(-|l|) and
// r = 1 / (1 + t), s is r or t r by the sign of l and the slope t r r for both: no difference is
// taken (1 - s has no digits left where s is 1 to the last bit, from l = 17 on) and t does not
// overflow.
__device__ __forceinline__ float2 sigmoid_and_slope(float l) {
  l = fmaxf(l, -INFINITY);  // (a maximum drops NaN)
  const float t = expf(-fabsf(l)), r = __frcp_rn(__fadd_rn(1.0f, t)), u = __fmul_rn(t, r);
  return make_float2(l < 0.0f ? u : r, __fmul_rn(u, r));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
  return key_float(__reduce_max_sync(kFull, float_key(v)));
}

// the lane's NV values to a shared row of EP
template <int EP>
__device__ __forceinline__ void store_row(float* row, int e0, const float (&v)[EP / 32]) {
  store_floats<float, EP / 32>(row + e0, v);
}

// The block's column sums: every warp's columns through shared memory, in warp order.
template <int EP>
__device__ __forceinline__ void write_partial(float (*s_row)[EP], int warp, int e0,
                                              const float (&col)[EP / 32], int E,
                                              float* __restrict__ partial) {
  store_row<EP>(s_row[warp], e0, col);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSelThreads) {
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < kSelWarps; ++q) v += s_row[q][e];
    partial[(size_t)blockIdx.x * E + e] = v;
  }
}

// ------------------------------------------------------------------ forward ---
template <typename Tin, int EP, int KIND, bool PROB>
__global__ void __launch_bounds__(kSelThreads, kSelBlocksPerSm) select_kernel(SelectArgs a,
                                                             int32_t* __restrict__ topk_idx,
                                                             float* __restrict__ topk_w,
                                                             float* __restrict__ partial) {
  constexpr int NV = EP / 32;
  if constexpr (PROB) pdl_launch_dependents();  // the column sums, which wait for this kernel
  __shared__ __align__(16) float s_row[kSelWarps][EP];  // keys
  __shared__ __align__(16) float s_score[KIND == 1 ? kSelWarps : 1][KIND == 1 ? EP : 4];
  __shared__ __align__(16) uint32_t s_key[kSelWarps][32];  // candidates in expert order
  __shared__ int s_expert[kSelWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e0 = lane * NV;
  const int E = a.E, k = a.k;
  const Tin* logits = static_cast<const Tin*>(a.logits);
  const bool vec = rows_aligned<Tin, NV>(logits, a.ld);
  float b[NV];
  lane_bias<NV>(a.bias, e0, E, b);
  // all experts of a lane are in one group (their count past e0 is then 0 or NV), or not
  const bool whole = a.n_group == 1 || a.per % NV == 0;
  const int inside = min(max(E - e0, 0), NV);
  // a group is the experts of 2^lane_shift lanes
  const bool by_lane = a.per == NV << a.lane_shift;
  float col[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) col[i] = 0.0f;
  float bound = INFINITY;  // of the token before
  const long long t0 = (long long)blockIdx.x * kSelWarps + warp;
  const long long stride = (long long)gridDim.x * kSelWarps;
  // the next token's logits are in flight while this one's experts are chosen
  float l[NV];
  if (t0 < a.T) load_row<Tin, NV>(logits + t0 * a.ld, e0, E, vec, l);
  bool open = true;  // the bias masks none of the lane's experts
#pragma unroll
  for (int i = 0; i < NV; ++i) open = open && b[i] > -INFINITY;

  for (long long t = t0; t < a.T; t += stride) {
    float key[NV], sc[NV];
    keys_of<KIND, NV>(l, b, open, inside, key, sc);
    if (t + stride < a.T) load_row<Tin, NV>(logits + (t + stride) * a.ld, e0, E, vec, l);
    // the row's softmax: its maximum and the sum relative to it (sigmoid: the sum of scores)
    float mx = -INFINITY, z = 0.0f;
    if (PROB || (KIND == 0 && !a.renorm)) {
      if constexpr (KIND == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) mx = fmaxf(mx, key[i]);
        mx = warp_max(mx);
      }
      // (with renorm they only make prob_sum, a sum of many terms: the special-function unit)
      const bool fast = a.renorm && fabsf(mx) < INFINITY;
      float p[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if constexpr (KIND == 0) p[i] = fast ? __expf(key[i] - mx) : exp_rel(key[i], mx);
        else p[i] = sc[i];
        z += p[i];
      }
      z = warp_sum(z);
      if constexpr (PROB) {
        const float r = z > 0.0f ? __frcp_rn(z) : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) col[i] += p[i] * r;
      }
    }
    // groups that stay: L lanes per group, each over every L-th of its keys
    unsigned keep = kFull;
    if (a.topk_group < a.n_group) {
      const int g = lane >> a.lane_shift, sub = lane & ((1 << a.lane_shift) - 1);
      float g1 = -INFINITY, g2 = -INFINITY;
      if (by_lane) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          g2 = fmaxf(g2, fminf(g1, key[i]));
          g1 = fmaxf(g1, key[i]);
        }
      } else {
        store_row<EP>(s_row[warp], e0, key);
        __syncwarp();
        if (g < a.n_group) {
          for (int i = sub; i < a.per; i += 1 << a.lane_shift) {
            const float v = s_row[warp][g * a.per + i];
            g2 = fmaxf(g2, fminf(g1, v));
            g1 = fmaxf(g1, v);
          }
        }
      }
      for (int o = 1; o < (1 << a.lane_shift); o <<= 1) {
        const float o1 = __shfl_xor_sync(kFull, g1, o), o2 = __shfl_xor_sync(kFull, g2, o);
        g2 = fmaxf(fmaxf(g2, o2), fminf(g1, o1));
        g1 = fmaxf(g1, o1);
      }
      // (two keys of FP32's lowest values add up to that lowest value, not to a masked group's -inf)
      const float gs = (a.group_top == 2 && g2 > -INFINITY) ? fmaxf(__fadd_rn(g1, g2), kLowest) : g1;
      // the largest score's first lane (so its lowest group) topk_group times
      uint32_t gk = (g < a.n_group) ? float_key(gs) : 0u;
      keep = 0u;
      for (int j = 0; j < a.topk_group; ++j) {
        const uint32_t m = __reduce_max_sync(kFull, gk);
        const uint32_t who = __ballot_sync(kFull, gk == m);
        keep |= who & (0u - who);  // bit g << lane_shift: group g stays
        if ((keep >> (lane & ~((1 << a.lane_shift) - 1))) & 1u) gk = 0u;
      }
    }
    // experts of this lane that may be chosen: all of a lane in one group, or one by one
    // (others get -inf here; the rare case where masked experts must be chosen sorts them out)
    bool lane_in = true;
    if (whole) {
      const int g = (e0 * a.per_magic) >> 16;  // e0 / per
      lane_in = inside > 0 && ((keep >> (g << a.lane_shift)) & 1u);
    }
    auto may = [&](int i) {
      if (whole) return lane_in && i < inside;
      const int g = ((e0 + i) * a.per_magic) >> 16;
      return i < inside && ((keep >> (g << a.lane_shift)) & 1u) != 0;
    };
    if (!whole) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (!may(i)) key[i] = -INFINITY;
    }
    // A lower bound of the k-th largest key: the k-th largest of the lanes' maxima (at
    // least k keys are not below it).  Few keys reach it, mostly one a lane.  The bound of
    // the token before is tried first: any bound that k to 32 keys reach will do.
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) top = fmaxf(top, key[i]);
    if (!lane_in) top = -INFINITY;
    int mine, before, n;
    unsigned mask;  // this lane's candidates
    auto count = [&]() {
      mask = 0u;
#pragma unroll
      for (int i = 0; i < NV; ++i) mask |= (key[i] >= bound ? 1u : 0u) << i;
      if (top < bound) mask = 0u;  // (a lane outside the groups that stay)
      mine = __popc(mask);
      before = mine;  // inclusive scan: candidates in expert order
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, before, o);
        if (lane >= o) before += v;
      }
      n = __shfl_sync(kFull, before, 31);
      before -= mine;
    };
    count();
    if (n < k || n > 32) {
      uint32_t tu = float_key(top), bu;
      for (int left = k;;) {
        bu = __reduce_max_sync(kFull, tu);
        const bool hit = tu == bu;
        left -= __popc(__ballot_sync(kFull, hit));
        if (left <= 0 || bu <= float_key(-INFINITY)) break;
        tu = hit ? 0u : tu;
      }
      bound = fmaxf(key_float(max(bu, 1u)), kLowest);  // (not the masked keys)
      count();
    }

    // lane j < k: slot j's expert, key and score
    int ce = 0;
    float ck = -INFINITY, cs = 0.0f;
    if (n >= k && n <= 32) {
      // one candidate a lane, ranked against the others
      store_row<EP>(s_row[warp], e0, key);
      if constexpr (KIND == 1) store_row<EP>(s_score[warp], e0, sc);
      for (; mask != 0u; mask &= mask - 1u) s_expert[warp][before++] = e0 + __ffs(mask) - 1;
      __syncwarp();
      const int mine_e = lane < n ? s_expert[warp][lane] : 0;
      const uint32_t cu = lane < n ? float_key(s_row[warp][mine_e]) : 0u;
      s_key[warp][lane] = cu;
      __syncwarp();
      int slot = lane < n ? 0 : 32;  // this lane's candidate's (k or more: not chosen)
      for (int j = 0; j < n; j += 4) {
        const uint4 o = *reinterpret_cast<const uint4*>(&s_key[warp][j]);
        slot += (o.x > cu || (o.x == cu && j + 0 < lane)) ? 1 : 0;
        slot += (o.y > cu || (o.y == cu && j + 1 < lane)) ? 1 : 0;
        slot += (o.z > cu || (o.z == cu && j + 2 < lane)) ? 1 : 0;
        slot += (o.w > cu || (o.w == cu && j + 3 < lane)) ? 1 : 0;
      }
      // slot j to lane j, so that sums over the chosen are in slot order
      if (slot < k) s_expert[warp][slot] = mine_e;
      __syncwarp();
      if (lane < k) {
        ce = s_expert[warp][lane];
        ck = s_row[warp][ce];
        if constexpr (KIND == 1) cs = s_score[warp][ce];
      }
      __syncwarp();
    } else {
      // many equal keys at the bound, or fewer than k that are not masked: k rounds of a
      // warp-wide maximum; 0 = cannot be chosen, masked below every number
      uint32_t u[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) u[i] = may(i) ? float_key(key[i]) : 0u;
      for (int j = 0; j < k; ++j) {
        uint32_t bk = 0u;
        int bi = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (u[i] > bk) {
            bk = u[i];
            bi = i;
          }
        const uint32_t m = __reduce_max_sync(kFull, bk);
        const int owner = __ffs(__ballot_sync(kFull, bk == m)) - 1;  // lanes hold ascending experts
        const int be = __shfl_sync(kFull, e0 + bi, owner);
        float sv = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (i == bi) {
            sv = sc[i];
            if (lane == owner) u[i] = 0u;
          }
        sv = __shfl_sync(kFull, sv, owner);
        if (lane == j) {
          ck = key_float(m);
          cs = sv;
          ce = be;
        }
      }
    }
    const bool chosen = lane < k;
    float w;
    if constexpr (KIND == 0) {
      // relative to the best chosen key, or the row's plain probability
      if (a.renorm) {
        const float best = warp_max(chosen ? ck : -INFINITY);
        w = chosen ? exp_rel(ck, best) : 0.0f;
        z = warp_sum(w);
      } else {
        w = chosen ? exp_rel(ck, mx) : 0.0f;
      }
      w = z > 0.0f ? __fdiv_rn(w, z) : 0.0f;
    } else {
      w = chosen ? cs : 0.0f;
      if (a.renorm) {
        const float S = warp_sum(w);
        w = S > 0.0f ? __fdiv_rn(w, S) : 0.0f;
      }
    }
    if (chosen) {
      topk_idx[t * k + lane] = ce;
      topk_w[t * k + lane] = w;
    }
  }
  if constexpr (PROB) write_partial<EP>(s_row, warp, e0, col, E, partial);
}

// ----------------------------------------------------------------- gradient ---
// add[i] = the sum of v over the lanes j < k whose expert e is this lane's e0 + i (e < 0:
// none), through a shared row; repeated experts (never from the forward pass) add up in
// slot order.
template <int EP>
__device__ __forceinline__ void spread(float* row, int e0, int lane, int e, float v, int k,
                                       float (&add)[EP / 32]) {
  constexpr int NV = EP / 32;
#pragma unroll
  for (int i = 0; i < NV; ++i) add[i] = 0.0f;
  __syncwarp();
  if (e >= 0) row[e] = __int_as_float(lane);  // who has this expert
  __syncwarp();
  const bool again = e >= 0 && __float_as_int(row[e]) != lane;
  if (__any_sync(kFull, again)) {
    for (int j = 0; j < k; ++j) {
      const int ej = __shfl_sync(kFull, e, j);
      const float vj = __shfl_sync(kFull, v, j);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (ej == e0 + i) add[i] += vj;
    }
    return;
  }
  store_row<EP>(row, e0, add);
  __syncwarp();
  if (e >= 0) row[e] = v;
  __syncwarp();
  load_floats<float, NV>(row + e0, add);
}

// The dense gradient's exponentials on the special-function unit: 2 FP32 steps plus |x| / 2
// (the product with log2 e is rounded), which a gradient of many summed terms absorbs.  With
// the library's exponential and rounded reciprocal they were a quarter of the kernel's
// instructions (T = 32768, E = 256: 22.5 us against 18.4 with these and the loads ahead).  Without
// d_prob_sum the chosen experts' sigmoid is expf's: the two calls' gradients of a chosen logit
// agree to these steps, not to the last bit.
__device__ __forceinline__ float2 sigmoid_and_slope_fast(float l) {
  l = fmaxf(l, -INFINITY);
  const float t = __expf(-fabsf(l)), r = __fdividef(1.0f, 1.0f + t), u = t * r;
  return make_float2(l < 0.0f ? u : r, u * r);
}

// DENSE: every expert of a row has a gradient (d_prob, or the plain softmax probability);
// otherwise only the chosen ones, and only their logits are read.
template <typename Tin, int EP, int KIND, bool DENSE, bool DBIAS>
__global__ void __launch_bounds__(kSelThreads, DENSE ? kSelBlocksPerSm : 6) select_bwd_kernel(
    SelectArgs a, const int32_t* __restrict__ topk_idx, const float* __restrict__ d_w,
    const float* __restrict__ d_prob, Tin* __restrict__ d_logits, long long ldd,
    float* __restrict__ partial) {
  constexpr int NV = EP / 32;
  if constexpr (DBIAS) pdl_launch_dependents();
  __shared__ __align__(16) float s_row[kSelWarps][EP];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e0 = lane * NV;
  const int E = a.E, k = a.k;
  const Tin* logits = static_cast<const Tin*>(a.logits);
  const bool vec = rows_aligned<Tin, NV>(logits, a.ld);
  const bool vecd = rows_aligned<Tin, NV>(d_logits, ldd);
  float b[DENSE ? NV : 1], g[DENSE ? NV : 1], col[DBIAS ? NV : 1];
  if constexpr (DENSE) {
    lane_bias<NV>(a.bias, e0, E, b);
    lane_vector<NV>(d_prob, e0, E, g);
  }
  if constexpr (DBIAS) {
#pragma unroll
    for (int i = 0; i < NV; ++i) col[i] = 0.0f;
  }
  const long long t0 = (long long)blockIdx.x * kSelWarps + warp;
  const long long stride = (long long)gridDim.x * kSelWarps;
  // the next token's loads are in flight while this one is computed
  float next[DENSE ? NV : 1];
  int next_e = -1;
  float next_d = 0.0f;
  auto fetch = [&](long long t) {
    if (t >= a.T) return;
    if (lane < k) {
      next_e = topk_idx[t * k + lane];
      next_d = d_w[t * k + lane];
    }
    if constexpr (DENSE) load_row<Tin, NV>(logits + t * a.ld, e0, E, vec, next);
  };
  fetch(t0);
  // sigmoid: experts that the bias masks (it joins nothing else here)
  unsigned off = 0u;
  if constexpr (DENSE && KIND == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (b[i] == -INFINITY) off |= 1u << i;
  }
  const bool any_off = __any_sync(kFull, off != 0u);
  for (long long t = t0; t < a.T; t += stride) {
    const int ej = next_e;
    const float dj = next_d;
    const bool valid = ej >= 0 && ej < E;
    float d[NV];
    float picked = KIND == 0 ? -INFINITY : 0.0f;  // slot j's key or score, in lane j
    float slope = 0.0f;                               // slot j's s (1 - s)
    // the lane's keys, then probabilities; sigmoid: scores, then slopes
    float sc[DENSE ? NV : 1], m = -INFINITY;
    float z = 0.0f, dot = 0.0f;  // sigmoid: the lane's sums of scores and of g times them
    if constexpr (DENSE) {
      float l[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) l[i] = next[i];
      fetch(t + stride);
      // the choice is made: any exponential will do
      __syncwarp();
      if constexpr (KIND == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const float v = __fadd_rn(l[i], b[i]);
          sc[i] = (v > -INFINITY) ? v : -INFINITY;
          m = fmaxf(m, sc[i]);
        }
      } else {
        float s[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const float2 v = sigmoid_and_slope_fast(l[i]);
          s[i] = v.x;
          sc[i] = v.y;
        }
        if (any_off) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if ((off >> i) & 1u) s[i] = sc[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          z += s[i];
          dot += g[i] * s[i];
        }
        store_row<EP>(s_row[warp], e0, s);
      }
      if constexpr (KIND == 0) store_row<EP>(s_row[warp], e0, sc);
      __syncwarp();
      if (valid) picked = s_row[warp][ej];
    } else {
      fetch(t + stride);
    }
    if (!DENSE && valid) {
      const float l = to_float(logits[t * a.ld + ej]);
      if constexpr (KIND == 0) {
        const float v = l + (a.bias != nullptr ? __ldg(a.bias + ej) : 0.0f);
        picked = (v > -INFINITY) ? v : -INFINITY;
      } else {
        const bool open = a.bias == nullptr || __ldg(a.bias + ej) > -INFINITY;
        const float2 v = sigmoid_and_slope(open ? l : -INFINITY);
        picked = v.x;
        slope = v.y;
      }
    }
    if constexpr (KIND == 0) {
      float rz = 0.0f;
      if constexpr (DENSE) {
        m = warp_max(m);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          sc[i] = exp_rel_fast(sc[i], m);
          z += sc[i];
        }
        z = warp_sum(z);
        rz = z > 0.0f ? 1.0f / z : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          sc[i] *= rz;
          dot += g[i] * sc[i];
        }
      }
      float cd;  // what the chosen logit gets beside the dense part
      if (!DENSE || a.renorm) {
        const float e = exp_rel(picked, warp_max(picked));
        const float S = warp_sum(e);
        const float w = S > 0.0f ? e / S : 0.0f;
        cd = w * (dj - warp_sum(dj * w));
      } else {
        cd = dj * (exp_rel(picked, m) * rz);
        dot += cd;
      }
      spread<EP>(s_row[warp], e0, lane, valid ? ej : -1, cd, k, d);
      if constexpr (DENSE) {
        dot = warp_sum(dot);
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] += sc[i] * (g[i] - dot);
      }
    } else {
      float cd = dj;
      if (a.renorm) {
        const float S = warp_sum(picked);
        cd = S > 0.0f ? __fdiv_rn(dj - __fdiv_rn(warp_sum(__fmul_rn(dj, picked)), S), S) : 0.0f;
      }
      if constexpr (DENSE) {
        z = warp_sum(z);
        const float rz = z > 0.0f ? 1.0f / z : 0.0f;
        const float mean = warp_sum(dot) * rz;
        spread<EP>(s_row[warp], e0, lane, valid ? ej : -1, cd, k, d);
#pragma unroll
        for (int i = 0; i < NV; ++i)
          d[i] = ((g[i] - mean) * rz + d[i]) * sc[i];
      } else {
        cd = __fmul_rn(cd, slope);
        spread<EP>(s_row[warp], e0, lane, valid ? ej : -1, cd, k, d);
      }
    }
    Tin* row = d_logits + t * ldd;
    if (vecd && e0 + NV <= E) {
      store_floats<Tin, NV>(row + e0, d);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (e0 + i < E) row[e0 + i] = from_float<Tin>(d[i]);
    }
    if constexpr (DBIAS) {
#pragma unroll
      for (int i = 0; i < NV; ++i) col[i] += d[i];
    }
  }
  if constexpr (DBIAS) {
    __syncwarp();
    write_partial<EP>(s_row, warp, e0, col, E, partial);
  }
}

// out[e] = sum over b of partial[b][e], in a fixed order
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* __restrict__ partial, int nb,
                                                          int E, float* __restrict__ out) {
  __shared__ float s[32][33];
  const int e = blockIdx.x * 32 + threadIdx.x;
  float v = 0.0f;
  pdl_wait();  // the partial sums are complete
  if (e < E)
    for (int b = threadIdx.y; b < nb; b += 32) v += partial[(size_t)b * E + e];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && e < E) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][threadIdx.x];
    out[e] = t;
  }
}

int select_blocks(int T) {
  const long long need = ((long long)T + kSelWarps - 1) / kSelWarps;
  const long long most = (long long)device_sm_count() * kSelBlocksPerSm;
  return (int)(need < most ? need : most);
}

template <typename Tin, int EP, int KIND>
cudaError_t fwd_ep(const SelectArgs& a, int32_t* idx, float* w, float* prob_sum, float* partial,
                   cudaStream_t s) {
  const int nb = select_blocks(a.T);
  if (prob_sum == nullptr) {
    select_kernel<Tin, EP, KIND, false><<<nb, kSelThreads, 0, s>>>(a, idx, w, nullptr);
    return cudaGetLastError();
  }
  select_kernel<Tin, EP, KIND, true><<<nb, kSelThreads, 0, s>>>(a, idx, w, partial);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_pdl(column_sum_kernel, dim3((a.E + 31) / 32), dim3(32, 32), 0, s,
                    static_cast<const float*>(partial), nb, a.E, prob_sum);
}

template <typename Tin, int EP, int KIND>
cudaError_t bwd_ep(const SelectArgs& a, const int32_t* idx, const float* d_w, const float* d_prob,
                   void* d_logits, long long ldd, float* d_bias, float* partial, cudaStream_t s) {
  const int nb = select_blocks(a.T);
  const bool dense = d_prob != nullptr || (KIND == 0 && !a.renorm);
  auto go = [&](auto kern) {
    kern<<<nb, kSelThreads, 0, s>>>(a, idx, d_w, d_prob, static_cast<Tin*>(d_logits), ldd, partial);
    return cudaGetLastError();
  };
  if (d_bias == nullptr)
    return dense ? go(select_bwd_kernel<Tin, EP, KIND, true, false>)
                 : go(select_bwd_kernel<Tin, EP, KIND, false, false>);
  if constexpr (KIND == 0) {
    const cudaError_t e = dense ? go(select_bwd_kernel<Tin, EP, KIND, true, true>)
                                : go(select_bwd_kernel<Tin, EP, KIND, false, true>);
    if (e != cudaSuccess) return e;
    return launch_pdl(column_sum_kernel, dim3((a.E + 31) / 32), dim3(32, 32), 0, s,
                      static_cast<const float*>(partial), nb, a.E, d_bias);
  }
  return cudaErrorInvalidValue;  // the selection-only bias has no gradient
}

// f(type tag, EP constant) for the logits' type and the experts rounded up to 32 * 2^n
template <typename F>
cudaError_t by_type_and_experts(int dtype, int E, F&& f) {
  auto by_e = [&](auto tag) -> cudaError_t {
    using Tin = decltype(tag);
    if (E <= 32) return f(Tin{}, std::integral_constant<int, 32>{});
    if (E <= 64) return f(Tin{}, std::integral_constant<int, 64>{});
    if (E <= 128) return f(Tin{}, std::integral_constant<int, 128>{});
    return f(Tin{}, std::integral_constant<int, 256>{});
  };
  if (dtype == MOE_DTYPE_F32) return by_e(float{});
  if (dtype == MOE_DTYPE_BF16) return by_e(__nv_bfloat16{});
  return by_e(__half{});
}

SelectArgs args_of(const void* logits, long long ld, const float* bias, const moe_select_opts& o,
                   int T, int E, int k) {
  const int per = E / o.n_group;
  int shift = 5;
  while ((1 << (5 - shift)) < o.n_group) --shift;
  return SelectArgs{logits,       ld,          bias,     T,   E,
                    k,            o.n_group,   o.topk_group, o.group_top, o.renorm,
                    per,          (65536 + per - 1) / per, shift};
}

}  // namespace

size_t select_partial_bytes(int T, int E) { return (size_t)select_blocks(T) * E * sizeof(float); }

cudaError_t launch_select(const void* logits, int dtype, long long ld, const float* bias,
                          const moe_select_opts& o, int T, int E, int k, int32_t* topk_idx,
                          float* topk_w, float* prob_sum, float* partial, cudaStream_t s) {
  const SelectArgs a = args_of(logits, ld, bias, o, T, E, k);
  return by_type_and_experts(dtype, E, [&](auto tin, auto ep) -> cudaError_t {
    using Tin = decltype(tin);
    constexpr int EP = decltype(ep)::value;
    return o.kind == MOE_ROUTER_SOFTMAX
               ? fwd_ep<Tin, EP, 0>(a, topk_idx, topk_w, prob_sum, partial, s)
               : fwd_ep<Tin, EP, 1>(a, topk_idx, topk_w, prob_sum, partial, s);
  });
}

cudaError_t launch_select_bwd(const void* logits, int dtype, long long ld, const float* bias,
                              const moe_select_opts& o, int T, int E, int k,
                              const int32_t* topk_idx, const float* d_topk_w,
                              const float* d_prob_sum, void* d_logits, long long ld_d,
                              float* d_bias, float* partial, cudaStream_t s) {
  const SelectArgs a = args_of(logits, ld, bias, o, T, E, k);
  return by_type_and_experts(dtype, E, [&](auto tin, auto ep) -> cudaError_t {
    using Tin = decltype(tin);
    constexpr int EP = decltype(ep)::value;
    return o.kind == MOE_ROUTER_SOFTMAX
               ? bwd_ep<Tin, EP, 0>(a, topk_idx, d_topk_w, d_prob_sum, d_logits, ld_d, d_bias,
                                    partial, s)
               : bwd_ep<Tin, EP, 1>(a, topk_idx, d_topk_w, d_prob_sum, d_logits, ld_d, d_bias,
                                    partial, s);
  });
}

}  // namespace moe

// Scoring and top-k of one token's router logits by one wave, shared by the
// router kernels and the whole-layer kernel.
//
// Lane l holds the experts l, l + 64, ...  A candidate's key is a float64
// (the logit, or its score plus the selection bias), mapped to an unsigned
// 64-bit integer of the same order with 0 for an expert that cannot be
// chosen, and the top-k is k rounds of a wave-wide maximum: the high words'
// maximum, then the low words' among the lanes that hold it, both with DPP
// (no LDS traffic).  Keys are float64 because experts whose scores agree to
// float32 rounding must still come out in the order of their exact scores:
// with 8192 tokens of 512 experts some token's 8th and 9th lie that close
// in a good part of all batches.
#pragma once

#include <float.h>

#include "device_common.h"
#include "kernels.h"

namespace moe {

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}

// Maximum over the 64 lanes, uniform: row shifts by 1, 2, 4 and 8, then the
// last lane of a row to the next rows; lane 63 has seen every lane.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, dpp_u32<0x111, 0xf>(v));
  v = max(v, dpp_u32<0x112, 0xf>(v));
  v = max(v, dpp_u32<0x114, 0xf>(v));
  v = max(v, dpp_u32<0x118, 0xf>(v));
  v = max(v, dpp_u32<0x142, 0xa>(v));
  v = max(v, dpp_u32<0x143, 0xc>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ double wave_max_f64(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = fmax(v, __shfl_xor(v, d));
  return v;
}

// The logit an expert competes with: -inf when it cannot be chosen (NaN or
// -inf), +inf taken as the largest finite float32.
__device__ __forceinline__ double route_logit(double l) {
  if (!(l > -INFINITY)) return -INFINITY;
  return fmax(fmin(l, (double)FLT_MAX), -(double)FLT_MAX);
}

__device__ __forceinline__ double sigmoid_f64(double l) { return 1.0 / (1.0 + exp(-l)); }

// float64 -> unsigned of the same order, > 0 for every number but NaN and
// -inf (which give 0); -0.0 counts as +0.0.
__device__ __forceinline__ uint64_t order_key(double v) {
  if (!(v > -INFINITY)) return 0;
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

// Ranks one token.  l[i]: route_logit of expert lane + 64 i (-inf past E).
// s_key: LDS of this wave, E doubles, used
// only with groups.  Returns in lane j < topk the j-th chosen expert (-1:
// none left) and its weight; the other lanes get -1 and 0.
template <int NV>
__device__ __forceinline__ void route_token(const RouterArgs& r, const double (&l)[NV],
                                            const float* __restrict__ bias, double* s_key,
                                            int& my_id, float& my_w) {
  const int lane = threadIdx.x & 63;
  const bool softmax = r.scoring == 0;
  const bool by_score = r.bias_kind == 2 || r.groups > 1;
  double top = -INFINITY, total = 0.0;
  if (softmax && (by_score || !r.renormalize)) {
    // the row's maximum and the sum of its exponentials
#pragma unroll
    for (int i = 0; i < NV; ++i) top = fmax(top, l[i]);
    top = wave_max_f64(top);
    if (by_score) {
#pragma unroll
      for (int i = 0; i < NV; ++i) total += l[i] > -INFINITY ? exp(l[i] - top) : 0.0;
    } else {
      // only a weight's denominator: 32-bit exponentials are enough
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) t += l[i] > -INFINITY ? expf((float)(l[i] - top)) : 0.f;
      total = t;
    }
    total = wave_sum_f64(total);
  }
  uint64_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    double k = l[i];
    if (by_score && l[i] > -INFINITY) {
      k = softmax ? exp(l[i] - top) / total : sigmoid_f64(l[i]);
      if (r.bias_kind == 2) k += (double)bias[lane + 64 * i];
    }
    key[i] = order_key(k);
    if (r.groups > 1 && lane + 64 * i < r.E) s_key[lane + 64 * i] = key[i] ? k : -INFINITY;
  }
  if (r.groups > 1) {
    // lane g scores group g: the sum of its two best keys (of the one there
    // is, or -inf); the topk_groups best groups stay
    __builtin_amdgcn_wave_barrier();
    const int per = r.E / r.groups;
    double b0 = -INFINITY, b1 = -INFINITY;
    if (lane < r.groups) {
      for (int q = 0; q < per; ++q) {
        const double k = s_key[lane * per + q];
        if (k > b0) { b1 = b0; b0 = k; } else if (k > b1) b1 = k;
      }
    }
    uint64_t gk = order_key(b1 > -INFINITY ? b0 + b1 : b0);
    uint64_t keep = 0;
    for (int n = 0; n < r.topk_groups; ++n) {
      const uint32_t hi = wave_max_u32((uint32_t)(gk >> 32));
      const bool in = (uint32_t)(gk >> 32) == hi;
      const uint32_t lo = wave_max_u32(in ? (uint32_t)gk : 0u);
      const uint64_t tie = __ballot(in && (uint32_t)gk == lo);
      if ((hi | lo) == 0) break;
      const int g = __ffsll((unsigned long long)tie) - 1;
      keep |= 1ull << g;
      if (lane == g) gk = 0;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 64 * i < r.E && !((keep >> ((lane + 64 * i) / per)) & 1)) key[i] = 0;
  }

  my_id = -1;
  double my_l = -INFINITY;
  for (int j = 0; j < r.topk; ++j) {
    uint64_t best = key[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < NV; ++i)
      if (key[i] > best) { best = key[i]; bi = i; }
    const uint32_t hi = wave_max_u32((uint32_t)(best >> 32));
    const bool in = (uint32_t)(best >> 32) == hi;
    const uint32_t lo = wave_max_u32(in ? (uint32_t)best : 0u);
    if ((hi | lo) == 0) break;   // nothing left to choose
    const bool tied = in && (uint32_t)best == lo;
    const uint64_t who = __ballot(tied);
    int e;
    if (NV == 1 || (who & (who - 1)) == 0) {
      const int src = __ffsll((unsigned long long)who) - 1;
      e = src + 64 * __builtin_amdgcn_readlane(bi, src);
    } else {
      // several lanes hold the same key: the lowest expert
      e = (int)(0x7fffffffu - wave_max_u32(tied ? 0x7fffffffu - (uint32_t)(lane + 64 * bi) : 0u));
    }
    e = __builtin_amdgcn_readfirstlane(e);
    double v = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i == (e >> 6)) {
        v = l[i];
        if (lane == (e & 63)) key[i] = 0;
      }
    v = __shfl(v, e & 63);
    if (lane == j) { my_id = e; my_l = v; }
  }

  // the weights of the chosen, in float64 (one exponential per slot)
  double w = 0.0;
  const bool have = my_id >= 0;
  if (softmax) {
    if (r.renormalize) {
      const double m = wave_max_f64(my_l);
      w = have ? exp(my_l - m) : 0.0;
      const double sum = wave_sum_f64(w);
      w = have ? w / sum : 0.0;
    } else {
      w = have ? exp(my_l - top) / total : 0.0;
    }
  } else {
    w = have ? sigmoid_f64(my_l) : 0.0;
    if (r.renormalize) {
      const double sum = wave_sum_f64(w);
      w = sum > 0.0 ? w / sum : 0.0;
    }
  }
  my_w = (float)(w * (double)r.scale);
}

}  // namespace moe

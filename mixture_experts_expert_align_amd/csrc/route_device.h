// Scoring and top-k of one token's router logits by one wave, shared by the
// router kernels and the whole-layer kernel.
//
// Lane l holds the experts l, l + 64, ...  A candidate's key is a float64
// (the logit, or its score plus the selection bias), mapped to an unsigned
// 64-bit integer of the same order with 0 for an expert that cannot be
// chosen, and the top-k is k rounds of a wave-wide maximum: the high words'
// maximum, then (where several lanes hold it) the low words' among those,
// both with DPP (no LDS traffic).  Keys are float64 because experts whose scores agree to
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

__device__ __forceinline__ double readlane_f64(double v, int from) {   // from: uniform
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, from);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), from);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
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

// The token's groups: expert e is in group e / per, as e * inv >> 21 (exact
// for e < 2048, per <= 1024); its key lies at LDS place e + group, so that
// the groups' scans start in different banks.
struct GroupIndex {
  int per;
  uint32_t inv;
  __device__ __forceinline__ explicit GroupIndex(const RouterArgs& r)
      : per(r.E / r.groups), inv((1u << 21) / (uint32_t)per + 1) {}
  __device__ __forceinline__ int of(int e) const { return (int)(((uint32_t)e * inv) >> 21); }
};

// Lane (g, s) of the first groups * lanes ones: the group key of group g (the
// sum of its two best keys, of the one there is, or 0 for none), scanned by
// `lanes` lanes (a power of two), in lane s = 0; 0 elsewhere.
__device__ __forceinline__ uint64_t group_key(const RouterArgs& r, const GroupIndex& gi, const double* s_key, int i,
                                              int lanes) {
  const int g = i / lanes;
  double b0 = -INFINITY, b1 = -INFINITY;
  if (g < r.groups) {
#pragma unroll 4
    for (int q = i % lanes; q < gi.per; q += lanes) {
      const double k = s_key[g * (gi.per + 1) + q];
      b1 = fmax(b1, fmin(b0, k));
      b0 = fmax(b0, k);
    }
  }
  for (int d = 1; d < lanes; d *= 2) {
    const double o0 = __shfl_xor(b0, d), o1 = __shfl_xor(b1, d);
    b1 = fmax(fmin(b0, o0), fmax(b1, o1));
    b0 = fmax(b0, o0);
  }
  return i % lanes ? 0 : order_key(b1 > -INFINITY ? b0 + b1 : b0);
}
// Lanes that can share a group's scan among n.
__device__ __forceinline__ int group_lanes(const RouterArgs& r, int n) {
  int lanes = 1;
  while (2 * lanes * r.groups <= n) lanes *= 2;
  return lanes;
}

// Ranks one token.  l[i]: route_logit of expert lane + 64 i (-inf past E).
// s_key: LDS of this wave, E + groups doubles, used
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
  const GroupIndex gi(r);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    double k = l[i];
    if (by_score && l[i] > -INFINITY) {
      k = softmax ? exp(l[i] - top) / total : sigmoid_f64(l[i]);
      if (r.bias_kind == 2) k += (double)bias[lane + 64 * i];
    }
    key[i] = order_key(k);
    if (r.groups > 1 && lane + 64 * i < r.E)
      s_key[lane + 64 * i + gi.of(lane + 64 * i)] = key[i] ? k : -INFINITY;
  }
  if (r.groups > 1) {
    // the topk_groups best groups stay
    __builtin_amdgcn_wave_barrier();
    const int lanes = group_lanes(r, 64);
    uint64_t gk = group_key(r, gi, s_key, lane, lanes);
    uint64_t keep = 0;
    for (int n = 0; n < r.topk_groups; ++n) {
      const uint32_t hi = wave_max_u32((uint32_t)(gk >> 32));
      const bool in = (uint32_t)(gk >> 32) == hi;
      const uint32_t lo = wave_max_u32(in ? (uint32_t)gk : 0u);
      const uint64_t tie = __ballot(in && (uint32_t)gk == lo);
      if ((hi | lo) == 0) break;
      const int first = __ffsll((unsigned long long)tie) - 1;
      keep |= 1ull << (first / lanes);
      if (lane == first) gk = 0;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 64 * i < r.E && !((keep >> gi.of(lane + 64 * i)) & 1)) key[i] = 0;
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
    if (hi == 0) break;   // nothing left to choose (a key's high word is not 0)
    bool tied = (uint32_t)(best >> 32) == hi;
    uint64_t who = __ballot(tied);
    if (who & (who - 1)) {
      const uint32_t lo = wave_max_u32(tied ? (uint32_t)best : 0u);
      tied = tied && (uint32_t)best == lo;
      who = __ballot(tied);
    }
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
    v = readlane_f64(v, e & 63);
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

// ------------------------------------------------ four tokens to a wave --
// The same with 16 lanes to a token, so that a round's reductions, which stay
// within a row of 16 lanes, serve four tokens at once.  Lane c of a row holds
// the experts c, c + 16, ...

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = dpp_u32<CTRL, 0xf>((uint32_t)u), hi = dpp_u32<CTRL, 0xf>((uint32_t)(u >> 32));
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
// Quads by lane 1 and 2 apart, then the mirrored half row, then the mirrored
// row: every lane of a row ends with the same bits.
template <typename F>
__device__ __forceinline__ double row_reduce_f64(double v, F f) {
  v = f(v, dpp_f64<0xb1>(v));
  v = f(v, dpp_f64<0x4e>(v));
  v = f(v, dpp_f64<0x141>(v));
  return f(v, dpp_f64<0x140>(v));
}
__device__ __forceinline__ double row_sum_f64(double v) {
  return row_reduce_f64(v, [](double a, double b) { return a + b; });
}
__device__ __forceinline__ double row_max_f64(double v) {
  return row_reduce_f64(v, [](double a, double b) { return fmax(a, b); });
}
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
  v = max(v, dpp_u32<0xb1, 0xf>(v));
  v = max(v, dpp_u32<0x4e, 0xf>(v));
  v = max(v, dpp_u32<0x141, 0xf>(v));
  return max(v, dpp_u32<0x140, 0xf>(v));
}

// Ranks one token per row; topk <= 16, groups <= 16.  logit(e): route_logit
// of the row's expert e.  As route_token, slot j in lane j of the row.
template <int NV, typename Logit>
__device__ __forceinline__ void route_row(const RouterArgs& r, Logit logit, const float* __restrict__ bias,
                                          double* s_key, int& my_id, float& my_w) {
  const int lane = threadIdx.x & 63, c = lane & 15;
  const bool softmax = r.scoring == 0;
  const bool by_score = r.bias_kind == 2 || r.groups > 1;
  uint32_t hi[NV], lo[NV];
  double top = -INFINITY, total = 0.0;
  {
    double l[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = c + 16 * i < r.E ? logit(c + 16 * i) : -INFINITY;
    if (softmax && (by_score || !r.renormalize)) {
#pragma unroll
      for (int i = 0; i < NV; ++i) top = fmax(top, l[i]);
      top = row_max_f64(top);
      if (by_score) {
#pragma unroll
        for (int i = 0; i < NV; ++i) total += l[i] > -INFINITY ? exp(l[i] - top) : 0.0;
      } else {
        float t = 0.f;   // only a weight's denominator
#pragma unroll
        for (int i = 0; i < NV; ++i) t += l[i] > -INFINITY ? expf((float)(l[i] - top)) : 0.f;
        total = t;
      }
      total = row_sum_f64(total);
    }
    const GroupIndex gi(r);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = c + 16 * i;
      double k = l[i];
      if (by_score && l[i] > -INFINITY) {
        k = softmax ? exp(l[i] - top) / total : sigmoid_f64(l[i]);
        if (r.bias_kind == 2) k += (double)bias[e];
      }
      const uint64_t key = order_key(k);
      hi[i] = (uint32_t)(key >> 32);
      lo[i] = (uint32_t)key;
      if (r.groups > 1 && e < r.E) s_key[e + gi.of(e)] = key ? k : -INFINITY;
    }
    if (r.groups > 1) {
      __builtin_amdgcn_wave_barrier();
      const int lanes = group_lanes(r, 16);
      const uint64_t gk = group_key(r, gi, s_key, c, lanes);
      uint32_t ghi = (uint32_t)(gk >> 32), keep = 0;
      for (int n = 0; n < r.topk_groups; ++n) {
        const uint32_t h = row_max_u32(ghi);
        const uint32_t w = row_max_u32(ghi == h ? (uint32_t)gk : 0u);
        const uint32_t first = 16u - row_max_u32(h && ghi == h && (uint32_t)gk == w ? 16u - c : 0u);
        if (first < 16) keep |= 1u << (first / lanes);
        if ((uint32_t)c == first) ghi = 0;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (c + 16 * i < r.E && !((keep >> gi.of(c + 16 * i)) & 1)) hi[i] = 0;
    }
  }

  my_id = -1;
  for (int j = 0; j < r.topk; ++j) {
    uint32_t m = hi[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = max(m, hi[i]);
    m = row_max_u32(m);
    int n = 0, at = 0;   // this lane's experts with it, and the last of them
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      n += hi[i] == m;
      at = hi[i] == m ? i : at;
    }
    n = m ? n : 0;   // m == 0: the row has nothing left
    const uint32_t who = (uint32_t)(__ballot(n > 0) >> (lane & 48)) & 0xffffu;
    if (!__any(n > 1 || (who & (who - 1)))) {
      const uint32_t e1 = row_max_u32(n ? (uint32_t)(c + 16 * at + 1) : 0u);
      if (c == j) my_id = (int)e1 - 1;
#pragma unroll
      for (int i = 0; i < NV; ++i) hi[i] = hi[i] == m ? 0 : hi[i];
    } else {   // equal high words in some row: the low words, then the lowest expert
      uint32_t w = 0, first = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) w = max(w, hi[i] == m ? lo[i] : 0u);
      w = row_max_u32(w);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        first = max(first, m && hi[i] == m && lo[i] == w ? 0x10000u - (uint32_t)(c + 16 * i) : 0u);
      first = row_max_u32(first);
      const int e = first ? (int)(0x10000u - first) : -1;
      if (c == j) my_id = e;
#pragma unroll
      for (int i = 0; i < NV; ++i) hi[i] = c + 16 * i == e ? 0 : hi[i];
    }
  }

  double w = 0.0;
  const bool have = my_id >= 0;
  const double my_l = have ? logit(my_id) : -INFINITY;
  if (softmax) {
    if (r.renormalize) {
      const double m = row_max_f64(my_l);
      w = have ? exp(my_l - m) : 0.0;
      const double sum = row_sum_f64(w);
      w = have ? w / sum : 0.0;
    } else {
      w = have ? exp(my_l - top) / total : 0.0;
    }
  } else {
    w = have ? sigmoid_f64(my_l) : 0.0;
    if (r.renormalize) {
      const double sum = row_sum_f64(w);
      w = sum > 0.0 ? w / sum : 0.0;
    }
  }
  my_w = (float)(w * (double)r.scale);
}

}  // namespace moe

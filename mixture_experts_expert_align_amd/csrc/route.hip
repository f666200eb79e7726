// The router's scoring and top-k, and the gradient of its weights.
//
// For token t with logits l (plus a bias per expert): the topk experts with
// the largest keys, ties to the lowest expert, and their weights
//   w_j = scale * s_j          or, renormalised,  scale * s_j / sum_k s_k
// where s is the softmax over the experts or the sigmoid of each.  The
// gradient takes d(sum_j dw_j w_j) / dl with the choice held fixed:
//   softmax, renormalised: dl_j = scale p_j (dw_j - sum_k p_k dw_k) over the
//     chosen, p their softmax among themselves (the others cancel: 0);
//   softmax: dl_i = scale p_i (dw_i - sum_k p_k dw_k), dw_i = 0 unless chosen
//     (in float64 for the chosen: where one of them has nearly all of the
//     softmax, the difference is a small part of its terms);
//   sigmoid: dl_j = ds_j s_j (1 - s_j), ds_j = scale dw_j, or renormalised
//     scale (dw_j - sum_k dw_k s_k / S) / S with S = sum_k s_k.
//
// Nothing but the logits is read, once, and nothing but the result written, so
// the memory is never the bound: with few tokens it is one token's latency
// (the float64 exponentials and divisions of the scores, then k rounds of
// reductions), with many the instructions issued for that (4096 x 512 with 16
// groups: vector instructions issue in 59 to 68% of the cycles; 8192 x 128, two
// waves a SIMD: 29 to 38%, the rest is their latency).  Hence two forms.
// A wave per token: the shortest rounds; 3.3 us for 4 x 64, top-8, 18.8 us for
// 4096 x 512 with 16 groups (29 by the other form).  And 16 lanes per token,
// where a round's reductions serve four tokens at once but a lane has four
// times the experts to look through: forward beyond 4096 tokens (more than
// four waves per SIMD of the first form) of up to 128 experts, beyond 6144 of
// up to 256.  Replayed from a graph, a wave / 16 lanes per token, us:
//   tokens                           4096       5000       6000       8192      16384
//   128, softmax                   6.5/6.7    7.3/6.7    8.0/6.8    9.4/6.8  15.8/8.9
//   128 in 8 groups, softmax     10.7/11.3  12.1/11.4  13.5/11.5  16.5/11.5 28.4/17.0
//   256, softmax                   8.0/9.7    8.9/9.7    9.8/9.9   11.6/9.8 20.0/13.0
//   256 in 8 groups, sel. bias   12.1/16.4  13.9/16.4  15.7/16.4  19.0/16.3 33.2/23.4
//   256, sigmoid, sel. bias       9.3/14.0  10.6/14.1  11.8/14.1  14.4/14.2 24.9/20.0
// Backward, whose rows have no rounds, from 2048 tokens; where every expert has
// a gradient (softmax, not renormalised) and there are more than 128, whose
// exponentials a lane then takes 16 or 32 of, from 4097:
//   tokens                           2048       3000       4096       8192      16384
//   128, chosen only               4.6/3.7    4.8/3.9    5.4/4.0    7.0/4.3  11.2/5.8
//   512, chosen only               7.5/6.3    8.2/6.9    9.1/7.2   12.9/8.3 22.0/13.9
//   128, every expert              6.2/6.0    6.6/6.7    7.3/6.8   10.8/7.2  18.4/9.8
//   256, every expert              8.4/9.0   9.0/10.1  10.1/10.3  15.5/11.2 26.6/16.4
//   512, every expert            12.5/15.0  13.9/17.1  16.1/17.4  24.3/20.0 44.3/32.7
#include "kernels.h"
#include "route_device.h"

namespace moe {
namespace {

constexpr int kRouteWaves = 4;

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  return BF16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

template <int NV, bool BF16>
__global__ void __launch_bounds__(64 * kRouteWaves) route_topk_kernel(RouterArgs r, int64_t M,
                                                                     const void* __restrict__ logits, int64_t ld,
                                                                     const float* __restrict__ bias,
                                                                     int32_t* __restrict__ ids,
                                                                     float* __restrict__ weights) {
  extern __shared__ double s_keys[];   // with groups: E + groups doubles per wave
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (t >= M) return;
  double l[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    double v = -INFINITY;
    if (e < r.E) {
      v = load_logit<BF16>(logits, t * ld + e);
      if (r.bias_kind == 1) v += (double)bias[e];
    }
    l[i] = route_logit(v);
  }
  int id;
  float w;
  route_token<NV>(r, l, bias, s_keys + (r.groups > 1 ? wave * (r.E + r.groups) : 0), id, w);
  if (lane < r.topk) {
    ids[t * r.topk + lane] = id;
    weights[t * r.topk + lane] = w;
  }
}

constexpr int kRowWaves = 2;
constexpr int64_t kRowsForwardTokens = 4097, kRowsForwardTokens256 = 6145;   // up to 128 experts, up to 256
constexpr int64_t kRowsBackwardTokens = 2048, kRowsBackwardTokensEvery = 4097;   // chosen or <= 128 experts; others
constexpr int kRowsForwardExperts = 256, kRowsBackwardExperts = 512;

template <int NV, bool BF16>
__global__ void __launch_bounds__(64 * kRowWaves) route_rows_kernel(RouterArgs r, int64_t M,
                                                                    const void* __restrict__ logits, int64_t ld,
                                                                    const float* __restrict__ bias,
                                                                    int32_t* __restrict__ ids,
                                                                    float* __restrict__ weights) {
  extern __shared__ double s_keys[];   // with groups: E + groups doubles per token
  const int row = threadIdx.x >> 4, c = threadIdx.x & 15;
  const int64_t t = (int64_t)blockIdx.x * (4 * kRowWaves) + row;
  const int64_t in = min(t, M - 1);    // past the last token: the last one again, not stored
  int id;
  float w;
  route_row<NV>(r, [&](int e) {
    double v = load_logit<BF16>(logits, in * ld + e);
    if (r.bias_kind == 1) v += (double)bias[e];
    return route_logit(v);
  }, bias, s_keys + (r.groups > 1 ? row * (r.E + r.groups) : 0), id, w);
  if (t < M && c < r.topk) {
    ids[t * r.topk + c] = id;
    weights[t * r.topk + c] = w;
  }
}

// e^x for x <= 0 to float32 precision: expf of the nearest float32, times e to
// the rest.  (Far below the smallest float32 the rest must not grow with x.)
__device__ __forceinline__ float exp_f32(double x) {
  x = fmax(x, -1000.0);
  const float h = (float)x;
  return expf(h) * (1.0f + (float)(x - (double)h));
}

template <bool BF16>
__global__ void __launch_bounds__(64 * kRouteWaves) route_topk_backward_kernel(
    RouterArgs r, int64_t M, const void* __restrict__ logits, int64_t ld, const float* __restrict__ bias,
    const int32_t* __restrict__ ids, const float* __restrict__ dw, void* __restrict__ dl, int64_t dl_ld) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (t >= M) return;
  const bool softmax = r.scoring == 0;
  auto logit = [&](int e) {
    double v = load_logit<BF16>(logits, t * ld + e);
    if (r.bias_kind == 1) v += (double)bias[e];
    return route_logit(v);
  };
  // slot j of the token in lane j
  int id = lane < r.topk ? ids[t * r.topk + lane] : -1;
  if (id < 0 || id >= r.E) id = -1;
  const double lj = id >= 0 ? logit(id) : -INFINITY;
  const bool have = lj > -INFINITY;
  const double g = have ? (double)dw[t * r.topk + lane] * (double)r.scale : 0.0;
  double top = -INFINITY, d = 0.0;
  float rest = 0.f;   // dense: an unchosen expert's gradient is e^(l - top) rest
  const bool dense = softmax && !r.renormalize;   // every expert has a gradient
  if (dense) {
    for (int e = lane; e < r.E; e += 64) top = fmax(top, logit(e));
    top = wave_max_f64(top);
    double s = 0.0;
    for (int e = lane; e < r.E; e += 64) {
      const double v = logit(e);
      s += v > -INFINITY ? exp(v - top) : 0.0;
    }
    const double total = wave_sum_f64(s);
    const double inv = total > 0.0 ? 1.0 / total : 0.0;
    const double p = have ? exp(lj - top) * inv : 0.0;
    const double dot = wave_sum_f64(p * g);
    double own = 0.0;   // of all slots with this one's expert
    for (int j = 0; j < r.topk; ++j) own += __builtin_amdgcn_readlane(id, j) == id ? readlane_f64(g, j) : 0.0;
    d = p * (own - dot);
    rest = (float)((0.0 - dot) * inv);
  } else if (softmax) {
    const double m = wave_max_f64(lj);
    const double e = have ? exp(lj - m) : 0.0;
    const double sum = wave_sum_f64(e);
    const double p = have ? e / sum : 0.0;
    d = p * (g - wave_sum_f64(p * g));
  } else {
    const double s = have ? sigmoid_f64(lj) : 0.0;
    d = g;
    if (r.renormalize) {
      const double S = wave_sum_f64(s);
      const double gs = wave_sum_f64(g * s);
      d = S > 0.0 ? (g - gs / S) / S : 0.0;
    }
    d *= have ? s * (1.0 - s) : 0.0;
  }
  const float df = (float)d;
  for (int e = lane; e - lane < r.E; e += 64) {
    // an expert named in several slots gets the sum of their gradients (dense:
    // each of them is that sum already; the unchosen get -p_e dot)
    float v = 0.f;
    auto slot = [&](int j) {
      return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(df), j));
    };
    if (dense) {
      const double le = e < r.E ? logit(e) : -INFINITY;
      if (le > -INFINITY) v = exp_f32(le - top) * rest;
      for (int j = 0; j < r.topk; ++j) v = __builtin_amdgcn_readlane(id, j) == e ? slot(j) : v;
    } else {
      for (int j = 0; j < r.topk; ++j) v += __builtin_amdgcn_readlane(id, j) == e ? slot(j) : 0.f;
    }
    if (e < r.E) {
      if (BF16)
        static_cast<uint16_t*>(dl)[t * dl_ld + e] = (uint16_t)f32_to_bf16_rne(v);
      else
        static_cast<float*>(dl)[t * dl_ld + e] = v;
    }
  }
}

// The same, a token per row of 16 lanes.
template <int NV, bool BF16>
__global__ void __launch_bounds__(64 * kRowWaves) route_rows_backward_kernel(
    RouterArgs r, int64_t M, const void* __restrict__ logits, int64_t ld, const float* __restrict__ bias,
    const int32_t* __restrict__ ids, const float* __restrict__ dw, void* __restrict__ dl, int64_t dl_ld) {
  const int lane = threadIdx.x & 63, row = threadIdx.x >> 4, c = lane & 15;
  const int64_t t = (int64_t)blockIdx.x * (4 * kRowWaves) + row;
  const int64_t in = min(t, M - 1);    // past the last token: the last one again, not stored
  auto logit = [&](int e) {
    double v = load_logit<BF16>(logits, in * ld + e);
    if (r.bias_kind == 1) v += (double)bias[e];
    return route_logit(v);
  };
  int id = c < r.topk ? ids[in * r.topk + c] : -1;
  if (id < 0 || id >= r.E) id = -1;
  const double lj = id >= 0 ? logit(id) : -INFINITY;
  const bool have = lj > -INFINITY;
  const double g = have ? (double)dw[in * r.topk + c] * (double)r.scale : 0.0;
  double d = g;
  const bool softmax = r.scoring == 0, dense = softmax && !r.renormalize;
  float p[NV], rest = 0.f;   // dense: an unchosen expert's gradient is p rest
  if (dense) {
    double top = -INFINITY, s = 0.0;
    double l[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      l[i] = c + 16 * i < r.E ? logit(c + 16 * i) : -INFINITY;
      top = fmax(top, l[i]);
    }
    top = row_max_f64(top);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const double e = l[i] > -INFINITY ? exp(l[i] - top) : 0.0;
      s += e;
      p[i] = (float)e;
    }
    const double total = row_sum_f64(s);
    const double inv = total > 0.0 ? 1.0 / total : 0.0;
    const double q = have ? exp(lj - top) * inv : 0.0;
    const double dot = row_sum_f64(q * g);
    double own = 0.0;   // of all slots with this one's expert
    for (int j = 0; j < r.topk; ++j) {
      const double gj = __shfl(g, (lane & 48) | j);
      own += __shfl(id, (lane & 48) | j) == id ? gj : 0.0;
    }
    d = q * (own - dot);
    rest = (float)((0.0 - dot) * inv);
  } else if (softmax) {
    const double m = row_max_f64(lj);
    const double e = have ? exp(lj - m) : 0.0;
    const double sum = row_sum_f64(e);
    const double q = have ? e / sum : 0.0;
    d = q * (g - row_sum_f64(q * g));
  } else {
    const double s = have ? sigmoid_f64(lj) : 0.0;
    if (r.renormalize) {
      const double S = row_sum_f64(s);
      const double gs = row_sum_f64(g * s);
      d = S > 0.0 ? (g - gs / S) / S : 0.0;
    }
    d *= have ? s * (1.0 - s) : 0.0;
  }
  const float df = (float)d;
  float v[NV];
  // an expert named in several slots gets their sum (dense: each slot has it)
  auto slots = [&](auto put) {
    for (int j = 0; j < r.topk; ++j) {
      const int ej = __shfl(id, (lane & 48) | j);
      const float dj = __shfl(df, (lane & 48) | j);
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = put(ej == c + 16 * i, v[i], dj);
    }
  };
  if (dense) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = p[i] * rest;
    slots([](bool own, float old, float dj) { return own ? dj : old; });
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = 0.f;
    slots([](bool own, float old, float dj) { return old + (own ? dj : 0.f); });
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = c + 16 * i;
    if (t < M && e < r.E) {
      if (BF16)
        static_cast<uint16_t*>(dl)[t * dl_ld + e] = (uint16_t)f32_to_bf16_rne(v[i]);
      else
        static_cast<float*>(dl)[t * dl_ld + e] = v[i];
    }
  }
}

template <int NV>
hipError_t launch_topk(const RouterArgs& r, int64_t M, const void* logits, bool bf16, int64_t ld, const float* bias,
                       int32_t* ids, float* weights, hipStream_t s) {
  const dim3 grid((unsigned)((M + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
  const size_t lds = r.groups > 1 ? sizeof(double) * (r.E + r.groups) * kRouteWaves : 0;
  if (bf16)
    hipLaunchKernelGGL((route_topk_kernel<NV, true>), grid, block, lds, s, r, M, logits, ld, bias, ids, weights);
  else
    hipLaunchKernelGGL((route_topk_kernel<NV, false>), grid, block, lds, s, r, M, logits, ld, bias, ids, weights);
  return hipGetLastError();
}

template <int NV>
hipError_t launch_rows(const RouterArgs& r, int64_t M, const void* logits, bool bf16, int64_t ld, const float* bias,
                       int32_t* ids, float* weights, hipStream_t s) {
  const dim3 grid((unsigned)((M + 4 * kRowWaves - 1) / (4 * kRowWaves))), block(64 * kRowWaves);
  const size_t lds = r.groups > 1 ? sizeof(double) * (r.E + r.groups) * 4 * kRowWaves : 0;
  if (bf16)
    hipLaunchKernelGGL((route_rows_kernel<NV, true>), grid, block, lds, s, r, M, logits, ld, bias, ids, weights);
  else
    hipLaunchKernelGGL((route_rows_kernel<NV, false>), grid, block, lds, s, r, M, logits, ld, bias, ids, weights);
  return hipGetLastError();
}

template <int NV>
hipError_t launch_rows_backward(const RouterArgs& r, int64_t M, const void* logits, bool bf16, int64_t ld,
                                const float* bias, const int32_t* ids, const float* dw, void* dl, int64_t dl_ld,
                                hipStream_t s) {
  const dim3 grid((unsigned)((M + 4 * kRowWaves - 1) / (4 * kRowWaves))), block(64 * kRowWaves);
  if (bf16)
    hipLaunchKernelGGL((route_rows_backward_kernel<NV, true>), grid, block, 0, s, r, M, logits, ld, bias, ids, dw, dl,
                       dl_ld);
  else
    hipLaunchKernelGGL((route_rows_backward_kernel<NV, false>), grid, block, 0, s, r, M, logits, ld, bias, ids, dw,
                       dl, dl_ld);
  return hipGetLastError();
}

// Tokens of a launch: it takes fewer than 2^32 threads (HIP drops the rest of a
// larger grid without an error), up to 64 of them to a token.
constexpr int64_t kLaunchTokens = 1 << 25;

const void* token_rows(const void* p, bool bf16, int64_t elements) {
  return static_cast<const char*>(p) + elements * (bf16 ? 2 : 4);
}

// many: the call has enough tokens for 16 lanes each
hipError_t launch_forward(const RouterArgs& r, bool many, int64_t M, const void* logits, bool bf16, int64_t ld,
                          const float* bias, int32_t* ids, float* weights, hipStream_t s) {
  if (many && r.E <= kRowsForwardExperts && r.topk <= 16 && r.groups <= 16) {
    if (r.E <= 128) return launch_rows<8>(r, M, logits, bf16, ld, bias, ids, weights, s);
    return launch_rows<16>(r, M, logits, bf16, ld, bias, ids, weights, s);
  }
  if (r.E <= 64) return launch_topk<1>(r, M, logits, bf16, ld, bias, ids, weights, s);
  if (r.E <= 128) return launch_topk<2>(r, M, logits, bf16, ld, bias, ids, weights, s);
  if (r.E <= 256) return launch_topk<4>(r, M, logits, bf16, ld, bias, ids, weights, s);
  if (r.E <= 512) return launch_topk<8>(r, M, logits, bf16, ld, bias, ids, weights, s);
  return launch_topk<32>(r, M, logits, bf16, ld, bias, ids, weights, s);
}

hipError_t launch_backward(const RouterArgs& r, bool many, int64_t M, const void* logits, bool bf16, int64_t ld,
                           const float* bias, const int32_t* ids, const float* dw, void* dl, int64_t dl_ld,
                           hipStream_t s) {
  if (many && r.E <= kRowsBackwardExperts && r.topk <= 16) {
    if (r.E <= 128) return launch_rows_backward<8>(r, M, logits, bf16, ld, bias, ids, dw, dl, dl_ld, s);
    if (r.E <= 256) return launch_rows_backward<16>(r, M, logits, bf16, ld, bias, ids, dw, dl, dl_ld, s);
    return launch_rows_backward<32>(r, M, logits, bf16, ld, bias, ids, dw, dl, dl_ld, s);
  }
  const dim3 grid((unsigned)((M + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
  if (bf16)
    hipLaunchKernelGGL((route_topk_backward_kernel<true>), grid, block, 0, s, r, M, logits, ld, bias, ids, dw, dl,
                       dl_ld);
  else
    hipLaunchKernelGGL((route_topk_backward_kernel<false>), grid, block, 0, s, r, M, logits, ld, bias, ids, dw, dl,
                       dl_ld);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route_topk(const RouterArgs& r, int64_t M, const void* logits, bool bf16, int64_t ld,
                             const float* bias, int32_t* ids, float* weights, hipStream_t s) {
  const bool many = M >= (r.E <= 128 ? kRowsForwardTokens : kRowsForwardTokens256);
  hipError_t e = hipSuccess;
  for (int64_t t = 0; t < M && e == hipSuccess; t += kLaunchTokens)
    e = launch_forward(r, many, M - t < kLaunchTokens ? M - t : kLaunchTokens, token_rows(logits, bf16, t * ld),
                       bf16, ld, bias, ids + t * r.topk, weights + t * r.topk, s);
  return e;
}

hipError_t launch_route_topk_backward(const RouterArgs& r, int64_t M, const void* logits, bool bf16, int64_t ld,
                                      const float* bias, const int32_t* ids, const float* dw, void* dl,
                                      int64_t dl_ld, hipStream_t s) {
  const bool every = r.scoring == 0 && !r.renormalize && r.E > 128;
  const bool many = M >= (every ? kRowsBackwardTokensEvery : kRowsBackwardTokens);
  hipError_t e = hipSuccess;
  for (int64_t t = 0; t < M && e == hipSuccess; t += kLaunchTokens)
    e = launch_backward(r, many, M - t < kLaunchTokens ? M - t : kLaunchTokens,
                        token_rows(logits, bf16, t * ld), bf16, ld, bias, ids + t * r.topk, dw + t * r.topk,
                        const_cast<void*>(token_rows(dl, bf16, t * dl_ld)), dl_ld, s);
  return e;
}

}  // namespace moe

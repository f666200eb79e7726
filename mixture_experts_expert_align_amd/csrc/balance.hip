// The load balance of a router's choice: counts per expert, the balance loss
// of each packed sequence, and its gradient over the logits.
//
// With p_t the softmax of token t's logits (or its sigmoids over their sum),
// c_s,e the routes of sequence s to expert e and T_s its tokens:
//   loss_s = E / (topk T_s^2) sum_e c_s,e sum_t p_t,e
//   dl_t,e = dloss_s E / (topk T_s^2) p_t,e (c_s,e - sum_f c_s,f p_t,f)
// (sigmoid: times 1 - sigmoid(l_t,e), from p = s / sum s).  The scores add up to 1, so
// any number may be taken off all counts: the count of the token's best expert
// is (in integers), which keeps a confident token's gradient, a small
// difference of large counts, to float32 precision.
//
// The forward is two launches.  In the first a workgroup takes a chunk of
// consecutive tokens, LANES lanes a token, and writes for each sequence that
// it meets the sums of p, the routes and the tokens that count, into slot
// chunk + sequence (both only grow along the tokens, so every pair that meets
// has a slot of its own).  In the second a workgroup adds the slots of one
// sequence, kBalanceExperts experts of it, and the last of a sequence's
// workgroups the loss.  Floats are added in a fixed order, over a chunk's
// tokens in float32, over the chunks in float64.
#include "kernels.h"
#include "route_device.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr float kLog2e = 1.44269504088896341f;

// Maximum and sums over the token's LANES lanes, the same bits in each: every
// step adds two values that the two lanes hold in either order.
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __uint_as_float(dpp_u32<CTRL, 0xf>(__float_as_uint(v)));
}
template <int LANES, class F>
__device__ __forceinline__ float lanes_all(float v, F f) {
  static_assert(LANES == 16 || LANES == 64, "a row of 16 lanes, or the wave");
  v = f(v, dpp_f32<0x128>(v));   // rotations within the row by 8, 4, 2, 1
  v = f(v, dpp_f32<0x124>(v));
  v = f(v, dpp_f32<0x122>(v));
  v = f(v, dpp_f32<0x121>(v));
  if (LANES == 64) {
    v = f(v, __shfl_xor(v, 16));
    v = f(v, __shfl_xor(v, 32));
  }
  return v;
}
template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
  return lanes_all<LANES>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  return lanes_all<LANES>(v, [](float a, float b) { return a + b; });
}

// Logits of a token: expert c + LANES i in l[i]; -inf for one that cannot be chosen.
template <int LANES, int NV, bool BF16>
__device__ __forceinline__ void token_logits(const BalanceArgs& a, int64_t t, int c, float (&l)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = c + LANES * i;
    float v = -INFINITY;
    if (e < a.E) {
      v = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(a.logits)[t * a.ld + e])
               : static_cast<const float*>(a.logits)[t * a.ld + e];
      if (a.add_bias) v += a.bias[e];
    }
    l[i] = v > -INFINITY ? fmaxf(fminf(v, FLT_MAX), -FLT_MAX) : -INFINITY;
  }
}

// Scores: p[i] of l[i], 0 where it is -inf; returns the largest logit.  The
// sigmoids are taken times e^-min(top, 0), which their quotient does not see
// and which keeps them from all underflowing.
template <int LANES, int NV>
__device__ __forceinline__ float token_scores(bool sigmoid, const float (&l)[NV], float (&p)[NV]) {
  float top = l[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) top = fmaxf(top, l[i]);
  top = lanes_max<LANES>(top);
  const float shift = sigmoid ? fminf(top, 0.f) : top;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float v = 0.f;
    if (l[i] > -INFINITY) {
      if (!sigmoid)
        v = __builtin_amdgcn_exp2f((l[i] - shift) * kLog2e);
      else if (l[i] > 0.f)
        v = 1.0f / (1.0f + __builtin_amdgcn_exp2f(-l[i] * kLog2e));
      else
        v = __builtin_amdgcn_exp2f((l[i] - shift) * kLog2e) / (1.0f + __builtin_amdgcn_exp2f(l[i] * kLog2e));
    }
    p[i] = v;
    s += v;
  }
  s = lanes_sum<LANES>(s);
  const float inv = s > 0.f ? 1.0f / s : 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) p[i] *= inv;
  return top;
}

// Whether one of the token's ids names an expert; the same in all its lanes.
template <int LANES>
__device__ __forceinline__ bool token_counts(const BalanceArgs& a, int64_t t, int c) {
  float any = 0.f;
  for (int j = c; j < a.topk; j += LANES) {
    const int id = a.ids[t * a.topk + j];
    if (id >= 0 && id < a.E) any = 1.f;
  }
  return lanes_max<LANES>(any) > 0.f;
}

// Offset i of the sequences, within [0, M] whatever the array holds.
__device__ __forceinline__ int64_t seq_offset(const BalanceArgs& a, int i) {
  if (!a.offsets) return i == 0 ? 0 : a.M;
  return min(max((int64_t)a.offsets[i], (int64_t)0), a.M);
}

// The last sequence that starts at or before token t, or -1: the one t is in,
// if it is in any.
__device__ __forceinline__ int seq_of(const BalanceArgs& a, int64_t t) {
  int lo = -1, hi = a.S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seq_offset(a, mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <int LANES, int NV, bool BF16>
__global__ void __launch_bounds__(kThreads) balance_tokens_kernel(BalanceArgs a) {
  constexpr int TOK = kThreads / LANES;          // tokens at a time
  __shared__ float s_p[kWaves][LANES * NV];
  __shared__ int s_c[LANES * NV];
  __shared__ int s_t;
  const int tid = threadIdx.x, c = tid % LANES, wave = tid >> 6;
  const int64_t first = (int64_t)blockIdx.x * a.chunk;
  const int64_t last = min(first + a.chunk, a.M);
  if (blockIdx.x == 0)
    for (int s = tid; s < a.S; s += kThreads) a.done[s] = 0;
  for (int64_t at = first; at < last;) {
    const int s = seq_of(a, at);
    if (s < 0) {                                 // before the first sequence
      at = min(max(seq_offset(a, 0), at + 1), last);
      continue;
    }
    const int64_t end = min(seq_offset(a, s + 1), last);
    if (end <= at) break;                        // behind the last sequence
    for (int e = tid; e < LANES * NV; e += kThreads) s_c[e] = 0;
    if (tid == 0) s_t = 0;
    __syncthreads();
    float acc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] = 0.f;
    int n = 0;
    for (int64_t t0 = at; t0 < end; t0 += TOK) {
      const int64_t t = t0 + tid / LANES;
      const int64_t in = min(t, end - 1);        // past the last token: that one again, not counted
      float l[NV], p[NV];
      token_logits<LANES, NV, BF16>(a, in, c, l);
      token_scores<LANES, NV>(a.sigmoid, l, p);
      bool any = false;
      for (int j = c; j < a.topk; j += LANES) {
        const int id = a.ids[in * a.topk + j];
        if (id >= 0 && id < a.E) {
          any = true;
          if (t < end) atomicAdd(&s_c[id], 1);
        }
      }
      const bool on = t < end && lanes_max<LANES>(any ? 1.f : 0.f) > 0.f;
      n += on;
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] += on ? p[i] : 0.f;
    }
    if (LANES == 16) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        acc[i] += __shfl_xor(acc[i], 16);
        acc[i] += __shfl_xor(acc[i], 32);
      }
    }
    if ((tid & 63) < LANES) {
#pragma unroll
      for (int i = 0; i < NV; ++i) s_p[wave][c + LANES * i] = acc[i];
    }
    if (c == 0) atomicAdd(&s_t, n);
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + s;
    for (int e = tid; e < a.E; e += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += s_p[w][e];
      a.psum[slot * a.E + e] = v;
      a.csum[slot * a.E + e] = s_c[e];
    }
    if (tid == 0) a.tsum[slot] = s_t;
    __syncthreads();
    at = end;
  }
}

// Workgroup (sequence, block of its experts): the waves share the sequence's slots.
constexpr int kSumWaves = 16;

__global__ void __launch_bounds__(64 * kSumWaves) balance_sums_kernel(BalanceArgs a) {
  __shared__ double s_p[kSumWaves][kBalanceExperts];
  __shared__ int s_c[kSumWaves][kBalanceExperts];
  __shared__ int s_t[kSumWaves];
  const int nb = (a.E + kBalanceExperts - 1) / kBalanceExperts;
  const int s = blockIdx.x / nb, b = blockIdx.x % nb;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = b * kBalanceExperts + lane;
  const int64_t lo = seq_offset(a, s), hi = seq_offset(a, s + 1);
  double p = 0.0;
  int c = 0, t = 0;
  if (lo < hi) {
    const int64_t i1 = (hi - 1) / a.chunk;
    for (int64_t i = lo / a.chunk + wave; i <= i1; i += kSumWaves) {
      const int64_t slot = i + s;
      if (e < a.E) {
        p += (double)a.psum[slot * a.E + e];
        c += a.csum[slot * a.E + e];
      }
      t += a.tsum[slot];
    }
  }
  s_p[wave][lane] = p;
  s_c[wave][lane] = c;
  if (lane == 0) s_t[wave] = t;
  __syncthreads();
  if (wave != 0) return;
  p = 0.0, c = 0, t = 0;
  for (int w = 0; w < kSumWaves; ++w) {
    p += s_p[w][lane];
    c += s_c[w][lane];
    t += s_t[w];
  }
  const double mean = t > 0 ? p / t : 0.0;
  if (e < a.E) {
    a.counts[(int64_t)s * a.E + e] = c;
    a.probs[(int64_t)s * a.E + e] = (float)mean;
  }
  if (b == 0 && lane == 0) a.tokens[s] = t;
  const double part = wave_sum_f64(e < a.E ? mean * c : 0.0);
  const double scale = t > 0 ? (double)a.E / ((double)a.topk * t) : 0.0;
  if (nb == 1) {
    if (lane == 0) a.loss[s] = (float)(part * scale);
    return;
  }
  // the last of the sequence's workgroups adds their parts, in their order
  if (lane == 0) {
    __hip_atomic_store(a.lpart + (int64_t)s * nb + b, part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__hip_atomic_fetch_add(a.done + s, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == nb - 1) {
      double sum = 0.0;
      for (int i = 0; i < nb; ++i)
        sum += __hip_atomic_load(a.lpart + (int64_t)s * nb + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      a.loss[s] = (float)(sum * scale);
    }
  }
}

template <int LANES, int NV, bool BF16>
__global__ void __launch_bounds__(kThreads) balance_backward_kernel(BalanceArgs a) {
  constexpr int TOK = kThreads / LANES;
  const int c = threadIdx.x % LANES;
  const int64_t t = a.t0 + (int64_t)blockIdx.x * TOK + threadIdx.x / LANES;
  const int64_t in = min(t, a.M - 1);            // past the last token: that one again, not stored
  const int s = seq_of(a, in);
  const bool on = token_counts<LANES>(a, in, c) && s >= 0 && in < seq_offset(a, s + 1);
  if (a.accumulate && !on) return;               // (no barrier below)
  float d[NV];
  if (on) {
    float l[NV], p[NV];
    token_logits<LANES, NV, BF16>(a, in, c, l);
    const float top = token_scores<LANES, NV>(a.sigmoid, l, p);
    const int32_t* cnt = a.counts_in + (int64_t)s * a.E;
    int ci[NV];
    float best = -1.f;                           // the position of the best expert
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = c + LANES * i;
      ci[i] = e < a.E ? cnt[e] : 0;
      if (l[i] == top) best = (float)e;
    }
    best = lanes_max<LANES>(best);
    const int ref = best >= 0.f && best < (float)a.E ? cnt[(int)best] : 0;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      d[i] = (float)(ci[i] - ref);
      dot += p[i] * d[i];
    }
    dot = lanes_sum<LANES>(dot);
    const double T = a.tokens_in[s];
    const float k = T > 0 ? (float)((double)a.dloss[s] * a.E / ((double)a.topk * T * T)) : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      d[i] = l[i] > -INFINITY ? k * (p[i] * (d[i] - dot)) : 0.f;
      if (a.sigmoid && l[i] > -INFINITY) d[i] /= 1.0f + __builtin_amdgcn_exp2f(l[i] * kLog2e);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) d[i] = 0.f;
  }
  if (t >= a.M) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = c + LANES * i;
    if (e >= a.E) continue;
    if (BF16) {
      uint16_t* o = static_cast<uint16_t*>(a.dlogits) + t * a.dld + e;
      *o = (uint16_t)f32_to_bf16_rne(a.accumulate ? bf16_to_f32(*o) + d[i] : d[i]);
    } else {
      float* o = static_cast<float*>(a.dlogits) + t * a.dld + e;
      *o = a.accumulate ? *o + d[i] : d[i];
    }
  }
}

template <int LANES, int NV>
hipError_t launch_tokens(const BalanceArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.nchunk > 0 ? a.nchunk : 1)), block(kThreads);
  if (a.bf16)
    hipLaunchKernelGGL((balance_tokens_kernel<LANES, NV, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((balance_tokens_kernel<LANES, NV, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

// Tokens of a launch: it takes fewer than 2^32 threads, up to 64 to a token.
constexpr int64_t kLaunchTokens = 1 << 25;

template <int LANES, int NV>
hipError_t launch_backward(BalanceArgs a, hipStream_t s) {
  constexpr int TOK = kThreads / LANES;
  hipError_t e = hipSuccess;
  for (a.t0 = 0; a.t0 < a.M && e == hipSuccess; a.t0 += kLaunchTokens) {
    const int64_t n = a.M - a.t0 < kLaunchTokens ? a.M - a.t0 : kLaunchTokens;
    const dim3 grid((unsigned)((n + TOK - 1) / TOK)), block(kThreads);
    if (a.bf16)
      hipLaunchKernelGGL((balance_backward_kernel<LANES, NV, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((balance_backward_kernel<LANES, NV, false>), grid, block, 0, s, a);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

// Tokens of a workgroup of the first launch: at most 512 workgroups.
int32_t balance_chunk(int64_t M) {
  const int64_t c = ((M + 511) / 512 + 15) / 16 * 16;
  return (int32_t)(c < 32 ? 32 : c);
}

hipError_t launch_balance(const BalanceArgs& a, hipStream_t s) {
  hipError_t e;
  if (a.E <= 16) e = launch_tokens<16, 1>(a, s);
  else if (a.E <= 64) e = launch_tokens<16, 4>(a, s);
  else if (a.E <= 128) e = launch_tokens<16, 8>(a, s);
  else if (a.E <= 256) e = launch_tokens<64, 4>(a, s);
  else if (a.E <= 512) e = launch_tokens<64, 8>(a, s);
  else e = launch_tokens<64, 32>(a, s);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((a.E + kBalanceExperts - 1) / kBalanceExperts * a.S));
  hipLaunchKernelGGL(balance_sums_kernel, grid, dim3(64 * kSumWaves), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceArgs& a, hipStream_t s) {
  if (a.E <= 16) return launch_backward<16, 1>(a, s);
  if (a.E <= 64) return launch_backward<16, 4>(a, s);
  if (a.E <= 128) return launch_backward<16, 8>(a, s);
  if (a.E <= 256) return launch_backward<64, 4>(a, s);
  if (a.E <= 512) return launch_backward<64, 8>(a, s);
  return launch_backward<64, 32>(a, s);
}

}  // namespace moe

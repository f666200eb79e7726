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
// has a slot of its own).  (Few tokens: one workgroup, which finishes the
// sequences itself.)  In the second a workgroup adds the slots of one
// sequence, kBalanceExperts experts of it, and the last of a sequence's
// workgroups the loss.  Floats are added in a fixed order, over a chunk's
// tokens in float32, over the chunks in float64.
//
// Bound by latency more than by bytes: 65536 x 256 bf16 is 36 MB, read in 14 us
// (2.5 TB/s), and 8 us of sums; 16381 x 512 (sigmoid, 13 sequences) takes 14 and 9
// us and its gradient, 34 MB, 14; 8192 x 128 float32 5, 6 and 5 us.
#include "kernels.h"
#include "lanes.h"
#include "route_device.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr float kLog2e = 1.44269504088896341f;

// A token's E values over LANES lanes: lane c holds VEC consecutive experts
// from VEC (c + LANES i) on, NV values in all, loaded VEC at a time.
template <int LANES_, int NV_, int VEC_, bool BF16_>
struct Shape {
  static constexpr int LANES = LANES_, NV = NV_, VEC = VEC_, NI = NV / VEC;
  static constexpr bool BF16 = BF16_;
  static constexpr int EL = BF16 ? 2 : 4, W = VEC * EL >= 4 ? VEC * EL / 4 : 1;   // words of a load
  static_assert(NI * VEC == NV, "whole loads");
  static __device__ __forceinline__ int expert(int c, int i) { return VEC * (c + LANES * i); }
};

template <class S>
struct Raw {
  uint32_t w[S::NI][S::W];
  __device__ __forceinline__ void clear() {   // -inf: what lies past E
#pragma unroll
    for (int i = 0; i < S::NI; ++i)
#pragma unroll
      for (int k = 0; k < S::W; ++k) w[i][k] = S::BF16 ? 0xff80ff80u : 0xff800000u;
  }
  __device__ __forceinline__ void load(const void* row, int E, int c) {
    const char* p = static_cast<const char*>(row);
#pragma unroll
    for (int i = 0; i < S::NI; ++i) {
      const int e = S::expert(c, i);
      if (e < E) {
        if constexpr (S::VEC * S::EL == 2) w[i][0] = *reinterpret_cast<const uint16_t*>(p + 2 * e);
        else __builtin_memcpy(w[i], __builtin_assume_aligned(p + (int64_t)S::EL * e, 4 * S::W), 4 * S::W);
      }
    }
  }
  // value k of load i
  __device__ __forceinline__ float get(int i, int k) const {
    if constexpr (!S::BF16) return __uint_as_float(w[i][k]);
    return __uint_as_float(k & 1 ? w[i][k / 2] & 0xffff0000u : w[i][k / 2] << 16);
  }
};

// The token's logits (plus a bias, LDS), its scores before their division by the
// returned sum, and the largest logit.  Nothing is done about special values
// until they show: with a NaN, a +inf or no expert at all the sum is not a
// positive number, past 2^29 the products with log2(e) are off by more than
// exponentials hold, and a sigmoid's whole row may underflow where none is
// positive; then, and only then, the row is taken again with the logits that
// compete (-inf for one that cannot be chosen, +inf as the largest float32) and
// sigmoids times e^-min(top, 0), which their quotient does not see.
// REST: also 1 - sigmoid in q, without cancellation (1 without sigmoids).
template <class S, bool REST>
__device__ __forceinline__ float token_scores(const Raw<S>& r, int c, bool add, const float* bias, bool sigmoid,
                                              float (&l)[S::NV], float (&p)[S::NV], float (&q)[REST ? S::NV : 1],
                                              float& top) {
  top = -INFINITY;
#pragma unroll
  for (int i = 0; i < S::NI; ++i)
#pragma unroll
    for (int k = 0; k < S::VEC; ++k) l[S::VEC * i + k] = r.get(i, k);
  if (add) {
#pragma unroll
    for (int i = 0; i < S::NI; ++i)
#pragma unroll
      for (int k = 0; k < S::VEC; ++k) l[S::VEC * i + k] += bias[S::expert(c, i) + k];
  }
#pragma unroll
  for (int i = 0; i < S::NV; ++i) top = fmaxf(top, l[i]);
  top = lanes_max<S::LANES>(top);
  float s = 0.f;
  if (!sigmoid) {
    // one fused operation: the rounding of top log2(e) is common to the row, and
    // the quotient does not see it
    const float m = -top * kLog2e;
#pragma unroll
    for (int i = 0; i < S::NV; ++i) {
      p[i] = __builtin_amdgcn_exp2f(fmaf(l[i], kLog2e, m));
      s += p[i];
      if (REST) q[REST ? i : 0] = 1.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < S::NV; ++i) {
      // 1 / (1 + e^-l), or e^l / (1 + e^l) below 0: no overflow in either
      const float e = __builtin_amdgcn_exp2f(-fabsf(l[i]) * kLog2e);
      const float d = __builtin_amdgcn_rcpf(1.0f + e);
      p[i] = (l[i] > 0.f ? 1.0f : e) * d;
      if (REST) q[REST ? i : 0] = (l[i] > 0.f ? e : 1.0f) * d;
      s += p[i];
    }
  }
  s = lanes_sum<S::LANES>(s);
  // (decided by the token, not by its wave: its bits are its own.  Under 2^29 the
  // rounding of top log2(e) is 2^5 at most, so the sum lies between 2^-32 and 2^43 and
  // has a reciprocal; at 2 10^9 it reached 2^127, whose reciprocal is subnormal, taken as 0)
  if (s > 0.f && s < INFINITY && fabsf(top) < 0x1p29f && (!sigmoid || top > 0.f)) return s;
  top = -INFINITY;
#pragma unroll
  for (int i = 0; i < S::NV; ++i) {
    l[i] = l[i] > -INFINITY ? fmaxf(fminf(l[i], FLT_MAX), -FLT_MAX) : -INFINITY;
    top = fmaxf(top, l[i]);
  }
  top = lanes_max<S::LANES>(top);
  const float shift = top == -INFINITY ? 0.f : sigmoid ? fminf(top, 0.f) : top;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < S::NV; ++i) {
    p[i] = __builtin_amdgcn_exp2f((l[i] - shift) * kLog2e);   // (0 for -inf)
    if (sigmoid) {
      const float e = __builtin_amdgcn_exp2f(-fabsf(l[i]) * kLog2e), d = __builtin_amdgcn_rcpf(1.0f + e);
      p[i] = (l[i] > 0.f ? 1.0f : p[i]) * d;
      if (REST) q[REST ? i : 0] = (l[i] > 0.f ? e : 1.0f) * d;
    }
    s += p[i];
  }
  return lanes_sum<S::LANES>(s);
}

// Offset i of the sequences, within [0, M] whatever the array holds.
__device__ __forceinline__ int64_t seq_offset(const BalanceArgs& a, int i) {
  if (!a.offsets) return i == 0 ? 0 : a.M;
  return min(max((int64_t)a.offsets[i], (int64_t)0), a.M);
}

// The last sequence that starts at or before token t, or -1: the one t is in,
// if it is in any.  64 of the sequences are looked at together; t is the same
// in all lanes, which are all here.
__device__ __forceinline__ int seq_of(const BalanceArgs& a, int64_t t) {
  int lo = -1, n = a.S;                          // it is lo or one of the n behind it
  while (n > 0) {
    const int step = (n + 63) / 64, i = step * (int)__lane_id();
    const int c = __popcll(__ballot(i < n && seq_offset(a, min(lo + 1 + i, a.S)) <= t));
    if (c == 0) break;
    lo += 1 + step * (c - 1);
    n = min(step - 1, n - 1 - step * (c - 1));
  }
  return lo;
}

template <class S>
__device__ __forceinline__ const void* token_row(const BalanceArgs& a, int64_t t) {
  return static_cast<const char*>(a.logits) + t * a.ld * S::EL;
}

template <class S>
__global__ void __launch_bounds__(kThreads) balance_tokens_kernel(BalanceArgs a) {
  constexpr int LANES = S::LANES, NE = LANES * S::NV;
  constexpr int TOK = kThreads / LANES;          // tokens at a time
  __shared__ float s_p[kWaves][NE];
  __shared__ float s_b[NE];
  __shared__ int s_c[NE];
  __shared__ int s_t;
  __shared__ double s_l[kWaves];
  const int tid = threadIdx.x, c = tid % LANES, wave = tid >> 6;
  const int64_t first = (int64_t)blockIdx.x * a.chunk;
  const int last = (int)min((int64_t)a.chunk, a.M - first);   // tokens, counted from the chunk's first below
  if (a.one) {                                   // there is no second launch; sequences without tokens
    for (int64_t i = tid; i < (int64_t)a.S * a.E; i += kThreads) {
      a.counts[i] = 0;
      a.probs[i] = 0.f;
    }
    for (int s = tid; s < a.S; s += kThreads) {
      a.loss[s] = 0.f;
      a.tokens[s] = 0;
    }
  } else if (blockIdx.x == 0) {
    for (int s = tid; s < a.S; s += kThreads) a.done[s] = 0;
  }
  for (int e = tid; e < NE; e += kThreads) s_b[e] = a.add_bias && e < a.E ? a.bias[e] : 0.f;
  // logits and first ids of the tokens t0 .. t0 + TOK - 1 (past the last token:
  // that one again, not counted), requested before the sequences are looked up
  Raw<S> raw;
  raw.clear();
  int id = -1;
  auto load = [&](int t0) {
    const int64_t in = first + min(t0 + tid / LANES, last - 1);
    raw.load(token_row<S>(a, in), a.E, c);
    if (c < a.topk) id = a.ids[in * a.topk + c];
  };
  if (last <= 0) return;                         // no tokens at all
  load(0);
  // the sequence at hand, its tokens [from, to) up to the chunk's end; between
  // sequences from is the chunk's end
  int s;
  int from, to;
  auto in_chunk = [&](int64_t t) { return (int)min(max(t - first, (int64_t)-1), (int64_t)last); };
  auto enter = [&](int at) {
    s = seq_of(a, first + at);
    from = s < 0 ? last : in_chunk(seq_offset(a, s));
    to = in_chunk(s < 0 ? seq_offset(a, 0) : seq_offset(a, s + 1));
    if (to <= at) {                              // behind the last sequence, or offsets in no order
      to = s < 0 ? at + 1 : last;
      from = last;
    }
  };
  enter(0);
  float acc[S::NV];
  int n = 0;
  auto clear = [&]() {
    for (int e = tid; e < NE; e += kThreads) s_c[e] = 0;
    if (tid == 0) s_t = 0;
#pragma unroll
    for (int i = 0; i < S::NV; ++i) acc[i] = 0.f;
    n = 0;
    __syncthreads();
  };
  auto flush = [&]() {
    if (LANES == 16) {
#pragma unroll
      for (int i = 0; i < S::NV; ++i) {
        acc[i] += __shfl_xor(acc[i], 16);
        acc[i] += __shfl_xor(acc[i], 32);
      }
    }
    if ((tid & 63) < LANES) {
#pragma unroll
      for (int i = 0; i < S::NI; ++i)
#pragma unroll
        for (int k = 0; k < S::VEC; ++k) s_p[wave][S::expert(c, i) + k] = acc[S::VEC * i + k];
    }
    if (c == 0) atomicAdd(&s_t, n);
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + s;
    double loss = 0.0;
    const int T = s_t;
    for (int e = tid; e < a.E; e += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += s_p[w][e];
      if (!a.one) {
        a.part[slot * a.E + e] = make_int2((int)__float_as_uint(v), s_c[e]);
      } else if (T > 0) {
        const double mean = (double)v / T;
        a.counts[(int64_t)s * a.E + e] = s_c[e];
        a.probs[(int64_t)s * a.E + e] = (float)mean;
        loss += mean * s_c[e];
      }
    }
    if (a.one) {
      loss = wave_sum_f64(loss);
      if ((tid & 63) == 0) s_l[wave] = loss;
      __syncthreads();
      if (tid == 0 && T > 0) {
        for (int w = 1; w < kWaves; ++w) loss += s_l[w];
        a.tokens[s] = T;
        a.loss[s] = (float)(loss * ((double)a.E / ((double)a.topk * T)));
      }
    } else if (tid == 0) {
      a.tsum[slot] = T;
    }
    __syncthreads();
  };
  clear();
  for (int t0 = 0; t0 < last; t0 += TOK) {
    const int t = t0 + tid / LANES, next = min(t0 + TOK, last);
    const Raw<S> now = raw;
    const int now_id = id;
    if (next < last) load(next);
    float l[S::NV], p[S::NV], q[1], top;
    const float sum = token_scores<S, false>(now, c, a.add_bias, s_b, a.sigmoid, l, p, q, top);
    const float inv = sum > 0.f ? __builtin_amdgcn_rcpf(sum) : 0.f;
    for (;;) {
      // the tokens of this group that are in the sequence
      const bool in = t >= from && t < to;
      bool any = in && now_id >= 0 && now_id < a.E;
      if (any) atomicAdd(&s_c[now_id], 1);
      if (in)
        for (int j = c + LANES; j < a.topk; j += LANES) {
          const int more = a.ids[(first + t) * a.topk + j];
          if (more >= 0 && more < a.E) {
            any = true;
            atomicAdd(&s_c[more], 1);
          }
        }
      const bool on = lanes_max<LANES>(any ? 1 : 0) != 0;
      n += on;
      const float f = on ? inv : 0.f;
#pragma unroll
      for (int i = 0; i < S::NV; ++i) acc[i] += p[i] * f;
      if (to > next || to == last) break;        // goes on in the next group, or the chunk ends
      const bool some = from < to, group = to < next;
      if (some) flush();
      enter(to);
      if (some) clear();
      if (!group) break;
    }
  }
  if (from < to) flush();
}

// Workgroup (sequence, block of its experts): 16 experts a row of lanes, the
// rows of all waves sharing the sequence's slots.
constexpr int kSumWaves = 16;

__global__ void __launch_bounds__(64 * kSumWaves) balance_sums_kernel(BalanceArgs a) {
  constexpr int kSumRows = 4 * kSumWaves;
  static_assert(kBalanceExperts == 16, "a row of lanes");
  __shared__ double s_p[kSumRows][kBalanceExperts];
  __shared__ int s_c[kSumRows][kBalanceExperts];
  __shared__ int s_t[kSumWaves];
  const int nb = (a.E + kBalanceExperts - 1) / kBalanceExperts;
  const int s = a.s0 + (int)(blockIdx.x / nb), b = blockIdx.x % nb;
  const int col = threadIdx.x % kBalanceExperts, row = threadIdx.x / kBalanceExperts;
  const int e = b * kBalanceExperts + col;
  const int64_t lo = seq_offset(a, s), hi = seq_offset(a, s + 1);
  double p = 0.0;
  int c = 0, t = 0;
  if (lo < hi) {
    const int64_t i0 = lo / a.chunk, i1 = (hi - 1) / a.chunk;
    if (e < a.E) {
#pragma unroll 8
      for (int64_t i = i0 + row; i <= i1; i += kSumRows) {
        const int2 v = a.part[(i + s) * a.E + e];
        p += (double)__uint_as_float((uint32_t)v.x);
        c += v.y;
      }
    }
    for (int64_t i = i0 + threadIdx.x; i <= i1; i += 64 * kSumWaves) t += a.tsum[i + s];
  }
  for (int d = 32; d; d >>= 1) t += __shfl_xor(t, d);
  s_p[row][col] = p;
  s_c[row][col] = c;
  if ((threadIdx.x & 63) == 0) s_t[threadIdx.x >> 6] = t;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  // lane (row, col): a quarter of the rows, then their sum
  p = 0.0, c = 0, t = 0;
#pragma unroll
  for (int w = 0; w < kSumRows / 4; ++w) {
    p += s_p[w * 4 + row][col];
    c += s_c[w * 4 + row][col];
  }
#pragma unroll
  for (int d = 16; d < 64; d *= 2) {
    p += __shfl_xor(p, d);
    c += __shfl_xor(c, d);
  }
#pragma unroll
  for (int w = 0; w < kSumWaves; ++w) t += s_t[w];
  const double mean = t > 0 ? p / t : 0.0;
  const bool mine = row == 0 && e < a.E;
  if (mine) {
    a.counts[(int64_t)s * a.E + e] = c;
    a.probs[(int64_t)s * a.E + e] = (float)mean;
  }
  if (b == 0 && threadIdx.x == 0) a.tokens[s] = t;
  const double part = wave_sum_f64(mine ? mean * c : 0.0);
  const double scale = t > 0 ? (double)a.E / ((double)a.topk * t) : 0.0;
  if (nb == 1) {
    if (threadIdx.x == 0) a.loss[s] = (float)(part * scale);
    return;
  }
  // the last of the sequence's workgroups adds their parts, in a fixed order; each
  // part is where all can read it before its workgroup is counted
  int done = 0;
  double* parts = a.lpart + (int64_t)s * nb;
  if (threadIdx.x == 0) {
    __hip_atomic_store(parts + b, part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    wait_vm<0>();
    done = __hip_atomic_fetch_add(a.done + s, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (__builtin_amdgcn_readfirstlane(done) != nb - 1) return;
  double sum = 0.0;
  for (int i = threadIdx.x; i < nb; i += 64)
    sum += __hip_atomic_load(parts + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  sum = wave_sum_f64(sum);
  if (threadIdx.x == 0) a.loss[s] = (float)(sum * scale);
}

template <class S>
__global__ void __launch_bounds__(kThreads) balance_backward_kernel(BalanceArgs a) {
  constexpr int LANES = S::LANES, TOK = kThreads / LANES, NE = LANES * S::NV;
  __shared__ float s_b[NE];
  const int c = threadIdx.x % LANES;
  const int64_t first = a.t0 + (int64_t)blockIdx.x * TOK;
  const int64_t t = first + threadIdx.x / LANES;
  const int64_t in = min(t, a.M - 1);            // past the last token: that one again, not stored
  Raw<S> raw;
  raw.clear();
  raw.load(token_row<S>(a, in), a.E, c);
  bool any = false;
  for (int j = c; j < a.topk; j += LANES) {
    const int id = a.ids[in * a.topk + j];
    any |= id >= 0 && id < a.E;
  }
  if (a.add_bias) {
    for (int e = threadIdx.x; e < NE; e += kThreads) s_b[e] = e < a.E ? a.bias[e] : 0.f;
    __syncthreads();
  }
  // the first token's sequence (-1: it lies before them all), or one of the next few, or
  // that of a search by itself
  int s = seq_of(a, min(first, a.M - 1));
  if (LANES < 64 && a.offsets) {
    int k = 0;
    while (k < 4 && s + 1 < a.S && seq_offset(a, s + 1) <= in) ++s, ++k;
    if (k == 4) {
      int lo = s, hi = a.S - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (seq_offset(a, mid) <= in) lo = mid; else hi = mid - 1;
      }
      s = lo;
    }
  } else if (a.offsets) {
    s = seq_of(a, in);
  }
  const bool on = lanes_max<LANES>(any ? 1 : 0) != 0 && s >= 0 && in < seq_offset(a, s + 1);
  if (t >= a.M || (a.accumulate && !on)) return;   // whole tokens; no barrier below
  float d[S::NV];
  if (on) {
    const int32_t* cnt = a.counts_in + (int64_t)s * a.E;
    int ci[S::NV];
#pragma unroll
    for (int i = 0; i < S::NI; ++i) {
      constexpr int B = S::VEC >= 4 ? 16 : 4;   // by_alignment has seen to it
#pragma unroll
      for (int k = 0; k < S::VEC; ++k) ci[S::VEC * i + k] = 0;
      if (S::expert(c, i) < a.E)
        __builtin_memcpy(ci + S::VEC * i, __builtin_assume_aligned(cnt + S::expert(c, i), B), 4 * S::VEC);
    }
    const double T = a.tokens_in[s];
    const float k = T > 0 ? (float)((double)a.dloss[s] * a.E / ((double)a.topk * T * T)) : 0.f;
    float l[S::NV], p[S::NV], q[S::NV], top;
    const float sum = token_scores<S, true>(raw, c, a.add_bias, s_b, a.sigmoid, l, p, q, top);
    const float inv = sum > 0.f ? __builtin_amdgcn_rcpf(sum) : 0.f;
    int ref = -1;                                // the best expert's count (of several, the largest)
#pragma unroll
    for (int i = 0; i < S::NV; ++i) ref = max(ref, l[i] == top ? ci[i] : -1);
    ref = lanes_max<LANES>(ref);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < S::NV; ++i) {
      p[i] *= inv;
      d[i] = (float)(ci[i] - ref);
      dot += p[i] * d[i];
    }
    dot = lanes_sum<LANES>(dot);
#pragma unroll
    for (int i = 0; i < S::NV; ++i) {
      d[i] = k * (p[i] * (d[i] - dot));   // p is 0 where l is -inf
      if (a.sigmoid) d[i] *= q[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < S::NV; ++i) d[i] = 0.f;
  }
  char* out = static_cast<char*>(a.dlogits) + t * a.dld * S::EL;
#pragma unroll
  for (int i = 0; i < S::NI; ++i) {
    const int e = S::expert(c, i);
    if (e >= a.E) continue;
    char* o = out + (int64_t)S::EL * e;
    uint32_t w[S::W];
    if (a.accumulate) {
      if constexpr (S::VEC * S::EL == 2) w[0] = *reinterpret_cast<uint16_t*>(o);
      else __builtin_memcpy(w, __builtin_assume_aligned(o, 4 * S::W), 4 * S::W);
#pragma unroll
      for (int k = 0; k < S::VEC; ++k) {
        const uint32_t u = S::BF16 ? (k & 1 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16) : w[k];
        d[S::VEC * i + k] += __uint_as_float(u);
      }
    }
    if constexpr (!S::BF16) {
#pragma unroll
      for (int k = 0; k < S::VEC; ++k) w[k] = __float_as_uint(d[S::VEC * i + k]);
    } else if constexpr (S::VEC == 1) {
      w[0] = bf16_pack2(d[i], 0.f);
    } else {
#pragma unroll
      for (int k = 0; k < S::VEC / 2; ++k) w[k] = bf16_pack2(d[S::VEC * i + 2 * k], d[S::VEC * i + 2 * k + 1]);
    }
    if constexpr (S::VEC * S::EL == 2) *reinterpret_cast<uint16_t*>(o) = (uint16_t)w[0];
    else __builtin_memcpy(__builtin_assume_aligned(o, 4 * S::W), w, 4 * S::W);
  }
}

struct Forward {
  template <class S>
  static hipError_t go(const BalanceArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(balance_tokens_kernel<S>, dim3((unsigned)(a.nchunk > 0 ? a.nchunk : 1)), dim3(kThreads), 0, s,
                       a);
    return hipGetLastError();
  }
};

// Tokens of a launch: it takes fewer than 2^32 threads, up to 64 to a token.
constexpr int64_t kLaunchTokens = 1 << 25;

struct Backward {
  template <class S>
  static hipError_t go(BalanceArgs a, hipStream_t s) {
    constexpr int TOK = kThreads / S::LANES;
    hipError_t e = hipSuccess;
    for (a.t0 = 0; a.t0 < a.M && e == hipSuccess; a.t0 += kLaunchTokens) {
      const int64_t n = a.M - a.t0 < kLaunchTokens ? a.M - a.t0 : kLaunchTokens;
      hipLaunchKernelGGL(balance_backward_kernel<S>, dim3((unsigned)((n + TOK - 1) / TOK)), dim3(kThreads), 0, s, a);
      e = hipGetLastError();
    }
    return e;
  }
};

// VEC values of EL bytes a load where every row allows it.
template <class L, int LANES, int NV, int VEC, bool BF16>
hipError_t by_alignment(const BalanceArgs& a, hipStream_t s) {
  if constexpr (VEC > 1) {
    constexpr uintptr_t B = VEC * (BF16 ? 2 : 4);
    const bool ok = a.E % VEC == 0 && a.ld % VEC == 0 && a.dld % VEC == 0 && (uintptr_t)a.logits % B == 0 &&
                    (uintptr_t)a.dlogits % B == 0 && (VEC < 4 || (uintptr_t)a.counts_in % 16 == 0);
    if (ok) return L::template go<Shape<LANES, NV, VEC, BF16>>(a, s);
  }
  return L::template go<Shape<LANES, NV, 1, BF16>>(a, s);
}

template <class L, int LANES, int NV>
hipError_t by_type(const BalanceArgs& a, hipStream_t s) {
  return a.bf16 ? by_alignment<L, LANES, NV, (NV < 8 ? NV : 8), true>(a, s)
                : by_alignment<L, LANES, NV, (NV < 4 ? NV : 4), false>(a, s);
}

// 16 lanes a token for up to 512 experts, a wave for more.  (At 512 experts in bf16, 16
// lanes and a wave of 8 values a lane, from a graph: 65536 tokens 25.0 and 35.1 us, their
// gradient 31.6 and 36.4; 16381 tokens 20.8 and 20.4, 12.3 and 13.2; 4096 tokens 11.9 and
// 11.9, 5.2 and 4.9.)
template <class L>
hipError_t by_experts(const BalanceArgs& a, hipStream_t s) {
  if (a.E <= 16) return by_type<L, 16, 1>(a, s);
  if (a.E <= 64) return by_type<L, 16, 4>(a, s);
  if (a.E <= 128) return by_type<L, 16, 8>(a, s);
  if (a.E <= 256) return by_type<L, 16, 16>(a, s);
  if (a.E <= 512) return by_type<L, 16, 32>(a, s);
  return by_type<L, 64, 32>(a, s);
}

}  // namespace

// Tokens of a workgroup of the first launch: at most 512 workgroups, whose parts
// the second has to add (65536 x 256, both launches: 512 workgroups 20.6 us, 1024
// 21.5, 2048 26.2), of 16 tokens at least (8192 x 128: 10.9 us, of 32 12.1), and of
// 4096 at most, whatever their number, since a chunk is summed in float32.
// Up to four rounds of a workgroup's tokens are left to one workgroup (64 x 8,
// loss and gradient, host included: 16.8 us, in two launches 19.5).
static int64_t one_workgroup(int64_t E) { return 4 * (kThreads / (E <= 512 ? 16 : 64)); }

int32_t balance_chunk(int64_t M, int64_t E) {
  if (M <= one_workgroup(E)) return (int32_t)one_workgroup(E);
  const int64_t c = ((M + 511) / 512 + 15) / 16 * 16;
  return (int32_t)(c < 16 ? 16 : c > 4096 ? 4096 : c);
}

// One workgroup also clears the outputs of all sequences: not too many of them.
bool balance_one(int64_t M, int64_t E, int64_t S) { return M <= one_workgroup(E) && S * E <= 8192; }

hipError_t launch_balance(BalanceArgs a, hipStream_t s) {
  hipError_t e = by_experts<Forward>(a, s);
  if (e != hipSuccess || a.one) return e;
  // whole sequences, and fewer than 2^32 threads, to a launch
  const int64_t nb = (a.E + kBalanceExperts - 1) / kBalanceExperts, most = (1 << 21) / nb, S = a.S;
  for (int64_t s0 = 0; s0 < S && e == hipSuccess; s0 += most) {
    a.s0 = (int32_t)s0;
    const int64_t n = S - s0 < most ? S - s0 : most;
    hipLaunchKernelGGL(balance_sums_kernel, dim3((unsigned)(nb * n)), dim3(64 * kSumWaves), 0, s, a);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_balance_backward(const BalanceArgs& a, hipStream_t s) { return by_experts<Backward>(a, s); }

}  // namespace moe

// A whole mixture-of-experts layer for a few tokens (M <= 64) in two
// launches: router, routing, W1 with SiLU-and-mul in the first, W2 with the
// weighted sum over each token's experts in the second.
//
//   logits = x Wr^T ; (ids, w) = the router's top-k of them
//   z_{e,t} = w_{t,e} silu(W1g_e x_t) (W1u_e x_t)      for the routed (e, t)
//   out_t = sum_e W2_e z_{e,t}        (shared experts: every t, weight 1)
//
// The weight is folded into z before its rounding to bf16 (one rounding, as
// without it), so W2 and the weighted sum are one contraction over (expert,
// feature) pairs: the second kernel gives each 32 output features to the
// waves of a few workgroups, whose MFMA accumulators run through all active
// experts in float32, and no per-route rows are written or re-read.
//
// What bounds it is reading the active experts' weights once; everything
// else is arranged to stay out of that stream's way.  Weight rows go from
// memory straight into the row operand of v_mfma_f32_16x16x32_bf16, the
// tokens sit in the column operand: up to 8 tokens of an expert by whole
// lines (stream_lines), more in tiles of 16 (stream_rows).  MXFP8 codes are
// widened to bf16 in registers (v_cvt_scalef32_pk_bf16_fp8: code times block
// scale, exact in the normal range of bf16), the activations stay bf16.
//
// Measured, first launch + second: 4 tokens, 27 of 64 bf16 experts of 8192
// features, K = 4096: 581 + 307 us for 5.4 GB of weights, 6.1 TB/s; 16
// tokens, 27 of 33 MXFP8 experts of 2048, K = 6144: 161 + 74 us for 1.04 GB,
// 4.4 TB/s (18 us of routing first, 20 us from the median workgroup's end to
// the last one's); 61 tokens, 128 bf16 experts of 1024 and 2 shared, K = 4096: 386 + 192
// us for 3.2 GB, 5.6 TB/s; 7 tokens, 8 experts of 512, K = 256: 9.8 + 8.6 us, latency
// (launch, router, ranking, two streams' round trips).  What such reads reach
// at best is 6.2 to 6.3 TB/s (W2 and W1 of the two-launch streaming path, which
// have no routing in front and no other sums to join).
//
// Inside the first launch the router comes before everything else.  Its work
// (units of 16 experts x 1024 of K, then of 8 tokens to rank) is claimed from
// a counter by whichever workgroups run, so a unit only ever waits for units
// that running workgroups hold; the workgroup that ranks last writes the slot
// list and publishes it, and every workgroup goes on to claim (slot, 8 or 16
// features) items.  The waits are bounded: after about a second a workgroup
// gives up, counts a time-out and leaves, and the second launch, which reads
// that count, writes NaN.  Data that crosses workgroups inside
// a launch goes through device-coherent accesses (the XCDs' L2s are not
// coherent).  A small router (solo) is computed by every workgroup on its
// own, which is faster than passing the result on.
//
// Every sum has a fixed order: the bits do not depend on the run.
#include "kernels.h"
#include "route_device.h"

namespace moe {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kSpinLimit = 1 << 20;   // polls, each a round trip to memory
constexpr uint32_t kPast = 0x80000000u;   // an offset past every buffer: loads give 0
constexpr int kUnitSteps = kWaves;    // 128-wide blocks of K per router unit, one per wave
constexpr int kDownTiles = 2;         // tiles of 16 output features per strip of the second launch

__device__ __forceinline__ int load_relaxed(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float load_relaxed(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ void store_relaxed(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// s_waitcnt vmcnt(0): this wave's loads and stores are done
__device__ __forceinline__ void wait_memory() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | 0x0f00);
  asm volatile("" ::: "memory");
}

// Polls until *p >= target, or the limit (a time-out is counted).
__device__ __forceinline__ bool wait_at_least(const int32_t* p, int target, int32_t* timeouts) {
  for (int n = 0; load_relaxed(p) < target; ++n) {
    if (n > kSpinLimit) {
      atomicAdd(timeouts, 1);
      return false;
    }
    __builtin_amdgcn_s_sleep(2);
  }
  return true;
}

// The thread index, opaque to the compiler: what one phase of the first launch
// derives from it is computed in that phase.  Hoisted out of the phases' loops,
// those values pushed the streaming loop's registers into spills.
__device__ __forceinline__ int phase_thread() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// ------------------------------------------------------------ the stream --
// The weight rows are read in pieces of 16 bytes a lane: 32 of the contraction
// for bf16 (lane group q holds k = 8 q .. +7), 64 for MXFP8 (k = 16 q .. +15,
// all of one 32-wide block), P pieces a step, D steps in flight; the
// activations of CT column tiles come along in the same order of k.  NT: row
// tiles that share the activations (gate and up).
// Steps past the end are loaded from past the buffers, as zeros: every load in
// the loop is unconditional, so the waits count exactly the loads they need.
//
// MXFP8 scales: a 128-wide block has 4 scale bytes a row.  One load gives
// each row's words of 4 blocks, one to each lane group, and each step takes
// its own from the lane that holds it.  A load of its word by every step
// (16 separate lines a load) cost 15% of the first launch and 17% of the
// second at K = 6144, I = 2048 and 33 experts.  (The half-block steps of the
// slots with more than 16 tokens keep that form: they are bound elsewhere, and
// the group's registers would spill.)
template <bool MX, int NT, int CT, int P>
struct Step {
  i32x4 w[NT][P];
  i32x4 a[CT][P][MX ? 2 : 1];
};

template <bool MX>
struct Weights {
  __amdgpu_buffer_rsrc_t w, s;
};

// One expert's matrix of `elems` elements.
template <bool MX>
__device__ __forceinline__ Weights<MX> expert_weights(const void* w, const uint8_t* ws, int64_t e, int64_t elems) {
  const int64_t bytes = elems * (MX ? 1 : 2);
  Weights<MX> r;
  r.w = buffer_rsrc(static_cast<const uint8_t*>(w) + e * bytes, bytes);
  r.s = MX ? buffer_rsrc(ws + e * (elems / 32), elems / 32) : r.w;
  return r;
}
// A lane's first byte of a row, of the row's scales and of a row of activations.
template <bool MX>
__device__ __forceinline__ uint32_t lane_w(int64_t row, int64_t ld, int q) {
  return (uint32_t)(row * ld * (MX ? 1 : 2) + 16 * q);
}
__device__ __forceinline__ uint32_t lane_s(int64_t row, int64_t ld) { return (uint32_t)(row * (ld / 32)); }
template <bool MX>
__device__ __forceinline__ uint32_t lane_a(int64_t row, int64_t ld, int q) {
  return (uint32_t)(row * ld * 2 + (MX ? 32 : 16) * q);
}

// Step `step` of the rows, or zeros when !in.
template <bool MX, int NT, int CT, int P>
__device__ __forceinline__ void load_step(Step<MX, NT, CT, P>& f, const Weights<MX>& wr, __amdgpu_buffer_rsrc_t ar,
                                          const uint32_t (&wo)[NT], const uint32_t (&ao)[CT], int step,
                                          bool in) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const uint32_t o = in ? wo[t] : kPast;
#pragma unroll
    for (int p = 0; p < P; ++p)
      f.w[t][p] = __builtin_amdgcn_raw_buffer_load_b128(wr.w, o + 64 * p, 64 * P * step, 0);
  }
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const uint32_t o = in ? ao[c] : kPast;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int h = 0; h < (MX ? 2 : 1); ++h)
        f.a[c][p][h] =
            __builtin_amdgcn_raw_buffer_load_b128(ar, o + (MX ? 128 : 64) * p + 16 * h, (MX ? 128 : 64) * P * step, 0);
  }
  issue_order();   // steps land in the order they are waited for
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Half h of a piece in bf16: the codes times their block's scale, the lowest
// byte of s.
__device__ __forceinline__ bf16x8 widen(const i32x4& w, uint32_t s, int h) {
  const float sc = __uint_as_float((s & 0xffu) << 23);
  const uint32_t lo = (uint32_t)w[2 * h], hi = (uint32_t)w[2 * h + 1];
  const bf16x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, sc, false),
                       __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, sc, true),
                       __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, sc, false),
                       __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, sc, true)};
  return __builtin_bit_cast(bf16x8, v);
}

// acc += the nb 128-wide blocks b0, b0 + stride, ... of the rows.
template <bool MX, int NT, int CT, int P, int D>
__device__ __forceinline__ void stream_rows(const Weights<MX>& wr, __amdgpu_buffer_rsrc_t ar, const uint32_t (&wo)[NT],
                                            const uint32_t (&so)[NT], const uint32_t (&ao)[CT], int b0,
                                            int stride, int nb, f32x4 (&acc)[NT][CT]) {
  constexpr int kPer = 128 / (P * (MX ? 64 : 32));   // steps of a block
  const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
  const int n = nb * kPer;
  auto at = [&](int i) { return (b0 + i / kPer * stride) * kPer + i % kPer; };
  Step<MX, NT, CT, P> st[D];
  // multiplies step i, held in f; sw: the lane's two scale bytes of its block
  // (0 and 2)
  auto mma = [&](const Step<MX, NT, CT, P>& f, int i, const uint32_t (&sw)[NT]) {
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int h = 0; h < (MX ? 2 : 1); ++h) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const bf16x8 w = MX ? widen(f.w[t][p], sw[t] >> (16 * (i % kPer * P + p)), h) : as_bf16x8(f.w[t][p]);
#pragma unroll
          for (int c = 0; c < CT; ++c)
            acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, as_bf16x8(f.a[c][p][h]), acc[t][c], 0, 0, 0);
        }
      }
    issue_order();
  };
  if constexpr (MX && P == 2) {
    // groups of 4 blocks with one load of scale words each, a group ahead
    static_assert(4 % D == 0, "a group takes whole rounds of the steps in flight");
    uint32_t next[NT], words[NT], sw[NT];
    auto load_words = [&](int b) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
        next[t] = __builtin_amdgcn_raw_buffer_load_b32(wr.s, b + q < nb ? so[t] + 4 * (b0 + (b + q) * stride) : kPast, 0, 0);
      issue_order();
    };
    load_words(0);
#pragma unroll
    for (int d = 0; d < D; ++d) load_step(st[d], wr, ar, wo, ao, at(d), d < n);
    for (int it = 0; it < n; it += 4) {
#pragma unroll
      for (int t = 0; t < NT; ++t) words[t] = next[t];
      load_words(it + 4);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (it + u >= n) return;
#pragma unroll
        for (int t = 0; t < NT; ++t) sw[t] = (uint32_t)__shfl((int)words[t], l16 + 16 * u) >> (8 * (q >> 1));
        mma(st[u % D], it + u, sw);
        load_step(st[u % D], wr, ar, wo, ao, at(it + u + D), it + u + D < n);
      }
    }
  } else {
    uint32_t sw[D][NT];
    auto load = [&](int d, int i) {
      if (MX) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
          sw[d][t] = __builtin_amdgcn_raw_buffer_load_b32(wr.s, i < n ? so[t] : kPast, 4 * (at(i) / kPer), 0);
      }
      load_step(st[d], wr, ar, wo, ao, at(i), i < n);
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, d);
    for (int it = 0; it < n; it += D)
#pragma unroll
      for (int d = 0; d < D; ++d) {
        uint32_t s[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) s[t] = MX ? sw[d][t] >> (8 * (q >> 1)) : 0;
        mma(st[d], it + d, s);
        load(d, it + d + D);
      }
  }
}
// ------------------------------------------------------------- whole lines --
// Up to 8 tokens.  The form above asks the cache for 16 rows of 64 bytes a
// load, half a line each, and a CU gets 28 KB/us of such requests, little more
// than its share of the memory bandwidth and less with the activations'.
// Here a load covers 8 rows of 128 bytes: row slots 2 r and 2 r + 1 of the
// MFMA both stand for row r, the even one for the first half of each line (4
// chunks of 16 bytes, one per lane group), the odd one for the second; column
// c holds token c at the first half's contraction, column c + 8 at the
// second's.  Of the products, (even slot, column < 8) and (odd slot, column
// >= 8) are wanted, and a row's sum is the two together; the rest is not
// used.  As many matrix instructions per byte of weights as before, and half
// the activation loads.
// NR: groups of 8 rows (they share the activations).
template <bool MX, int NR>
struct LineStep {
  i32x4 w[NR][MX ? 1 : 2];   // bf16: two lines of a 128-wide block; MXFP8: one
  i32x4 a[2];
};
// A lane's first byte: of row r of a group (its slot's row is l16 / 2), of
// the activations (row: of token l16 % 8).
template <bool MX>
__device__ __forceinline__ uint32_t line_w(int64_t row, int64_t ld, int l16, int q) {
  return (uint32_t)(row * ld * (MX ? 1 : 2) + 64 * (l16 & 1) + 16 * q);
}
template <bool MX>
__device__ __forceinline__ uint32_t line_a(int64_t row, int64_t ld, int l16, int q) {
  return (uint32_t)(row * ld * 2 + (MX ? 2 : 1) * (64 * (l16 >> 3) + 16 * q));
}

// acc += the nb 128-wide blocks b0, b0 + stride, ... of NR groups of 8 rows:
// group t's begin dr[t] (uniform) after the first's.  so: the scales of the
// lane's row; one load gives a row's words of 8 blocks, one to each of its
// lanes.
template <bool MX, int NR, int D>
__device__ __forceinline__ void stream_lines(const Weights<MX>& wr, __amdgpu_buffer_rsrc_t ar, uint32_t wo, uint32_t so,
                                             const int (&dr)[NR], int ld, uint32_t ao, int b0, int stride, int nb,
                                             f32x4 (&acc)[NR]) {
  const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
  LineStep<MX, NR> st[D];
  auto load = [&](LineStep<MX, NR>& f, int i) {   // past the end: zeros
    const bool in = i < nb;
    const int b = b0 + i * stride;
#pragma unroll
    for (int t = 0; t < NR; ++t)
#pragma unroll
      for (int p = 0; p < (MX ? 1 : 2); ++p)
        f.w[t][p] = __builtin_amdgcn_raw_buffer_load_b128(wr.w, in ? wo + 128 * p : kPast,
                                                          (MX ? 1 : 2) * (dr[t] * ld + 128 * b), 0);
#pragma unroll
    for (int p = 0; p < 2; ++p)
      f.a[p] = __builtin_amdgcn_raw_buffer_load_b128(ar, in ? ao + (MX ? 16 : 128) * p : kPast, 256 * b, 0);
    issue_order();
  };
  auto mma = [&](const LineStep<MX, NR>& f, const uint32_t (&sw)[NR]) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int t = 0; t < NR; ++t) {
        const bf16x8 w = MX ? widen(f.w[t][0], sw[t], p) : as_bf16x8(f.w[t][MX ? 0 : p]);
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, as_bf16x8(f.a[p]), acc[t], 0, 0, 0);
      }
    issue_order();
  };
  uint32_t sw[NR];
#pragma unroll
  for (int t = 0; t < NR; ++t) sw[t] = 0;
  if constexpr (MX) {
    static_assert(8 % D == 0, "8 blocks take whole rounds of the steps in flight");
    uint32_t next[NR], words[NR];
    const int mine = 4 * (l16 & 1) + q;   // which of 8 blocks' words this lane holds
    auto load_words = [&](int b) {
#pragma unroll
      for (int t = 0; t < NR; ++t)
        next[t] = __builtin_amdgcn_raw_buffer_load_b32(wr.s, b + mine < nb ? so + 4 * (b0 + (b + mine) * stride) : kPast,
                                                       dr[t] * (ld / 32), 0);
      issue_order();
    };
    load_words(0);
#pragma unroll
    for (int d = 0; d < D; ++d) load(st[d], d);
    for (int it = 0; it < nb; it += D) {
      if (it % 8 == 0) {
#pragma unroll
        for (int t = 0; t < NR; ++t) words[t] = next[t];
        load_words(it + 8);
      }
#pragma unroll
      for (int d = 0; d < D; ++d) {
        // block u's word is with the row's lane (parity u / 4, group u % 4);
        // this lane's chunk is scaled by its byte 2 parity + q / 2
        const int u = (it + d) % 8, from = ((l16 & ~1) | (u >> 2)) + 16 * (u & 3);
#pragma unroll
        for (int t = 0; t < NR; ++t)
          sw[t] = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * from, (int)words[t]) >> (8 * (2 * (l16 & 1) + (q >> 1)));
        mma(st[d], sw);
        load(st[d], it + d + D);
      }
    }
  } else {
#pragma unroll
    for (int d = 0; d < D; ++d) load(st[d], d);
    for (int it = 0; it < nb; it += D)
#pragma unroll
      for (int d = 0; d < D; ++d) {
        mma(st[d], sw);
        load(st[d], it + d + D);
      }
  }
}

__device__ __forceinline__ uint64_t below(int t) { return t == 0 ? 0ull : (~0ull >> (64 - t)); }

// -------------------------------------------------------------- routing --
constexpr int kSoloRows = kWaves * (kLayerMaxTopk + kLayerMaxShared);

// What a workgroup keeps of the routing while it streams.
struct SlotLds {
  int32_t e[kLayerMaxE + kLayerMaxShared];
  int32_t pos[kLayerMaxE + kLayerMaxShared + 1];     // first row; the next slot's is one past the last
  float w[kSoloRows];                                 // solo only: the rows' weights
  uint8_t tok[kLayerMaxRoutes + kLayerMaxM * kLayerMaxShared];
};

struct RouteLds {
  uint64_t mask[kLayerMaxE];            // tokens of each expert
  int32_t pos[kLayerMaxE];              // their first row
  int32_t id[kLayerMaxRoutes];          // the tokens' choices
  float w[kLayerMaxRoutes];
  int32_t wave_n[kWaves], wave_c[kWaves];
};

// Ranks tokens t0 .. t0 + 7, one per wave.  partial(n, t, e): the n-th partial
// logit; all of a lane's are requested before the first is added.
template <int NV, typename Partial>
__device__ __forceinline__ void rank_tokens(const LayerArgs& g, int t0, RouteLds& s, double* keys, bool publish,
                                            Partial partial) {
  const int tid = phase_thread(), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t = t0 + wave;
  if (t >= g.M) return;
  float sum[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) sum[i] = 0.f;
  constexpr int kBatch = 8;
  for (int n0 = 0; n0 < g.rsplit; n0 += kBatch) {
    float v[NV][kBatch];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int n = 0; n < kBatch; ++n) v[i][n] = partial(min(n0 + n, g.rsplit - 1), t, min(lane + 64 * i, g.r.E - 1));
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int n = 0; n < kBatch; ++n)
        if (n0 + n < g.rsplit) sum[i] += v[i][n];
  }
  double l[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    double v = -INFINITY;
    if (e < g.r.E) {
      v = sum[i];
      if (g.r.bias_kind == 1) v += (double)g.rbias[e];
    }
    l[i] = route_logit(v);
  }
  int id;
  float w;
  route_token<NV>(g.r, l, g.rbias, keys + (g.r.groups > 1 ? wave * (g.r.E + g.r.groups) : 0), id, w);
  if (lane < g.r.topk) {
    const int i = t * g.r.topk + lane;
    s.id[i] = id;
    s.w[i] = w;
    if (publish) {
      store_relaxed(g.ids + i, id);
      store_relaxed(g.wts + i, w);
    }
  }
}

// From the tokens' choices (s.id, s.w), the slots: the experts that got a
// token, in ascending order, each with the rows [pos0, pos0 + cnt) of z for
// its tokens in ascending order; the shared experts last, with every token.
// To memory (publish) and, with lds, to the workgroup's own copy.
__device__ __forceinline__ void build_slots(const LayerArgs& g, RouteLds& s, bool publish, SlotLds* lds) {
  const int tid = phase_thread(), lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < g.r.E; e += kThreads) s.mask[e] = 0;
  __syncthreads();
  for (int i = tid; i < g.M * g.r.topk; i += kThreads)
    if (s.id[i] >= 0) atomicOr((unsigned long long*)&s.mask[s.id[i]], 1ull << (i / g.r.topk));
  __syncthreads();
  // one expert per thread (E <= kThreads): sums of (has tokens, tokens)
  const uint64_t m = tid < g.r.E ? s.mask[tid] : 0;
  const int cnt = __popcll(m);
  int n = cnt > 0, c = cnt;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int a = __shfl_up(n, d), b = __shfl_up(c, d);
    if (lane >= d) { n += a; c += b; }
  }
  if (lane == 63) { s.wave_n[wave] = n; s.wave_c[wave] = c; }
  __syncthreads();
  int n0 = 0, c0 = 0, nt = 0, ct = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) { n0 += s.wave_n[w]; c0 += s.wave_c[w]; }
    nt += s.wave_n[w];
    ct += s.wave_c[w];
  }
  n += n0;
  c += c0;
  if (tid < g.r.E) s.pos[tid] = c - cnt;
  auto slot = [&](int at, int e, int count, int pos0, uint64_t mask) {
    if (publish) g.slots[at] = LayerSlot{e, count, pos0, 0, mask, 0};
    if (lds) { lds->e[at] = e; lds->pos[at] = pos0; }
  };
  if (cnt > 0) slot(n - 1, tid, cnt, c - cnt, m);
  if (tid < g.S) slot(nt + tid, g.r.E + tid, g.M, ct + tid * g.M, below(g.M));
  __syncthreads();
  auto row = [&](int p, int t, float w) {
    if (publish) { g.rows[p] = t; g.roww[p] = w; }
    if (lds) { lds->tok[p] = (uint8_t)t; lds->w[p] = w; }
  };
  for (int i = tid; i < g.M * g.r.topk; i += kThreads) {
    const int e = s.id[i], t = i / g.r.topk;
    if (e >= 0) row(s.pos[e] + __popcll(s.mask[e] & below(t)), t, s.w[i]);
  }
  for (int i = tid; i < g.S * g.M; i += kThreads) row(ct + i, i % g.M, 1.0f);
  if (tid == 0) {
    if (publish) {
      g.sync[kLayerNumSlots] = nt + g.S;
      g.sync[kLayerNumRows] = ct + g.S * g.M;
    }
    if (lds) {
      lds->pos[nt + g.S] = ct + g.S * g.M;
      s.wave_n[0] = nt + g.S;
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------- first launch --
// Partial logits of 16 experts over 1024 of K (one 128-wide step per wave).
// put(n, t, e, v): partial logits e .. e + 3 of token t, split n.
template <int CT, typename Put>
__device__ __forceinline__ void router_unit(const LayerArgs& g, int unit, f32x4* red, Put put) {
  const int tid = phase_thread(), lane = tid & 63, q = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int e0 = 16 * (unit / g.rsplit), n = unit % g.rsplit;
  const int step = n * kUnitSteps + wave;
  f32x4 acc[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) acc[c] = (f32x4){0.f, 0.f, 0.f, 0.f};
  if (128 * step < g.K) {
    Weights<false> wr;
    wr.w = wr.s = buffer_rsrc(g.wr, (int64_t)g.r.E * g.K * 2);
    const __amdgpu_buffer_rsrc_t ar = buffer_rsrc(g.x, (int64_t)g.M * g.K * 2);
    const uint32_t wo[1] = {e0 + l16 < g.r.E ? lane_w<false>(e0 + l16, g.K, q) : kPast};
    uint32_t ao[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) ao[c] = 16 * c + l16 < g.M ? lane_a<false>(16 * c + l16, g.K, q) : kPast;
    f32x4 sum[1][CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) sum[0][c] = acc[c];
    stream_rows<false, 1, CT, 4, 1>(wr, ar, wo, wo, ao, step, 1, 1, sum);
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[c] = sum[0][c];
  }
#pragma unroll
  for (int c = 0; c < CT; ++c) red[(wave * CT + c) * 64 + lane] = acc[c];
  __syncthreads();
  if (wave < CT) {
    f32x4 sum = red[wave * 64 + lane];
    for (int w = 1; w < kWaves; ++w) sum += red[(w * CT + wave) * 64 + lane];
    const int t = 16 * wave + l16;   // sum[r]: expert e0 + 4 q + r, token t
    if (t < g.M) put(n, t, e0 + 4 * q, sum);
  }
  __syncthreads();
}

// z of 16 features of one slot with up to 16 CT tokens: wave kw of ks takes
// the 128-wide blocks kw, kw + ks, ... of K (the waves together read each
// weight row in long runs: contiguous parts per wave measured 5% slower) of
// the gate and up rows.
template <bool MX, int CT, int P, int D>
__device__ __forceinline__ void gate_up_strip(const LayerArgs& g, const SlotLds& s, int slot, int f0, int kw, bool live,
                                              f32x4* red) {
  const int lane = phase_thread() & 63, q = lane >> 4, l16 = lane & 15;
  const int e = __builtin_amdgcn_readfirstlane(s.e[slot]);
  const int pos0 = s.pos[slot], cnt = s.pos[slot + 1] - pos0;
  const int n = live ? (g.K / 128 - kw + g.ks - 1) / g.ks : 0;
  const Weights<MX> wr = expert_weights<MX>(g.w1, g.w1s, e, 2ll * g.I * g.K);
  uint32_t wo[2], so[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int row = w1_row(f0 + l16, t != 0, g.I, g.w1_order);
    wo[t] = lane_w<MX>(row, g.K, q);
    so[t] = lane_s(row, g.K);
  }
  float wt[CT];
  f32x4 acc[2][CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    wt[c] = 16 * c + l16 >= cnt ? 0.f : g.solo ? s.w[pos0 + 16 * c + l16] : load_relaxed(g.roww + pos0 + 16 * c + l16);
#pragma unroll
    for (int t = 0; t < 2; ++t) acc[t][c] = (f32x4){0.f, 0.f, 0.f, 0.f};
  }
  const __amdgpu_buffer_rsrc_t ar = buffer_rsrc(g.x, (int64_t)g.M * g.K * 2);
  uint32_t ao[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c)
    ao[c] = 16 * c + l16 < cnt ? lane_a<MX>(s.tok[pos0 + 16 * c + l16], g.K, q) : kPast;
  stream_rows<MX, 2, CT, P, D>(wr, ar, wo, so, ao, kw, g.ks, n, acc);
#pragma unroll
  for (int c = 0; c < CT; ++c) {
#pragma unroll
    for (int t = 0; t < 2; ++t) red[(kw * 2 + t) * 64 + lane] = acc[t][c];
    __syncthreads();
    const int tk = 16 * c + l16;
    if (live && c % g.ks == kw && tk < cnt) {   // column tile c: one of the strip's waves
      f32x4 gate = red[lane], up = red[64 + lane];
      for (int k = 1; k < g.ks; ++k) {
        gate += red[2 * k * 64 + lane];
        up += red[(2 * k + 1) * 64 + lane];
      }
      uint32_t h[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) h[r] = f32_to_bf16_rne(wt[c] * (silu_f32(gate[r]) * up[r]));
      *reinterpret_cast<uint2*>(g.z + (int64_t)(pos0 + tk) * g.I + f0 + 4 * q) =
          make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    }
    __syncthreads();
  }
}

// The same of F features (8 or 16) for a slot of up to 8 tokens, by whole
// lines.
template <bool MX, int F>
__device__ __forceinline__ void gate_up_lines(const LayerArgs& g, const SlotLds& s, int slot, int f0, int kw, bool live,
                                              f32x4* red) {
  constexpr int H = F / 8, NR = 2 * H;   // groups of 8 rows: the features' gates, then their ups
  const int lane = phase_thread() & 63, q = lane >> 4, l16 = lane & 15;
  const int e = __builtin_amdgcn_readfirstlane(s.e[slot]);
  const int pos0 = s.pos[slot], cnt = s.pos[slot + 1] - pos0;
  const int n = live ? (g.K / 128 - kw + g.ks - 1) / g.ks : 0;
  const Weights<MX> wr = expert_weights<MX>(g.w1, g.w1s, e, 2ll * g.I * g.K);
  const __amdgpu_buffer_rsrc_t ar = buffer_rsrc(g.x, (int64_t)g.M * g.K * 2);
  const int row = w1_row(f0 + (l16 >> 1), 0, g.I, g.w1_order);
  const int up = __builtin_amdgcn_readfirstlane(w1_row(f0, 1, g.I, g.w1_order) - w1_row(f0, 0, g.I, g.w1_order));
  int dr[NR];
#pragma unroll
  for (int t = 0; t < NR; ++t) dr[t] = 8 * (t % H) + (t / H) * up;
  const int tk = l16 & 7, hh = l16 >> 3;
  const uint32_t ao = tk < cnt ? line_a<MX>(s.tok[pos0 + tk], g.K, l16, q) : kPast;
  const float wt = tk >= cnt ? 0.f : g.solo ? s.w[pos0 + tk] : load_relaxed(g.roww + pos0 + tk);
  f32x4 acc[NR];
#pragma unroll
  for (int t = 0; t < NR; ++t) acc[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
  stream_lines<MX, NR, 2>(wr, ar, line_w<MX>(row, g.K, l16, q), lane_s(row, g.K), dr, g.K, ao, kw, g.ks, n, acc);
#pragma unroll
  for (int t = 0; t < NR; ++t) red[(kw * NR + t) * 64 + lane] = acc[t];
  __syncthreads();
  if (live && kw == 0 && tk < cnt && hh < H) {
    // lane (token tk, features 8 hh + 2 q, + 1): even slots from the token's
    // column, odd ones from the column 8 on
    const int at = 16 * q + tk;
    float v[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
    for (int k = 0; k < g.ks; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const f32x4 lo = red[(k * NR + H * t + hh) * 64 + at], hi = red[(k * NR + H * t + hh) * 64 + at + 8];
        v[t][0] += lo[0] + hi[1];
        v[t][1] += lo[2] + hi[3];
      }
    const uint32_t a = f32_to_bf16_rne(wt * (silu_f32(v[0][0]) * v[1][0]));
    const uint32_t b = f32_to_bf16_rne(wt * (silu_f32(v[0][1]) * v[1][1]));
    *reinterpret_cast<uint32_t*>(g.z + (int64_t)(pos0 + tk) * g.I + f0 + 8 * hh + 2 * q) = a | (b << 16);
  }
  __syncthreads();
}

// Features of an item of the first launch.
__host__ __device__ constexpr int item_features(bool mx, bool wide) { return mx || wide ? 16 : 8; }

// WIDE: M > 8 (a slot may hold up to 64 tokens).  At most 128 registers, so
// two workgroups share a CU and one's joins overlap the other's streaming.
template <bool MX, bool WIDE, int NV>
__global__ void __launch_bounds__(kThreads, 4) layer_gate_up_kernel(LayerArgs g) {
  // streaming: the strips' sums, the slots; before that the routing, in front
  // of the slots
  constexpr int kSums = kWaves * 4 * 64 * 16;
  constexpr int kRoute = (int)sizeof(RouteLds) + kWaves * 64 * (NV + 1) * 8 +
                         (NV == 1 ? 16 + kLayerSoloUnits * kWaves * 64 * 4 : 0);
  constexpr int kStream = ((kSums > kRoute ? kSums : kRoute) + 15) / 16 * 16;
  constexpr int kSlots = ((int)sizeof(SlotLds) + 15) / 16 * 16;
  static_assert(kRoute <= kStream && kWaves * (WIDE ? 4 : 1) * 64 * 16 <= kStream, "routing and router units fit");
  __shared__ __attribute__((aligned(16))) char smem[kStream + kSlots];
  __shared__ int s_claim, s_last, s_slots;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  f32x4* red = reinterpret_cast<f32x4*>(smem);
  RouteLds& rl = *reinterpret_cast<RouteLds*>(smem);
  double* keys = reinterpret_cast<double*>(smem + sizeof(RouteLds));
  SlotLds& s = *reinterpret_cast<SlotLds*>(smem + kStream);
  int nslots;

  // The second launch's arrival counters start at 0.  Cleared here and not by
  // their last reader: a plan with another K has other data at their place.
  if (g.splits > 1 && blockIdx.x == gridDim.x - 1)
    for (int i = threadIdx.x; i < g.K / (16 * kDownTiles); i += kThreads) store_relaxed(g.sync + kLayerStrips + i, 0);

  if (NV == 1 && !WIDE && g.solo) {
    // a small router: every workgroup computes the whole routing by itself
    constexpr int kLogits = ((int)sizeof(RouteLds) + kWaves * 64 * 2 * 8 + 15) / 16 * 16;
    float* logits = reinterpret_cast<float*>(smem + kLogits);   // [rsplit][8][64]
    static_assert(kLogits >= kWaves * 64 * 16 && kLogits + kLayerSoloUnits * kWaves * 64 * 4 <= kStream, "logits fit");
    for (int unit = 0; unit < g.runits; ++unit)
      router_unit<1>(g, unit, red, [&](int n, int t, int e, f32x4 v) {
        *reinterpret_cast<f32x4*>(logits + (n * kWaves + t) * 64 + e) = v;
      });
    const bool first = blockIdx.x == 0;
    rank_tokens<NV>(g, 0, rl, keys, first, [&](int n, int t, int e) { return logits[(n * kWaves + t) * 64 + e]; });
    __syncthreads();
    build_slots(g, rl, first, &s);
    nslots = __builtin_amdgcn_readfirstlane(rl.wave_n[0]);
    if (first && threadIdx.x == 0) g.sync[kLayerRouted] = 1;
    __syncthreads();
  } else {
    // The routing's units, until none is left: the router's, then ranking 8
    // tokens each.  A ranking unit waits for the router's units, which
    // running workgroups have claimed before it.
    const int tunits = (g.M + kWaves - 1) / kWaves;
    for (;;) {
      if (threadIdx.x == 0)
        s_claim = __hip_atomic_fetch_add(g.sync + kLayerClaim, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __syncthreads();
      const int unit = s_claim;
      if (unit >= g.runits + tunits) break;
      if (unit < g.runits) {
        router_unit<WIDE ? 4 : 1>(g, unit, red, [&](int n, int t, int e, f32x4 v) {
          float* o = g.logits + ((int64_t)n * g.M + t) * g.logit_ld + e;
#pragma unroll
          for (int r = 0; r < 4; ++r) store_relaxed(o + r, v[r]);
        });
        wait_memory();
        __syncthreads();
        if (threadIdx.x == 0)
          __hip_atomic_fetch_add(g.sync + kLayerArrived, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      } else {
        if (threadIdx.x == 0) s_last = wait_at_least(g.sync + kLayerArrived, g.runits, g.status);
        __syncthreads();
        const bool ready = s_last;
        __syncthreads();
        if (ready) {
          rank_tokens<NV>(g, (unit - g.runits) * kWaves, rl, keys, true, [&](int n, int t, int e) {
            return load_relaxed(g.logits + ((int64_t)n * g.M + t) * g.logit_ld + e);
          });
          wait_memory();
          __syncthreads();
          if (threadIdx.x == 0)
            s_last = tunits == 1 || __hip_atomic_fetch_add(g.sync + kLayerRanked, 1, __ATOMIC_RELAXED,
                                                           __HIP_MEMORY_SCOPE_AGENT) == tunits - 1;
          __syncthreads();
          if (s_last) {   // every token is ranked: the slots
            if (tunits > 1) {
              for (int i = phase_thread(); i < g.M * g.r.topk; i += kThreads) {
                rl.id[i] = load_relaxed(g.ids + i);
                rl.w[i] = load_relaxed(g.wts + i);
              }
            }
            __syncthreads();
            build_slots(g, rl, true, nullptr);
            wait_memory();
            __syncthreads();
            if (threadIdx.x == 0)
              __hip_atomic_store(g.sync + kLayerRouted, 1, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
          }
        }
      }
      // Keeps this unit's work of thread 0 apart from the next claim's: with no
      // barrier between the two, the compiler may run thread 0 through both
      // while the other lanes of its wave go round without it, and the
      // wave's barriers no longer match the other waves'.
      __syncthreads();
    }

    if (threadIdx.x == 0)
      s_slots = wait_at_least(g.sync + kLayerRouted, 1, g.status) ? load_relaxed(g.sync + kLayerNumSlots) : 0;
    __syncthreads();
    nslots = s_slots;
    {
      const int tid = phase_thread();
      const int total = nslots ? load_relaxed(g.sync + kLayerNumRows) : 0;
      for (int i = tid; i < nslots; i += kThreads) {
        s.e[i] = load_relaxed(&g.slots[i].e);
        s.pos[i] = load_relaxed(&g.slots[i].pos0);
      }
      if (tid == 0) s.pos[nslots] = total;
      for (int i = tid; i < total; i += kThreads) s.tok[i] = (uint8_t)load_relaxed(g.rows + i);
    }
    __syncthreads();
  }

  // Items (slot, nh strips of F features): a workgroup starts with its own and
  // then claims one after another, the last slots first (the shared experts
  // hold every token and take longest).  With a fixed share each, the
  // workgroups that got the shared experts' strips ended last by half the
  // launch; in chunks of several items the ends lay further apart.  bf16 of
  // few tokens does best with short items (4 tokens, 4096 x 8192: F = 8 583 us,
  // 16 605); with MXFP8's shorter rows a start and a join for each 8 features
  // cost more than the closer ends bring (6144 x 2048: 8 185 us, 16 163; the
  // last item of each workgroup halved, 172).
  constexpr int F = item_features(MX, WIDE);
  const int nh = kWaves / g.ks;
  const int h = wave / g.ks, kw = wave % g.ks;
  const int strips = g.I / F, per = (strips + nh - 1) / nh;
  const int items = nslots * per;
  f32x4* mine = red + h * g.ks * 4 * 64;
  for (int claim = blockIdx.x; claim < items;) {
    int next = 0;   // the claim's answer is used an item later
    if (threadIdx.x == 0)
      next = __hip_atomic_fetch_add(g.sync + kLayerItems, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const int item = items - 1 - claim;
    const int slot = item / per;
    const int strip = item % per * nh + h;
    const bool live = strip < strips;
    const int pos0 = s.pos[slot];
    const int cnt = __builtin_amdgcn_readfirstlane(s.pos[slot + 1] - pos0);
    if (!WIDE || cnt <= 8) gate_up_lines<MX, F>(g, s, slot, F * strip, kw, live, mine);
    else if (cnt <= 16) gate_up_strip<MX, 1, MX ? 2 : 4, 2>(g, s, slot, 16 * strip, kw, live, mine);
    else if (cnt <= 32) gate_up_strip<MX, 2, MX ? 1 : 2, 2>(g, s, slot, 16 * strip, kw, live, mine);
    else gate_up_strip<MX, 4, 1, MX ? 1 : 2>(g, s, slot, 16 * strip, kw, live, mine);
    if (threadIdx.x == 0) s_claim = next;
    __syncthreads();
    claim = __builtin_amdgcn_readfirstlane((int)gridDim.x + s_claim);
    __syncthreads();   // read before the next claim's answer overwrites it
  }
}

// --------------------------------------------------------- second launch --
// Workgroup (strip, split): the 32 output features of the strip over its
// share of the active slots' features, one contiguous run per wave, slot by
// slot.  Up to 8 tokens the MFMA columns are the tokens; beyond, they are the
// slot's own (most slots hold a few of the 64).  Each slot's sums are added to
// the wave's [token][32] tile in LDS.  The waves' sums meet in LDS in wave order; with
// more than one split the workgroup that arrives last adds the splits' sums
// in order.
template <bool MX, int CT, int P, int D>
__device__ __forceinline__ void down_run(const LayerArgs& g, const LayerSlot& sl, const uint32_t (&wo)[kDownTiles],
                                         const uint32_t (&so)[kDownTiles], int b0, int nb, f32x4* tile) {
  const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
  const int e = __builtin_amdgcn_readfirstlane(sl.e), cnt = sl.cnt, pos0 = sl.pos0;
  const Weights<MX> wr = expert_weights<MX>(g.w2, g.w2s, e, (int64_t)g.K * g.I);
  const __amdgpu_buffer_rsrc_t ar = buffer_rsrc(g.z, (int64_t)g.cap * g.I * 2);
  uint32_t ao[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) ao[c] = 16 * c + l16 < cnt ? lane_a<MX>(pos0 + 16 * c + l16, g.I, q) : kPast;
  f32x4 acc[kDownTiles][CT];
#pragma unroll
  for (int t = 0; t < kDownTiles; ++t)
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[t][c] = (f32x4){0.f, 0.f, 0.f, 0.f};
  int tok[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) tok[c] = 16 * c + l16 < cnt ? g.rows[pos0 + 16 * c + l16] : -1;
  stream_rows<MX, kDownTiles, CT, P, D>(wr, ar, wo, so, ao, b0, 1, nb, acc);
#pragma unroll
  for (int c = 0; c < CT; ++c)
    if (tok[c] >= 0) {
#pragma unroll
      for (int t = 0; t < kDownTiles; ++t) tile[(tok[c] * kDownTiles + t) * 4 + q] += acc[t][c];
    }
}

// The same for a slot of up to 8 tokens, by whole lines: acc[t] += 8 output
// features of tile t each; down_lines_add puts a slot's (or, up to 8 tokens,
// all slots') sums into the wave's tile, tok: the token of column l16 % 8.
constexpr int kDownGroups = 2 * kDownTiles;

template <bool MX>
__device__ __forceinline__ void down_lines(const LayerArgs& g, int e, int strip, int zrow, int b0, int nb,
                                           f32x4 (&acc)[kDownGroups]) {
  const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
  const Weights<MX> wr = expert_weights<MX>(g.w2, g.w2s, e, (int64_t)g.K * g.I);
  const __amdgpu_buffer_rsrc_t ar = buffer_rsrc(g.z, (int64_t)g.cap * g.I * 2);
  const int row = 8 * kDownGroups * strip + (l16 >> 1);
  int dr[kDownGroups];
#pragma unroll
  for (int t = 0; t < kDownGroups; ++t) dr[t] = 8 * t;
  stream_lines<MX, kDownGroups, 2>(wr, ar, line_w<MX>(row, g.I, l16, q), lane_s(row, g.I), dr, g.I,
                                   zrow >= 0 ? line_a<MX>(zrow, g.I, l16, q) : kPast, b0, 1, nb, acc);
}
__device__ __forceinline__ void down_lines_add(const f32x4 (&acc)[kDownGroups], int tok, f32x4* tile) {
  const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
  float* f = reinterpret_cast<float*>(tile);
#pragma unroll
  for (int t = 0; t < kDownGroups; ++t) {
    const float a = acc[t][0] + __shfl_xor(acc[t][1], 8), b = acc[t][2] + __shfl_xor(acc[t][3], 8);
    if (l16 < 8 && tok >= 0) {
      float2* dst = reinterpret_cast<float2*>(f + tok * (16 * kDownTiles) + 8 * t + 2 * q);
      const float2 old = *dst;
      *dst = make_float2(old.x + a, old.y + b);
    }
  }
}

template <bool MX, bool WIDE>
__global__ void __launch_bounds__(kThreads, 4) layer_down_kernel(LayerArgs g) {
  // [wave][token][4 of the 32 features]
  constexpr int kTok = WIDE ? kLayerMaxM : 8;
  constexpr int kQ = 4 * kDownTiles;
  __shared__ __attribute__((aligned(16))) f32x4 red[kWaves * kTok * kQ];
  // the slots (dynamic: the launch passes room for the most there can be) are
  // requested before their number is known
  extern __shared__ LayerSlot s_slots[];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int strip = blockIdx.x / g.splits, split = blockIdx.x % g.splits;
  for (int i = threadIdx.x; i < g.max_slots; i += kThreads) s_slots[i] = g.slots[i];
  // after a wait that gave up: nothing of the first launch is used, out is NaN
  const int gave_up = g.sync[kLayerStatus], routed = g.sync[kLayerRouted], slots = g.sync[kLayerNumSlots];
  const bool failed = gave_up != 0 || routed == 0;
  const int nslots = failed ? 0 : slots;
  __syncthreads();
  const int spe = g.I / 128;                             // blocks per slot
  const int64_t total = (int64_t)nslots * spe;
  const int parts = g.splits * kWaves, part = split * kWaves + wave;
  int64_t b = part * total / parts;
  const int64_t end = (part + 1) * total / parts;
  uint32_t wo[kDownTiles], so[kDownTiles];
#pragma unroll
  for (int t = 0; t < kDownTiles; ++t) {
    wo[t] = lane_w<MX>(16 * (kDownTiles * strip + t) + l16, g.I, q);
    so[t] = lane_s(16 * (kDownTiles * strip + t) + l16, g.I);
  }
  const int col = l16 & 7;
  f32x4* tile = red + wave * kTok * kQ;
#pragma unroll
  for (int i = 0; i < kTok * kQ; i += 64) tile[i + lane] = (f32x4){0.f, 0.f, 0.f, 0.f};

  // A slot's sums are added to its own tokens only: a token takes no part in
  // other experts' products, not even as a zero, so an infinite weight stays
  // with the tokens of its expert.
  while (b < end) {
    const int slot = (int)(b / spe), b0 = (int)(b % spe);
    const int n = (int)min<int64_t>(spe - b0, end - b);
    const LayerSlot& sl = s_slots[slot];
    const int cnt = __builtin_amdgcn_readfirstlane(sl.cnt);
    if (!WIDE || cnt <= 8) {
      // columns: the tokens, or beyond 8 tokens the slot's (listed in rows)
      const int tok = WIDE ? (col < cnt ? g.rows[sl.pos0 + col] : -1) : ((sl.mask >> col) & 1 ? col : -1);
      const int zrow = sl.pos0 + (WIDE ? col : __popcll(sl.mask & below(col)));
      f32x4 acc[kDownGroups];
#pragma unroll
      for (int t = 0; t < kDownGroups; ++t) acc[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
      down_lines<MX>(g, __builtin_amdgcn_readfirstlane(sl.e), strip, tok >= 0 ? zrow : -1, b0, n, acc);
      down_lines_add(acc, tok, tile);
    } else if (cnt <= 16) down_run<MX, 1, MX ? 2 : 4, 2>(g, sl, wo, so, b0, n, tile);
    else if (cnt <= 32) down_run<MX, 2, MX ? 1 : 2, 2>(g, sl, wo, so, b0, n, tile);
    else down_run<MX, 4, 1, MX ? 1 : 2>(g, sl, wo, so, b0, n, tile);
    b += n;
  }
  __syncthreads();
  // thread (t, quarter) finishes 4 features of token t
  const int t = threadIdx.x / kQ, qt = threadIdx.x % kQ;
  const bool mine = t < g.M;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  if (mine)
    for (int k = 0; k < kWaves; ++k) sum += red[(k * kTok + t) * kQ + qt];
  bool finish = mine;
  if (g.splits > 1) {
    // [strip][split][token][32] partial sums
    float* p = g.part + ((int64_t)strip * g.splits * g.M + t) * (4 * kQ) + 4 * qt;
    if (mine) {
#pragma unroll
      for (int r = 0; r < 4; ++r) store_relaxed(p + (int64_t)split * g.M * 4 * kQ + r, sum[r]);
    }
    wait_memory();
    __syncthreads();
    if (threadIdx.x == 0)
      s_last = __hip_atomic_fetch_add(g.sync + kLayerStrips + strip, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
               g.splits - 1;
    __syncthreads();
    finish = mine && s_last;
    if (finish) {
      sum = (f32x4){0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < g.splits; ++k)
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[r] += load_relaxed(p + (int64_t)k * g.M * 4 * kQ + r);
    }
  }
  if (finish) {
    uint32_t h[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) h[r] = failed ? 0x7fc0u : f32_to_bf16_rne(sum[r]);
    *reinterpret_cast<uint2*>(g.out + (int64_t)t * g.K + 4 * kQ * strip + 4 * qt) =
        make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  }
  // the last workgroup of the launch clears the first launch's counters
  if (threadIdx.x == 0) {
    const int done = __hip_atomic_fetch_add(g.sync + kLayerDone, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (done == (int)gridDim.x - 1) {
      store_relaxed(g.sync + kLayerClaim, 0);
      store_relaxed(g.sync + kLayerItems, 0);
      store_relaxed(g.sync + kLayerArrived, 0);
      store_relaxed(g.sync + kLayerRanked, 0);
      store_relaxed(g.sync + kLayerRouted, 0);
      store_relaxed(g.sync + kLayerDone, 0);
    }
  }
}

template <bool MX, bool WIDE>
hipError_t launch(const LayerArgs& g, unsigned grid1, hipStream_t s) {
  if (g.r.E <= 64)
    hipLaunchKernelGGL((layer_gate_up_kernel<MX, WIDE, 1>), dim3(grid1), dim3(kThreads), 0, s, g);
  else if (g.r.E <= 128)
    hipLaunchKernelGGL((layer_gate_up_kernel<MX, WIDE, 2>), dim3(grid1), dim3(kThreads), 0, s, g);
  else
    hipLaunchKernelGGL((layer_gate_up_kernel<MX, WIDE, 8>), dim3(grid1), dim3(kThreads), 0, s, g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((layer_down_kernel<MX, WIDE>), dim3((unsigned)(g.K / (16 * kDownTiles) * g.splits)), dim3(kThreads),
                     sizeof(LayerSlot) * g.max_slots, s, g);
  return hipGetLastError();
}

}  // namespace

// Splits of the second launch: the smallest power of two, up to 8, that gives
// the chip its two workgroups per CU, but not so many that a wave has fewer
// than 4 blocks of 128 features to read with every slot filled (`blocks` in
// all; 2 while there are fewer than 64 workgroups, where it is the few CUs'
// loads that take the time).  1 / 2 / 4 / 8 splits, us: the second launch at K =
// 6144 (192 strips), MXFP8, 33 experts of 2048, 127 / 92 / 80 / 101 (more
// workgroups than fit pay their start and their join again).  The whole layer,
// bf16: one token, K = 7168, 2 of 64 experts of 2048 (32 blocks) 48 / 50 / 56 / -;
// one, K = 2048, 8 of 64 of 1024 (64) 43 / 42 / 43 / 47; 4 tokens, K = 2048, 27 of
// 64 of 512 (at most 128) 63 / 57 / 55 / 62; with fewer than 64 workgroups, 7
// tokens, K = 256 (32) 19.2 / 18.1 / 17.9 / 18.3; 4, K = 512 (32) 19.2 / 19.1 /
// 18.5 / 19.7; 4, K = 512 (128) 33.0 / 29.6 / 27.3 / 27.7; 40, K = 512 (64) 43.0 /
// 36.9 / 33.8 / 32.9; 8, MXFP8, K = 256 (32) 16.4 / 16.9 / 17.3 / 18.0.
int32_t layer_splits(int64_t K, int64_t blocks) {
  int32_t s = 1;
  const int64_t strips = K / (16 * kDownTiles);
  while (s < 8 && strips * s < 512 && blocks >= 2 * s * kWaves * (strips * s < 64 ? 2 : 4)) s *= 2;
  return s;
}

int32_t layer_router_splits(int64_t K) { return (int32_t)((K / 128 + kUnitSteps - 1) / kUnitSteps); }

hipError_t launch_layer(LayerArgs g, bool mxfp8, hipStream_t s) {
  g.rsplit = layer_router_splits(g.K);
  g.runits = (g.r.E + 15) / 16 * g.rsplit;
  g.splits = layer_splits(g.K, (int64_t)g.max_slots * (g.I / 128));
  g.solo = g.runits <= kLayerSoloUnits && g.M <= kWaves && g.r.E <= 64;
  g.ks = g.K >= 1024 ? 8 : g.K >= 512 ? 4 : g.K >= 256 ? 2 : 1;
  const int nh = kWaves / g.ks, f = item_features(mxfp8, g.M > 8);
  const int64_t items = (int64_t)g.max_slots * ((g.I / f + nh - 1) / nh);
  const int64_t units = g.runits + (g.M + kWaves - 1) / kWaves;
  int64_t grid = items > units ? items : units;
  if (grid > 512) grid = 512;
  if (g.M > 8) return mxfp8 ? launch<true, true>(g, (unsigned)grid, s) : launch<false, true>(g, (unsigned)grid, s);
  return mxfp8 ? launch<true, false>(g, (unsigned)grid, s) : launch<false, false>(g, (unsigned)grid, s);
}

}  // namespace moe

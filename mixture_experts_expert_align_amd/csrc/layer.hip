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
// feature) pairs: the second kernel gives each 16 output features to the
// waves of a few workgroups, whose MFMA accumulators run through all active
// experts in float32, and no per-route rows are written or re-read.
//
// What bounds it is reading the active experts' weights once; everything
// else is arranged to stay out of that stream's way.  Weight rows go from
// memory straight into the row operand of v_mfma_f32_16x16x32_bf16, the
// tokens (16 per column tile, CT tiles) sit in the column operand.  MXFP8
// codes are widened to bf16 in registers (v_cvt_scalef32_pk_bf16_fp8: code
// times block scale, exact in bf16), the activations stay bf16.
//
// Inside the first launch the router comes before everything else.  Its work
// (16 experts x 1024 of K per unit) is claimed from a counter by whichever
// workgroups run, so it never depends on a workgroup that has not started;
// the workgroup that finishes the last unit adds the partial logits (in
// order), ranks the tokens, writes the slot list and publishes it; every
// workgroup then goes through its share of (slot, 16 features) items.  The
// wait for the list is bounded: after about a second a workgroup gives up,
// counts a time-out and leaves.  Data that crosses workgroups inside a launch
// goes through device-coherent accesses (the XCDs' L2s are not coherent).
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
constexpr int kUnitSteps = kWaves;    // 128-wide steps per router unit, one per wave

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

// The thread index, opaque to the compiler: what one phase of the first launch
// derives from it is computed in that phase.  Hoisted out of the phases' loops,
// those values pushed the streaming loop's registers into spills.
__device__ __forceinline__ int phase_thread() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// ------------------------------------------------------------ the stream --
// One 128-wide step of 16 weight rows.  bf16: piece j of lane (row l16,
// group q) holds k = 32 j + 8 q .. +7.  MXFP8: piece p holds the codes of
// k = 64 p + 16 q .. +15, half h of it feeds MFMA 2 p + h; the lane's block
// scale is byte 2 p + q / 2 of the row's 4 scale bytes of the step.
template <bool MX>
struct WStep {
  i32x4 w[MX ? 2 : 4];
  uint32_t s;
};

template <bool MX>
__device__ __forceinline__ void load_w(WStep<MX>& f, __amdgpu_buffer_rsrc_t wr, __amdgpu_buffer_rsrc_t sr,
                                       uint32_t wo, uint32_t so, int step) {
  if (MX) {
#pragma unroll
    for (int p = 0; p < 2; ++p) f.w[p] = __builtin_amdgcn_raw_buffer_load_b128(wr, wo + 64 * p, 128 * step, 0);
    f.s = __builtin_amdgcn_raw_buffer_load_b32(sr, so, 4 * step, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f.w[j] = __builtin_amdgcn_raw_buffer_load_b128(wr, wo + 64 * j, 256 * step, 0);
  }
}

// The step's activations of one column tile, in the weights' order of k.
template <bool MX>
__device__ __forceinline__ void load_a(i32x4 (&a)[4], __amdgpu_buffer_rsrc_t ar, uint32_t ao, int step) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    a[j] = __builtin_amdgcn_raw_buffer_load_b128(ar, ao + (MX ? 128 * (j >> 1) + 16 * (j & 1) : 64 * j), 256 * step, 0);
}
// a lane's first k of a step, in bytes of bf16
template <bool MX>
__device__ __forceinline__ int lane_k(int q) { return MX ? 32 * q : 16 * q; }

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <bool MX>
__device__ __forceinline__ bf16x8 widen(const WStep<MX>& f, int j, int q) {
  if (!MX) return as_bf16x8(f.w[j]);
  const float sc = __uint_as_float(((f.s >> (8 * (2 * (j >> 1) + (q >> 1)))) & 0xffu) << 23);
  const uint32_t lo = (uint32_t)f.w[j >> 1][2 * (j & 1)], hi = (uint32_t)f.w[j >> 1][2 * (j & 1) + 1];
  const bf16x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, sc, false),
                       __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, sc, true),
                       __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, sc, false),
                       __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, sc, true)};
  return __builtin_bit_cast(bf16x8, v);
}

// Buffers of one expert's weight matrix of `elems` elements.
template <bool MX>
__device__ __forceinline__ void expert_rsrc(const void* w, const uint8_t* ws, int64_t e, int64_t elems,
                                            __amdgpu_buffer_rsrc_t& wr, __amdgpu_buffer_rsrc_t& sr) {
  const int64_t bytes = elems * (MX ? 1 : 2);
  wr = buffer_rsrc(static_cast<const uint8_t*>(w) + e * bytes, bytes);
  sr = MX ? buffer_rsrc(ws + e * (elems / 32), elems / 32) : wr;
}

__device__ __forceinline__ uint64_t below(int t) { return t == 0 ? 0ull : (~0ull >> (64 - t)); }

// -------------------------------------------------------------- routing --
struct RouteLds {
  uint64_t mask[kLayerMaxE];            // tokens of each expert
  int32_t slot[kLayerMaxE];             // inclusive sums, then slot and first row
  int32_t pos[kLayerMaxE];
  int32_t id[kLayerMaxRoutes];          // the tokens' choices
  float w[kLayerMaxRoutes];
  int32_t wave_n[kWaves], wave_c[kWaves];
};

template <int NV>
__device__ __forceinline__ void rank_tokens(const LayerArgs& g, RouteLds& s, double* keys, int lane, int wave) {
  const int ep = g.logit_ld;
  for (int t = wave; t < g.M; t += kWaves) {
    double l[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      double v = -INFINITY;
      if (e < g.r.E) {
        float sum = 0.f;
        for (int n = 0; n < g.rsplit; ++n) sum += load_relaxed(g.logits + ((int64_t)n * g.M + t) * ep + e);
        v = sum;
        if (g.r.bias_kind == 1) v += (double)g.rbias[e];
      }
      l[i] = route_logit(v);
    }
    int id;
    float w;
    route_token<NV>(g.r, l, g.rbias, keys + (g.r.groups > 1 ? wave * g.r.E : 0), id, w);
    if (lane < g.r.topk) {
      g.ids[t * g.r.topk + lane] = id;
      g.wts[t * g.r.topk + lane] = w;
      s.id[t * g.r.topk + lane] = id;
      s.w[t * g.r.topk + lane] = w;
      if (id >= 0) atomicOr((unsigned long long*)&s.mask[id], 1ull << t);
    }
  }
}

// The tokens' choices, then the slots: the experts that got a token, in
// ascending order, each with the rows [pos0, pos0 + cnt) of z for its
// tokens in ascending order; the shared experts last, with every token.
template <int NV>
__device__ __forceinline__ void route(const LayerArgs& g, RouteLds& s, double* keys) {
  const int tid = phase_thread(), lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < g.r.E; e += kThreads) s.mask[e] = 0;
  __syncthreads();
  rank_tokens<NV>(g, s, keys, lane, wave);
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
  if (cnt > 0) g.slots[n - 1] = LayerSlot{tid, cnt, c - cnt, 0, m, 0};
  if (tid < g.S) g.slots[nt + tid] = LayerSlot{g.r.E + tid, g.M, ct + tid * g.M, 0, below(g.M), 0};
  __syncthreads();
  for (int i = tid; i < g.M * g.r.topk; i += kThreads) {
    const int e = s.id[i], t = i / g.r.topk;
    if (e < 0) continue;
    const int p = s.pos[e] + __popcll(s.mask[e] & below(t));
    g.rows[p] = t;
    g.roww[p] = s.w[i];
  }
  for (int i = tid; i < g.S * g.M; i += kThreads) {
    g.rows[ct + i] = i % g.M;
    g.roww[ct + i] = 1.0f;
  }
  if (tid == 0) g.sync[kLayerNumSlots] = nt + g.S;
}

// ---------------------------------------------------------- first launch --
constexpr int kKeyBytes = kWaves * kLayerMaxE * 8;

template <int CT>
constexpr int gate_up_lds() {
  constexpr int red = kWaves * CT * 64 * 16;
  constexpr int rt = (int)sizeof(RouteLds) + kKeyBytes;
  return red > rt ? red : rt;
}

// Partial logits of 16 experts over 1024 of K (one 128-wide step per wave).
template <int CT>
__device__ __forceinline__ void router_unit(const LayerArgs& g, int unit, f32x4* red) {
  const int tid = phase_thread(), lane = tid & 63, q = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int e0 = 16 * (unit / g.rsplit), n = unit % g.rsplit;
  const int step = n * kUnitSteps + wave;
  f32x4 acc[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) acc[c] = (f32x4){0.f, 0.f, 0.f, 0.f};
  if (128 * step < g.K) {
    const __amdgpu_buffer_rsrc_t wr = buffer_rsrc(g.wr, (int64_t)g.r.E * g.K * 2);
    const __amdgpu_buffer_rsrc_t ar = buffer_rsrc(g.x, (int64_t)g.M * g.K * 2);
    WStep<false> w;
    load_w<false>(w, wr, wr, e0 + l16 < g.r.E ? (uint32_t)((e0 + l16) * g.K * 2 + 16 * q) : kPast, 0, step);
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int t = 16 * c + l16;
      i32x4 a[4];
      load_a<false>(a, ar, t < g.M ? (uint32_t)(t * g.K * 2 + 16 * q) : kPast, step);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w.w[j]), as_bf16x8(a[j]), acc[c], 0, 0, 0);
    }
  }
#pragma unroll
  for (int c = 0; c < CT; ++c) red[(wave * CT + c) * 64 + lane] = acc[c];
  __syncthreads();
  if (wave < CT) {
    f32x4 sum = red[wave * 64 + lane];
    for (int w = 1; w < kWaves; ++w) sum += red[(w * CT + wave) * 64 + lane];
    const int t = 16 * wave + l16;   // sum[r]: expert e0 + 4 q + r, token t
    if (t < g.M) {
      float* o = g.logits + ((int64_t)n * g.M + t) * g.logit_ld + e0 + 4 * q;
#pragma unroll
      for (int r = 0; r < 4; ++r) store_relaxed(o + r, sum[r]);
    }
  }
  __syncthreads();
}

// z of 16 features of one slot: ks waves per operand (gate, up) split K.
template <bool MX, int CT, int D>
__device__ __forceinline__ void gate_up_strip(const LayerArgs& g, const LayerSlot& sl, int f0, int kw, int ut,
                                              bool live, f32x4* red) {
  const int lane = phase_thread() & 63, q = lane >> 4, l16 = lane & 15;
  const int ks = g.ks;
  const int nsteps = g.K / 128;
  const int s0 = kw * nsteps / ks, n = live ? (kw + 1) * nsteps / ks - s0 : 0;
  __amdgpu_buffer_rsrc_t wr, sr;
  expert_rsrc<MX>(g.w1, g.w1s, sl.e, 2ll * g.I * g.K, wr, sr);
  const __amdgpu_buffer_rsrc_t ar = buffer_rsrc(g.x, (int64_t)g.M * g.K * 2);
  const int row = w1_row(f0 + l16, ut != 0, g.I, g.w1_order);
  const uint32_t wo = (uint32_t)row * (uint32_t)g.K * (MX ? 1u : 2u) + 16 * q;
  const uint32_t so = (uint32_t)row * (uint32_t)(g.K / 32);
  uint32_t ao[CT];
  float wt[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int tk = 16 * c + l16;
    ao[c] = kPast;
    wt[c] = 0.f;
    if (live && tk < sl.cnt) {
      ao[c] = (uint32_t)(load_relaxed(g.rows + sl.pos0 + tk) * g.K * 2 + lane_k<MX>(q));
      wt[c] = load_relaxed(g.roww + sl.pos0 + tk);
    }
  }
  f32x4 acc[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) acc[c] = (f32x4){0.f, 0.f, 0.f, 0.f};
  WStep<MX> w[D];
  i32x4 a[D][CT][4];
  auto load = [&](int d, int it) {
    load_w<MX>(w[d], wr, sr, wo, so, s0 + it);
#pragma unroll
    for (int c = 0; c < CT; ++c) load_a<MX>(a[d][c], ar, ao[c], s0 + it);
  };
  auto mma = [&](int d) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x8 wf = widen<MX>(w[d], j, q);
#pragma unroll
      for (int c = 0; c < CT; ++c)
        acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, as_bf16x8(a[d][c][j]), acc[c], 0, 0, 0);
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < n) load(d, d);
  for (int it = 0; it < n; it += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (it + d < n) mma(d);
      if (it + d + D < n) load(d, it + d + D);
    }
  }
#pragma unroll
  for (int c = 0; c < CT; ++c) red[((ut * ks + kw) * CT + c) * 64 + lane] = acc[c];
  __syncthreads();
  // column tile c of the strip: wave c of its 2 ks waves (or all by the first)
  const int me = ut * ks + kw;
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    if (!live || c % (2 * ks) != me) continue;
    f32x4 gate = red[c * 64 + lane], up = red[(ks * CT + c) * 64 + lane];
    for (int k = 1; k < ks; ++k) {
      gate += red[(k * CT + c) * 64 + lane];
      up += red[((ks + k) * CT + c) * 64 + lane];
    }
    const int tk = 16 * c + l16;
    if (tk < sl.cnt) {
      uint32_t h[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) h[r] = f32_to_bf16_rne(wt[c] * (silu_f32(gate[r]) * up[r]));
      *reinterpret_cast<uint2*>(g.z + (int64_t)(sl.pos0 + tk) * g.I + f0 + 4 * q) =
          make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    }
  }
  __syncthreads();
}

template <bool MX, int CT, int D, int NV>
__global__ void __launch_bounds__(kThreads, CT == 4 ? 2 : 4) layer_gate_up_kernel(LayerArgs g) {
  __shared__ __attribute__((aligned(16))) char smem[gate_up_lds<CT>()];
  __shared__ int s_claim, s_last, s_slots;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  f32x4* red = reinterpret_cast<f32x4*>(smem);

  // the router's units, until none is left
  for (;;) {
    if (threadIdx.x == 0)
      s_claim = __hip_atomic_fetch_add(g.sync + kLayerClaim, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    const int unit = s_claim;
    if (unit >= g.runits) break;
    router_unit<CT>(g, unit, red);
    wait_memory();
    __syncthreads();
    if (threadIdx.x == 0)
      s_last = __hip_atomic_fetch_add(g.sync + kLayerArrived, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
               g.runits - 1;
    __syncthreads();
    if (s_last) {
      RouteLds* rl = reinterpret_cast<RouteLds*>(smem);
      route<NV>(g, *rl, reinterpret_cast<double*>(smem + sizeof(RouteLds)));
      wait_memory();
      __syncthreads();
      if (threadIdx.x == 0)
        __hip_atomic_store(g.sync + kLayerRouted, 1, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
    }
    // Keeps this round's work of thread 0 apart from the next claim's: with no
    // barrier between the two, the compiler may run thread 0 through both
    // while the other lanes of its wave go round without it, and the
    // wave's barriers no longer match the other waves'.
    __syncthreads();
  }

  if (threadIdx.x == 0) {
    int n = 0, ok = 1;
    while (load_relaxed(g.sync + kLayerRouted) == 0) {
      if (++n > kSpinLimit) {
        atomicAdd(g.status, 1);
        ok = 0;
        break;
      }
      __builtin_amdgcn_s_sleep(2);
    }
    s_slots = ok ? load_relaxed(g.sync + kLayerNumSlots) : 0;
  }
  __syncthreads();
  const int nslots = s_slots;

  const int nh = kWaves / (2 * g.ks);             // strips a workgroup takes at once
  const int h = wave / (2 * g.ks), ut = (wave / g.ks) & 1, kw = wave % g.ks;
  const int strips = g.I / 16, per = (strips + nh - 1) / nh;
  for (int64_t item = blockIdx.x; item < (int64_t)nslots * per; item += gridDim.x) {
    const int slot = (int)(item / per);
    const int strip = (int)(item % per) * nh + h;
    const int32_t* rec = reinterpret_cast<const int32_t*>(g.slots + slot);
    LayerSlot sl;
    sl.e = load_relaxed(rec);
    sl.cnt = load_relaxed(rec + 1);
    sl.pos0 = load_relaxed(rec + 2);
    sl.e = __builtin_amdgcn_readfirstlane(sl.e);
    sl.cnt = __builtin_amdgcn_readfirstlane(sl.cnt);
    sl.pos0 = __builtin_amdgcn_readfirstlane(sl.pos0);
    gate_up_strip<MX, CT, D>(g, sl, 16 * strip, kw, ut, strip < strips, red + h * 2 * g.ks * CT * 64);
  }
}

// --------------------------------------------------------- second launch --
// Workgroup (strip, split): the 16 output features of the strip over its
// share of the active slots' features, one contiguous run per wave.  The
// waves' sums meet in LDS in wave order; with more than one split the
// workgroup that arrives last adds the splits' sums in order.
template <bool MX, int CT, int D>
__global__ void __launch_bounds__(kThreads, CT == 4 ? 2 : 4) layer_down_kernel(LayerArgs g) {
  __shared__ __attribute__((aligned(16))) f32x4 red[kWaves * CT * 64];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int strip = blockIdx.x / g.splits, split = blockIdx.x % g.splits;
  // a first launch that timed out published nothing: no rows to add
  const int nslots = g.sync[kLayerRouted] ? g.sync[kLayerNumSlots] : 0;
  const int spe = g.I / 128;                             // steps per slot
  const int64_t total = (int64_t)nslots * spe;
  const int parts = g.splits * kWaves, part = split * kWaves + wave;
  const int64_t s0 = part * total / parts;
  const int n = (int)((part + 1) * total / parts - s0);

  const __amdgpu_buffer_rsrc_t ar = buffer_rsrc(g.z, (int64_t)g.cap * g.I * 2);
  const int row = 16 * strip + l16;
  const uint32_t wo = (uint32_t)row * (uint32_t)g.I * (MX ? 1u : 2u) + 16 * q;
  const uint32_t so = (uint32_t)row * (uint32_t)(g.I / 32);
  // cursor of the next step to load
  int slot = (int)(s0 / spe), step = (int)(s0 % spe);
  __amdgpu_buffer_rsrc_t wr, sr;
  uint32_t ao[CT];
  auto enter = [&]() {
    const LayerSlot& sl = g.slots[slot];
    expert_rsrc<MX>(g.w2, g.w2s, sl.e, (int64_t)g.K * g.I, wr, sr);
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int t = 16 * c + l16;
      ao[c] = (sl.mask >> t) & 1
                  ? (uint32_t)(sl.pos0 + __popcll(sl.mask & below(t))) * (uint32_t)g.I * 2u + lane_k<MX>(q)
                  : kPast;
    }
  };
  f32x4 acc[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) acc[c] = (f32x4){0.f, 0.f, 0.f, 0.f};
  WStep<MX> w[D];
  i32x4 a[D][CT][4];
  auto load = [&](int d) {
    if (step == spe) {
      ++slot;
      step = 0;
      enter();
    }
    load_w<MX>(w[d], wr, sr, wo, so, step);
#pragma unroll
    for (int c = 0; c < CT; ++c) load_a<MX>(a[d][c], ar, ao[c], step);
    ++step;
  };
  auto mma = [&](int d) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x8 wf = widen<MX>(w[d], j, q);
#pragma unroll
      for (int c = 0; c < CT; ++c)
        acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, as_bf16x8(a[d][c][j]), acc[c], 0, 0, 0);
    }
  };
  if (n > 0) enter();
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < n) load(d);
  for (int it = 0; it < n; it += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (it + d < n) mma(d);
      if (it + d + D < n) load(d);
    }
  }
#pragma unroll
  for (int c = 0; c < CT; ++c) red[(wave * CT + c) * 64 + lane] = acc[c];
  __syncthreads();
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  const int t = 16 * wave + l16;           // wave c < CT finishes column tile c
  if (wave < CT)
    for (int k = 0; k < kWaves; ++k) sum += red[(k * CT + wave) * 64 + lane];
  if (g.splits > 1) {
    // [strip][split][token][16] partial sums
    float* p = g.part + ((int64_t)strip * g.splits * g.M + t) * 16 + 4 * q;
    if (wave < CT && t < g.M) {
#pragma unroll
      for (int r = 0; r < 4; ++r) store_relaxed(p + (int64_t)split * g.M * 16 + r, sum[r]);
    }
    wait_memory();
    __syncthreads();
    if (threadIdx.x == 0)
      s_last = __hip_atomic_fetch_add(g.sync + kLayerStrips + strip, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
               g.splits - 1;
    __syncthreads();
    if (s_last && wave < CT && t < g.M) {
      sum = (f32x4){0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < g.splits; ++k)
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[r] += load_relaxed(p + (int64_t)k * g.M * 16 + r);
    }
    if (s_last && threadIdx.x == 0) store_relaxed(g.sync + kLayerStrips + strip, 0);
  }
  if (wave < CT && t < g.M && (g.splits == 1 || s_last)) {
    uint32_t h[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) h[r] = f32_to_bf16_rne(sum[r]);
    *reinterpret_cast<uint2*>(g.out + (int64_t)t * g.K + 16 * strip + 4 * q) =
        make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  }
  // the last workgroup of the launch clears the first launch's counters
  if (threadIdx.x == 0) {
    const int done = __hip_atomic_fetch_add(g.sync + kLayerDone, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (done == (int)gridDim.x - 1) {
      store_relaxed(g.sync + kLayerClaim, 0);
      store_relaxed(g.sync + kLayerArrived, 0);
      store_relaxed(g.sync + kLayerRouted, 0);
      store_relaxed(g.sync + kLayerDone, 0);
    }
  }
}

template <bool MX, int CT, int D>
hipError_t launch(const LayerArgs& g, unsigned grid1, hipStream_t s) {
  if (g.r.E <= 64)
    hipLaunchKernelGGL((layer_gate_up_kernel<MX, CT, D, 1>), dim3(grid1), dim3(kThreads), 0, s, g);
  else if (g.r.E <= 128)
    hipLaunchKernelGGL((layer_gate_up_kernel<MX, CT, D, 2>), dim3(grid1), dim3(kThreads), 0, s, g);
  else
    hipLaunchKernelGGL((layer_gate_up_kernel<MX, CT, D, 8>), dim3(grid1), dim3(kThreads), 0, s, g);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((layer_down_kernel<MX, CT, D>), dim3((unsigned)(g.K / 16 * g.splits)), dim3(kThreads), 0, s, g);
  return hipGetLastError();
}

}  // namespace

// Splits of the second launch: with two workgroups per CU the chip holds
// 512; of 1 .. 8 splits the one whose last round of workgroups is fullest
// (the fewest splits among equals).
int32_t layer_splits(int64_t K) {
  int best = 1;
  double waste = 1e9;
  for (int s = 1; s <= 8; ++s) {
    const int64_t wg = K / 16 * s;
    const double w = (double)((wg + 511) / 512 * 512) / (double)wg;
    if (w < waste - 1e-3) { waste = w; best = s; }
  }
  return best;
}

int32_t layer_router_splits(int64_t K) { return (int32_t)((K / 128 + kUnitSteps - 1) / kUnitSteps); }

hipError_t launch_layer(LayerArgs g, bool mxfp8, hipStream_t s) {
  g.rsplit = layer_router_splits(g.K);
  g.runits = (g.r.E + 15) / 16 * g.rsplit;
  g.splits = layer_splits(g.K);
  g.ks = g.K >= 512 ? 4 : g.K >= 256 ? 2 : 1;
  const int nh = kWaves / (2 * g.ks);
  const int64_t items = (int64_t)g.max_slots * ((g.I / 16 + nh - 1) / nh);
  int64_t grid = items > g.runits ? items : g.runits;
  if (grid > 512) grid = 512;
  const int ct = (g.M + 15) / 16;
  if (mxfp8) {
    if (ct == 1) return launch<true, 1, 3>(g, (unsigned)grid, s);
    if (ct == 2) return launch<true, 2, 2>(g, (unsigned)grid, s);
    return launch<true, 4, 2>(g, (unsigned)grid, s);
  }
  if (ct == 1) return launch<false, 1, 3>(g, (unsigned)grid, s);
  if (ct == 2) return launch<false, 2, 2>(g, (unsigned)grid, s);
  return launch<false, 4, 2>(g, (unsigned)grid, s);
}

}  // namespace moe

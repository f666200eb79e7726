// The norms before and after a block with its gate and residual scale:
//   u = b rb w_post,  rb = 1 / sqrt(mean b^2 + eps)      (or u = b)
//   x' = res_scale x + gate u,  h = x' rx w_pre,  rx = 1 / sqrt(mean x'^2 + eps)
// and the gradients of both, at the stored x'.
//
// One pass over the data: a row stays in registers between its statistics and
// its results, 8 consecutive values (a 16-byte load of bf16) a thread and chunk,
// up to NC chunks a thread.  TPR threads take a row (a wave: no barrier; more:
// one barrier a statistic).  A workgroup takes rows at a stride, the weights
// (and in the backward the sums over its rows) in registers throughout, and
// loads its next row while it works on this one.
//
// Bound by memory: the backward of 8192 x 6144 bf16 moves 604 MB in 124 us, 4.9
// TB/s, what a large copy reaches, and adds its workgroups' sums in 5 us more; the
// forward of 8192 x 4096 moves 268 MB in 42 us, some of it from the last-level
// cache.  A single token costs 4 us, the latency of its loads and two statistics.
#include "device_common.h"
#include "kernels.h"
#include "lanes.h"

namespace moe {
namespace {

// 8 consecutive values of float32 or bf16, as loaded.
template <bool F32>
struct Raw8 {
  i32x4 v[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const i32x4* q = reinterpret_cast<const i32x4*>(static_cast<const char*>(p) + i * (F32 ? 4 : 2));
#pragma unroll
    for (int j = 0; j < (F32 ? 2 : 1); ++j) v[j] = q[j];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < (F32 ? 2 : 1); ++j) v[j] = (i32x4){0, 0, 0, 0};
  }
  __device__ __forceinline__ float get(int k) const {
    if constexpr (F32) return __uint_as_float((uint32_t)v[k / 4][k % 4]);
    const uint32_t w = (uint32_t)v[0][k / 2];
    return __uint_as_float(k & 1 ? w & 0xffff0000u : w << 16);
  }
};

template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&f)[8]) {
  i32x4* q = reinterpret_cast<i32x4*>(static_cast<char*>(p) + i * (F32 ? 4 : 2));
  if constexpr (F32) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      i32x4 v;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = (int)__float_as_uint(f[4 * j + k]);
      q[j] = v;
    }
  } else {
    i32x4 v;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = (int)bf16_pack2(f[2 * k], f[2 * k + 1]);
    q[0] = v;
  }
}

// 8 weights (1 without an array).
__device__ __forceinline__ void weights8(const void* p, bool bf16, int i, float (&w)[8]) {
  if (!p) {
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = 1.f;
  } else if (bf16) {
    Raw8<false> r;
    r.load(p, i);
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = r.get(k);
  } else {
    Raw8<true> r;
    r.load(p, i);
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = r.get(k);
  }
}

// Sums of N values over the TPR threads of a row, the same bits in each.
// s: LDS of the workgroup for this statistic, another for every second row: a
// wave that writes one again has passed the next row's barrier, so every wave
// has read it.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*s)[TPR / 64]) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = lanes_sum<64>(v[n]);
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) s[n][wave] = v[n];
    }
    lds_barrier();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = s[n][0];
#pragma unroll
      for (int w = 1; w < TPR / 64; ++w) v[n] += s[n][w];
    }
  }
}

template <int TPR>
constexpr int threads_of() {
  return TPR < 256 ? 256 : TPR;
}

template <bool XF, int TPR, int NC>
__global__ void __launch_bounds__(threads_of<TPR>()) norm_forward_kernel(NormArgs a) {
  constexpr int RW = threads_of<TPR>() / TPR;   // rows of a workgroup at a time
  __shared__ __attribute__((aligned(16))) float s_b[2][1][TPR / 64], s_x[2][1][TPR / 64];
  const int c0 = threadIdx.x % TPR;
  const bool block = a.block != nullptr, post = a.w_post != nullptr, pre = a.w_pre != nullptr;
  float wu[NC][8], wh[NC][8];                   // w_post times the channels' gate; w_pre
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int k = 8 * (c0 + TPR * j);
    if (k >= a.K) continue;
    weights8(a.w_post, a.wbf16, k, wu[j]);
    weights8(a.w_pre, a.wbf16, k, wh[j]);
    if (a.gate_kind == 1) {
      float g[8];
      weights8(a.gate, a.wbf16, k, g);
#pragma unroll
      for (int q = 0; q < 8; ++q) wu[j][q] *= g[q];
    }
  }
  const float inv_k = 1.0f / (float)a.K;
  Raw8<XF> x[NC];
  Raw8<false> b[NC];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int k = 8 * (c0 + TPR * j);
      x[j].zero();
      b[j].zero();
      if (k < a.K && r < a.M) {
        x[j].load(a.x, r * a.K + k);
        if (block) b[j].load(a.block, r * a.K + k);
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * RW;
  int64_t r = (int64_t)blockIdx.x * RW + threadIdx.x / TPR;
  load(r);
  for (int odd = 0; r < a.M; r += step, odd ^= 1) {
    float y[NC][8];
    float u[NC][8];
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        y[j][q] = x[j].get(q);
        u[j][q] = b[j].get(q);
      }
    load(r + step);
    if (block) {
      float scale = 1.f;
      if (post) {
        float v[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int q = 0; q < 8; ++q) v[0] += u[j][q] * u[j][q];
        row_sums<TPR, 1>(v, s_b[odd]);
        scale = __builtin_amdgcn_rsqf(v[0] * inv_k + a.eps);
      }
      if (a.gate_kind == 2) scale *= static_cast<const float*>(a.gate)[r];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int k = 8 * (c0 + TPR * j);
        if (k >= a.K) continue;
#pragma unroll
        for (int q = 0; q < 8; ++q) y[j][q] = a.res_scale * y[j][q] + scale * u[j][q] * wu[j][q];
        store8<XF>(a.x_out, r * a.K + k, y[j]);
      }
    }
    if (pre) {
      float v[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int q = 0; q < 8; ++q) v[0] += y[j][q] * y[j][q];
      row_sums<TPR, 1>(v, s_x[odd]);
      const float rx = __builtin_amdgcn_rsqf(v[0] * inv_k + a.eps);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int k = 8 * (c0 + TPR * j);
        if (k >= a.K) continue;
#pragma unroll
        for (int q = 0; q < 8; ++q) y[j][q] = y[j][q] * rx * wh[j][q];
        store8<false>(a.h, r * a.K + k, y[j]);
      }
    }
  }
}

// Backward of one junction, and the sums of dh n and of gate d (b rb) (gate
// per token; else of d (b rb)) over the workgroup's rows into its part of ws.
template <bool XF, int TPR, int NC>
__global__ void __launch_bounds__(threads_of<TPR>()) norm_backward_kernel(NormArgs a) {
  constexpr int NT = threads_of<TPR>(), RW = NT / TPR;
  __shared__ __attribute__((aligned(16))) float s_1[2][3][TPR / 64], s_2[2][1][TPR / 64];
  const int c0 = threadIdx.x % TPR;
  const bool block = a.block != nullptr, post = a.w_post != nullptr, pre = a.w_pre != nullptr;
  // four chunks a thread (K past 8192): the sums go to LDS, and no second row
  // waits, for want of registers (some of the weights still go to scratch and back,
  // 72 bytes a lane for bf16 and 152 for float32 rows, at no cost that shows: 8192 x
  // 12288 252 us, 4.8 TB/s, 8192 x 16384 322 us, 5.0; float32 rows 381 and 487)
  constexpr bool kKeep = NC <= 2;
  __shared__ f32x4 s_acc[kKeep ? 1 : 4 * NC][kKeep ? 1 : TPR];
  float qu[kKeep ? NC : 1][8], qh[kKeep ? NC : 1][8];
  // sums of chunk j += v: of dh n (which 0) or of d (b rb) (1)
  auto add = [&](int j, int which, const float (&v)[8]) {
    if constexpr (kKeep) {
      float(&q)[8] = which ? qu[j] : qh[j];
#pragma unroll
      for (int k = 0; k < 8; ++k) q[k] += v[k];
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f32x4& q = s_acc[4 * j + 2 * which + h][c0];
        q = (f32x4){q[0] + v[4 * h], q[1] + v[4 * h + 1], q[2] + v[4 * h + 2], q[3] + v[4 * h + 3]};
      }
    }
  };
  float wu[NC][8], wh[NC][8];                   // as in the forward; 0 past K
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int k = 8 * (c0 + TPR * j);
    if constexpr (!kKeep) {
#pragma unroll
      for (int q = 0; q < 4; ++q) s_acc[4 * j + q][c0] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      wu[j][q] = wh[j][q] = 0.f;
      if constexpr (kKeep) qu[j][q] = qh[j][q] = 0.f;
    }
    if (k >= a.K) continue;
    weights8(a.w_post, a.wbf16, k, wu[j]);
    weights8(a.w_pre, a.wbf16, k, wh[j]);
    if (a.gate_kind == 1) {
      float g[8];
      weights8(a.gate, a.wbf16, k, g);
#pragma unroll
      for (int q = 0; q < 8; ++q) wu[j][q] *= g[q];
    }
  }
  const float inv_k = 1.0f / (float)a.K;
  struct Row {
    Raw8<XF> x[NC], dy[NC];
    Raw8<false> b[NC], dh[NC];
  };
  Row next;
  auto load = [&](int64_t r) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int k = 8 * (c0 + TPR * j);
      next.x[j].zero();
      next.dy[j].zero();
      next.b[j].zero();
      next.dh[j].zero();
      if (k < a.K && r < a.M) {
        if (pre) next.x[j].load(a.x, r * a.K + k);
        if (a.dx_out) next.dy[j].load(a.dx_out, r * a.K + k);
        if (block) next.b[j].load(a.block, r * a.K + k);
        if (pre) next.dh[j].load(a.dh, r * a.K + k);
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * RW;
  int odd = 0;
  int64_t r = (int64_t)blockIdx.x * RW + threadIdx.x / TPR;
  if (kKeep) load(r);
  for (; r < a.M; r += step, odd ^= 1) {
    if (!kKeep) load(r);
    const Row now = next;
    if (kKeep) load(r + step);
    const auto& x = now.x;
    const auto& dy = now.dy;
    const auto& b = now.b;
    const auto& dh = now.dh;
    // mean squares of x' and b, and the product of w_pre dh with x'
    float v[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NC; ++j) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float xv = x[j].get(q), bv = b[j].get(q);
        v[0] += xv * xv;
        v[1] += wh[j][q] * dh[j].get(q) * xv;
        v[2] += bv * bv;
      }
    }
    row_sums<TPR, 3>(v, s_1[odd]);
    const float rx = pre ? __builtin_amdgcn_rsqf(v[0] * inv_k + a.eps) : 0.f;
    const float rb = post ? __builtin_amdgcn_rsqf(v[2] * inv_k + a.eps) : 1.f;
    const float gate = a.gate_kind == 2 ? static_cast<const float*>(a.gate)[r] : 1.f;
    const float mx = v[1] * inv_k * rx;           // mean of w_pre dh n
    float d[NC][8];
    float w[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int k = 8 * (c0 + TPR * j);
      float o[8], ah[8], au[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float xv = x[j].get(q), bv = b[j].get(q), hv = dh[j].get(q);
        float e = dy[j].get(q);
        const float n = xv * rx;             // (without w_pre: rx is 0, and so are x' and dh here)
        e += rx * (wh[j][q] * hv - n * mx);
        ah[q] = hv * n;
        o[q] = block ? a.res_scale * e : e;
        au[q] = gate * e * (bv * rb);
        e *= wu[j][q];
        w[0] += e * bv;
        d[j][q] = e;
      }
      add(j, 0, ah);
      add(j, 1, au);
      if (k < a.K) store8<XF>(a.dx, r * a.K + k, o);
    }
    if (!block) continue;
    if (post || a.gate_kind == 2) row_sums<TPR, 1>(w, s_2[odd]);
    if (a.gate_kind == 2 && a.dgate && c0 == 0) a.dgate[r] = w[0] * rb;
    const float mb = post ? w[0] * inv_k * rb : 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int k = 8 * (c0 + TPR * j);
      if (k >= a.K) continue;
      float o[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) o[q] = gate * (rb * (d[j][q] - b[j].get(q) * rb * mb));
      store8<false>(a.dblock, r * a.K + k, o);
    }
  }
  // rows of one workgroup side by side: added through LDS, in order
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.K;
  if constexpr (RW == 1) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int k = 8 * (c0 + TPR * j);
      if (k >= a.K) continue;
      if constexpr (kKeep) {
        store8<true>(part, k, qh[j]);
        store8<true>(part, a.K + k, qu[j]);
      } else {
#pragma unroll
        for (int h = 0; h < 4; ++h)
          *reinterpret_cast<f32x4*>(part + (h / 2) * a.K + k + 4 * (h % 2)) = s_acc[4 * j + h][c0];
      }
    }
  } else {
    __shared__ float s_q[RW][2][8 * TPR * NC];
    const int row = threadIdx.x / TPR;
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        s_q[row][0][8 * (c0 + TPR * j) + q] = qh[j][q];
        s_q[row][1][8 * (c0 + TPR * j) + q] = qu[j][q];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.K; i += NT) {
      const int h = i >= a.K, k = i - h * a.K;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < RW; ++w) v += s_q[w][h][k];
      part[i] = v;
    }
  }
}

// The workgroups' sums, added in float64 (their number grows with M): 64 columns a
// workgroup, its waves sharing the parts.
constexpr int kJoinWaves = 16;

__global__ void __launch_bounds__(64 * kJoinWaves) norm_join_kernel(NormArgs a, int nparts) {
  __shared__ double s_v[kJoinWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = blockIdx.x * 64 + lane;
  double v = 0.0;
  if (i < 2 * a.K) {
#pragma unroll 8
    for (int p = wave; p < nparts; p += kJoinWaves) v += a.part[(int64_t)p * 2 * a.K + i];
  }
  s_v[wave][lane] = v;
  __syncthreads();
  if (wave != 0 || i >= 2 * a.K) return;
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kJoinWaves; ++w) v += s_v[w][lane];
  auto put = [&](float* out, int k, double d) {
    const float f = (float)d;
    if (out) out[k] = a.accumulate ? out[k] + f : f;
  };
  auto weight = [&](const void* p, int k) {
    return a.wbf16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[k]) : static_cast<const float*>(p)[k];
  };
  if (i < a.K) {
    put(a.dw_pre, i, v);
    return;
  }
  // the sum of d n: w_post's gradient over the gate, the gate's over w_post
  const int k = i - a.K;
  if (a.gate_kind == 1) put(a.dgate, k, a.w_post && nparts ? v * weight(a.w_post, k) : v);
  put(a.dw_post, k, a.gate_kind == 1 && nparts ? v * weight(a.gate, k) : v);
}

template <bool XF, int TPR, int NC>
hipError_t forward(const NormArgs& a, hipStream_t s) {
  constexpr int NT = threads_of<TPR>(), RW = NT / TPR;
  const int64_t rows = (a.M + RW - 1) / RW, most = 256 * (2048 / NT);   // what is resident at once
  hipLaunchKernelGGL((norm_forward_kernel<XF, TPR, NC>), dim3((unsigned)(rows < most ? rows : most)), dim3(NT), 0, s,
                     a);
  return hipGetLastError();
}

template <bool XF>
hipError_t forward_of(const NormArgs& a, hipStream_t s) {
  if (a.K <= 512) return forward<XF, 64, 1>(a, s);
  if (a.K <= 1024) return forward<XF, 64, 2>(a, s);
  if (a.K <= 2048) return forward<XF, 256, 1>(a, s);
  if (a.K <= 4096) return forward<XF, 256, 2>(a, s);
  if (a.K <= 8192) return forward<XF, 512, 2>(a, s);
  return forward<XF, 1024, 2>(a, s);
}

// Threads of a row in the backward, by K.
int backward_tpr(int64_t K) { return K <= 1024 ? 64 : K <= 4096 ? 256 : 512; }

template <bool XF, int TPR, int NC>
hipError_t backward(const NormArgs& a, int blocks, hipStream_t s) {
  if (blocks > 0) {
    hipLaunchKernelGGL((norm_backward_kernel<XF, TPR, NC>), dim3((unsigned)blocks), dim3(threads_of<TPR>()), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.dw_pre && !a.dw_post && (!a.dgate || a.gate_kind != 1)) return hipSuccess;
  hipLaunchKernelGGL(norm_join_kernel, dim3((unsigned)((2 * a.K + 63) / 64)), dim3(64 * kJoinWaves), 0, s, a, blocks);
  return hipGetLastError();
}

template <bool XF>
hipError_t backward_of(const NormArgs& a, int blocks, hipStream_t s) {
  if (a.K <= 512) return backward<XF, 64, 1>(a, blocks, s);
  if (a.K <= 1024) return backward<XF, 64, 2>(a, blocks, s);
  if (a.K <= 2048) return backward<XF, 256, 1>(a, blocks, s);
  if (a.K <= 4096) return backward<XF, 256, 2>(a, blocks, s);
  if (a.K <= 8192) return backward<XF, 512, 2>(a, blocks, s);
  return backward<XF, 512, 4>(a, blocks, s);
}

}  // namespace

// Workgroups of the backward, each with sums of its own that are added afterwards:
// what is resident at once, one of 512 threads or two of 256 a CU (8192 x 4096
// bf16: 512 workgroups 90 us, 256 107, 768 101; 8192 x 6144, whose rows take 512
// threads: 256 workgroups 128 us, 512 134, 128 207).  A workgroup adds its rows in
// float32, whose rounding may be off in one direction throughout (equal rows): n in
// turn by up to n / 2 half steps of the sum.  So none takes more than kRun; past that
// there are more rounds of workgroups (of 64 instead of 128 in turn 17000 x 6144 took
// 259 us, not 248).
int32_t norm_backward_blocks(int64_t M, int64_t K) {
  constexpr int64_t kRun = 128;
  const int tpr = backward_tpr(K), rw = tpr < 256 ? 256 / tpr : 1;
  const int64_t rows = (M + rw - 1) / rw;
  const int64_t most = tpr <= 256 ? 512 : 256;
  return (int32_t)(rows < most ? rows : (rows + most * kRun - 1) / (most * kRun) * most);
}

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
  return a.xf32 ? forward_of<true>(a, s) : forward_of<false>(a, s);
}

hipError_t launch_block_norm_backward(const NormArgs& a, hipStream_t s) {
  const int blocks = norm_backward_blocks(a.M, a.K);
  return a.xf32 ? backward_of<true>(a, blocks, s) : backward_of<false>(a, blocks, s);
}

}  // namespace moe

// The orthogonalised update of the experts' matrices by Newton-Schulz steps:
//   X = U / (|U|_F + eps), then  X <- X (a I + B),  B = b A + c A^2,  A = X^T X
// on X [n, m] with n >= m (U itself, or its transpose).
//
// Three products a step, all of the form C[q][p] = sum_k P[p][k] Q[q][k] with
// the contraction contiguous in both operands: A from X^T (kept beside X), A^2
// from A (symmetric), X B from X and B (symmetric).  A and B are symmetric, so
// only the tiles on and above the diagonal are computed, and stored twice:
// 3 m^2 n + m^3 operations a step.
//
// Precision.  The steps multiply a singular value far below the largest by
// about a each time, and what rounding adds in its direction with it, so bf16
// operands (8 bits) leave errors of 1 to 9%.  Here operands are float16 (11
// bits), scaled by powers of two to its range; the term a X takes X in two
// pieces, float16 and the rest in float16 times 2^11 (22 bits); and the
// diagonals of A and B, which hold most of them where X is near orthogonal,
// stay in float32 outside the products:
//   A = D + O, A^2 = O O + D O + O D + D^2,  X (a I + B) = X (a I + D_B) + X O_B.
// What is left is 1e-4 to 1.4e-3 of the result (2-norm; Gaussian, low-rank and
// decaying spectra, 256 x 256 to 4096 x 64, 5 steps), under the 1.7e-3 of its
// rounding to bf16.
#include <math.h>

#include <type_traits>

#include "device_common.h"
#include "kernels.h"
#include "tile_common.h"

namespace moe {
namespace ortho {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t f32_to_f16(float f) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f);
}
__device__ __forceinline__ float f16_to_f32(uint32_t u) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)u);
}
__device__ __forceinline__ float half_of(const uint2& v, int h) {
  return f16_to_f32((h & 2 ? v.y : v.x) >> (h & 1 ? 16 : 0));
}

// 2^s
__host__ __device__ __forceinline__ float pow2(int s) { return ldexpf(1.0f, s); }

constexpr float kLow = 2048.f;   // the second piece of X is the rest times this

// Matrices in the workspace: m and n padded to mp and np (multiples of the
// tile) with zeros, which the steps keep.
struct Mats {
  int32_t E, np, mp;
  double* part;          // [E][kOrthoNormBlocks]
  uint16_t* hi[2];       // X [np][mp], first piece; of this step and of the next
  uint16_t* lo[2];       // second piece
  uint16_t* xt;          // X^T [mp][np], first piece
  uint16_t* a;           // off-diagonal part of A [mp][mp]
  uint16_t* b;           // of B
  float* da;             // diagonals [mp]
  float* db;
};

// ------------------------------------------------------------ norm, input --

// Sums of squares: kOrthoNormBlocks workgroups a matrix.
template <bool BF16>
__global__ void __launch_bounds__(256) ortho_norm_kernel(const void* u, int64_t per, double* part) {
  const int e = blockIdx.y;
  const int64_t base = (int64_t)e * per;
  const int64_t step = (int64_t)gridDim.x * 256;
  double s = 0.0;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < per; i += step) {
    const double v = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(u)[base + i]) : static_cast<const float*>(u)[base + i];
    s += v * v;
  }
  __shared__ double s_v[4];
#pragma unroll
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) s_v[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) part[(int64_t)e * gridDim.x + blockIdx.x] = (s_v[0] + s_v[1]) + (s_v[2] + s_v[3]);
}

// X and X^T from U, 64 x 64 values a workgroup: U [N, K] is X (wide = 0) or X^T.
template <bool BF16>
__global__ void __launch_bounds__(256) ortho_input_kernel(const void* u, int N, int K, int wide, double eps,
                                                          float scale, Mats M) {
  __shared__ float s_v[64][65];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int np = M.np, mp = M.mp;
  const int rows = wide ? mp : np, cols = wide ? np : mp;   // U, padded
  const int tc = cols / 64;
  const int64_t tiles = (int64_t)(rows / 64) * tc;
  const int e = (int)(blockIdx.x / tiles);
  const int t = (int)(blockIdx.x % tiles);
  const int r0 = t / tc * 64, c0 = t % tc * 64;
  double s = M.part[(int64_t)e * kOrthoNormBlocks + lane];
  static_assert(kOrthoNormBlocks == 64, "a lane each");
#pragma unroll
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  const double f = scale / (sqrt(s) + eps);
  // the pieces in U's own order
  const int64_t base = (int64_t)e * N * K;
  const int64_t at = (int64_t)e * np * mp;
  for (int i = wave; i < 64; i += 4) {
    const int r = r0 + i, c = c0 + lane;
    float v = 0.f;
    if (r < N && c < K) {
      const int64_t p = base + (int64_t)r * K + c;
      v = (float)((BF16 ? bf16_to_f32(static_cast<const uint16_t*>(u)[p]) : static_cast<const float*>(u)[p]) * f);
    }
    s_v[i][lane] = v;
    const uint32_t h = f32_to_f16(v);
    if (wide) {
      M.xt[at + (int64_t)r * np + c] = (uint16_t)h;
    } else {
      M.hi[0][at + (int64_t)r * mp + c] = (uint16_t)h;
      M.lo[0][at + (int64_t)r * mp + c] = (uint16_t)f32_to_f16((v - f16_to_f32(h)) * kLow);
    }
  }
  __syncthreads();
  for (int i = wave; i < 64; i += 4) {
    const int r = c0 + i, c = r0 + lane;   // of the transpose
    const float v = s_v[lane][i];
    const uint32_t h = f32_to_f16(v);
    if (wide) {
      M.hi[0][at + (int64_t)r * mp + c] = (uint16_t)h;
      M.lo[0][at + (int64_t)r * mp + c] = (uint16_t)f32_to_f16((v - f16_to_f32(h)) * kLow);
    } else {
      M.xt[at + (int64_t)r * np + c] = (uint16_t)h;
    }
  }
}

// --------------------------------------------------------------- products --

enum Product { kGram = 0, kSquare = 1, kApply = 2 };

struct StepArgs {
  Mats M;
  int32_t cur;            // which of hi and lo holds X
  int32_t last;           // the step's result is the output
  float ca, cb, cc;       // the step's coefficients
  float in, out;          // products -> values, values -> what is stored
  float aux;              // kSquare: stored A -> values; kApply: stored X -> values
  // output
  uint16_t* y;            // bf16 [E, N, K]
  int32_t N, K, wide;
  float scale;
  int32_t chunk;          // consecutive tiles of an XCD
  int64_t total;          // tiles
};

// Tile of C: T x T, waves WI (along p) x WJ (along q) of TI x TJ MFMA tiles.
template <int T>
struct Shape;
template <>
struct Shape<256> {
  static constexpr int WI = 2, WJ = 4, TI = 4, TJ = 2;
};
template <>
struct Shape<128> {
  static constexpr int WI = 2, WJ = 2, TI = 2, TJ = 2;
};
template <>
struct Shape<64> {
  static constexpr int WI = 2, WJ = 2, TI = 1, TJ = 1;
};

constexpr int kBK = 64;   // contraction of a slice

template <int T, int MODE>
__global__ void __launch_bounds__(64 * Shape<T>::WI * Shape<T>::WJ, T == 256 ? 2 : T == 128 ? 2 : 4)
    ortho_product_kernel(StepArgs a) {
  using S = Shape<T>;
  constexpr int WI = S::WI, WJ = S::WJ, TI = S::TI, TJ = S::TJ, NW = WI * WJ;
  static_assert(32 * WI * TI == T && 32 * WJ * TJ == T, "the waves cover the tile");
  constexpr int kSlot = T * kBK;          // uint16 elements
  constexpr int L = T / 8 / NW;           // 1 KB loads a wave, operand and slice
  constexpr int NSTEP = kBK / 16;
  __shared__ __attribute__((aligned(1024))) uint16_t smem[5 * kSlot];
  uint16_t* const pbase = smem;               // 3 slots of P
  uint16_t* const qbase = smem + 3 * kSlot;   // 2 slots of Q

  const Mats& M = a.M;
  const int np = M.np, mp = M.mp;
  // block b runs on XCD b % 8: runs of `chunk` tiles go to one XCD
  const int64_t kx = blockIdx.x / tile::NXCD;
  const int64_t tl = ((kx / a.chunk) * tile::NXCD + blockIdx.x % tile::NXCD) * a.chunk + kx % a.chunk;
  if (tl >= a.total) return;
  const int nm = mp / T;
  int e, tp, tq;
  if (MODE == kApply) {
    const int nn = np / T;
    e = (int)(tl / ((int64_t)nn * nm));
    const int r = (int)(tl % ((int64_t)nn * nm));
    tq = r / nm;
    tp = r % nm;
  } else {
    const int nt = nm * (nm + 1) / 2;
    e = (int)(tl / nt);
    int r = (int)(tl % nt);
    tq = 0;
    while (r >= nm - tq) r -= nm - tq++;      // row tq holds the tiles tp >= tq
    tp = tq + r;
  }
  const int p0 = tp * T, q0 = tq * T;
  const int kd = MODE == kGram ? np : mp;     // contraction, also the row length of P and Q
  const uint16_t *P, *Q;
  int64_t qrows;
  if (MODE == kGram) {
    P = Q = M.xt + (int64_t)e * mp * np;
    qrows = mp;
  } else if (MODE == kSquare) {
    P = Q = M.a + (int64_t)e * mp * mp;
    qrows = mp;
  } else {
    P = M.b + (int64_t)e * mp * mp;
    Q = M.hi[a.cur] + (int64_t)e * np * mp;
    qrows = np;
  }
  const int nk = kd / kBK;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave / WJ, wj = wave % WJ;
  const __amdgpu_buffer_rsrc_t pr = buffer_rsrc(P, (int64_t)mp * kd * 2);
  const __amdgpu_buffer_rsrc_t qr = buffer_rsrc(Q, qrows * kd * 2);
  // load i of this wave: slot rows 8 (wave + NW i) .. +7, lane l -> row l / 8,
  // physical chunk l % 8 (lds_off's swizzle: logical chunk ^ (row / 2) % 8)
  uint32_t op[L], oq[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int r = 8 * (wave + NW * i) + lane / 8;
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    op[i] = (uint32_t)(((int64_t)(p0 + r) * kd + 8 * c) * 2);
    oq[i] = (uint32_t)(((int64_t)(q0 + r) * kd + 8 * c) * 2);
  }
  auto issue_p = [&](int kt) {
    uint16_t* slot = pbase + (kt % 3) * kSlot;
#pragma unroll
    for (int i = 0; i < L; ++i) lds_load16(pr, slot + (wave + NW * i) * 512, op[i], kt * kBK * 2);
    issue_order();
  };
  auto issue_q = [&](int kt) {
    uint16_t* slot = qbase + (kt % 2) * kSlot;
#pragma unroll
    for (int i = 0; i < L; ++i) lds_load16(qr, slot + (wave + NW * i) * 512, oq[i], kt * kBK * 2);
    issue_order();
  };

  f32x16 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  i32x4 fp[2][TI], fq[2][TJ];
  auto fload = [&](int fb, int kt, int st) {
    const uint16_t* ps = pbase + (kt % 3) * kSlot;
    const uint16_t* qs = qbase + (kt % 2) * kSlot;
    const int c = 2 * st + (lane >> 5);
#pragma unroll
    for (int i = 0; i < TI; ++i)
      fp[fb][i] = *reinterpret_cast<const i32x4*>(ps + tile::lds_off<kBK>((wi * TI + i) * 32 + (lane & 31), c));
#pragma unroll
    for (int j = 0; j < TJ; ++j)
      fq[fb][j] = *reinterpret_cast<const i32x4*>(qs + tile::lds_off<kBK>((wj * TJ + j) * 32 + (lane & 31), c));
  };
  auto mma = [&](int fb) {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, fp[fb][i]),
                                                           __builtin_bit_cast(f16x8, fq[fb][j]), acc[i][j], 0, 0, 0);
  };

  // prologue: P 0, Q 0 and 1, P 1 and 2; the wait leaves only P's loads of
  // slices 1 and 2 outstanding
  issue_p(0);
  issue_q(0);
  if (nk > 1) { issue_q(1); issue_p(1); }
  if (nk > 2) issue_p(2);
  if (nk > 2) wait_vm<2 * L>();
  else if (nk > 1) wait_vm<L>();
  else wait_vm<0>();
  lds_barrier();
  // slice kt; F 2: slices kt+2 and kt+3 exist, 1: only kt+2, 0: only kt+1, -1:
  // kt is the last
  auto slice = [&](int kt, auto mode) {
    constexpr int F = decltype(mode)::value;
#pragma unroll
    for (int st = 0; st + 1 < NSTEP; ++st) {
      fload((st + 1) & 1, kt, st + 1);
      mma(st & 1);
    }
    if (F >= 0) {
      if (F >= 1) wait_vm<L>();   // slice kt+1 is in; P of kt+2 may fly
      else wait_vm<0>();
      lds_barrier();              // nobody reads slice kt's slots any more
      if (F >= 1) issue_q(kt + 2);
      if (F >= 2) issue_p(kt + 3);
      fload(0, kt + 1, 0);
    }
    mma((NSTEP - 1) & 1);
  };
  fload(0, 0, 0);
  int kt = 0;
  for (; kt + 3 < nk; ++kt) slice(kt, std::integral_constant<int, 2>());
  if (kt + 2 < nk) slice(kt++, std::integral_constant<int, 1>());
  if (kt + 1 < nk) slice(kt++, std::integral_constant<int, 0>());
  slice(kt, std::integral_constant<int, -1>());

  // acc[i][j][4 g + h]: p = p0 + 32 (wi TI + i) + 8 g + 4 (lane / 32) + h,
  // q = q0 + 32 (wj TJ + j) + lane % 32
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int q = q0 + 32 * (wj * TJ + j) + (lane & 31);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int p = p0 + 32 * (wi * TI + i) + 8 * g + 4 * (lane >> 5);
        float v[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) v[h] = acc[i][j][4 * g + h] * a.in;
        if (MODE == kApply) {
          const int64_t at = ((int64_t)e * np + q) * mp + p;
          const uint2 xh = *reinterpret_cast<const uint2*>(M.hi[a.cur] + at);
          const uint2 xl = *reinterpret_cast<const uint2*>(M.lo[a.cur] + at);
          const f32x4 d = *reinterpret_cast<const f32x4*>(M.db + (int64_t)e * mp + p);
#pragma unroll
          for (int h = 0; h < 4; ++h)
            v[h] += (a.ca + d[h]) * ((half_of(xh, h) + half_of(xl, h) * (1.0f / kLow)) * a.aux);
          if (a.last) {
            // X [n, m] is the output [N, K], or its transpose
            const int n = a.wide ? a.K : a.N, m = a.wide ? a.N : a.K;
#pragma unroll
            for (int h = 0; h < 4; ++h)
              if (q < n && p + h < m) {
                const int64_t o = (int64_t)e * a.N * a.K + (a.wide ? (int64_t)(p + h) * a.K + q : (int64_t)q * a.K + p + h);
                a.y[o] = (uint16_t)f32_to_bf16_rne(v[h] * a.scale);
              }
          } else {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const float w = v[h] * a.out;
              hi[h] = f32_to_f16(w);
              lo[h] = f32_to_f16((w - f16_to_f32(hi[h])) * kLow);
              M.xt[((int64_t)e * mp + p + h) * np + q] = (uint16_t)hi[h];
            }
            *reinterpret_cast<uint2*>(M.hi[a.cur ^ 1] + at) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
            *reinterpret_cast<uint2*>(M.lo[a.cur ^ 1] + at) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
          }
        } else {
          const int64_t me = (int64_t)e * mp;
          if (MODE == kSquare) {
            const uint2 o = *reinterpret_cast<const uint2*>(M.a + (me + q) * mp + p);
            const f32x4 dp = *reinterpret_cast<const f32x4*>(M.da + me + p);
            const float dq = M.da[me + q];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const float off = half_of(o, h) * a.aux;   // 0 on the diagonal
              v[h] = p + h == q ? a.cb * dq + a.cc * (v[h] + dq * dq)
                                : a.cb * off + a.cc * (v[h] + (dp[h] + dq) * off);
            }
          }
          uint16_t* C = (MODE == kGram ? M.a : M.b);
          float* D = (MODE == kGram ? M.da : M.db);
          uint32_t s[4];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const bool diag = p + h == q;
            if (diag) D[me + q] = v[h];
            s[h] = diag ? 0u : f32_to_f16(v[h] * a.out);
          }
          *reinterpret_cast<uint2*>(C + (me + q) * mp + p) = make_uint2(s[0] | (s[1] << 16), s[2] | (s[3] << 16));
          if (tp != tq) {
#pragma unroll
            for (int h = 0; h < 4; ++h) C[(me + p + h) * mp + q] = (uint16_t)s[h];
          }
        }
      }
    }
}

template <int T, int MODE>
hipError_t launch_product(StepArgs a, hipStream_t s) {
  const int64_t nm = a.M.mp / T, nn = a.M.np / T;
  a.total = a.M.E * (MODE == kApply ? nm * nn : nm * (nm + 1) / 2);
  // few tiles are dealt evenly, many in runs of 32, a tile for each CU of an XCD
  const int64_t even = (a.total + tile::NXCD - 1) / tile::NXCD;
  a.chunk = (int32_t)(even < tile::kXcdChunk ? even : tile::kXcdChunk);
  const int64_t unit = (int64_t)tile::NXCD * a.chunk;
  const int64_t grid = (a.total + unit - 1) / unit * unit;
  hipLaunchKernelGGL((ortho_product_kernel<T, MODE>), dim3((unsigned)grid), dim3(64 * Shape<T>::WI * Shape<T>::WJ), 0,
                     s, a);
  return hipGetLastError();
}

template <int MODE>
hipError_t product(const StepArgs& a, int T, hipStream_t s) {
  if (T == 256) return launch_product<256, MODE>(a, s);
  if (T == 128) return launch_product<128, MODE>(a, s);
  return launch_product<64, MODE>(a, s);
}

// What m and n are padded to: tiles of 256 where they fill the CUs and the
// padding costs little.
int tile_of(int64_t E, int64_t n, int64_t m) {
  for (int T = 256; T > 64; T /= 2) {
    const int64_t nm = (m + T - 1) / T, nn = (n + T - 1) / T;
    if (E * nm * nn >= 192 && nm * T <= m + m / 8) return T;
  }
  return 64;
}

struct Layout {
  int T;
  int64_t np, mp, hi[2], lo[2], xt, a, b, da, db, part, end;
};

Layout layout(int64_t E, int64_t N, int64_t K) {
  Layout L;
  const int64_t n = N >= K ? N : K, m = N >= K ? K : N;
  L.T = tile_of(E, n, m);
  L.np = (n + L.T - 1) / L.T * L.T;
  L.mp = (m + L.T - 1) / L.T * L.T;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  L.part = take(8 * E * kOrthoNormBlocks);
  for (int i = 0; i < 2; ++i) {
    L.hi[i] = take(2 * E * L.np * L.mp);
    L.lo[i] = take(2 * E * L.np * L.mp);
  }
  L.xt = take(2 * E * L.np * L.mp);
  L.a = take(2 * E * L.mp * L.mp);
  L.b = take(2 * E * L.mp * L.mp);
  L.da = take(4 * E * L.mp);
  L.db = take(4 * E * L.mp);
  L.end = at;
  return L;
}

}  // namespace ortho

int64_t ortho_ws_bytes(int64_t E, int64_t N, int64_t K) { return ortho::layout(E, N, K).end; }

// Singular values start in [0, 1]; one in [0, u] goes to |a s + b s^3 + c s^5|,
// whose largest value is at u or where the derivative is 0.  X's entries stay
// under u, A's under u^2, B's under the largest |b s^2 + c s^4|; each is scaled
// to at most 2^14, a quarter of float16's range, which leaves room for what
// rounding adds.
bool ortho_scales(const OrthoArgs& o, int32_t (*s)[3]) {
  double u = 1.0;
  auto power = [](double v) { return 14 - (int)ceil(log2(v > 1e-6 ? v : 1e-6)); };
  for (int i = 0; i < o.steps; ++i) {
    const double a = o.coef[i][0], b = o.coef[i][1], c = o.coef[i][2];
    if (!(a - a == 0.0) || !(b - b == 0.0) || !(c - c == 0.0) || !(u <= 4096.0)) return false;
    auto f = [&](double x) { return fabs(x * (a + x * x * (b + x * x * c))); };
    auto g = [&](double x) { return fabs(x * x * (b + x * x * c)); };
    double next = f(u), most = g(u);
    // a + 3 b y + 5 c y^2 = 0 and b + 2 c y = 0, y = s^2
    auto at = [&](double y) {
      if (y > 0.0 && y < u * u) {
        next = fmax(next, f(sqrt(y)));
        most = fmax(most, g(sqrt(y)));
      }
    };
    if (c != 0.0) {
      const double d = 9 * b * b - 20 * a * c;
      if (d >= 0.0) {
        at((-3 * b + sqrt(d)) / (10 * c));
        at((-3 * b - sqrt(d)) / (10 * c));
      }
      at(-b / (2 * c));
    } else if (b != 0.0) {
      at(-a / (3 * b));
    }
    s[i][0] = power(u);
    s[i][1] = power(u * u);
    s[i][2] = power(most);
    if (!(most <= 1e9)) return false;
    u = next;
  }
  return u <= 4096.0;
}

hipError_t launch_orthogonalize(const OrthoArgs& o, hipStream_t st) {
  using namespace ortho;
  const Layout L = layout(o.E, o.N, o.K);
  int32_t s[kOrthoMaxSteps][3];
  if (!ortho_scales(o, s)) return hipErrorInvalidValue;
  char* ws = static_cast<char*>(o.ws);
  Mats M{};
  M.E = o.E;
  M.np = (int32_t)L.np;
  M.mp = (int32_t)L.mp;
  M.part = reinterpret_cast<double*>(ws + L.part);
  for (int i = 0; i < 2; ++i) {
    M.hi[i] = reinterpret_cast<uint16_t*>(ws + L.hi[i]);
    M.lo[i] = reinterpret_cast<uint16_t*>(ws + L.lo[i]);
  }
  M.xt = reinterpret_cast<uint16_t*>(ws + L.xt);
  M.a = reinterpret_cast<uint16_t*>(ws + L.a);
  M.b = reinterpret_cast<uint16_t*>(ws + L.b);
  M.da = reinterpret_cast<float*>(ws + L.da);
  M.db = reinterpret_cast<float*>(ws + L.db);
  const int wide = o.N < o.K;
  const int64_t per = (int64_t)o.N * o.K;
  hipError_t e;
  {
    const dim3 g(kOrthoNormBlocks, (unsigned)o.E);
    if (o.bf16)
      hipLaunchKernelGGL(ortho_norm_kernel<true>, g, dim3(256), 0, st, o.update, per, M.part);
    else
      hipLaunchKernelGGL(ortho_norm_kernel<false>, g, dim3(256), 0, st, o.update, per, M.part);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const dim3 gi((unsigned)(o.E * (L.np / 64) * (L.mp / 64)));
    const float sc = pow2(s[0][0]);
    if (o.bf16)
      hipLaunchKernelGGL(ortho_input_kernel<true>, gi, dim3(256), 0, st, o.update, o.N, o.K, wide, (double)o.eps, sc, M);
    else
      hipLaunchKernelGGL(ortho_input_kernel<false>, gi, dim3(256), 0, st, o.update, o.N, o.K, wide, (double)o.eps, sc,
                         M);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  StepArgs a{};
  a.M = M;
  a.y = o.out;
  a.N = o.N;
  a.K = o.K;
  a.wide = wide;
  a.scale = o.scale;
  for (int i = 0; i < o.steps; ++i) {
    const int sx = s[i][0], sa = s[i][1], sb = s[i][2];
    a.cur = i & 1;
    a.last = i + 1 == o.steps;
    a.ca = o.coef[i][0];
    a.cb = o.coef[i][1];
    a.cc = o.coef[i][2];
    a.in = pow2(-2 * sx);
    a.out = pow2(sa);
    if ((e = product<kGram>(a, L.T, st)) != hipSuccess) return e;
    a.in = pow2(-2 * sa);
    a.out = pow2(sb);
    a.aux = pow2(-sa);
    if ((e = product<kSquare>(a, L.T, st)) != hipSuccess) return e;
    a.in = pow2(-sx - sb);
    a.out = a.last ? 1.0f : pow2(s[i + 1][0]);
    a.aux = pow2(-sx);
    if ((e = product<kApply>(a, L.T, st)) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe

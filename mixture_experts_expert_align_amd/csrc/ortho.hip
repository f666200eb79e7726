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
// pieces, float16 and the rest in float16 times 2^11 (22 bits), and so do X B up to
// m = 512 and, up to m = 64, also X^T X, and X B with B in two pieces too (the
// smaller m, the more one entry's rounding counts); and the diagonals of A and B,
// which hold most of them where X is near orthogonal, stay in float32 outside the
// products:
//   A = D + O, A^2 = O O + D O + O D + D^2,  X (a I + B) = X (a I + D_B) + X O_B.
// What is left of 5 steps' result is (2-norm, relative; Gaussian matrices, decaying
// spectra, and r singular values of 1 over others of 3e-2 to 1e-5, the worst of
// all) up to 1.4e-3 for m up to 64, 1.1e-3 up to 512 and 2e-3 past it, a worst
// case about as large as the rounding to bf16 that follows (1.7e-3).
//
// Large matrices are bound by the matrix units and by what the epilogues move: 8 of
// 4096 x 6144 take 841 us for A, 593 for B and 1555 for X B a step (1.04, 0.96 and
// 1.06 PFLOP/s of what the tiles compute; 820, 577 and 1524 on another card), A and B
// 7 to 8% of the whole in a last round that fills a quarter of the CUs.  A tile of X B
// is 1.4 us a slice and 37 us besides, in which 650 KB of X come and go; workgroups
// that start at different times, requests a slice earlier, tiles of 128 (11% slower)
// and tiles of two products in one launch (9 to 17%) did not shorten it.
// Small ones are bound by the latency of three dependent launches a step (8 of 256 x
// 512: 5.6, 4.6 and 7.1 us), m <= 64 of one (64 x 4096: 13.4 us).
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
  float* gpart;          // [E][tiles of 64 of A][splits][64][64]: sums over parts of n
  int32_t* gdone;        // [E][tiles]: how many of them are there, 0 between the steps
  int32_t gtiles;        // E tiles
};

// ------------------------------------------------------------ norm, input --

// Sums of squares: kOrthoNormBlocks workgroups a matrix, 16 bytes a load between
// the first and the last aligned address of the matrix, the ends by themselves.
// (One value a load reached 1.2 TB/s.)
template <bool BF16>
__global__ void __launch_bounds__(1024) ortho_norm_kernel(const void* u, int64_t per, double* part) {
  constexpr int EL = BF16 ? 2 : 4, V = 16 / EL;   // bytes of a value, values of a load
  const int e = blockIdx.y;
  const char* base = static_cast<const char*>(u) + (int64_t)e * per * EL;
  const int64_t head = min((int64_t)((16 - ((uintptr_t)base & 15)) & 15) / EL, per);
  const int64_t nv = (per - head) / V;
  auto value = [&](int64_t i) {
    const char* p = base + i * EL;
    return BF16 ? bf16_to_f32(*reinterpret_cast<const uint16_t*>(p)) : *reinterpret_cast<const float*>(p);
  };
  double s = 0.0;
  const i32x4* body = reinterpret_cast<const i32x4*>(base + head * EL);
  const int64_t step = (int64_t)gridDim.x * 1024;
  auto add = [&](const i32x4& x) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w = (uint32_t)x[k];
      const double a = __uint_as_float(BF16 ? w << 16 : w);
      s += a * a;
      if (BF16) {
        const double b = __uint_as_float(w & 0xffff0000u);
        s += b * b;
      }
    }
  };
  int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x;
  for (; i + 3 * step < nv; i += 4 * step) {
    i32x4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = body[i + k * step];
#pragma unroll
    for (int k = 0; k < 4; ++k) add(x[k]);
  }
  for (; i < nv; i += step) add(body[i]);
  if (blockIdx.x == 0) {
    const int64_t tail = head + nv * V;
    if (threadIdx.x < head) {
      const double a = value(threadIdx.x);
      s += a * a;
    }
    if (tail + threadIdx.x < per) {
      const double a = value(tail + threadIdx.x);
      s += a * a;
    }
  }
  __shared__ double s_v[16];
#pragma unroll
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) s_v[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 16; ++w) s += s_v[w];
    part[(int64_t)e * gridDim.x + blockIdx.x] = s;
  }
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
  // the pieces in U's own order; all values requested before the first is stored
  const int64_t base = (int64_t)e * N * K;
  const int64_t at = (int64_t)e * np * mp;
  float v[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int r = min(r0 + wave + 4 * k, N - 1), c = min(c0 + lane, K - 1);   // past the matrix: not taken
    const int64_t p = base + (int64_t)r * K + c;
    v[k] = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(u)[p]) : static_cast<const float*>(u)[p];
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int i = wave + 4 * k, r = r0 + i, c = c0 + lane;
    const float x = r < N && c < K ? (float)(v[k] * f) : 0.f;
    s_v[i][lane] = x;
    const uint32_t h = f32_to_f16(x);
    if (wide) {
      M.xt[at + (int64_t)r * np + c] = (uint16_t)h;
    } else {
      M.hi[0][at + (int64_t)r * mp + c] = (uint16_t)h;
      M.lo[0][at + (int64_t)r * mp + c] = (uint16_t)f32_to_f16((x - f16_to_f32(h)) * kLow);
    }
  }
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < M.gtiles; i += (int64_t)gridDim.x * 256) M.gdone[i] = 0;
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

enum Product { kGram = 0, kSquare = 1, kApply = 2, kApplyBoth = 3 };   // both pieces of X in X B

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
  int32_t vec;            // rows of y take 16-byte stores
  float scale;
  int32_t chunk;          // consecutive tiles of an XCD
  int64_t total;          // tiles
  int32_t splits;         // kGram, tiles of 64: workgroups that share a tile's contraction
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
constexpr int kBand = 4;  // rows of tiles that are gone through together

// 8 values (or what the row has of them) of output row `row` from column c on.
__device__ __forceinline__ void store_row(const StepArgs& a, int64_t row, int c, const i32x4& s) {
  uint16_t* o = a.y + row * a.K + c;
  if (a.vec && c + 8 <= a.K) {
    *reinterpret_cast<i32x4*>(o) = s;
    return;
  }
#pragma unroll
  for (int h = 0; h < 8; ++h)
    if (c + h < a.K) o[h] = (uint16_t)((uint32_t)s[h / 2] >> (h & 1 ? 16 : 0));
}

template <int T, int MODE>
__global__ void __launch_bounds__(64 * Shape<T>::WI * Shape<T>::WJ, T == 256 ? 2 : T == 128 ? 2 : 4)
    ortho_product_kernel(StepArgs a) {
  using S = Shape<T>;
  constexpr bool kXB = MODE == kApply || MODE == kApplyBoth, kBoth = MODE == kApplyBoth;
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
  int64_t tl = ((kx / a.chunk) * tile::NXCD + blockIdx.x % tile::NXCD) * a.chunk + kx % a.chunk;
  if (tl >= a.total) return;
  constexpr bool kSplit = MODE == kGram && T == 64;   // may share a tile
  const int sp = kSplit ? (int)(tl % a.splits) : 0;
  if (kSplit) tl /= a.splits;
  const int nm = mp / T;
  int e, tp, tq;
  if (kXB) {
    // bands of kBand rows of tiles, column by column: 32 tiles in a row read 4
    // row tiles of X and 8 of B
    const int nn = np / T, per = nn * nm;
    e = (int)(tl / per);
    const int r = (int)(tl % per), band = r / (kBand * nm), in = r % (kBand * nm);
    const int h = min(kBand, nn - band * kBand);
    tp = in / h;
    tq = band * kBand + in % h;
  } else {
    // the same over the tiles tp >= tq: the band from row t has its columns t,
    // t + 1, ... 1, 2, ... up to h rows high
    const int nt = nm * (nm + 1) / 2;
    e = (int)(tl / nt);
    int r = (int)(tl % nt), t = 0, h = min(kBand, nm);
    for (;;) {
      const int in = h * (nm - t) - h * (h - 1) / 2;
      if (r < in) break;
      r -= in;
      t += h;
      h = min(kBand, nm - t);
    }
    tp = t;
    while (r >= min(h, tp - t + 1)) r -= min(h, tp++ - t + 1);
    tq = t + r;
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
  const int ns = kd / kBK;                    // slices; this workgroup's: nk from k0 on
  const int k0 = kSplit ? (int)((int64_t)ns * sp / a.splits) : 0;
  const int nk = kSplit ? (int)((int64_t)ns * (sp + 1) / a.splits) - k0 : kBoth ? 2 * ns : ns;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave / WJ, wj = wave % WJ;
  const __amdgpu_buffer_rsrc_t pr = buffer_rsrc(P, (int64_t)mp * kd * 2);
  const __amdgpu_buffer_rsrc_t qr = buffer_rsrc(Q, qrows * kd * 2);
  // both pieces: X's second, kLow times its value, in the first ns slices
  const __amdgpu_buffer_rsrc_t q2 = kBoth ? buffer_rsrc(M.lo[a.cur] + (int64_t)e * np * mp, qrows * kd * 2) : qr;
  auto column = [&](int kt) { return (kBoth && kt >= ns ? kt - ns : k0 + kt) * kBK * 2; };
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
    for (int i = 0; i < L; ++i) lds_load16(pr, slot + (wave + NW * i) * 512, op[i], column(kt));
    issue_order();
  };
  auto issue_q = [&](int kt) {
    uint16_t* slot = qbase + (kt % 2) * kSlot;
#pragma unroll
    for (int i = 0; i < L; ++i)
      lds_load16(kBoth && kt < ns ? q2 : qr, slot + (wave + NW * i) * 512, oq[i], column(kt));
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
  auto mma = [&](int fb, int i0, int i1) {
#pragma unroll
    for (int i = i0; i < i1; ++i)
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
  // a step's reads for the next step go between its MFMAs, one each
  auto interleave = [&](auto mfmas) {
    constexpr int R = TI + TJ, N = decltype(mfmas)::value;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < R) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    if constexpr (R > N) __builtin_amdgcn_sched_group_barrier(0x100, R - N, 0);
  };
  // slice kt; F 1: slice kt+2 exists, 0: only kt+1, -1: kt is the last
  auto slice = [&](int kt, auto mode) {
    constexpr int F = decltype(mode)::value;
    if (kBoth && kt == ns) {   // (all products of the slices before are in)
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][j][r] *= 1.0f / kLow;
    }
#pragma unroll
    for (int st = 0; st + 1 < NSTEP; ++st) {
      // (P's loads have a slice more to arrive than Q's: issued later, they leave
      // the way to Q's, which cuts 9% of the cycles of a slice)
      if (st == NSTEP - 2 && F >= 1 && kt > 0) issue_p(kt + 2);
      fload((st + 1) & 1, kt, st + 1);
      mma(st & 1, 0, TI);
      interleave(std::integral_constant<int, TI * TJ>());
      __builtin_amdgcn_sched_barrier(0);
    }
    if (F >= 0) {
      mma((NSTEP - 1) & 1, 0, TI / 2);
      __builtin_amdgcn_sched_barrier(0);
      if (F >= 1) wait_vm<L>();   // slice kt+1 is in; P of kt+2 may fly
      else wait_vm<0>();
      lds_barrier();              // nobody reads slice kt's slots any more
      if (F >= 1) issue_q(kt + 2);
      fload(0, kt + 1, 0);
      mma((NSTEP - 1) & 1, TI / 2, TI);
      interleave(std::integral_constant<int, (TI - TI / 2) * TJ>());
      __builtin_amdgcn_sched_barrier(0);
    } else {
      mma((NSTEP - 1) & 1, 0, TI);
    }
  };
  fload(0, 0, 0);
  int kt = 0;
  for (; kt + 2 < nk; ++kt) slice(kt, std::integral_constant<int, 1>());
  if (kt + 1 < nk) slice(kt++, std::integral_constant<int, 0>());
  slice(kt, std::integral_constant<int, -1>());

  // Epilogue through LDS, HR rows q of the tile at a time as float32 rows of T:
  // rows are read back 8 values a thread, finished and stored by whole lines;
  // where the transpose is stored too, the finished 16-bit values take the place
  // of the first of their two 16-byte chunks and are read by columns.  A row's
  // even chunks lie before its odd ones, and chunk i of either at i ^ r ^ (r / 8):
  // 8 rows of a chunk (the accumulators), 8 chunks of a row, and a column of every
  // eighth row all lie in different banks.  (With i ^ r alone the columns met in
  // one, 29000 cycles a tile of 256.)
  constexpr int NT = 64 * NW;
  constexpr int HR = T == 256 ? 128 : T;
  constexpr int CH = T / 4, SW = CH / 2 - 1;
  static_assert(HR * T * 4 <= 5 * kSlot * 2, "the rows fit the slots");
  float* const stage = reinterpret_cast<float*>(smem);
  auto chunk = [&](int r, int c) {
    return stage + r * T + ((((c >> 1) ^ ((r ^ (r >> 3)) & SW)) + (c & 1) * (CH / 2)) << 2);
  };
  const int64_t me = (int64_t)e * mp;
  const bool turned = kXB ? !a.last || a.wide : tp != tq;
#pragma unroll
  for (int hf = 0; hf < T / HR; ++hf) {
    constexpr int UR = T / 8, U = HR * UR / NT;   // units of a row; of a thread
    static_assert(U * NT == HR * UR, "units fill the threads");
    const int u = threadIdx.x % UR, p = p0 + 8 * u;
    auto unit_row = [&](int w) { return (int)threadIdx.x / UR + NT / UR * w; };
    // what is read besides, all of it requested before the rows are written (a
    // load behind another unit's stores would wait for each in turn)
    f16x8 x1[U], x2[kXB ? U : 1];
    float xq[MODE == kSquare ? U : 1];
    if (MODE != kGram) {
#pragma unroll
      for (int w = 0; w < U; ++w) {
        const int q = q0 + hf * HR + unit_row(w);
        if constexpr (kXB) {
          const int64_t at = ((int64_t)e * np + q) * mp + p;
          x1[w] = *reinterpret_cast<const f16x8*>(M.hi[a.cur] + at);
          x2[w] = *reinterpret_cast<const f16x8*>(M.lo[a.cur] + at);
        } else {
          x1[w] = *reinterpret_cast<const f16x8*>(M.a + (me + q) * mp + p);   // 0 on the diagonal
          xq[w] = M.da[me + q];
        }
      }
    }
    lds_barrier();
    // acc[i][j][4 g + h]: p = 32 (wi TI + i) + 8 g + 4 (lane / 32) + h,
    // q = 32 (wj TJ + j) + lane % 32
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int r = 32 * (wj * TJ + j) + (lane & 31) - hf * HR;
      if (32 * (wj * TJ + j) / HR != hf) continue;
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<f32x4*>(chunk(r, 8 * (wi * TI + i) + 2 * g + (lane >> 5))) =
              (f32x4){acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
    }
    lds_barrier();
    if constexpr (kSplit) {
      // the tile's sums over its share of n; the last workgroup of the tile adds all of
      // them, in their order, and goes on alone.  A part is where all can read it
      // before its workgroup is counted.
      if (a.splits > 1) {
        constexpr int kCoherent = 16;   // sc1: past the XCD's own L2, to where all XCDs read
        const __amdgpu_buffer_rsrc_t pr4 = buffer_rsrc(M.gpart + tl * a.splits * (T * T), (int64_t)a.splits * T * T * 4);
        int* const s_last = reinterpret_cast<int*>(smem + 4 * kSlot);
        uint32_t place[U];
#pragma unroll
        for (int w = 0; w < U; ++w) {
          place[w] = (uint32_t)(unit_row(w) * T + 8 * u) * 4;
#pragma unroll
          for (int c = 0; c < 2; ++c)
            __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<const i32x4*>(chunk(unit_row(w), 2 * u + c)), pr4,
                                                   place[w] + 16 * c, sp * T * T * 4, kCoherent);
        }
        wait_vm<0>();
        lds_barrier();
        if (threadIdx.x == 0)
          *s_last = __hip_atomic_fetch_add(M.gdone + tl, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.splits - 1;
        lds_barrier();
        if (!*s_last) return;
        if (threadIdx.x == 0) M.gdone[tl] = 0;
        f32x4 sum[U][2] = {};
        for (int s = 0; s < a.splits; s += 4) {
          i32x4 part[4][U][2];   // past the last part: beyond the buffer, zeros
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int w = 0; w < U; ++w)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                part[k][w][c] = __builtin_amdgcn_raw_buffer_load_b128(pr4, place[w] + 16 * c + (uint32_t)(s + k) * (T * T * 4),
                                                                      0, kCoherent);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int w = 0; w < U; ++w)
#pragma unroll
              for (int c = 0; c < 2; ++c) sum[w][c] += __builtin_bit_cast(f32x4, part[k][w][c]);
        }
#pragma unroll
        for (int w = 0; w < U; ++w)
#pragma unroll
          for (int c = 0; c < 2; ++c) *reinterpret_cast<f32x4*>(chunk(unit_row(w), 2 * u + c)) = sum[w][c];
      }
    }
    // (powers of two go into the columns' factors: a value costs a few fused
    // operations that take float16 operands as they are; written out, with each
    // step by itself, the arithmetic took 20000 cycles a tile of 256)
    float kp[8];
    if (kXB) {
#pragma unroll
      for (int h = 0; h < 8; ++h) kp[h] = (a.ca + M.db[me + p + h]) * (a.aux * a.out);
    } else if (MODE == kSquare) {
#pragma unroll
      for (int h = 0; h < 8; ++h) kp[h] = (a.cb + a.cc * M.da[me + p + h]) * (a.aux * a.out);
    }
    const float k_acc = MODE == kSquare ? a.cc * (a.in * a.out) : a.in * a.out;
#pragma unroll
    for (int w = 0; w < U; ++w) {
      const int r = unit_row(w), q = q0 + hf * HR + r;
      float v[8];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const f32x4 f = *reinterpret_cast<const f32x4*>(chunk(r, 2 * u + c));
#pragma unroll
        for (int h = 0; h < 4; ++h) v[4 * c + h] = f[h];
      }
      i32x4 s;   // the 8 finished values, 16 bits each
      if (kXB) {
        const int64_t at = ((int64_t)e * np + q) * mp + p;
#pragma unroll
        for (int h = 0; h < 8; ++h) v[h] = ((float)x2[w][h] * (1.0f / kLow) + (float)x1[w][h]) * kp[h] + v[h] * k_acc;
        if (a.last) {
          // X [n, m] is the output [N, K], or its transpose.  (The scale by itself: times
          // the powers of two above a small one would be subnormal.)
#pragma unroll
          for (int h = 0; h < 4; ++h) s[h] = (int)bf16_pack2(v[2 * h] * a.scale, v[2 * h + 1] * a.scale);
          if (!a.wide && q < a.N) store_row(a, (int64_t)e * a.N + q, p, s);
        } else {
          f16x8 hi, lo;
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            hi[h] = (_Float16)v[h];
            lo[h] = (_Float16)(v[h] * kLow - (float)hi[h] * kLow);
          }
          s = __builtin_bit_cast(i32x4, hi);
          *reinterpret_cast<i32x4*>(M.hi[a.cur ^ 1] + at) = s;
          *reinterpret_cast<f16x8*>(M.lo[a.cur ^ 1] + at) = lo;
        }
      } else {
        if (MODE == kSquare) {
          const float kq = a.cc * xq[w] * (a.aux * a.out);
#pragma unroll
          for (int h = 0; h < 8; ++h) v[h] = (float)x1[w][h] * (kp[h] + kq) + v[h] * k_acc;
        } else {
#pragma unroll
          for (int h = 0; h < 8; ++h) v[h] *= k_acc;
        }
        if (tp == tq) {   // the diagonal stays in float32, outside
#pragma unroll
          for (int h = 0; h < 8; ++h)
            if (p + h == q) {
              const float back = 1.0f / a.out, d = MODE == kSquare ? xq[MODE == kSquare ? w : 0] : 0.f;
              (MODE == kGram ? M.da : M.db)[me + q] = v[h] * back + (MODE == kSquare ? d * (a.cb + a.cc * d) : 0.f);
              v[h] = 0.f;
            }
        }
        f16x8 c;
#pragma unroll
        for (int h = 0; h < 8; ++h) c[h] = (_Float16)v[h];
        s = __builtin_bit_cast(i32x4, c);
        *reinterpret_cast<i32x4*>((MODE == kGram ? M.a : M.b) + (me + q) * mp + p) = s;
      }
      if (turned) *reinterpret_cast<i32x4*>(chunk(r, 2 * u)) = s;
    }
    if (turned) {
      lds_barrier();
      // columns, 8 rows of one a lane: a group of 16 lanes reads 16 columns of 4
      // rows transposed (lane L: row L / 4, columns 4 (L % 4) .. + 3; received:
      // column L of the 4 rows), the wave 32 rows of the 16 columns
      constexpr int UC = HR / 32 * (T / 16) / NW;   // such blocks of a wave
      static_assert(UC * NW * 32 * 16 == HR * T, "blocks fill the waves");
      const int L16 = lane & 15, grp = lane >> 4;
#pragma unroll
      for (int w = 0; w < UC; ++w) {
        const int b = wave + NW * w, c0 = b / (HR / 32) * 16, r0 = b % (HR / 32) * 32 + 8 * grp;
        const int c = c0 + 4 * (L16 & 3), r = r0 + (L16 >> 2);
        const uint32_t a0 = (uint32_t)(uintptr_t)(lds_void*)(reinterpret_cast<uint16_t*>(chunk(r, c / 8 * 2)) + c % 8);
        const uint32_t a1 = (uint32_t)(uintptr_t)(lds_void*)(reinterpret_cast<uint16_t*>(chunk(r + 4, c / 8 * 2)) + c % 8);
        tile::v4i16 f[2];
        asm volatile("ds_read_b64_tr_b16 %0, %2\n\tds_read_b64_tr_b16 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(f[0]), "=&v"(f[1])
                     : "v"(a0), "v"(a1)
                     : "memory");
        const i32x4 s = __builtin_bit_cast(i32x4, f);
        const int row = p0 + c0 + L16, col = q0 + hf * HR + r0;
        if (kXB && a.last) {
          if (row < a.N) store_row(a, (int64_t)e * a.N + row, col, s);
        } else if (kXB) {
          *reinterpret_cast<i32x4*>(M.xt + (me + row) * np + col) = s;
        } else {
          *reinterpret_cast<i32x4*>((MODE == kGram ? M.a : M.b) + (me + row) * mp + col) = s;
        }
      }
    }
  }
}

template <int T, int MODE>
hipError_t launch_product(StepArgs a, hipStream_t s) {
  const int64_t nm = a.M.mp / T, nn = a.M.np / T;
  a.total = a.M.E * (MODE >= kApply ? nm * nn : nm * (nm + 1) / 2) * (MODE == kGram && T == 64 ? a.splits : 1);
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

// ----------------------------------------------------------------- narrow --
// m <= 64: a launch a step.  Every workgroup of a matrix adds the workgroups'
// parts of A, squares it and forms B by itself, in LDS, applies B to its rows of
// X and leaves its part of the next A.  The three products by themselves are
// chains of launches of a few microseconds each, and A's a few tiles with all
// of n to add (4096 x 64: 18 of a step's 27 us, in one launch 11).
//
// Here X enters A and X B in two pieces, and B the latter (the product of two second
// pieces is left out): with the first pieces alone the rounding of a few strong
// directions reached the weak ones, at up to 4e-2 of the result (n x 2 to n x 64, r
// singular values of 1, the others 1e-2 to 1e-5); so it is 1.4e-3.  64 x 4096: 66.5 us
// with the first pieces, 71.3 with both in X B, 75.6 with both in A too.

// (For m <= 128 the same, with two halves of columns and twice the threads, took 15
// us a step and more, the three launches 13.)

constexpr int kNarrow = 64;       // m, padded
constexpr int kNarrowRows = 128;  // rows of a round: 32 a wave

struct NarrowArgs {
  int32_t E, N, K, wide, n, m;
  int32_t W, rows;        // workgroups of a matrix; rows of one, a multiple of kNarrowRows
  const void* u;
  const double* part;     // sums of squares
  double eps;
  float first;            // 2^ of the first X's scale
  uint16_t* hi;           // X [E][W rows][64], two pieces, updated in place
  uint16_t* lo;
  const float* gin;       // parts of A [E][W][64][64], of the stored X's products
  float* gout;
  int32_t last;
  float ca, cb, cc;
  float to_a, sa, from_sa, sb, from_b, from_x, out;   // scales, as in StepArgs
  float scale;
  uint16_t* y;
};

enum Narrow { kNarrowInput = 0, kNarrowInputBf16 = 1, kNarrowStep = 2 };

// Lanes l and l + 32 hold 8 values each of 16 in a row, the first and the last 8, as
// loaded; or, as a product leaves them, values 0 .. 3 and 8 .. 11, and 4 .. 7 and 12 ..
// 15.  One to the other, either way.
__device__ __forceinline__ void halves_to_groups(i32x4& v) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const auto r = __builtin_amdgcn_permlane32_swap((uint32_t)v[k], (uint32_t)v[2 + k], false, false);
    v[k] = (int)r[0];
    v[2 + k] = (int)r[1];
  }
}

// Transposed fragments of a round's rows (columns j .. + 31 of the 16 rows from 16 ST
// on) for two column starts j: a lane's first read of the round's first 16 rows is at
// a[.][0], its second, 4 rows further, at a[.][1]; 16 rows further the swizzle is the
// same, so that a slice is a constant offset.  Reads and their wait in one statement
// (the builtins wait for the stores in flight as well).
__device__ __forceinline__ void narrow_places(const uint16_t* s, const int (&j)[2], int lane, uint32_t (&a)[2][2]) {
  const int gq = lane >> 4, L = lane & 15;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      a[i][h] = (uint32_t)(uintptr_t)(tile::lds_v4i16*)(
          s + tile::wt_off_n<kNarrow>(8 * (gq >> 1) + (L >> 2) + 4 * h, j[i] + 16 * (gq & 1) + 4 * (L & 3)));
}

// acc += the products of the two fragments over slices ST .. of a round, low += those with
// a second piece, which lies a round behind the first, at kLow times their value.
template <int ST>
__device__ __forceinline__ void narrow_gram(const uint32_t (&a)[2][2], f32x16& acc, f32x16& low) {
  if constexpr (ST < kNarrowRows / 16) {
    tile::v4i16 v[8];
    constexpr int at = ST * 16 * kNarrow * 2;
    asm volatile("ds_read_b64_tr_b16 %0, %8 offset:%12\n\tds_read_b64_tr_b16 %1, %9 offset:%12\n\t"
                 "ds_read_b64_tr_b16 %2, %10 offset:%12\n\tds_read_b64_tr_b16 %3, %11 offset:%12\n\t"
                 "ds_read_b64_tr_b16 %4, %8 offset:%13\n\tds_read_b64_tr_b16 %5, %9 offset:%13\n\t"
                 "ds_read_b64_tr_b16 %6, %10 offset:%13\n\tds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]),
                   "=&v"(v[7])
                 : "v"(a[0][0]), "v"(a[0][1]), "v"(a[1][0]), "v"(a[1][1]), "n"(at), "n"(at + kNarrowRows * kNarrow * 2)
                 : "memory");
    f16x8 f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const tile::v4i16 v8[2] = {v[2 * i], v[2 * i + 1]};
      f[i] = __builtin_bit_cast(f16x8, v8);
    }
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[0], f[1], acc, 0, 0, 0);
    low = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[2], f[1], low, 0, 0, 0);
    low = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[0], f[3], low, 0, 0, 0);
    narrow_gram<ST + 1>(a, acc, low);
  }
}

template <int MODE>
__global__ void __launch_bounds__(256) ortho_narrow_kernel(NarrowArgs a) {
  constexpr int MP = kNarrow, SQ = MP * MP;
  constexpr int NK = MP / 16;       // MFMA steps along m
  __shared__ __attribute__((aligned(16))) uint16_t s_o[MODE == kNarrowStep ? SQ : 8], s_b[MODE == kNarrowStep ? SQ : 8],
      s_bl[MODE == kNarrowStep ? SQ : 8];   // B's second piece
  __shared__ __attribute__((aligned(16))) uint16_t s_x[2 * kNarrowRows * MP];   // both pieces
  __shared__ __attribute__((aligned(16))) float s_d[MP], s_e[MP];
  const int e = blockIdx.x / a.W, wg = blockIdx.x % a.W;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave >> 1, wj = wave & 1, l32 = lane & 31, up = lane >> 5;
  auto frag = [&](const uint16_t* s, int row, int st) {
    return *reinterpret_cast<const f16x8*>(s + tile::lds_off<MP>(row, 2 * st + up));
  };
  // A round: row t of the lane in two pieces, columns 16 st + 8 up .. + 7, 16-byte loads
  // (x: also the product's operand); or the update's values (u: 4 g + h of [i] is column
  // 32 i + 8 g + 4 up + h, as in the product).  Requested a round ahead, the first
  // before anything else.
  const int tl = 32 * wave + l32;
  const int64_t row0 = (int64_t)wg * a.rows + tl;
  const int64_t x0 = ((int64_t)e * a.W * a.rows + row0) * MP;
  i32x4 x[NK], xl[NK];
  float u[2][16];
  auto request = [&](int rb) {
    if constexpr (MODE == kNarrowStep) {
      const int64_t at = x0 + (int64_t)rb * MP + 8 * up;
#pragma unroll
      for (int st = 0; st < NK; ++st) {
        x[st] = *reinterpret_cast<const i32x4*>(a.hi + at + 16 * st);
        xl[st] = *reinterpret_cast<const i32x4*>(a.lo + at + 16 * st);
      }
    } else {
      // past the matrix: an offset past the buffer, which gives 0
      constexpr int EL = MODE == kNarrowInputBf16 ? 2 : 4;
      const int64_t per = (int64_t)a.N * a.K * EL;
      const __amdgpu_buffer_rsrc_t r = buffer_rsrc(static_cast<const char*>(a.u) + e * per, per);
      const int t = (int)(row0 + rb);
      const uint32_t vo = (uint32_t)(a.wide ? 4 * up * a.K + t : t * a.K + 4 * up) * EL;
      const int step = (a.wide ? a.K : 1) * EL;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int p = 32 * i + 8 * (k / 4) + k % 4;
          const uint32_t o = t < a.n && p + 4 * up < a.m ? vo : 0x80000000u;
          if constexpr (EL == 2)
            u[i][k] = bf16_to_f32((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, o, p * step, 0));
          else
            u[i][k] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, o, p * step, 0));
        }
    }
  };
  request(0);
  double f = 0.0;
  if constexpr (MODE != kNarrowStep) {
    double s = a.part[(int64_t)e * kOrthoNormBlocks + lane];
#pragma unroll
    for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
    f = a.first / (sqrt(s) + a.eps);
  } else {
    // A: a thread holds 4 columns from c on of every RS-th row from r0 on; some
    // parts are requested together (past the last: that one again, not added)
    constexpr int RS = 256 / (MP / 4), NI = MP / RS, AHEAD = 16 / NI;
    const int c = 4 * (threadIdx.x % (MP / 4)), r0 = threadIdx.x / (MP / 4);
    f32x4 v[NI] = {};
    const float* g = a.gin + (int64_t)e * a.W * SQ + r0 * MP + c;
    for (int w = 0; w < a.W; w += AHEAD) {
      f32x4 part[AHEAD][NI];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
#pragma unroll
        for (int i = 0; i < NI; ++i)
          part[k][i] = *reinterpret_cast<const f32x4*>(g + (int64_t)min(w + k, a.W - 1) * SQ + RS * i * MP);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (w + k < a.W) {
#pragma unroll
          for (int i = 0; i < NI; ++i) v[i] += part[k][i];
        }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = r0 + RS * i, k = r - c;   // the diagonal is value k of this thread, if 0 <= k < 4
      uint32_t o[4];
      float d = 0.f;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float w = v[i][h] * a.to_a;
        d = k == h ? w : d;
        o[h] = f32_to_f16(k == h ? 0.f : w * a.sa);
      }
      if ((unsigned)k < 4u) s_d[r] = d;
      *reinterpret_cast<uint2*>(s_o + tile::lds_off<MP>(r, c / 8) + c % 8) =
          make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
    }
    lds_barrier();
    // B: wave (wi, wj) the tile of 32 p by 32 q
    f32x16 acc = {};
#pragma unroll
    for (int st = 0; st < NK; ++st)
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(frag(s_o, 32 * wi + l32, st), frag(s_o, 32 * wj + l32, st), acc, 0,
                                                   0, 0);
    const float sq = a.from_sa * a.from_sa;
    const int q = 32 * wj + l32;
    const float dq = s_d[q];
#pragma unroll
    for (int g4 = 0; g4 < 4; ++g4) {
      const int p = 32 * wi + 8 * g4 + 4 * up;
      const uint2 o = *reinterpret_cast<const uint2*>(s_o + tile::lds_off<MP>(q, p / 8) + p % 8);
      const f32x4 dp = *reinterpret_cast<const f32x4*>(s_d + p);
      uint32_t b[4], bl[4];
      float diag = 0.f;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float off = f16_to_f32((h & 2 ? o.y : o.x) >> (h & 1 ? 16 : 0)) * a.from_sa;   // 0 on the diagonal
        const float oo = acc[4 * g4 + h] * sq;
        diag = p + h == q ? oo : diag;
        const float v = p + h == q ? 0.f : (a.cb * off + a.cc * (oo + (dp[h] + dq) * off)) * a.sb;
        b[h] = f32_to_f16(v);
        bl[h] = f32_to_f16((v - f16_to_f32(b[h])) * kLow);
      }
      if ((unsigned)(q - p) < 4u) s_e[q] = a.ca + (a.cb * dq + a.cc * (diag + dq * dq));
      *reinterpret_cast<uint2*>(s_b + tile::lds_off<MP>(q, p / 8) + p % 8) =
          make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
      *reinterpret_cast<uint2*>(s_bl + tile::lds_off<MP>(q, p / 8) + p % 8) =
          make_uint2(bl[0] | (bl[1] << 16), bl[2] | (bl[3] << 16));
    }
    lds_barrier();
  }
  f32x16 gram = {}, gram_low = {};
  uint32_t places[2][2];
  narrow_places(s_x, {32 * wi, 32 * wj}, lane, places);
  for (int rb = 0; rb < a.rows; rb += kNarrowRows) {
    const int64_t t = row0 + rb, at = x0 + (int64_t)rb * MP;
    float val[2][16];
    if constexpr (MODE == kNarrowStep) {
      // X B in pieces: both products with a second piece, at kLow times their value, then
      // the one of the first
      f32x16 acc[2] = {};
      auto add = [&](const uint16_t* s_p, const i32x4(&xp)[NK]) {
#pragma unroll
        for (int st = 0; st < NK; ++st)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(frag(s_p, 32 * i + l32, st),
                                                            __builtin_bit_cast(f16x8, xp[st]), acc[i], 0, 0, 0);
      };
      add(s_bl, x);
      add(s_b, xl);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[i][k] *= 1.0f / kLow;
      add(s_b, x);
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        halves_to_groups(x[st]);
        halves_to_groups(xl[st]);
        const f16x8 h = __builtin_bit_cast(f16x8, x[st]), l = __builtin_bit_cast(f16x8, xl[st]);
#pragma unroll
        for (int g2 = 0; g2 < 2; ++g2) {
          const int i = st / 2, g4 = 2 * (st % 2) + g2;
          const f32x4 se = *reinterpret_cast<const f32x4*>(s_e + 16 * st + 8 * g2 + 4 * up);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float v = (float)l[4 * g2 + k] * (1.0f / kLow) + (float)h[4 * g2 + k];
            val[i][4 * g4 + k] = (se[k] * a.from_x * v + acc[i][4 * g4 + k] * a.from_b) * a.out;
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k) val[i][k] = (float)(u[i][k] * f);
    }
    if (rb + kNarrowRows < a.rows) request(rb + kNarrowRows);
    if (MODE == kNarrowStep && a.last) {
      // past the matrix: an offset past the buffer, which stores nothing
      const int64_t per = (int64_t)a.N * a.K;
      const __amdgpu_buffer_rsrc_t r = buffer_rsrc(a.y + e * per, per * 2);
      const uint32_t vo = (uint32_t)(a.wide ? 4 * up * a.K + (int)t : (int)t * a.K + 4 * up) * 2;
      const int step = (a.wide ? a.K : 1) * 2;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          const uint32_t w = bf16_pack2(val[i][k] * a.scale, val[i][k + 1] * a.scale);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int p = 32 * i + 8 * (k / 4) + (k + h) % 4;
            const uint32_t o = t < a.n && p + 4 * up < a.m ? vo : 0x80000000u;
            __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(w >> (16 * h)), r, o, p * step, 0);
          }
        }
      continue;
    }
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      f16x8 hi, lo;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = val[st / 2][8 * (st % 2) + k];
        hi[k] = (_Float16)v;
        lo[k] = (_Float16)(v * kLow - (float)hi[k] * kLow);
      }
      i32x4 h = __builtin_bit_cast(i32x4, hi), l = __builtin_bit_cast(i32x4, lo);
#pragma unroll
      for (int g2 = 0; g2 < 2; ++g2) {
        uint16_t* const place = s_x + tile::wt_off_n<MP>(tl, 16 * st + 8 * g2 + 4 * up);
        *reinterpret_cast<int2*>(place) = make_int2(h[2 * g2], h[2 * g2 + 1]);
        *reinterpret_cast<int2*>(place + kNarrowRows * MP) = make_int2(l[2 * g2], l[2 * g2 + 1]);
      }
      halves_to_groups(h);
      halves_to_groups(l);
      *reinterpret_cast<i32x4*>(a.hi + at + 16 * st + 8 * up) = h;
      *reinterpret_cast<i32x4*>(a.lo + at + 16 * st + 8 * up) = l;
    }
    lds_barrier();
    narrow_gram<0>(places, gram, gram_low);
    lds_barrier();
  }
  if (MODE == kNarrowStep && a.last) return;
  float* g = a.gout + ((int64_t)e * a.W + wg) * SQ;
#pragma unroll
  for (int g4 = 0; g4 < 4; ++g4)
    *reinterpret_cast<f32x4*>(g + (32 * wj + l32) * MP + 32 * wi + 8 * g4 + 4 * up) =
        (f32x4){gram[4 * g4] + gram_low[4 * g4] * (1.0f / kLow),
                gram[4 * g4 + 1] + gram_low[4 * g4 + 1] * (1.0f / kLow),
                gram[4 * g4 + 2] + gram_low[4 * g4 + 2] * (1.0f / kLow),
                gram[4 * g4 + 3] + gram_low[4 * g4 + 3] * (1.0f / kLow)};
}

// Rows of a workgroup: two rounds, or what leaves 16 workgroups (whose parts of A
// each of them adds) and not many more than there are CUs.
int64_t narrow_rows(int64_t E, int64_t n) {
  const int64_t by_cus = (256 + E - 1) / E, W = by_cus < 16 ? by_cus : 16;
  const int64_t r = (n + W - 1) / W;
  const int64_t rows = (r + kNarrowRows - 1) / kNarrowRows * kNarrowRows;
  if (n <= kNarrowRows) return kNarrowRows;
  return rows < 2 * kNarrowRows ? 2 * kNarrowRows : rows;
}

// Time of a slice of `tiles` tiles of T over 256 CUs, in that of a tile of 256 alone on
// its CU (1.3 us): a smaller tile has room for 2 or 4 on a CU and costs more for its
// size.  (16 of 1536 x 4096, the products for A: 336 tiles of 256 240 us, 1248 of 128
// 201, 4992 of 64 309; 8 of 4096 x 6144: 1088 of 256 827 us, 4224 of 128 866; X B of
// the latter in tiles of 256 1523 us, of 128 1895.)
double slice_time(int T, int64_t tiles) {
  const double q = (double)((tiles + 255) / 256);
  if (T == 256) return q;
  const double alone = T == 128 ? 0.35 : 0.2, each = T == 128 ? 0.295 : 0.13;
  return q * each > alone ? q * each : alone;
}

// What m and n are padded to, and the tiles of X B.
int tile_of(int64_t E, int64_t n, int64_t m) {
  int best = 0;
  double least = 0.0;
  for (int T = 64; T <= 256; T *= 2) {
    const int64_t nm = (m + T - 1) / T, nn = (n + T - 1) / T;
    const double time = slice_time(T, E * nm * nn) * (double)(nm * T);
    if (best == 0 || time < least) {
      best = T;
      least = time;
    }
  }
  return best;
}

// Tiles of the symmetric products, as the padding allows.
int symmetric_tile(int64_t E, int64_t mp, int most) {
  int best = 64;
  for (int T = 128; T <= most; T *= 2) {
    auto time = [&](int t) { return slice_time(t, E * (mp / t) * (mp / t + 1) / 2); };
    if (time(T) < time(best)) best = T;
  }
  return best;
}

// Workgroups that share the contraction of a tile of A, of 8 slices at least and three
// of them (128 x 4096: 8 of them 109 us, one 172; 512 x 2048: 4 134, one 155; but two
// for 1000 x 1000 170, one 165; of 4 slices 512 x 2048 155).
int gram_splits(int64_t E, int64_t np, int64_t mp) {
  const int64_t tiles = E * (mp / 64) * (mp / 64 + 1) / 2, by_cus = 512 / tiles, by_slices = np / kBK / 8;
  const int64_t s = by_cus < by_slices ? by_cus : by_slices;
  return (int)(s < 3 ? 1 : s > 16 ? 16 : s);
}

// Matrices up to this m take both pieces of X in X B.  With the first alone the
// rounding of a few strong directions that reaches the weak ones is up to 4.4e-3 of
// the result for 4096 x 128 (spectra as above), 2.8e-3 for 4096 x 256, 2e-3 for
// 4096 x 513, 1.2e-3 for 1024 x 1024; with both 1.1e-3 and less.  8 of 256 x 512: 85.8
// us with the first piece, 91.5 with both; 32 of 512 x 2048 835 and 929, 64 of 256 x
// 4096 1254 and 1319.
constexpr int64_t kBothMost = 512;

struct Layout {
  int T;                  // 0: narrow
  int Ts, splits;         // tiles of the symmetric products; of A, if 64
  bool both;              // both pieces of X in X B
  int64_t np, mp, W, hi[2], lo[2], xt, a, b, da, db, part, gpart, gdone, end;
};

Layout layout(int64_t E, int64_t N, int64_t K) {
  Layout L{};
  const int64_t n = N >= K ? N : K, m = N >= K ? K : N;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  L.part = take(8 * E * kOrthoNormBlocks);
  if (m <= kNarrow) {
    L.mp = kNarrow;
    const int64_t rows = narrow_rows(E, n);
    L.W = (n + rows - 1) / rows;
    L.np = L.W * rows;
    L.hi[0] = take(2 * E * L.np * L.mp);
    L.lo[0] = take(2 * E * L.np * L.mp);
    L.a = take(4 * E * L.W * L.mp * L.mp);   // parts of A, of this step and of the next
    L.b = take(4 * E * L.W * L.mp * L.mp);
    L.end = at;
    return L;
  }
  L.T = tile_of(E, n, m);
  L.both = m <= kBothMost;
  L.np = (n + L.T - 1) / L.T * L.T;
  L.mp = (m + L.T - 1) / L.T * L.T;
  L.Ts = symmetric_tile(E, L.mp, L.T);
  L.splits = L.Ts == 64 ? gram_splits(E, L.np, L.mp) : 1;
  for (int i = 0; i < 2; ++i) {
    L.hi[i] = take(2 * E * L.np * L.mp);
    L.lo[i] = take(2 * E * L.np * L.mp);
  }
  L.xt = take(2 * E * L.np * L.mp);
  L.a = take(2 * E * L.mp * L.mp);
  L.b = take(2 * E * L.mp * L.mp);
  L.da = take(4 * E * L.mp);
  L.db = take(4 * E * L.mp);
  if (L.splits > 1) {
    const int64_t tiles = E * (L.mp / 64) * (L.mp / 64 + 1) / 2;
    L.gpart = take(4 * tiles * L.splits * 64 * 64);
    L.gdone = take(4 * tiles);
  }
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
    // (the root whose numerator does not cancel, and the other by their product: for
    // c = 0 too, and where c is so small that the two of a numerator would be one
    // number; a division by 0 leaves nothing inside)
    const double d = 9 * b * b - 20 * a * c;
    if (d >= 0.0) {
      const double q = -(3 * b + copysign(sqrt(d), b)) / 2;
      at(q / (5 * c));
      at(a / q);
    }
    at(-b / (2 * c));
    s[i][0] = power(u);
    s[i][1] = power(u * u);
    s[i][2] = power(most);
    if (!(most <= 1e9)) return false;
    u = next;
  }
  return u <= 4096.0;
}

static hipError_t launch_narrow(const OrthoArgs& o, const ortho::Layout& L, const int32_t (*s)[3], hipStream_t st) {
  using namespace ortho;
  char* ws = static_cast<char*>(o.ws);
  NarrowArgs a{};
  a.E = o.E;
  a.N = o.N;
  a.K = o.K;
  a.wide = o.N < o.K;
  a.n = a.wide ? o.K : o.N;
  a.m = a.wide ? o.N : o.K;
  a.W = (int32_t)L.W;
  a.rows = (int32_t)(L.np / L.W);
  a.u = o.update;
  a.part = reinterpret_cast<const double*>(ws + L.part);
  a.eps = o.eps;
  a.first = pow2(s[0][0]);
  a.hi = reinterpret_cast<uint16_t*>(ws + L.hi[0]);
  a.lo = reinterpret_cast<uint16_t*>(ws + L.lo[0]);
  a.scale = o.scale;
  a.y = o.out;
  float* g[2] = {reinterpret_cast<float*>(ws + L.a), reinterpret_cast<float*>(ws + L.b)};
  a.gout = g[0];
  const dim3 grid((unsigned)(o.E * L.W)), block(256);
  if (o.bf16)
    hipLaunchKernelGGL(ortho_narrow_kernel<kNarrowInputBf16>, grid, block, 0, st, a);
  else
    hipLaunchKernelGGL(ortho_narrow_kernel<kNarrowInput>, grid, block, 0, st, a);
  hipError_t e = hipGetLastError();
  for (int i = 0; i < o.steps && e == hipSuccess; ++i) {
    a.gin = g[i & 1];
    a.gout = g[(i & 1) ^ 1];
    a.last = i + 1 == o.steps;
    a.ca = o.coef[i][0];
    a.cb = o.coef[i][1];
    a.cc = o.coef[i][2];
    a.to_a = pow2(-2 * s[i][0]);
    a.sa = pow2(s[i][1]);
    a.from_sa = pow2(-s[i][1]);
    a.sb = pow2(s[i][2]);
    a.from_b = pow2(-s[i][0] - s[i][2]);
    a.from_x = pow2(-s[i][0]);
    a.out = a.last ? 1.0f : pow2(s[i + 1][0]);
    hipLaunchKernelGGL(ortho_narrow_kernel<kNarrowStep>, grid, block, 0, st, a);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_orthogonalize(const OrthoArgs& o, hipStream_t st) {
  using namespace ortho;
  const Layout L = layout(o.E, o.N, o.K);
  int32_t s[kOrthoMaxSteps][3];
  if (!ortho_scales(o, s)) return hipErrorInvalidValue;
  char* ws = static_cast<char*>(o.ws);
  const int wide = o.N < o.K;
  const int64_t per = (int64_t)o.N * o.K;
  double* part = reinterpret_cast<double*>(ws + L.part);
  const dim3 gn(kOrthoNormBlocks, (unsigned)o.E);
  if (o.bf16)
    hipLaunchKernelGGL(ortho_norm_kernel<true>, gn, dim3(1024), 0, st, o.update, per, part);
  else
    hipLaunchKernelGGL(ortho_norm_kernel<false>, gn, dim3(1024), 0, st, o.update, per, part);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (L.T == 0) return launch_narrow(o, L, s, st);
  Mats M{};
  M.E = o.E;
  M.np = (int32_t)L.np;
  M.mp = (int32_t)L.mp;
  M.part = part;
  for (int i = 0; i < 2; ++i) {
    M.hi[i] = reinterpret_cast<uint16_t*>(ws + L.hi[i]);
    M.lo[i] = reinterpret_cast<uint16_t*>(ws + L.lo[i]);
  }
  M.xt = reinterpret_cast<uint16_t*>(ws + L.xt);
  M.a = reinterpret_cast<uint16_t*>(ws + L.a);
  M.b = reinterpret_cast<uint16_t*>(ws + L.b);
  M.da = reinterpret_cast<float*>(ws + L.da);
  M.db = reinterpret_cast<float*>(ws + L.db);
  if (L.splits > 1) {
    M.gpart = reinterpret_cast<float*>(ws + L.gpart);
    M.gdone = reinterpret_cast<int32_t*>(ws + L.gdone);
    M.gtiles = (int32_t)(o.E * (L.mp / 64) * (L.mp / 64 + 1) / 2);
  }
  {
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
  a.vec = o.K % 8 == 0 && ((uintptr_t)o.out & 15) == 0;
  a.scale = o.scale;
  a.splits = L.splits;
  for (int i = 0; i < o.steps; ++i) {
    const int sx = s[i][0], sa = s[i][1], sb = s[i][2];
    a.cur = i & 1;
    a.last = i + 1 == o.steps;
    a.ca = o.coef[i][0];
    a.cb = o.coef[i][1];
    a.cc = o.coef[i][2];
    a.in = pow2(-2 * sx);
    a.out = pow2(sa);
    if ((e = product<kGram>(a, L.Ts, st)) != hipSuccess) return e;
    a.in = pow2(-2 * sa);
    a.out = pow2(sb);
    a.aux = pow2(-sa);
    if ((e = product<kSquare>(a, L.Ts, st)) != hipSuccess) return e;
    a.in = pow2(-sx - sb);
    a.out = a.last ? 1.0f : pow2(s[i + 1][0]);
    a.aux = pow2(-sx);
    if ((e = L.both ? product<kApplyBoth>(a, L.T, st) : product<kApply>(a, L.T, st)) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe

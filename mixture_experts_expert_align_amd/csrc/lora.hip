// Low-rank adapters of many requests at once beside a shared projection, and
// their gradients.  Row r takes adapter g = adapter[r] (or none):
//   s_r = scale_g A_g x_r         y_r  = W x_r + B_g s_r
//   t_r = scale_g B_g^T dy_r      dx_r = W^T dy_r + A_g^T t_r
//   dA_g = sum over its rows of t_r x_r^T      dB_g = sum of dy_r s_r^T
// with x [R, K], W [N, K], A [G, rank, K], B [G, N, rank].
//
// The rows may come in any order of adapters.  The narrow products s and t
// come first (shrink); the projection's kernels then treat the adapters'
// part as more of the same contraction.  s and t are kept to float32
// precision as three bf16 pieces, hi + mid + lo (3 x 8 significand bits): the
// matrix units take bf16 operands, and one piece alone would put an error of
// 2^-8 into dA and dB, which are float32, and a second rounding of the size
// of y's own into y.
#include "kernels.h"
#include "tile_common.h"

namespace moe {
namespace {

constexpr uint32_t kPast = 0x80000000u;   // an offset past every buffer: loads give 0
constexpr int kPieces = kLoraPieces;

__device__ __forceinline__ int row_adapter(const int32_t* adapter, int64_t r, int64_t R, int G) {
  if (r >= R) return -1;
  const int g = adapter[r];
  return g >= 0 && g < G ? g : -1;
}

// The three bf16 pieces of a float32.  A finite value past bf16's largest (from
// 2^128 - 2^119 on the nearest is infinity) has that one as its first piece,
// and the rest fits the other two.
__device__ __forceinline__ void split3(float v, uint32_t (&p)[3]) {
  p[0] = f32_to_bf16_rne(v);
  if ((p[0] & 0x7fffu) == 0x7f80u && v - v == 0.0f) p[0] -= 1;
  const float r1 = v - bf16_to_f32(p[0]);
  p[1] = f32_to_bf16_rne(r1);
  p[2] = f32_to_bf16_rne(r1 - bf16_to_f32(p[1]));
  if (!(v - v == 0.0f)) p[1] = p[2] = 0;   // inf, NaN: the first piece says it
}

typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;

// MFMA operand fragment (16 outputs x 8 contraction rows a lane group) of a
// row-major LDS block whose rows are the contraction: lane (l16, q) gets
// column col0 + l16 of rows 8 q .. 8 q + 7, by two transposing reads whose
// lane L of each group of 16 points at row 8 q + L / 4 (+ 4), columns
// col0 + 4 (L % 4) .. + 3.  off(row, col): element offset, 4 columns together.
template <typename Off>
__device__ __forceinline__ bf16x8 col_frag(const uint16_t* base, int col0, int lane, Off off) {
  const int q = lane >> 4, L = lane & 15;
  const int r = 8 * q + (L >> 2), c = col0 + 4 * (L & 3);
  const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(base + off(r, c)));
  const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(base + off(r + 4, c)));
  const v4i16 v8[2] = {lo, hi};
  return __builtin_bit_cast(bf16x8, v8);
}

// Blocks that are read transposed (rows of `chunks` 16-byte chunks): rows lie
// an odd multiple of 128 bytes apart, chunk pairs XORed by the row, so that a
// read's 4 consecutive rows and its lane groups' rows 8 apart fall on
// different banks.  Pitch and position in chunks.
__host__ __device__ constexpr int tr_pitch(int chunks) { return ((chunks + 7) / 8 | 1) * 8; }
__device__ __forceinline__ int tr_at(int r, int c, int pitch) {
  return r * pitch + (c ^ (((r & 3) ^ ((r >> 3) & 1)) << 1));
}

// ---------------------------------------------------------------- shrink --
// low[r] = scale_g M_g v_r for 16 CT rows a workgroup: the rows in the MFMA
// column operand, 16 of the rank's outputs per row tile (JT tiles), the
// contraction split over the 4 waves in steps of 64 (wave w takes steps w,
// w + 4, ...), whose sums meet in LDS in wave order.  One pass per adapter
// among the workgroup's rows; each pass reads and writes its own rows.
//   T = false: M = A [rank, C], contraction contiguous;
//   T = true:  M = B^T, B [C, rank]: a step's 64 rows are read transposed.
// Each wave has a ring of D steps in LDS to itself, filled by loads that
// write LDS (no barrier: it waits for its own loads; T: one step in LDS, D on
// their way in registers, since the compiler waits for every load that writes
// LDS before a transposing read).  That is for the lines:
// the MFMA layout wants 16 rows of 64 bytes from a load, which asks the cache
// for half a line at a time, and a CU got 28 KB/us that way; loads of 8 rows
// of 128 bytes reach 70.  Chunks are XOR-swizzled so that the 16 rows of a
// read spread over the banks.
// Grid (row blocks, passes in flight, row tile groups): with few row blocks
// the adapters of one block go to different workgroups.
constexpr int kShrinkWaves = 4;
constexpr int64_t kShrinkSplitRows = 320;

template <int JT, int CT, bool T, int D>
__global__ void __launch_bounds__(64 * kShrinkWaves) lora_shrink_kernel(LoraArgs a, const uint16_t* __restrict__ v,
                                                                       const uint16_t* __restrict__ m, int C) {
  // a step: 16 CT rows, then 16 JT rows of A, of 128 bytes of contraction
  // each, or 64 rows of B (rank <= 16 JT)
  constexpr int kStep = CT * 1024 + (T ? 64 * 8 * tr_pitch(2 * JT) : JT * 1024);   // elements
  constexpr int kRing = kStep * (T ? 1 : D);
  constexpr int kLoads = 2 * (CT + JT);           // 1 KB each
  constexpr int kRed = kShrinkWaves * JT * CT * 64 * 16, kRings = kShrinkWaves * kRing * 2;
  static_assert((D - 1) * kLoads < 64, "wait counts");
  __shared__ __attribute__((aligned(1024))) char smem[kRed > kRings ? kRed : kRings];
  const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t r0 = (int64_t)blockIdx.x * 16 * CT;
  const int rank = a.rank;
  const int j0 = T ? 0 : JT * blockIdx.z;   // first row tile
  int mine[CT];                             // adapter of row 16 c + l16
#pragma unroll
  for (int c = 0; c < CT; ++c) mine[c] = row_adapter(a.adapter, r0 + 16 * c + l16, a.R, a.G);
  const __amdgpu_buffer_rsrc_t vr = buffer_rsrc(v + r0 * C, min<int64_t>(16 * CT, a.R - r0) * C * 2);
  f32x4* red = reinterpret_cast<f32x4*>(smem);
  uint16_t* ring = reinterpret_cast<uint16_t*>(smem) + wave * kRing;

  if (blockIdx.y == 0 && blockIdx.z == 0) {   // rows without an adapter: zeros
    for (int i = threadIdx.x; i < 16 * CT * kPieces * rank / 8; i += 64 * kShrinkWaves) {
      const int64_t r = r0 + 8 * i / (kPieces * rank);
      if (r < a.R && row_adapter(a.adapter, r, a.R, a.G) < 0)
        reinterpret_cast<i32x4*>(a.low + r0 * kPieces * rank)[i] = (i32x4){0, 0, 0, 0};
    }
  }

  uint64_t left = 0;   // rows whose adapter has not had its pass
#pragma unroll
  for (int c = 0; c < CT; ++c) left |= (__ballot(mine[c] >= 0) & 0xffffull) << (16 * c);
  for (int pass = 0; left; ++pass) {
    const int row = __ffsll((unsigned long long)left) - 1;
    int g = 0;
#pragma unroll
    for (int c = 0; c < CT; ++c)
      if (row >> 4 == c) g = __builtin_amdgcn_readlane(mine[c], row & 15);
    uint64_t rows = 0;
#pragma unroll
    for (int c = 0; c < CT; ++c) rows |= (__ballot(mine[c] == g) & 0xffffull) << (16 * c);
    left &= ~rows;
    if (pass % gridDim.y != blockIdx.y) continue;
    const __amdgpu_buffer_rsrc_t mr = buffer_rsrc(m + (int64_t)g * rank * C, (int64_t)rank * C * 2);
    const float sc = a.scale[g];
    // load i of a step: rows 8 i + lane / 8, physical chunk lane % 8; only
    // this adapter's rows are read
    auto chunk = [&](int r) { return 16 * ((lane & 7) ^ ((r >> 1) & 7)); };
    uint32_t vo[2 * CT], mo[2 * JT];
#pragma unroll
    for (int i = 0; i < 2 * CT; ++i) {
      const int r = 8 * i + (lane >> 3);
      vo[i] = (rows >> r) & 1 ? (uint32_t)(r * C * 2 + chunk(r)) : kPast;
    }
#pragma unroll
    for (int i = 0; i < 2 * JT; ++i) {
      const int r = 8 * i + (lane >> 3), e = 64 * i + lane;
      mo[i] = T ? (e < 8 * rank ? 16 * e : kPast)
                : (16 * j0 + r < rank ? (uint32_t)((16 * j0 + r) * C * 2 + chunk(r)) : kPast);
    }
    constexpr int kPitch = tr_pitch(2 * JT);
    int bo[T ? 2 * JT : 1];   // where this lane's chunks of B go
    if (T) {
#pragma unroll
      for (int i = 0; i < 2 * JT; ++i) {
        const int e = min(64 * i + lane, 8 * rank - 1), r = e / (rank / 8);
        bo[i] = tr_at(r, e - r * (rank / 8), kPitch);
      }
    }
    f32x4 acc[JT][CT];
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[j][c] = (f32x4){0.f, 0.f, 0.f, 0.f};
    const int n = (C / 64 - wave + kShrinkWaves - 1) / kShrinkWaves;
    i32x4 reg[T ? D : 1][T ? kLoads : 1];
    auto load = [&](int d, int i) {   // past the end: zeros
      const int k0 = 64 * (wave + kShrinkWaves * i);
      const bool in = i < n;
      uint16_t* s = ring + d * kStep;
#pragma unroll
      for (int l = 0; l < 2 * CT; ++l) {
        if constexpr (T) reg[d][l] = __builtin_amdgcn_raw_buffer_load_b128(vr, in ? vo[l] : kPast, 2 * k0, 0);
        else lds_load16(vr, s + 512 * l, in ? vo[l] : kPast, 2 * k0);
      }
#pragma unroll
      for (int l = 0; l < 2 * JT; ++l) {
        if constexpr (T)
          reg[d][2 * CT + l] = __builtin_amdgcn_raw_buffer_load_b128(mr, in ? mo[l] : kPast, 2 * k0 * rank, 0);
        else
          lds_load16(mr, s + CT * 1024 + 512 * l, in ? mo[l] : kPast, 2 * k0);
      }
      issue_order();
    };
    auto mma = [&](int d) {
      if constexpr (T) {
        __builtin_amdgcn_wave_barrier();   // the last step's reads come first
#pragma unroll
        for (int l = 0; l < 2 * CT; ++l) *reinterpret_cast<i32x4*>(ring + 512 * l + 8 * lane) = reg[d][l];
#pragma unroll
        for (int l = 0; l < 2 * JT; ++l)
          if (64 * l + lane < 8 * rank) *reinterpret_cast<i32x4*>(ring + CT * 1024 + 8 * bo[l]) = reg[d][2 * CT + l];
        __builtin_amdgcn_wave_barrier();
      }
      const uint16_t* s = ring + (T ? 0 : d) * kStep;
      const uint16_t* sm = s + CT * 1024;
      auto frag = [&](const uint16_t* p, int t, int h) {   // 16 rows from 16 t, 32 of the step's contraction
        return as_bf16x8(*reinterpret_cast<const i32x4*>(p + (16 * t + l16) * 64 + 8 * ((4 * h + q) ^ ((l16 >> 1) & 7))));
      };
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bf16x8 x[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) x[c] = frag(s, c, h);
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          const bf16x8 w = T ? col_frag(sm, 16 * j, lane,
                                        [&](int r, int c) { return 8 * tr_at(32 * h + r, c >> 3, kPitch) + (c & 7); })
                             : frag(sm, j, h);
#pragma unroll
          for (int c = 0; c < CT; ++c) acc[j][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x[c], acc[j][c], 0, 0, 0);
        }
      }
      issue_order();
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, d);
    for (int it = 0; it < n; it += D)
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if constexpr (!T) wait_vm<(D - 1) * kLoads>();
        mma(d);
        load(d, it + d + D);
      }
    wait_vm<0>();
    __syncthreads();   // every wave is done with its ring
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int c = 0; c < CT; ++c) red[((wave * JT + j) * CT + c) * 64 + lane] = acc[j][c];
    __syncthreads();
    // (row tile j, column tile c): one wave; sum[r]: output 16 j + 4 q + r
#pragma unroll
    for (int t = 0; t < JT * CT; ++t) {
      const int j = t / CT, c = t % CT;
      if (t % kShrinkWaves != wave) continue;
      f32x4 sum = red[t * 64 + lane];
      for (int w = 1; w < kShrinkWaves; ++w) sum += red[(w * JT * CT + t) * 64 + lane];
      const int o = 16 * (j0 + j) + 4 * q;
      if (mine[c] == g && o < rank) {
        uint32_t p[4][3];
#pragma unroll
        for (int r = 0; r < 4; ++r) split3(sc * sum[r], p[r]);
        uint16_t* dst = a.low + (r0 + 16 * c + l16) * kPieces * rank + o;
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
          *reinterpret_cast<uint2*>(dst + k * rank) =
              make_uint2(p[0][k] | (p[1][k] << 16), p[2][k] | (p[3][k] << 16));
      }
    }
    __syncthreads();
  }
}

// ----------------------------------------------------- few rows: streaming --
// y of 16 output features for up to 8 CT rows, the contraction split over the
// waves.  W streams from memory by whole lines: a load covers 8 rows of 128
// bytes, the row slots 2 f and 2 f + 1 of the MFMA are the two halves of
// feature f's line, column c holds row c's activations at the first half,
// column c + 8 at the second, and of the products the matching ones (even
// slot, column < 8) and (odd slot, column >= 8) are added; the others are not
// used.  (Loads of 16 rows by 64 bytes, all products used, reach 28 KB/us on a
// CU; these about 70.)  Wave j also adds the adapters' product of the ranks
// 8 j .. 8 j + 7 to its sums, each row with its own B_g.
// Whole calls by lines / by tiles, us, 1, 16, 32, 48, 64 rows: 4096 x 4096, rank 16
// 11.1/24.5 16.6/27.2 19.7/29.3 25.7/30.5 29.1/31.5; 2048 x 2048, rank 8 9.0/16.1
// 11.0/16.8 13.3/17.1 17.0/17.7 19.6/18.0; N = 4096, K = 14336, rank 16 28.2/60.6
// 33.6/64.7 45.2/65.9 61.7/68.9 71.4/70.9.
constexpr int kStreamWaves = 16;

__device__ __forceinline__ float ror8(float v) {   // lane c of a row of 16: from lane (c + 8) % 16
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x128, 0xf, 0xf, false));
}

struct AdapterPart {   // 8 ranks of one row's s and of two features' B rows
  i32x4 p[kPieces], b[2];
};

template <int CT, int D>
__global__ void __launch_bounds__(64 * kStreamWaves) lora_stream_kernel(LoraArgs a, const uint16_t* __restrict__ x,
                                                                       const uint16_t* __restrict__ w,
                                                                       const uint16_t* __restrict__ b,
                                                                       uint16_t* __restrict__ y, int N, int K) {
  __shared__ float2 red[kStreamWaves * CT * 64];
  const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15, hh = l16 >> 3;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = 16 * blockIdx.x, n = n0 + 8 * hh + 2 * q;   // the lane's features n, n + 1
  const int row0 = l16 & 7;                                  // of row 8 c + row0
  const int rank0 = 8 * wave;
  auto adapter_load = [&](AdapterPart& v, int c) {
    const int64_t r = 8 * c + row0;
    const int g = r < a.R ? row_adapter(a.adapter, r, a.R, a.G) : -1;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) v.p[k] = (i32x4){0, 0, 0, 0};
    v.b[0] = v.b[1] = (i32x4){0, 0, 0, 0};
    if (g >= 0) {
#pragma unroll
      for (int k = 0; k < kPieces; ++k)
        v.p[k] = *reinterpret_cast<const i32x4*>(a.low + (r * kPieces + k) * a.rank + rank0);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v.b[i] = *reinterpret_cast<const i32x4*>(b + ((int64_t)g * N + n + i) * a.rank + rank0);
    }
  };
  auto adapter_add = [&](const AdapterPart& v, float2& sum) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      float s = 0.f;
#pragma unroll
      for (int k = kPieces - 1; k >= 0; --k) s += bf16_to_f32(((uint32_t)v.p[k][u / 2] >> (16 * (u & 1))) & 0xffffu);
      sum.x += s * bf16_to_f32(((uint32_t)v.b[0][u / 2] >> (16 * (u & 1))) & 0xffffu);
      sum.y += s * bf16_to_f32(((uint32_t)v.b[1][u / 2] >> (16 * (u & 1))) & 0xffffu);
    }
  };
  const bool adds = rank0 < a.rank;
  // up to two tiles of rows: requested before the projection's loads
  constexpr int kEarly = CT <= 2 ? CT : 0;
  AdapterPart part[kEarly ? kEarly : 1];
#pragma unroll
  for (int c = 0; c < kEarly; ++c)
    if (adds) adapter_load(part[c], c);

  const __amdgpu_buffer_rsrc_t wr = buffer_rsrc(w + (int64_t)n0 * K, 16ll * K * 2);
  const __amdgpu_buffer_rsrc_t xr = buffer_rsrc(x, a.R * K * 2);
  const uint32_t wo = (uint32_t)((l16 >> 1) * K * 2 + 64 * (l16 & 1) + 16 * q);
  const uint32_t xo = (uint32_t)(row0 * K * 2 + 64 * hh + 16 * q);
  f32x4 acc[2][CT];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[t][c] = (f32x4){0.f, 0.f, 0.f, 0.f};
  struct Step {
    i32x4 w[2], x[CT];
  } st[D];
  const int lines = K / 64;
  auto load = [&](Step& f, int line) {   // past the end: zeros
    const bool in = line < lines;
#pragma unroll
    for (int t = 0; t < 2; ++t)
      f.w[t] = __builtin_amdgcn_raw_buffer_load_b128(wr, in ? wo : kPast, 128 * line + 16 * t * K, 0);
#pragma unroll
    for (int c = 0; c < CT; ++c)
      f.x[c] = __builtin_amdgcn_raw_buffer_load_b128(xr, in && 8 * c + row0 < a.R ? xo : kPast,
                                                     128 * line + 16 * c * K, 0);
    issue_order();
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(st[d], wave + kStreamWaves * d);
  for (int line = wave; line < lines; line += kStreamWaves * D)
#pragma unroll
    for (int d = 0; d < D; ++d) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int c = 0; c < CT; ++c)
          acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(st[d].w[t]), as_bf16x8(st[d].x[c]), acc[t][c], 0, 0, 0);
      issue_order();
      load(st[d], line + kStreamWaves * (d + D));
    }
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    // Lanes l16 < 8 take the first 8 features' sums of their row, the others the
    // second 8.  (Every lane takes part in every exchange.)
    const float e0 = ror8(acc[1][c][0]), o0 = ror8(acc[0][c][1]), e1 = ror8(acc[1][c][2]), o1 = ror8(acc[0][c][3]);
    float2 v;
    v.x = hh ? e0 + acc[1][c][1] : acc[0][c][0] + o0;
    v.y = hh ? e1 + acc[1][c][3] : acc[0][c][2] + o1;
    if (adds) {
      if (!kEarly) adapter_load(part[0], c);
      adapter_add(part[kEarly ? c : 0], v);
    }
    red[(wave * CT + c) * 64 + lane] = v;
  }
  __syncthreads();
  if (wave >= CT) return;
  float2 sum = red[wave * 64 + lane];
  for (int k = 1; k < kStreamWaves; ++k) {
    const float2 v = red[(k * CT + wave) * 64 + lane];
    sum.x += v.x;
    sum.y += v.y;
  }
  const int64_t r = 8 * wave + row0;
  if (r >= a.R) return;
  *reinterpret_cast<uint32_t*>(y + r * N + n) = f32_to_bf16_rne(sum.x) | ((uint32_t)f32_to_bf16_rne(sum.y) << 16);
}

// ----------------------------------------------------------------- wgrad --
// One workgroup: one adapter, 256 columns of x (for dA) or of dy (for dB) and
// a share of the adapter's rows, taken from the rows sorted by adapter.  32
// rows at a time go through LDS, the next 64 on their way in registers: the
// columns (512 bytes a row, swizzled) and the pieces of t or s beside them;
// both operands are read transposed, the rows being the contraction, and the
// three pieces add into the same accumulators.  A wave owns 64 columns: with
// 32 the pieces' fragments, which every wave reads, were most of the LDS
// traffic.  (Through registers, not by loads that write LDS: the compiler
// waits for all of those before a transposing read, 88 us instead of 65
// at 8192 rows, K = 6144, N = 4096, 4 adapters of rank 64.)  With more than
// one share the sums go to the workspace and a second launch adds them in
// order.
constexpr int kWgCols = 256, kWgRows = 32, kWgWaves = 4, kWgList = 1024;

// chunk c of row r: 4 consecutive rows on distinct chunk pairs, rows 8 apart
// on opposite halves of the banks (its own inverse)
__device__ __forceinline__ int wg_chunk(int r, int c) { return c ^ ((r & 3) << 1) ^ (((r >> 3) & 1) << 3); }

template <int JT, bool IS_A>
__device__ __forceinline__ void wgrad_tile(const LoraGradArgs& a, int c0, uint16_t* smem, int32_t* list) {
  constexpr int NT = 64 * kWgWaves;
  constexpr int kColLoads = kWgRows * kWgCols / 8 / NT;                // 16-byte chunks a thread
  constexpr int kLowLoads = (kWgRows * 6 * JT + NT - 1) / NT;          // 32 rows of 3 rank <= 48 JT
  constexpr int kPitch = tr_pitch(6 * JT);                             // chunks
  constexpr int kCols = kWgRows * kWgCols, kBuf = kCols + kWgRows * 8 * kPitch;   // elements
  constexpr int D = 2;                                                 // stages on their way
  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = blockIdx.y;
  const int C = IS_A ? a.K : a.N;
  const int rank = a.rank, pr = kPieces * rank, cpr = pr / 8;   // chunks of a row of low
  const int cnt = a.counts[g];
  const int32_t* rows = a.sorted + a.offsets[g];
  const int i0 = (int)((int64_t)cnt * blockIdx.z / gridDim.z), i1 = (int)((int64_t)cnt * (blockIdx.z + 1) / gridDim.z);
  const __amdgpu_buffer_rsrc_t vr = buffer_rsrc(IS_A ? a.x : a.dy, a.R * C * 2);
  const __amdgpu_buffer_rsrc_t lr = buffer_rsrc(IS_A ? a.low_dy : a.low_x, a.R * pr * 2);
  const int ccol = c0 + 8 * (tid & 31);
  int lrow[kLowLoads], lcol[kLowLoads];   // (row, chunk) of this thread's pieces of low
#pragma unroll
  for (int b = 0; b < kLowLoads; ++b) {
    lrow[b] = (tid + NT * b) / cpr;
    lcol[b] = tid + NT * b - lrow[b] * cpr;
  }
  f32x4 acc[JT][4];
#pragma unroll
  for (int j = 0; j < JT; ++j)
#pragma unroll
    for (int h = 0; h < 4; ++h) acc[j][h] = (f32x4){0.f, 0.f, 0.f, 0.f};

  for (int base = i0; base < i1; base += kWgList) {
    const int m = min(kWgList, i1 - base);   // rows of this part of the list
    for (int i = tid; i < m; i += NT) list[i] = rows[base + i];
    __syncthreads();
    i32x4 vc[D][kColLoads], vl[D][kLowLoads];
    auto load = [&](int d, int st) {   // past the end: zeros
#pragma unroll
      for (int b = 0; b < kColLoads; ++b) {
        const int i = st * kWgRows + (tid >> 5) + NT / 32 * b;
        vc[d][b] = __builtin_amdgcn_raw_buffer_load_b128(
            vr, i < m && ccol < C ? (uint32_t)(list[min(i, m - 1)] * C + ccol) * 2u : kPast, 0, 0);
      }
#pragma unroll
      for (int b = 0; b < kLowLoads; ++b) {
        const int i = st * kWgRows + lrow[b];
        vl[d][b] = __builtin_amdgcn_raw_buffer_load_b128(
            lr, lrow[b] < kWgRows && i < m ? (uint32_t)(list[min(i, m - 1)] * cpr + lcol[b]) * 16u : kPast, 0, 0);
      }
      issue_order();
    };
    const int ns = (m + kWgRows - 1) / kWgRows;
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, d);
    for (int it = 0; it < ns; it += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        uint16_t* cols = smem + (d & 1) * kBuf;
        uint16_t* low = cols + kCols;
#pragma unroll
        for (int b = 0; b < kColLoads; ++b) {
          const int r = (tid >> 5) + NT / 32 * b;
          *reinterpret_cast<i32x4*>(cols + r * kWgCols + 8 * wg_chunk(r, tid & 31)) = vc[d][b];
        }
#pragma unroll
        for (int b = 0; b < kLowLoads; ++b)
          if (lrow[b] < kWgRows) *reinterpret_cast<i32x4*>(low + 8 * tr_at(lrow[b], lcol[b], kPitch)) = vl[d][b];
        issue_order();
        load(d, it + d + D);
        // one barrier a stage: the other buffer's readers have passed it
        lds_barrier();
        bf16x8 f[4];
#pragma unroll
        for (int h = 0; h < 4; ++h)
          f[h] = col_frag(cols, 64 * wave + 16 * h, lane,
                          [&](int r, int c) { return r * kWgCols + 8 * wg_chunk(r, c >> 3) + (c & 7); });
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
#pragma unroll
          for (int j = 0; j < JT; ++j) {
            const bf16x8 t = col_frag(low, p * rank + 16 * j, lane,
                                      [&](int r, int c) { return 8 * tr_at(r, c >> 3, kPitch) + (c & 7); });
#pragma unroll
            for (int h = 0; h < 4; ++h)
              acc[j][h] = IS_A ? __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[h], t, acc[j][h], 0, 0, 0)
                               : __builtin_amdgcn_mfma_f32_16x16x32_bf16(t, f[h], acc[j][h], 0, 0, 0);
          }
      }
    }
    lds_barrier();   // the list and the buffers are read
  }
  // dA [G, rank, K]: lane: output 16 j + l16, columns 4 q ..; dB [G, N, rank]:
  // lane: column l16, outputs 16 j + 4 q ..
  const int64_t na = (int64_t)a.G * rank * a.K, nb = (int64_t)a.G * rank * a.N;
  float* out = gridDim.z > 1 ? a.part + blockIdx.z * (na + nb) + (IS_A ? 0 : na) : IS_A ? a.da : a.db;
  const bool add = gridDim.z == 1 && a.accumulate;
#pragma unroll
  for (int j = 0; j < JT; ++j)
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int col = c0 + 64 * wave + 16 * h + (IS_A ? 4 * q : l16);
      const int o = 16 * j + (IS_A ? l16 : 4 * q);
      if (col >= C || o >= rank) continue;
      f32x4* dst = reinterpret_cast<f32x4*>(out + (IS_A ? ((int64_t)g * rank + o) * a.K + col
                                                        : ((int64_t)g * a.N + col) * rank + o));
      f32x4 r = acc[j][h];
      if (add) {
        const f32x4 old = *dst;
#pragma unroll
        for (int u = 0; u < 4; ++u) r[u] = old[u] + r[u];
      }
      *dst = r;
    }
}

template <int JT>
__global__ void __launch_bounds__(64 * kWgWaves) lora_wgrad_kernel(LoraGradArgs a) {
  __shared__ __attribute__((aligned(16))) uint16_t smem[2 * (kWgRows * kWgCols + kWgRows * 8 * tr_pitch(6 * JT))];
  __shared__ int32_t list[kWgList];
  const int kt = (a.K + kWgCols - 1) / kWgCols;
  if ((int)blockIdx.x < kt) wgrad_tile<JT, true>(a, blockIdx.x * kWgCols, smem, list);
  else wgrad_tile<JT, false>(a, (blockIdx.x - kt) * kWgCols, smem, list);
}

// dA and dB from the shares' sums, four values a thread.
__global__ void __launch_bounds__(256) lora_wgrad_join_kernel(LoraGradArgs a, int shares) {
  const int64_t na = (int64_t)a.G * a.rank * a.K, n = na + (int64_t)a.G * a.rank * a.N;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  f32x4 s = *reinterpret_cast<const f32x4*>(a.part + i);
  for (int k = 1; k < shares; ++k) s += *reinterpret_cast<const f32x4*>(a.part + k * n + i);
  f32x4* dst = reinterpret_cast<f32x4*>(i < na ? a.da + i : a.db + (i - na));
  if (a.accumulate) {
    const f32x4 old = *dst;
#pragma unroll
    for (int u = 0; u < 4; ++u) s[u] = old[u] + s[u];
  }
  *dst = s;
}

template <int JT, int CT, int D>
hipError_t launch_shrink(const LoraArgs& a, const uint16_t* v, const uint16_t* m, int C, bool t, hipStream_t s) {
  const int64_t blocks = (a.R + 16 * CT - 1) / (16 * CT);
  int64_t passes = 1024 / blocks;
  passes = passes < 1 ? 1 : passes > 16 * CT ? 16 * CT : passes;
  const dim3 block(64 * kShrinkWaves);
  if (t)
    hipLaunchKernelGGL((lora_shrink_kernel<JT, CT, true, D>), dim3((unsigned)blocks, (unsigned)passes), block, 0, s, a,
                       v, m, C);
  else
    hipLaunchKernelGGL((lora_shrink_kernel<JT, CT, false, D>),
                       dim3((unsigned)blocks, (unsigned)passes, (unsigned)((a.rank + 16 * JT - 1) / (16 * JT))), block, 0,
                       s, a, v, m, C);
  return hipGetLastError();
}

// low[r] = scale_g (T ? B_g^T : A_g) v_r, contraction C.  With few rows each
// 16 of the rank's outputs go to a workgroup of their own (forward of N = 1024, K
// = 4096, 4 adapters, each on its own / all in one, us: rank 128, 65 rows 39.0 /
// 46.6, 300 47.1 / 48.7, 512 52.5 / 48.7, 1024 66.6 / 52.3; rank 32, 65 rows 28.6 /
// 30.3, 300 32.1 / 31.2, 1024 34.3 / 31.4; 300 rows of 48, rank 32, N = K = 4096,
// 49.2 / 50.0).  (Blocks of 32 rows
// read each adapter's matrix half as often but put one workgroup on a CU: 24
// against 17 us at 8192 x 4096, rank 16, no difference at rank 64.)
hipError_t shrink(const LoraArgs& a, const uint16_t* v, const uint16_t* m, int C, bool t, hipStream_t s) {
  if (a.rank <= 16 || (!t && a.R <= kShrinkSplitRows)) return launch_shrink<1, 1, 4>(a, v, m, C, t, s);
  if (a.rank <= 32) return launch_shrink<2, 1, 3>(a, v, m, C, t, s);
  if (a.rank <= 64) return launch_shrink<4, 1, 2>(a, v, m, C, t, s);
  return launch_shrink<8, 1, 2>(a, v, m, C, t, s);
}

}  // namespace

hipError_t launch_lora_forward(const LoraArgs& a, const uint16_t* x, const uint16_t* w, const uint16_t* am,
                               const uint16_t* b, uint16_t* y, int N, int K, hipStream_t s) {
  if (a.R == 0) return hipSuccess;
  hipError_t e = shrink(a, x, am, K, false, s);
  if (e != hipSuccess) return e;
  if (a.R <= kLoraStreamRows) {
    static_assert(kLoraStreamRows == 64 && kLoraMaxRank <= 8 * kStreamWaves, "8 tiles of rows, 8 ranks a wave");
    const dim3 grid(N / 16), block(64 * kStreamWaves);
    if (a.R <= 8) hipLaunchKernelGGL((lora_stream_kernel<1, 4>), grid, block, 0, s, a, x, w, b, y, N, K);
    else if (a.R <= 16) hipLaunchKernelGGL((lora_stream_kernel<2, 3>), grid, block, 0, s, a, x, w, b, y, N, K);
    else if (a.R <= 32) hipLaunchKernelGGL((lora_stream_kernel<4, 2>), grid, block, 0, s, a, x, w, b, y, N, K);
    else hipLaunchKernelGGL((lora_stream_kernel<8, 1>), grid, block, 0, s, a, x, w, b, y, N, K);
    return hipGetLastError();
  }
  return launch_tile_lora_bf16(a, x, w, b, y, K, N, false, s);
}

hipError_t launch_lora_dgrad(const LoraArgs& a, const uint16_t* dy, const uint16_t* w, const uint16_t* am,
                             const uint16_t* b, uint16_t* dx, int N, int K, hipStream_t s) {
  if (a.R == 0) return hipSuccess;
  hipError_t e = shrink(a, dy, b, N, true, s);
  if (e != hipSuccess) return e;
  return launch_tile_lora_bf16(a, dy, w, am, dx, N, K, true, s);
}

// Shares of each adapter's rows: at most two workgroups per CU, 256 rows of an
// even split at least.  1 / 2 / 3 / 4 / 8 / 16 shares, whole call, us: 8192 rows of
// 4, 4096 x 6144, rank 64 (rule: 3) 87 / 73 / 62 / 73 / 84 / 119; 1001 of 3, 2048 x
// 2048, rank 8 (4) 16.8 / 15.5 / 14.7 / 15.0 / 16.5 / 21.0; 4096 of one, 1024 x 1024,
// rank 32 (16) 111 / 65 / 50 / 42 / 31 / 29; 300 of 48, 4096 x 4096, rank 32 (1) 26 /
// 65 / 86 / 107 / 229 / 412.
int32_t lora_wgrad_shares(int64_t R, int64_t N, int64_t K, int64_t G) {
  const int64_t wgs = G * ((K + kWgCols - 1) / kWgCols + (N + kWgCols - 1) / kWgCols);
  int64_t n = 512 / wgs;
  const int64_t most = (R + 255) / 256;
  if (n > most) n = most;
  return (int32_t)(n < 1 ? 1 : n > 16 ? 16 : n);
}

hipError_t launch_lora_wgrad(const LoraGradArgs& a, int32_t shares, hipStream_t s) {
  const dim3 grid((unsigned)((a.K + kWgCols - 1) / kWgCols + (a.N + kWgCols - 1) / kWgCols), (unsigned)a.G,
                  (unsigned)shares);
  const dim3 block(64 * kWgWaves);
  if (a.rank <= 16) hipLaunchKernelGGL((lora_wgrad_kernel<1>), grid, block, 0, s, a);
  else if (a.rank <= 32) hipLaunchKernelGGL((lora_wgrad_kernel<2>), grid, block, 0, s, a);
  else if (a.rank <= 64) hipLaunchKernelGGL((lora_wgrad_kernel<4>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((lora_wgrad_kernel<8>), grid, block, 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || shares == 1) return e;
  const int64_t n = (int64_t)a.G * a.rank * (a.K + a.N) / 4;
  hipLaunchKernelGGL(lora_wgrad_join_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a, shares);
  return hipGetLastError();
}

}  // namespace moe

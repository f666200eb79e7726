// The C ABI declared in include/moe_mi355x.h: validation, planning,
// workspace layout and the launch sequences.  Host code, plus the one device
// array that moe_apply_contiguous_static uses as its workspace; it enqueues
// kernels on the caller's stream and never allocates or synchronises.
#include <stdio.h>
#include <string.h>

#include <mutex>

#include "../../include/moe_mi355x.h"
#include "kernels.h"

using namespace moe;

namespace {

constexpr int64_t kAlign = 256;
inline int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
inline bool aligned16(const void* p) { return p && ((uintptr_t)p & 15u) == 0; }
inline bool aligned4(const void* p) { return p && ((uintptr_t)p & 3u) == 0; }
// MXFP8 weights, with row-major or grouped scale arrays
inline bool is_mxfp8(const moe_problem& P) { return P.w_dtype == MOE_W_MXFP8 || P.w_dtype == MOE_W_MXFP8_GROUPED; }

int fail(moe_plan* plan, int code, const char* msg) {
  if (plan) snprintf(plan->reason, sizeof(plan->reason), "%s", msg);
  return code;
}

struct AlignLayout {
  int64_t counts, offsets, sorted, block_bucket, num_post, active, status, scratch, end;
};

AlignLayout layout_align(int64_t base, int64_t nb, int64_t capacity, int64_t max_tiles,
                         int64_t max_active, int64_t nblocks) {
  AlignLayout L;
  int64_t o = base;
  L.counts = o;       o = up(o + 4 * nb, kAlign);
  L.offsets = o;      o = up(o + 4 * (nb + 1), kAlign);
  L.sorted = o;       o = up(o + 4 * capacity, kAlign);
  L.block_bucket = o; o = up(o + 4 * max_tiles, kAlign);
  L.num_post = o;     o = up(o + 4, kAlign);
  L.active = o;       o = up(o + 4 * (max_active + 1), kAlign);
  L.status = o;       o = up(o + 16, kAlign);
  L.scratch = o;      o = up(o + 4 * nblocks * (nb + 1), kAlign);
  L.end = o;
  return L;
}

int64_t align_nblocks_of(int64_t R) {
  const int64_t n = (R + kAlignChunk - 1) / kAlignChunk;
  return n < kAlignMaxBlocks ? n : kAlignMaxBlocks;
}
int64_t align_nblocks(int64_t R) { return R <= kAlignSmallMaxR ? 0 : align_nblocks_of(R); }

template <typename T>
T* at(void* base, int64_t off) { return reinterpret_cast<T*>(static_cast<char*>(base) + off); }

AlignArgs align_args(const moe_plan* p, const int32_t* keys, const int32_t* expert_map, void* ws13) {
  AlignArgs a{};
  a.keys = keys;
  a.key_map = expert_map;
  a.key_range = (int32_t)p->prob.global_experts;
  a.R = p->routes;
  a.nb = (int32_t)p->prob.E;
  a.B = p->block_m;
  a.counts = at<int32_t>(ws13, p->off_counts);
  a.offsets = at<int32_t>(ws13, p->off_offsets);
  a.sorted = at<int32_t>(ws13, p->off_sorted_ids);
  a.block_bucket = at<int32_t>(ws13, p->off_block_expert);
  a.num_post = at<int32_t>(ws13, p->off_num_post_padded);
  a.active = at<int32_t>(ws13, p->off_active);
  a.status = at<int32_t>(ws13, p->off_status);
  a.block_hist = at<int32_t>(ws13, p->off_align_scratch);
  a.capacity = p->sorted_capacity;
  a.max_tiles = p->max_tiles;
  a.max_active = p->max_active;
  a.sentinel = (int32_t)p->routes;
  a.nblocks = (int32_t)p->align_blocks;
  return a;
}

}  // namespace

// ------------------------------------------------ the allocation-free call ----
// The workspaces of moe_apply_contiguous_static: one array per GPU, held from
// the library's load until the process ends.  Host code never uses the
// array's name as an address (in host code it names a host-side stand-in);
// it takes the device address hipGetSymbolAddress returns for the current
// device, once per device.
static __device__ __align__(256) uint8_t scratch[MOE_STATIC_SCRATCH_BYTES];

namespace {
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices];

// Device address of `scratch` on the current device, or nullptr.
void* scratch_on_current_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* ptr = nullptr;
    if (hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)) != hipSuccess || !ptr) return nullptr;
    g_scratch_ptr[dev] = ptr;
  }
  return g_scratch_ptr[dev];
}
}  // namespace

extern "C" {

int moe_abi_version(void) { return MOE_ABI_VERSION; }

const char* moe_status_string(int status) {
  switch (status) {
    case MOE_OK: return "ok";
    case MOE_EINVAL: return "invalid argument";
    case MOE_EUNSUPPORTED: return "unsupported problem";
    case MOE_EHIP: return "HIP launch error";
    default: return "unknown status";
  }
}

void moe_struct_sizes(int64_t* problem, int64_t* plan, int64_t* weights) {
  if (problem) *problem = sizeof(moe_problem);
  if (plan) *plan = sizeof(moe_plan);
  if (weights) *weights = sizeof(moe_weights);
}

const char* moe_plan_reason(const moe_plan* plan) { return plan ? plan->reason : ""; }

int moe_plan_init(moe_plan* plan, const moe_problem* prob) {
  if (!plan || !prob) return MOE_EINVAL;
  memset(plan, 0, sizeof(*plan));
  plan->prob = *prob;
  plan->abi_version = MOE_ABI_VERSION;
  const moe_problem& P = *prob;
  if (P.M <= 0 || P.K <= 0 || P.I <= 0 || P.E <= 0)
    return fail(plan, MOE_EINVAL, "M, K, I and E must be positive");
  if (P.layout != MOE_LAYOUT_CONTIGUOUS && P.layout != MOE_LAYOUT_BATCHED)
    return fail(plan, MOE_EINVAL, "unknown layout");
  if (P.w_dtype != MOE_W_BF16 && !is_mxfp8(P))
    return fail(plan, MOE_EINVAL, "unknown weight dtype");
  if (P.w1_order != MOE_W1_HALVES && P.w1_order != MOE_W1_INTERLEAVE16)
    return fail(plan, MOE_EINVAL, "unknown W1 row order");
  if (P.variant < MOE_VARIANT_AUTO || P.variant > MOE_VARIANT_FUSED)
    return fail(plan, MOE_EINVAL, "unknown variant");
  const bool contiguous = P.layout == MOE_LAYOUT_CONTIGUOUS;
  if (contiguous) {
    if (P.global_experts != 0 && (P.global_experts < P.E || P.global_experts >= (1ll << 31)))
      return fail(plan, MOE_EINVAL, "global_experts must be 0 or in [E, 2^31)");
    const int64_t id_space = P.global_experts ? P.global_experts : P.E;
    if (P.topk <= 0 || P.topk > id_space)
      return fail(plan, MOE_EINVAL, "topk must be in [1, E] (or [1, global_experts])");
  } else {
    if (P.max_tokens <= 0) return fail(plan, MOE_EINVAL, "max_tokens must be positive");
    if (P.global_experts != 0) return fail(plan, MOE_EINVAL, "the batched format takes local experts only");
  }
  const int64_t R = contiguous ? P.M * P.topk : P.E * P.max_tokens;
  // flat slot ids, positions and the sentinel are int32; rows are addressed
  // in 64-bit, so only these ranges matter
  if (R >= (1ll << 31) - 1 || P.M >= (1ll << 31) || P.E > kAlignMaxBuckets)
    return fail(plan, MOE_EINVAL, "routes or experts past the 32-bit index range");
  if (P.w1_order == MOE_W1_INTERLEAVE16 && P.I % 16)
    return fail(plan, MOE_EINVAL, "the 16-row interleave needs I % 16 == 0");

  int variant = P.variant;
  if (is_mxfp8(P)) {
    if (!contiguous)
      return fail(plan, MOE_EUNSUPPORTED, "MXFP8 weights are built for the contiguous format only");
    if (variant == MOE_VARIANT_FUSED)
      return fail(plan, MOE_EUNSUPPORTED, "MXFP8 weights have no single-launch kernel");
    if (P.K % 128 || P.I % 128)
      return fail(plan, MOE_EUNSUPPORTED, "MXFP8 kernels need K % 128 == 0 and I % 128 == 0");
    if (2 * P.I * P.K >= (1ll << 31))
      return fail(plan, MOE_EUNSUPPORTED, "MXFP8 kernels address one expert with 32-bit offsets");
    // the tiles (128 weight rows: 64 W1 features, 128 W2 rows, covered by
    // the checks above) unless the streaming kernels are asked for
    if (variant == MOE_VARIANT_AUTO) variant = MOE_VARIANT_TILE;
    if (P.w_dtype == MOE_W_MXFP8_GROUPED) {
      if (variant != MOE_VARIANT_TILE)
        return fail(plan, MOE_EUNSUPPORTED, "grouped MXFP8 scales are read by the tile kernels only");
      if (P.K % 512 || P.I % 512)
        return fail(plan, MOE_EUNSUPPORTED, "grouped MXFP8 scales need K % 512 == 0 and I % 512 == 0");
    }
    if (variant == MOE_VARIANT_TILE) {
      snprintf(plan->reason, sizeof(plan->reason),
               "tile (MXFP8): 128 weight rows x 64 routes per workgroup, both operands staged in LDS");
    } else {
      snprintf(plan->reason, sizeof(plan->reason),
               "stream (MXFP8): weight rows streamed into scaled MFMA, 64 tokens per pass");
    }
  } else {
    if (variant == MOE_VARIANT_AUTO) {
      // small layers (all weights within 1 GiB, at most 32 rows per expert
      // that can hold a route, one-workgroup align): one launch plus the
      // reduce, where launch latency is most of the time; few rows per
      // expert: the two streaming launches; otherwise the tiles
      const int64_t slots = P.E < R ? P.E : R;
      const bool small = 6 * P.E * P.I * P.K <= (1ll << 30) && R <= 32 * slots && R <= kAlignSmallMaxR &&
                         P.E <= kFusedMaxExperts && P.K % 128 == 0 && P.I % 128 == 0;
      variant = !contiguous ? MOE_VARIANT_TILE
                : small     ? MOE_VARIANT_FUSED
                : P.M <= 16 ? MOE_VARIANT_STREAM
                            : MOE_VARIANT_TILE;
    }
    if (variant == MOE_VARIANT_STREAM || variant == MOE_VARIANT_FUSED) {
      if (!contiguous) return fail(plan, MOE_EUNSUPPORTED, "the streaming kernels take the contiguous format only");
      if (P.K % 128 || P.I % 128)
        return fail(plan, MOE_EUNSUPPORTED, "streaming kernels need K % 128 == 0 and I % 128 == 0");
      // 32-bit buffer offsets: one expert's W1 and the activation buffers
      if (4 * P.I * P.K >= (1ll << 31) || 2 * P.M * P.K >= (1ll << 31))
        return fail(plan, MOE_EUNSUPPORTED, "streaming kernels address one expert with 32-bit offsets");
      if (variant == MOE_VARIANT_FUSED) {
        if (R > kAlignSmallMaxR || P.E > kFusedMaxExperts)
          return fail(plan, MOE_EUNSUPPORTED, "the single-launch kernel needs M*topk <= 8192 and E <= 2048");
        snprintf(plan->reason, sizeof(plan->reason),
                 "fused: align, W1 and W2 streaming strips in one launch (device work queue), then the reduce");
      } else {
        snprintf(plan->reason, sizeof(plan->reason),
                 "stream: M <= 16 rows per expert, weights streamed into the MFMA row operand");
      }
    } else {
      // 32-bit buffer offsets: one expert's W1, the activation rows and z
      const int64_t act_rows = contiguous ? P.M : P.E * P.max_tokens;
      if (4 * P.I * P.K >= (1ll << 31) || 2 * act_rows * P.K >= (1ll << 31) ||
          2 * (contiguous ? R + P.E * kTileRoutesContiguous : act_rows) * P.I >= (1ll << 31))
        return fail(plan, MOE_EUNSUPPORTED, "tiled kernels address one expert and the activations with 32-bit offsets");
      if (contiguous) {
        if (P.K % 256 || P.I % 128)
          return fail(plan, MOE_EUNSUPPORTED, "contiguous tiled kernels need K % 256 == 0 and I % 128 == 0");
        snprintf(plan->reason, sizeof(plan->reason),
                 "tile: 256 weight rows x 256 routes per workgroup, slices loaded straight into LDS");
      } else {
        if (P.K % 128 || P.I % 64)
          return fail(plan, MOE_EUNSUPPORTED, "batched tiled kernels need K % 128 == 0 and I % 64 == 0");
        snprintf(plan->reason, sizeof(plan->reason),
                 "tile: 128 weight rows x 128 rows per workgroup, route-tile-major order");
      }
    }
  }
  plan->variant = variant;
  plan->block_m = variant != MOE_VARIANT_TILE   ? 16
                  : !contiguous                  ? kTileRowsBatched
                  : is_mxfp8(P)                  ? kTileRoutesMxfp8
                                                 : kTileRoutesContiguous;
  plan->reduce_kind = contiguous ? MOE_REDUCE_NOOP : MOE_REDUCE_NAIVE_BATCHED;
  plan->routes = R;
  const int64_t B = plan->block_m;
  if (contiguous) {
    plan->max_active = P.E < R ? P.E : R;
    plan->max_tiles = (R + plan->max_active * (B - 1)) / B;
    plan->sorted_capacity = plan->max_tiles * B;
    plan->align_blocks = variant == MOE_VARIANT_FUSED ? 0 : align_nblocks(R);
  } else {
    plan->max_active = P.E;
    plan->max_tiles = 0;
    plan->sorted_capacity = 0;
    plan->align_blocks = 0;
  }
  if (plan->max_tiles > 65535 || plan->max_active > 65535)
    return fail(plan, MOE_EUNSUPPORTED, "grid too large");
  if (contiguous && (variant != MOE_VARIANT_TILE || is_mxfp8(P))) {
    // the streaming and MXFP8 kernels read z (and for MXFP8 the gathered
    // activation codes) through one buffer resource with 32-bit offsets,
    // whose range check stops at 2^31 - 1 bytes: rows past it would read 0
    const int64_t zbytes = plan->sorted_capacity * P.I * (is_mxfp8(P) ? 1 : 2);
    const int64_t xqbytes = is_mxfp8(P) ? plan->sorted_capacity * P.K : 0;
    if (zbytes >= (1ll << 31) - 1 || xqbytes >= (1ll << 31) - 1)
      return fail(plan, MOE_EUNSUPPORTED,
                  "streaming/MXFP8 kernels address z and the gathered activations with 32-bit offsets");
  }

  AlignLayout L = layout_align(0, P.E, plan->sorted_capacity, plan->max_tiles, plan->max_active,
                               plan->align_blocks);
  plan->off_counts = L.counts;
  plan->off_offsets = L.offsets;
  plan->off_sorted_ids = L.sorted;
  plan->off_block_expert = L.block_bucket;
  plan->off_num_post_padded = L.num_post;
  plan->off_active = L.active;
  plan->off_status = L.status;
  plan->off_align_scratch = L.scratch;
  int64_t o = L.end;
  const int64_t zrows = contiguous ? plan->sorted_capacity : P.E * P.max_tokens;
  plan->off_z = o;
  if (is_mxfp8(P)) {
    o = up(o + zrows * P.I, kAlign);
    plan->off_z_scale = o;
    o = up(o + zrows * (P.I / 32), kAlign);
    plan->off_xq = o;
    o = up(o + zrows * P.K, kAlign);
    plan->off_xq_scale = o;
    o = up(o + zrows * (P.K / 32), kAlign);
  } else {
    o = up(o + zrows * P.I * 2, kAlign);
    plan->off_z_scale = plan->off_xq = plan->off_xq_scale = -1;
  }
  if (variant == MOE_VARIANT_FUSED) {
    plan->off_sync = o;
    o = up(o + 4 * sync_words(plan->max_active), kAlign);
  } else {
    plan->off_sync = -1;
  }
  plan->ws13_bytes = o;
  plan->ws2_bytes = contiguous ? up(R * P.K * 2, kAlign) : 0;
  plan->out_rows = contiguous ? P.M : P.E * P.max_tokens;
  plan->out_cols = P.K;
  return MOE_OK;
}

// An expert map is given exactly when the plan's ids are global.
static bool map_ok(const moe_plan* plan, const int32_t* expert_map) {
  return plan->prob.global_experts ? aligned4(expert_map) : expert_map == nullptr;
}

int moe_align_permute(const moe_plan* plan, const int32_t* topk_ids, const int32_t* expert_map,
                      void* ws13, void* stream) {
  if (!plan || plan->abi_version != MOE_ABI_VERSION) return MOE_EINVAL;
  if (plan->prob.layout != MOE_LAYOUT_CONTIGUOUS) return MOE_EINVAL;
  if (!aligned4(topk_ids) || !aligned16(ws13) || !map_ok(plan, expert_map)) return MOE_EINVAL;
  AlignArgs a = align_args(plan, topk_ids, expert_map, ws13);
  return launch_align(a, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_EHIP;
}

static GemmArgs gemm_common(const moe_plan* p, void* ws13) {
  GemmArgs g{};
  const moe_problem& P = p->prob;
  g.rows.layout = P.layout;
  g.rows.sorted_ids = at<int32_t>(ws13, p->off_sorted_ids);
  g.rows.block_expert = at<int32_t>(ws13, p->off_block_expert);
  g.rows.num_post = at<int32_t>(ws13, p->off_num_post_padded);
  g.rows.offsets = at<int32_t>(ws13, p->off_offsets);
  g.rows.counts = at<int32_t>(ws13, p->off_counts);
  g.rows.active = at<int32_t>(ws13, p->off_active);
  g.rows.topk = (int32_t)P.topk;
  g.rows.sentinel = (int32_t)p->routes;
  g.rows.max_tokens = (int32_t)P.max_tokens;
  g.I = (int32_t)P.I;
  g.w1_order = P.w1_order;
  g.E = (int32_t)P.E;
  g.max_tiles = p->max_tiles;
  g.max_active = p->max_active;
  return g;
}

static bool contiguous_args_ok(const moe_plan* plan, const moe_weights* w) {
  if (!plan || plan->abi_version != MOE_ABI_VERSION || !w) return false;
  const moe_problem& P = plan->prob;
  if (P.layout != MOE_LAYOUT_CONTIGUOUS) return false;
  if (!aligned16(w->w1) || !aligned16(w->w2)) return false;
  if (P.w_dtype == MOE_W_MXFP8 && (!aligned4(w->w1_scale) || !aligned4(w->w2_scale))) return false;
  if (P.w_dtype == MOE_W_MXFP8_GROUPED && (!aligned16(w->w1_scale) || !aligned16(w->w2_scale))) return false;
  return true;
}

static GemmArgs w1_args(const moe_plan* plan, const moe_weights* w, void* ws13) {
  const moe_problem& P = plan->prob;
  GemmArgs g = gemm_common(plan, ws13);
  g.epi = kEpiGateUp;
  g.w = w->w1;
  g.w_scale = w->w1_scale;
  g.w_expert_stride = 2 * P.I * P.K;
  g.kdim = (int32_t)P.K;
  g.nfeat = (int32_t)P.I;
  g.out = at<void>(ws13, plan->off_z);
  g.out_ld = P.I;
  return g;
}

static GemmArgs w2_args(const moe_plan* plan, const moe_weights* w, void* ws13, void* ws2) {
  const moe_problem& P = plan->prob;
  GemmArgs g = gemm_common(plan, ws13);
  g.epi = kEpiDown;
  g.w = w->w2;
  g.w_scale = w->w2_scale;
  g.w_expert_stride = P.K * P.I;
  g.kdim = (int32_t)P.I;
  g.nfeat = (int32_t)P.K;
  g.act = at<void>(ws13, plan->off_z);
  g.act_ld = P.I;
  g.act_bytes = plan->sorted_capacity * P.I * 2;
  g.out = ws2;
  g.out_ld = P.K;
  return g;
}

// Grouped MXFP8 scales: bytes between the 16-byte groups of the gathered
// activations' and z's scale arrays (sorted_capacity rows each); 0 for
// row-major scales.
static int64_t scale_group(const moe_plan* plan) {
  return plan->prob.w_dtype == MOE_W_MXFP8_GROUPED ? plan->sorted_capacity * 16 : 0;
}

static int gate_up_act(const moe_plan* plan, const void* a, const moe_weights* w, void* ws13,
                       hipStream_t s) {
  const moe_problem& P = plan->prob;
  GemmArgs g = w1_args(plan, w, ws13);
  if (is_mxfp8(P)) {
    uint8_t* xq = at<uint8_t>(ws13, plan->off_xq);
    uint8_t* xqs = at<uint8_t>(ws13, plan->off_xq_scale);
    g.scale_group = scale_group(plan);
    if (launch_quantize_gather_mxfp8(static_cast<const uint16_t*>(a), g.rows.sorted_ids,
                                     g.rows.num_post, (int32_t)P.topk, g.rows.sentinel,
                                     plan->sorted_capacity, P.K, xq, xqs, g.scale_group, s) != hipSuccess)
      return MOE_EHIP;
    g.act = xq;
    g.act_scale = xqs;
    g.act_ld = P.K;
    g.act_bytes = plan->sorted_capacity * P.K;
    g.out_scale = at<uint8_t>(ws13, plan->off_z_scale);
    const hipError_t e = plan->variant == MOE_VARIANT_TILE ? launch_gemm_tile_mxfp8(g, s) : launch_gemm_stream_mxfp8(g, s);
    return e == hipSuccess ? MOE_OK : MOE_EHIP;
  }
  g.act = a;
  g.act_ld = P.K;
  g.act_bytes = P.M * P.K * 2;
  hipError_t e = plan->variant != MOE_VARIANT_TILE ? launch_gemm_stream_bf16(g, s)
                                                     : launch_gemm_tile_bf16(g, s);
  return e == hipSuccess ? MOE_OK : MOE_EHIP;
}

static int down_unpermute(const moe_plan* plan, const moe_weights* w, void* ws13, void* ws2,
                          hipStream_t s) {
  const moe_problem& P = plan->prob;
  GemmArgs g = w2_args(plan, w, ws13, ws2);
  hipError_t e;
  if (is_mxfp8(P)) {
    g.act_scale = at<uint8_t>(ws13, plan->off_z_scale);
    g.scale_group = scale_group(plan);
    g.act_bytes = plan->sorted_capacity * P.I;
    e = plan->variant == MOE_VARIANT_TILE ? launch_gemm_tile_mxfp8(g, s) : launch_gemm_stream_mxfp8(g, s);
  } else {
    e = plan->variant != MOE_VARIANT_TILE ? launch_gemm_stream_bf16(g, s)
                                            : launch_gemm_tile_bf16(g, s);
  }
  return e == hipSuccess ? MOE_OK : MOE_EHIP;
}

int moe_gate_up_act(const moe_plan* plan, const void* a, const moe_weights* w, void* ws13,
                    void* stream) {
  if (!contiguous_args_ok(plan, w) || !aligned16(a) || !aligned16(ws13)) return MOE_EINVAL;
  return gate_up_act(plan, a, w, ws13, (hipStream_t)stream);
}

int moe_down_unpermute(const moe_plan* plan, const moe_weights* w, void* ws13, void* ws2,
                       void* stream) {
  if (!contiguous_args_ok(plan, w) || !aligned16(ws13) || !aligned16(ws2)) return MOE_EINVAL;
  return down_unpermute(plan, w, ws13, ws2, (hipStream_t)stream);
}

// The launches of moe_apply_contiguous (arguments already validated).
static int apply_contiguous(const moe_plan* plan, const void* a, const int32_t* topk_ids,
                            const float* topk_weights, const moe_weights* w, void* out, void* ws13,
                            void* ws2, hipStream_t s) {
  const moe_problem& P = plan->prob;
  AlignArgs al = align_args(plan, topk_ids, w->expert_map, ws13);
  if (plan->variant == MOE_VARIANT_FUSED) {
    FusedArgs f{};
    f.align = al;
    f.w1 = w1_args(plan, w, ws13);
    f.w1.act = a;
    f.w1.act_ld = P.K;
    f.w1.act_bytes = P.M * P.K * 2;
    f.w2 = w2_args(plan, w, ws13, ws2);
    f.sync = at<int32_t>(ws13, plan->off_sync);
    f.max_active = plan->max_active;
    if (launch_fused_stream_bf16(f, s) != hipSuccess) return MOE_EHIP;
  } else {
    if (launch_align(al, s) != hipSuccess) return MOE_EHIP;
    int st = gate_up_act(plan, a, w, ws13, s);
    if (st != MOE_OK) return st;
    st = down_unpermute(plan, w, ws13, ws2, s);
    if (st != MOE_OK) return st;
  }
  const bool fused = plan->variant == MOE_VARIANT_FUSED;
  hipError_t e = launch_reduce_contiguous(static_cast<const uint16_t*>(ws2), topk_ids, topk_weights,
                                          w->expert_map, (int32_t)P.global_experts,
                                          static_cast<uint16_t*>(out), P.M, (int32_t)P.topk, P.K,
                                          (int32_t)P.E,
                                          fused ? at<int32_t>(ws13, plan->off_sync) : nullptr,
                                          fused ? sync_counter_lines(plan->max_active) : 0, s);
  return e == hipSuccess ? MOE_OK : MOE_EHIP;
}

static bool apply_args_ok(const moe_plan* plan, const void* a, const int32_t* topk_ids,
                          const float* topk_weights, const moe_weights* w, const void* out) {
  return contiguous_args_ok(plan, w) && map_ok(plan, w->expert_map) && aligned16(a) &&
         aligned4(topk_ids) && aligned4(topk_weights) && aligned16(out);
}

int moe_apply_contiguous(const moe_plan* plan, const void* a, const int32_t* topk_ids,
                         const float* topk_weights, const moe_weights* w, void* out, void* ws13,
                         void* ws2, void* stream) {
  if (!apply_args_ok(plan, a, topk_ids, topk_weights, w, out) || !aligned16(ws13) || !aligned16(ws2))
    return MOE_EINVAL;
  return apply_contiguous(plan, a, topk_ids, topk_weights, w, out, ws13, ws2, (hipStream_t)stream);
}

int moe_apply_contiguous_static(const moe_plan* plan, const void* a, const int32_t* topk_ids,
                                const float* topk_weights, const moe_weights* w, void* out,
                                void* stream) {
  if (!apply_args_ok(plan, a, topk_ids, topk_weights, w, out)) return MOE_EINVAL;
  const int64_t ws2_off = up(plan->ws13_bytes, kAlign);
  if (plan->ws13_bytes <= 0 || ws2_off + plan->ws2_bytes > (int64_t)MOE_STATIC_SCRATCH_BYTES)
    return MOE_EUNSUPPORTED;
  uint8_t* base = static_cast<uint8_t*>(scratch_on_current_device());
  if (!base) return MOE_EHIP;
  hipStream_t s = (hipStream_t)stream;
  void* ws13 = base;
  void* ws2 = base + ws2_off;
  // The array keeps whatever the previous call (of any plan) left in it.
  // Every buffer the kernels read is written earlier in the same call,
  // except the single-launch variant's work-queue counters and the status
  // words it counts into: clear those first, with a kernel rather than a
  // memset node, so the call stays capturable.
  if (launch_zero_words(at<int32_t>(ws13, plan->off_status), 4, 1, s) != hipSuccess) return MOE_EHIP;
  if (plan->variant == MOE_VARIANT_FUSED &&
      launch_zero_words(at<int32_t>(ws13, plan->off_sync), sync_counter_lines(plan->max_active), kSyncLine,
                        s) != hipSuccess)
    return MOE_EHIP;
  return apply_contiguous(plan, a, topk_ids, topk_weights, w, out, ws13, ws2, s);
}

int moe_apply_batched(const moe_plan* plan, const void* a, const int32_t* expert_num_tokens,
                      const moe_weights* w, void* y, void* ws13, void* stream) {
  if (!plan || plan->abi_version != MOE_ABI_VERSION || !w) return MOE_EINVAL;
  const moe_problem& P = plan->prob;
  if (P.layout != MOE_LAYOUT_BATCHED) return MOE_EINVAL;
  if (!aligned16(a) || !aligned4(expert_num_tokens) || !aligned16(y) || !aligned16(ws13) ||
      !aligned16(w->w1) || !aligned16(w->w2))
    return MOE_EINVAL;
  hipStream_t s = (hipStream_t)stream;
  GemmArgs g1 = gemm_common(plan, ws13);
  g1.rows.counts = expert_num_tokens;
  g1.epi = kEpiGateUp;
  g1.act = a;
  g1.act_ld = P.K;
  g1.act_bytes = P.E * P.max_tokens * P.K * 2;
  g1.w = w->w1;
  g1.w_expert_stride = 2 * P.I * P.K;
  g1.kdim = (int32_t)P.K;
  g1.nfeat = (int32_t)P.I;
  g1.out = at<void>(ws13, plan->off_z);
  g1.out_ld = P.I;
  GemmArgs g2 = g1;
  g2.epi = kEpiDown;
  g2.act = at<void>(ws13, plan->off_z);
  g2.act_ld = P.I;
  g2.act_bytes = P.E * P.max_tokens * P.I * 2;
  g2.w = w->w2;
  g2.w_expert_stride = P.K * P.I;
  g2.kdim = (int32_t)P.I;
  g2.nfeat = (int32_t)P.K;
  g2.out = y;
  g2.out_ld = P.K;
  if (launch_gemm_tile_bf16(g1, s) != hipSuccess) return MOE_EHIP;
  if (launch_gemm_tile_bf16(g2, s) != hipSuccess) return MOE_EHIP;
  return MOE_OK;
}

int moe_topk_reduce_contiguous(const moe_plan* plan, const void* y, const int32_t* topk_ids,
                               const float* topk_weights, const int32_t* expert_map, void* out,
                               void* stream) {
  if (!plan || plan->abi_version != MOE_ABI_VERSION) return MOE_EINVAL;
  const moe_problem& P = plan->prob;
  if (P.layout != MOE_LAYOUT_CONTIGUOUS) return MOE_EINVAL;
  if (!aligned16(y) || !aligned4(topk_ids) || !aligned4(topk_weights) || !aligned16(out) ||
      !map_ok(plan, expert_map))
    return MOE_EINVAL;
  hipError_t e = launch_reduce_contiguous(static_cast<const uint16_t*>(y), topk_ids, topk_weights,
                                          expert_map, (int32_t)P.global_experts,
                                          static_cast<uint16_t*>(out), P.M, (int32_t)P.topk, P.K,
                                          (int32_t)P.E, nullptr, 0, (hipStream_t)stream);
  return e == hipSuccess ? MOE_OK : MOE_EHIP;
}

static AlignLayout batched_reduce_layout(const moe_plan* p, int64_t n_out) {
  const int64_t R = p->prob.E * p->prob.max_tokens;
  const int64_t max_active = n_out < R ? n_out : R;
  // the first 256 bytes hold the status word (out-of-range tokens seen)
  return layout_align(kAlign, n_out, R, R, max_active, align_nblocks(R));
}

int64_t moe_naive_batched_ws_bytes(const moe_plan* plan, int64_t n_out) {
  if (!plan || plan->prob.layout != MOE_LAYOUT_BATCHED || n_out <= 0 || n_out > kAlignMaxBuckets)
    return -1;
  return batched_reduce_layout(plan, n_out).end;
}

int moe_topk_reduce_naive_batched(const moe_plan* plan, const void* y,
                                  const int32_t* expert_num_tokens, const int32_t* row_token,
                                  const float* row_weight, int64_t n_out, void* out, void* ws,
                                  void* stream) {
  if (!plan || plan->abi_version != MOE_ABI_VERSION) return MOE_EINVAL;
  const moe_problem& P = plan->prob;
  if (P.layout != MOE_LAYOUT_BATCHED || n_out <= 0 || n_out > kAlignMaxBuckets) return MOE_EINVAL;
  if (!aligned16(y) || !aligned4(expert_num_tokens) || !aligned4(row_token) ||
      !aligned4(row_weight) || !aligned16(out) || !aligned16(ws))
    return MOE_EINVAL;
  const int64_t R = P.E * P.max_tokens;
  hipStream_t s = (hipStream_t)stream;
  if (P.K <= 8192 && P.E <= kReduceBatchedMaxE) {
    // one launch: each token's workgroup finds its rows itself
    const hipError_t e = launch_reduce_batched(static_cast<const uint16_t*>(y), expert_num_tokens, row_token,
                                               row_weight, (int32_t)P.max_tokens, (int32_t)P.E,
                                               static_cast<uint16_t*>(out), n_out, P.K, at<int32_t>(ws, 0), s);
    return e == hipSuccess ? MOE_OK : MOE_EHIP;
  }
  AlignLayout L = batched_reduce_layout(plan, n_out);
  AlignArgs a{};
  a.keys = row_token;
  a.R = R;
  a.nb = (int32_t)n_out;
  a.B = 1;
  a.group_count = expert_num_tokens;
  a.rows_per_group = (int32_t)P.max_tokens;
  a.counts = at<int32_t>(ws, L.counts);
  a.offsets = at<int32_t>(ws, L.offsets);
  a.sorted = at<int32_t>(ws, L.sorted);
  a.block_bucket = at<int32_t>(ws, L.block_bucket);
  a.num_post = at<int32_t>(ws, L.num_post);
  a.active = at<int32_t>(ws, L.active);
  a.status = at<int32_t>(ws, 0);
  a.block_hist = at<int32_t>(ws, L.scratch);
  a.capacity = R;
  a.max_tiles = R;
  a.max_active = n_out < R ? n_out : R;
  a.sentinel = (int32_t)R;
  a.nblocks = (int32_t)align_nblocks(R);
  if (launch_align(a, s) != hipSuccess) return MOE_EHIP;
  hipError_t e = launch_reduce_csr(static_cast<const uint16_t*>(y), row_weight, a.offsets, a.sorted,
                                   static_cast<uint16_t*>(out), n_out, P.K, s);
  return e == hipSuccess ? MOE_OK : MOE_EHIP;
}

int moe_quantize_mxfp8(const void* x, int x_dtype, int64_t rows, int64_t cols, uint8_t* codes,
                       uint8_t* scales, void* stream) {
  if (rows <= 0 || cols <= 0 || cols % 32 || (x_dtype != 0 && x_dtype != 1)) return MOE_EINVAL;
  if (!aligned16(x) || !aligned16(codes) || !scales) return MOE_EINVAL;
  hipError_t e = launch_quantize_mxfp8(x, x_dtype, rows, cols, codes, scales, (hipStream_t)stream);
  return e == hipSuccess ? MOE_OK : MOE_EHIP;
}

int moe_pack_mxfp8_scales(const uint8_t* src, uint8_t* dst, int64_t mats, int64_t rows, int64_t cols,
                          void* stream) {
  if (mats <= 0 || rows <= 0 || cols <= 0 || cols % 512) return MOE_EINVAL;
  if (!aligned16(src) || !aligned16(dst)) return MOE_EINVAL;
  const int64_t bytes = mats * rows * (cols / 32);
  if (bytes / mats / rows != cols / 32) return MOE_EINVAL;   // overflow
  // the buffers must not overlap
  if ((uintptr_t)src < (uintptr_t)dst + bytes && (uintptr_t)dst < (uintptr_t)src + bytes) return MOE_EINVAL;
  hipError_t e = launch_pack_mxfp8_scales(src, dst, mats, rows, cols, (hipStream_t)stream);
  return e == hipSuccess ? MOE_OK : MOE_EHIP;
}


// ------------------------------------------------------------- training ----

static int grouped_ok(const moe_grouped_problem* p, const int32_t* offsets) {
  if (!p || !aligned4(offsets)) return MOE_EINVAL;
  if (p->E < 1 || p->E > 65535 || p->R < 0 || p->R >= (1ll << 31) || p->N <= 0 || p->K <= 0)
    return MOE_EINVAL;
  if (p->N % 128 || p->K % 128) return MOE_EUNSUPPORTED;
  const int64_t wide = p->N > p->K ? p->N : p->K;
  if (p->R * wide * 2 >= (1ll << 31) || p->N * p->K * 2 >= (1ll << 31)) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

static TrainArgs train_args(const moe_grouped_problem* p, int mode, const int32_t* offsets, void* out) {
  TrainArgs t{};
  t.mode = mode;
  t.offsets = offsets;
  t.out = out;
  t.R = p->R;
  t.N = (int32_t)p->N;
  t.K = (int32_t)p->K;
  t.E = (int32_t)p->E;
  return t;
}

int moe_grouped_forward(const moe_grouped_problem* p, const void* x, const void* w,
                        const int32_t* group_offsets, void* y, void* stream) {
  const int st = grouped_ok(p, group_offsets);
  if (st != MOE_OK) return st;
  if (p->R > 0 && (!aligned16(x) || !aligned16(w) || !aligned16(y))) return MOE_EINVAL;
  TrainArgs t = train_args(p, kTrainForward, group_offsets, y);
  t.x = static_cast<const uint16_t*>(x);
  t.w = static_cast<const uint16_t*>(w);
  return launch_train(t, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_EHIP;
}

int moe_grouped_dgrad(const moe_grouped_problem* p, const void* dy, const void* w,
                      const int32_t* group_offsets, void* dx, void* stream) {
  const int st = grouped_ok(p, group_offsets);
  if (st != MOE_OK) return st;
  if (p->R > 0 && (!aligned16(dy) || !aligned16(w) || !aligned16(dx))) return MOE_EINVAL;
  TrainArgs t = train_args(p, kTrainDgrad, group_offsets, dx);
  t.dy = static_cast<const uint16_t*>(dy);
  t.w = static_cast<const uint16_t*>(w);
  return launch_train(t, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_EHIP;
}

int moe_grouped_wgrad(const moe_grouped_problem* p, const void* dy, const void* x,
                      const int32_t* group_offsets, float* dw, int accumulate, void* stream) {
  const int st = grouped_ok(p, group_offsets);
  if (st != MOE_OK) return st;
  if (!aligned16(dw) || (accumulate != 0 && accumulate != 1)) return MOE_EINVAL;
  if (p->R > 0 && (!aligned16(dy) || !aligned16(x))) return MOE_EINVAL;
  TrainArgs t = train_args(p, kTrainWgrad, group_offsets, dw);
  t.dy = static_cast<const uint16_t*>(dy);
  t.x = static_cast<const uint16_t*>(x);
  t.accumulate = accumulate;
  return launch_train(t, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_EHIP;
}


// --------------------------------------------------------------- router ----

static bool router_args(const moe_router* r, RouterArgs* a) {
  if (!r || r->E < 1 || r->E > kRouterMaxE || r->topk < 1 || r->topk > kRouterMaxTopk || r->topk > r->E) return false;
  if (r->groups < 1 || r->groups > kRouterMaxGroups || r->E % r->groups || r->topk_groups < 1 ||
      r->topk_groups > r->groups)
    return false;
  if (r->scoring != MOE_ROUTE_SOFTMAX && r->scoring != MOE_ROUTE_SIGMOID) return false;
  if (r->bias_kind < MOE_ROUTE_BIAS_NONE || r->bias_kind > MOE_ROUTE_BIAS_SELECT) return false;
  if ((r->renormalize != 0 && r->renormalize != 1) || !(r->scale - r->scale == 0.0f)) return false;
  *a = RouterArgs{(int32_t)r->E, (int32_t)r->topk, (int32_t)r->groups, (int32_t)r->topk_groups,
                  r->scoring, r->bias_kind, r->renormalize, r->scale};
  return true;
}

// Logits or their gradient: M rows, ld elements apart, dtype 0 float32 or 1 bf16.
static bool logits_ok(const void* p, int dtype, int64_t M, int64_t E, int64_t ld) {
  if ((dtype != 0 && dtype != 1) || M < 0 || M >= (1ll << 31) || ld < E || ld >= (1ll << 31)) return false;
  return M == 0 || (p && ((uintptr_t)p & (dtype == 0 ? 3u : 1u)) == 0);
}

static bool router_bias_ok(const RouterArgs& a, const float* bias) {
  return a.bias_kind == MOE_ROUTE_BIAS_NONE ? bias == nullptr : aligned4(bias);
}

int moe_route_topk(const moe_router* r, int64_t M, const void* logits, int dtype, int64_t logits_ld,
                   const float* bias, int32_t* topk_ids, float* topk_weights, void* stream) {
  RouterArgs a;
  if (!router_args(r, &a) || !logits_ok(logits, dtype, M, r->E, logits_ld) || !router_bias_ok(a, bias))
    return MOE_EINVAL;
  if (M > 0 && (!aligned4(topk_ids) || !aligned4(topk_weights))) return MOE_EINVAL;
  hipError_t e = launch_route_topk(a, M, logits, dtype == 1, logits_ld, bias, topk_ids, topk_weights,
                                   (hipStream_t)stream);
  return e == hipSuccess ? MOE_OK : MOE_EHIP;
}

int moe_route_topk_backward(const moe_router* r, int64_t M, const void* logits, int dtype, int64_t logits_ld,
                            const float* bias, const int32_t* topk_ids, const float* dweights, void* dlogits,
                            int64_t dlogits_ld, void* stream) {
  RouterArgs a;
  if (!router_args(r, &a) || !logits_ok(logits, dtype, M, r->E, logits_ld) || !router_bias_ok(a, bias) ||
      !logits_ok(dlogits, dtype, M, r->E, dlogits_ld))
    return MOE_EINVAL;
  if (M > 0 && (!aligned4(topk_ids) || !aligned4(dweights))) return MOE_EINVAL;
  hipError_t e = launch_route_topk_backward(a, M, logits, dtype == 1, logits_ld, bias, topk_ids, dweights, dlogits,
                                            dlogits_ld, (hipStream_t)stream);
  return e == hipSuccess ? MOE_OK : MOE_EHIP;
}

// ---------------------------------------------------------------- layer ----

void moe_layer_struct_sizes(int64_t* router, int64_t* problem, int64_t* plan) {
  if (router) *router = sizeof(moe_router);
  if (problem) *problem = sizeof(moe_layer_problem);
  if (plan) *plan = sizeof(moe_layer_plan);
}

static int layer_fail(moe_layer_plan* plan, int code, const char* msg) {
  snprintf(plan->reason, sizeof(plan->reason), "%s", msg);
  return code;
}

int moe_layer_plan_init(moe_layer_plan* plan, const moe_layer_problem* prob) {
  if (!plan || !prob) return MOE_EINVAL;
  memset(plan, 0, sizeof(*plan));
  plan->prob = *prob;
  const moe_layer_problem& P = *prob;
  RouterArgs r;
  if (!router_args(&P.router, &r)) return layer_fail(plan, MOE_EINVAL, "bad router");
  if (P.M <= 0 || P.K <= 0 || P.I <= 0 || P.shared_experts < 0)
    return layer_fail(plan, MOE_EINVAL, "M, K and I must be positive, shared_experts not negative");
  if (P.w_dtype != MOE_W_BF16 && P.w_dtype != MOE_W_MXFP8 && P.w_dtype != MOE_W_MXFP8_GROUPED)
    return layer_fail(plan, MOE_EINVAL, "unknown weight dtype");
  if (P.w1_order != MOE_W1_HALVES && P.w1_order != MOE_W1_INTERLEAVE16)
    return layer_fail(plan, MOE_EINVAL, "unknown W1 row order");
  if (P.w_dtype == MOE_W_MXFP8_GROUPED)
    return layer_fail(plan, MOE_EUNSUPPORTED, "the layer reads row-major MXFP8 scales");
  if (P.M > kLayerMaxM || r.E > kLayerMaxE || r.topk > kLayerMaxTopk || P.shared_experts > kLayerMaxShared)
    return layer_fail(plan, MOE_EUNSUPPORTED, "the layer takes M <= 64, E <= 512, topk <= 32, shared_experts <= 16");
  if (P.K % 128 || P.I % 128) return layer_fail(plan, MOE_EUNSUPPORTED, "the layer needs K % 128 == 0 and I % 128 == 0");
  const int64_t rows = P.M * (r.topk + P.shared_experts);
  // 32-bit buffer offsets: one expert's W1, x, the router's weights, z
  if (P.K >= (1ll << 29) || P.I >= (1ll << 29) || 4 * P.I * P.K >= (1ll << 31) || 2 * P.M * P.K >= (1ll << 31) ||
      2ll * r.E * P.K >= (1ll << 31) || 2 * rows * P.I >= (1ll << 31))
    return layer_fail(plan, MOE_EUNSUPPORTED, "the layer addresses one expert and the intermediate with 32-bit offsets");
  plan->abi_version = MOE_ABI_VERSION;
  plan->max_slots = (r.E < P.M * r.topk ? r.E : P.M * r.topk) + P.shared_experts;
  plan->splits = layer_splits(P.K, plan->max_slots * (P.I / 128));
  plan->rows = rows;
  int64_t o = 0;
  auto take = [&](int64_t bytes) {
    const int64_t at = o;
    o = up(o + bytes, kAlign);
    return at;
  };
  plan->off_sync = take(4 * (kLayerStrips + P.K / 32));
  plan->off_status = plan->off_sync + 4 * kLayerStatus;
  plan->off_logits = take(4 * layer_router_splits(P.K) * P.M * up(r.E, 16));
  plan->off_slots = take((int64_t)sizeof(LayerSlot) * plan->max_slots);
  plan->off_rows = take(4 * rows);
  plan->off_row_weights = take(4 * rows);
  plan->off_z = take(2 * rows * P.I);
  plan->off_partial = take(plan->splits > 1 ? 4 * plan->splits * P.M * P.K : 0);
  plan->ws_bytes = o;
  return MOE_OK;
}

int moe_layer_apply(const moe_layer_plan* plan, const void* x, const void* router_w, const float* router_bias,
                    const moe_weights* w, void* out, int32_t* topk_ids, float* topk_weights, void* ws,
                    void* stream) {
  if (!plan || plan->abi_version != MOE_ABI_VERSION || !w) return MOE_EINVAL;
  const moe_layer_problem& P = plan->prob;
  const bool mx = P.w_dtype == MOE_W_MXFP8;
  LayerArgs g{};
  if (!router_args(&P.router, &g.r) || !router_bias_ok(g.r, router_bias)) return MOE_EINVAL;
  if (!aligned16(x) || !aligned16(router_w) || !aligned16(w->w1) || !aligned16(w->w2) || !aligned16(out) ||
      !aligned4(topk_ids) || !aligned4(topk_weights) || !aligned16(ws) || w->expert_map)
    return MOE_EINVAL;
  if (mx && (!aligned4(w->w1_scale) || !aligned4(w->w2_scale))) return MOE_EINVAL;
  g.M = (int32_t)P.M;
  g.K = (int32_t)P.K;
  g.I = (int32_t)P.I;
  g.S = (int32_t)P.shared_experts;
  g.w1_order = P.w1_order;
  g.x = static_cast<const uint16_t*>(x);
  g.wr = static_cast<const uint16_t*>(router_w);
  g.rbias = router_bias;
  g.w1 = w->w1;
  g.w1s = w->w1_scale;
  g.w2 = w->w2;
  g.w2s = w->w2_scale;
  g.out = static_cast<uint16_t*>(out);
  g.ids = topk_ids;
  g.wts = topk_weights;
  g.sync = at<int32_t>(ws, plan->off_sync);
  g.status = at<int32_t>(ws, plan->off_status);
  g.logits = at<float>(ws, plan->off_logits);
  g.slots = at<LayerSlot>(ws, plan->off_slots);
  g.rows = at<int32_t>(ws, plan->off_rows);
  g.roww = at<float>(ws, plan->off_row_weights);
  g.z = at<uint16_t>(ws, plan->off_z);
  g.part = at<float>(ws, plan->off_partial);
  g.logit_ld = (int32_t)up(g.r.E, 16);
  g.max_slots = (int32_t)plan->max_slots;
  g.cap = (int32_t)plan->rows;
  return launch_layer(g, mx, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_EHIP;
}

// ----------------------------------------------------------------- lora ----

static int lora_ok(const moe_lora_problem* p) {
  if (!p || p->R < 0 || p->R >= (1ll << 31) || p->N <= 0 || p->K <= 0 || p->G <= 0 || p->rank <= 0) return MOE_EINVAL;
  if (p->N % 64 || p->K % 64 || p->rank % 8 || p->rank > kLoraMaxRank || p->G > 4096) return MOE_EUNSUPPORTED;
  const int64_t wide = p->N > p->K ? p->N : p->K, lim = 1ll << 30;   // elements of 2 bytes
  if (wide >= lim || p->N >= lim / p->K + (lim % p->K != 0) || wide * p->R >= lim || p->G * p->rank >= lim / wide + 1 ||
      p->G * p->rank * wide >= lim || kLoraPieces * p->R * p->rank >= lim)
    return MOE_EUNSUPPORTED;
  return MOE_OK;
}

static LoraArgs lora_args(const moe_lora_problem* p, const float* scale, const int32_t* adapter, void* low) {
  LoraArgs a{};
  a.scale = scale;
  a.adapter = adapter;
  a.low = static_cast<uint16_t*>(low);
  a.R = p->R;
  a.G = (int32_t)p->G;
  a.rank = (int32_t)p->rank;
  return a;
}

int64_t moe_lora_low_bytes(const moe_lora_problem* p) {
  return lora_ok(p) == MOE_OK ? 2 * kLoraPieces * p->R * p->rank : -1;
}

// Chunks of the rows' sort (the gradients' whole call, 4 adapters of rank 16, N =
// K = 256, one workgroup / several, us: 1024 rows 14.5 / 17.4, 2048 18.6 / 19.3,
// 3000 22.0 / 20.5, 8192 38.2 / 23.7).
static int64_t lora_align_blocks(int64_t R) { return R <= 2 * kAlignChunk ? 0 : align_nblocks_of(R); }

static AlignLayout lora_layout(const moe_lora_problem* p) {
  return layout_align(0, p->G, p->R, p->R, p->G < p->R ? p->G : p->R, lora_align_blocks(p->R));
}

int64_t moe_lora_ws_bytes(const moe_lora_problem* p) {
  if (lora_ok(p) != MOE_OK) return -1;
  const int64_t shares = lora_wgrad_shares(p->R, p->N, p->K, p->G);
  return lora_layout(p).end + (shares > 1 ? 4 * shares * p->G * p->rank * (p->N + p->K) : 0);
}

static int lora_project(const moe_lora_problem* p, bool dgrad, const void* in, const void* w, const void* a,
                        const void* b, const float* scale, const int32_t* adapter, void* out, void* low,
                        void* stream) {
  const int st = lora_ok(p);
  if (st != MOE_OK) return st;
  if (!aligned16(w) || !aligned16(a) || !aligned16(b) || !aligned4(scale)) return MOE_EINVAL;
  if (p->R > 0 && (!aligned16(in) || !aligned4(adapter) || !aligned16(out) || !aligned16(low))) return MOE_EINVAL;
  const LoraArgs l = lora_args(p, scale, adapter, low);
  auto u16 = [](const void* q) { return static_cast<const uint16_t*>(q); };
  const hipError_t e =
      dgrad ? launch_lora_dgrad(l, u16(in), u16(w), u16(a), u16(b), static_cast<uint16_t*>(out), (int)p->N, (int)p->K,
                                (hipStream_t)stream)
            : launch_lora_forward(l, u16(in), u16(w), u16(a), u16(b), static_cast<uint16_t*>(out), (int)p->N,
                                  (int)p->K, (hipStream_t)stream);
  return e == hipSuccess ? MOE_OK : MOE_EHIP;
}

int moe_lora_forward(const moe_lora_problem* p, const void* x, const void* w, const void* a, const void* b,
                     const float* scale, const int32_t* adapter, void* y, void* low, void* stream) {
  return lora_project(p, false, x, w, a, b, scale, adapter, y, low, stream);
}

int moe_lora_dgrad(const moe_lora_problem* p, const void* dy, const void* w, const void* a, const void* b,
                   const float* scale, const int32_t* adapter, void* dx, void* low, void* stream) {
  return lora_project(p, true, dy, w, a, b, scale, adapter, dx, low, stream);
}

int moe_lora_wgrad(const moe_lora_problem* p, const void* x, const void* dy, const void* low_x, const void* low_dy,
                   const int32_t* adapter, float* da, float* db, int accumulate, void* ws, void* stream) {
  const int st = lora_ok(p);
  if (st != MOE_OK) return st;
  if (!aligned16(da) || !aligned16(db) || !aligned16(ws) || (accumulate != 0 && accumulate != 1)) return MOE_EINVAL;
  if (p->R > 0 &&
      (!aligned16(x) || !aligned16(dy) || !aligned16(low_x) || !aligned16(low_dy) || !aligned4(adapter)))
    return MOE_EINVAL;
  // the rows of each adapter, in row order
  const AlignLayout L = lora_layout(p);
  AlignArgs al{};
  al.keys = adapter;
  al.R = p->R;
  al.nb = (int32_t)p->G;
  al.B = 1;
  al.counts = at<int32_t>(ws, L.counts);
  al.offsets = at<int32_t>(ws, L.offsets);
  al.sorted = at<int32_t>(ws, L.sorted);
  al.block_bucket = at<int32_t>(ws, L.block_bucket);
  al.num_post = at<int32_t>(ws, L.num_post);
  al.active = at<int32_t>(ws, L.active);
  al.status = at<int32_t>(ws, L.status);
  al.block_hist = at<int32_t>(ws, L.scratch);
  al.capacity = p->R;
  al.max_tiles = p->R;
  al.max_active = p->G < p->R ? p->G : p->R;
  al.sentinel = (int32_t)p->R;
  al.nblocks = (int32_t)lora_align_blocks(p->R);
  if (launch_align(al, (hipStream_t)stream) != hipSuccess) return MOE_EHIP;
  LoraGradArgs g{};
  g.x = static_cast<const uint16_t*>(x);
  g.dy = static_cast<const uint16_t*>(dy);
  g.low_x = static_cast<const uint16_t*>(low_x);
  g.low_dy = static_cast<const uint16_t*>(low_dy);
  g.counts = al.counts;
  g.offsets = al.offsets;
  g.sorted = al.sorted;
  g.da = da;
  g.db = db;
  g.part = at<float>(ws, L.end);
  g.R = p->R;
  g.N = (int32_t)p->N;
  g.K = (int32_t)p->K;
  g.G = (int32_t)p->G;
  g.rank = (int32_t)p->rank;
  g.accumulate = accumulate;
  return launch_lora_wgrad(g, lora_wgrad_shares(p->R, p->N, p->K, p->G), (hipStream_t)stream) == hipSuccess ? MOE_OK
                                                                                                            : MOE_EHIP;
}

// -------------------------------------------------------------- balance ----

constexpr int64_t kBalanceMaxS = 65536;

struct BalanceLayout {
  int64_t part, tsum, lpart, done, end;
};

static bool balance_layout(const moe_router* r, int64_t M, int64_t S, BalanceLayout* L) {
  RouterArgs a;
  if (!router_args(r, &a) || M < 0 || M * r->topk >= (1ll << 31) || S < 1 || S > kBalanceMaxS) return false;
  const int64_t chunk = balance_chunk(M, r->E), slots = (M + chunk - 1) / chunk + S;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += up(bytes, 256);
    return o;
  };
  L->lpart = take(8 * S * ((r->E + kBalanceExperts - 1) / kBalanceExperts));
  L->part = take(8 * slots * r->E);
  L->tsum = take(4 * slots);
  L->done = take(4 * S);
  L->end = at;
  return true;
}

int64_t moe_balance_ws_bytes(const moe_router* r, int64_t M, int64_t S) {
  BalanceLayout L;
  return M < (1ll << 31) && balance_layout(r, M, S, &L) ? L.end : -1;
}

static bool balance_args(const moe_router* r, int64_t M, int64_t S, const void* logits, int dtype, int64_t ld,
                         const float* bias, const int32_t* ids, const int32_t* offsets, BalanceArgs* b) {
  RouterArgs a;
  if (!router_args(r, &a) || !logits_ok(logits, dtype, M, r->E, ld) || !router_bias_ok(a, bias)) return false;
  if (M * r->topk >= (1ll << 31) || S < 1 || S > kBalanceMaxS || (S > 1 && !offsets) || ((uintptr_t)offsets & 3))
    return false;
  if (M > 0 && !aligned4(ids)) return false;
  b->M = M;
  b->S = (int32_t)S;
  b->E = a.E;
  b->topk = a.topk;
  b->sigmoid = a.scoring;
  b->add_bias = a.bias_kind == MOE_ROUTE_BIAS_LOGIT;
  b->logits = logits;
  b->bf16 = dtype;
  b->ld = ld;
  b->bias = bias;
  b->ids = ids;
  b->offsets = offsets;
  return true;
}

int moe_balance_loss(const moe_router* r, int64_t M, int64_t S, const void* logits, int dtype, int64_t logits_ld,
                     const float* bias, const int32_t* topk_ids, const int32_t* seq_offsets, float* loss,
                     int32_t* counts, int32_t* tokens, float* probs, void* ws, void* stream) {
  BalanceArgs b{};
  BalanceLayout L;
  if (!balance_args(r, M, S, logits, dtype, logits_ld, bias, topk_ids, seq_offsets, &b) ||
      !balance_layout(r, M, S, &L) || !aligned4(loss) || !aligned4(counts) || !aligned4(tokens) || !aligned4(probs) ||
      !aligned16(ws))
    return MOE_EINVAL;
  b.loss = loss;
  b.counts = counts;
  b.tokens = tokens;
  b.probs = probs;
  b.chunk = balance_chunk(M, r->E);
  b.one = balance_one(M, r->E, S);
  b.nchunk = (int32_t)((M + b.chunk - 1) / b.chunk);
  b.part = at<int2>(ws, L.part);
  b.tsum = at<int32_t>(ws, L.tsum);
  b.lpart = at<double>(ws, L.lpart);
  b.done = at<int32_t>(ws, L.done);
  return launch_balance(b, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_EHIP;
}

int moe_balance_loss_backward(const moe_router* r, int64_t M, int64_t S, const void* logits, int dtype,
                              int64_t logits_ld, const float* bias, const int32_t* topk_ids,
                              const int32_t* seq_offsets, const int32_t* counts, const int32_t* tokens,
                              const float* dloss, void* dlogits, int64_t dlogits_ld, int accumulate, void* stream) {
  BalanceArgs b{};
  if (!balance_args(r, M, S, logits, dtype, logits_ld, bias, topk_ids, seq_offsets, &b) ||
      !logits_ok(dlogits, dtype, M, r->E, dlogits_ld) || !aligned4(counts) || !aligned4(tokens) || !aligned4(dloss) ||
      (accumulate != 0 && accumulate != 1))
    return MOE_EINVAL;
  b.counts_in = counts;
  b.tokens_in = tokens;
  b.dloss = dloss;
  b.dlogits = dlogits;
  b.dld = dlogits_ld;
  b.accumulate = accumulate;
  return launch_balance_backward(b, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_EHIP;
}

// ----------------------------------------------------------------- norm ----

void moe_block_struct_sizes(int64_t* norm, int64_t* ortho) {
  if (norm) *norm = sizeof(moe_norm_problem);
  if (ortho) *ortho = sizeof(moe_ortho_problem);
}

static bool finite_f32(float v) { return v - v == 0.0f; }

static int norm_ok(const moe_norm_problem* p) {
  if (!p || p->M < 0 || p->M >= (1ll << 31) || p->K <= 0) return MOE_EINVAL;
  if ((p->x_dtype != 0 && p->x_dtype != 1) || (p->w_dtype != 0 && p->w_dtype != 1)) return MOE_EINVAL;
  if (p->gate_kind < MOE_GATE_NONE || p->gate_kind > MOE_GATE_TOKEN) return MOE_EINVAL;
  // (the kernels' reciprocal square root takes a subnormal value as 0)
  if (!(p->eps >= 0x1p-126f) || !finite_f32(p->eps) || !finite_f32(p->res_scale)) return MOE_EINVAL;
  if (p->K % 8 || p->K > kNormMaxK) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

// Null, or 16-byte aligned.
static bool optional16(const void* q) { return ((uintptr_t)q & 15) == 0; }

// What forward and backward ask of the weights and the gate alike.
static bool norm_weights(const moe_norm_problem* p, const void* w_post, const void* gate, const void* w_pre) {
  if (!optional16(w_post) || !optional16(w_pre)) return false;
  const bool empty = p->gate_kind == MOE_GATE_TOKEN && p->M == 0;   // a gate of no elements may be null
  if (!empty && (p->gate_kind == MOE_GATE_NONE) != (gate == nullptr)) return false;
  return ((uintptr_t)gate & (p->gate_kind == MOE_GATE_TOKEN ? 3 : 15)) == 0;
}

// Without a block there is nothing to norm behind it or to gate.
static bool norm_block(const void* block, const void* w_post, const void* gate, const void* w_pre) {
  return block ? optional16(block) : w_pre && !w_post && !gate;
}

static NormArgs norm_args(const moe_norm_problem* p, const void* x, const void* block, const void* w_post,
                          const void* gate, const void* w_pre) {
  NormArgs a{};
  a.M = p->M;
  a.K = (int32_t)p->K;
  a.xf32 = p->x_dtype == 0;
  a.wbf16 = p->w_dtype;
  a.gate_kind = p->gate_kind;
  a.eps = p->eps;
  a.res_scale = p->res_scale;
  a.x = x;
  a.block = static_cast<const uint16_t*>(block);
  a.w_post = w_post;
  a.gate = gate;
  a.w_pre = w_pre;
  return a;
}

int moe_block_norm(const moe_norm_problem* p, const void* x, const void* block, const void* w_post,
                   const void* gate, const void* w_pre, void* x_out, void* h, void* stream) {
  const int st = norm_ok(p);
  if (st != MOE_OK) return st;
  if (p->M == 0) return MOE_OK;
  if (!norm_weights(p, w_post, gate, w_pre) || !norm_block(block, w_post, gate, w_pre) || !aligned16(x) || !optional16(x_out) ||
      !optional16(h) || (block != nullptr) != (x_out != nullptr) || (w_pre != nullptr) != (h != nullptr))
    return MOE_EINVAL;
  NormArgs a = norm_args(p, x, block, w_post, gate, w_pre);
  a.x_out = x_out;
  a.h = static_cast<uint16_t*>(h);
  return launch_block_norm(a, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_EHIP;
}

int64_t moe_block_norm_ws_bytes(const moe_norm_problem* p) {
  return norm_ok(p) == MOE_OK ? 8 * (int64_t)norm_backward_blocks(p->M, p->K) * p->K : -1;
}

int moe_block_norm_backward(const moe_norm_problem* p, const void* x_out, const void* block, const void* w_post,
                            const void* gate, const void* w_pre, const void* dx_out, const void* dh, void* dx,
                            void* dblock, float* dw_post, float* dgate, float* dw_pre, int accumulate, void* ws,
                            void* stream) {
  const int st = norm_ok(p);
  if (st != MOE_OK) return st;
  const bool rows = p->M > 0;
  if (!norm_weights(p, w_post, gate, w_pre) || (accumulate != 0 && accumulate != 1) || !optional16(dw_post) || !optional16(dw_pre) || !aligned16(ws) ||
      (dw_post && !w_post) || (dw_pre && !w_pre) || (dgate && p->gate_kind == MOE_GATE_NONE) ||
      ((uintptr_t)dgate & 3))
    return MOE_EINVAL;
  if (rows && (!norm_block(block, w_post, gate, w_pre) || !aligned16(x_out) || !aligned16(dx) ||
               !optional16(dblock) || !optional16(dx_out) || !optional16(dh) ||
               (block != nullptr) != (dblock != nullptr) || (w_pre != nullptr) != (dh != nullptr) ||
               (!dx_out && !w_pre)))
    return MOE_EINVAL;
  NormArgs a = norm_args(p, x_out, block, w_post, gate, w_pre);
  a.dx_out = dx_out;
  a.dh = static_cast<const uint16_t*>(dh);
  a.dx = dx;
  a.dblock = static_cast<uint16_t*>(dblock);
  a.dw_post = dw_post;
  a.dgate = dgate;
  a.dw_pre = dw_pre;
  a.accumulate = accumulate;
  a.part = static_cast<float*>(ws);
  return launch_block_norm_backward(a, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_EHIP;
}

// ---------------------------------------------------------------- ortho ----

static int ortho_ok(const moe_ortho_problem* p, OrthoArgs* a) {
  if (!p || p->E < 1 || p->N < 1 || p->K < 1 || (p->dtype != 0 && p->dtype != 1)) return MOE_EINVAL;
  if (p->steps < 1 || p->steps > MOE_ORTHO_MAX_STEPS || !(p->eps > 0.0f) || !finite_f32(p->eps) ||
      !finite_f32(p->scale))
    return MOE_EINVAL;
  if (p->N > 32768 || p->K > 32768 || p->E > 65535 || up(p->N, 256) * up(p->K, 256) >= (1ll << 30) ||
      p->E * up(p->N, 256) * up(p->K, 256) >= (1ll << 36))
    return MOE_EUNSUPPORTED;
  static_assert(kOrthoMaxSteps == MOE_ORTHO_MAX_STEPS, "steps");
  a->E = (int32_t)p->E;
  a->N = (int32_t)p->N;
  a->K = (int32_t)p->K;
  a->bf16 = p->dtype;
  a->steps = p->steps;
  a->eps = p->eps;
  a->scale = p->scale;
  for (int i = 0; i < p->steps; ++i)
    for (int j = 0; j < 3; ++j) a->coef[i][j] = p->coef[i][j];
  int32_t s[kOrthoMaxSteps][3];
  return ortho_scales(*a, s) ? MOE_OK : MOE_EUNSUPPORTED;
}

int64_t moe_ortho_ws_bytes(const moe_ortho_problem* p) {
  OrthoArgs a{};
  return ortho_ok(p, &a) == MOE_OK ? ortho_ws_bytes(a.E, a.N, a.K) : -1;
}

int moe_orthogonalize(const moe_ortho_problem* p, const void* update, void* out, void* ws, void* stream) {
  OrthoArgs a{};
  const int st = ortho_ok(p, &a);
  if (st != MOE_OK) return st;
  if (!update || ((uintptr_t)update & (p->dtype == 0 ? 3 : 1)) || !out || ((uintptr_t)out & 1) || !aligned16(ws))
    return MOE_EINVAL;
  a.update = update;
  a.out = static_cast<uint16_t*>(out);
  a.ws = ws;
  return launch_orthogonalize(a, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_EHIP;
}

}  // extern "C"

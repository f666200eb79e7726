"""Python binding of libmoe_mi355x.so, the fused-MoE expert computation for
one MI355X (gfx950).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI of ``include/moe_mi355x.h``.  torch supplies device
memory and the stream.  The functions carry the C names.  Loading fails
loudly when the library has not been built; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

__all__ = [
    "ABI_VERSION", "LAYOUT_CONTIGUOUS", "LAYOUT_BATCHED", "W_BF16", "W_MXFP8", "W_MXFP8_GROUPED", "W1_HALVES",
    "W1_INTERLEAVE16", "VARIANT_AUTO", "VARIANT_TILE", "VARIANT_STREAM", "VARIANT_FUSED", "REDUCE_NOOP",
    "REDUCE_CONTIGUOUS", "REDUCE_NAIVE_BATCHED", "MoeError", "MoeProblem", "MoePlan", "MoeWeights",
    "load_library", "library_path", "moe_abi_version", "moe_status_string", "moe_plan_init",
    "moe_apply_contiguous_static", "STATIC_SCRATCH_BYTES",
    "moe_plan_reason", "moe_align_permute", "moe_apply_contiguous", "moe_apply_batched",
    "moe_gate_up_act", "moe_down_unpermute",
    "moe_topk_reduce_contiguous", "moe_naive_batched_ws_bytes", "moe_topk_reduce_naive_batched",
    "moe_quantize_mxfp8", "moe_pack_mxfp8_scales", "make_problem", "allocate_workspaces", "ws_view", "status_words",
    "check_status",
    "MoeGroupedProblem", "moe_grouped_forward", "moe_grouped_dgrad", "moe_grouped_wgrad",
    "ROUTE_SOFTMAX", "ROUTE_SIGMOID", "BIAS_NONE", "BIAS_LOGIT", "BIAS_SELECT", "MoeRouter", "make_router",
    "moe_route_topk", "moe_route_topk_backward",
    "MoeLayerProblem", "MoeLayerPlan", "make_layer_problem", "moe_layer_plan_init", "allocate_layer_workspace",
    "moe_layer_apply", "check_layer_status",
    "MoeLoraProblem", "moe_lora_low_bytes", "moe_lora_ws_bytes", "allocate_lora_low", "allocate_lora_workspace",
    "moe_lora_forward", "moe_lora_dgrad", "moe_lora_wgrad",
]

ABI_VERSION = 6
STATIC_SCRATCH_BYTES = 64 << 20     # MOE_STATIC_SCRATCH_BYTES
MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_EHIP = 0, 1, 2, 3
LAYOUT_CONTIGUOUS, LAYOUT_BATCHED = 0, 1
W_BF16, W_MXFP8, W_MXFP8_GROUPED = 0, 1, 2
W1_HALVES, W1_INTERLEAVE16 = 0, 1
VARIANT_AUTO, VARIANT_TILE, VARIANT_STREAM, VARIANT_FUSED = -1, 0, 1, 2
REDUCE_NOOP, REDUCE_CONTIGUOUS, REDUCE_NAIVE_BATCHED = 0, 1, 2
ROUTE_SOFTMAX, ROUTE_SIGMOID = 0, 1                  # MOE_ROUTE_SOFTMAX, MOE_ROUTE_SIGMOID
BIAS_NONE, BIAS_LOGIT, BIAS_SELECT = 0, 1, 2         # MOE_ROUTE_BIAS_*

_i64, _i32, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p


class MoeProblem(ctypes.Structure):
    _fields_ = [("M", _i64), ("K", _i64), ("I", _i64), ("E", _i64), ("topk", _i64),
                ("max_tokens", _i64), ("global_experts", _i64), ("layout", _i32), ("w_dtype", _i32),
                ("w1_order", _i32), ("variant", _i32)]


class MoeGroupedProblem(ctypes.Structure):
    _fields_ = [("R", _i64), ("N", _i64), ("K", _i64), ("E", _i64)]


class MoeRouter(ctypes.Structure):
    _fields_ = [("E", _i64), ("topk", _i64), ("groups", _i64), ("topk_groups", _i64), ("scoring", _i32),
                ("bias_kind", _i32), ("renormalize", _i32), ("scale", ctypes.c_float)]


class MoeLayerProblem(ctypes.Structure):
    _fields_ = [("M", _i64), ("K", _i64), ("I", _i64), ("shared_experts", _i64), ("router", MoeRouter),
                ("w_dtype", _i32), ("w1_order", _i32)]


class MoeLayerPlan(ctypes.Structure):
    _fields_ = [("prob", MoeLayerProblem), ("abi_version", _i32), ("splits", _i32), ("max_slots", _i64),
                ("rows", _i64), ("ws_bytes", _i64), ("off_sync", _i64), ("off_status", _i64), ("off_logits", _i64),
                ("off_slots", _i64), ("off_rows", _i64), ("off_row_weights", _i64), ("off_z", _i64),
                ("off_partial", _i64), ("reason", ctypes.c_char * 192)]


class MoeLoraProblem(ctypes.Structure):
    _fields_ = [("R", _i64), ("N", _i64), ("K", _i64), ("G", _i64), ("rank", _i64)]


class MoePlan(ctypes.Structure):
    _fields_ = [("prob", MoeProblem), ("abi_version", _i32), ("variant", _i32), ("block_m", _i32),
                ("reduce_kind", _i32), ("routes", _i64), ("sorted_capacity", _i64),
                ("max_tiles", _i64), ("max_active", _i64), ("align_blocks", _i64),
                ("ws13_bytes", _i64), ("ws2_bytes", _i64), ("out_rows", _i64), ("out_cols", _i64),
                ("off_counts", _i64), ("off_offsets", _i64), ("off_sorted_ids", _i64),
                ("off_block_expert", _i64), ("off_num_post_padded", _i64), ("off_active", _i64),
                ("off_status", _i64), ("off_align_scratch", _i64), ("off_z", _i64),
                ("off_z_scale", _i64), ("off_xq", _i64), ("off_xq_scale", _i64), ("off_sync", _i64),
                ("reason", ctypes.c_char * 192)]


class MoeWeights(ctypes.Structure):
    _fields_ = [("w1", _vp), ("w1_scale", _vp), ("w2", _vp), ("w2_scale", _vp), ("expert_map", _vp)]


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int, reason: str = ""):
        self.status = status
        msg = f"{fn}: {_status_name(status)}"
        if reason:
            msg += f" ({reason})"
        super().__init__(msg)


_LIB: Optional[ctypes.CDLL] = None


def library_path() -> str:
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_mi355x.so")


def load_library() -> ctypes.CDLL:
    """Load the in-tree library (once).  Raises if it is missing or stale."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run mixture_experts_expert_align_amd/build.py "
                           "(or __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    sig = {
        "moe_abi_version": (_i32, []),
        "moe_status_string": (ctypes.c_char_p, [_i32]),
        "moe_struct_sizes": (None, [_vp, _vp, _vp]),
        "moe_plan_init": (_i32, [_vp, _vp]),
        "moe_plan_reason": (ctypes.c_char_p, [_vp]),
        "moe_align_permute": (_i32, [_vp] * 5),
        "moe_apply_contiguous": (_i32, [_vp] * 9),
        "moe_apply_contiguous_static": (_i32, [_vp] * 7),
        "moe_apply_batched": (_i32, [_vp] * 7),
        "moe_gate_up_act": (_i32, [_vp] * 5),
        "moe_down_unpermute": (_i32, [_vp] * 5),
        "moe_topk_reduce_contiguous": (_i32, [_vp] * 7),
        "moe_naive_batched_ws_bytes": (_i64, [_vp, _i64]),
        "moe_topk_reduce_naive_batched": (_i32, [_vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp]),
        "moe_quantize_mxfp8": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp, _vp]),
        "moe_pack_mxfp8_scales": (_i32, [_vp, _vp, _i64, _i64, _i64, _vp]),
        "moe_grouped_forward": (_i32, [_vp] * 6),
        "moe_grouped_dgrad": (_i32, [_vp] * 6),
        "moe_grouped_wgrad": (_i32, [_vp] * 5 + [_i32, _vp]),
        "moe_layer_struct_sizes": (None, [_vp, _vp, _vp]),
        "moe_layer_plan_init": (_i32, [_vp, _vp]),
        "moe_layer_apply": (_i32, [_vp] * 10),
        "moe_lora_low_bytes": (_i64, [_vp]),
        "moe_lora_ws_bytes": (_i64, [_vp]),
        "moe_lora_forward": (_i32, [_vp] * 10),
        "moe_lora_dgrad": (_i32, [_vp] * 10),
        "moe_lora_wgrad": (_i32, [_vp] * 8 + [_i32, _vp, _vp]),
        "moe_route_topk": (_i32, [_vp, _i64, _vp, _i32, _i64, _vp, _vp, _vp, _vp]),
        "moe_route_topk_backward": (_i32, [_vp, _i64, _vp, _i32, _i64, _vp, _vp, _vp, _vp, _i64, _vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    v = lib.moe_abi_version()
    if v != ABI_VERSION:
        raise RuntimeError(f"{path}: ABI version {v}, binding expects {ABI_VERSION}; rebuild it")
    sizes = [ctypes.c_int64() for _ in range(3)]
    lib.moe_struct_sizes(*[ctypes.byref(s) for s in sizes])
    want = [ctypes.sizeof(MoeProblem), ctypes.sizeof(MoePlan), ctypes.sizeof(MoeWeights)]
    if [s.value for s in sizes] != want:
        raise RuntimeError(f"struct layout mismatch: library {[s.value for s in sizes]}, binding {want}")
    lib.moe_layer_struct_sizes(*[ctypes.byref(s) for s in sizes])
    want = [ctypes.sizeof(MoeRouter), ctypes.sizeof(MoeLayerProblem), ctypes.sizeof(MoeLayerPlan)]
    if [s.value for s in sizes] != want:
        raise RuntimeError(f"struct layout mismatch: library {[s.value for s in sizes]}, binding {want}")
    _LIB = lib
    return lib


def _status_name(status: int) -> str:
    return {0: "ok", 1: "invalid argument", 2: "unsupported problem", 3: "HIP launch error"}.get(
        status, f"status {status}")


def _check(fn: str, status: int, plan: Optional[MoePlan] = None):
    if status != MOE_OK:
        raise MoeError(fn, status, plan.reason.decode() if plan is not None else "")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _arg(t: Optional[torch.Tensor], name: str, dtypes, numel: int) -> Optional[int]:
    """Device pointer of ``t`` after checking its dtype and that it holds at
    least ``numel`` elements (the kernels read or write that many)."""
    if t is None:
        return None
    if not isinstance(dtypes, tuple):
        dtypes = (dtypes,)
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, the call needs {numel}")
    return _ptr(t)


def _ws(t: torch.Tensor, name: str, nbytes: int) -> int:
    """A workspace: any dtype, at least ``nbytes`` bytes."""
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name}: {t.numel() * t.element_size()} bytes, the plan needs {nbytes}")
    return _ptr(t)


def _stream(stream) -> int:
    if stream is None:
        # the handle of torch.cuda.current_stream() (2.9 us), without the object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ------------------------------------------------------------------ calls --

def moe_abi_version() -> int:
    return load_library().moe_abi_version()


def moe_status_string(status: int) -> str:
    return load_library().moe_status_string(status).decode()


def make_problem(M, K, I, E, topk=0, max_tokens=0, layout=LAYOUT_CONTIGUOUS, w_dtype=W_BF16,
                 w1_order=W1_HALVES, variant=VARIANT_AUTO, global_experts=0) -> MoeProblem:
    return MoeProblem(M, K, I, E, topk, max_tokens, global_experts, layout, w_dtype, w1_order, variant)


def moe_plan_init(prob: MoeProblem) -> MoePlan:
    plan = MoePlan()
    st = load_library().moe_plan_init(ctypes.byref(plan), ctypes.byref(prob))
    _check("moe_plan_init", st, plan)
    return plan


def moe_plan_reason(plan: MoePlan) -> str:
    return load_library().moe_plan_reason(ctypes.byref(plan)).decode()


def allocate_workspaces(plan: MoePlan, device="cuda"):
    """ws13 and ws2 as uint8 device tensors of the sizes the plan states
    (ws13 zero-filled: the single-launch variant keeps its counters there)."""
    ws13 = torch.zeros(max(plan.ws13_bytes, 16), dtype=torch.uint8, device=device)
    ws2 = torch.empty(max(plan.ws2_bytes, 16), dtype=torch.uint8, device=device)
    return ws13, ws2


def ws_view(ws: torch.Tensor, offset: int, count: int, dtype=torch.int32) -> torch.Tensor:
    """A typed view of ``count`` elements at byte ``offset`` of a workspace."""
    nbytes = count * torch.empty((), dtype=dtype).element_size()
    return ws[offset: offset + nbytes].view(dtype)


def _ids_arg(plan: MoePlan, topk_ids: torch.Tensor, name="topk_ids") -> int:
    p = plan.prob
    if topk_ids.dtype != torch.int32:
        raise ValueError(f"{name}: dtype {topk_ids.dtype}, expected torch.int32 (e.g. topk ids .int())")
    if topk_ids.numel() != p.M * p.topk:
        raise ValueError(f"{name}: {topk_ids.numel()} elements, expected M*topk = {p.M * p.topk}")
    return _ptr(topk_ids)


def _map_arg(plan: MoePlan, expert_map: Optional[torch.Tensor]) -> Optional[int]:
    return _arg(expert_map, "expert_map", torch.int32, plan.prob.global_experts)


def status_words(plan: MoePlan, ws13: torch.Tensor):
    """(ids outside {-1} U [0,E) seen by the last align, waits of the
    single-launch variant that timed out, summed over calls) from the status
    words in ws13.  Synchronises with the device (a copy to the host)."""
    w = ws_view(ws13, plan.off_status, 2).cpu()
    return int(w[0]), int(w[1])


def check_status(plan: MoePlan, ws13: torch.Tensor):
    """Raise MoeError when a single-launch call on this ws13 gave up a bounded
    wait (its outputs are then undefined).  The count stays until ws13 is
    cleared, so every later check fails too."""
    _, timeouts = status_words(plan, ws13)
    if timeouts:
        raise MoeError("moe_apply_contiguous", MOE_EHIP,
                       f"{timeouts} bounded waits of the single-launch kernel timed out; outputs undefined")


def moe_align_permute(plan: MoePlan, topk_ids: torch.Tensor, ws13: torch.Tensor, stream=None,
                      expert_map: Optional[torch.Tensor] = None):
    st = load_library().moe_align_permute(ctypes.byref(plan), _ids_arg(plan, topk_ids),
                                          _map_arg(plan, expert_map), _ws(ws13, "ws13", plan.ws13_bytes),
                                          _stream(stream))
    _check("moe_align_permute", st)


def _weights(plan: MoePlan, w1, w2, w1_scale=None, w2_scale=None, expert_map=None) -> MoeWeights:
    p = plan.prob
    mx = p.w_dtype in (W_MXFP8, W_MXFP8_GROUPED)
    wt = torch.uint8 if mx else torch.bfloat16
    n1, n2 = p.E * 2 * p.I * p.K, p.E * p.K * p.I
    if mx and (w1_scale is None or w2_scale is None):
        raise ValueError("MXFP8 weights need w1_scale and w2_scale")
    return MoeWeights(_arg(w1, "w1", wt, n1), _arg(w1_scale, "w1_scale", torch.uint8, n1 // 32 if mx else 0),
                      _arg(w2, "w2", wt, n2), _arg(w2_scale, "w2_scale", torch.uint8, n2 // 32 if mx else 0),
                      _map_arg(plan, expert_map))


def moe_apply_contiguous(plan: MoePlan, a, topk_ids, topk_weights, w1, w2, out, ws13, ws2,
                         w1_scale=None, w2_scale=None, stream=None, expert_map=None):
    w = _weights(plan, w1, w2, w1_scale, w2_scale, expert_map)
    p = plan.prob
    st = load_library().moe_apply_contiguous(
        ctypes.byref(plan), _arg(a, "a", torch.bfloat16, p.M * p.K), _ids_arg(plan, topk_ids),
        _arg(topk_weights, "topk_weights", torch.float32, p.M * p.topk), ctypes.byref(w),
        _arg(out, "out", torch.bfloat16, p.M * p.K), _ws(ws13, "ws13", plan.ws13_bytes),
        _ws(ws2, "ws2", plan.ws2_bytes), _stream(stream))
    _check("moe_apply_contiguous", st)


def moe_apply_contiguous_static(plan: MoePlan, a, topk_ids, topk_weights, w1, w2, out, w1_scale=None,
                                w2_scale=None, stream=None, expert_map=None):
    """moe_apply_contiguous with the workspaces inside the library's own
    per-GPU array (no allocation by anyone; calls that overlap on one GPU
    race).  Raises MoeError(MOE_EUNSUPPORTED) when the plan's workspaces do
    not fit in STATIC_SCRATCH_BYTES."""
    w = _weights(plan, w1, w2, w1_scale, w2_scale, expert_map)
    p = plan.prob
    st = load_library().moe_apply_contiguous_static(
        ctypes.byref(plan), _arg(a, "a", torch.bfloat16, p.M * p.K), _ids_arg(plan, topk_ids),
        _arg(topk_weights, "topk_weights", torch.float32, p.M * p.topk), ctypes.byref(w),
        _arg(out, "out", torch.bfloat16, p.M * p.K), _stream(stream))
    _check("moe_apply_contiguous_static", st)


def moe_gate_up_act(plan: MoePlan, a, w1, w2, ws13, w1_scale=None, w2_scale=None, stream=None):
    w = _weights(plan, w1, w2, w1_scale, w2_scale)
    st = load_library().moe_gate_up_act(ctypes.byref(plan), _arg(a, "a", torch.bfloat16, plan.prob.M * plan.prob.K),
                                        ctypes.byref(w), _ws(ws13, "ws13", plan.ws13_bytes), _stream(stream))
    _check("moe_gate_up_act", st)


def moe_down_unpermute(plan: MoePlan, w1, w2, ws13, ws2, w1_scale=None, w2_scale=None, stream=None):
    w = _weights(plan, w1, w2, w1_scale, w2_scale)
    st = load_library().moe_down_unpermute(ctypes.byref(plan), ctypes.byref(w), _ws(ws13, "ws13", plan.ws13_bytes),
                                           _ws(ws2, "ws2", plan.ws2_bytes), _stream(stream))
    _check("moe_down_unpermute", st)


def moe_apply_batched(plan: MoePlan, a, expert_num_tokens, w1, w2, y, ws13, stream=None):
    w = _weights(plan, w1, w2)
    p = plan.prob
    slab = p.E * p.max_tokens * p.K
    st = load_library().moe_apply_batched(ctypes.byref(plan), _arg(a, "a", torch.bfloat16, slab),
                                          _arg(expert_num_tokens, "expert_num_tokens", torch.int32, p.E),
                                          ctypes.byref(w), _arg(y, "y", torch.bfloat16, slab),
                                          _ws(ws13, "ws13", plan.ws13_bytes), _stream(stream))
    _check("moe_apply_batched", st)


def moe_topk_reduce_contiguous(plan: MoePlan, y, topk_ids, topk_weights, out, stream=None,
                               expert_map: Optional[torch.Tensor] = None):
    p = plan.prob
    st = load_library().moe_topk_reduce_contiguous(ctypes.byref(plan), _arg(y, "y", torch.bfloat16, p.M * p.topk * p.K),
                                                   _ids_arg(plan, topk_ids),
                                                   _arg(topk_weights, "topk_weights", torch.float32, p.M * p.topk),
                                                   _map_arg(plan, expert_map),
                                                   _arg(out, "out", torch.bfloat16, p.M * p.K), _stream(stream))
    _check("moe_topk_reduce_contiguous", st)


def moe_naive_batched_ws_bytes(plan: MoePlan, n_out: int) -> int:
    v = load_library().moe_naive_batched_ws_bytes(ctypes.byref(plan), n_out)
    if v < 0:
        raise MoeError("moe_naive_batched_ws_bytes", MOE_EINVAL)
    return v


def moe_topk_reduce_naive_batched(plan: MoePlan, y, expert_num_tokens, row_token, row_weight,
                                  n_out: int, out, ws, stream=None):
    p = plan.prob
    rows = p.E * p.max_tokens
    st = load_library().moe_topk_reduce_naive_batched(
        ctypes.byref(plan), _arg(y, "y", torch.bfloat16, rows * p.K),
        _arg(expert_num_tokens, "expert_num_tokens", torch.int32, p.E),
        _arg(row_token, "row_token", torch.int32, rows), _arg(row_weight, "row_weight", torch.float32, rows),
        n_out, _arg(out, "out", torch.bfloat16, n_out * p.K),
        _ws(ws, "ws", moe_naive_batched_ws_bytes(plan, n_out)), _stream(stream))
    _check("moe_topk_reduce_naive_batched", st)


def moe_quantize_mxfp8(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None):
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("x must be float32 or bfloat16")
    rows = x.numel() // x.shape[-1]
    st = load_library().moe_quantize_mxfp8(_ptr(x), 0 if x.dtype == torch.float32 else 1, rows,
                                           x.shape[-1], _arg(codes, "codes", torch.uint8, x.numel()),
                                           _arg(scales, "scales", torch.uint8, x.numel() // 32),
                                           _stream(stream))
    _check("moe_quantize_mxfp8", st)


def moe_pack_mxfp8_scales(scales: torch.Tensor, packed: torch.Tensor, stream=None):
    """Row-major MXFP8 scale arrays ``[..., rows, cols/32]`` (as
    moe_quantize_mxfp8 writes them) into ``packed`` (same size) in the layout
    of W_MXFP8_GROUPED: each matrix of the last two dimensions in groups of
    16 bytes a row."""
    if scales.dim() < 2:
        raise ValueError("scales: expected [..., rows, cols/32]")
    rows, ncols = scales.shape[-2], scales.shape[-1] * 32
    mats = scales.numel() // max(rows * scales.shape[-1], 1)
    st = load_library().moe_pack_mxfp8_scales(_arg(scales, "scales", torch.uint8, scales.numel()),
                                              _arg(packed, "packed", torch.uint8, scales.numel()),
                                              mats, rows, ncols, _stream(stream))
    _check("moe_pack_mxfp8_scales", st)


# ------------------------------------------------------------- training ----

def _grouped(R, N, K, E) -> MoeGroupedProblem:
    return MoeGroupedProblem(R=R, N=N, K=K, E=E)


def moe_grouped_forward(x, w, group_offsets, y, stream=None):
    """y[r] = W[e] x[r] over the rows of each group (x [R,K], w [E,N,K], y [R,N] bf16)."""
    p = _grouped(x.shape[0], w.shape[1], w.shape[2], w.shape[0])
    st = load_library().moe_grouped_forward(ctypes.byref(p), _arg(x, "x", torch.bfloat16, p.R * p.K),
                                            _arg(w, "w", torch.bfloat16, p.E * p.N * p.K),
                                            _arg(group_offsets, "group_offsets", torch.int32, p.E + 1),
                                            _arg(y, "y", torch.bfloat16, p.R * p.N), _stream(stream))
    _check("moe_grouped_forward", st)


def moe_grouped_dgrad(dy, w, group_offsets, dx, stream=None):
    """dx[r] = W[e]^T dy[r] (dy [R,N], w [E,N,K], dx [R,K] bf16)."""
    p = _grouped(dy.shape[0], w.shape[1], w.shape[2], w.shape[0])
    st = load_library().moe_grouped_dgrad(ctypes.byref(p), _arg(dy, "dy", torch.bfloat16, p.R * p.N),
                                          _arg(w, "w", torch.bfloat16, p.E * p.N * p.K),
                                          _arg(group_offsets, "group_offsets", torch.int32, p.E + 1),
                                          _arg(dx, "dx", torch.bfloat16, p.R * p.K), _stream(stream))
    _check("moe_grouped_dgrad", st)


def moe_grouped_wgrad(dy, x, group_offsets, dw, accumulate: bool = False, stream=None):
    """dW[e] = sum over group e's rows of dy[r] x[r]^T into dw [E,N,K] float32
    (written, or added when ``accumulate``)."""
    p = _grouped(dy.shape[0], dw.shape[1], dw.shape[2], dw.shape[0])
    st = load_library().moe_grouped_wgrad(ctypes.byref(p), _arg(dy, "dy", torch.bfloat16, p.R * p.N),
                                          _arg(x, "x", torch.bfloat16, p.R * p.K),
                                          _arg(group_offsets, "group_offsets", torch.int32, p.E + 1),
                                          _arg(dw, "dw", torch.float32, p.E * p.N * p.K),
                                          1 if accumulate else 0, _stream(stream))
    _check("moe_grouped_wgrad", st)



# --------------------------------------------------------------- router ----

def make_router(E, topk, scoring=ROUTE_SOFTMAX, bias_kind=BIAS_NONE, renormalize=True, scale=1.0, groups=1,
                topk_groups=1) -> MoeRouter:
    return MoeRouter(E, topk, groups, topk_groups, scoring, bias_kind, 1 if renormalize else 0, scale)


def _current() -> int:
    """The device the kernels are launched on (torch.cuda.current_device())."""
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else torch.cuda.current_device()


def _device_for(t: torch.Tensor) -> int:
    """The current device; for a host tensor the refusal comes before CUDA is
    initialised for it."""
    return _current() if t.is_cuda else -2


def _on(dev: int, t: Optional[torch.Tensor], name: str, dtype, numel: int) -> Optional[int]:
    """_arg, and that the tensor lies on device ``dev``."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.numel() >= numel:
        return t.data_ptr()
    p = _arg(t, name, dtype, numel)   # names what is wrong
    raise ValueError(f"{name}: tensor on {t.device}, the current device is cuda:{dev} ({p:#x})")


def _ws_on(dev: int, t: torch.Tensor, name: str, nbytes: int) -> int:
    p = _ws(t, name, nbytes)
    if t.get_device() != dev:
        raise ValueError(f"{name}: tensor on {t.device}, the current device is cuda:{dev}")
    return p


def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


_LOGIT_DTYPES = {torch.float32: 0, torch.bfloat16: 1}


def _logits(dev: int, t: torch.Tensor, E: int, name: str):
    """(pointer, dtype code, row stride) of a [M, E] matrix whose rows are
    contiguous and may lie apart."""
    code = _LOGIT_DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: dtype {t.dtype}, expected torch.float32 or torch.bfloat16")
    if t.dim() != 2 or t.shape[1] != E:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [M, {E}]")
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError("expected a device tensor")
        raise ValueError(f"{name}: tensor on {t.device}, the current device is cuda:{dev}")
    M = t.shape[0]
    ld, one = t.stride()
    if (E > 1 and one != 1) or (M > 1 and ld < E):
        raise ValueError(f"{name}: strides {t.stride()}, expected contiguous rows that do not overlap")
    return t.data_ptr(), code, (ld if M > 1 else E)


def moe_route_topk(router: MoeRouter, logits, topk_ids, topk_weights, bias=None, stream=None):
    """The topk experts of each row of logits [M, E] (float32 or bf16, rows may
    lie apart) into topk_ids int32 [M, topk] and topk_weights float32 [M, topk]."""
    E, dev = router.E, _device_for(logits)
    ptr, code, ld = _logits(dev, logits, E, "logits")
    M = logits.shape[0]
    n = M * router.topk
    st = load_library().moe_route_topk(
        ctypes.byref(router), M, ptr, code, ld, _on(dev, bias, "bias", torch.float32, E),
        _on(dev, topk_ids, "topk_ids", torch.int32, n), _on(dev, topk_weights, "topk_weights", torch.float32, n),
        _raw_stream(stream, dev))
    _check("moe_route_topk", st)


def moe_route_topk_backward(router: MoeRouter, logits, topk_ids, dweights, dlogits, bias=None, stream=None):
    """dlogits [M, E] (the logits' dtype) from the gradient dweights [M, topk]
    of the weights moe_route_topk gave for topk_ids."""
    E, dev = router.E, _device_for(logits)
    ptr, code, ld = _logits(dev, logits, E, "logits")
    dptr, dcode, dld = _logits(dev, dlogits, E, "dlogits")
    M = logits.shape[0]
    n = M * router.topk
    if dcode != code or dlogits.shape[0] != M:
        raise ValueError("dlogits: expected the dtype and shape of logits")
    st = load_library().moe_route_topk_backward(
        ctypes.byref(router), M, ptr, code, ld, _on(dev, bias, "bias", torch.float32, E),
        _on(dev, topk_ids, "topk_ids", torch.int32, n), _on(dev, dweights, "dweights", torch.float32, n), dptr, dld,
        _raw_stream(stream, dev))
    _check("moe_route_topk_backward", st)


# ---------------------------------------------------------------- layer ----

def make_layer_problem(M, K, I, router: MoeRouter, shared_experts=0, w_dtype=W_BF16,
                       w1_order=W1_HALVES) -> MoeLayerProblem:
    return MoeLayerProblem(M, K, I, shared_experts, router, w_dtype, w1_order)


def moe_layer_plan_init(prob: MoeLayerProblem) -> MoeLayerPlan:
    plan = MoeLayerPlan()
    st = load_library().moe_layer_plan_init(ctypes.byref(plan), ctypes.byref(prob))
    _check("moe_layer_plan_init", st, plan)
    return plan


def allocate_layer_workspace(plan: MoeLayerPlan, device="cuda") -> torch.Tensor:
    """The layer's workspace, zero-filled (its counters start at zero); it also
    serves any other plan whose ws_bytes it holds."""
    return torch.zeros(plan.ws_bytes, dtype=torch.uint8, device=device)


def check_layer_status(plan: MoeLayerPlan, ws: torch.Tensor):
    """Raise MoeError when a call on this workspace gave up its bounded wait:
    its ``out`` and every later one's is NaN until the workspace is zero-filled
    again.  Synchronises with the device."""
    timeouts = int(ws_view(ws, plan.off_status, 1).cpu()[0])
    if timeouts:
        raise MoeError("moe_layer_apply", MOE_EHIP, f"{timeouts} bounded waits timed out; out is NaN")


def moe_layer_apply(plan: MoeLayerPlan, x, router_w, w1, w2, out, topk_ids, topk_weights, ws, router_bias=None,
                    w1_scale=None, w2_scale=None, stream=None):
    """out [M, K] = the whole layer on x [M, K] (bf16); also the router's choice
    (topk_ids int32, topk_weights float32, [M, topk]).  ws: from
    allocate_layer_workspace; calls that share it must not overlap."""
    p = plan.prob
    r = p.router
    mx = p.w_dtype == W_MXFP8
    wt = torch.uint8 if mx else torch.bfloat16
    n1 = (r.E + p.shared_experts) * 2 * p.I * p.K
    n2 = n1 // 2
    if mx and (w1_scale is None or w2_scale is None):
        raise ValueError("MXFP8 weights need w1_scale and w2_scale")
    dev = _device_for(x)
    w = MoeWeights(_on(dev, w1, "w1", wt, n1), _on(dev, w1_scale, "w1_scale", torch.uint8, n1 // 32 if mx else 0),
                   _on(dev, w2, "w2", wt, n2), _on(dev, w2_scale, "w2_scale", torch.uint8, n2 // 32 if mx else 0), None)
    st = load_library().moe_layer_apply(
        ctypes.byref(plan), _on(dev, x, "x", torch.bfloat16, p.M * p.K),
        _on(dev, router_w, "router_w", torch.bfloat16, r.E * p.K),
        _on(dev, router_bias, "router_bias", torch.float32, r.E), ctypes.byref(w),
        _on(dev, out, "out", torch.bfloat16, p.M * p.K), _on(dev, topk_ids, "topk_ids", torch.int32, p.M * r.topk),
        _on(dev, topk_weights, "topk_weights", torch.float32, p.M * r.topk), _ws_on(dev, ws, "ws", plan.ws_bytes),
        _raw_stream(stream, dev))
    _check("moe_layer_apply", st)


# ----------------------------------------------------------------- lora ----

def _lora_bytes(fn: str, R, N, K, G, rank) -> int:
    v = getattr(load_library(), fn)(ctypes.byref(MoeLoraProblem(R, N, K, G, rank)))
    if v < 0:
        raise MoeError(fn, MOE_EINVAL)
    return v


def moe_lora_low_bytes(R, N, K, G, rank) -> int:
    return _lora_bytes("moe_lora_low_bytes", R, N, K, G, rank)


def moe_lora_ws_bytes(R, N, K, G, rank) -> int:
    return _lora_bytes("moe_lora_ws_bytes", R, N, K, G, rank)


def allocate_lora_low(R, rank, device="cuda") -> torch.Tensor:
    """The narrow products of R rows, as moe_lora_forward and moe_lora_dgrad
    write them (moe_lora_low_bytes)."""
    return torch.empty(max(moe_lora_low_bytes(R, 64, 64, 1, rank), 16), dtype=torch.uint8, device=device)


def allocate_lora_workspace(R, N, K, G, rank, device="cuda") -> torch.Tensor:
    """moe_lora_wgrad's workspace (moe_lora_ws_bytes)."""
    return torch.empty(max(moe_lora_ws_bytes(R, N, K, G, rank), 16), dtype=torch.uint8, device=device)


def _lora_project(fn, v, C, w, a, b, scale, adapter, out, out_cols, low, stream):
    if w.dim() != 2 or a.dim() != 3 or b.dim() != 3:
        raise ValueError("expected w [N, K], a [G, rank, K], b [G, N, rank]")
    (N, K), (G, rank) = w.shape, a.shape[:2]
    if a.shape[2] != K or tuple(b.shape) != (G, N, rank):
        raise ValueError(f"w {tuple(w.shape)}, a {tuple(a.shape)}, b {tuple(b.shape)}: "
                         "expected [N, K], [G, rank, K], [G, N, rank]")
    R = v.shape[0]
    if v.shape[1:] != w.shape[C:C + 1] or tuple(out.shape) != (R, w.shape[out_cols]):
        raise ValueError(f"rows {tuple(v.shape)} and {tuple(out.shape)} do not fit w {tuple(w.shape)}")
    p, dev = MoeLoraProblem(R, N, K, G, rank), _device_for(v)
    st = getattr(load_library(), fn)(
        ctypes.byref(p), _on(dev, v, "rows", torch.bfloat16, 0), _on(dev, w, "w", torch.bfloat16, 0),
        _on(dev, a, "a", torch.bfloat16, 0), _on(dev, b, "b", torch.bfloat16, 0),
        _on(dev, scale, "scale", torch.float32, G), _on(dev, adapter, "adapter", torch.int32, R),
        _on(dev, out, "output rows", torch.bfloat16, 0), _ws_on(dev, low, "low", 6 * R * rank),
        _raw_stream(stream, dev))
    _check(fn, st)


def moe_lora_forward(x, w, a, b, scale, adapter, y, low, stream=None):
    """y [R, N] = x [R, K] W^T + scale_g (x A_g^T) B_g^T, g = adapter[r] (int32
    [R], -1: none); w [N, K], a [G, rank, K], b [G, N, rank], scale float32 [G];
    low: from allocate_lora_low, read again by moe_lora_wgrad."""
    _lora_project("moe_lora_forward", x, 1, w, a, b, scale, adapter, y, 0, low, stream)


def moe_lora_dgrad(dy, w, a, b, scale, adapter, dx, low, stream=None):
    """dx [R, K] = dy [R, N] W + scale_g (dy B_g) A_g."""
    _lora_project("moe_lora_dgrad", dy, 0, w, a, b, scale, adapter, dx, 1, low, stream)


def moe_lora_wgrad(x, dy, low_x, low_dy, adapter, da, db, ws, accumulate: bool = False, stream=None):
    """da [G, rank, K] and db [G, N, rank] (float32, written, or added to when
    ``accumulate``) from the forward's low (of x) and the dgrad's (of dy)."""
    (R, K), N = x.shape, dy.shape[1]
    G, rank = da.shape[:2]
    if dy.shape[0] != R or da.shape[2] != K or tuple(db.shape) != (G, N, rank):
        raise ValueError(f"x {tuple(x.shape)}, dy {tuple(dy.shape)}, da {tuple(da.shape)}, db {tuple(db.shape)} "
                         "do not fit")
    p, dev = MoeLoraProblem(R, N, K, G, rank), _device_for(x)
    low = 6 * R * rank
    st = load_library().moe_lora_wgrad(
        ctypes.byref(p), _on(dev, x, "x", torch.bfloat16, 0), _on(dev, dy, "dy", torch.bfloat16, 0),
        _ws_on(dev, low_x, "low_x", low), _ws_on(dev, low_dy, "low_dy", low),
        _on(dev, adapter, "adapter", torch.int32, R), _on(dev, da, "da", torch.float32, 0),
        _on(dev, db, "db", torch.float32, 0), 1 if accumulate else 0,
        _ws_on(dev, ws, "ws", max(load_library().moe_lora_ws_bytes(ctypes.byref(p)), 0)), _raw_stream(stream, dev))
    _check("moe_lora_wgrad", st)

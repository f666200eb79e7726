"""The router (moe_route_topk, moe_route_topk_backward) against the 64-bit
reference: choices exactly, values within bounds derived below.

Weights: computed in float64 from the chosen logits and rounded once, 2^-24
relative; without renormalisation a softmax's denominator is a float32 sum of
float32 exponentials, each off by 2 units in the last place at most (2^-22)
plus its argument's rounding (|d| e^-d <= 0.37 times 2^-24), added per lane in
at most 32 steps (2^-19).  Gradients: the same, times the magnitude of the
terms they are differences of; bf16 outputs add half a step, 2^-8.
"""
import numpy as np
import pytest
import torch

import mixture_experts_expert_align_amd as moe
from operator_refs import route_backward, route_topk

W_EXACT = 2.0 ** -23
W_SUM = 2.0 ** -24 + 2.0 ** -21 + 32 * 2.0 ** -24
SCORING = {"softmax": moe.ROUTE_SOFTMAX, "sigmoid": moe.ROUTE_SIGMOID}
BIAS = {"none": moe.BIAS_NONE, "logit": moe.BIAS_LOGIT, "select": moe.BIAS_SELECT}

gpu = pytest.mark.gpu


# ----------------------------------------------------------------- refusals --

@pytest.mark.parametrize("kw", [
    dict(E=0), dict(E=2049), dict(topk=0), dict(topk=17), dict(E=128, topk=65), dict(groups=0), dict(groups=3),
    dict(E=130, groups=65), dict(groups=4, topk_groups=5), dict(groups=4, topk_groups=0), dict(scoring=2),
    dict(bias_kind=3), dict(scale=float("inf")), dict(scale=float("nan")),
])
def test_router_refuses(kw):
    base = dict(E=16, topk=2)
    base.update(kw)
    r = moe.make_router(**base)
    lib = moe.load_library()
    import ctypes
    # every pointer is a plausible address: only the router is wrong
    a = 4096
    bias = a if r.bias_kind else None
    assert lib.moe_route_topk(ctypes.byref(r), 4, a, 0, base["E"], bias, a, a, None) == moe.MOE_EINVAL
    assert lib.moe_route_topk_backward(ctypes.byref(r), 4, a, 0, base["E"], bias, a, a, a, base["E"],
                                       None) == moe.MOE_EINVAL


def test_router_refuses_arguments():
    import ctypes
    lib = moe.load_library()
    r, rb = moe.make_router(16, 2), moe.make_router(16, 2, bias_kind=moe.BIAS_SELECT)
    a = 4096

    def fwd(rr=r, M=4, logits=a, dtype=0, ld=16, bias=None, ids=a, w=a):
        return lib.moe_route_topk(ctypes.byref(rr), M, logits, dtype, ld, bias, ids, w, None)

    def bwd(rr=r, M=4, logits=a, dtype=0, ld=16, bias=None, ids=a, w=a, dl=a, dld=16):
        return lib.moe_route_topk_backward(ctypes.byref(rr), M, logits, dtype, ld, bias, ids, w, dl, dld, None)

    for bad in (dict(M=-1), dict(M=1 << 31), dict(logits=None), dict(logits=a + 2), dict(dtype=2), dict(ld=15),
                dict(bias=a), dict(ids=None), dict(ids=a + 2), dict(w=None), dict(rr=rb, bias=None),
                dict(rr=rb, bias=a + 1), dict(dtype=1, logits=a + 1)):
        assert fwd(**bad) == moe.MOE_EINVAL, bad
        assert bwd(**bad) == moe.MOE_EINVAL, bad
    assert bwd(dl=None) == moe.MOE_EINVAL and bwd(dld=15) == moe.MOE_EINVAL and bwd(dl=a + 1) == moe.MOE_EINVAL
    assert fwd(M=0, logits=None, ids=None, w=None) == moe.MOE_OK      # nothing to do
    assert bwd(M=0, logits=None, ids=None, w=None, dl=None) == moe.MOE_OK
    assert lib.moe_route_topk(None, 4, a, 0, 16, None, a, a, None) == moe.MOE_EINVAL


def test_binding_refuses_shapes():
    r = moe.make_router(16, 2)
    x = torch.zeros(4, 16)
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_route_topk(r, x, ids, w)
    with pytest.raises(ValueError, match="dtype"):
        moe.moe_route_topk(r, x.half(), ids, w)
    with pytest.raises(ValueError, match="shape"):
        moe.moe_route_topk(r, torch.zeros(4, 15), ids, w)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_reference_gradient_is_the_difference_quotient(scoring, renorm):
    rng = np.random.default_rng(5)
    l = rng.normal(size=(3, 9))
    dw = rng.normal(size=(3, 4))
    ids, _ = route_topk(l, 4, scoring, renorm=renorm, scale=1.5)
    d, _ = route_backward(l, ids, dw, scoring, renorm=renorm, scale=1.5)
    h = 1e-6
    for t in range(3):
        for e in range(9):
            f = []
            for sgn in (1, -1):
                lp = l.copy()
                lp[t, e] += sgn * h
                ids2, w = route_topk(lp, 4, scoring, renorm=renorm, scale=1.5)
                assert np.array_equal(ids2, ids)
                f.append((w * dw).sum())
            assert abs((f[0] - f[1]) / (2 * h) - d[t, e]) < 1e-8


# ---------------------------------------------------------------------- GPU --

def run(l, topk, scoring, bias, bias_kind, renorm, scale, groups, topk_groups, dw=None):
    r = moe.make_router(l.shape[1], topk, SCORING[scoring], BIAS[bias_kind], renorm, scale, groups, topk_groups)
    M = l.shape[0]
    # one row more than the call writes
    ids = torch.full((M + 1, topk), 77, dtype=torch.int32, device="cuda")
    w = torch.full((M + 1, topk), 7.0, device="cuda")
    b = None if bias is None else torch.from_numpy(bias).cuda()
    moe.moe_route_topk(r, l, ids, w, bias=b)
    assert (ids[M] == 77).all() and (w[M] == 7.0).all()
    dl = None
    if dw is not None:
        dl = torch.full_like(l, float("nan"))
        moe.moe_route_topk_backward(r, l, ids, torch.from_numpy(dw).cuda(), dl, bias=b)
    return ids[:M].cpu().numpy(), w[:M].cpu().numpy(), dl


def check(l, topk, scoring="softmax", bias=None, bias_kind="none", renorm=True, scale=1.0, groups=1, topk_groups=1,
          seed=0):
    M = l.shape[0]
    dw = np.random.default_rng(seed).normal(size=(M, topk)).astype(np.float32)
    ids, w, dl = run(l, topk, scoring, bias, bias_kind, renorm, scale, groups, topk_groups, dw)
    lh = l.float().cpu().numpy()
    rid, rw = route_topk(lh, topk, scoring, bias, bias_kind, renorm, scale, groups, topk_groups)
    assert np.array_equal(ids, rid), np.argwhere(ids != rid)[:4]
    tol = W_SUM if scoring == "softmax" and not renorm else W_EXACT
    assert np.all(np.abs(w - rw) <= tol * np.abs(rw) + 1e-37)
    rd, mag = route_backward(lh, rid, dw, scoring, bias, bias_kind, renorm, scale)
    got = dl.float().cpu().numpy().astype(np.float64)
    # the dense softmax gradient: score, sum and difference each rounded in float32
    gt = 3 * W_SUM if scoring == "softmax" and not renorm else W_EXACT
    bound = gt * mag + 1e-37
    if l.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * np.abs(rd)
    assert np.all(np.abs(got - rd) <= bound), (np.abs(got - rd) - bound).max()


def logits(M, E, dtype, seed):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.normal(size=(M, E)).astype(np.float32)).to("cuda", dtype)


@gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias_kind", ["none", "logit", "select"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("M,E,topk,groups,tg", [(1, 1, 1, 1, 1), (3, 5, 5, 1, 1), (130, 64, 8, 1, 1), (7, 65, 3, 1, 1),
                                                (33, 128, 8, 8, 3), (9, 320, 64, 1, 1), (17, 512, 8, 16, 4),
                                                (5, 600, 7, 1, 1), (3, 2048, 6, 64, 2), (21, 99, 4, 3, 2),
                                                (4, 256, 12, 1, 1)])
def test_router(scoring, bias_kind, renorm, M, E, topk, groups, tg):
    for dtype in (torch.float32, torch.bfloat16):
        rng = np.random.default_rng(E)
        bias = None if bias_kind == "none" else (0.25 * rng.normal(size=E)).astype(np.float32)
        check(logits(M, E, dtype, M + E), topk, scoring, bias, bias_kind, renorm, 2.5, groups, tg)


@gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias_kind", ["none", "logit", "select"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("M,E,topk,groups,tg", [(4097, 1, 1, 1, 1), (4101, 65, 3, 1, 1), (4099, 128, 16, 16, 3),
                                                (4098, 99, 4, 3, 2), (4100, 256, 12, 2, 1), (2049, 512, 8, 16, 4),
                                                (2051, 300, 16, 1, 1), (4098, 200, 17, 1, 1),
                                                (4098, 160, 4, 32, 9)])
def test_router_many_rows(scoring, bias_kind, renorm, M, E, topk, groups, tg):
    """Enough tokens for several of them to a wave (up to 16 choices and 16 groups)."""
    rng = np.random.default_rng(E)
    bias = None if bias_kind == "none" else (0.25 * rng.normal(size=E)).astype(np.float32)
    dtype = torch.float32 if renorm else torch.bfloat16
    check(logits(M, E, dtype, M + E), topk, scoring, bias, bias_kind, renorm, 2.5, groups, tg)


@gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias_kind", ["none", "logit", "select"])
@pytest.mark.parametrize("groups,tg", [(1, 1), (4, 2)])
def test_router_masks_and_special_values(scoring, bias_kind, groups, tg, rows=16):
    E, topk = 64, 6
    l = logits(16, E, torch.float32, 3)
    low = torch.finfo(torch.float32).min
    l[0] = float("-inf")                      # nothing left
    l[1, 3:] = float("-inf")                  # fewer than topk left
    l[2] = float("nan")
    l[3, ::2] = float("nan")
    l[4] = low                                # a mask of the lowest value in every place
    l[5, 1:] = low
    l[6, 7] = float("inf")
    l[7, 7:9] = float("inf")
    l[8] = 0.0                                # all tied
    l[9, 10:20] = 3.0
    l[10, 5], l[10, 6] = -0.0, 0.0
    l[11] = 60.0 + l[11]
    l[12] = -200.0 + l[12]
    l[13, 16:32] = float("-inf")              # a whole group
    l[14, :63] = float("-inf")
    bias = None
    if bias_kind != "none":
        bias = np.zeros(E, np.float32)
        bias[5] = float("-inf")
        bias[6] = float("nan")
        bias[40] = 0.5
    l = l[torch.arange(rows) % 16].contiguous()
    for renorm in (True, False):
        check(l, topk, scoring, bias, bias_kind, renorm, 1.0, groups, tg)


@gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias_kind", ["none", "logit", "select"])
@pytest.mark.parametrize("groups,tg", [(1, 1), (4, 2), (16, 5)])
def test_router_masks_and_special_values_many_rows(scoring, bias_kind, groups, tg):
    test_router_masks_and_special_values(scoring, bias_kind, groups, tg, rows=4101)


@gpu
def test_router_ties_go_to_the_lowest():
    l = torch.zeros(5, 200, device="cuda", dtype=torch.bfloat16)
    l[1, 130:] = 1.0
    l[2, ::3] = -1.0
    l[3, 199] = 1.0
    ids, w, _ = run(l, 4, "softmax", None, "none", True, 1.0, 1, 1)
    assert ids.tolist() == [[0, 1, 2, 3], [130, 131, 132, 133], [1, 2, 4, 5], [199, 0, 1, 2], [0, 1, 2, 3]]
    assert np.all(w[0] == 0.25)


@gpu
@pytest.mark.parametrize("M", [37, 4103])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_router_row_strides(dtype, M):
    """Rows inside a wider matrix (at an odd column for the alignment), and the
    gradient into one: the columns between stay as they were."""
    wide = logits(M, 150, dtype, 9)
    l = wide[:, 3:131]
    dw = np.random.default_rng(1).normal(size=(M, 8)).astype(np.float32)
    r = moe.make_router(128, 8, renormalize=False)
    out = {}
    for name, src in (("view", l), ("dense", l.contiguous())):
        ids = torch.empty(M, 8, dtype=torch.int32, device="cuda")
        w = torch.empty(M, 8, device="cuda")
        moe.moe_route_topk(r, src, ids, w)
        big = torch.full((M, 140), 5.0, dtype=dtype, device="cuda")
        dl = big[:, 5:133] if name == "view" else torch.empty(M, 128, dtype=dtype, device="cuda")
        moe.moe_route_topk_backward(r, src, ids, torch.from_numpy(dw).cuda(), dl)
        if name == "view":
            assert (big[:, :5] == 5.0).all() and (big[:, 133:] == 5.0).all()
        out[name] = (ids, w, dl)
    for a, b in zip(out["view"], out["dense"]):
        assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("copies", [1, 701])
def test_router_backward_skips_bad_slots_and_adds_repeated_ones(copies):
    l = logits(3 * copies, 32, torch.float32, 4)
    dw = np.random.default_rng(2).normal(size=(3 * copies, 4)).astype(np.float32)
    ids = np.array([[1, -1, 5, 99], [4, 4, 2, 31], [-1, -1, -1, -5]] * copies, np.int32)
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            r = moe.make_router(32, 4, SCORING[scoring], renormalize=renorm)
            dl = torch.full_like(l, float("nan"))
            moe.moe_route_topk_backward(r, l, torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(), dl)
            rd, mag = route_backward(l.cpu().numpy(), ids, dw, scoring, renorm=renorm)
            assert np.all(np.abs(dl.cpu().numpy() - rd) <= 3 * W_SUM * mag + 1e-37)


@gpu
def test_router_many_tokens_feeds_the_experts():
    """The workload's router output through the experts' own path: ids and
    weights go straight into moe_align_permute (a -1 slot is skipped)."""
    M, E, topk = 8192, 128, 8
    l = logits(M, E, torch.float32, 11)
    l[100] = float("-inf")
    check(l, topk, "softmax", np.zeros(E, np.float32), "logit")
    r = moe.make_router(E, topk)
    ids = torch.empty(M, topk, dtype=torch.int32, device="cuda")
    w = torch.empty(M, topk, device="cuda")
    moe.moe_route_topk(r, l, ids, w)
    plan = moe.moe_plan_init(moe.make_problem(M, 256, 128, E, topk=topk))
    ws13, _ = moe.allocate_workspaces(plan)
    moe.moe_align_permute(plan, ids, ws13)
    counts = moe.ws_view(ws13, plan.off_counts, E).cpu().numpy()
    assert np.array_equal(counts, np.bincount(ids.cpu().numpy()[ids.cpu().numpy() >= 0], minlength=E))
    assert counts.sum() == (M - 1) * topk and moe.status_words(plan, ws13)[0] == 0


@gpu
def test_router_graph_replays_and_streams():
    l = logits(64, 128, torch.float32, 21)
    dw = torch.randn(64, 8, device="cuda")
    r = moe.make_router(128, 8, moe.ROUTE_SIGMOID, groups=8, topk_groups=3, scale=2.5)

    def call(o):
        moe.moe_route_topk(r, l, o[0], o[1])
        moe.moe_route_topk_backward(r, l, o[0], dw, o[2])

    def bufs():
        return (torch.zeros(64, 8, dtype=torch.int32, device="cuda"), torch.zeros(64, 8, device="cuda"),
                torch.zeros_like(l))

    ref, out = bufs(), bufs()
    call(ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(out)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(ref, out))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    for i in range(4):
        l.add_(0.125 * i)
        l[:, i] -= 1.0
        call(ref)
        for o in out:
            o.fill_(-3)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, out)), i


@gpu
@pytest.mark.parametrize("M,E,topk", [((1 << 26) + 5, 17, 17), ((1 << 28) + 5, 1, 1)])
def test_router_tokens_past_one_launch(M, E, topk):
    """More tokens than the threads of one launch can take (a wave, and 16
    lanes, to a token); rows at the ends and about every power of two."""
    l = torch.empty(M, E, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    for i in range(0, M, 1 << 24):
        l[i:i + (1 << 24)].normal_(generator=g)
    r = moe.make_router(E, topk, moe.ROUTE_SIGMOID, renormalize=False)
    ids = torch.full((M, topk), 99, dtype=torch.int32, device="cuda")
    w = torch.full((M, topk), float("nan"), device="cuda")
    moe.moe_route_topk(r, l, ids, w)
    dl = torch.full_like(l, float("nan"))
    dw = torch.full((M, topk), 0.5, device="cuda")
    moe.moe_route_topk_backward(r, l, ids, dw, dl)
    assert bool((ids >= 0).all()) and bool((ids < E).all()) and bool(w.isfinite().all()) and bool(dl.isfinite().all())
    at = sorted({t for p in range(1, 29) for t in range((1 << p) - 2, (1 << p) + 3) if t < M} | set(range(M - 40, M)))
    rows = torch.tensor(at, device="cuda")
    lh = l[rows].float().cpu().numpy()
    rid, rw = route_topk(lh, topk, "sigmoid", renorm=False)
    assert np.array_equal(ids[rows].cpu().numpy(), rid)
    assert np.all(np.abs(w[rows].cpu().numpy() - rw) <= W_EXACT * np.abs(rw))
    rd, _ = route_backward(lh, rid, np.full(rid.shape, 0.5, np.float32), "sigmoid", renorm=False)
    assert np.all(np.abs(dl[rows].double().cpu().numpy() - rd) <= (2.0 ** -8 + W_EXACT) * np.abs(rd))


@gpu
@pytest.mark.parametrize("M", [40, 2053])
@pytest.mark.parametrize("E,topk", [(64, 4), (100, 8), (300, 1), (500, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_router_gradient_of_confident_tokens(M, E, topk, dtype):
    """Softmax over all experts, one of which has nearly all of it: its gradient
    g (1 - p) is small and must come out to the result's own precision.  In
    float64 (some 2^-46 of the terms, of exponentials and their sum) but for
    the unchosen's float32 exponential (2^-22) and at most four more float32
    roundings (2^-24 each), and half a bf16 step."""
    l = logits(M, E, torch.float32, E + topk)
    gap = torch.linspace(4.0, 22.0, M, device="cuda")
    l[torch.arange(M), torch.arange(M) % E] += gap
    l = l.to(dtype)
    dw = np.random.default_rng(M).normal(size=(M, topk)).astype(np.float32)
    r = moe.make_router(E, topk, renormalize=False, scale=1.5)
    ids = torch.empty(M, topk, dtype=torch.int32, device="cuda")
    w = torch.empty(M, topk, device="cuda")
    moe.moe_route_topk(r, l, ids, w)
    dl = torch.full_like(l, float("nan"))
    moe.moe_route_topk_backward(r, l, ids, torch.from_numpy(dw).cuda(), dl)
    rd, mag = route_backward(l.float().cpu().numpy(), ids.cpu().numpy(), dw, renorm=False, scale=1.5)
    bound = 2.0 ** -21 * np.abs(rd) + 2.0 ** -46 * mag + (2.0 ** -8 * np.abs(rd) if dtype == torch.bfloat16 else 0) + 1e-37
    d = np.abs(dl.double().cpu().numpy() - rd)
    assert np.all(d <= bound), (np.nanmax(d / bound), np.argwhere(~(d <= bound))[:3])


@gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias_kind", ["none", "logit", "select"])
@pytest.mark.parametrize("M,E,topk,groups,tg", [(6147, 256, 12, 2, 1), (6145, 129, 16, 1, 1), (6150, 240, 5, 16, 4),
                                                (6144, 200, 8, 8, 3)])
def test_router_many_rows_of_more_than_128_experts(scoring, bias_kind, M, E, topk, groups, tg):
    """On either side of the number of tokens from which several share a wave."""
    rng = np.random.default_rng(E)
    bias = None if bias_kind == "none" else (0.25 * rng.normal(size=E)).astype(np.float32)
    for renorm, dtype in ((True, torch.float32), (False, torch.bfloat16)):
        check(logits(M, E, dtype, M + E), topk, scoring, bias, bias_kind, renorm, 2.5, groups, tg)


@gpu
@pytest.mark.parametrize("E,topk", [(129, 3), (300, 8), (500, 16)])
def test_router_gradient_of_confident_tokens_many_rows(E, topk):
    """The same where several tokens of more than 128 experts share a wave."""
    test_router_gradient_of_confident_tokens(4101, E, topk, torch.float32)


@gpu
@pytest.mark.parametrize("M", [24, 4104])
@pytest.mark.parametrize("E", [64, 200, 700])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_router_largest_differences_between_logits(M, E, scoring):
    """A logit that counts as the largest float32 beside ones of the lowest, of
    every size between, and masked ones: no NaN, and what the formulas give."""
    l = logits(M, E, torch.float32, E)
    low, top = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    l[0::8, 1::3] = low
    l[0::8, 5] = float("inf")
    l[1::8, ::2] = low
    l[1::8, 7] = top
    l[2::8] *= 1e37
    l[3::8] *= 1e4
    l[4::8, 9] = 1e30
    l[5::8, ::5] = -1e30
    l[6::8, 1:] = float("-inf")
    l[7::8, :3] = top
    l[7::8, 4:] = low
    for renorm in (True, False):
        check(l, 6, scoring, renorm=renorm)

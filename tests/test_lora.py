"""Adapters beside a shared projection (moe_lora_forward, _dgrad, _wgrad)
against the formulas in 64 bits.

Bounds per element, u = 2^-23 (a float32 operation; the matrix units may
truncate): the narrow product s is off by (C + 64) u sum |A| |x| |scale| from
its sum of C terms and 2^-23 |s| from its three pieces; y by that times |B|,
by 2^-17 of |B| |s| (the tiles use two pieces of s), by (K + 3 rank + 64) u
of the sum of the magnitudes, and by half a bf16 step, 2^-8 |y|.  dA and dB
(float32) by the error of t or s times |x| or |dy| and (3 rows + 64) u of
the sum of magnitudes; their root mean square error is also held to 2^-18 of
the result's, far below what one bf16 piece would leave (2^-9)."""
import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_expert_align_amd as moe

gpu = pytest.mark.gpu
U = 2.0 ** -23


# ----------------------------------------------------------------- refusals --

@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), moe.MOE_EINVAL), (dict(R=1 << 31), moe.MOE_EINVAL), (dict(N=0), moe.MOE_EINVAL),
    (dict(K=-64), moe.MOE_EINVAL), (dict(G=0), moe.MOE_EINVAL), (dict(rank=0), moe.MOE_EINVAL),
    (dict(N=96), moe.MOE_EUNSUPPORTED), (dict(K=32), moe.MOE_EUNSUPPORTED), (dict(rank=12), moe.MOE_EUNSUPPORTED),
    (dict(rank=136), moe.MOE_EUNSUPPORTED), (dict(G=4097), moe.MOE_EUNSUPPORTED),
    (dict(R=1 << 24), moe.MOE_EUNSUPPORTED), (dict(N=1 << 15, K=1 << 15), moe.MOE_EUNSUPPORTED),
    (dict(N=1 << 40), moe.MOE_EUNSUPPORTED), (dict(G=4096, rank=128, N=2048), moe.MOE_EUNSUPPORTED),
])
def test_lora_refuses_problems(kw, code):
    base = dict(R=4, N=128, K=64, G=2, rank=8)
    base.update(kw)
    p = ctypes.byref(moe.MoeLoraProblem(**base))
    lib = moe.load_library()
    a = 4096
    assert lib.moe_lora_low_bytes(p) == -1 and lib.moe_lora_ws_bytes(p) == -1
    assert lib.moe_lora_forward(p, a, a, a, a, a, a, a, a, None) == code
    assert lib.moe_lora_dgrad(p, a, a, a, a, a, a, a, a, None) == code
    assert lib.moe_lora_wgrad(p, a, a, a, a, a, a, a, 0, a, None) == code


def test_lora_refuses_pointers():
    lib = moe.load_library()
    p = ctypes.byref(moe.MoeLoraProblem(4, 128, 64, 2, 8))
    z = ctypes.byref(moe.MoeLoraProblem(0, 128, 64, 2, 8))
    a = 4096
    assert lib.moe_lora_low_bytes(p) == 4 * 8 * 3 * 2 and lib.moe_lora_ws_bytes(p) > 0
    for i in range(8):
        for bad in (None, a + 2):
            args = [a] * 8
            args[i] = bad
            assert lib.moe_lora_forward(p, *args, None) == moe.MOE_EINVAL, i
            assert lib.moe_lora_dgrad(p, *args, None) == moe.MOE_EINVAL, i
    for i in range(9):
        if i == 7:
            continue
        for bad in (None, a + 2):
            args = [a] * 7 + [0, a]
            args[i] = bad
            assert lib.moe_lora_wgrad(p, *args, None) == moe.MOE_EINVAL, i
    assert lib.moe_lora_wgrad(p, *([a] * 7), 2, a, None) == moe.MOE_EINVAL
    assert lib.moe_lora_forward(z, None, a, a, a, a, None, None, None, None) == moe.MOE_OK
    assert lib.moe_lora_dgrad(z, None, a, a, a, a, None, None, None, None) == moe.MOE_OK


def test_lora_binding_refuses_shapes():
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    args = lambda **k: {**dict(x=t(4, 64), w=t(128, 64), a=t(2, 8, 64), b=t(2, 128, 8), scale=torch.ones(2),
                               adapter=torch.zeros(4, dtype=torch.int32), y=t(4, 128),
                               low=torch.zeros(192, dtype=torch.uint8)), **k}
    for bad in (dict(a=t(2, 8, 128)), dict(b=t(2, 8, 128)), dict(x=t(4, 128)), dict(y=t(4, 64)), dict(w=t(2, 128, 64))):
        with pytest.raises(ValueError):
            moe.moe_lora_forward(**args(**bad))
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_lora_forward(**args())


# ---------------------------------------------------------------------- GPU --

class Case:
    def __init__(self, R, N, K, G, rank, order="mixed", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.R, self.N, self.K, self.G, self.rank = R, N, K, G, rank
        self.x, self.dy = rn(R, K).bfloat16(), rn(R, N).bfloat16()
        self.w = (rn(N, K) * K ** -0.5).bfloat16()
        self.a = (rn(G, rank, K) * K ** -0.5).bfloat16()
        self.b = (rn(G, N, rank) * rank ** -0.5).bfloat16()
        self.scale = 0.5 + torch.rand(G, generator=g, device="cuda")
        ad = torch.randint(-1, G, (R,), generator=g, device="cuda", dtype=torch.int32)
        self.adapter = ad.sort().values if order == "runs" else ad if order == "mixed" else torch.full_like(ad, order)

    def buffers(self):
        nan = lambda *s, dt=torch.bfloat16: torch.full(s, float("nan"), dtype=dt, device="cuda")
        o = {"y": nan(self.R, self.N), "dx": nan(self.R, self.K), "da": nan(self.G, self.rank, self.K, dt=torch.float32),
             "db": nan(self.G, self.N, self.rank, dt=torch.float32)}
        o["low"], o["low_dy"] = (moe.allocate_lora_low(self.R, self.rank).fill_(0xff) for _ in range(2))
        o["ws"] = moe.allocate_lora_workspace(self.R, self.N, self.K, self.G, self.rank)
        return o

    def call(self, o, stream=None, accumulate=False):
        moe.moe_lora_forward(self.x, self.w, self.a, self.b, self.scale, self.adapter, o["y"], o["low"], stream=stream)
        moe.moe_lora_dgrad(self.dy, self.w, self.a, self.b, self.scale, self.adapter, o["dx"], o["low_dy"],
                           stream=stream)
        moe.moe_lora_wgrad(self.x, self.dy, o["low"], o["low_dy"], self.adapter, o["da"], o["db"], o["ws"],
                           accumulate=accumulate, stream=stream)

    def check(self, o):
        x, dy, w = self.x.double(), self.dy.double(), self.w.double()
        ref = {"y": x @ w.t(), "dx": dy @ w}
        mag = {"y": x.abs() @ w.abs().t(), "dx": dy.abs() @ w.abs()}
        err = {k: (c + 3 * self.rank + 64) * U * mag[k] for k, c in (("y", self.K), ("dx", self.N))}
        z = lambda t: torch.zeros(t.shape, dtype=torch.float64, device="cuda")
        ref.update(da=z(o["da"]), db=z(o["db"]))
        err.update(da=z(o["da"]), db=z(o["db"]))
        for g in range(self.G):
            rows = torch.nonzero(self.adapter == g)[:, 0]
            if rows.numel() == 0:
                continue
            sc = self.scale[g].double()
            a, b, xr, dr = self.a[g].double(), self.b[g].double(), x[rows], dy[rows]
            s, t = sc * (xr @ a.t()), sc * (dr @ b)
            es = (self.K + 64) * U * sc * (xr.abs() @ a.abs().t()) + U * s.abs()
            et = (self.N + 64) * U * sc * (dr.abs() @ b.abs()) + U * t.abs()
            n = 3 * rows.numel() + 64
            ref["y"][rows] += s @ b.t()
            ref["dx"][rows] += t @ a
            extra = 2.0 ** -17 + (self.K + 3 * self.rank + 64) * U
            err["y"][rows] += es @ b.abs().t() + extra * (s.abs() @ b.abs().t())
            extra = 2.0 ** -17 + (self.N + 3 * self.rank + 64) * U
            err["dx"][rows] += et @ a.abs() + extra * (t.abs() @ a.abs())
            ref["da"][g], ref["db"][g] = t.t() @ xr, dr.t() @ s
            err["da"][g] = et.t() @ xr.abs() + n * U * (t.abs().t() @ xr.abs())
            err["db"][g] = dr.abs().t() @ es + n * U * (dr.abs().t() @ s.abs())
        for k in ("y", "dx", "da", "db"):
            if o[k].numel() == 0:
                continue
            d = (o[k].double() - ref[k]).abs()
            bound = err[k] + (2.0 ** -8 * ref[k].abs() if k in ("y", "dx") else 0) + 1e-30
            assert bool((d <= bound).all()), (k, (d / bound).max().item(), torch.nonzero(~(d <= bound))[:3].tolist())
            if k in ("da", "db") and self.R:
                rms = (d.pow(2).mean() / ref[k].pow(2).mean().clamp_min(1e-30)).sqrt().item()
                assert rms <= 2.0 ** -18 or bool((ref[k] == 0).all()), (k, rms)


CASES = [
    # R, N, K, G, rank, order
    (1, 64, 64, 1, 8, "mixed"), (1, 128, 320, 5, 16, 4), (3, 192, 64, 2, 8, "mixed"), (13, 512, 1024, 32, 16, "mixed"),
    (16, 256, 128, 3, 24, "runs"), (17, 64, 256, 4, 32, "mixed"), (33, 320, 192, 40, 40, "mixed"),
    (64, 1024, 512, 64, 64, "mixed"), (64, 128, 128, 2, 128, "runs"), (65, 128, 192, 3, 8, "mixed"),
    (100, 64, 64, 7, 72, "mixed"), (255, 320, 448, 300, 8, "mixed"), (300, 512, 256, 48, 32, "mixed"),
    (513, 256, 320, 4, 128, "runs"), (700, 832, 576, 8, 16, "runs"), (1025, 384, 512, 2, 56, "mixed"),
    (40, 256, 256, 4, 16, -1), (300, 256, 256, 4, 16, -1), (300, 128, 256, 1, 16, 0), (9000, 128, 64, 3, 8, "mixed"),
    # 128 x 64, 128 x 128 and 256 x 256 tiles, of y and of dx; few and many adapters in a tile
    (1001, 2048, 192, 3, 8, "mixed"), (290, 4160, 128, 48, 32, "mixed"), (1001, 192, 2048, 3, 24, "mixed"),
    (290, 128, 4160, 48, 8, "mixed"), (2048, 2048, 64, 5, 16, "mixed"), (2040, 2112, 64, 40, 8, "mixed"),
    (2048, 64, 2048, 8, 64, "mixed"), (2040, 128, 2112, 40, 16, "mixed"), (4096, 4096, 64, 3, 16, "runs"),
    (4090, 4160, 64, 24, 8, "mixed"), (4096, 64, 4096, 5, 128, "runs"), (4090, 64, 4160, 24, 8, "mixed"),
    # 9 to 64 rows by whole lines: every count of row tiles, one and many adapters
    (8, 256, 704, 3, 128, "mixed"), (9, 64, 64, 4, 8, "mixed"), (24, 128, 1088, 30, 16, "mixed"),
    (32, 192, 4096, 2, 16, "runs"), (47, 64, 2048, 9, 88, "mixed"), (64, 192, 4160, 64, 16, "mixed"),
]


@gpu
@pytest.mark.parametrize("R,N,K,G,rank,order", CASES)
def test_lora(R, N, K, G, rank, order):
    c = Case(R, N, K, G, rank, order)
    o = c.buffers()
    c.call(o)
    c.check(o)
    p = c.buffers()
    c.call(p)
    for k in ("y", "dx", "da", "db", "low", "low_dy"):
        assert torch.equal(o[k], p[k]), f"{k}: run-to-run bits differ"


@gpu
@pytest.mark.parametrize("R,N,K,G,order", [
    (7, 128, 256, 4, "mixed"), (50, 128, 256, 4, "mixed"), (100, 192, 320, 4, "mixed"), (130, 320, 256, 60, "mixed"),
    (2048, 2048, 64, 4, "mixed"), (2048, 64, 2048, 4, "mixed"), (2048, 2048, 64, 40, "mixed"),
    (2048, 64, 2048, 40, "mixed"), (4096, 4096, 64, 4, "mixed"), (4096, 64, 4096, 4, "mixed"),
])
def test_lora_nonfinite_stays_with_its_adapter(R, N, K, G, order):
    """An adapter's infinities and NaN, and a row's, reach the outputs that the
    formulas give them to and no other."""
    c = Case(R, N, K, G, 16, order)
    c.adapter[3] = -1
    c.adapter[1], c.adapter[2] = 1, 2
    o = c.buffers()
    c.call(o)
    c.b[1, 5, 3], c.b[1, 40, 0], c.b[1, N - 1, 15] = float("inf"), float("nan"), float("-inf")
    c.a[2, 4, 7], c.a[2, 15, K - 1] = float("nan"), float("inf")
    p = c.buffers()
    c.call(p)
    one, two = c.adapter == 1, c.adapter == 2
    # y: B's element reaches its feature; A's reach s, and with it the whole row
    bad = torch.zeros(R, N, dtype=torch.bool, device="cuda")
    for f in (5, 40, N - 1):
        bad[:, f] = one
    bad |= two[:, None]
    assert torch.equal(~p["y"].isfinite(), bad) and torch.equal(p["y"][~bad], o["y"][~bad])
    bad = torch.zeros(R, K, dtype=torch.bool, device="cuda")
    bad[:, 7] = bad[:, K - 1] = two
    bad |= one[:, None]
    assert torch.equal(~p["dx"].isfinite(), bad) and torch.equal(p["dx"][~bad], o["dx"][~bad])
    # the gradients: t of adapter 1's rows and s of adapter 2's are not finite
    for k, g in (("da", 1), ("db", 2)):
        rest = [i for i in range(G) if i != g]
        assert not p[k][g].isfinite().all() and torch.equal(p[k][rest], o[k][rest])
    # a row's own infinity: its y, and its adapter's dA
    c = Case(R, N, K, G, 16, order)
    c.adapter[1] = 1
    o = c.buffers()
    c.call(o)
    c.x[1, 3] = float("inf")
    p = c.buffers()
    c.call(p)
    rows = [i for i in range(R) if i != 1]
    rest = [i for i in range(G) if i != 1]
    assert not p["y"][1].isfinite().any() and torch.equal(p["y"][rows], o["y"][rows])
    assert torch.equal(p["dx"], o["dx"])
    assert torch.equal(p["da"][rest], o["da"][rest]) and torch.equal(p["db"][rest], o["db"][rest])


@gpu
def test_lora_ids_outside_mean_no_adapter():
    c = Case(70, 128, 128, 3, 16)
    o, p = c.buffers(), c.buffers()
    c.adapter[::5] = -1
    c.call(o)
    c.adapter[::10] = 3
    c.adapter[5::10] = -2 ** 31
    c.call(p)
    for k in ("y", "dx", "da", "db"):
        assert torch.equal(o[k], p[k])
    c.adapter[:] = 2 ** 31 - 1
    c.call(p)
    assert (p["da"] == 0).all() and (p["db"] == 0).all() and (p["low"] == 0).all()
    c.check(p)


@gpu
def test_lora_no_rows():
    c = Case(0, 128, 64, 2, 8)
    o = c.buffers()
    c.call(o)
    assert (o["da"] == 0).all() and (o["db"] == 0).all()


@gpu
@pytest.mark.parametrize("R,G", [(50, 3), (900, 2)])
def test_lora_accumulate_adds_the_finished_sum(R, G):
    c = Case(R, 192, 128, G, 24)
    c.adapter[c.adapter == 1] = 0        # adapter 1 has no rows
    o, p = c.buffers(), c.buffers()
    c.call(o)
    for k in ("da", "db"):
        p[k].copy_(torch.randn_like(p[k]))
    p["da"][1] = -0.0
    want = {k: p[k] + o[k] for k in ("da", "db")}
    c.call(p, accumulate=True)
    for k in ("da", "db"):
        assert torch.equal(p[k].view(torch.int32), want[k].view(torch.int32)), k
    assert not torch.signbit(p["da"][1]).any()


@gpu
def test_lora_rows_are_independent():
    """A row's output does not depend on its place, its neighbours or a NaN in
    another row, within one kernel (the streaming one, and the tiles)."""
    for R in (40, 400):
        c = Case(R, 256, 192, 6, 16)
        o = c.buffers()
        c.call(o)
        perm = torch.randperm(R, device="cuda")
        d = Case(R, 256, 192, 6, 16)
        d.x, d.dy, d.adapter = c.x[perm].contiguous(), c.dy[perm].contiguous(), c.adapter[perm].contiguous()
        p = d.buffers()
        d.call(p)
        assert torch.equal(p["y"], o["y"][perm]) and torch.equal(p["dx"], o["dx"][perm])
        c.x[7] = float("nan")
        c.dy[9] = float("inf")
        q = c.buffers()
        c.call(q)
        keep = torch.arange(R, device="cuda")
        assert torch.equal(q["y"][keep != 7], o["y"][keep != 7])
        assert torch.equal(q["dx"][keep != 9], o["dx"][keep != 9])
        assert q["y"][7].isnan().all()


@gpu
def test_lora_equals_the_plain_projection_without_adapters():
    """No adapter anywhere: the tiles give moe_grouped_forward's bits."""
    c = Case(300, 256, 256, 2, 8, -1)
    o = c.buffers()
    c.call(o)
    y, dx = torch.empty_like(o["y"]), torch.empty_like(o["dx"])
    off = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    moe.moe_grouped_forward(c.x, c.w[None].contiguous(), off, y)
    moe.moe_grouped_dgrad(c.dy, c.w[None].contiguous(), off, dx)
    assert torch.equal(o["y"], y) and torch.equal(o["dx"], dx)


@gpu
def test_lora_gradients_are_difference_quotients():
    """The calls' own gradients against differences of the formula in 64 bits
    (the loss is linear in every argument, so any step is exact)."""
    c = Case(6, 64, 64, 2, 8)
    o = c.buffers()
    c.call(o)

    def loss(x, a, b):
        y = x @ c.w.double().t()
        for r in range(6):
            g = int(c.adapter[r])
            if g >= 0:
                y[r] += c.scale[g].double() * (b[g] @ (a[g] @ x[r]))
        return (y * c.dy.double()).sum()

    x, a, b = c.x.double(), c.a.double(), c.b.double()
    base = loss(x, a, b)
    for name, t, grad in (("x", x, o["dx"]), ("a", a, o["da"]), ("b", b, o["db"])):
        flat = t.view(-1)
        for i in range(0, flat.numel(), flat.numel() // 37):
            keep = flat[i].item()
            flat[i] = keep + 1.0
            d = (loss(x, a, b) - base).item()
            flat[i] = keep
            got = grad.reshape(-1)[i].double().item()
            assert abs(got - d) <= 2.0 ** -8 * abs(d) + 2.0 ** -8 * 0.05, (name, i, got, d)


@gpu
@pytest.mark.parametrize("R", [21, 300])
def test_lora_graph_replays_and_streams(R):
    c = Case(R, 256, 192, 5, 16)
    ref, o = c.buffers(), c.buffers()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.call(o, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    c.call(ref)
    keys = ("y", "dx", "da", "db")
    assert all(torch.equal(ref[k], o[k]) for k in keys)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(o)
    for i in range(4):
        c.x.copy_(torch.randn(R, 192, device="cuda"))
        c.adapter.copy_(torch.randint(-1, 5, (R,), device="cuda", dtype=torch.int32))
        c.call(ref)
        for k in keys:
            o[k].fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(ref[k], o[k]) for k in keys), i


@gpu
def test_lora_projection_then_layer():
    """As used: a projection with adapters in front of a MoE layer for a few
    tokens, both on one stream."""
    c = Case(12, 256, 128, 4, 8)
    o = c.buffers()
    c.call(o)
    c.check(o)
    r = moe.make_router(8, 2)
    plan = moe.moe_layer_plan_init(moe.make_layer_problem(12, 256, 128, r))
    ws = moe.allocate_layer_workspace(plan)
    g = torch.Generator(device="cuda").manual_seed(5)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").mul(0.06).bfloat16()
    wr, w1, w2 = rn(8, 256), rn(8, 256, 256), rn(8, 256, 128)
    out = torch.empty(12, 256, dtype=torch.bfloat16, device="cuda")
    ids, wt = torch.empty(12, 2, dtype=torch.int32, device="cuda"), torch.empty(12, 2, device="cuda")
    moe.moe_layer_apply(plan, o["y"], wr, w1, w2, out, ids, wt, ws)
    moe.check_layer_status(plan, ws)
    x = o["y"].double()
    want = torch.zeros(12, 256, dtype=torch.float64, device="cuda")
    for t in range(12):
        for j in range(2):
            e = int(ids[t, j])
            h = w1[e].double() @ x[t]
            want[t] += wt[t, j].double() * (w2[e].double() @ (h[:128] * torch.sigmoid(h[:128]) * h[128:]))
    assert ((out.double() - want).pow(2).mean() / want.pow(2).mean()).sqrt() <= 1.5 * 2 ** 0.5 * 2.0 ** -8 / 3 ** 0.5


@gpu
def test_lora_and_router_training_step():
    """As used in training: logits from an adapted projection, the router's
    weights, their gradient back through the router into the adapters; eager
    and captured, every stage against its formula at the values it was given."""
    from operator_refs import route_backward, route_topk

    c = Case(200, 64, 128, 3, 8)
    r = moe.make_router(64, 4, moe.ROUTE_SIGMOID, renormalize=True, scale=2.0)
    dw = torch.randn(200, 4, device="cuda")

    def buffers():
        o = c.buffers()
        o["ids"] = torch.full((200, 4), 99, dtype=torch.int32, device="cuda")
        o["wt"] = torch.full((200, 4), float("nan"), device="cuda")
        o["dl"] = torch.full((200, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        return o

    def step(o):
        moe.moe_lora_forward(c.x, c.w, c.a, c.b, c.scale, c.adapter, o["y"], o["low"])
        moe.moe_route_topk(r, o["y"], o["ids"], o["wt"])
        moe.moe_route_topk_backward(r, o["y"], o["ids"], dw, o["dl"])
        moe.moe_lora_dgrad(o["dl"], c.w, c.a, c.b, c.scale, c.adapter, o["dx"], o["low_dy"])
        moe.moe_lora_wgrad(c.x, o["dl"], o["low"], o["low_dy"], c.adapter, o["da"], o["db"], o["ws"])

    ref, o = buffers(), buffers()
    step(o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(o)
    keys = ("y", "ids", "wt", "dl", "dx", "da", "db")
    for i in range(3):
        c.x.copy_(torch.randn(200, 128, device="cuda"))
        c.adapter.copy_(torch.randint(-1, 3, (200,), device="cuda", dtype=torch.int32))
        step(ref)
        for k in keys:
            o[k].fill_(99)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(ref[k], o[k]) for k in keys), i
    logits = o["y"].float().cpu().numpy()
    ids, wt = route_topk(logits, 4, "sigmoid", scale=2.0)
    assert np.array_equal(o["ids"].cpu().numpy(), ids)
    assert np.all(np.abs(o["wt"].cpu().numpy() - wt) <= 2.0 ** -23 * np.abs(wt))
    dl, mag = route_backward(logits, ids, dw.cpu().numpy(), "sigmoid", scale=2.0)
    got = o["dl"].double().cpu().numpy()
    assert np.all(np.abs(got - dl) <= 2.0 ** -8 * np.abs(dl) + 2.0 ** -23 * mag + 1e-37)
    c.dy = o["dl"]
    c.check(o)


@gpu
def test_lora_workspaces_and_ids_in_succession():
    """One workspace and one narrow-product buffer for problems of different
    sizes one after another, with nothing cleared in between."""
    sizes = [(9000, 128, 64, 3, 8), (33, 320, 192, 40, 40), (300, 64, 448, 4096, 8), (1, 64, 64, 1, 128)]
    cases = [Case(*z) for z in sizes]
    ws = torch.full((max(moe.moe_lora_ws_bytes(*z) for z in sizes),), 0xff, dtype=torch.uint8, device="cuda")
    low = [torch.full((max(moe.moe_lora_low_bytes(*z) for z in sizes),), 0xff, dtype=torch.uint8, device="cuda")
           for _ in range(2)]
    for c in cases + cases[::-1]:
        o = c.buffers()
        o["low"], o["low_dy"], o["ws"] = low[0], low[1], ws
        c.call(o)
        c.check(o)


@gpu
@pytest.mark.parametrize("R,G,N,K", [(5, 3, 128, 64), (40, 40, 64, 128), (300, 3, 256, 320), (300, 60, 320, 256),
                                     (2048, 4, 2048, 64), (2048, 4, 64, 2048), (2048, 40, 2048, 64), (4096, 2, 4096, 64),
                                     (4096, 2, 64, 4096)])
def test_lora_narrow_products_near_the_largest_float(R, G, N, K):
    """s and t up to the largest float32 are finite, and what is made of them
    is: y = W x + B s with s near 2^128 and B = 2^-20, the same for dx, and the
    gradients with 2^-20 on their other side.  One product per sum, so y and dx
    are off by 2^-17 (two pieces) and half a bf16 step, dA and dB by the 3
    pieces' sums over the adapter's rows."""
    c = Case(R, N, K, G, 8, "mixed", seed=R)
    top = float(torch.finfo(torch.float32).max)
    c.scale[:] = top
    c.scale[1:] = -3.397e38
    c.scale[2:] = 3.4e38
    small = 2.0 ** -20

    def unit(t):
        t.zero_()
        t[..., 0] = 1.0

    for side in ("y", "dx"):
        for t in (c.a, c.b):
            t.zero_()
        c.a[:, 0, 0] = 1.0 if side == "y" else small
        c.b[:, 0, 0] = small if side == "y" else 1.0
        unit(c.x)
        unit(c.dy)
        if side == "y":
            c.dy.mul_(small)
        else:
            c.x.mul_(small)
        o = c.buffers()
        c.call(o)
        on = c.adapter >= 0
        s = torch.where(on, c.scale.double()[c.adapter.clamp_min(0).long()], 0.0)   # s of side y, t of side dx
        got = o[side].double()
        want = s * small
        bound = (2.0 ** -8 + 2.0 ** -17 + 256 * U) * want.abs() + 16.0              # |W| < 16
        assert bool(((got[:, 0] - want).abs() <= bound).all()) and bool(got.isfinite().all())
        # dB[g, 0, 0] = sum dy s (side y), dA[g, 0, 0] = sum t x (side dx); the other one's own product is small^2
        k = "db" if side == "y" else "da"
        for g in range(G):
            n = int((c.adapter == g).sum())
            want = n * c.scale[g].double().item() * small
            assert abs(o[k][g, 0, 0].double().item() - want) <= (3 * n + 64) * U * abs(want), (side, g)
        assert bool(o["da"].isfinite().all()) and bool(o["db"].isfinite().all())


@gpu
@pytest.mark.parametrize("R,N,K,G,rank", [((1 << 24) - 1, 64, 64, 5, 8), (5, 32704, 32704, 3, 8), (300, 32704, 32704, 40, 8),
                                          (32768, 32704, 32704, 4, 16), (200, 64, (1 << 22) - 64, 3, 40),
                                          (40, (1 << 20) - 64, 64, 7, 128), (130, 192, 64, 4096, 128)])
def test_lora_largest_sizes(R, N, K, G, rank):
    """Rows, W and the adapters near 2^31 bytes, offsets past 2^30: rows from all
    over, and the adapters' gradients by their root mean square.  A float32 sum of
    n terms of random sign, one by one, has partial sums that grow like sqrt(i)
    and is off by at most half a step of each: 2^-24 sqrt(sum of i / n) =
    2^-24 sqrt(n / 2) of its size.  For s or t, C / 4 terms to a wave; for dA and
    dB three pieces of every row; and 2^-23 for the pieces and the last sums."""
    g = torch.Generator(device="cuda").manual_seed(R)

    def rn(*s, std=1.0):
        t = torch.empty(*s, dtype=torch.bfloat16, device="cuda")
        for i in range(0, t.numel(), 1 << 28):
            t.view(-1)[i:i + (1 << 28)].normal_(0.0, std, generator=g)
        return t

    c = Case(1, 64, 64, 1, 8)
    c.R, c.N, c.K, c.G, c.rank = R, N, K, G, rank
    c.x, c.dy, c.w, c.a, c.b = rn(R, K), rn(R, N), rn(N, K, std=K ** -0.5), rn(G, rank, K, std=K ** -0.5), rn(G, N, rank, std=rank ** -0.5)
    c.scale = 0.5 + torch.rand(G, generator=g, device="cuda")
    c.adapter = torch.randint(-1, G, (R,), generator=g, device="cuda", dtype=torch.int32)
    o = c.buffers()
    c.call(o)
    at = torch.unique(torch.cat([torch.arange(2, device="cuda"), torch.arange(R - 3, R, device="cuda"),
                                 torch.randint(0, R, (40,), generator=g, device="cuda")]))

    def by_rows(rows, m, t):   # rows [n, C] times m's rows (t: columns), m in pieces
        v, n = rows.double(), (1 << 27) // m.shape[1]
        if t:
            out = torch.zeros(v.shape[0], m.shape[1], dtype=torch.float64, device="cuda")
            for i in range(0, m.shape[0], n):
                out += v[:, i:i + n] @ m[i:i + n].double()
            return out
        return torch.cat([v @ m[i:i + n].double().t() for i in range(0, m.shape[0], n)], 1)

    y, dx = by_rows(c.x[at], c.w, False), by_rows(c.dy[at], c.w, True)
    for i, r in enumerate(at.tolist()):
        q = int(c.adapter[r])
        if q >= 0:
            y[i] += c.scale[q].double() * (c.b[q].double() @ (c.a[q].double() @ c.x[r].double()))
            dx[i] += c.scale[q].double() * ((c.dy[r].double() @ c.b[q].double()) @ c.a[q].double())
    for got, want, n in ((o["y"], y, K), (o["dx"], dx, N)):
        d = (got[at].double() - want).abs()
        # n terms of random sign, each of size / sqrt(n): U n of their magnitudes is U sqrt(n) of the size
        size = want.pow(2).mean().sqrt()
        assert bool((d <= 2.0 ** -8 * want.abs() + (2.0 ** -15 + 4 * U * n ** 0.5) * size).all()), d.max().item()
        assert bool(got.isfinite().all())
    for q in range(0, G, max(G // 5, 1)):
        rows = torch.nonzero(c.adapter == q)[:, 0]
        da, db = (torch.zeros(t.shape[1:], dtype=torch.float64, device="cuda") for t in (o["da"], o["db"]))
        step = max(1, (1 << 27) // (N + K))
        for i in range(0, rows.numel(), step):
            k = rows[i:i + step]
            x, dy = c.x[k].double(), c.dy[k].double()
            s, t = c.scale[q].double() * (x @ c.a[q].double().t()), c.scale[q].double() * (dy @ c.b[q].double())
            da += t.t() @ x
            db += dy.t() @ s
        for got, want, C in ((o["da"][q], da, N), (o["db"][q], db, K)):
            if rows.numel() == 0:
                assert (got == 0).all()
                continue
            rms = ((got.double() - want).pow(2).mean() / want.pow(2).mean()).sqrt().item()
            assert rms <= 2.0 ** -24 * ((C / 8) ** 0.5 + (3 * rows.numel() / 2) ** 0.5 + 2), (q, rms)

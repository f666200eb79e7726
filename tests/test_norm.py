"""The norms around a block (moe_block_norm, moe_block_norm_backward) against
64 bits.  Bounds: the errors of float32 arithmetic as block_refs derives them,
and half a step of each output's type."""
import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_expert_align_amd as moe
from block_refs import norm_backward, norm_forward

gpu = pytest.mark.gpu
GATE = {"none": moe.GATE_NONE, "channel": moe.GATE_CHANNEL, "token": moe.GATE_TOKEN}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


# ------------------------------------------------------------- on the host --

def test_refusals():
    lib, a = moe.load_library(), 4096

    def problem(**kw):
        p = moe.make_norm_problem(4, 64)
        for k, v in kw.items():
            setattr(p, k, v)
        return p

    def fwd(p=None, x=a, block=a, w_post=a, gate=None, w_pre=a, x_out=a, h=a, **kw):
        return lib.moe_block_norm(ctypes.byref(p or problem(**kw)), x, block, w_post, gate, w_pre, x_out, h, None)

    def bwd(p=None, x=a, block=a, w_post=a, gate=None, w_pre=a, dx_out=a, dh=a, dx=a, db=a, dwp=a, dg=None, dwr=a,
            acc=0, ws=a, **kw):
        return lib.moe_block_norm_backward(ctypes.byref(p or problem(**kw)), x, block, w_post, gate, w_pre, dx_out, dh,
                                           dx, db, dwp, dg, dwr, acc, ws, None)

    inf, nan = float("inf"), float("nan")
    for kw in (dict(M=-1), dict(M=1 << 31), dict(K=0), dict(x_dtype=2), dict(w_dtype=-1), dict(gate_kind=3),
               dict(eps=0.0), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(res_scale=inf), dict(res_scale=nan),
               dict(x=None), dict(x=a + 8), dict(block=a + 2), dict(w_post=a + 4), dict(gate=a),
               dict(gate_kind=moe.GATE_CHANNEL), dict(gate_kind=moe.GATE_CHANNEL, gate=a + 4),
               dict(gate_kind=moe.GATE_TOKEN, gate=a + 2), dict(w_pre=a + 8)):
        assert fwd(**kw) == moe.MOE_EINVAL, kw
        assert bwd(**kw) == moe.MOE_EINVAL, kw
    for kw in (dict(K=60), dict(K=16392)):
        assert fwd(**kw) == moe.MOE_EUNSUPPORTED and bwd(**kw) == moe.MOE_EUNSUPPORTED
        assert lib.moe_block_norm_ws_bytes(ctypes.byref(problem(**kw))) == -1
    for kw in (dict(x_out=None), dict(x_out=a + 8), dict(h=None), dict(h=a + 2), dict(w_pre=None),
               dict(block=None), dict(block=None, x_out=None), dict(block=None, x_out=None, w_post=None, w_pre=None, h=None)):
        assert fwd(**kw) == moe.MOE_EINVAL, kw
    for kw in (dict(dh=None), dict(w_pre=None, dwr=None), dict(dx=None), dict(dx=a + 8), dict(db=None),
               dict(block=None, w_post=None, dwp=None), dict(dx_out=a + 4), dict(dh=a + 2),
               dict(w_pre=None, dh=None, dx_out=None, dwr=None), dict(w_post=None), dict(dg=a), dict(dwp=a + 4),
               dict(dwr=a + 8), dict(acc=2), dict(ws=None), dict(ws=a + 8)):
        assert bwd(**kw) == moe.MOE_EINVAL, kw
    assert fwd(M=0, x=None, block=None, x_out=None, h=None) == moe.MOE_OK      # nothing to do
    with pytest.raises(ValueError, match="x_dtype"):
        moe.make_norm_problem(4, 64, x_dtype=torch.float16)
    with pytest.raises(ValueError, match="device tensor|cuda"):
        moe.moe_block_norm(moe.make_norm_problem(4, 64), torch.zeros(4, 64, dtype=torch.bfloat16))


def test_reference_gradients_are_difference_quotients():
    rng = np.random.default_rng(0)
    M, K, eps, a = 3, 5, 1e-3, 0.7
    x0, b, wp, wr = (rng.normal(size=s) for s in ((M, K), (M, K), K, K))
    dx_out, dh = rng.normal(size=(M, K)), rng.normal(size=(M, K))
    for kind in ("none", "channel", "token"):
        g = {"none": np.ones((1, 1)), "channel": rng.normal(size=(1, K)), "token": rng.normal(size=(M, 1))}[kind]

        def f(x0, b, wp, g, wr):
            y, _, h, _ = norm_forward(x0, b, wp, g, wr, eps, a)
            return (y * dx_out).sum() + (h * dh).sum()

        args = [x0, b, wp, g, wr]
        y = norm_forward(*args, eps, a)[0]
        d = norm_backward(y, b, wp, g, wr, dx_out, dh, eps, a)
        want = {0: "dx", 1: "dblock", 2: "dw_post", 4: "dw_pre"}
        if kind != "none":
            want[3] = "dgate_" + kind
        for i, name in want.items():
            flat = args[i].reshape(-1)
            for j in range(flat.size):
                q = []
                for h in (1e-6, -1e-6):
                    p = flat.copy()
                    p[j] += h
                    q.append(f(*[p.reshape(args[i].shape) if k == i else v for k, v in enumerate(args)]))
                assert abs((q[0] - q[1]) / 2e-6 - d[name][0].reshape(-1)[j]) < 1e-7, (kind, name)


# ---------------------------------------------------------------------- GPU --

def operands(M, K, xt, wt, gate, post, pre, seed, block=True, spread=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rnd(*s, t=torch.float32, k=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * k).to(t)
    o = dict(x=rnd(M, K, t=xt, k=spread), block=rnd(M, K, t=torch.bfloat16, k=0.3) if block else None,
             w_post=(1 + rnd(K, k=0.3)).to(wt) if post else None, w_pre=(1 + rnd(K, k=0.3)).to(wt) if pre else None,
             gate={"none": None, "channel": rnd(K, t=wt), "token": rnd(M)}[gate],
             dx_out=rnd(M, K, t=xt), dh=rnd(M, K, t=torch.bfloat16) if pre else None)
    return o


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def gate64(o, kind):
    g = f64(o["gate"])
    return np.ones((1, 1)) if kind == "none" else g[None, :] if kind == "channel" else g[:, None]


def guarded(shape, dtype):
    """A buffer with one more row, and the part of it that is to be written."""
    n = int(np.prod(shape))
    buf = torch.full((n + 64,), 3.0, dtype=dtype, device="cuda")
    return buf, buf[:n].view(shape)


def within(got, ref, err, half, what=""):
    got = f64(got)
    bound = err + half * (np.abs(ref) + err) + 1e-37
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, np.argwhere(bad)[:4], (np.abs(got - ref) - bound).max())


def check(M, K, xt=torch.bfloat16, wt=torch.float32, gate="none", post=True, pre=True, block=True, scale=1.0, eps=1e-6,
          seed=0, with_dx=True, o=None, sums=True):
    o = o or operands(M, K, xt, wt, gate, post, pre, seed, block)
    p = moe.make_norm_problem(M, K, xt, wt, GATE[gate], eps, scale)
    bx, x_out = guarded((M, K), xt)
    bh, h = guarded((M, K), torch.bfloat16)
    moe.moe_block_norm(p, o["x"], x_out if block else None, o["block"], o["w_post"], o["gate"], o["w_pre"],
                       h if pre else None)
    y, ey, rh, eh = norm_forward(f64(o["x"]), f64(o["block"]), f64(o["w_post"]), gate64(o, gate), f64(o["w_pre"]), p.eps,
                                 p.res_scale)
    assert (bx[M * K:] == 3).all() and (bh[M * K:] == 3).all()
    if block:
        within(x_out, y, ey, HALF[xt], "x_out")
    if pre:
        within(h, rh, eh, 2.0 ** -8, "h")
    # backward at the stored x_out (any other would do)
    stored = x_out if block else o["x"]
    dx_out = o["dx_out"] if with_dx else None
    bufs = {n: guarded(s, t) for n, s, t in (("dx", (M, K), xt), ("dblock", (M, K), torch.bfloat16),
                                             ("dw_post", (K,), torch.float32), ("dw_pre", (K,), torch.float32),
                                             ("dgate", (M if gate == "token" else K,), torch.float32))}
    given = {n: v[1] for n, v in bufs.items()}
    wanted = dict(dblock=block, dw_post=post and block and sums, dw_pre=pre and sums, dgate=gate != "none" and sums)
    ws = moe.allocate_norm_workspace(p).fill_(255)
    moe.moe_block_norm_backward(p, stored, dx_out, given["dx"], ws, o["block"], o["w_post"], o["gate"], o["w_pre"],
                                o["dh"], **{n: given[n] if w else None for n, w in wanted.items()})
    ref = norm_backward(f64(stored), f64(o["block"]), f64(o["w_post"]), gate64(o, gate), f64(o["w_pre"]),
                        f64(dx_out) if with_dx else np.zeros((M, K)), f64(o["dh"]), p.eps, p.res_scale)
    within(given["dx"], *ref["dx"], HALF[xt], "dx")
    if block:
        within(given["dblock"], *ref["dblock"], 2.0 ** -8, "dblock")
    for n in ("dw_post", "dw_pre"):
        if wanted[n]:
            within(given[n], *ref[n], 2.0 ** -24, n)
    if wanted["dgate"]:
        within(given["dgate"], *ref["dgate_" + gate], 2.0 ** -24, "dgate")
    for n, (buf, view) in bufs.items():
        assert (buf[view.numel():] == 3).all(), n
        if not wanted.get(n, True):
            assert (buf == 3).all(), n


@gpu
@pytest.mark.parametrize("K", [8, 64, 504, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 6144, 8192, 8200, 16384])
@pytest.mark.parametrize("M", [1, 3, 37])
def test_sizes(M, K):
    check(M, K, gate="channel", scale=0.5, seed=K)
    check(M, K, torch.float32, torch.bfloat16, gate="token", seed=K + 1)


@gpu
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16])
def test_forms(gate, post, pre, xt):
    for K in (256, 2560):
        check(21, K, xt, torch.bfloat16 if pre else torch.float32, gate, post, pre, scale=0.75, eps=1e-5, seed=K)


@gpu
@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [256, 2560])
def test_first_norm(xt, K):
    check(19, K, xt, post=False, block=False, seed=4)
    check(19, K, xt, post=False, block=False, seed=5, with_dx=False)


@gpu
def test_no_gradient_from_behind_and_no_sums():
    check(9, 512, gate="channel", with_dx=False)
    check(9, 512, gate="channel", sums=False)
    check(9, 2560, gate="token", sums=False)


@gpu
@pytest.mark.parametrize("M,K", [(2500, 256), (1100, 2048), (700, 4096), (600, 6144)])
def test_many_rows_to_a_workgroup(M, K):
    check(M, K, gate="channel", seed=M)
    check(M, K, torch.float32, gate="token", post=False, seed=M + 1)


@gpu
def test_rows_of_zeros_and_of_small_and_large_values():
    for K in (256, 2560):
        o = operands(8, K, torch.float32, torch.float32, "channel", True, True, 3)
        o["x"][0], o["block"][0] = 0, 0
        o["x"][1] *= 1e-12
        o["block"][1] *= 1e-12
        o["x"][2] *= 1e15
        o["block"][3] *= 1e15
        o["block"][4] = 0
        o["dh"][5] = 0
        check(8, K, torch.float32, gate="channel", o=o)


@gpu
@pytest.mark.parametrize("K", [256, 2560])
def test_nan_and_infinity_stay_in_their_row(K):
    o = operands(6, K, torch.bfloat16, torch.float32, "channel", True, True, 7)
    clean = {k: None if v is None else v.clone() for k, v in o.items()}
    o["x"][1, 5] = float("nan")
    o["block"][3, 7] = float("inf")
    outs = []
    for q in (clean, o):
        p = moe.make_norm_problem(6, K, gate_kind=moe.GATE_CHANNEL)
        y, h = torch.empty_like(q["x"]), torch.empty_like(q["x"])
        moe.moe_block_norm(p, q["x"], y, q["block"], q["w_post"], q["gate"], q["w_pre"], h)
        dx, db = torch.empty_like(y), torch.empty_like(y)
        moe.moe_block_norm_backward(p, q["x"], q["dx_out"], dx, moe.allocate_norm_workspace(p), q["block"], q["w_post"],
                                    q["gate"], q["w_pre"], q["dh"], db)
        outs.append((y, h, dx, db))
    keep = [0, 2, 4, 5]
    for a, b in zip(*outs):
        assert torch.equal(a[keep], b[keep])
    y, h, dx, db = outs[1]
    assert h[1].isnan().all() and y[1, 5].isnan() and dx[1].isnan().all() and db[1].isnan().all()
    assert y[3, 7].isnan() and db[3, 7].isnan()


@gpu
def test_in_place():
    """x_out may be x, dx may be dx_out."""
    for K in (256, 2560):
        o = operands(70, K, torch.bfloat16, torch.float32, "channel", True, True, 8)
        p = moe.make_norm_problem(70, K, gate_kind=moe.GATE_CHANNEL, res_scale=0.5)
        y, h, h2 = torch.empty_like(o["x"]), torch.empty_like(o["x"]), torch.empty_like(o["x"])
        moe.moe_block_norm(p, o["x"], y, o["block"], o["w_post"], o["gate"], o["w_pre"], h)
        dx, db, db2 = torch.empty_like(y), torch.empty_like(y), torch.empty_like(y)
        ws = moe.allocate_norm_workspace(p)
        args = (o["block"], o["w_post"], o["gate"], o["w_pre"], o["dh"])
        moe.moe_block_norm_backward(p, y, o["dx_out"], dx, ws, *args, db)
        x = o["x"].clone()
        moe.moe_block_norm(p, x, x, o["block"], o["w_post"], o["gate"], o["w_pre"], h2)
        assert torch.equal(x, y) and torch.equal(h, h2)
        d = o["dx_out"].clone()
        moe.moe_block_norm_backward(p, y, d, d, ws, *args, db2)
        assert torch.equal(d, dx) and torch.equal(db, db2)


@gpu
@pytest.mark.parametrize("M", [0, 5, 900])
def test_accumulate_adds_the_finished_sums(M):
    K = 520
    o = operands(M, K, torch.bfloat16, torch.float32, "channel", True, True, 9)
    p = moe.make_norm_problem(M, K, gate_kind=moe.GATE_CHANNEL)
    ws = moe.allocate_norm_workspace(p)
    sums = []
    for acc in (False, True):
        s = [torch.full((K,), -0.0 if M == 0 else 2.5, device="cuda") for _ in range(3)]
        dx, db = torch.empty_like(o["x"]), torch.empty_like(o["x"])
        moe.moe_block_norm_backward(p, o["x"], o["dx_out"], dx, ws, o["block"], o["w_post"], o["gate"], o["w_pre"],
                                    o["dh"], db, *s, accumulate=acc)
        sums.append(s)
    for a, b in zip(*sums):
        assert torch.equal(b, a + (-0.0 if M == 0 else 2.5))
        if M == 0:
            assert not a.any() and not torch.signbit(a).any() and not torch.signbit(b).any()


@gpu
def test_same_bits_again():
    o = operands(1500, 2048, torch.bfloat16, torch.float32, "channel", True, True, 10)
    p = moe.make_norm_problem(1500, 2048, gate_kind=moe.GATE_CHANNEL)
    runs = []
    for _ in range(2):
        s = [torch.empty(2048, device="cuda") for _ in range(3)]
        dx, db = torch.empty_like(o["x"]), torch.empty_like(o["x"])
        moe.moe_block_norm_backward(p, o["x"], o["dx_out"], dx, moe.allocate_norm_workspace(p).fill_(255), o["block"],
                                    o["w_post"], o["gate"], o["w_pre"], o["dh"], db, *s)
        runs.append([dx, db, *s])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


@gpu
def test_offsets_past_32_bits():
    """M K past 2^31 elements: the last rows."""
    M, K = 140000, 16384
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, K, device="cuda").to(torch.bfloat16)
    w = torch.ones(K, device="cuda")
    h = torch.empty_like(x)
    moe.moe_block_norm(moe.make_norm_problem(M, K), x, w_pre=w, h=h)
    _, _, r, e = norm_forward(f64(x[-3:]), None, None, 1.0, np.ones(K), 1e-6, 1.0)
    within(h[-3:], r, e, 2.0 ** -8)
    assert not h[:100].any() and not h[70000:70100].any()


@gpu
@pytest.mark.parametrize("M,K", [(600, 16384), (530, 9000)])
def test_many_long_rows(M, K):
    check(M, K, gate="channel", seed=M)
    check(M, K, torch.float32, torch.bfloat16, gate="token", seed=M + 1)


def test_subnormal_eps_is_refused():
    p = moe.make_norm_problem(4, 64)
    # 8 bytes a column and workgroup; one takes all four rows
    for eps, st in ((2.0 ** -127, -1), (1e-45, -1), (2.0 ** -126, 8 * 64)):
        p.eps = eps
        assert moe.load_library().moe_block_norm_ws_bytes(ctypes.byref(p)) == st


@gpu
def test_zero_rows_at_the_least_eps():
    """1 / rms is 2^63 there, and 0 stays 0 in the results and the gradients."""
    M, K = 3, 64
    p = moe.make_norm_problem(M, K, x_dtype=torch.float32, eps=2.0 ** -126)
    z, b = torch.zeros(M, K, device="cuda"), torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    w, x_out, h = torch.ones(K, device="cuda"), torch.full_like(z, 7.0), torch.full_like(b, 7.0)
    moe.moe_block_norm(p, z, x_out, b, w, None, w, h)
    assert not x_out.any() and not h.any()
    dx, db = torch.full_like(z, 7.0), torch.full_like(b, 7.0)
    dw = [torch.full_like(w, 7.0) for _ in range(2)]
    moe.moe_block_norm_backward(p, x_out, z, dx, moe.allocate_norm_workspace(p), block=b, w_post=w, w_pre=w, dh=b,
                                dblock=db, dw_post=dw[0], dw_pre=dw[1])
    assert not any(t.any() for t in (dx, db, *dw))

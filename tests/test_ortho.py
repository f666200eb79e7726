"""The orthogonalised update (moe_orthogonalize) against 64 bits.

One step has a bound for every element, from the roundings of its operands
(float16: 2^-11 relative, 2^-38 absolute at the scale used; sums of n float32
terms: n 2^-24), with absolute values carried through the products.  Over
several steps such a bound says nothing (each multiplies it by ||abs(X)||), so
there the distance (2-norm) is bounded by twice that of a 64-bit evaluation
with the same roundings, and by the 2e-3 that the interface states, besides
half a step of bf16."""
import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_expert_align_amd as moe
from block_refs import ortho, ortho_rounded

gpu = pytest.mark.gpu
MUON = [moe.MUON_COEF] * 5
HALF = 2.0 ** -8


# ------------------------------------------------------------- on the host --

def test_refusals():
    lib, a = moe.load_library(), 4096

    def call(update=a, out=a, ws=a, coef=None, **kw):
        p = moe.make_ortho_problem(2, 48, 64)
        for k, v in kw.items():
            setattr(p, k, v)
        if coef:
            p.coef[1][:] = coef
        return lib.moe_orthogonalize(ctypes.byref(p), update, out, ws, None), lib.moe_ortho_ws_bytes(ctypes.byref(p))

    inf, nan = float("inf"), float("nan")
    for kw in (dict(E=0), dict(N=0), dict(K=-1), dict(dtype=2), dict(steps=0), dict(steps=17), dict(eps=0.0),
               dict(eps=nan), dict(eps=inf), dict(scale=inf), dict(scale=nan)):
        assert call(**kw) == (moe.MOE_EINVAL, -1), kw
    for kw in (dict(E=65536), dict(N=32769), dict(K=32769), dict(N=32768, K=32768), dict(E=65535, N=2048, K=2048),
               dict(coef=(inf, 0, 0)), dict(coef=(0, nan, 0)), dict(coef=(1e5, 0, 0)), dict(coef=(1, 1e10, 0)),
               dict(coef=(0, 0, 3e38))):
        assert call(**kw) == (moe.MOE_EUNSUPPORTED, -1), kw
    for kw in (dict(update=None), dict(update=a + 2), dict(out=None), dict(out=a + 1), dict(ws=None), dict(ws=a + 8)):
        assert call(**kw)[0] == moe.MOE_EINVAL, kw
    with pytest.raises(ValueError, match="coef"):
        moe.make_ortho_problem(1, 4, 4, steps=3, coef=[(1, 2, 3)] * 2)
    with pytest.raises(ValueError, match="dtype"):
        moe.make_ortho_problem(1, 4, 4, dtype=torch.float16)
    with pytest.raises(ValueError, match="device tensor|cuda"):
        moe.moe_orthogonalize(moe.make_ortho_problem(1, 4, 4), torch.zeros(1, 4, 4), torch.zeros(1, 4, 4), torch.zeros(1))


def matrix(kind, n, m, seed):
    rng = np.random.default_rng(seed)
    u = rng.normal(size=(n, m))
    if kind == "low rank":
        u = 0.1 * u + rng.normal(size=(n, 6)) @ rng.normal(size=(6, m))
    elif kind == "decay":
        q = np.linalg.svd(u, full_matrices=False)
        u = q[0] * np.logspace(0, -3, min(n, m)) @ q[2]
    return u


@pytest.mark.parametrize("kind", ["gauss", "low rank", "decay"])
@pytest.mark.parametrize("n,m", [(40, 40), (64, 200), (300, 96), (1024, 32)])
def test_the_roundings_leave_less_than_stated(kind, n, m):
    u = matrix(kind, n, m, n + m)
    e = ortho(u, MUON, 1e-7)
    assert np.linalg.norm(ortho_rounded(u, MUON, 1e-7) - e) < 2e-3 * np.linalg.norm(e)


# ---------------------------------------------------------------------- GPU --

def run(u, dtype=torch.float32, coef=MUON, eps=1e-7, scale=1.0, stream=None):
    t = torch.from_numpy(np.asarray(u, np.float64)).to("cuda", dtype)
    p = moe.make_ortho_problem(*t.shape, dtype=dtype, steps=len(coef), coef=coef, eps=eps, scale=scale)
    buf = torch.full((t.numel() + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:t.numel()].view(t.shape)
    ws = torch.full((moe.moe_ortho_ws_bytes(p) + 256,), 255, dtype=torch.uint8, device="cuda")
    moe.moe_orthogonalize(p, t, out, ws, stream=stream)
    assert (buf[t.numel():] == 3).all() and (ws[-256:] == 255).all()
    return t.double().cpu().numpy(), out.double().cpu().numpy(), p


def one_step_bound(x, a, b, c):
    """|error| of one step on X [n, m] whose float16 pieces are exact to 2^-11 and 2^-22."""
    n, m = x.shape
    u, tiny = 2.0 ** -11, 2.0 ** -38
    gn, gm = 2 * n * 2.0 ** -24, 2 * m * 2.0 ** -24
    ax = np.abs(x)
    ex = u * ax + tiny
    A = x.T @ x
    aa = ax.T @ ax
    ea = ax.T @ ex + ex.T @ ax + ex.T @ ex + gn * aa
    off = ~np.eye(m, dtype=bool)
    eo = ea + off * (u * (np.abs(A) + ea) + tiny)
    B = b * A + c * (A @ A)
    bA = np.abs(A) + eo
    eb = abs(b) * eo + abs(c) * (bA @ eo + eo @ bA + gm * bA @ bA) + 2.0 ** -21 * (abs(b) * bA + abs(c) * bA @ bA)
    eq = eb + off * (u * (np.abs(B) + eb) + tiny)
    bB = np.abs(B) + eq
    return ax @ eq + ex @ (off * bB) + gm * ax @ bB + (2.0 ** -21 * ax + tiny) * (abs(a) + np.diag(bB))


@gpu
@pytest.mark.parametrize("N,K", [(1, 1), (1, 9), (7, 1), (2, 3), (16, 16), (31, 33), (64, 64), (65, 64), (64, 130),
                                 (100, 40), (200, 72), (129, 256), (320, 96), (515, 33)])
@pytest.mark.parametrize("coef", [moe.MUON_COEF, (1.5, -0.5, 0.0), (1.0, 0.0, 0.0), (0.0, 0.0, 2.0)])
def test_one_step(N, K, coef):
    for E, dtype in ((1, torch.float32), (3, torch.bfloat16)):
        u, got, p = run(np.stack([matrix("gauss", N, K, s + N) for s in range(E)]), dtype, [coef], scale=0.5)
        a, b, c = (float(v) for v in p.coef[0])
        for e in range(E):
            ref = 0.5 * ortho(u[e], [(a, b, c)], p.eps)
            x = u[e] if N >= K else u[e].T
            x = x / (np.linalg.norm(x) + p.eps)
            err = 0.5 * one_step_bound(x, a, b, c)
            if N < K:
                err = err.T
            assert np.all(np.abs(got[e] - ref) <= err + HALF * (np.abs(ref) + err) + 1e-37), (e, np.abs(got[e] - ref).max())


def check(u, got, p, e):
    coef = [tuple(float(v) for v in p.coef[i]) for i in range(p.steps)]
    ref = p.scale * ortho(u, coef, p.eps)
    size = np.linalg.norm(ref)
    rounded = np.linalg.norm(p.scale * ortho_rounded(u, coef, p.eps) - ref)
    off = np.linalg.norm(got - ref)
    assert off <= 2 * rounded + 2.0 ** -16 * size + HALF * size, (e, off / size, rounded / size)
    assert off <= 2e-3 * size + HALF * size


@gpu
@pytest.mark.parametrize("kind", ["gauss", "low rank", "decay"])
@pytest.mark.parametrize("N,K", [(40, 40), (64, 200), (300, 96), (1024, 32), (256, 512), (500, 333)])
def test_five_steps(kind, N, K):
    u, got, p = run(np.stack([matrix(kind, N, K, s + K) for s in range(3)]))
    for e in range(3):
        check(u[e], got[e], p, e)


@gpu
@pytest.mark.parametrize("E,N,K", [(40, 256, 300), (9, 1024, 700), (7, 1100, 1500), (13, 1024, 1024), (33, 640, 768)])
def test_larger_tiles(E, N, K):
    """Enough matrices for each tile size; the first and the last of them."""
    u, got, p = run(np.stack([matrix("gauss", N, K, s) for s in range(E)]), torch.bfloat16, scale=0.2)
    for e in (0, E // 2, E - 1):
        check(u[e], got[e], p, e)


@gpu
@pytest.mark.parametrize("steps", [2, 3, 8, 16])
def test_other_steps_and_coefficients(steps):
    coef = [(1.5, -0.5, 0.0)] * steps if steps > 8 else [(2.0 + 0.1 * i, -1.5, 0.5) for i in range(steps)]
    if steps == 8:
        # a singular value of 1 goes to a + b + c = 1.7 at (2.7, -1.5, 0.5), and from 1.7 on to 4.3, 580, ...: refused
        with pytest.raises(moe.MoeError):
            run(matrix("gauss", 96, 64, 3)[None], coef=coef)
        coef = [(1.9 - 0.1 * i, -1.2 + 0.1 * i, 0.3) for i in range(steps)]   # a + b + c = 1 at each
    u, got, p = run(matrix("gauss", 96, 64, 3)[None], coef=coef)
    check(u[0], got[0], p, 0)


@gpu
def test_a_matrix_by_itself():
    """Zero, infinite and NaN matrices, and scales from 1e-30 to 1e30, beside each other."""
    E, N, K = 8, 72, 100
    u = np.stack([matrix("gauss", N, K, s) for s in range(E)])
    u[1] = 0.0
    u[2, 5, 7] = np.inf
    u[3, 71, 99] = np.nan
    u[4] *= 1e30
    u[5] *= 1e-4
    u[6, 0] = 0.0
    x, got, p = run(u)
    assert not got[1].any() and np.isnan(got[2]).all() and np.isnan(got[3]).all()
    for e in (0, 4, 5, 6, 7):
        check(x[e], got[e], p, e)
    _, alone, _ = run(u[7:])
    assert np.array_equal(alone[0], got[7])
    # eps is felt where the norm is of its size
    x, got, p = run(u[:1] * 1e-9)
    check(x[0], got[0], p, 0)


@gpu
def test_the_transpose_gives_the_transpose():
    """The same bits: both work on the taller of the two."""
    u = matrix("gauss", 200, 90, 5)
    _, a, _ = run(u[None])
    _, b, _ = run(u.T[None].copy())
    assert np.array_equal(a[0], b[0].T)


@gpu
def test_same_bits_again_and_on_another_stream():
    u = np.stack([matrix("gauss", 256, 512, s) for s in range(8)])
    _, a, _ = run(u)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _, b, _ = run(u)
    torch.cuda.synchronize()
    assert np.array_equal(a, b)


@gpu
@pytest.mark.parametrize("E,N,K", [(1, 130, 4100), (2, 3001, 200), (1, 70, 1600), (3, 65, 2000), (40, 33, 700),
                                   (300, 20, 40)])
def test_long_contractions_and_many_narrow_matrices(E, N, K):
    """A's tiles shared by several workgroups; narrow matrices with several workgroups each, or one."""
    u, got, p = run(np.stack([matrix("gauss", N, K, s) for s in range(E)]))
    for e in (0, E // 2, E - 1):
        check(u[e], got[e], p, e)
    _, again, _ = run(u)
    assert np.array_equal(got, again)


@gpu
def test_workspace_serves_one_problem_after_another():
    """Its contents do not matter: problems of different sizes in turn, on one workspace, give the bits they
    give alone, and so do two streams with a workspace each."""
    shapes = [(1, 128, 4096), (2, 64, 300), (1, 128, 4096), (3, 200, 256), (1, 130, 4100)]
    probs, ins, want = [], [], []
    for i, (E, N, K) in enumerate(shapes):
        p = moe.make_ortho_problem(E, N, K)
        t = torch.from_numpy(np.stack([matrix("gauss", N, K, 10 * i + s) for s in range(E)])).float().cuda()
        out = torch.empty(t.shape, dtype=torch.bfloat16, device="cuda")
        moe.moe_orthogonalize(p, t, out, moe.allocate_ortho_workspace(p))
        probs.append(p), ins.append(t), want.append(out)
    size = max(moe.moe_ortho_ws_bytes(p) for p in probs)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
            for p, t in zip(probs, ins):
                out = torch.empty(t.shape, dtype=torch.bfloat16, device="cuda")
                moe.moe_orthogonalize(p, t, out, ws)
                outs.append((out, ws))
    torch.cuda.synchronize()
    for i, (out, _) in enumerate(outs):
        assert torch.equal(out, want[i % len(want)])


@gpu
@pytest.mark.parametrize("E,N,K", [(2, 64, 40), (2, 40, 64), (2, 96, 200), (2, 200, 96), (1, 32768, 8), (1, 3, 32768),
                                   (2000, 3, 2)])
def test_out_and_update_aligned_to_their_elements(E, N, K):
    for dtype in (torch.float32, torch.bfloat16):
        u = np.stack([matrix("gauss", N, K, s % 7) for s in range(E)])
        t, want, p = run(u, dtype)
        src = torch.empty(t.size + 1, dtype=dtype, device="cuda")[1:].view(E, N, K)
        src.copy_(torch.from_numpy(t))
        buf = torch.full((t.size + 66,), 3.0, dtype=torch.bfloat16, device="cuda")
        out = buf[1:1 + t.size].view(E, N, K)
        moe.moe_orthogonalize(p, src, out, moe.allocate_ortho_workspace(p))
        assert np.array_equal(out.double().cpu().numpy(), want)
        assert buf[0] == 3 and (buf[1 + t.size:] == 3).all()
    for e in (0, E - 1):
        check(t[e], want[e], p, e)


@gpu
@pytest.mark.parametrize("E,N,K", [(4, 40, 700), (4, 700, 40), (4, 1, 5), (4, 3, 1), (20, 520, 640), (30, 1024, 600)])
def test_not_finite_in_each_path(E, N, K):
    """The one-launch steps, and the tiles of 64 and more: NaN in all of a bad matrix, none beside it."""
    u = np.stack([matrix("gauss", N, K, s) for s in range(E)])
    u[1, N - 1, 0] = np.nan
    u[2, 0, K - 1] = -np.inf
    for dtype in (torch.float32, torch.bfloat16):
        x, got, p = run(u, dtype)
        assert np.isnan(got[1]).all() and np.isnan(got[2]).all()
        for e in (0, 3, E - 1):
            check(x[e], got[e], p, e)

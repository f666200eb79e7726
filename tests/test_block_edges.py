"""Calls at the edges of what the interface allows, for the operators of a
block's training: a sequence that begins inside a workgroup's tokens, logits of
10^9, sums over very many rows, batches of no tokens, matrices of a few strong
directions, tiny coefficients and scales."""
import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_expert_align_amd as moe
from block_refs import U24, norm_backward, ortho, scores
from test_balance import check, make, run
from test_norm import GATE, f64, gate64, operands, within
from test_ortho import check as ortho_check, run as ortho_run

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [12, 64, 512, 513, 600])
def test_one_sequence_that_begins_inside_a_workgroup(E, dtype, scoring):
    """seq_offsets with S = 1: 16 tokens a workgroup up to 512 experts, 4 past them."""
    l, ids, _ = make(50, E, 3, 1, dtype, E)
    for off in ([5, 50], [17, 40], [3, 4], [1, 50], [0, 49], [49, 50], [16, 50], [50, 50]):
        check(l, ids, off, scoring)
        base = torch.randn(l.shape, device="cuda").to(dtype) * 0.01
        dloss = np.ones(1, np.float32)
        *_, plain = run(l, ids, off, scoring, dloss=dloss)
        *_, got = run(l, ids, off, scoring, dloss=dloss, accumulate=True, dl=base.clone())
        out = torch.ones(50, dtype=torch.bool, device="cuda")
        out[off[0]:off[1]] = False
        assert torch.equal(got[out], base[out]) and not plain[out].any()
        if dtype == torch.float32:
            assert torch.equal(got, base + plain)
        else:   # one rounding of the sum; the addend there is not rounded
            err = (got.double() - base.double() - plain.double()).abs()
            assert (err <= 2.0 ** -8 * (got.double().abs() + plain.double().abs()) + 1e-37).all()


@gpu
@pytest.mark.parametrize("E", [8, 100, 600])
def test_logits_of_a_billion_and_more(E):
    """Rows of equal or nearly equal logits t: the float32 product of t and log2(e) is off by 2^-24 of itself,
    up to 2^6 at 10^9 and 2^8 at 5 10^9, which must not meet an exponential's range.  A token a sequence, so
    probs are its scores."""
    top = [-2.06e9, -2.68e9, -6.19e9, -10.94e9, 5.58e9, 7.81e9, 14.79e9, -1e9, -1e10, 1e12, -1e29, 1e30, 3e38, -1e37,
           2.0 ** 29, -2.0 ** 29, 2.0 ** 31, -2.0 ** 31, 3e8]
    M = 2 * len(top)
    l = np.repeat(np.array(top, np.float32), 2)[:, None] * np.ones((M, E), np.float32)
    l[1::2, 1:] = -np.inf if E == 100 else -3e38      # every other row: one expert, the others far below
    ids = np.stack([np.arange(M) % E, (np.arange(M) + 3) % E], 1).astype(np.int32)
    dloss = np.ones(M, np.float32)
    ref, _ = scores(l.astype(np.float64), "softmax")
    loss, counts, tokens, probs, dl = run(torch.from_numpy(l).cuda(), ids, list(range(M + 1)), "softmax", dloss=dloss)
    assert (tokens == 1).all() and (counts.sum(1) == 2).all()
    # equal logits, equal scores: 56 half steps for the exponential, the sum and the quotient
    assert np.all(np.abs(probs - ref) <= 56 * U24 * ref), np.abs(probs / np.maximum(ref, 1e-30) - 1).max()
    assert np.all(np.abs(loss - E / 2 * (counts * ref).sum(1)) <= E / 2 * 60 * U24 * (counts * ref).sum(1))
    want = E / 2 * ref * (counts - (counts * ref).sum(1, keepdims=True))
    # |c - dot| and dot are at most 1 here: 56 half steps of p each, 44 of the sum, 10 of the rest
    assert np.all(np.abs(dl.double().cpu().numpy() - want) <= E / 2 * ref * 2 * (56 + 56 + 44 + 10) * U24)


@gpu
@pytest.mark.parametrize("M,K,gate", [(1 << 20, 64, "channel"), (1 << 18, 1032, "none"), (1 << 16, 4104, "channel"),
                                      (1 << 16, 9000, "none")])
def test_sums_over_many_equal_rows(M, K, gate):
    """Every row adds the same term, so a run of n float32 additions can be off in one direction by half a step of
    the sum each, n / 2 half steps of the last.  The bound is block_refs' 100 half steps, whatever M."""
    o = operands(1, K, torch.bfloat16, torch.float32, gate, True, True, K)
    p = moe.make_norm_problem(M, K, gate_kind=GATE[gate])
    rows = {n: o[n].expand(M, K).contiguous() for n in ("x", "block", "dx_out", "dh")}
    sums = {n: torch.empty(K, device="cuda") for n in ("dw_post", "dw_pre") + (("dgate",) if gate != "none" else ())}
    dx, db = torch.empty_like(rows["x"]), torch.empty_like(rows["x"])
    moe.moe_block_norm_backward(p, rows["x"], rows["dx_out"], dx, moe.allocate_norm_workspace(p), rows["block"],
                                o["w_post"], o["gate"], o["w_pre"], rows["dh"], db, **sums)
    ref = norm_backward(f64(o["x"]), f64(o["block"]), f64(o["w_post"]), gate64(o, gate), f64(o["w_pre"]),
                        f64(o["dx_out"]), f64(o["dh"]), p.eps, p.res_scale)
    for n, got in sums.items():
        want, err = ref["dgate_channel" if n == "dgate" else n]
        within(got, M * want, M * err, 2.0 ** -24, n)
    assert (dx == dx[0]).all() and (db == db[0]).all()


@gpu
def test_no_tokens_with_a_gate_per_token():
    """An empty gate has no address; the sums are written, or left by accumulate."""
    K = 520
    p = moe.make_norm_problem(0, K, gate_kind=moe.GATE_TOKEN)
    none = torch.empty(0, K, dtype=torch.bfloat16, device="cuda")
    w, empty = torch.ones(K, device="cuda"), torch.empty(0, device="cuda")
    ws = moe.allocate_norm_workspace(p)
    moe.moe_block_norm(p, none, none, none, w, empty, w, none)
    for dgate in (empty, None):
        s = [torch.full((K,), -0.0, device="cuda") for _ in range(2)]
        moe.moe_block_norm_backward(p, none, none, none, ws, none, w, empty, w, none, none, s[0], dgate, s[1])
        assert all(not t.any() and not torch.signbit(t).any() for t in s)
        s = [torch.full((K,), 2.5, device="cuda") for _ in range(2)]
        moe.moe_block_norm_backward(p, none, none, none, ws, none, w, empty, w, none, none, s[0], dgate, s[1],
                                    accumulate=True)
        assert all((t == 2.5).all() for t in s)


def test_a_gate_per_token_is_asked_for_where_there_are_tokens():
    lib, a = moe.load_library(), 4096
    p = moe.make_norm_problem(4, 64, gate_kind=moe.GATE_TOKEN)
    assert lib.moe_block_norm(ctypes.byref(p), a, a, a, None, a, a, a, None) == moe.MOE_EINVAL
    args = [a, a, a, None, a, a, a, a, a, a, None, a, 0, a, None]
    assert lib.moe_block_norm_backward(ctypes.byref(p), *args) == moe.MOE_EINVAL
    # without tokens too, a gate's gradient per channel needs the gate, and a gate needs its kind
    p = moe.make_norm_problem(0, 64, gate_kind=moe.GATE_CHANNEL)
    assert lib.moe_block_norm_backward(ctypes.byref(p), *args) == moe.MOE_EINVAL
    p = moe.make_norm_problem(0, 64)
    args[3] = a
    assert lib.moe_block_norm_backward(ctypes.byref(p), *args) == moe.MOE_EINVAL


@gpu
@pytest.mark.parametrize("M,E", [(100, 12), (1500, 12), (700, 600)])
def test_malformed_offsets_write_nothing_past_workspace_or_gradient(M, E):
    """Offsets that descend or leave [0, M], in one launch and in two: the slots that depend on them stay within the
    workspace, the gradient within its rows."""
    l, ids, _ = make(M, E, 2, 1, torch.float32, 13)
    r, dev_ids = moe.make_router(E, 2), torch.from_numpy(ids).cuda()
    for off in ([0, M - 10, M // 5, M], [-5, 30, 2 * M, 10 * M], [M, 0, M, 0], [1 << 30, -(1 << 30), 5, M // 2],
                [M // 2, -(1 << 31), (1 << 31) - 1, 0]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        ws = torch.full((moe.moe_balance_ws_bytes(r, M, 3) + 4096,), 255, dtype=torch.uint8, device="cuda")
        f = torch.full((2, 4, E), 7.0, device="cuda")
        n = torch.full((2, 4, E), 77, dtype=torch.int32, device="cuda")
        loss, probs, tokens, counts = f[0, :3, 0].contiguous(), f[1, :3], n[0, :3, 0].contiguous(), n[1, :3]
        grad = torch.full((M + 2, E), 7.0, device="cuda")
        moe.moe_balance_loss(r, l, dev_ids, loss, counts, tokens, probs, ws, seq_offsets=o)
        moe.moe_balance_loss_backward(r, l, dev_ids, counts, tokens, torch.ones(3, device="cuda"), grad[1:M + 1],
                                      seq_offsets=o)
        assert (ws[-4096:] == 255).all() and (f[1, 3] == 7).all() and (n[1, 3] == 77).all()
        assert (grad[0] == 7).all() and (grad[M + 1] == 7).all()


def test_workspace_sizes_of_refused_problems_name_the_reason():
    for call, p, status in ((moe.moe_block_norm_ws_bytes, moe.make_norm_problem(4, 60), moe.MOE_EUNSUPPORTED),
                            (moe.moe_block_norm_ws_bytes, moe.make_norm_problem(4, 1 << 20), moe.MOE_EUNSUPPORTED),
                            (moe.moe_block_norm_ws_bytes, moe.make_norm_problem(-1, 64), moe.MOE_EINVAL),
                            (moe.moe_ortho_ws_bytes, moe.make_ortho_problem(1, 40000, 8), moe.MOE_EUNSUPPORTED),
                            (moe.moe_ortho_ws_bytes, moe.make_ortho_problem(1, 8, 8, coef=(1e9, 0, 0)),
                             moe.MOE_EUNSUPPORTED),
                            (moe.moe_ortho_ws_bytes, moe.make_ortho_problem(0, 8, 8), moe.MOE_EINVAL)):
        with pytest.raises(moe.MoeError) as e:
            call(p)
        assert e.value.status == status


# ---------------------------------------------------------------- ortho ----

def few_strong(n, m, r, w, seed):
    """n x m with r singular values of 1 and the others w."""
    g = np.random.default_rng(seed)
    u, s, v = np.linalg.svd(g.normal(size=(max(n, m), min(n, m))), full_matrices=False)
    x = (u * np.where(np.arange(s.size) < r, 1.0, w)) @ v
    return x if n >= m else x.T.copy()


def least_error(u, coef, steps):
    """2-norm, relative, of what the result is off by before its rounding to bf16, at least: the result times 16
    scales of [1, 2), each rounded to bf16, leaves an interval for every element."""
    t = torch.from_numpy(u).to("cuda", torch.float32)
    ref = np.stack([ortho(x, [coef] * steps, 1e-7) for x in t.double().cpu().numpy()])
    lo, hi = np.full(u.shape, -np.inf), np.full(u.shape, np.inf)
    for k in range(16):
        scale = 1.0 + k / 16
        p = moe.make_ortho_problem(*u.shape, steps=steps, coef=coef, scale=scale)
        out = torch.empty(u.shape, dtype=torch.bfloat16, device="cuda")
        moe.moe_orthogonalize(p, t, out, moe.allocate_ortho_workspace(p))
        v = out.double().cpu().numpy()
        half = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 1e-30))) - 8), 1e-37)   # of a bf16 step
        lo, hi = np.maximum(lo, (v - half) / scale), np.minimum(hi, (v + half) / scale)
    # (the scale enters in float32: the intervals of one value may miss each other by a few of its half steps)
    assert np.all(lo <= hi + 64 * U24 * (np.abs(ref) + np.sqrt((ref ** 2).mean()))), (lo - hi).max()
    off = np.maximum(np.maximum(lo - ref, ref - hi), 0.0)
    return np.sqrt((off ** 2).sum((1, 2)) / (ref ** 2).sum((1, 2)))


def a_few_strong_directions(n, m):
    r = [k for k in (1, 4, 8, min(n, m) // 2) if 0 < k < min(n, m)] or [1]
    u = np.stack([few_strong(n, m, k, w, i) for k in r for i, w in enumerate((1e-2, 3e-4, 1e-5))])
    e = least_error(u, moe.MUON_COEF, 5)
    assert e.max() <= 2e-3, e


@gpu
@pytest.mark.parametrize("n,m", [(64, 2), (2, 2), (64, 5), (5, 5), (6, 7), (9, 9), (17, 16), (1000, 12),
                                 (16, 300), (1024, 32), (4096, 64), (64, 64)])
def test_a_few_strong_directions_of_a_narrow_matrix(n, m):
    """Singular values far below others: what rounding adds in a strong direction must not reach the weak ones.
    Within the 2e-3 that the interface states (64-bit evaluations with the kernel's roundings leave up to 1.4e-3)."""
    a_few_strong_directions(n, m)


@gpu
@pytest.mark.parametrize("n,m", [(65, 65), (1024, 96), (96, 1000), (2048, 128), (256, 256), (260, 1030), (1536, 384),
                                 (700, 512), (1024, 520), (768, 768)])
def test_a_few_strong_directions(n, m):
    a_few_strong_directions(n, m)


@gpu
@pytest.mark.parametrize("N,K", [(96, 40), (130, 200)])
@pytest.mark.parametrize("coef", [(3.0, -3.0, 1e-20), (3.0, -3.0, -1e-20), (2.0, -2.0, 1e-30), (2.0, 1e-25, 1e-30),
                                  (1.5, -0.5, 1e-18)])
def test_coefficients_beside_far_larger_ones(coef, N, K):
    """The largest value that a singular value can take lies at a root of a + 3 b y + 5 c y^2, whose usual formula
    cancels for small c: a bound that misses it scales X past float16's range."""
    u, got, p = ortho_run(np.stack([few_strong(N, K, 3, 0.5, s) for s in range(2)]), coef=[coef] * 2)
    for e in range(2):
        ortho_check(u[e], got[e], p, e)


@gpu
@pytest.mark.parametrize("N,K", [(40, 64), (96, 66), (66, 200), (300, 400)])
@pytest.mark.parametrize("scale", [1e-37, -2e-37, 1e37, 2e38])
def test_scales_at_the_ends_of_float32(scale, N, K):
    """Values near 1 in blocks of 2 x 2, so that the result is a normal number wherever it is not 0: the scale meets
    X itself, not the powers of two that the products carry."""
    u = np.zeros((2, N, K))
    g = np.random.default_rng(N + K)
    for i in range(0, min(N, K) - 1, 2):
        u[:, i:i + 2, i:i + 2] = np.eye(2) + 0.6 * g.uniform(-1, 1, (2, 2, 2))
    u, got, p = ortho_run(u, scale=scale)
    for e in range(2):
        ortho_check(u[e], got[e], p, e)

"""The balance loss, its counts and its gradient (moe_balance_loss,
moe_balance_loss_backward) against 64 bits.  Counts are exact; the scores'
errors are derived in block_refs.scores; a sum over a chunk's tokens in float32
(at most M / 512 + 16 + 32 tokens, four or sixteen at a time) adds at most
chunk / 4 + 8 half steps, the sum over the chunks is float64."""
import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_expert_align_amd as moe
from block_refs import U24, balance, balance_backward, scores

SCORING = {"softmax": moe.ROUTE_SOFTMAX, "sigmoid": moe.ROUTE_SIGMOID}
gpu = pytest.mark.gpu


# ------------------------------------------------------------- on the host --

def test_refusals():
    lib, r, a = moe.load_library(), moe.make_router(16, 2), 4096
    rb = moe.make_router(16, 2, bias_kind=moe.BIAS_LOGIT)

    def fwd(rr=r, M=4, S=2, logits=a, dtype=0, ld=16, bias=None, ids=a, off=a, loss=a, counts=a, tokens=a, probs=a,
            ws=a):
        return lib.moe_balance_loss(ctypes.byref(rr), M, S, logits, dtype, ld, bias, ids, off, loss, counts, tokens,
                                    probs, ws, None)

    def bwd(rr=r, M=4, S=2, logits=a, dtype=0, ld=16, bias=None, ids=a, off=a, counts=a, tokens=a, dloss=a, dl=a,
            dld=16, acc=0):
        return lib.moe_balance_loss_backward(ctypes.byref(rr), M, S, logits, dtype, ld, bias, ids, off, counts, tokens,
                                             dloss, dl, dld, acc, None)

    both = [dict(M=-1), dict(M=1 << 31), dict(M=1 << 30), dict(S=0), dict(S=65537), dict(off=None), dict(off=a + 2),
            dict(logits=None), dict(logits=a + 2), dict(dtype=2), dict(ld=15), dict(bias=a), dict(rr=rb), dict(ids=None),
            dict(ids=a + 1), dict(counts=None), dict(counts=a + 2), dict(tokens=None), dict(tokens=a + 1),
            dict(rr=moe.make_router(0, 1)), dict(rr=moe.make_router(4, 5)), dict(rr=moe.make_router(2049, 1))]
    for kw in both:
        assert fwd(**kw) == moe.MOE_EINVAL, kw
        assert bwd(**kw) == moe.MOE_EINVAL, kw
    for kw in (dict(loss=None), dict(loss=a + 2), dict(probs=None), dict(ws=None), dict(ws=a + 8)):
        assert fwd(**kw) == moe.MOE_EINVAL, kw
    for kw in (dict(dloss=None), dict(dl=None), dict(dl=a + 2), dict(dld=15), dict(acc=2)):
        assert bwd(**kw) == moe.MOE_EINVAL, kw
    assert bwd(M=0, logits=None, ids=None, dl=None) == moe.MOE_OK      # nothing to do
    assert lib.moe_balance_ws_bytes(ctypes.byref(r), 4, 0) == -1
    assert lib.moe_balance_ws_bytes(ctypes.byref(r), -1, 1) == -1
    with pytest.raises(moe.MoeError):
        moe.moe_balance_ws_bytes(moe.make_router(4, 5), 4)


def test_binding_refuses():
    r, x = moe.make_router(16, 2), torch.zeros(4, 16)
    i32 = dict(dtype=torch.int32)
    ids, c, t = torch.zeros(4, 2, **i32), torch.zeros(1, 16, **i32), torch.zeros(1, **i32)
    f, ws = torch.zeros(1), torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_balance_loss(r, x, ids, f, c, t, torch.zeros(1, 16), ws)
    with pytest.raises(ValueError, match="shape"):
        moe._sequences(torch.zeros(1, 15, **i32), 16, None)
    with pytest.raises(ValueError, match="need seq_offsets"):
        moe._sequences(torch.zeros(2, 16, **i32), 16, None)
    with pytest.raises(ValueError, match="expected 3"):
        moe._sequences(torch.zeros(2, 16, **i32), 16, torch.zeros(2, **i32))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_reference_gradient_is_the_difference_quotient(scoring):
    rng = np.random.default_rng(1)
    l, ids, off = rng.normal(size=(7, 6)), rng.integers(-1, 6, size=(7, 2)), [0, 3, 3, 7]
    ids[2] = -1
    dloss = rng.normal(size=3)
    loss, counts, tokens, _, _ = balance(l, ids, off, scoring)
    d, _ = balance_backward(l, ids, off, scoring, counts, tokens, dloss)
    for t in range(7):
        for e in range(6):
            q = []
            for h in (1e-6, -1e-6):
                lp = l.copy()
                lp[t, e] += h
                q.append((balance(lp, ids, off, scoring)[0] * dloss).sum())
            assert abs((q[0] - q[1]) / 2e-6 - d[t, e]) < 1e-8


# ---------------------------------------------------------------------- GPU --

def make(M, E, topk, S, dtype, seed, ld=None, scale=1.0, padded=False):
    rng = np.random.default_rng(seed)
    full = torch.from_numpy((rng.normal(size=(M, ld or E)) * scale).astype(np.float32)).to("cuda", dtype)
    ids = np.argsort(-(rng.normal(size=(M, E)) + np.linspace(1, -1, E)), 1)[:, :topk].astype(np.int32)
    if padded:
        ids[rng.random(M) < 0.2] = -1
        ids[rng.random((M, topk)) < 0.1] = -1
    off = np.concatenate([[0], np.sort(rng.integers(0, M + 1, S - 1)), [M]]).astype(np.int32)
    return full[:, :E], ids, off


def run(l, ids, off, scoring, bias=None, bias_kind=moe.BIAS_NONE, dloss=None, accumulate=None, dl=None, router=None):
    M, E = l.shape
    S = len(off) - 1
    r = router or moe.make_router(E, ids.shape[1], SCORING[scoring], bias_kind)
    dev_ids = torch.from_numpy(np.ascontiguousarray(ids)).cuda()
    o = torch.from_numpy(np.asarray(off, np.int32)).cuda() if S > 1 or off[0] != 0 or off[-1] != M else None
    # one element more than the call writes
    loss, tokens = torch.full((S + 1,), 7.0, device="cuda"), torch.full((S + 1,), 77, dtype=torch.int32, device="cuda")
    counts = torch.full((S + 1, E), 77, dtype=torch.int32, device="cuda")
    probs = torch.full((S + 1, E), 7.0, device="cuda")
    ws = moe.allocate_balance_workspace(r, M, S).fill_(255)
    b = None if bias is None else torch.from_numpy(bias).cuda()
    moe.moe_balance_loss(r, l, dev_ids, loss, counts[:S], tokens, probs, ws, bias=b, seq_offsets=o)
    assert loss[S] == 7.0 and tokens[S] == 77 and (counts[S] == 77).all() and (probs[S] == 7.0).all()
    if dloss is not None:
        dl = torch.full_like(l, float("nan")) if dl is None else dl
        moe.moe_balance_loss_backward(r, l, dev_ids, counts[:S], tokens, torch.from_numpy(dloss).cuda(), dl, bias=b,
                                      seq_offsets=o, accumulate=bool(accumulate))
    return (loss[:S].cpu().numpy().astype(np.float64), counts[:S].cpu().numpy(), tokens[:S].cpu().numpy(),
            probs[:S].cpu().numpy().astype(np.float64), dl)


def check(l, ids, off, scoring="softmax", bias=None, bias_kind=moe.BIAS_NONE):
    M, E = l.shape
    topk, S = ids.shape[1], len(off) - 1
    lh = l.float().cpu().numpy().astype(np.float64)
    if bias_kind == moe.BIAS_LOGIT:
        lh = lh + bias.astype(np.float64)
    dloss = np.random.default_rng(9).normal(size=S).astype(np.float32)
    loss, counts, tokens, probs, dl = run(l, ids, off, scoring, bias, bias_kind, dloss)
    rl, rc, rt, rp, tol = balance(lh, ids, off, scoring)
    assert np.array_equal(counts, rc) and np.array_equal(tokens, rt)
    chunk = max(32, -(-M // 512) + 16)
    tol = tol + rp * U24 * (chunk / 4 + 10) + 1e-37
    assert np.all(np.abs(probs - rp) <= tol), (np.abs(probs - rp) - tol).max()
    per = E / (topk * np.maximum(rt, 1))
    assert np.all(np.abs(loss - rl) <= per * (rc * tol).sum(1) + 2 * U24 * np.abs(rl))
    rd, bound = balance_backward(lh, ids, off, scoring, rc, rt, dloss.astype(np.float64))
    got = dl.float().cpu().numpy().astype(np.float64)
    bound = bound + (2.0 ** -8 if l.dtype == torch.bfloat16 else U24) * np.abs(rd)
    assert np.all(np.abs(got - rd) <= bound), (np.abs(got - rd) - bound).max()
    assert np.all(got[(rd == 0) & (bound == 0)] == 0)


@gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,topk,S", [(1, 1, 1, 1), (1, 8, 2, 1), (5, 16, 3, 2), (64, 8, 2, 1), (33, 17, 4, 5),
                                        (130, 64, 8, 3), (31, 65, 8, 31), (257, 128, 8, 4), (77, 129, 5, 1),
                                        (40, 256, 8, 7), (65, 300, 16, 2), (70, 512, 8, 3), (35, 513, 64, 2),
                                        (34, 2048, 7, 2), (1500, 60, 4, 9)])
def test_balance(scoring, M, E, topk, S):
    for dtype in (torch.float32, torch.bfloat16):
        l, ids, off = make(M, E, topk, S, dtype, M + E, padded=M % 2 == 1)
        check(l, ids, off, scoring)


@gpu
def test_many_tokens_to_a_workgroup():
    l, ids, off = make(20011, 24, 2, 3, torch.float32, 3)
    check(l, ids, off)


@gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_bias_strides_and_scale(scoring):
    l, ids, off = make(97, 48, 4, 3, torch.float32, 5, ld=53, scale=6.0)
    bias = np.random.default_rng(2).normal(size=48).astype(np.float32)
    check(l, ids, off, scoring, bias, moe.BIAS_LOGIT)
    check(l, ids, off, scoring, bias, moe.BIAS_SELECT)      # plays no part
    l, ids, off = make(97, 48, 4, 3, torch.bfloat16, 6, ld=49)
    check(l, ids, off, scoring)


@gpu
def test_strided_gradient_leaves_the_gaps():
    l, ids, off = make(20, 24, 2, 1, torch.float32, 8)
    buf = torch.full((20, 31), 5.0, device="cuda")
    dl = buf[:, :24]
    *_, _ = run(l, ids, off, "softmax", dloss=np.ones(1, np.float32), dl=dl)
    assert (buf[:, 24:] == 5.0).all() and not (dl == 5.0).any()


@gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_masks_and_special_values(scoring):
    E, low = 40, float(torch.finfo(torch.float32).min)
    l, ids, off = make(16, E, 3, 2, torch.float32, 11)
    l[0] = float("-inf")                       # no expert to choose from
    l[1, 3:] = float("-inf")
    l[2] = float("nan")
    l[3, ::2] = float("nan")
    l[4] = low
    l[5, 1:] = low
    l[6, 7] = float("inf")
    l[7, 7:9] = float("inf")
    l[8] = 0.0
    l[9] = -200.0 + l[9]                       # sigmoids under float32's smallest number
    l[10] = 90.0 + l[10]
    l[11, 5] = 60.0                            # a confident token
    check(l, ids, off, scoring)


@gpu
def test_tokens_outside_every_sequence_and_repeated_ids():
    l, ids, _ = make(50, 12, 3, 1, torch.float32, 12)
    ids[:, 1] = ids[:, 0]                      # the same expert twice
    ids[7] = [-1, 99, -5]                      # ids that name nothing
    ids[9] = [2, 99, -1]
    check(l, ids, [5, 5, 17, 40, 40])          # tokens 0 .. 4 and 40 .. 49 in no sequence
    check(l, ids, [0, 0])                      # nothing at all
    check(l, ids, [50, 50, 50])


@gpu
def test_no_tokens():
    r = moe.make_router(12, 2)
    loss, counts, tokens, probs, _ = run(torch.zeros(0, 12, device="cuda"), np.zeros((0, 2), np.int32), [0, 0, 0],
                                         "softmax", router=r)
    assert not loss.any() and not counts.any() and not tokens.any() and not probs.any()


@gpu
def test_malformed_offsets_stay_in_bounds():
    """Offsets that descend or leave [0, M]: some result, nothing past the buffers (run() looks)."""
    l, ids, _ = make(100, 12, 2, 1, torch.float32, 13)
    for off in ([0, 90, 20, 100], [-5, 30, 200, 1000], [100, 0, 100, 0], [1 << 30, -(1 << 30), 5, 50]):
        run(l, ids, off, "softmax", dloss=np.ones(3, np.float32))


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_accumulate(dtype):
    """The gradient is added in one rounding; tokens that do not count stay as they are."""
    l, ids, off = make(61, 20, 2, 3, dtype, 14)
    ids[4] = -1
    off[0] = 2
    dloss = np.array([1.0, 2.0, 3.0], np.float32)
    base = torch.randn(61, 20, device="cuda").to(dtype) * 0.01
    base[0, 0] = -0.0
    *_, plain = run(l, ids, off, "softmax", dloss=dloss)
    *_, got = run(l, ids, off, "softmax", dloss=dloss, accumulate=True, dl=base.clone())
    same = torch.tensor([0, 1, 4], device="cuda")
    assert torch.equal(got[same].view(torch.uint8), base[same].view(torch.uint8))
    assert not plain[same].any()
    if dtype == torch.float32:
        assert torch.equal(got, base + plain)
    else:   # the addend itself is float32 there: a step of the sum, half a step of the addend
        err = (got.double() - base.double() - plain.double()).abs()
        assert (err <= 2.0 ** -8 * got.double().abs() + 2.0 ** -8 * plain.double().abs() + 1e-37).all()


@gpu
def test_same_bits_again_and_on_another_stream():
    l, ids, off = make(3000, 96, 8, 5, torch.bfloat16, 15)
    dloss = np.ones(5, np.float32)
    a = run(l, ids, off, "sigmoid", dloss=dloss)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        b = run(l, ids, off, "sigmoid", dloss=dloss)
    torch.cuda.synchronize()
    for x, y in zip(a[:4], b[:4]):
        assert np.array_equal(x, y)
    assert torch.equal(a[4], b[4])


@gpu
def test_sequences_do_not_see_each_other():
    """A sequence's results are its own, whatever stands beside it."""
    l, ids, off = make(300, 32, 4, 3, torch.float32, 16)
    off = [0, 90, 200, 300]
    a = run(l, ids, off, "softmax", dloss=np.ones(3, np.float32))
    l2 = l.clone()
    l2[:90] = float("nan")
    b = run(l2, ids, off, "softmax", dloss=np.ones(3, np.float32))
    for x, y in zip(a[:4], b[:4]):
        assert np.array_equal(x[1:], y[1:])
    assert torch.equal(a[4][90:], b[4][90:])


@gpu
def test_many_empty_sequences():
    """More sequences than one workgroup clears by itself, nearly all of them empty."""
    l, ids, _ = make(50, 16, 2, 1, torch.float32, 17)
    off = np.sort(np.concatenate([[0], np.repeat([3, 20, 47], 300), [50]])).astype(np.int32)
    check(l, ids, off)
    l, ids, _ = make(700, 16, 2, 1, torch.bfloat16, 18)
    off = np.sort(np.concatenate([[0], np.repeat([1, 2, 350, 699], 200), [700]])).astype(np.int32)
    check(l, ids, off, "sigmoid")


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [64, 128])
def test_operands_off_the_wide_alignment(dtype, E):
    """Logits, gradient or counts aligned to their elements only, each against 64 bits.  A lane then holds
    other experts of the row, so a row's sum is added in another order: each result is within the bounds of
    `balance` (whose sum of up to 38 steps holds for any order), and two need not be the same bits."""
    l, ids, _ = make(40, E, 3, 1, dtype, 19)
    dloss = np.ones(1, np.float32)
    lh = l.float().cpu().numpy().astype(np.float64)
    rl, rc, rt, rp, tol = balance(lh, ids, [0, 40], "softmax")
    tol = tol + rp * U24 * (48 / 4 + 10) + 1e-37
    rd, bound = balance_backward(lh, ids, [0, 40], "softmax", rc, rt, dloss.astype(np.float64))
    bound = bound + (2.0 ** -8 if dtype == torch.bfloat16 else U24) * np.abs(rd)

    def right(result):
        loss, counts, tokens, probs, dl = result
        assert np.array_equal(counts, rc) and np.array_equal(tokens, rt)
        assert np.all(np.abs(probs - rp) <= tol)
        assert np.all(np.abs(loss - rl) <= E / (3 * rt) * (rc * tol).sum(1) + 2 * U24 * np.abs(rl))
        gradient(dl)

    def gradient(dl):
        assert np.all(np.abs(dl.float().cpu().numpy().astype(np.float64) - rd) <= bound)

    def shifted(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        v = b[1:].view(t.shape)
        v.copy_(t)
        return v
    want = run(l, ids, [0, 40], "softmax", dloss=dloss)
    right(want)
    off = shifted(l)
    first = run(off, ids, [0, 40], "softmax", dloss=dloss)
    right(first)
    again = run(off, ids, [0, 40], "softmax", dloss=dloss)     # the same call again: the same bits
    assert all(np.array_equal(a, b) for a, b in zip(first[:4], again[:4])) and torch.equal(first[4], again[4])
    gradient(run(l, ids, [0, 40], "softmax", dloss=dloss, dl=shifted(torch.empty_like(l)))[4])
    r = moe.make_router(E, 3)
    i32 = torch.from_numpy(want[1].astype(np.int32)).cuda()
    dl = torch.empty_like(l)
    moe.moe_balance_loss_backward(r, l, torch.from_numpy(ids).cuda(), shifted(i32),
                                  torch.from_numpy(want[2].astype(np.int32)).cuda(), torch.ones(1, device="cuda"), dl)
    gradient(dl)


@gpu
def test_more_sequences_than_one_launch_takes():
    """65536 sequences of 2048 experts: 2^33 threads' worth of sums; three sequences hold the tokens."""
    E, topk, S, M, full = 2048, 2, 65536, 24, [0, 20000, 65535]
    l, ids, _ = make(M, E, topk, 1, torch.bfloat16, 23)
    ends = [0, 9, 10, M]
    off = np.zeros(S + 1, np.int32)
    for i, s in enumerate(full):
        off[s + 1:] = ends[i + 1]
    lh = l.float().cpu().numpy().astype(np.float64)
    rl, rc, rt, rp, tol = balance(lh, ids, ends, "softmax")
    tol = tol + rp * U24 * (48 / 4 + 10) + 1e-37
    r = moe.make_router(E, topk)
    d_ids, d_off = torch.from_numpy(ids).cuda(), torch.from_numpy(off).cuda()
    loss, tokens = torch.full((S,), 7.0, device="cuda"), torch.full((S,), 77, dtype=torch.int32, device="cuda")
    counts = torch.full((S, E), 77, dtype=torch.int32, device="cuda")
    probs = torch.full((S, E), 7.0, device="cuda")
    moe.moe_balance_loss(r, l, d_ids, loss, counts, tokens, probs, moe.allocate_balance_workspace(r, M, S),
                         seq_offsets=d_off)
    assert np.array_equal(counts[full].cpu().numpy(), rc) and np.array_equal(tokens[full].cpu().numpy(), rt)
    assert np.all(np.abs(probs[full].double().cpu().numpy() - rp) <= tol)
    per = E / (topk * rt)
    assert np.all(np.abs(loss[full].double().cpu().numpy() - rl) <= per * (rc * tol).sum(1) + 2 * U24 * np.abs(rl))
    dl = torch.full_like(l, float("nan"))
    moe.moe_balance_loss_backward(r, l, d_ids, counts, tokens, torch.ones(S, device="cuda"), dl, seq_offsets=d_off)
    rd, bound = balance_backward(lh, ids, ends, "softmax", rc, rt, np.ones(3))
    assert np.all(np.abs(dl.double().cpu().numpy() - rd) <= bound + 2.0 ** -8 * np.abs(rd))
    for t in (loss, tokens, counts, probs):    # the empty ones
        t[full] = 0
        assert not t.any()


@gpu
def test_more_tokens_than_one_launch_takes():
    """2^25 + 3 tokens of two experts: the ends of the gradient, and the sums."""
    M = (1 << 25) + 3
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    l = torch.randn(M, 2, generator=g, device="cuda")
    ids = (torch.rand(M, 1, generator=g, device="cuda") < 0.3).to(torch.int32)
    r = moe.make_router(2, 1)
    loss, tokens = torch.empty(1, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    counts, probs = torch.empty(1, 2, dtype=torch.int32, device="cuda"), torch.empty(1, 2, device="cuda")
    moe.moe_balance_loss(r, l, ids, loss, counts, tokens, probs, moe.allocate_balance_workspace(r, M))
    one = ids.sum(dtype=torch.int64).item()
    assert tokens.item() == M and counts[0].tolist() == [M - one, one]
    mean = torch.softmax(l.double(), 1).mean(0)
    # 56 half steps of a score, and of a chunk's 4096 tokens 4096 / 4 + 8 more
    assert ((probs[0].double() - mean).abs() <= (80 + 4096 / 4 + 10) * U24 * mean).all()
    dl = torch.empty_like(l)
    moe.moe_balance_loss_backward(r, l, ids, counts, tokens, torch.ones(1, device="cuda"), dl)
    for s in (slice(0, 5), slice((1 << 25) - 4, M)):
        p = torch.softmax(l[s].double(), 1)
        c = counts[0].double()
        want = 2.0 / M ** 2 * p * (c - (c * p).sum(1, keepdim=True))
        assert ((dl[s].double() - want).abs() <= 300 * U24 * (2.0 / M ** 2 * p * (c[0] - c[1]).abs())).all()

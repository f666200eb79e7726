"""64-bit references of the balance loss, the block's norms and the
orthogonalised update, written from their formulas, with the magnitudes that
float32 rounding errors scale with."""
import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)
U24 = 2.0 ** -24          # half a step of float32


# -------------------------------------------------------------- balance ----

def scores(l, scoring):
    """(p [M, E], tol [M, E]): the scores of logits l (float64 [M, E], NaN and
    -inf never chosen) and the error float32 arithmetic may leave in them.

    An exponential's argument is a difference times a constant, 3 roundings
    relative to its size |x|, and as many more for the sum's terms; the
    exponential, the quotient and a sum of up to 32 + 6 steps add at most 56
    half steps.  A bias is added in float32, one rounding of |l|."""
    ok = ~np.isnan(l) & (l > -np.inf)
    z = np.where(ok, np.clip(np.where(ok, l, 0.0), -FLT_MAX, FLT_MAX), 0.0)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        top = np.where(ok, z, -np.inf).max(1, keepdims=True)
        top = np.where(np.isfinite(top), top, 0.0)
        if scoring == "softmax":
            x = z - top
            e = np.where(ok, np.exp(x), 0.0)
        else:
            # sigmoid over the sum of sigmoids, both times e^-min(top, 0)
            m = np.minimum(top, 0.0)
            x = np.abs(z) + np.abs(m)
            e = np.where(ok, np.exp(np.where(z > 0, 0.0, z - m)) / (1.0 + np.exp(-np.abs(z))), 0.0)
        s = e.sum(1, keepdims=True)
        p = np.where(s > 0, e / np.where(s > 0, s, 1.0), 0.0)
        size = np.where(p > 0, np.minimum(np.abs(x), 200.0) + np.minimum(np.abs(z), 1e6), 0.0)
    mean = (p * size).sum(1, keepdims=True)
    return p, p * U24 * (3 * size + 3 * mean + 56) + 1e-37


def balance(l, ids, offsets, scoring):
    """loss, counts, tokens, probs and their tolerances (but for the sum over tokens)."""
    E, topk = l.shape[1], ids.shape[1]
    p, tol = scores(l, scoring)
    S = len(offsets) - 1
    loss, counts, tokens = np.zeros(S), np.zeros((S, E), np.int64), np.zeros(S, np.int64)
    probs, ptol = np.zeros((S, E)), np.zeros((S, E))
    for s in range(S):
        for t in range(offsets[s], offsets[s + 1]):
            good = [i for i in ids[t] if 0 <= i < E]
            if not good:
                continue
            tokens[s] += 1
            for i in good:
                counts[s, i] += 1
            probs[s] += p[t]
            ptol[s] += tol[t]
        if tokens[s]:
            probs[s] /= tokens[s]
            ptol[s] /= tokens[s]
            loss[s] = E / (topk * tokens[s]) * (counts[s] * probs[s]).sum()
    return loss, counts, tokens, probs, ptol


def balance_backward(l, ids, offsets, scoring, counts, tokens, dloss):
    """(dlogits, tolerance).  The count of the token's best expert is taken off
    all counts; what is left enters a sum of E terms (44 half steps)."""
    M, E = l.shape
    topk = ids.shape[1]
    p, tol = scores(l, scoring)
    d, bound = np.zeros((M, E)), np.zeros((M, E))
    for s in range(len(offsets) - 1):
        for t in range(offsets[s], offsets[s + 1]):
            if not any(0 <= i < E for i in ids[t]) or not (p[t] > 0).any():
                continue
            k = abs(dloss[s]) * E / (topk * float(tokens[s]) ** 2)
            ok = ~np.isnan(l[t]) & (l[t] > -np.inf)
            z = np.clip(np.where(ok, l[t], 0.0), -FLT_MAX, FLT_MAX)
            best = np.where(ok, z, -np.inf)
            ref = counts[s][np.flatnonzero(best == best.max())[-1]]
            c = (counts[s] - ref).astype(np.float64)
            dot = (c * p[t]).sum()
            inner = c - dot
            err_dot = (tol[t] * np.abs(c)).sum() + 44 * U24 * (p[t] * np.abs(c)).sum()
            v = p[t] * inner
            e = tol[t] * np.abs(inner) + p[t] * (err_dot + 2 * U24 * np.abs(c)) + 8 * U24 * np.abs(v)
            if scoring == "sigmoid":
                with np.errstate(over="ignore"):
                    f = 1.0 / (1.0 + np.exp(z))
                v = v * f
                e = e * f + np.abs(v) * U24 * (3 * np.minimum(np.abs(z), 200.0) + 8)
            d[t] = np.where(ok, v, 0.0) * (dloss[s] * E / (topk * float(tokens[s]) ** 2))
            bound[t] = np.where(ok, e, 0.0) * k + 1e-37
    return d, bound


# ----------------------------------------------------------------- norm ----
# Row sums of K float32 terms: at most 16 terms a thread, 6 steps over a wave
# and 16 over its waves, so 38 half steps, 20 of them left in a root.

def norm_forward(x, block, w_post, gate, w_pre, eps, scale):
    """x_out, h and the errors of float32 arithmetic before their rounding;
    gate broadcast to [M, K] or 1."""
    K = x.shape[1]
    if block is None:
        y, ey = x, np.zeros_like(x)
    else:
        u = block
        if w_post is not None:
            u = block / np.sqrt((block ** 2).mean(1, keepdims=True) + eps) * w_post
        u = gate * u
        y = scale * x + u
        ey = U24 * (3 * np.abs(scale * x) + 30 * np.abs(u))
    if w_pre is None:
        return y, ey, None, None
    r = 1.0 / np.sqrt((y ** 2).mean(1, keepdims=True) + eps)
    h = y * r * w_pre
    # an error in y reaches h directly and through the mean square
    through = (np.abs(y) * ey).mean(1, keepdims=True) * r * r
    return y, ey, h, np.abs(w_pre) * r * (ey + np.abs(y) * through) + 30 * U24 * np.abs(h)


def norm_backward(x, block, w_post, gate, w_pre, dx_out, dh, eps, scale):
    """dict of (gradient, error of float32 arithmetic), from the stored x; sums
    over tokens: at most 100 half steps besides the terms' own errors (parts of
    a row each, their sum over the workgroups in 16 waves)."""
    out = {}
    d, ed = dx_out, 2 * U24 * np.abs(dx_out)
    if w_pre is not None:
        r = 1.0 / np.sqrt((x ** 2).mean(1, keepdims=True) + eps)
        n, g = x * r, w_pre * dh
        d = dx_out + r * (g - n * (g * n).mean(1, keepdims=True))
        ed = U24 * (4 * np.abs(dx_out) + r * (30 * np.abs(g) + 90 * np.abs(n) * (np.abs(g * n)).mean(1, keepdims=True)))
        t = np.abs(dh * n)
        out["dw_pre"] = ((dh * n).sum(0), (30 + 100) * U24 * t.sum(0))
    if block is None:
        out["dx"] = (d, ed)
        return out
    out["dx"] = (scale * d, abs(scale) * (ed + U24 * np.abs(d)))
    rb = 1.0 if w_post is None else 1.0 / np.sqrt((block ** 2).mean(1, keepdims=True) + eps)
    w = 1.0 if w_post is None else w_post
    n = block * rb
    t, et = d * w * n, (ed + 30 * U24 * np.abs(d)) * np.abs(w * n)
    out["dgate_channel"] = (t.sum(0), et.sum(0) + 100 * U24 * np.abs(t).sum(0))
    out["dgate_token"] = (t.sum(1), et.sum(1) + 40 * U24 * np.abs(t).sum(1))
    g, eg = gate * d, np.abs(gate) * (ed + 4 * U24 * np.abs(d))
    if w_post is None:
        out["dblock"] = (g, eg)
        return out
    out["dw_post"] = ((g * n).sum(0), ((eg + 30 * U24 * np.abs(g)) * np.abs(n) + 100 * U24 * np.abs(g * n)).sum(0))
    wd, ewd = g * w, eg * np.abs(w) + U24 * np.abs(g * w)
    m = (wd * n).mean(1, keepdims=True)
    em = (ewd * np.abs(n)).mean(1, keepdims=True) + 70 * U24 * np.abs(wd * n).mean(1, keepdims=True)
    out["dblock"] = (rb * (wd - n * m), rb * (ewd + 30 * U24 * np.abs(wd) + np.abs(n) * (em + 50 * U24 * np.abs(m))))
    return out


# ---------------------------------------------------------------- ortho ----

def ortho(u, coef, eps):
    """Newton-Schulz steps on one matrix, in float64."""
    x = u if u.shape[0] >= u.shape[1] else u.T
    x = x / (np.sqrt((x ** 2).sum()) + eps)
    for a, b, c in coef:
        g = x.T @ x
        x = a * x + x @ (b * g + c * (g @ g))
    return x if u.shape[0] >= u.shape[1] else x.T


def ortho_rounded(u, coef, eps):
    """The same with the kernels' roundings: float16 operands (two pieces of X
    for a X), the diagonals of A and B apart, float64 elsewhere."""
    def f16(v, bits):
        return (v * 2.0 ** bits).astype(np.float16).astype(np.float64) * 2.0 ** -bits
    x = u if u.shape[0] >= u.shape[1] else u.T
    x = x / (np.sqrt((x ** 2).sum()) + eps)
    for a, b, c in coef:
        h = f16(x, 12)
        x = h + f16((x - h) * 2048, 12) / 2048
        g = h.T @ h
        d = np.diag(g).copy()
        o = f16(g - np.diag(d), 12)
        full = o + np.diag(d)
        q = b * full + c * (full @ full)
        e = np.diag(q).copy()
        x = x * (a + e) + h @ f16(q - np.diag(e), 12)
    return x if u.shape[0] >= u.shape[1] else x.T

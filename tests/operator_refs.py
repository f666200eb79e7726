"""Plain 64-bit references of the router, layer and adapter operators, written
from their definitions with loops over tokens (numpy, no HIP)."""
import math

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)


def route_scores(logits, bias, scoring, bias_kind):
    """Per token: the logits that compete (-inf: out) and the scores, float64.
    scoring: "softmax" | "sigmoid"; bias_kind: "none" | "logit" | "select"."""
    l = np.asarray(logits, np.float64).copy()
    if bias_kind == "logit":
        l = l + np.asarray(bias, np.float64)[None, :]
    out = np.isnan(l) | np.isneginf(l)
    l = np.where(out, -np.inf, np.clip(np.where(out, 0.0, l), -FLT_MAX, FLT_MAX))
    s = np.zeros_like(l)
    for t in range(l.shape[0]):
        ok = ~out[t]
        if not ok.any():
            continue
        if scoring == "softmax":
            e = np.exp(l[t, ok] - l[t, ok].max())
            s[t, ok] = e / e.sum()
        else:
            with np.errstate(over="ignore"):
                s[t, ok] = 1.0 / (1.0 + np.exp(-l[t, ok]))
    return l, s


def route_topk(logits, topk, scoring="softmax", bias=None, bias_kind="none", renorm=True, scale=1.0, groups=1,
               topk_groups=1):
    """ids int32 [M, topk] (-1: none left) and float64 weights."""
    l, s = route_scores(logits, bias, scoring, bias_kind)
    M, E = l.shape
    ids = np.full((M, topk), -1, np.int32)
    w = np.zeros((M, topk))
    per = E // groups
    for t in range(M):
        key = l[t].copy()
        if bias_kind == "select":
            key = s[t] + np.asarray(bias, np.float64)
        elif groups > 1:
            key = s[t].copy()
        key[np.isneginf(l[t]) | np.isnan(key)] = -np.inf
        if groups > 1:
            gs = []
            for g in range(groups):
                best = sorted((k for k in key[g * per:(g + 1) * per] if k > -np.inf), reverse=True)[:2]
                gs.append(sum(best) if best else -np.inf)
            keep = sorted(range(groups), key=lambda g: (-gs[g], g))[:topk_groups]
            for g in range(groups):
                if g not in keep:
                    key[g * per:(g + 1) * per] = -np.inf
        order = [e for e in sorted(range(E), key=lambda e: (-key[e], e)) if key[e] > -np.inf][:topk]
        n = len(order)
        ids[t, :n] = order
        if n == 0:
            continue
        if scoring == "softmax" and renorm:
            c = np.exp(l[t, order] - l[t, order].max())
        else:
            c = s[t, order]
        if renorm:
            c = c / c.sum() if c.sum() > 0 else np.zeros_like(c)
        w[t, :n] = scale * c
    return ids, w


def route_backward(logits, ids, dw, scoring="softmax", bias=None, bias_kind="none", renorm=True, scale=1.0):
    """d(sum dw w) / d(logits) with the choice held fixed, float64, and per
    element the magnitude of the terms it is the difference of."""
    l, s = route_scores(logits, bias, scoring, bias_kind)
    M, E = l.shape
    d = np.zeros((M, E))
    mag = np.zeros((M, E))
    for t in range(M):
        sel = [(int(e), scale * float(g)) for e, g in zip(ids[t], dw[t]) if 0 <= e < E and l[t, e] > -np.inf]
        if not sel:
            continue
        e = np.array([i for i, _ in sel])
        g = np.array([v for _, v in sel])
        if scoring == "softmax" and renorm:
            p = np.exp(l[t, e] - l[t, e].max())
            p /= p.sum()
            np.add.at(d[t], e, p * (g - (p * g).sum()))
            np.add.at(mag[t], e, p * (abs(g) + abs(p * g).sum()))
        elif scoring == "softmax":
            full = np.zeros(E)
            np.add.at(full, e, g)
            dot = (s[t, e] * g).sum()
            d[t] = s[t] * (full - dot)
            mag[t] = s[t] * (abs(full) + abs(s[t, e] * g).sum())
        else:
            c = s[t, e]
            ds = g
            m = abs(g)
            if renorm:
                S = c.sum()
                ds = (g - (g * c).sum() / S) / S if S > 0 else np.zeros_like(g)
                m = (abs(g) + (abs(g) * c).sum() / S) / S if S > 0 else np.zeros_like(g)
            np.add.at(d[t], e, ds * c * (1 - c))
            np.add.at(mag[t], e, m * c * (1 - c))
    return d, mag

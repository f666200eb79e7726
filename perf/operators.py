"""The router, whole-layer and adapter operators as measured calls.

Each case is one pass through one operator.  With ``own`` false the pass is
written in elementary torch operations (32-bit arithmetic, 64-bit where a
choice between experts hangs on it); with ``own`` true it is the framework's
call.  Sizes are those of the repository's workloads (hidden 256, 4096 and
6144, intermediate 512, 2048 and 8192, 8 / 32 / 64 / 128 / 512 experts, top-2
and top-8) or generic ones near them.
"""
import math

import torch

own = False

DEV = "cuda"
FLT_MAX = torch.finfo(torch.float32).max


def _moe():
    import mixture_experts_expert_align_amd as moe
    return moe


# ------------------------------------------------------------------ cases --

def _route(name, M, E, topk, scoring, bias, renorm, groups=1, topk_groups=1, scale=1.0, dtype="f32",
           train=False, masked=False):
    return dict(name=name, op="route", M=M, E=E, topk=topk, scoring=scoring, bias=bias, renorm=renorm,
                groups=groups, topk_groups=topk_groups, scale=scale, dtype=dtype, train=train, masked=masked)


def _layer(name, M, K, I, E, topk, w, order, shared=0, scoring="softmax", bias="none", renorm=True, groups=1,
           topk_groups=1, scale=1.0):
    return dict(name=name, op="layer", M=M, K=K, I=I, E=E, topk=topk, w=w, order=order, shared=shared,
                scoring=scoring, bias=bias, renorm=renorm, groups=groups, topk_groups=topk_groups, scale=scale)


def _lora(name, R, N, K, G, rank, mix, train):
    return dict(name=name, op="lora", R=R, N=N, K=K, G=G, rank=rank, mix=mix, train=train)


def listed():
    return [
        # the router of one decode step: four tokens, softmax top-8 of 64
        _route("route_decode", 4, 64, 8, "softmax", "none", True),
        # the router of a long prompt on a layer of 512 experts: sigmoid scores, a load-balancing
        # bias that only selects, experts in 16 groups of which 4 stay, bf16 logits
        _route("route_groups", 4096, 512, 8, "sigmoid", "select", True, 16, 4, 2.5, "bf16"),
        # training: 8192 tokens over 128 experts, forward and the logits' gradient
        _route("route_train", 8192, 128, 8, "softmax", "logit", True, train=True),
        # a small layer for a handful of tokens: launch latency
        _layer("layer_tiny", 7, 256, 512, 8, 2, "bf16", "halves"),
        # one decode step of four sequences on a large bf16 layer
        _layer("layer_decode", 4, 4096, 8192, 64, 8, "bf16", "halves"),
        # decode of 16 sequences, MXFP8 weights, one shared expert
        _layer("layer_mxfp8", 16, 6144, 2048, 32, 8, "mxfp8", "interleave16", shared=1, scoring="sigmoid",
               bias="select", scale=2.5),
        # a decode batch of 61 sequences: most experts hold several rows
        _layer("layer_batch", 61, 4096, 1024, 128, 8, "bf16", "halves", shared=2, renorm=False),
        # decode of 13 requests, each with an adapter of its own or none
        _lora("lora_decode", 13, 4096, 4096, 32, 16, "mixed", False),
        # a mixed batch: 300 rows of many requests in any order
        _lora("lora_mixed", 300, 4096, 4096, 48, 32, "mixed", False),
        # long prompts of a few requests, one after another
        _lora("lora_prefill", 8192, 4096, 4096, 8, 16, "runs", False),
        # one training step of four adapters of rank 64 on a wide projection
        _lora("lora_train", 8192, 4096, 6144, 4, 64, "runs", True),
        # a short training step, odd row count, rank 8
        _lora("lora_train_short", 1001, 2048, 2048, 3, 8, "mixed", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "layer", "layer", "lora", "lora"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        per = rng.choice([8, 12, 16, 33, 64]) if groups > 1 else rng.choice([8, 24, 60, 64, 128, 160, 256, 512])
        E = groups * per
        tg = rng.randint(2, groups) if groups > 1 else 1
        topk = rng.randint(1, min(8, tg * per))
        return _route(None, _log(rng, 1, 8192), E, topk, rng.choice(["softmax", "sigmoid"]),
                      rng.choice(["none", "logit", "select"]), rng.random() < 0.6, groups, tg,
                      rng.choice([1.0, 2.5]), rng.choice(["f32", "bf16"]), rng.random() < 0.4, rng.random() < 0.3)
    if op == "layer":
        w = rng.choice(["bf16", "mxfp8"])
        return _layer(None, _log(rng, 1, 64), 128 * _log(rng, 1, 48), 128 * _log(rng, 1, 16),
                      rng.choice([4, 8, 16, 31, 32, 64]), rng.randint(1, 4), w,
                      rng.choice(["halves", "interleave16"]), rng.choice([0, 0, 1, 2]),
                      rng.choice(["softmax", "sigmoid"]), rng.choice(["none", "logit", "select"]),
                      rng.random() < 0.6, scale=rng.choice([1.0, 2.5]))
    train = rng.random() < 0.4
    return _lora(None, _log(rng, 1, 6000), 64 * _log(rng, 2, 64), 64 * _log(rng, 2, 64), _log(rng, 1, 64),
                 8 * rng.randint(1, 8), rng.choice(["mixed", "runs"]), train)


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    if dtype == torch.float32 or math.prod(shape) < 1 << 24:
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)
    out = torch.empty(*shape, device=DEV, dtype=dtype)
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        flat[i:i + step].normal_(0.0, std, generator=g)
    return out


def _mx_weights(g, *shape, std):
    """E4M3 codes and one UE8M0 scale per 32: codes of N(0, 1) * 2^6 blocks whose
    exponents differ by block, so decoded weights have deviation about std."""
    codes = torch.empty(*shape, device=DEV, dtype=torch.uint8)
    for i in range(shape[0]):
        v = torch.randn(*shape[1:], generator=g, device=DEV).mul_(64.0).clamp_(-448.0, 448.0)
        codes[i] = v.to(torch.float8_e4m3fn).view(torch.uint8)
    base = 127 - 6 + round(math.log2(std))
    scales = torch.randint(base - 1, base + 2, shape[:-1] + (shape[-1] // 32,), generator=g, device=DEV)
    return codes, scales.to(torch.uint8)


def _router(case):
    moe = _moe()
    return moe.make_router(
        case["E"], case["topk"],
        scoring=moe.ROUTE_SOFTMAX if case["scoring"] == "softmax" else moe.ROUTE_SIGMOID,
        bias_kind={"none": moe.BIAS_NONE, "logit": moe.BIAS_LOGIT, "select": moe.BIAS_SELECT}[case["bias"]],
        renormalize=case["renorm"], scale=case["scale"], groups=case["groups"], topk_groups=case["topk_groups"])


def _adapters(case, g):
    R, G = case["R"], case["G"]
    if case["mix"] == "mixed":
        return torch.randint(-1, G, (R,), generator=g, device=DEV, dtype=torch.int32)
    # runs: the requests' rows one after another, the last tenth without an adapter
    cut = torch.sort(torch.randint(0, max(R - R // 10, 1), (G - 1,), generator=g, device=DEV)).values
    row = torch.arange(R, device=DEV)
    ids = torch.searchsorted(cut, row, right=True).to(torch.int32)
    return torch.where(row < R - R // 10, ids, torch.full_like(ids, -1))


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "route":
        M, E, k = case["M"], case["E"], case["topk"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s["logits"] = _normal(g, M, E, dtype=dt)
        if case["masked"]:
            s["logits"][torch.rand(M, E, generator=g, device=DEV) < 0.5] = float("-inf")
        s["bias"] = None if case["bias"] == "none" else _normal(g, E, std=0.25, dtype=torch.float32)
        if case["train"]:
            s["dw"] = _normal(g, M, k, dtype=torch.float32)
        if own:
            s["router"] = _router(case)
            s["ids"] = torch.empty(M, k, dtype=torch.int32, device=DEV)
            s["wts"] = torch.empty(M, k, dtype=torch.float32, device=DEV)
            if case["train"]:
                s["dl"] = torch.empty_like(s["logits"])
    elif case["op"] == "layer":
        M, K, I, E, S = case["M"], case["K"], case["I"], case["E"], case["shared"]
        s["x"] = _normal(g, M, K)
        s["wr"] = _normal(g, E, K, std=K ** -0.5)
        s["bias"] = None if case["bias"] == "none" else _normal(g, E, std=0.25, dtype=torch.float32)
        if case["w"] == "bf16":
            s["w1"], s["s1"] = _normal(g, E + S, 2 * I, K, std=K ** -0.5), None
            s["w2"], s["s2"] = _normal(g, E + S, K, I, std=I ** -0.5), None
        else:
            s["w1"], s["s1"] = _mx_weights(g, E + S, 2 * I, K, std=K ** -0.5)
            s["w2"], s["s2"] = _mx_weights(g, E + S, K, I, std=I ** -0.5)
        if own:
            moe = _moe()
            s["plan"] = moe.moe_layer_plan_init(moe.make_layer_problem(
                M, K, I, _router(case), shared_experts=S,
                w_dtype=moe.W_BF16 if case["w"] == "bf16" else moe.W_MXFP8,
                w1_order=moe.W1_HALVES if case["order"] == "halves" else moe.W1_INTERLEAVE16))
            s["ws"] = moe.allocate_layer_workspace(s["plan"], DEV)
            s["out"] = torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
            s["ids"] = torch.empty(M, case["topk"], dtype=torch.int32, device=DEV)
            s["wts"] = torch.empty(M, case["topk"], dtype=torch.float32, device=DEV)
    else:
        R, N, K, G, r = case["R"], case["N"], case["K"], case["G"], case["rank"]
        s["x"] = _normal(g, R, K)
        s["w"] = _normal(g, N, K, std=K ** -0.5)
        s["a"] = _normal(g, G, r, K, std=K ** -0.5)
        s["b"] = _normal(g, G, N, r, std=0.5 * r ** -0.5)
        s["scale"] = torch.rand(G, generator=g, device=DEV) + 0.5
        s["adapter"] = _adapters(case, g)
        if case["train"]:
            s["dy"] = _normal(g, R, N)
        if own:
            moe = _moe()
            s["y"] = torch.empty(R, N, dtype=torch.bfloat16, device=DEV)
            s["low"] = moe.allocate_lora_low(R, r, DEV)
            if case["train"]:
                s["dx"] = torch.empty(R, K, dtype=torch.bfloat16, device=DEV)
                s["low_dy"] = moe.allocate_lora_low(R, r, DEV)
                s["da"] = torch.empty(G, r, K, dtype=torch.float32, device=DEV)
                s["db"] = torch.empty(G, N, r, dtype=torch.float32, device=DEV)
                s["ws"] = moe.allocate_lora_workspace(R, N, K, G, r, DEV)
    return s


# -------------------------------------------------------------- the passes --

def _plain_route(case, logits, bias):
    """ids, weights and what the gradient needs, from logits of any type."""
    E, k = case["E"], case["topk"]
    l = logits.double()
    if case["bias"] == "logit":
        l = l + bias.double()
    ok = ~torch.isnan(l) & (l > float("-inf"))
    l = torch.where(ok, l.clamp(-FLT_MAX, FLT_MAX), torch.full_like(l, float("-inf")))
    if case["scoring"] == "softmax":
        top = l.amax(1, keepdim=True)
        e = torch.where(ok, torch.exp(l - torch.where(top > float("-inf"), top, torch.zeros_like(top))),
                        torch.zeros_like(l))
        score = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        score = torch.where(ok, 1.0 / (1.0 + torch.exp(-l)), torch.zeros_like(l))
    if case["bias"] == "select":
        key = score + bias.double()
    else:
        key = score if case["groups"] > 1 else l
    key = torch.where(ok & ~torch.isnan(key), key, torch.full_like(key, float("-inf")))
    if case["groups"] > 1:
        gk = key.view(-1, case["groups"], E // case["groups"])
        best = torch.sort(gk, dim=2, descending=True).values[:, :, :2]
        gs = torch.where((best > float("-inf")).any(2),
                         torch.where(best > float("-inf"), best, torch.zeros_like(best)).sum(2),
                         torch.full_like(best[:, :, 0], float("-inf")))
        keep = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        on = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, keep, True)
        key = torch.where(on[:, :, None], gk, torch.full_like(gk, float("-inf"))).reshape(-1, E)
    sk, order = torch.sort(key, dim=1, descending=True, stable=True)
    have = sk[:, :k] > float("-inf")
    ids = torch.where(have, order[:, :k], torch.full_like(order[:, :k], -1))
    chosen = torch.where(have, torch.gather(score, 1, order[:, :k]), torch.zeros_like(sk[:, :k]))
    w = chosen
    total = chosen.sum(1, keepdim=True)
    if case["renorm"]:
        w = torch.where(total > 0, chosen / torch.where(total > 0, total, torch.ones_like(total)),
                        torch.zeros_like(chosen))
    return ids.to(torch.int32), (w * case["scale"]).float(), score.float(), chosen.float()


def _plain_route_grad(case, ids, score, chosen, dw, dtype):
    have = ids >= 0
    dw = torch.where(have, dw, torch.zeros_like(dw)) * case["scale"]
    total = chosen.sum(1, keepdim=True)
    if case["renorm"]:
        inv = torch.where(total > 0, 1.0 / total, torch.zeros_like(total))
        dc = (dw - (dw * chosen).sum(1, keepdim=True) * inv) * inv
    else:
        dc = dw
    ds = torch.zeros_like(score).scatter_add_(1, ids.clamp_min(0).long(), torch.where(have, dc, torch.zeros_like(dc)))
    if case["scoring"] == "softmax":
        dl = score * (ds - (ds * score).sum(1, keepdim=True))
    else:
        dl = ds * score * (1.0 - score)
    return dl.to(dtype)


def _expert_rows(w, scales, e):
    """One expert's weights in 32 bits (e: an index on the device)."""
    c = w.index_select(0, e)[0]
    if scales is None:
        return c.float()
    f = scales.index_select(0, e)[0].float()
    v = c.view(torch.float8_e4m3fn).float()
    return (v.view(v.shape[0], -1, 32) * torch.exp2(f - 127.0)[:, :, None]).view(v.shape)


def _gate_up(h, I, order):
    if order == "halves":
        return h[..., :I], h[..., I:]
    b = h.view(*h.shape[:-1], I // 16, 2, 16)
    return b[..., 0, :].reshape(*h.shape[:-1], I), b[..., 1, :].reshape(*h.shape[:-1], I)


def _plain_layer(case, s):
    M, I, E = case["M"], case["I"], case["E"]
    logits = s["x"].double() @ s["wr"].double().t()
    ids, wts, _, _ = _plain_route(case, logits, s["bias"])
    x = s["x"].float()
    out = torch.zeros(M, case["K"], device=DEV)

    def ffn(e, rows):
        gate, up = _gate_up(rows @ _expert_rows(s["w1"], s["s1"], e).t(), I, case["order"])
        z = gate / (1.0 + torch.exp(-gate)) * up
        return z @ _expert_rows(s["w2"], s["s2"], e).t()

    flat = ids.reshape(-1)
    if flat.numel() <= E:
        for i in range(flat.numel()):
            t = i // case["topk"]
            y = ffn(flat[i:i + 1].clamp_min(0).long(), x[t:t + 1])
            out[t] += torch.where(flat[i] >= 0, wts.view(-1)[i], torch.zeros((), device=DEV)) * y[0]
    else:
        for e in range(E):
            we = torch.where(ids == e, wts, torch.zeros_like(wts)).sum(1, keepdim=True)
            out += we * ffn(torch.full((1,), e, dtype=torch.long, device=DEV), x)
    for j in range(case["shared"]):
        out += ffn(torch.full((1,), E + j, dtype=torch.long, device=DEV), x)
    return {"out": out.to(torch.bfloat16), "ids": ids, "weights": wts}


def _plain_lora(case, s):
    x, w = s["x"].float(), s["w"].float()
    G = case["G"]
    ad = s["adapter"]
    if case["R"] <= 64 and not case["train"]:
        g = ad.clamp_min(0).long()
        sc = torch.where(ad >= 0, s["scale"][g], torch.zeros_like(s["scale"][g]))
        low = (s["a"].float()[g] * x[:, None, :]).sum(2) * sc[:, None]
        return {"y": (x @ w.t() + (s["b"].float()[g] * low[:, None, :]).sum(2)).to(torch.bfloat16)}
    y = x @ w.t()
    if case["train"]:
        dy = s["dy"].float()
        dx = dy @ w
        da, db = [], []
    for g in range(G):
        m = torch.where(ad == g, s["scale"][g], torch.zeros((), device=DEV))[:, None]
        a, b = s["a"][g].float(), s["b"][g].float()
        low = (x @ a.t()) * m
        y += low @ b.t()
        if case["train"]:
            t = (dy @ b) * m
            dx += t @ a
            da.append(t.t() @ x)
            db.append(dy.t() @ low)
    out = {"y": y.to(torch.bfloat16)}
    if case["train"]:
        out.update(dx=dx.to(torch.bfloat16), da=torch.stack(da), db=torch.stack(db))
    return out


def run(state):
    s, case = state, state["case"]
    if own:
        moe = _moe()
        if case["op"] == "route":
            moe.moe_route_topk(s["router"], s["logits"], s["ids"], s["wts"], bias=s["bias"])
            out = {"ids": s["ids"], "weights": s["wts"]}
            if case["train"]:
                moe.moe_route_topk_backward(s["router"], s["logits"], s["ids"], s["dw"], s["dl"], bias=s["bias"])
                out["dlogits"] = s["dl"]
            return out
        if case["op"] == "layer":
            moe.moe_layer_apply(s["plan"], s["x"], s["wr"], s["w1"], s["w2"], s["out"], s["ids"], s["wts"], s["ws"],
                                router_bias=s["bias"], w1_scale=s["s1"], w2_scale=s["s2"])
            return {"out": s["out"], "ids": s["ids"], "weights": s["wts"]}
        moe.moe_lora_forward(s["x"], s["w"], s["a"], s["b"], s["scale"], s["adapter"], s["y"], s["low"])
        out = {"y": s["y"]}
        if case["train"]:
            moe.moe_lora_dgrad(s["dy"], s["w"], s["a"], s["b"], s["scale"], s["adapter"], s["dx"], s["low_dy"])
            moe.moe_lora_wgrad(s["x"], s["dy"], s["low"], s["low_dy"], s["adapter"], s["da"], s["db"], s["ws"])
            out.update(dx=s["dx"], da=s["da"], db=s["db"])
        return out
    if case["op"] == "route":
        ids, wts, score, chosen = _plain_route(case, s["logits"], s["bias"])
        out = {"ids": ids, "weights": wts}
        if case["train"]:
            out["dlogits"] = _plain_route_grad(case, ids, score, chosen, s["dw"], s["logits"].dtype)
        return out
    return _plain_layer(case, s) if case["op"] == "layer" else _plain_lora(case, s)


# ------------------------------------------------------- what a pass needs --

def work(case):
    if case["op"] == "route":
        M, E, k = case["M"], case["E"], case["topk"]
        el = 4 if case["dtype"] == "f32" else 2
        b = M * E * el + M * k * 8 + (0 if case["bias"] == "none" else 4 * E)
        f = M * E * 4
        if case["train"]:
            b += M * k * 4 + M * E * el
            f += M * E * 4
        return {"bytes": b, "flops": f}
    if case["op"] == "layer":
        M, K, I, E, k, S = (case[n] for n in ("M", "K", "I", "E", "topk", "shared"))
        active = E * (1.0 - (1.0 - k / E) ** M) + S     # expected over routings
        per = 2.0 if case["w"] == "bf16" else 1.0 + 1.0 / 32
        b = active * 3 * I * K * per + 2 * E * K + 4 * M * K + 8 * M * k
        return {"bytes": int(b), "flops": int(2 * M * K * E + (M * k + M * S) * 6 * I * K)}
    R, N, K, G, r = (case[n] for n in ("R", "N", "K", "G", "rank"))
    used = G * (1.0 - (1.0 - 1.0 / (G + 1)) ** R) if case["mix"] == "mixed" else min(G, R)
    b = 2 * N * K + 2 * R * (K + N) + 2 * used * r * (K + N) + 4 * R
    f = 2 * R * N * K + 2 * R * r * (K + N)
    if case["train"]:
        b = 2 * N * K + 4 * R * (K + N) + 2 * used * r * (K + N) + 4 * R + 4 * G * r * (K + N)
        f = 2 * f + 2 * R * r * (K + N)
    return {"bytes": int(b), "flops": int(f)}


# ------------------------------------------------------------ in 64 bits ----

def _exact_route(case, logits, bias):
    """Selection and weights by their definition, token rows as a batch: the best
    eligible key is taken topk times."""
    M, E, k = logits.shape[0], case["E"], case["topk"]
    l = logits.to(torch.float64)
    if case["bias"] == "logit":
        l = l + bias.to(torch.float64)
    bad = torch.isnan(l) | torch.isneginf(l)
    l = torch.clamp(l.masked_fill(bad, 0.0), -FLT_MAX, FLT_MAX)
    if case["scoring"] == "softmax":
        m = l.masked_fill(bad, -math.inf).max(1, keepdim=True).values.nan_to_num(neginf=0.0)
        num = torch.exp(l - m).masked_fill(bad, 0.0)
        den = num.sum(1, keepdim=True)
        sc = torch.where(den > 0, num / den, torch.zeros_like(num))
    else:
        sc = torch.sigmoid(l).masked_fill(bad, 0.0)
    key = l if case["bias"] != "select" and case["groups"] == 1 else sc
    if case["bias"] == "select":
        key = sc + bias.to(torch.float64)
    key = key.masked_fill(bad | torch.isnan(key), -math.inf)
    G = case["groups"]
    rows = torch.arange(M, device=DEV)
    if G > 1:
        g = key.reshape(M, G, E // G).clone()
        first, at = g.max(2)
        rest = g.scatter(2, at[:, :, None], -math.inf)
        second = rest.max(2).values
        gs = first + second.masked_fill(torch.isneginf(second), 0.0)
        alive = torch.zeros(M, G, dtype=torch.bool, device=DEV)
        left = gs.clone()
        for _ in range(case["topk_groups"]):
            best = left.max(1, keepdim=True).values
            pick = (left == best).to(torch.int8).argmax(1)
            alive[rows, pick] = True
            left[rows, pick] = -math.inf
        key = g.masked_fill(~alive[:, :, None], -math.inf).reshape(M, E)
    ids, val = [], []
    key = key.clone()
    for _ in range(k):
        best = key.max(1, keepdim=True).values
        pick = (key == best).to(torch.int8).argmax(1)
        got = ~torch.isneginf(best[:, 0])
        ids.append(torch.where(got, pick, torch.full_like(pick, -1)))
        val.append(torch.where(got, sc[rows, pick], torch.zeros_like(best[:, 0])))
        key[rows, pick] = -math.inf
    ids, val = torch.stack(ids, 1), torch.stack(val, 1)
    S = val.sum(1, keepdim=True)
    w = val
    if case["renorm"]:
        w = torch.where(S > 0, val / S, torch.zeros_like(val))
    return ids.to(torch.int32), w * case["scale"], sc, val


def _exact_expert(w, scales, e):
    if scales is None:
        return w[e].to(torch.float64)
    v = w[e].view(torch.float8_e4m3fn).to(torch.float64)
    return v * torch.pow(2.0, scales[e].to(torch.float64) - 127.0).repeat_interleave(32, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        ids, w, sc, val = _exact_route(case, s["logits"], s["bias"])
        out = {"ids": ids, "weights": w}
        if case["train"]:
            # d(sum dw w) / dl through the score's Jacobian, on the chosen entries
            M, E = case["M"], case["E"]
            take = torch.zeros(M, E, dtype=torch.float64, device=DEV)
            have = (ids >= 0).to(torch.float64)
            S = val.sum(1, keepdim=True)
            g = s["dw"].to(torch.float64) * have * case["scale"]
            if case["renorm"]:
                g = torch.where(S > 0, g / S - (g * val).sum(1, keepdim=True) / (S * S), torch.zeros_like(g))
            idx = ids.long().clamp_min(0)
            for j in range(case["topk"]):
                take[torch.arange(M, device=DEV), idx[:, j]] += g[:, j] * have[:, j]
            if case["scoring"] == "softmax":
                out["dlogits"] = sc * take - sc * (sc * take).sum(1, keepdim=True)
            else:
                out["dlogits"] = take * (sc - sc * sc)
        return out
    if case["op"] == "layer":
        M, I, E = case["M"], case["I"], case["E"]
        x = s["x"].to(torch.float64)
        ids, w, _, _ = _exact_route(case, x @ s["wr"].to(torch.float64).t(), s["bias"])
        out = torch.zeros(M, case["K"], dtype=torch.float64, device=DEV)
        for e in range(E + case["shared"]):
            c = torch.ones(M, dtype=torch.float64, device=DEV) if e >= E else (w * (ids == e)).sum(1)
            rows = torch.nonzero((ids == e).any(1) if e < E else c > 0)[:, 0]
            if rows.numel() == 0:
                continue
            h = _exact_expert(s["w1"], s["s1"], e) @ x[rows].t()
            if case["order"] == "halves":
                gate, up = h[:I], h[I:]
            else:
                hb = h.reshape(I // 16, 32, -1)
                gate, up = hb[:, :16].reshape(I, -1), hb[:, 16:].reshape(I, -1)
            z = gate * torch.sigmoid(gate) * up
            out[rows] += c[rows][:, None] * (_exact_expert(s["w2"], s["s2"], e) @ z).t()
        return {"out": out, "ids": ids, "weights": w}
    x, w = s["x"].to(torch.float64), s["w"].to(torch.float64)
    y = torch.matmul(x, w.t())
    train = case["train"]
    if train:
        dy = s["dy"].to(torch.float64)
        dx = torch.matmul(dy, w)
        da = torch.zeros(case["G"], case["rank"], case["K"], dtype=torch.float64, device=DEV)
        db = torch.zeros(case["G"], case["N"], case["rank"], dtype=torch.float64, device=DEV)
    for g in range(case["G"]):
        rows = torch.nonzero(s["adapter"] == g)[:, 0]
        if rows.numel() == 0:
            continue
        c = s["scale"][g].to(torch.float64)
        a, b = s["a"][g].to(torch.float64), s["b"][g].to(torch.float64)
        xr = x[rows]
        y[rows] += c * torch.matmul(torch.matmul(xr, a.t()), b.t())
        if train:
            dr = dy[rows]
            dx[rows] += c * torch.matmul(torch.matmul(dr, b), a)
            da[g] = c * torch.matmul(torch.matmul(dr, b).t(), xr)
            db[g] = c * torch.matmul(dr.t(), torch.matmul(xr, a.t()))
    out = {"y": y}
    if train:
        out.update(dx=dx, da=da, db=db)
    return out

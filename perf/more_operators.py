"""Training a mixture-of-experts block around its products, as measured calls:
the router's balance loss with its gradient, the norms before and after the
block with gate and residual scale, and the orthogonalised update of the
experts' matrices.

Each case is one pass through one operator.  With ``own`` false the pass is
written in elementary torch operations (32-bit arithmetic, 64-bit for sums
over many tokens); with ``own`` true it is the framework's call.  Sizes are
those of the repository's workloads (hidden 256, 2048, 4096 and 6144,
intermediate 512, 1536 and 2048, 8 / 64 / 128 / 512 experts, top-2 and top-8)
or generic ones near them.
"""
import math

import torch

own = False

DEV = "cuda"
FLT_MAX = torch.finfo(torch.float32).max
MUON = (3.4445, -4.7750, 2.0315)


def _moe():
    import mixture_experts_expert_align_amd as moe
    return moe


# ------------------------------------------------------------------ cases --

def _balance(name, M, E, topk, S, scoring, bias, dtype, train, padded=False):
    return dict(name=name, op="balance", M=M, E=E, topk=topk, S=S, scoring=scoring, bias=bias, dtype=dtype,
                train=train, padded=padded)


def _norm(name, M, K, x, gate, post, pre, train, scale=1.0):
    return dict(name=name, op="norm", M=M, K=K, x=x, gate=gate, post=post, pre=pre, train=train, scale=scale)


def _ortho(name, E, N, K, dtype, steps=5, scale=1.0):
    return dict(name=name, op="ortho", E=E, N=N, K=K, dtype=dtype, steps=steps, scale=scale)


def listed():
    return [
        # the loss of one small batch on a layer of 8 experts: launch latency
        _balance("balance_small", 64, 8, 2, 1, "softmax", "none", "f32", True),
        # a training step of 8192 tokens over 128 experts, loss and gradient over the whole batch
        _balance("balance_train", 8192, 128, 8, 1, "softmax", "logit", "f32", True),
        # 13 packed sequences of different lengths and some padding on a layer of 512 experts,
        # sigmoid scores, bf16 logits, a loss per sequence
        _balance("balance_sequences", 16381, 512, 8, 13, "sigmoid", "none", "bf16", True, padded=True),
        # the counts and the loss of a large batch, watched without a gradient
        _balance("balance_watch", 65536, 256, 8, 32, "softmax", "none", "bf16", False),
        # a decode step of four sequences: the block's output into the residual stream, and the
        # next block's input
        _norm("norm_decode", 4, 4096, "bf16", "channel", True, True, False),
        # a long prompt
        _norm("norm_prefill", 8192, 4096, "bf16", "channel", True, True, False, 0.5),
        # training, backward of the same junction, hidden size 6144
        _norm("norm_train", 8192, 6144, "bf16", "channel", True, True, True),
        # training with a float32 residual stream and a gate per token, odd number of tokens
        _norm("norm_train_f32", 1001, 2048, "f32", "token", True, True, True, 0.75),
        # the update of a small layer's second matrices: latency of the dependent products
        _ortho("ortho_small", 8, 256, 512, "f32"),
        # a router's own matrix: 64 experts by the hidden size
        _ortho("ortho_router", 1, 64, 4096, "f32"),
        # the first matrices of 16 experts of 1536 (gate and up), bf16 momentum
        _ortho("ortho_experts", 16, 1536, 4096, "bf16", scale=0.2),
        # the wide projections of a large layer
        _ortho("ortho_large", 8, 4096, 6144, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "norm", "ortho"])
    if op == "balance":
        E = rng.choice([4, 8, 60, 64, 99, 128, 160, 256, 512])
        M = _log(rng, 1, 65536 * 128 // max(E, 128))
        return _balance(None, M, E, rng.randint(1, min(8, E // 2)), rng.choice([1, 1, min(M, 3), min(M, _log(rng, 2, 64))]),
                        rng.choice(["softmax", "sigmoid"]), rng.choice(["none", "logit"]),
                        rng.choice(["f32", "bf16"]), rng.random() < 0.6, rng.random() < 0.3)
    if op == "norm":
        K = 8 * _log(rng, 16, 1024)
        train = rng.random() < 0.5
        M = _log(rng, 1, min(16384, 30_000_000 // K))
        post = rng.random() < 0.8
        return _norm(None, M, K, rng.choice(["f32", "bf16"]), rng.choice(["none", "channel", "token"]), post,
                     not post or rng.random() < 0.8, train, rng.choice([1.0, 0.5]))
    a, b = _log(rng, 16, 3000), _log(rng, 16, 5000)
    m, n = min(a, b), max(a, b)
    most = 8 * (3 * 4096 * 4096 * 6144 + 4096 ** 3)
    E = min(_log(rng, 1, 32), max(1, most // (3 * m * m * n + m ** 3)))
    return _ortho(None, E, a, b, rng.choice(["f32", "bf16"]), rng.choice([5, 5, 3, 6]), rng.choice([1.0, 0.2]))


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "balance":
        M, E, k, S = case["M"], case["E"], case["topk"], case["S"]
        # some experts are liked by every token, as in an unbalanced layer
        s["logits"] = (_normal(g, M, E, dtype=torch.float32)
                       + _normal(g, 1, E, std=0.7, dtype=torch.float32)).to(_type(case["dtype"]))
        s["bias"] = None if case["bias"] == "none" else _normal(g, E, std=0.25, dtype=torch.float32)
        key = s["logits"].float() if s["bias"] is None else s["logits"].float() + s["bias"]
        s["ids"] = torch.topk(key, k, dim=1).indices.to(torch.int32).contiguous()
        if case["padded"]:   # padding tokens take no expert
            s["ids"][torch.rand(M, generator=g, device=DEV) < 0.1] = -1
        cut = torch.sort(torch.randint(0, M + 1, (S - 1,), generator=g, device=DEV)).values
        ends = torch.tensor([0, M], device=DEV)
        s["offsets"] = torch.cat([ends[:1], cut, ends[1:]]).to(torch.int32)
        s["dloss"] = torch.rand(S, generator=g, device=DEV) + 0.5
        if own:
            moe = _moe()
            s["router"] = moe.make_router(
                E, k, scoring=moe.ROUTE_SOFTMAX if case["scoring"] == "softmax" else moe.ROUTE_SIGMOID,
                bias_kind=moe.BIAS_NONE if case["bias"] == "none" else moe.BIAS_LOGIT)
            s["loss"] = torch.empty(S, device=DEV)
            s["counts"] = torch.empty(S, E, dtype=torch.int32, device=DEV)
            s["tokens"] = torch.empty(S, dtype=torch.int32, device=DEV)
            s["probs"] = torch.empty(S, E, device=DEV)
            s["ws"] = moe.allocate_balance_workspace(s["router"], M, S, DEV)
            if case["train"]:
                s["dl"] = torch.empty_like(s["logits"])
    elif case["op"] == "norm":
        M, K, dt = case["M"], case["K"], _type(case["x"])
        # a residual stream whose channels differ in size, a block output of another size
        chan = torch.exp(0.5 * torch.randn(K, generator=g, device=DEV))
        s["x"] = (_normal(g, M, K, dtype=torch.float32) * chan).to(dt)
        s["block"] = _normal(g, M, K, std=0.3)
        s["w_post"] = _normal(g, K, std=0.2, dtype=torch.float32).add_(1.0) if case["post"] else None
        s["w_pre"] = _normal(g, K, std=0.2, dtype=torch.float32).add_(1.0) if case["pre"] else None
        s["gate"] = None
        if case["gate"] == "channel":
            s["gate"] = _normal(g, K, std=0.3, dtype=torch.float32).add_(0.5)
        elif case["gate"] == "token":
            s["gate"] = torch.rand(M, generator=g, device=DEV)
        if case["train"]:   # x stands for the stream behind the block; its gradients
            s["dx_out"] = _normal(g, M, K, std=0.02, dtype=dt)
            s["dh"] = _normal(g, M, K, std=0.02) if case["pre"] else None
        if own:
            moe = _moe()
            s["problem"] = moe.make_norm_problem(
                M, K, x_dtype=dt, gate_kind={"none": moe.GATE_NONE, "channel": moe.GATE_CHANNEL,
                                             "token": moe.GATE_TOKEN}[case["gate"]], res_scale=case["scale"])
            if case["train"]:
                s["dx"] = torch.empty_like(s["x"])
                s["dblock"] = torch.empty_like(s["block"])
                s["dw_post"] = torch.empty(K, device=DEV) if case["post"] else None
                s["dw_pre"] = torch.empty(K, device=DEV) if case["pre"] else None
                s["dgate"] = torch.empty_like(s["gate"]) if s["gate"] is not None else None
                s["ws"] = moe.allocate_norm_workspace(s["problem"], DEV)
            else:
                s["x_out"] = torch.empty_like(s["x"])
                s["h"] = torch.empty(M, K, dtype=torch.bfloat16, device=DEV) if case["pre"] else None
    else:
        E, N, K = case["E"], case["N"], case["K"]
        # a momentum: a few strong directions over noise
        u = torch.randn(E, N, K, generator=g, device=DEV)
        r = min(8, N, K)
        u += 2.0 * torch.matmul(torch.randn(E, N, r, generator=g, device=DEV),
                                torch.randn(E, r, K, generator=g, device=DEV)) / r
        s["update"] = (1e-3 * u).to(_type(case["dtype"]))
        if own:
            moe = _moe()
            s["problem"] = moe.make_ortho_problem(E, N, K, dtype=_type(case["dtype"]), steps=case["steps"], coef=MUON,
                                                  scale=case["scale"])
            s["out"] = torch.empty(E, N, K, dtype=torch.bfloat16, device=DEV)
            s["ws"] = moe.allocate_ortho_workspace(s["problem"], DEV)
    return s


# -------------------------------------------------------------- the passes --

def _plain_balance(case, s):
    M, E, k, S = case["M"], case["E"], case["topk"], case["S"]
    l = s["logits"].float()
    if s["bias"] is not None:
        l = l + s["bias"]
    if case["scoring"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        sg = 1.0 / (1.0 + torch.exp(-l))
        total = sg.sum(1, keepdim=True)
        p = sg / total
    # which sequence a token is of, as rows of zeros and ones; padding tokens are of none
    t = torch.arange(M, device=DEV, dtype=torch.int32)
    on = (s["ids"] >= 0).any(1)
    member = (t >= s["offsets"][:-1, None]) & (t < s["offsets"][1:, None]) & on
    route = torch.zeros(M, E + 1, device=DEV)
    route.scatter_(1, torch.where(s["ids"] >= 0, s["ids"], E).long(), 1.0)   # ids of a token differ
    # sums over the tokens of each sequence: 32 bits over 256 tokens at a time, 64 over those
    n = (M + 255) // 256
    member = torch.nn.functional.pad(member.float(), (0, 256 * n - M))
    part = member.view(S, n, 256).transpose(0, 1).contiguous()

    def over_tokens(v):
        v = torch.nn.functional.pad(v, (0, 0, 0, 256 * n - M)).view(n, 256, -1)
        return torch.matmul(part, v).double().sum(0)

    counts = over_tokens(route[:, :E])
    tokens = part.sum((0, 2)).double()
    per = tokens.clamp_min(1.0)
    probs = over_tokens(p) / per[:, None]
    loss = (counts * probs).sum(1) * (E / k) / per
    out = {"loss": loss.float(), "counts": counts.to(torch.int32), "tokens": tokens.to(torch.int32),
           "probs": probs.float()}
    if case["train"]:
        # counts (times what multiplies them) of each token's own sequence, less their mean, which
        # changes nothing (the scores add up to 1) but would hide their differences in 32 bits
        c = (counts - counts.mean(1, keepdim=True)) * (s["dloss"].double() * (E / k) / (per * per))[:, None]
        c = member[:, :M].t().contiguous() @ c.float()
        inner = c - (c * p).sum(1, keepdim=True)
        dl = p * inner if case["scoring"] == "softmax" else sg * (1.0 - sg) / total * inner
        out["dlogits"] = torch.where(on[:, None], dl, torch.zeros_like(dl)).to(s["logits"].dtype)
    return out


EPS = 1e-6


def _plain_norm(case, s):
    x, b = s["x"].float(), s["block"].float()
    gate = 1.0
    if case["gate"] == "channel":
        gate = s["gate"]
    elif case["gate"] == "token":
        gate = s["gate"][:, None]
    n, w = b, 1.0
    if case["post"]:
        rb = torch.rsqrt((b * b).mean(1, keepdim=True) + EPS)
        n, w = b * rb, s["w_post"]
    if not case["train"]:
        y = case["scale"] * x + gate * (n * w)
        out = {"x_out": y.to(s["x"].dtype)}
        if case["pre"]:
            out["h"] = (y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) * s["w_pre"]).to(torch.bfloat16)
        return out
    out = {}
    dy = s["dx_out"].float()
    if case["pre"]:
        r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
        xn, dh = x * r, s["dh"].float()
        g = dh * s["w_pre"]
        dy = dy + r * (g - xn * (g * xn).mean(1, keepdim=True))
        out["dw_pre"] = (dh * xn).double().sum(0).float()
    out["dx"] = (case["scale"] * dy).to(s["x"].dtype)
    if case["gate"] == "channel":
        out["dgate"] = (dy * n * w).double().sum(0).float()
    elif case["gate"] == "token":
        out["dgate"] = (dy * n * w).sum(1)
    du = gate * dy
    if case["post"]:
        out["dw_post"] = (du * n).double().sum(0).float()
        g = du * w
        du = rb * (g - n * (g * n).mean(1, keepdim=True))
    out["dblock"] = du.to(torch.bfloat16)
    return out


def _plain_ortho(case, s):
    a, b, c = MUON
    x = s["update"].float()
    wide = case["N"] < case["K"]
    if not wide:
        x = x.transpose(1, 2).contiguous()
    x = x / ((x * x).double().sum((1, 2), keepdim=True).sqrt().float() + 1e-7)
    for _ in range(case["steps"]):
        gram = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    if not wide:
        x = x.transpose(1, 2).contiguous()
    return {"out": (case["scale"] * x).to(torch.bfloat16)}


def run(state):
    s, case = state, state["case"]
    if own:
        moe = _moe()
        if case["op"] == "balance":
            moe.moe_balance_loss(s["router"], s["logits"], s["ids"], s["loss"], s["counts"], s["tokens"], s["probs"],
                                 s["ws"], bias=s["bias"], seq_offsets=s["offsets"])
            out = {"loss": s["loss"], "counts": s["counts"], "tokens": s["tokens"], "probs": s["probs"]}
            if case["train"]:
                moe.moe_balance_loss_backward(s["router"], s["logits"], s["ids"], s["counts"], s["tokens"],
                                              s["dloss"], s["dl"], bias=s["bias"], seq_offsets=s["offsets"])
                out["dlogits"] = s["dl"]
            return out
        if case["op"] == "ortho":
            moe.moe_orthogonalize(s["problem"], s["update"], s["out"], s["ws"])
            return {"out": s["out"]}
        if not case["train"]:
            moe.moe_block_norm(s["problem"], s["x"], s["x_out"], block=s["block"], w_post=s["w_post"],
                               gate=s["gate"], w_pre=s["w_pre"], h=s["h"])
            out = {"x_out": s["x_out"]}
            if case["pre"]:
                out["h"] = s["h"]
            return out
        moe.moe_block_norm_backward(s["problem"], s["x"], s["dx_out"], s["dx"], s["ws"], block=s["block"],
                                    w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"], dh=s["dh"],
                                    dblock=s["dblock"], dw_post=s["dw_post"], dgate=s["dgate"], dw_pre=s["dw_pre"])
        out = {}
        if case["pre"]:
            out["dw_pre"] = s["dw_pre"]
        out["dx"] = s["dx"]
        if case["gate"] != "none":
            out["dgate"] = s["dgate"]
        if case["post"]:
            out["dw_post"] = s["dw_post"]
        out["dblock"] = s["dblock"]
        return out
    if case["op"] == "balance":
        return _plain_balance(case, s)
    return _plain_norm(case, s) if case["op"] == "norm" else _plain_ortho(case, s)


# ------------------------------------------------------- what a pass needs --

def work(case):
    if case["op"] == "balance":
        M, E, k, S = case["M"], case["E"], case["topk"], case["S"]
        el = 4 if case["dtype"] == "f32" else 2
        b = M * E * el + M * k * 4 + S * (E * 8 + 8) + 4 * (S + 1) + (0 if case["bias"] == "none" else 4 * E)
        f = 4 * M * E
        if case["train"]:
            b += M * E * el + 4 * S
            f += 6 * M * E
        return {"bytes": b, "flops": f}
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        el = 4 if case["x"] == "f32" else 2
        vec = 4 * K * (int(case["post"]) + int(case["pre"]) + int(case["gate"] == "channel"))
        vec += 4 * M if case["gate"] == "token" else 0
        pre = 2 if case["pre"] else 0
        if case["train"]:
            # x, dx_out, dx, block, dblock, dh; weights and their gradients
            return {"bytes": M * K * (3 * el + 4 + pre) + 2 * vec, "flops": 20 * M * K}
        return {"bytes": M * K * (2 * el + 2 + pre) + vec, "flops": 9 * M * K}
    E, N, K = case["E"], case["N"], case["K"]
    m, n = min(N, K), max(N, K)
    # X^T X and its square are symmetric: half of each is enough
    f = case["steps"] * E * (3 * m * m * n + m * m * m)
    return {"bytes": E * N * K * ((4 if case["dtype"] == "f32" else 2) + 2), "flops": f}


# ------------------------------------------------------------ in 64 bits ----

def _exact_balance(case, s):
    E, k = case["E"], case["topk"]
    z = s["logits"].to(torch.float64)
    if s["bias"] is not None:
        z = z + s["bias"].to(torch.float64)
    p = torch.softmax(z, 1)
    if case["scoring"] == "sigmoid":
        sig = torch.sigmoid(z)
        p = sig / sig.sum(1, keepdim=True)
    off = s["offsets"].tolist()
    loss, counts, tokens, probs = [], [], [], []
    dl = torch.zeros_like(z)
    for q in range(case["S"]):
        a, b = off[q], off[q + 1]
        ids = s["ids"][a:b].long()
        keep = torch.nonzero((ids >= 0).any(1))[:, 0]
        T = int(keep.numel())
        tokens.append(T)
        c = torch.bincount(ids[ids >= 0], minlength=E)
        counts.append(c.to(torch.int32))
        if T == 0:
            probs.append(torch.zeros(E, dtype=torch.float64, device=DEV))
            loss.append(torch.zeros((), dtype=torch.float64, device=DEV))
            continue
        pq = p[a:b][keep]
        mean = pq.mean(0)
        f = c.to(torch.float64) * E / (k * T)
        probs.append(mean)
        loss.append(torch.dot(f, mean))
        # dloss/dp is f / T for each of the sequence's tokens; through the scores' Jacobian
        gp = (f / T * s["dloss"][q].to(torch.float64)).expand(T, E)
        inner = gp - (gp * pq).sum(1, keepdim=True)
        if case["scoring"] == "softmax":
            d = pq * inner
        else:
            sq = sig[a:b][keep]
            d = inner / sq.sum(1, keepdim=True) * torch.sigmoid(z[a:b][keep]) * torch.sigmoid(-z[a:b][keep])
        dl[a + keep] = d
    out = {"loss": torch.stack(loss), "counts": torch.stack(counts),
           "tokens": torch.tensor(tokens, dtype=torch.int32, device=DEV), "probs": torch.stack(probs)}
    if case["train"]:
        out["dlogits"] = dl
    return out


def _exact_norm(case, s):
    d = torch.float64
    K = case["K"]
    x, b = s["x"].to(d), s["block"].to(d)
    one = torch.ones(1, 1, dtype=d, device=DEV)
    g = {"none": lambda: one, "channel": lambda: s["gate"].to(d)[None, :], "token": lambda: s["gate"].to(d)[:, None]}
    gate = g[case["gate"]]()

    def rms(v):
        return torch.sqrt(torch.linalg.vector_norm(v, dim=1, keepdim=True) ** 2 / K + EPS)

    hat = b / rms(b) if case["post"] else b
    wp = s["w_post"].to(d)[None, :] if case["post"] else one
    if not case["train"]:
        y = case["scale"] * x + gate * hat * wp
        out = {"x_out": y}
        if case["pre"]:
            out["h"] = y / rms(y) * s["w_pre"].to(d)
        return out
    out = {}
    dy = s["dx_out"].to(d)
    if case["pre"]:
        dh, r = s["dh"].to(d), rms(x)
        wd = dh * s["w_pre"].to(d)
        dy = dy + wd / r - x * (torch.linalg.vecdot(wd, x, dim=1)[:, None] / (K * r ** 3))
        out["dw_pre"] = torch.linalg.vecdot(dh, x / r, dim=0)
    out["dx"] = dy * case["scale"]
    if case["gate"] == "channel":
        out["dgate"] = torch.linalg.vecdot(dy, hat * wp, dim=0)
    elif case["gate"] == "token":
        out["dgate"] = torch.linalg.vecdot(dy, hat * wp, dim=1)
    du = dy * gate
    if case["post"]:
        r = rms(b)
        out["dw_post"] = torch.linalg.vecdot(du, hat, dim=0)
        wd = du * wp
        du = wd / r - b * (torch.linalg.vecdot(wd, b, dim=1)[:, None] / (K * r ** 3))
    out["dblock"] = du
    return out


def _exact_ortho(case, s):
    a, b, c = MUON
    out = []
    for e in range(case["E"]):
        x = s["update"][e].to(torch.float64)
        if case["N"] > case["K"]:
            x = x.t().contiguous()
        x = x / (torch.linalg.matrix_norm(x) + 1e-7)
        for _ in range(case["steps"]):
            q = x @ x.t()
            # a X + b Q X + c Q (Q X)
            y = q @ x
            x = a * x + b * y + c * (q @ y)
        if case["N"] > case["K"]:
            x = x.t()
        out.append(x * case["scale"])
    return {"out": torch.stack(out)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "balance":
        return _exact_balance(case, s)
    return _exact_norm(case, s) if case["op"] == "norm" else _exact_ortho(case, s)

"""One training step of a block with the operators around its products: norm,
router, balance loss, grouped products, the junction's norm and gate, all of
their gradients, and the orthogonalised update of the experts' matrices, eager
and replayed from a graph, against 64-bit arithmetic on the same weights.

The path from a leaf to an output passes at most 10 roundings to bf16 (h, the
rows, y, x', and as many gradients on the way back), each at most half a step,
2^-8: 2-norms may be off by 10 2^-8 = 0.04 of the result."""
import numpy as np
import pytest
import torch

import mixture_experts_expert_align_amd as moe
from block_refs import ortho

pytestmark = pytest.mark.gpu
M, K, E, TOPK = 250, 256, 8, 2
TOL = 10 * 2.0 ** -8


class Block:
    def __init__(self):
        g = torch.Generator(device="cuda")
        g.manual_seed(3)
        bf = torch.bfloat16

        def rnd(*s, k=1.0, t=torch.float32):
            return (torch.randn(*s, generator=g, device="cuda") * k).to(t)
        self.x = rnd(M, K, t=bf)
        self.w_pre, self.w_post, self.w_next = 1 + rnd(K, k=0.2), 1 + rnd(K, k=0.2), 1 + rnd(K, k=0.2)
        self.gate = rnd(K)
        self.router_w = rnd(E, K, k=K ** -0.5, t=bf)
        self.w = rnd(E, K, K, k=K ** -0.5, t=bf)
        self.dx_out, self.dh = rnd(M, K, k=0.1, t=bf), rnd(M, K, k=0.1, t=bf)
        self.dbalance = torch.tensor([0.01, 0.02], device="cuda")
        self.offsets = torch.tensor([0, 110, M], dtype=torch.int32, device="cuda")
        self.router = moe.make_router(E, TOPK, renormalize=True)
        self.first = moe.make_norm_problem(M, K)
        self.junction = moe.make_norm_problem(M, K, gate_kind=moe.GATE_CHANNEL, res_scale=0.9)
        self.update = moe.make_ortho_problem(E, K, K, scale=0.2)
        e = dict(device="cuda")
        self.b = {n: torch.empty(M, K, dtype=bf, **e) for n in
                  ("h", "block", "x_out", "h_next", "dx", "dblock", "dh1", "dx0")}
        self.ids = torch.empty(M, TOPK, dtype=torch.int32, **e)
        self.wts = torch.empty(M, TOPK, **e)
        self.loss, self.tokens = torch.empty(2, **e), torch.empty(2, dtype=torch.int32, **e)
        self.counts, self.probs = torch.empty(2, E, dtype=torch.int32, **e), torch.empty(2, E, **e)
        self.logits, self.dlogits = torch.empty(M, E, **e), torch.empty(M, E, **e)
        self.sums = {n: torch.empty(K, **e) for n in ("dw_pre", "dw_post", "dgate", "dw_next")}
        self.dw = torch.empty(E, K, K, **e)
        self.new = torch.empty(E, K, K, dtype=bf, **e)
        self.ws_b = moe.allocate_balance_workspace(self.router, M, 2)
        self.ws_n = moe.allocate_norm_workspace(self.junction)
        self.ws_o = moe.allocate_ortho_workspace(self.update)
        # the sort of the rows by expert, fixed from one eager routing (the grouped products' own input)
        self.front()
        key = self.ids.reshape(-1).long()
        self.order = torch.argsort(key, stable=True)
        self.token = self.order // TOPK
        self.goff = torch.cat([torch.zeros(1, device="cuda"), torch.cumsum(torch.bincount(key, minlength=E), 0)]).int()
        R = M * TOPK
        self.rows, self.y = torch.empty(R, K, dtype=bf, **e), torch.empty(R, K, dtype=bf, **e)
        self.dy, self.drows = torch.empty(R, K, dtype=bf, **e), torch.empty(R, K, dtype=bf, **e)
        # each token's rows, in slot order: sums without atomics
        self.inverse = torch.argsort(self.order).view(M, TOPK)

    def front(self):
        b = self.b
        moe.moe_block_norm(self.first, self.x, w_pre=self.w_pre, h=b["h"])
        self.logits.copy_(b["h"].float() @ self.router_w.float().t().contiguous())
        moe.moe_route_topk(self.router, self.logits, self.ids, self.wts)

    def step(self):
        b = self.b
        self.front()
        moe.moe_balance_loss(self.router, self.logits, self.ids, self.loss, self.counts, self.tokens, self.probs,
                             self.ws_b, seq_offsets=self.offsets)
        self.rows.copy_(b["h"][self.token])
        moe.moe_grouped_forward(self.rows, self.w, self.goff, self.y)
        y = self.y.float()[self.inverse]
        b["block"].copy_((y * self.wts[:, :, None]).sum(1))
        moe.moe_block_norm(self.junction, self.x, b["x_out"], b["block"], self.w_post, self.gate, self.w_next,
                           b["h_next"])
        # back
        s = self.sums
        moe.moe_block_norm_backward(self.junction, b["x_out"], self.dx_out, b["dx"], self.ws_n, b["block"], self.w_post,
                                    self.gate, self.w_next, self.dh, b["dblock"], s["dw_post"], s["dgate"],
                                    s["dw_next"])
        db = b["dblock"].float()
        dwts = (y * db[:, None, :]).sum(2)
        wrow = self.wts.reshape(-1)[self.order][:, None]
        self.dy.copy_(db[self.token] * wrow)
        moe.moe_grouped_dgrad(self.dy, self.w, self.goff, self.drows)
        moe.moe_grouped_wgrad(self.dy, self.rows, self.goff, self.dw)
        moe.moe_route_topk_backward(self.router, self.logits, self.ids, dwts, self.dlogits)
        moe.moe_balance_loss_backward(self.router, self.logits, self.ids, self.counts, self.tokens, self.dbalance,
                                      self.dlogits, seq_offsets=self.offsets, accumulate=True)
        b["dh1"].copy_(self.drows.float()[self.inverse].sum(1) + self.dlogits @ self.router_w.float())
        moe.moe_block_norm_backward(self.first, self.x, b["dx"], b["dx0"], self.ws_n, w_pre=self.w_pre, dh=b["dh1"],
                                    dw_pre=s["dw_pre"])
        moe.moe_orthogonalize(self.update, self.dw, self.new, self.ws_o)

    def results(self):
        return [self.b["x_out"], self.b["h_next"], self.loss, self.b["dx0"], self.dw, self.new, self.dlogits,
                *self.sums.values()]


def reference(blk):
    """x_out, h_next, losses and gradients by autograd in float64, the choice held fixed."""
    d = torch.float64
    leaf = {n: getattr(blk, n).to("cpu", d).requires_grad_() for n in
            ("x", "w_pre", "w_post", "w_next", "gate", "w")}
    ids, rw = blk.ids.cpu().long(), blk.router_w.to("cpu", d)

    def norm(v, w):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * w
    h = norm(leaf["x"], leaf["w_pre"])
    logits = h @ rw.t()
    p = torch.softmax(logits, 1)
    w = torch.gather(p, 1, ids)
    w = w / w.sum(1, keepdim=True)
    block = torch.zeros(M, K, dtype=d)
    for j in range(TOPK):
        block = block + w[:, j, None] * torch.stack([h[t] @ leaf["w"][ids[t, j]].t() for t in range(M)])
    x_out = 0.9 * leaf["x"] + leaf["gate"] * norm(block, leaf["w_post"])
    h_next = norm(x_out, leaf["w_next"])
    loss, off = [], blk.offsets.tolist()
    for s in range(2):
        c = torch.bincount(ids[off[s]:off[s + 1]].reshape(-1), minlength=E).to(d)
        T = off[s + 1] - off[s]
        loss.append(E / (TOPK * T) * (c * p[off[s]:off[s + 1]].mean(0)).sum())
    loss = torch.stack(loss)
    total = (x_out * blk.dx_out.to("cpu", d)).sum() + (h_next * blk.dh.to("cpu", d)).sum() + \
        (loss * blk.dbalance.to("cpu", d)).sum()
    total.backward()
    return x_out.detach(), h_next.detach(), loss.detach(), {n: v.grad for n, v in leaf.items()}


def off(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    return ((a - b).norm() / b.norm()).item()


def test_step():
    blk = Block()
    blk.step()
    x_out, h_next, loss, grad = reference(blk)
    assert off(blk.b["x_out"], x_out) < TOL and off(blk.b["h_next"], h_next) < TOL and off(blk.loss, loss) < TOL
    assert off(blk.b["dx0"], grad["x"]) < TOL and off(blk.dw, grad["w"]) < TOL
    for n, leaf in (("dw_pre", "w_pre"), ("dw_post", "w_post"), ("dw_next", "w_next"), ("dgate", "gate")):
        assert off(blk.sums[n], grad[leaf]) < TOL, n
    # the update of the gradients as they are (its own error: 2e-3, and half a step of bf16)
    coef = [tuple(float(v) for v in blk.update.coef[i]) for i in range(5)]
    for e in (0, E - 1):
        ref = torch.from_numpy(0.2 * ortho(blk.dw[e].double().cpu().numpy(), coef, 1e-7))
        assert off(blk.new[e], ref) < 2e-3 + 2.0 ** -8


def test_step_from_a_graph():
    """Captured once and replayed with eager work between the replays; two captured steps share no
    state but their own buffers."""
    blk = Block()
    blk.step()
    want = [t.clone() for t in blk.results()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        blk.step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        blk.step()
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        blk.step()
    for i in range(4):
        for t in blk.results():
            t.fill_(1.0)
        (g if i % 2 == 0 else g2).replay()
        torch.cuda.synchronize()
        for a, b in zip(blk.results(), want):
            assert torch.equal(a, b)
        blk.ws_b.fill_(i), blk.ws_n.fill_(i), blk.ws_o.fill_(i)      # contents of no matter
        other = Block()
        other.step()
        torch.cuda.synchronize()
        for a, b in zip(other.results(), want):
            assert torch.equal(a, b)

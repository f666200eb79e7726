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

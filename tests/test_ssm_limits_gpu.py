"""The selective scan from states that are infinite or NaN: an infinite state stays one, with its
sign, under every decay that FP32 holds; NaN stays NaN; their neighbours keep their bits."""
from __future__ import annotations

import pytest
import torch

from linear_attention_recurrent_kda_gb300.api import KdaSsmStep, kda_ssm_prompt
from tests.test_ssm_gpu import i32, make

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
INF, NAN = float("inf"), float("nan")


def poisoned(state, slot):
    """Infinities and a NaN in some states of `slot`; what each becomes."""
    bad = {(0, 0): INF, (1, 5): -INF, (2, 15): INF, (9, 3): NAN, (17, 8): -INF, (23, 1): INF}
    for (c, n), v in bad.items():
        state[slot, c, n] = v
    return bad


def decays(d, rate):
    """exp(-rate / 4) a step, or somewhat less of it, each state's its own."""
    g = torch.Generator().manual_seed(9)
    d["a"].copy_(-rate * (0.5 + 0.5 * torch.rand(d["a"].shape, generator=g)))
    d["dt"].fill_(0.25)


def holds(bad, got, clean):
    rest = torch.ones(got.shape, dtype=torch.bool, device="cuda")
    for (c, n), v in bad.items():
        assert got[c, n].item() == v or (v != v and torch.isnan(got[c, n])), (c, n, v, got[c, n].item())
        rest[c, n] = False
    assert torch.equal(got[rest], clean[rest])


# decays a step from nearly 1 over 2^-1/4, where the step's form changes, and 1/2, where the
# prompt's does, to 1e-4
@pytest.mark.parametrize("rate", [1e-5, 1e-2, 1.0, 4.0, 40.0])
def test_step(rate):
    C, B = 24, 3
    d, state = make(B, C, soft=False, seed=2)
    decays(d, rate)
    clean = state.clone()
    bad = poisoned(state, 2)
    outs = [torch.zeros(B, C, dtype=BF, device="cuda") for _ in range(2)]
    for pool, out in ((clean, outs[0]), (state, outs[1])):
        step = KdaSsmStep(**d, softplus=False, slots=i32([1, 2, 0]), state=pool, output=out)
        for _ in range(3):
            step()
    holds(bad, state[2], clean[2])
    assert torch.equal(state[1], clean[1])
    hit = torch.zeros(B, C, dtype=torch.bool, device="cuda")
    for c, _ in bad:
        hit[1, c] = True
    assert torch.equal(outs[1][~hit], outs[0][~hit]) and not torch.isfinite(outs[1][hit]).any()


@pytest.mark.parametrize("T,path,rate", [(1, 1, 1e-5), (40, 1, 1e-5), (40, 1, 1.0), (40, 1, 4.0), (500, 1, 1e-2),
                                         (300, 1, 1e-5), (900, 2, 1e-5), (900, 2, 1e-2), (1500, 2, 0.1)])
def test_prompt(T, path, rate):
    """(Decays over the whole sequence stay above 2^-126.)"""
    C = 24
    d, state = make(T, C, soft=False, seed=3)
    decays(d, rate)
    clean = state.clone()
    bad = poisoned(state, 1)
    outs = [torch.zeros(T, C, dtype=BF, device="cuda") for _ in range(2)]
    for pool, out in ((clean, outs[0]), (state, outs[1])):
        kda_ssm_prompt(**d, softplus=False, seq_starts=i32([0, T]), state=pool, src_slots=i32([1]),
                       dst_slots=i32([2]), output=out, path=path)
    holds(bad, state[2], clean[2])
    hit = torch.zeros(C, dtype=torch.bool, device="cuda")
    for c, _ in bad:
        hit[c] = True
    assert torch.equal(outs[1][:, ~hit], outs[0][:, ~hit]) and not torch.isfinite(outs[1][:, hit]).any()

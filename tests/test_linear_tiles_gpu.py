"""The product's form for many tiles on the GPU where a pair of CTAs takes several tiles, some
of them at the output's end: whole numbers bit for bit."""
from __future__ import annotations

import pytest
import torch

from linear_attention_recurrent_kda_gb300.api import kda_linear

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def whole(g, *shape, top):
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(BF)


def framed(rows, width, extra=0):
    """NaN all around [rows, width]: a row before and behind, columns behind."""
    wide = torch.full((rows + 2, -(-width // 8) * 8 + extra), float("nan"), dtype=BF, device="cuda")
    return wide, wide[1:rows + 1, :width]


SIZES = [(2000, 64, 4096), (600, 64, 20480), (10000, 64, 7168), (1500, 72, 4100), (5000, 64, 5000),
         (4163, 72, 7203), (16384, 64, 2881), (2049, 200, 4999), (700, 8, 30001)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_residual_over_several_tiles(M, K, N, in_place):
    """|sum| <= 16 K + 60 + 250: exact in FP32 in any order, so the output is its rounding."""
    g = torch.Generator(device="cuda").manual_seed(M + K + N)
    x, w = whole(g, M, K, top=4), whole(g, N, K, top=4)
    bias, values = whole(g, N, top=60), whole(g, M, N, top=250)
    wide, out = framed(M, N, 8)
    behind, res = framed(M, N, 16)
    if in_place:
        res = out
    res.copy_(values)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda_linear(x=x, weight=w, bias=bias, residual=res, output=out, err=err)
    want = (x.double() @ w.double().T + bias.double() + values.double()).to(BF)
    assert err.item() == 0
    assert torch.equal(out, want)
    assert torch.isnan(wide[0]).all() and torch.isnan(wide[-1]).all() and torch.isnan(wide[:, N:]).all()


def test_residual_of_one_call_after_another():
    """Calls without a synchronisation, each adding to what the one before left."""
    g = torch.Generator(device="cuda").manual_seed(7)
    M, K, N = 2100, 64, 4360
    x, w = whole(g, M, K, top=2), whole(g, N, K, top=2)
    out, want = torch.zeros(M, N, dtype=BF, device="cuda"), torch.zeros(M, N, dtype=BF, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(5):
        kda_linear(x=x, weight=w, residual=out, output=out, err=err)
    product = x.double() @ w.double().T
    for _ in range(5):
        want = (product + want.double()).to(BF)
    assert err.item() == 0
    assert torch.equal(out, want)

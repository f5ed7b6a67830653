"""The product's activations of infinities, of sums that overflow and of NaN, in each form."""
from __future__ import annotations

import math

import pytest
import torch

from linear_attention_recurrent_kda_gb300.api import kda_linear

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
INF, NAN = float("inf"), float("nan")


# (one token, few tiles, many tiles)
@pytest.mark.parametrize("rows,path", [(1, 0), (5, 1), (5, 2), (300, 2)])
@pytest.mark.parametrize("act,below", [("silu", None), ("gelu", 0.0), ("softplus", 0.0)])
def test_activations_of_infinities(act, below, rows, path):
    """+infinity stays, -infinity leaves the activation's limit (0; SiLU's quotient of two
    infinities is not looked at), NaN stays NaN."""
    w = torch.ones(16, 2, dtype=BF, device="cuda")
    out = torch.zeros(rows, 16, dtype=BF, device="cuda")
    x = torch.zeros(rows, 8, dtype=BF, device="cuda")[:, :2]
    wide = torch.zeros(16, 8, dtype=BF, device="cuda")
    wide[:, :2] = w
    for pair, want in (((INF, 1.0), INF), ((3e38, 3e38), INF), ((-INF, 1.0), below), ((-3e38, -3e38), below),
                       ((NAN, 1.0), NAN), ((INF, -INF), NAN)):
        x[rows - 1] = torch.tensor(pair)
        kda_linear(x=x, weight=wide[:, :2], output=out, activation=act, path=path)
        got = out[rows - 1].tolist()
        if want is not None:
            assert all(v == want or (math.isnan(v) and math.isnan(want)) for v in got), (pair, got)

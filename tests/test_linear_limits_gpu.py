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


@pytest.mark.parametrize("rows,inner,outer", [(2000, 72, 3), (700, 520, 7), (65, 8200, 1), (4100, 16, 5)])
def test_many_rows_of_fewer_than_8_columns(rows, inner, outer):
    """Whole numbers: |sum| <= 4 inner + 50 is exact in FP32, so the output is its rounding."""
    g = torch.Generator(device="cuda").manual_seed(rows)

    def whole(n, width, top):
        wide = torch.randint(-top, top + 1, (n, -(-width // 8) * 8 + 8), generator=g, device="cuda").to(BF)
        return wide[:, :width]
    x, w, res = whole(rows, inner, 2), whole(outer, inner, 2), whole(rows, outer, 50)
    wide = torch.full((rows, 16), NAN, dtype=BF, device="cuda")
    for path in (0, 1):
        kda_linear(x=x, weight=w, residual=res, output=wide[:, :outer], path=path)
        assert torch.equal(wide[:, :outer], (x.double() @ w.double().T + res.double()).to(BF))
        assert torch.isnan(wide[:, outer:]).all()

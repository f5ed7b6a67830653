"""The product in each of its forms on the GPU (``path`` 1 and 2), whichever it would take by
itself: sizes, epilogues, cut tiles, views, infinities and graphs as tests/test_linear_gpu.py
has them."""
from __future__ import annotations

import pytest
import torch

from linear_attention_recurrent_kda_gb300 import lib as kl
from linear_attention_recurrent_kda_gb300.api import kda_linear
from tests import mixref
from tests.test_linear_gpu import SIZES, padded, whole

pytestmark = [pytest.mark.gpu, pytest.mark.parametrize("path", [1, 2])]
BF = torch.bfloat16
CUT = [(1, 64, 8), (130, 64, 9), (255, 200, 63), (257, 72, 257), (383, 64, 321), (300, 136, 775), (513, 24, 1030)]


@pytest.mark.parametrize("M,K,N", [s for s in SIZES if s[2] >= 8] + CUT)
def test_whole_numbers_are_exact(M, K, N, path):
    g = torch.Generator().manual_seed(M * 7 + K * 3 + N)
    x, w = whole(g, M, K, top=4), whole(g, N, K, top=4)
    bias, res = whole(g, N, top=60), whole(g, M, N, top=200)
    product = x.double() @ w.double().T
    wide = torch.full((M + 2, -(-N // 8) * 8 + 8), float("nan"), dtype=BF, device="cuda")
    x, w = padded(x, 16), padded(w, 8)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for b, r in ((None, None), (bias, None), (None, res), (bias, res)):
        wide.fill_(float("nan"))
        kda_linear(x=x, weight=w, bias=None if b is None else b.to(BF).cuda(),
                   residual=None if r is None else padded(r, 24), output=wide[1:M + 1, :N], path=path, err=err)
        want = product + (0 if b is None else b.double()) + (0 if r is None else r.double())
        got = wide.cpu()
        assert torch.equal(got[1:M + 1, :N].double(), want.to(BF).double()), (b is None, r is None)
        assert torch.isnan(got[0]).all() and torch.isnan(got[-1]).all() and torch.isnan(got[:, N:]).all()
    assert err.item() == 0


@pytest.mark.parametrize("act", [None, "silu", "gelu", "softplus"])
@pytest.mark.parametrize("M,K,N", [(4, 1000, 129), (300, 256, 1001), (700, 96, 515), (2000, 72, 4100)])
def test_epilogue_within_its_bound(M, K, N, act, path):
    g = torch.Generator().manual_seed(M + K)
    x, w = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g) * K ** -0.5
    x, w = padded(x), padded(w)
    bias = (2 * torch.randn(N, generator=g)).to(BF).cuda()
    out = padded(torch.zeros(M, N))
    for b, r in ((None, None), (bias, None), (bias, padded(torch.randn(M, N, generator=g)))):
        kda_linear(x=x, weight=w, bias=b, residual=r, output=out, activation=act, path=path)
        want, bound = mixref.linear(x, w, b, r, act)
        mixref.inside(out, want, bound, (act, b is None, r is None))


@pytest.mark.parametrize("M,N", [(1, 264), (600, 264), (3000, 2051)])
def test_residual_in_place(M, N, path):
    g = torch.Generator().manual_seed(9)
    x, w, res = whole(g, M, 256, top=3), whole(g, N, 256, top=3), whole(g, M, N, top=50)
    out = padded(res, 8)
    kda_linear(x=padded(x), weight=padded(w), residual=out, output=out, path=path)
    assert torch.equal(out.cpu().double(), (x.double() @ w.double().T + res.double()).to(BF).double())


@pytest.mark.parametrize("M,N", [(40, 300), (600, 519), (2100, 2305)])
def test_infinities_and_nan_reach_their_own_sums(M, N, path):
    """In x, W, the bias and the residual, some of them beside the output's end."""
    g = torch.Generator().manual_seed(4)
    x, w = whole(g, M, 200, top=3).to(BF), whole(g, N, 200, top=3).to(BF)
    bias, res = whole(g, N, top=9).to(BF), whole(g, M, N, top=9).to(BF)
    want = (x.double() @ w.double().T + bias.double() + res.double()).to(BF)
    x[5, 3], w[17, 199], bias[N - 1], res[M - 1, 7] = float("nan"), float("inf"), float("inf"), float("nan")
    odd = torch.zeros(M, N, dtype=torch.bool)
    odd[5], odd[:, 17], odd[:, N - 1], odd[M - 1, 7] = True, True, True, True
    out = padded(torch.zeros(M, N))
    kda_linear(x=padded(x), weight=padded(w), bias=bias.cuda(), residual=padded(res), output=out, path=path)
    got = out.cpu()
    assert torch.equal(got[~odd], want[~odd]) and not torch.isfinite(got[odd]).any()


def test_views_reach_no_further_than_themselves(path):
    g = torch.Generator().manual_seed(12)
    for M, K, N in ((1, 24, 40), (5, 24, 40), (270, 136, 200)):
        big = torch.full((M + 9, K + 48), float("nan"), dtype=BF, device="cuda")
        bigw = torch.full((N + 9, K + 48), float("nan"), dtype=BF, device="cuda")
        x, w = big[3:3 + M, 8:8 + K], bigw[4:4 + N, 16:16 + K]
        x.copy_(whole(g, M, K, top=3)), w.copy_(whole(g, N, K, top=3))
        out = padded(torch.zeros(M, N))
        kda_linear(x=x, weight=w, output=out, path=path)
        assert torch.equal(out.cpu().double(), (x.cpu().double() @ w.cpu().double().T).to(BF).double())


def test_graphs_and_repeats(path):
    """Several tiles a pair, a residual that changes between replays, eager calls beside."""
    g = torch.Generator().manual_seed(3)
    x, w = padded(whole(g, 1500, 128, top=3)), padded(whole(g, 4104, 128, top=3))
    res, out, other = (padded(torch.zeros(1500, 4104)) for _ in range(3))
    product = x.double() @ w.double().T
    kda_linear(x=x, weight=w, residual=res, output=out, path=path)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            kda_linear(x=x, weight=w, residual=res, output=out, path=path)
    side = torch.cuda.Stream()
    for i in range(6):
        out.zero_(), other.zero_(), res.fill_(i)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        kda_linear(x=x, weight=w, residual=res, output=other, path=path, stream=side)
        torch.cuda.synchronize()
        want = (product + i).to(BF)
        assert torch.equal(out, want) and torch.equal(other, want)


def test_refusals(path):
    x = torch.zeros(8, 16, dtype=BF, device="cuda")
    with pytest.raises(kl.KdaError) as e:
        kda_linear(x=x, weight=x, output=torch.zeros(8, 8, dtype=BF, device="cuda"), path=path + (1 << 32))
    assert e.value.code == kl.KDA_ERR_PATH
    if path == 2:
        with pytest.raises(kl.KdaError) as e:
            kda_linear(x=x, weight=x[:7], output=torch.zeros(8, 8, dtype=BF, device="cuda")[:, :7], path=2)
        assert e.value.code == kl.KDA_ERR_SHAPE

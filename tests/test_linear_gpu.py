"""The product with its epilogue on the GPU: whole numbers bit for bit over odd
sizes, random values within the bounds of tests/mixref.py."""
from __future__ import annotations

import pytest
import torch

from linear_attention_recurrent_kda_gb300 import lib as kl
from linear_attention_recurrent_kda_gb300.api import kda_linear
from tests import mixref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def padded(t, extra=0):
    """The same values as a slice of wider rows (a multiple of 8 elements apart)."""
    rows, width = t.shape
    wide = torch.full((rows, -(-width // 8) * 8 + extra), float("nan"), dtype=BF, device="cuda")
    wide[:, :width] = t.to(BF)
    return wide[:, :width]


def whole(g, *shape, top):
    return torch.randint(-top, top + 1, shape, generator=g).float()


SIZES = [(1, 1, 1), (1, 8, 8), (1, 4097, 1001), (1, 7168, 64), (1, 300, 9001), (1, 33000, 70), (3, 7, 5), (2, 40, 33), (8, 4100, 1000), (5, 24, 17), (8, 31, 16), (7, 20000, 100), (6, 64, 40000), (16, 64, 128), (17, 65, 129), (31, 4096, 1024), (33, 72, 257),
         (64, 1000, 640), (61, 4096, 2049), (128, 128, 128), (129, 200, 300), (255, 96, 1000),
         (256, 512, 256), (257, 520, 511), (300, 1, 40), (513, 2048, 1111), (1024, 256, 4096),
         (4099, 64, 136), (700, 4096, 770), (2, 16384, 16), (5, 40, 20000)]


@pytest.mark.parametrize("M,K,N", SIZES)
def test_whole_numbers_are_exact(M, K, N):
    """Sums of products of small whole numbers are exact in FP32 in any order: the output
    is the rounding of the sum, and nothing around it is touched."""
    g = torch.Generator().manual_seed(M * 7 + K * 3 + N)
    x, w = whole(g, M, K, top=4), whole(g, N, K, top=4)
    bias, res = whole(g, N, top=60), whole(g, M, N, top=200)
    want = x.double() @ w.double().T + bias.double() + res.double()
    wide = torch.full((M + 2, -(-N // 8) * 8 + 8), float("nan"), dtype=BF, device="cuda")
    kda_linear(x=padded(x, 16), weight=padded(w, 8), bias=bias.to(BF).cuda(), residual=padded(res, 24),
               output=wide[1:M + 1, :N])
    got = wide.cpu()
    assert torch.equal(got[1:M + 1, :N].double(), want.to(BF).double())
    assert torch.isnan(got[0]).all() and torch.isnan(got[-1]).all() and torch.isnan(got[:, N:]).all()


@pytest.mark.parametrize("act", [None, "silu", "gelu", "softplus"])
@pytest.mark.parametrize("M,K,N", [(1, 4096, 1025), (4, 4096, 129), (8, 1000, 77), (61, 321, 640), (300, 256, 1001), (1025, 520, 264)])
def test_epilogue_within_its_bound(M, K, N, act):
    g = torch.Generator().manual_seed(M + K)
    x, w = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g) * K ** -0.5
    x, w = padded(x), padded(w)
    bias = (2 * torch.randn(N, generator=g)).to(BF).cuda()
    out = padded(torch.zeros(M, N))
    for b, r in ((None, None), (bias, None), (bias, padded(torch.randn(M, N, generator=g)))):
        kda_linear(x=x, weight=w, bias=b, residual=r, output=out, activation=act)
        want, bound = mixref.linear(x, w, b, r, act)
        mixref.inside(out, want, bound, (act, b is None, r is None))
        # over all values the rounding is the error: at most half a place each
        off = (out.cpu().double() - want).norm() / want.norm()
        assert off <= 2.0 ** -8, off


@pytest.mark.parametrize("act", ["silu", "gelu", "softplus"])
def test_activations_over_their_range(act):
    """Each BF16 value of a range through the product with a unit matrix: exact up to the
    activation."""
    v = torch.cat([torch.linspace(-120, 120, 4001), torch.linspace(-1, 1, 1001),
                   torch.logspace(-30, 0, 301), -torch.logspace(-30, 0, 301),
                   torch.tensor([float("inf"), 3e38, -3e38])]).to(BF)
    x = torch.zeros(v.numel(), 8, dtype=BF)
    x[:, 0] = v
    w = torch.eye(8, dtype=BF)
    out = torch.empty(v.numel(), 8, dtype=BF, device="cuda")
    kda_linear(x=x[:-3].cuda(), weight=w.cuda(), output=out[:-3], activation=act)
    want, bound = mixref.linear(x[:-3], w, act=act)
    mixref.inside(out[:-3], want, bound)
    kda_linear(x=x[-3:].cuda(), weight=w.cuda(), output=out[-3:], activation=act)
    got = out[-3:, 0].cpu()
    assert got[0] != got[0] or got[0] == float("inf")
    assert got[1] == v[-2] and got[2] == 0


@pytest.mark.parametrize("M", [1, 3, 7, 600])
def test_residual_in_place(M):
    g = torch.Generator().manual_seed(9)
    x, w, res = whole(g, M, 256, top=3), whole(g, 264, 256, top=3), whole(g, M, 264, top=50)
    out = padded(res, 8)
    kda_linear(x=padded(x), weight=padded(w), residual=out, output=out)
    assert torch.equal(out.cpu().double(), (x.double() @ w.double().T + res.double()).to(BF).double())


@pytest.mark.parametrize("M,N", [(40, 300), (600, 520)])
def test_infinities_and_nan_reach_their_own_sums(M, N):
    g = torch.Generator().manual_seed(4)
    x, w = whole(g, M, 200, top=3).to(BF), whole(g, N, 200, top=3).to(BF)
    x[5, 3], w[17, 199] = float("nan"), float("inf")
    out = padded(torch.zeros(M, N))
    kda_linear(x=padded(x), weight=padded(w), output=out)
    odd = torch.zeros(M, N, dtype=torch.bool)
    odd[5], odd[:, 17] = True, True
    x[5, 3], w[17, 199] = 0, 0
    want = (x.double() @ w.double().T).to(BF)
    got = out.cpu()
    assert torch.equal(got[~odd], want[~odd]) and not torch.isfinite(got[odd]).any()


def test_views_reach_no_further_than_themselves():
    """NaN all around the operands: rows before and behind, columns beside."""
    g = torch.Generator().manual_seed(12)
    for M, K, N in ((1, 24, 40), (5, 24, 40), (270, 136, 200)):
        big = torch.full((M + 9, K + 48), float("nan"), dtype=BF, device="cuda")
        bigw = torch.full((N + 9, K + 48), float("nan"), dtype=BF, device="cuda")
        x, w = big[3:3 + M, 8:8 + K], bigw[4:4 + N, 16:16 + K]
        x.copy_(whole(g, M, K, top=3)), w.copy_(whole(g, N, K, top=3))
        out = padded(torch.zeros(M, N))
        kda_linear(x=x, weight=w, output=out)
        assert torch.equal(out.cpu().double(), (x.cpu().double() @ w.cpu().double().T).to(BF).double())


def test_graphs_streams_and_repeats():
    g = torch.Generator().manual_seed(3)
    x, w = padded(torch.randn(900, 512, generator=g)), padded(torch.randn(700, 512, generator=g))
    few, out, little = x[:9], padded(torch.zeros(900, 700)), padded(torch.zeros(9, 700))
    kda_linear(x=x, weight=w, output=out, activation="silu")
    kda_linear(x=few, weight=w, output=little)
    first, second = out.clone(), little.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda_linear(x=x, weight=w, output=out, activation="silu")
        kda_linear(x=few, weight=w, output=little)
    side = torch.cuda.Stream()
    other = padded(torch.zeros(9, 700))
    for _ in range(20):
        out.zero_(), little.zero_(), other.zero_()
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        kda_linear(x=few, weight=w, output=other, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(little, second) and torch.equal(other, second)


def test_offsets_past_32_bits():
    """Operands and output whose last rows begin past 2^31 elements."""
    g = torch.Generator().manual_seed(8)
    for M, N in ((40, (1 << 16) + 70), ((1 << 16) + 300, 48)):
        x, w = whole(g, M, 64, top=3), whole(g, N, 64, top=3)
        want = (x.double() @ w.double().T).to(BF)
        big = [torch.zeros(r, 1 << 15, dtype=BF, device="cuda") for r in (max(M, N), M)]
        side = big[0][:, 8:72]
        side.copy_(w if N > M else x)
        out = big[1][:, :N] if N <= 1 << 15 else padded(torch.zeros(M, N))
        kda_linear(x=side if M > N else padded(x), weight=side if N > M else padded(w), output=out)
        assert torch.equal(out.cpu().double(), want.double())
        del big, side


def test_no_rows_or_columns():
    x, w = torch.zeros(0, 8, dtype=BF, device="cuda"), torch.zeros(8, 8, dtype=BF, device="cuda")
    kda_linear(x=x, weight=w, output=torch.zeros(0, 8, dtype=BF, device="cuda"))
    kda_linear(x=w, weight=x, output=torch.zeros(8, 0, dtype=BF, device="cuda"))


def test_binding_refuses():
    x = torch.zeros(8, 16, dtype=BF, device="cuda")
    good = dict(x=x, weight=x, output=torch.zeros(8, 8, dtype=BF, device="cuda"))
    for bad, what in ((dict(activation="relu"), ValueError), (dict(weight=x[:, :8]), ValueError),
                      (dict(output=x), ValueError), (dict(bias=x[0]), ValueError), (dict(x=x.float()), TypeError),
                      (dict(x=x.T), ValueError), (dict(residual=x), ValueError),
                      (dict(x=x[:, 1:9], weight=x[:, :8]), kl.KdaError),
                      (dict(weight=x.cpu()), ValueError), (dict(err=x[0]), TypeError)):
        with pytest.raises(what):
            kda_linear(**{**good, **bad})

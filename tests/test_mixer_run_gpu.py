"""The operators together, as a model's selective-state-space layer runs them: prompts
into slots, then decoding on those slots, against the layer in 64 bits (with BF16
between the operators, as the calls hand it on)."""
from __future__ import annotations

import pytest
import torch

from linear_attention_recurrent_kda_gb300.api import (KdaConvStep, KdaSsmStep, kda_conv_prompt,
                                                      kda_linear, kda_ssm_prompt)
from tests import mixref

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32
HIDDEN, C, N, RANK, TAPS = 128, 256, 16, 8, 4


def i32(v):
    return torch.tensor(v, dtype=I32, device="cuda")


class Layer:
    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)

        def w(*shape, scale):
            return (scale * torch.randn(*shape, generator=g)).to(BF).cuda()

        self.into = w(2 * C, HIDDEN, scale=HIDDEN ** -0.5)
        self.taps, self.bias = w(TAPS, C, scale=0.5), w(C, scale=0.2)
        self.mix = w(RANK + 2 * N, C, scale=C ** -0.5)
        self.step = w(C, RANK, scale=RANK ** -0.5)
        self.a = -torch.exp(torch.randn(C, N, generator=g)).cuda()
        self.d = torch.randn(C, generator=g).cuda()
        self.dt_bias = (torch.randn(C, generator=g) - 3.0).cuda()
        self.out = w(HIDDEN, C, scale=C ** -0.5)

    def run(self, u, conv, scan):
        """One pass over rows u, the residual stream added; conv and scan are called with
        their rows."""
        rows = u.shape[0]

        def empty(width):
            return torch.empty(rows, width, dtype=BF, device="cuda")

        xz, x, mixed, dt, y, out = (empty(n) for n in (2 * C, C, RANK + 2 * N, C, C, HIDDEN))
        kda_linear(x=u, weight=self.into, output=xz)
        conv(x=xz[:, :C], output=x)
        kda_linear(x=x, weight=self.mix, output=mixed)
        kda_linear(x=mixed[:, :RANK], weight=self.step, output=dt)
        scan(x=x, dt=dt, b=mixed[:, RANK:RANK + N], c=mixed[:, RANK + N:], z=xz[:, C:], output=y)
        kda_linear(x=y, weight=self.out, residual=u, output=out)
        return dict(xz=xz, x=x, mixed=mixed, dt=dt, y=y, out=out)

    def check(self, u, got, starts, window, state, src):
        """Each stage against its plain form on what the stage before handed on."""
        def near(name, pair):
            mixref.inside(got[name], *pair[:2], name)
        near("xz", mixref.linear(u, self.into))
        near("x", mixref.conv(got["xz"][:, :C], self.taps, starts, self.bias, window, src))
        near("mixed", mixref.linear(got["x"], self.mix))
        near("dt", mixref.linear(got["mixed"][:, :RANK], self.step))
        scan = mixref.ssm(got["x"], got["dt"], self.a, got["mixed"][:, RANK:RANK + N],
                          got["mixed"][:, RANK + N:], starts, self.d, got["xz"][:, C:], self.dt_bias,
                          state=state, src=src)
        near("y", scan)
        near("out", mixref.linear(got["y"], self.out, residual=u))
        return scan


def test_prompts_then_decoding():
    layer = Layer(1)
    g = torch.Generator().manual_seed(2)
    lens, slots = [37, 1, 300, 2], [4, 2, 1, 5]
    starts = [0, 37, 38, 338, 340]
    window = torch.zeros(6, C, TAPS - 1, dtype=BF, device="cuda")
    state = torch.zeros(6, C, N, device="cuda")
    u = torch.randn(340, HIDDEN, generator=g).to(BF).cuda()
    seq = dict(seq_starts=i32(starts), dst_slots=i32(slots))
    got = layer.run(
        u, lambda **r: kda_conv_prompt(**r, **seq, weight=layer.taps, bias=layer.bias, window=window),
        lambda **r: kda_ssm_prompt(**r, **seq, a=layer.a, d=layer.d, dt_bias=layer.dt_bias, state=state))
    _, _, h, hb = layer.check(u, got, starts, None, None, None)
    for r, slot in enumerate(slots):
        mixref.inside(state[slot], h[r], hb[r], "state")
    at = i32(slots + [0])                           # the last row is padding
    for t in range(4):
        u = torch.randn(5, HIDDEN, generator=g).to(BF).cuda()
        old_window, old_state = window.clone(), state.clone()
        got = layer.run(
            u, lambda **r: KdaConvStep(**r, weight=layer.taps, bias=layer.bias, slots=at, window=window)(),
            lambda **r: KdaSsmStep(**r, a=layer.a, d=layer.d, dt_bias=layer.dt_bias, slots=at, state=state)())
        assert (got["x"][4] == 0).all() and (got["y"][4] == 0).all()
        live = {k: v[:4] for k, v in got.items()}
        _, _, h, hb = layer.check(u[:4], live, [0, 1, 2, 3, 4], old_window, old_state, slots)
        for r, slot in enumerate(slots):
            mixref.inside(state[slot], h[r], hb[r], "state")
        assert torch.equal(got["out"][4], u[4])     # padding passes the residual stream on
        assert torch.equal(state[[0, 3]], old_state[[0, 3]])


def test_a_prompt_in_pieces_is_the_prompt():
    """Chunked prefill: the second half continues from the slots of the first, and gives
    the rows of the whole within twice the bounds of a row."""
    layer = Layer(3)
    u = torch.randn(200, HIDDEN, generator=torch.Generator().manual_seed(4)).to(BF).cuda()
    outs = []
    for cuts in ([200], [120, 80]):
        window = torch.zeros(2, C, TAPS - 1, dtype=BF, device="cuda")
        state = torch.zeros(2, C, N, device="cuda")
        lo, parts = 0, []
        for n in cuts:
            seq = dict(seq_starts=i32([0, n]), src_slots=i32([1]), dst_slots=i32([1]))
            parts.append(layer.run(
                u[lo:lo + n],
                lambda **r: kda_conv_prompt(**r, **seq, weight=layer.taps, bias=layer.bias, window=window),
                lambda **r: kda_ssm_prompt(**r, **seq, a=layer.a, d=layer.d, dt_bias=layer.dt_bias,
                                           state=state)))
            lo += n
        outs.append({k: torch.cat([p[k] for p in parts]) for k in parts[0]})
    for k in ("xz", "x", "mixed", "dt"):           # no scan before them: the same bits
        assert torch.equal(outs[0][k], outs[1][k]), k
    _, bound, _, _ = mixref.ssm(outs[0]["x"], outs[0]["dt"], layer.a, outs[0]["mixed"][:, RANK:RANK + N],
                                outs[0]["mixed"][:, RANK + N:], [0, 200], layer.d, outs[0]["xz"][:, C:],
                                layer.dt_bias)
    assert ((outs[0]["y"].double() - outs[1]["y"].double()).abs().cpu() <= 2 * bound).all()

"""Kernels that may start while the one before them ends: chains of calls without a
synchronisation between them, each reading what the one before wrote, leave the bits
that the same calls leave one at a time."""
from __future__ import annotations

import pytest
import torch

from linear_attention_recurrent_kda_gb300.api import (KdaConvStep, KdaSsmStep, kda_conv_prompt,
                                                      kda_linear, kda_ssm_prompt, step_from_inputs)
from linear_attention_recurrent_kda_gb300.workloads import make_inputs
from tests.test_graph_pdl_gpu import Launch, wl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Chain:
    """rows x wide -> product (long) -> convolution -> product -> scan -> product, each over
    what the one before wrote, and pools that a pass leaves to the next (the input stays:
    fed back it would grow with its fourth power)."""

    def __init__(self, rows, wide, prompt, seed):
        g = torch.Generator().manual_seed(seed)

        def w(*shape, scale):
            return (scale * torch.randn(*shape, generator=g)).to(BF).cuda()
        N, taps = 16, 4
        self.w1, self.w2 = w(wide, wide, scale=wide ** -0.5), w(wide, wide, scale=wide ** -0.5)
        self.wbc = w(2 * N, wide, scale=wide ** -0.5)
        self.x = w(rows, wide, scale=1.0)
        self.t, self.y, self.end = (torch.zeros_like(self.x) for _ in range(3))
        self.bc = torch.zeros(rows, 2 * N, dtype=BF, device="cuda")
        slots = i32(list(range(1, rows + 1)))
        self.window = torch.zeros(rows + 1, wide, taps - 1, dtype=BF, device="cuda")
        self.state = torch.zeros(rows + 1, wide, N, device="cuda")
        weights = dict(weight=w(taps, wide, scale=0.5))
        rest = dict(a=-torch.exp(torch.randn(wide, N, generator=g)).cuda(), state=self.state)
        scan = dict(x=self.t, dt=self.t, b=self.bc[:, :N], c=self.bc[:, N:], z=self.x, output=self.y)
        if prompt:
            seq = dict(seq_starts=i32([0, 1, rows // 3, rows]), src_slots=i32([1, 2, 3]), dst_slots=i32([1, 2, 3]))
            self.conv = lambda: kda_conv_prompt(x=self.y, output=self.t, window=self.window, **weights, **seq)
            self.scan = lambda: kda_ssm_prompt(**scan, **rest, **seq)
        else:
            self.conv = KdaConvStep(x=self.y, output=self.t, window=self.window, slots=slots, **weights)
            self.scan = KdaSsmStep(**scan, **rest, slots=slots)

    def calls(self):
        def into():
            kda_linear(x=self.x, weight=self.w1, output=self.y, activation="silu")

        def mixed():
            kda_linear(x=self.t, weight=self.wbc, output=self.bc)

        def out():
            kda_linear(x=self.y, weight=self.w2, residual=self.end, output=self.end)
        return [into, lambda: self.conv(), mixed, lambda: self.scan(), out]

    def left(self):
        return [self.end, self.window, self.state]


@pytest.mark.parametrize("rows,wide,prompt", [(1, 2048, False), (4, 4096, False), (100, 1024, False),
                                              (61, 512, True), (3000, 1024, True), (2, 64, False)])
@pytest.mark.parametrize("captured", [False, True])
def test_chains_leave_the_bits_of_single_calls(rows, wide, prompt, captured):
    a, b = Chain(rows, wide, prompt, 5), Chain(rows, wide, prompt, 5)
    for _ in range(6):
        for call in a.calls():
            call()
            torch.cuda.synchronize()
    if captured:
        b.calls()                                   # (nothing is launched here)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                for call in b.calls():
                    call()
        graph.replay()
        graph.replay()
    else:
        for _ in range(6):
            for call in b.calls():
                call()
    torch.cuda.synchronize()
    assert torch.isfinite(a.end).all()
    for u, v in zip(a.left(), b.left()):
        assert torch.equal(u, v)


@pytest.mark.parametrize("captured", [False, True])
def test_after_and_before_other_work(captured):
    """Copies, fills and torch's kernels before and behind a call, and a fork to a second
    stream and back, order it as any kernel."""
    g = torch.Generator().manual_seed(6)
    big = torch.randint(-2, 3, (4096, 4096), generator=g).to(BF).cuda()
    w = torch.randint(-2, 3, (512, 4096), generator=g).to(BF).cuda()
    x = torch.zeros(64, 4096, dtype=BF, device="cuda")
    out, copy, more = (torch.zeros(64, 512, dtype=BF, device="cuda") for _ in range(3))
    side = torch.cuda.Stream()

    def work():
        x.fill_(1)
        big.add_(0)                                 # some microseconds
        x.copy_(big[:64])                           # a copy before
        kda_linear(x=x, weight=w, output=out)
        copy.copy_(out)                             # and behind
        x.add_(1)                                   # torch's kernel writes what a call reads
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            big[64:].add_(0)
            kda_linear(x=x, weight=w, output=more)
        torch.cuda.current_stream().wait_stream(side)
        kda_linear(x=x, weight=w, output=out, residual=more)
        x.zero_()                                   # what it read is written over

    if captured:
        graph = torch.cuda.CUDAGraph()
        warm = torch.cuda.Stream()
        warm.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(warm):
            work()
        torch.cuda.current_stream().wait_stream(warm)
        with torch.cuda.graph(graph):
            work()
    for _ in range(5):
        out.zero_(), copy.zero_(), more.zero_()
        graph.replay() if captured else work()
    torch.cuda.synchronize()
    first = (big[:64].double().cpu() @ w.double().cpu().T)
    second = ((big[:64].double() + 1).cpu() @ w.double().cpu().T)
    assert torch.equal(copy.cpu(), first.to(BF))
    assert torch.equal(more.cpu(), second.to(BF))
    assert torch.equal(out.cpu(), (second + second.to(BF).double()).to(BF))


@pytest.mark.parametrize("rows", [1, 4, 600])
def test_a_kda_step_two_launches_behind(rows):
    """A KDA step that reads its pages before it waits for the kernel before (use_pdl): that
    one is a product, and the step before the product wrote the pages."""
    x, w = (torch.ones(n, 2048, dtype=BF, device="cuda") for n in (rows, 1024))
    between = torch.zeros(rows, 1024, dtype=BF, device="cuda")
    got = []
    for apart in (True, False):
        step = Launch(make_inputs(wl()))
        behind = step_from_inputs(step.d, step.out, err=step.err, dbg=step.dbg, use_pdl=True)
        for _ in range(4):
            for call in (step.step, lambda: kda_linear(x=x, weight=w, output=between), behind,
                         lambda: kda_linear(x=x, weight=w, output=between)):
                call()
                if apart:
                    torch.cuda.synchronize()
        got.append(step.snapshot())
    for u, v in zip(*got):
        assert torch.equal(u, v)

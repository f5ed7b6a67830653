"""Ways to call the convolution, scan and product: first calls from several host
threads, streams of the caller's, workspaces of the caller's, batches of padding
alone, prepared steps whose contents change."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from linear_attention_recurrent_kda_gb300 import lib as kl
from linear_attention_recurrent_kda_gb300.api import (KdaConvStep, KdaSsmStep, kda_conv_prompt,
                                                      kda_linear, kda_ssm_prompt)
from tests import mixref
from tests.test_conv_gpu import make as make_conv
from tests.test_ssm_gpu import i32
from tests.test_ssm_gpu import make as make_ssm

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

CHILD = r"""
import threading, torch
from linear_attention_recurrent_kda_gb300 import api
from tests.test_ssm_gpu import make, i32
from tests.test_conv_gpu import make as make_conv
BF = torch.bfloat16

def scan(T, path, seed):
    d, state = make(T, 64, seed=seed)
    out = torch.zeros(T, 64, dtype=BF, device="cuda")
    kw = dict(d, seq_starts=i32([0, 5, T]), output=out, state=state, src_slots=i32([1, 2]),
              dst_slots=i32([3, 4]), path=path)
    return (lambda s: api.kda_ssm_prompt(**kw, stream=s)), [out, state]

def scan_step(seed):
    d, state = make(6, 40, seed=seed)
    out = torch.zeros(6, 40, dtype=BF, device="cuda")
    kw = dict(d, slots=i32([1, 2, 3, 4, 5, 6]), state=state, output=out)
    return (lambda s: api.kda_ssm_step(s, **kw)), [out, state]

def conv(seed):
    d, out = make_conv(90, 48, seed=seed)
    out.zero_()
    kw = dict(d, output=out[:, :48], seq_starts=i32([0, 90]), src_slots=i32([1]), dst_slots=i32([2]))
    return (lambda s: api.kda_conv_prompt(**kw, stream=s)), [out, d["window"]]

def conv_step(seed):
    d, out = make_conv(6, 48, seed=seed)
    out.zero_()
    kw = dict(d, output=out[:, :48], slots=i32([1, 2, 3, 4, 5, 6]))
    return (lambda s: api.kda_conv_step(s, **kw)), [out, d["window"]]

def product(M, K, N, seed):
    g = torch.Generator().manual_seed(seed)
    x, w = (torch.randn(*s, generator=g).to(BF).cuda() for s in ((M, K), (N, K)))
    out = torch.zeros(M, N, dtype=BF, device="cuda")
    return (lambda s: api.kda_linear(x=x, weight=w, output=out, activation="gelu", stream=s)), [out]

def jobs():
    return [scan(1500, 2, 1), scan(300, 1, 2), scan_step(3), conv(4), conv_step(5), product(1, 512, 64, 6),
            product(40, 4096, 128, 7), product(2000, 256, 2048, 8), product(2000, 256, 2048, 9)]

mine, failures = jobs(), []
torch.cuda.synchronize()
gate = threading.Barrier(len(mine))

def work(run):
    try:
        s = torch.cuda.Stream()
        gate.wait()
        with torch.cuda.stream(s):
            run(s)
    except Exception as e:
        failures.append(repr(e))

threads = [threading.Thread(target=work, args=(run,)) for run, _ in mine]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not failures, failures
for (_, got), (run, want) in zip(mine, jobs()):
    run(None)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
print("same bits")
"""


def test_first_calls_from_several_host_threads():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", CHILD], cwd=root, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-3000:]
    assert "same bits" in res.stdout


def test_the_caller_s_workspace():
    T = 1500
    d, state = make_ssm(T, 64, seed=1)
    outs = [torch.empty(T, 64, dtype=BF, device="cuda") for _ in range(2)]
    args = dict(d, seq_starts=i32([0, T]), path=2)
    kda_ssm_prompt(**args, output=outs[0])
    need = kl.ssm_workspace(kl.KdaSsmPromptArgs(
        seqs=1, channels=64, states=16, groups=1, tokens=T, max_seq=T, path=2, softplus=1, x_stride=88,
        dt_stride=88, b_stride=40, c_stride=40, z_stride=88, o_stride=64))
    assert need > 0
    guard = torch.full((need + 4096,), 85, dtype=torch.uint8, device="cuda")
    kda_ssm_prompt(**args, output=outs[1], workspace=guard[:need])
    assert torch.equal(outs[0], outs[1]) and (guard[need:] == 85).all()
    for bad in (guard[:need - 1], guard[4:need + 4], None):
        with pytest.raises(kl.KdaError) as e:
            if bad is None:
                a = kl.KdaSsmPromptArgs(
                    1, 64, 16, 1, T, T, 0, 1, 2, 88, 88, 40, 40, 88, 64,
                    *(d[k].data_ptr() for k in ("x", "dt", "a", "b", "c", "d", "z", "dt_bias")),
                    args["seq_starts"].data_ptr(), None, None, None, outs[1].data_ptr(), None)
                raise kl.KdaError(kl.call("kda_ssm_prompt", a, 0), "")
            kda_ssm_prompt(**args, output=outs[1], workspace=bad)
        assert e.value.code == kl.KDA_ERR_WORKSPACE


def test_on_a_stream_of_the_caller_s():
    """Inputs come on a stream, the calls follow on it, and their results are used on it: the
    default stream is not waited for."""
    d, state = make_ssm(400, 64, seed=2)
    want, bound, _, _ = mixref.ssm(**d, starts=[0, 400])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = {k: torch.zeros_like(v) if v is not None and k != "a" else v for k, v in d.items()}
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        for k, v in late.items():
            if v is not None:
                v.copy_(d[k])
        out = torch.empty(400, 64, dtype=BF, device="cuda")
        y = torch.empty(400, 64, dtype=BF, device="cuda")
    starts = i32([0, 400])
    torch.cuda.current_stream().synchronize()
    kda_ssm_prompt(**late, seq_starts=starts, output=out, path=2, stream=side)
    kda_linear(x=out, weight=torch.eye(64, dtype=BF, device="cuda"), output=y, stream=side)
    side.synchronize()
    mixref.inside(out, want, bound)
    assert torch.equal(out, y)


def test_batches_of_padding_alone():
    d, state = make_ssm(5, 40, seed=3)
    before, out = state.clone(), torch.full((5, 40), float("nan"), dtype=BF, device="cuda")
    KdaSsmStep(**d, slots=i32([0, -1, 0, 0, -7]), state=state, output=out)()
    assert (out == 0).all() and torch.equal(state, before)
    window = torch.randn(3, 40, 3, device="cuda").to(BF)
    kept = window.clone()
    out.fill_(float("nan"))
    KdaConvStep(x=d["x"], weight=torch.ones(4, 40, dtype=BF, device="cuda"), slots=i32([0, -1, 0, 0, -7]),
                window=window, output=out)()
    assert (out == 0).all() and torch.equal(window, kept)


def test_prepared_steps_follow_their_tensors():
    """The contents of a prepared step's tensors change between calls, slots among them."""
    d, state = make_ssm(3, 40, seed=4)
    slots, out = i32([1, 2, 3]), torch.empty(3, 40, dtype=BF, device="cuda")
    step = KdaSsmStep(**d, slots=slots, state=state, output=out)
    step()
    for at in ([3, 1, 2], [5, 0, 6]):
        slots.copy_(i32(at))
        d["x"].copy_(torch.randn(3, 40))
        old = state.clone()
        step()
        want, bound, h, hb = mixref.ssm(**d, starts=[0, 1, 2, 3], state=old, src=at)
        for r, slot in enumerate(at):
            if slot:
                mixref.inside(out[r], want[r], bound[r])
                mixref.inside(state[slot], h[r], hb[r])
            else:
                assert (out[r] == 0).all()


def test_a_graph_of_the_whole_step_while_eager_calls_run():
    """Decode of a layer captured once and replayed, its buffers refilled, beside eager calls
    of the same operators on another stream."""
    C, B = 64, 4
    g = torch.Generator().manual_seed(5)
    d, state = make_ssm(B, C, seed=6)
    w_in, w_out = (0.2 * torch.randn(C, C, generator=g)).to(BF).cuda(), (0.2 * torch.randn(C, C, generator=g)).to(BF).cuda()
    taps = torch.randn(4, C, generator=g).to(BF).cuda()
    window = torch.randn(8, C, 3, generator=g).to(BF).cuda()
    u, x0, x1, y, out = (torch.zeros(B, C, dtype=BF, device="cuda") for _ in range(5))
    slots = i32([4, 1, 0, 2])
    conv = KdaConvStep(x=x0, weight=taps, slots=slots, window=window, output=x1)
    scan = KdaSsmStep(**dict(d, x=x1), slots=slots, state=state, output=y)

    def layer():
        kda_linear(x=u, weight=w_in, output=x0)
        conv()
        scan()
        kda_linear(x=y, weight=w_out, residual=u, output=out, activation="silu")

    first = window.clone(), state.clone()
    layer()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    side, other = torch.cuda.Stream(), torch.empty(300, C, dtype=BF, device="cuda")
    big, _ = make_ssm(300, C, seed=7)
    kda_ssm_prompt(**big, seq_starts=i32([0, 300]), output=other)
    clean = other.clone()
    inputs = [torch.randn(B, C, generator=g).to(BF).cuda() for _ in range(4)]

    def run(one):
        window.copy_(first[0]), state.copy_(first[1])
        got = []
        for v in inputs:
            u.copy_(v)
            one()
            got.append(out.clone())
        return got + [window.clone(), state.clone()]

    want = run(layer)
    torch.cuda.synchronize()
    for _ in range(3):
        kda_ssm_prompt(**big, seq_starts=i32([0, 300]), output=other, stream=side)
    for a, b in zip(run(graph.replay), want):
        assert torch.equal(a, b)
    side.synchronize()
    assert torch.equal(other, clean)


class Counted:
    """The short way from Python, with what it took counted; or one that takes nothing."""

    def __init__(self, inner):
        self.inner, self.took = inner, 0

    def __getattr__(self, name):
        def call(*args):
            rc = getattr(self.inner, name)(*args) if self.inner else None
            self.took += rc is not None
            return rc
        return call


def _three(stream, out):
    """A product, a convolution and a scan on slices, with everything that may be there."""
    g = torch.Generator().manual_seed(12)
    x, w = (torch.randn(*s, generator=g).to(BF).cuda() for s in ((5, 48), (24, 48)))
    torch.cuda.synchronize()
    kda_linear(x=x[:, :40], weight=torch.nn.Parameter(w[:, :40]), output=out["product"][:, :24],
               bias=w[0, :24].contiguous(), residual=x[:, 8:32], activation="gelu",
               err=out["err"], stream=stream)
    kda_linear(x=x[:1, :40], weight=w[:, :40], output=out["one"], stream=stream)
    seq = dict(seq_starts=i32([0, 1, 30]), src_slots=i32([1, 2]), dst_slots=i32([3, 2]))
    d, y = make_conv(30, 48, seed=3)
    torch.cuda.synchronize()
    kda_conv_prompt(**dict(d, output=out["conv"]), **seq, err=out["err"], stream=stream)
    out["window"] = d["window"]
    d, state = make_ssm(30, 64, seed=4)
    torch.cuda.synchronize()
    kda_ssm_prompt(**d, **seq, output=out["scan"], state=state, err=out["err"], max_seq=29, stream=stream)
    out["state"] = state
    torch.cuda.synchronize()


@pytest.mark.parametrize("own_stream", [False, True])
def test_the_short_way_and_the_general_one(monkeypatch, own_stream):
    """The same bits by both, and the short way takes all of them."""
    stream = torch.cuda.Stream() if own_stream else None
    short, general = Counted(kl.bind()), Counted(None)
    got = []
    for way in (short, general):
        monkeypatch.setattr(kl, "_bind", way)
        out = dict(product=torch.zeros(5, 32, dtype=BF, device="cuda"), one=torch.zeros(1, 24, dtype=BF, device="cuda"),
                   conv=torch.zeros(30, 48, dtype=BF, device="cuda"), scan=torch.zeros(30, 64, dtype=BF, device="cuda"),
                   err=torch.zeros(1, dtype=torch.int32, device="cuda"))
        _three(stream, out)
        got.append(out)
    assert short.took == 4 and general.took == 0
    for k in got[0]:
        assert torch.equal(got[0][k], got[1][k]), k
    assert (got[0]["product"][:, :24] != 0).any() and (got[0]["product"][:, 24:] == 0).all()


def test_the_short_way_leaves_rare_calls():
    bind = kl.bind()
    x, w = torch.zeros(4, 16, dtype=BF, device="cuda"), torch.zeros(8, 16, dtype=BF, device="cuda")
    out = torch.zeros(4, 8, dtype=BF, device="cuda")
    assert bind.linear(x, w, out, None, None, 0, None, None) == 0
    for args in ((x.float(), w, out), (x, w.float(), out), (x, w, out.T), (x.T, w, out), (x, w[:, :8], out),
                 (x, w, out[:, :7]), (x[0], w, out), (x, w, out.cpu()), (x, w, None), (x[:, ::2], w[:, :8], out)):
        assert bind.linear(*args, None, None, 0, None, None) is None
    for bias in (out[0, :7], out, out[0].float(), out[0].cpu()):
        assert bind.linear(x, w, out, bias, None, 0, None, None) is None
    assert bind.linear(x, w, out, None, None, 0, out, None) is None
    assert bind.linear(x, w, out, None, None, 0, None, "a stream") is None
    with pytest.raises(kl.KdaError):                  # it is the library that refuses this
        kda_linear(x=torch.zeros(4, 24, dtype=BF, device="cuda")[:, 1:17], weight=w, output=out)
    with pytest.raises(ValueError, match="shape"):
        kda_linear(x=x, weight=w, output=out[:, :7])
    with pytest.raises(ValueError, match="adjacent"):
        kda_linear(x=torch.zeros(16, 4, dtype=BF, device="cuda").T, weight=w, output=out)
    torch.cuda.synchronize()

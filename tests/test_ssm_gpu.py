"""The selective scan on the GPU against the recurrence in 64 bits, within the bounds
that tests/mixref.py derives."""
from __future__ import annotations

import math

import pytest
import torch

from linear_attention_recurrent_kda_gb300 import lib as kl
from linear_attention_recurrent_kda_gb300.api import KdaSsmStep, kda_ssm_prompt, kda_ssm_step
from tests import mixref

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def i32(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def make(rows, C, N=16, G=1, soft=True, gated=True, skip=True, slots=8, seed=0, rate=1.0, extra=24):
    """Inputs of the scan; rows are slices of wider ones."""
    g = torch.Generator().manual_seed(seed)

    def wide(width, scale=1.0):
        t = torch.full((rows, width + extra), float("nan"), dtype=BF)
        t[:, 8:8 + width] = (scale * torch.randn(rows, width, generator=g)).to(BF)
        return t.cuda()[:, 8:8 + width]

    step = torch.exp(torch.rand(C, generator=g) * math.log(100.0)) * 1e-2
    d = dict(x=wide(C), b=wide(G * N), c=wide(G * N),
             a=(-rate * (torch.rand(C, N, generator=g) * 4 + 0.02)).cuda(),
             d=torch.randn(C, generator=g).cuda() if skip else None, z=wide(C) if gated else None)
    if soft:
        d["dt"], d["dt_bias"] = wide(C), (step + torch.log(-torch.expm1(-step))).cuda()
    else:
        d["dt"], d["dt_bias"] = wide(C).abs_().mul_(0.1), None
    state = torch.randn(slots, C, N, generator=g).cuda()
    return d, state


def check(d, state, lens, src, dst, soft=True, first=0, path=0, max_seq=None, err=None):
    rows, C = d["x"].shape
    starts = [first]
    for n in lens:
        starts.append(starts[-1] + n)
    before = state.clone()
    out = torch.full((rows, C + 16), float("nan"), dtype=BF, device="cuda")
    kda_ssm_prompt(**d, softplus=soft, seq_starts=i32(starts), output=out[:, 8:8 + C], state=state,
                   src_slots=None if src is None else i32(src),
                   dst_slots=None if dst is None else i32(dst), path=path, max_seq=max_seq, err=err)
    want, bound, h, hb = mixref.ssm(**d, soft=soft, starts=starts, state=before, src=src)
    got = out.cpu()
    mixref.inside(got[:, 8:8 + C], want, bound, "output")
    assert torch.isnan(got[:, :8]).all() and torch.isnan(got[:, 8 + C:]).all()
    assert torch.isnan(got[:first]).all() and torch.isnan(got[starts[-1]:]).all()
    kept = torch.ones(state.shape[0], dtype=torch.bool)
    for r, slot in enumerate(dst or []):
        if slot > 0:
            mixref.inside(state[slot], h[r], hb[r], "state")
            kept[slot] = False
    assert torch.equal(state[kept.cuda()], before[kept.cuda()])
    return out[:, 8:8 + C]


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("C,N,G,soft,gated,skip", [
    (8, 16, 1, True, True, True), (24, 16, 3, False, False, False), (136, 16, 1, True, False, True),
    (264, 32, 1, True, True, False), (48, 32, 2, False, True, True), (72, 64, 1, True, True, True),
    (16, 64, 2, False, False, True), (200, 16, 1, False, True, False)])
def test_ragged_prompts(C, N, G, soft, gated, skip, path):
    lens = [17, 0, 1, 2, 3, 70, 16, 15, 33, 130, 0, 9]
    n = len(lens)
    d, state = make(sum(lens) + 7, C, N, G, soft, gated, skip, slots=2 * n + 2, seed=C + N)
    src = [1 + 2 * (r % 4) for r in range(n)]                # shared
    src[4], src[6] = 0, -3
    dst = [2 + 2 * r if r % 5 else 0 for r in range(n)]
    check(d, state, lens, src, dst, soft, first=3, path=path)


@pytest.mark.parametrize("path", [0, 1, 2])
@pytest.mark.parametrize("lens", [[1], [2], [0], [1500], [1, 0, 700, 3, 129]])
def test_state_in_place(lens, path):
    d, state = make(sum(lens) + 1, 40, seed=len(lens))
    slots = [1 + r for r in range(len(lens))]
    check(d, state, lens, slots, slots, path=path)


def test_many_pieces_in_place():
    """900 pieces, more than run at a time: a sequence's last piece writes the state that its
    first ones start from, and all give the bits of separate slots."""
    B, T, C = 300, 800, 64
    d, _ = make(B * T, C, seed=13, extra=8)
    state = torch.randn(2 * B + 1, C, 16, generator=torch.Generator().manual_seed(14)).cuda()
    starts = torch.arange(0, B * T + 1, T, dtype=I32, device="cuda")
    at = torch.arange(1, B + 1, dtype=I32, device="cuda")
    apart, place = state.clone(), state.clone()
    outs = [torch.empty(B * T, C, dtype=BF, device="cuda") for _ in range(2)]
    kda_ssm_prompt(**d, seq_starts=starts, output=outs[0], state=apart, src_slots=at, dst_slots=at + B,
                   path=2, max_seq=T)
    for _ in range(5):
        place.copy_(state)
        kda_ssm_prompt(**d, seq_starts=starts, output=outs[1], state=place, src_slots=at, dst_slots=at,
                       path=2, max_seq=T)
        assert torch.equal(outs[0], outs[1]) and torch.equal(place[1:B + 1], apart[B + 1:])


@pytest.mark.parametrize("path", [1, 2])
def test_without_states_and_without_tokens(path):
    d, state = make(300, 16)
    check(d, state, [17, 280], None, None, path=path)
    d, state = make(0, 16)
    check(d, state, [0, 0], [1, 0], [2, 3], path=path)      # copied, or cleared


@pytest.mark.parametrize("N", [16, 32, 64])
def test_long_sequences_beside_short_ones(N):
    """Automatic layout, a tight and a loose bound of the lengths."""
    lens = [5, 2100, 0, 64, 900]
    d, state = make(sum(lens), 24, N, seed=N, slots=12)
    src, dst = [1, 0, 3, 4, 5], [6, 7, 8, 9, 10]
    tight = check(d, state, lens, src, dst, max_seq=2100)
    loose = check(d, state, lens, src, dst)
    assert torch.equal(tight[:5], loose[:5])


@pytest.mark.parametrize("path", [1, 2])
def test_slow_states_do_not_drift(path):
    """4000 constant steps of decays exp(-1e-7) .. exp(-3e-3), nothing added.  Rounding the
    state itself, which FP32 does once a token, may go the same way every time where the
    decay is below a last place: 4000 x 2^-24 = 2.38e-4.  The exponents (12.5 at most in
    all) are off by three roundings and exp - 1 by 2^-22.9 of itself: 12.5 x 3.1e-7 = 3.9e-6.
    Together 2.43e-4; a factor rounded to FP32 could add 4000 x 2^-25 = 1.19e-4."""
    T, C = 4000, 64
    x = torch.zeros(T, C, dtype=BF, device="cuda")
    dt = torch.full((T, C), 2.0 ** -7, dtype=BF, device="cuda")
    a = -torch.logspace(-5, -0.4, C * 16, device="cuda").view(C, 16)
    b = torch.zeros(T, 16, dtype=BF, device="cuda")
    state = torch.zeros(3, C, 16, device="cuda")
    state[1] = torch.rand(C, 16, generator=torch.Generator().manual_seed(2)).cuda() + 1.0
    kda_ssm_prompt(x=x, dt=dt, a=a, b=b, c=b, softplus=False, seq_starts=i32([0, T]), state=state,
                   output=torch.empty_like(x), src_slots=i32([1]), dst_slots=i32([2]), path=path)
    want = state[1].double() * torch.exp(a.double() * 2.0 ** -7 * T)
    off = (state[2].double() - want) / want
    assert off.abs().max() < 2.43e-4, off.abs().max()
    again = torch.zeros(3, C, 16, device="cuda")
    again[1] = state[1]
    step = KdaSsmStep(x=x[:1], dt=dt[:1], a=a, b=b[:1], c=b[:1], softplus=False, slots=i32([1]), state=again,
                      output=torch.empty_like(x[:1]))
    for _ in range(T):
        step()
    off = (again[1].double() - want) / want
    assert off.abs().max() < 2.43e-4, off.abs().max()


@pytest.mark.parametrize("path", [1, 2])
def test_constant_steps_under_random_inputs(path):
    """Memories of 250 to 2500 tokens (decays exp(-4e-3) .. exp(-4e-4)), inputs of either
    sign.  The state's roundings are random here: 2^-24 / sqrt(3) each over the last
    m / 2 tokens in the square, sqrt(1250) x 3.4e-8 = 1.2e-6 of a state at most, the
    mean over the memories below 1e-6; allowed is twice that.  A factor that FP32 rounds
    is off by 2^-25 / sqrt(3) the same way for m tokens: 1.7e-8 x 2500 = 4.3e-5."""
    T, C = 6000, 64
    g = torch.Generator().manual_seed(12)
    x, b = (torch.randn(T, n, generator=g).to(BF).cuda() for n in (C, 16))
    dt = torch.full((T, C), 2.0 ** -7, dtype=BF, device="cuda")
    a = -torch.logspace(-1.29, -0.29, C * 16, device="cuda").view(C, 16)
    state = torch.zeros(2, C, 16, device="cuda")
    kda_ssm_prompt(x=x, dt=dt, a=a, b=b, c=b, softplus=False, seq_starts=i32([0, T]), state=state,
                   output=torch.empty_like(x), dst_slots=i32([1]), path=path)
    h = torch.zeros(C, 16, dtype=torch.float64, device="cuda")
    f = torch.exp(a.double() * 2.0 ** -7)
    for t in range(T):
        h = h * f + (x[t].double() * 2.0 ** -7)[:, None] * b[t].double()
    off = (state[1].double() - h).norm() / h.norm()
    assert off < 2e-6, off


@pytest.mark.parametrize("path", [1, 2])
def test_strong_decays_and_growth(path):
    """A state that one token wipes out (exp(-4000) = 0), and one that grows."""
    T, C = 600, 8
    d, state = make(T, C, soft=False, seed=3)
    d["dt"] = torch.full((T, C), 0.02, dtype=BF, device="cuda")
    d["dt"][40] = 1000.0
    d["a"][:, 8:] = 0.5                                     # grows by exp(0.01) a token
    d["a"][:, 8:].mul_(0.02)
    state[1] = 1e30
    d["dt"][40, 4:] = 0.02
    d["a"][:4, 8:] = -1.0
    state[1, :, 8:] = 1.0
    state[1, 4:] = 1.0
    check(d, state, [T], [1], [2], soft=False, path=path)


@pytest.mark.parametrize("path", [1, 2])
def test_softplus_over_its_range(path):
    """One token each: dt + bias from -60 (steps of 1e-26) to 60."""
    C = 512
    v = torch.linspace(-60, 60, C)
    d, state = make(1, C, seed=5, slots=3)
    d["dt_bias"] = v.cuda()
    d["a"] = d["a"] * 1e-3
    check(d, state, [1], [1], [2], path=path)


@pytest.mark.parametrize("path", [1, 2])
def test_nan_and_infinity_reach_later_tokens_of_their_channel(path):
    T, C = 700, 24
    d, state = make(T, C, seed=6)
    args = dict(softplus=True, seq_starts=i32([0, 300, T]), path=path)
    clean, out = (torch.empty(T, C, dtype=BF, device="cuda") for _ in range(2))
    kda_ssm_prompt(**d, **args, output=clean)
    e = dict(d, x=d["x"].clone(), dt=d["dt"].clone(), z=d["z"].clone())
    e["x"][100, 3], e["dt"][299, 5], e["z"][50, 7], e["x"][400, 9] = (float("nan"), float("nan"),
                                                                   float("nan"), float("inf"))
    kda_ssm_prompt(**e, **args, output=out)
    odd = torch.zeros(T, C, dtype=torch.bool)
    odd[100:300, 3], odd[299, 5], odd[50, 7], odd[400:, 9] = True, True, True, True
    got = out.cpu()
    assert torch.equal(got[~odd], clean.cpu()[~odd]) and not torch.isfinite(got[odd]).any()


@pytest.mark.parametrize("C,N,G,soft", [(8, 16, 1, True), (1032, 16, 1, False), (64, 32, 2, True),
                                        (40, 64, 1, True)])
def test_steps_follow_the_prompt(C, N, G, soft):
    """Five requests, one of them padding: token by token within the prompt's bounds."""
    T, B = 7, 5
    d, pool = make(T * B, C, N, G, soft, seed=C)
    state = pool.clone()
    slots = [3, 0, 1, 7, -2]
    live = [r for r, s in enumerate(slots) if s > 0]
    starts = [T * r for r in range(B + 1)]
    want, bound, h, hb = mixref.ssm(**d, soft=soft, starts=starts, state=pool, src=slots)
    rows = {k: torch.empty(B, d[k].shape[1], dtype=BF, device="cuda") for k in ("x", "dt", "b", "c", "z")}
    out, err = torch.empty(B, C, dtype=BF, device="cuda"), i32([0])
    step = KdaSsmStep(**rows, a=d["a"], d=d["d"], dt_bias=d["dt_bias"], softplus=soft, slots=i32(slots),
                      state=state, output=out, err=err)
    for t in range(T):
        for k, v in rows.items():
            v.copy_(d[k][t::T])
        out.fill_(float("nan"))
        step()
        got = out.cpu()
        for r in range(B):
            if r in live:
                mixref.inside(got[r], want[r * T + t], bound[r * T + t])
            else:
                assert (got[r] == 0).all()
    for r in live:
        mixref.inside(state[slots[r]], h[r], hb[r])
    rest = [s for s in range(8) if s not in slots]
    assert torch.equal(state[rest], pool[rest]) and int(err) == 0
    step.args.num_slots = 2
    pool = state.clone()
    step()
    assert int(err) == kl.KDA_DEVERR_SLOT and (out[[0, 3]] == 0).all() and (out[2] != 0).any()
    assert torch.equal(state[2:], pool[2:])


@pytest.mark.parametrize("path", [1, 2])
def test_flags(path):
    lens, starts = [5, 800, 7], [0, 5, 805, 812]
    for src, dst in (([1, 8, 2], [3, 4, 5]), ([1, 1, 2], [3, 9, 5])):
        d, state = make(820, 24)
        err, before = i32([0]), state.clone()
        out = torch.full((820, 24), float("nan"), dtype=BF, device="cuda")
        kda_ssm_prompt(**d, seq_starts=i32(starts), output=out, state=state, src_slots=i32(src),
                       dst_slots=i32(dst), err=err, path=path)
        assert int(err) == kl.KDA_DEVERR_SLOT
        want, bound, _, _ = mixref.ssm(**d, starts=starts, state=before, src=[1, 0, 2])
        want[5:805] = float("nan")
        mixref.inside(out, want, bound)
        assert torch.isnan(out[5:805]).all() and torch.equal(state[4], before[4])
    for bad in ([0, 5, 999, 45], [-1, 5, 9, 12], [0, 500, 9, 12], [2 ** 31 - 1, 5, 6, 7], [-2 ** 31, 1, 2, 3]):
        d, state = make(820, 24)
        err, before = i32([0]), state.clone()
        kda_ssm_prompt(**d, seq_starts=i32(bad), output=out, state=state, src_slots=i32([1, 1, 2]),
                       dst_slots=i32([3, 4, 5]), err=err, path=path)
        assert int(err) == kl.KDA_DEVERR_SEQ
        assert torch.equal(state[[0, 1, 2, 6, 7]], before[[0, 1, 2, 6, 7]])
    d, state = make(820, 24)
    err = i32([0])
    out.fill_(float("nan"))
    kda_ssm_prompt(**d, seq_starts=i32(starts), output=out, max_seq=700, err=err, path=path)
    assert int(err) == kl.KDA_DEVERR_SEQ and torch.isnan(out[5:805]).all()
    assert torch.isfinite(out[:5]).all() and torch.isfinite(out[805:812]).all()


@pytest.mark.parametrize("path", [1, 2])
def test_captured_and_replayed_with_other_sequences(path):
    """Two graphs (their workspaces are their own) and an eager call beside them."""
    d, state = make(900, 24, seed=8)
    calls = []
    for k in range(2):
        starts, src, dst = i32([0, 0, 0]), i32([0, 0]), i32([0, 0])
        out = torch.empty(900, 24, dtype=BF, device="cuda")
        args = dict(seq_starts=starts, output=out, state=state, src_slots=src, dst_slots=dst, path=path)
        kda_ssm_prompt(**d, **args)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kda_ssm_prompt(**d, **args)
        calls.append((graph, starts, src, dst, out))
    for lens, srcs, dsts in (([700, 200], [1, 0], [3, 4]), ([30, 860], [2, 1], [5, 6])):
        starts = [5, 5 + lens[0], 5 + sum(lens)] if sum(lens) < 896 else [0, lens[0], sum(lens)]
        for k, (graph, s, a, b, out) in enumerate(calls):
            s.copy_(i32(starts)), a.copy_(i32(srcs)), b.copy_(i32([v if k == 0 else 0 for v in dsts]))
            out.fill_(float("nan"))
        before = state.clone()
        eager = torch.empty(900, 24, dtype=BF, device="cuda")
        torch.cuda.synchronize()
        side = [torch.cuda.Stream() for _ in calls]
        for (graph, *_), stream in zip(calls, side):
            with torch.cuda.stream(stream):
                graph.replay()
        kda_ssm_prompt(**d, seq_starts=i32(starts), output=eager, state=state, src_slots=i32(srcs), path=path)
        torch.cuda.synchronize()
        want, bound, h, hb = mixref.ssm(**d, starts=starts, state=before, src=srcs)
        for got in (calls[0][4], calls[1][4], eager):
            mixref.inside(got, want, bound)
        for r, slot in enumerate(dsts):
            mixref.inside(state[slot], h[r], hb[r])


@pytest.mark.parametrize("path", [1, 2])
def test_repeats_give_the_same_bits(path):
    d, state = make(2000, 136, seed=9)
    outs = []
    for _ in range(10):
        s = state.clone()
        out = torch.empty(2000, 136, dtype=BF, device="cuda")
        kda_ssm_prompt(**d, seq_starts=i32([0, 1200, 1300, 2000]), output=out, state=s, path=path,
                       src_slots=i32([1, 2, 0]), dst_slots=i32([3, 4, 5]))
        outs.append((out, s))
    assert all(torch.equal(o, outs[0][0]) and torch.equal(s, outs[0][1]) for o, s in outs)


def test_rows_and_states_past_32_bit_offsets():
    stride, rows, C = 1 << 15, (1 << 16) + 40, 16
    d, _ = make(60, C, seed=4)
    big = {k: torch.zeros(rows, stride, dtype=BF, device="cuda") for k in ("x", "output")}
    big["x"][-60:, :C] = d["x"]
    state = torch.zeros((1 << 31) // (C * 16) + 3, C, 16, device="cuda")
    n = state.shape[0]
    state[n - 1] = torch.randn(C, 16, generator=torch.Generator().manual_seed(1)).cuda()
    e = dict(d)
    for k in ("dt", "b", "c", "z"):
        full = torch.zeros(rows, d[k].shape[1], dtype=BF, device="cuda")
        full[-60:] = d[k]
        e[k] = full
    e["x"] = big["x"][:, :C]
    for path in (1, 2):
        big["output"].zero_()
        kda_ssm_prompt(**e, seq_starts=i32([rows - 60, rows]), output=big["output"][:, :C], state=state,
                       src_slots=i32([n - 1]), dst_slots=i32([n - 2]), path=path)
        want, bound, h, hb = \
            mixref.ssm(**d, starts=[0, 60], state=torch.stack([state[n - 1], state[n - 1]]), src=[1])
        mixref.inside(big["output"][-60:, :C], want, bound)
        mixref.inside(state[n - 2], h[0], hb[0])
        assert int(torch.count_nonzero(big["output"][:-60])) == 0
    out = torch.zeros(1, C, dtype=BF, device="cuda")
    state[n - 2] = state[n - 1]
    kda_ssm_step(**{k: (v[:1] if k not in ("a", "d", "dt_bias") else v) for k, v in d.items()},
                 slots=i32([n - 2]), state=state, output=out)
    want, bound, h, hb = mixref.ssm(**d, starts=[0, 1], state=torch.stack([state[n - 1]] * 2), src=[1])
    mixref.inside(out, want[:1], bound[:1])
    mixref.inside(state[n - 2], h[0], hb[0])


def test_binding_refuses():
    d, state = make(10, 16)
    out = torch.full((10, 16), float("nan"), dtype=BF, device="cuda")
    good = dict(d, seq_starts=i32([0, 10]), output=out)
    for bad, what in ((dict(x=d["x"].float()), TypeError), (dict(dt=d["dt"][:, :8]), ValueError),
                      (dict(a=d["a"][:, :8].contiguous()), kl.KdaError), (dict(a=d["a"].T), (ValueError, TypeError)),
                      (dict(b=d["b"][:, :8]), ValueError), (dict(c=d["c"][:5]), ValueError),
                      (dict(d=d["d"].to(BF)), TypeError), (dict(z=d["z"].float()), TypeError),
                      (dict(src_slots=i32([1])), ValueError), (dict(state=state[:, :8]), ValueError),
                      (dict(state=state, dst_slots=i32([1, 2])), ValueError), (dict(path=5), kl.KdaError),
                      (dict(seq_starts=torch.tensor([0, 10], device="cuda")), TypeError)):
        with pytest.raises(what):
            kda_ssm_prompt(**{**good, **bad})
    assert torch.isnan(out).all()

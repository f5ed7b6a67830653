"""The short causal convolution on the GPU against its plain form in 64 bits, with
windows compared bit for bit, and against the KDA step's own convolution."""
from __future__ import annotations

import pytest
import torch

from linear_attention_recurrent_kda_gb300 import lib as kl
from linear_attention_recurrent_kda_gb300.api import (KdaConvStep, kda_conv_prompt, kda_conv_step,
                                                      step_from_inputs)
from tests import mixref

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def i32(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def make(rows, C, taps=4, parts=1, width=None, wide=False, bias=True, slots=8, seed=0, extra=40):
    """Inputs; x and output are slices of wider rows, the output's all NaN before."""
    g = torch.Generator().manual_seed(seed)
    shape = (taps, C) if parts == 1 else (parts, taps, C // parts)
    out = torch.full((rows, C + extra), float("nan"), dtype=BF, device="cuda")
    d = dict(x=torch.randn(rows, C + extra, generator=g).to(BF).cuda()[:, 8:8 + C],
             weight=(0.5 * torch.randn(shape, generator=g)).to(BF).cuda(),
             bias=torch.randn(C, generator=g).to(BF).cuda() if bias else None,
             window=torch.randn(slots, C, width or taps - 1, generator=g).to(F32 if wide else BF).cuda())
    return d, out


def check_prompt(d, out, lens, src, dst, silu=True, behind=0, first=0, err=None):
    C, taps = d["x"].shape[1], d["weight"].shape[-2]
    starts = [first]
    for n in lens:
        starts.append(starts[-1] + n)
    before = d["window"].clone()
    kda_conv_prompt(x=d["x"], weight=d["weight"], bias=d["bias"], seq_starts=i32(starts),
                    output=out[:, 16:16 + C], window=d["window"],
                    src_slots=None if src is None else i32(src),
                    dst_slots=None if dst is None else i32(dst), silu=silu, err=err)
    want, bound, last = mixref.conv(d["x"], d["weight"], starts, d["bias"], before, src, silu)
    got = out.cpu()
    mixref.inside(got[:, 16:16 + C], want, bound)
    # what no sequence covers, and the columns beside the output, are left
    assert torch.isnan(got[:, :16]).all() and torch.isnan(got[:, 16 + C:]).all()
    assert torch.isnan(got[:first]).all() and torch.isnan(got[starts[-1]:]).all()
    pool = before.cpu()
    for r, slot in enumerate(dst or []):
        if slot > 0:
            pool[slot, :, :taps - 1] = last[r].to(pool.dtype)
    assert torch.equal(d["window"].cpu(), pool)


@pytest.mark.parametrize("C,parts,taps,width,wide,silu,bias", [
    (8, 1, 4, 3, False, True, True), (24, 3, 4, 3, True, True, False), (264, 1, 3, 2, False, False, True),
    (1032, 1, 2, 1, True, True, True), (96, 3, 4, 6, False, True, False), (48, 2, 3, 5, True, False, False),
    (64, 1, 2, 4, False, True, False)])
def test_ragged_prompts(C, parts, taps, width, wide, silu, bias):
    lens = [33, 0, 1, 2, 3, 64, 31, 32, 5, 97, 0]
    n = len(lens)
    d, out = make(sum(lens) + 9, C, taps, parts, width, wide, bias, slots=2 * n + 2, seed=C)
    src = [1 + 2 * (r % 4) for r in range(n)]                 # shared
    src[4], src[6] = 0, -3
    dst = [2 + 2 * r if r % 5 else 0 for r in range(n)]
    check_prompt(d, out, lens, src, dst, silu, first=4)


@pytest.mark.parametrize("lens", [[1], [2], [3], [4], [200], [0], [1, 2, 0, 3]])
def test_window_in_place_and_short_sequences(lens):
    d, out = make(sum(lens) + 1, 40, seed=7)
    slots = [1 + r for r in range(len(lens))]
    check_prompt(d, out, lens, slots, slots)


def test_without_windows_and_without_tokens():
    d, out = make(40, 16)
    check_prompt(d, out, [17, 20], None, None)
    d, out = make(0, 16)
    check_prompt(d, out, [0, 0], [1, 0], [2, 3])     # windows are copied, or cleared


def test_pieces_chain_bit_for_bit():
    """A prompt in three calls leaves the bits of one call."""
    d, whole = make(150, 72, width=5, seed=3)
    check_prompt(d, whole, [150], [1], [2])
    parts = torch.full_like(whole, float("nan"))
    lo = 0
    for n, src in ((2, 1), (81, 3), (67, 3)):
        kda_conv_prompt(x=d["x"][lo:lo + n], weight=d["weight"], bias=d["bias"], seq_starts=i32([0, n]),
                        output=parts[lo:lo + n, 16:88], window=d["window"], src_slots=i32([src]),
                        dst_slots=i32([3]))
        lo += n
    assert torch.equal(parts[:, 16:88], whole[:, 16:88])
    assert torch.equal(d["window"][3, :, :3], d["window"][2, :, :3])


@pytest.mark.parametrize("C,parts,taps,width,wide", [(8, 1, 4, 3, False), (24, 3, 4, 6, True),
                                                     (2056, 1, 3, 2, True), (136, 1, 2, 3, False),
                                                     (1200, 3, 4, 3, True)])
def test_steps_leave_the_prompt_s_bits(C, parts, taps, width, wide):
    T, B = 5, 3
    d, out = make(T * B, C, taps, parts, width, wide, slots=9, seed=C + 1)
    check_prompt(d, out, [T] * B, [1, 2, 0], [4, 5, 6])
    for slot in (1, 2):
        assert not torch.equal(d["window"][slot, :, :taps - 1], d["window"][slot + 3, :, :taps - 1])
    d["window"][3, :, :taps - 1] = 0
    pool = d["window"].clone()
    y = torch.full((4, C + 8), float("nan"), dtype=BF, device="cuda")
    x = torch.empty(4, C, dtype=BF, device="cuda")
    err = i32([0])
    step = KdaConvStep(x=x, weight=d["weight"], bias=d["bias"], slots=i32([1, 2, 0, 3]), err=err,
                       window=d["window"], output=y[:, :C])
    for t in range(T):
        x.copy_(d["x"][torch.tensor([t, T + t, 0, 2 * T + t], device="cuda")])
        step()
        for row, r in ((0, 0), (1, 1), (3, 2)):
            assert torch.equal(y[row, :C], out[r * T + t, 16:16 + C])
        assert (y[2, :C] == 0).all() and torch.isnan(y[:, C:]).all()
    for slot in range(9):
        n = taps - 1 if slot in (1, 2, 3) else 0
        assert torch.equal(d["window"][slot, :, n:], pool[slot, :, n:])
        if n:
            assert torch.equal(d["window"][slot, :, :n], d["window"][slot + 3, :, :n])
    assert int(err) == 0
    step.args.num_slots = 2                                   # slots 2 and 3 are past the pool
    pool = d["window"].clone()
    step()
    assert int(err) == kl.KDA_DEVERR_SLOT and (y[1:, :C] == 0).all()
    assert torch.equal(d["window"][2:], pool[2:])


def test_flags():
    """Flagged sequences write nothing; in order, the others are as without them."""
    for lens, src, dst, flag in (([5, 40, 7], [1, 8, 2], [3, 4, 5], kl.KDA_DEVERR_SLOT),
                                 ([5, 40, 7], [1, 1, 2], [3, 9, 5], kl.KDA_DEVERR_SLOT)):
        d, out = make(60, 24)
        err, before = i32([0]), d["window"].clone()
        kda_conv_prompt(x=d["x"], weight=d["weight"], bias=d["bias"], seq_starts=i32([0, 5, 45, 52]),
                        output=out[:, 16:40], window=d["window"], src_slots=i32(src),
                        dst_slots=i32(dst), err=err)
        assert int(err) == flag
        want, bound, _ = mixref.conv(d["x"], d["weight"], [0, 5, 45, 52], d["bias"], before, [1, 1, 2])
        want[5:45] = float("nan")
        mixref.inside(out[:, 16:40].cpu(), want, bound)
        assert torch.isnan(out[5:45]).all() and torch.equal(d["window"][4], before[4])
    for starts in ([0, 5, 99, 45], [-1, 5, 9, 12], [0, 50, 9, 12], [2 ** 31 - 1, 5, 6, 7], [-2 ** 31, 1, 2, 3]):
        d, out = make(60, 24)
        err, before = i32([0]), d["window"].clone()
        kda_conv_prompt(x=d["x"], weight=d["weight"], bias=d["bias"], seq_starts=i32(starts),
                        output=out[:, 16:40], window=d["window"], src_slots=i32([1, 1, 2]),
                        dst_slots=i32([3, 4, 5]), err=err)
        assert int(err) == kl.KDA_DEVERR_SEQ
        assert torch.equal(d["window"][[0, 1, 2, 6, 7]], before[[0, 1, 2, 6, 7]])
        assert torch.isnan(out[:, :16]).all() and torch.isnan(out[:, 40:]).all()


def test_nan_and_infinity_reach_their_own_taps_only():
    d, out = make(80, 16, bias=False)
    clean = torch.full_like(out, float("nan"))
    args = dict(weight=d["weight"], seq_starts=i32([0, 30, 70]), window=d["window"], src_slots=i32([1, 2]),
                dst_slots=i32([3, 4]))
    kda_conv_prompt(x=d["x"], output=clean[:, :16], **args)
    x = d["x"].clone()
    x[29, 3], x[40, 5], x[75, 1], d["window"][1, 7, 2] = float("nan"), float("inf"), float("nan"), float("nan")
    kda_conv_prompt(x=x, output=out[:, :16], **args)
    odd = torch.zeros(80, 16, dtype=torch.bool)
    odd[29, 3], odd[40:44, 5], odd[0:3, 7] = True, True, True
    got, want = out[:, :16].cpu(), clean[:, :16].cpu()
    assert torch.equal(got[~odd][~torch.isnan(want[~odd])], want[~odd][~torch.isnan(want[~odd])])
    # an infinity is an infinity, NaN, or silu(-inf) = -0
    assert not torch.isfinite(got[odd & (torch.arange(16) != 5)]).any()
    assert torch.isnan(got[70:]).all()


def test_a_kda_layer_s_prompt_leaves_what_its_decode_would():
    """q, k, v of the KDA step's own convolution, token by token, and the prompt call on
    the same inputs, weights and pool: the same bits."""
    from linear_attention_recurrent_kda_gb300.workloads import WORKLOADS, make_inputs
    inp = make_inputs(WORKLOADS["decode_b4_h8"])
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in inp.items()}
    B, H, T = dev["x"].shape[0], dev["a_log"].shape[0], 6
    g = torch.Generator().manual_seed(11)
    xs = torch.randn(B, T, 3 * H * 128, generator=g).to(BF).cuda()
    window = dev["conv_state"].clone()
    out = torch.empty(B * T, 3 * H * 128, dtype=BF, device="cuda")
    slots = dev["slots"].clone()
    kda_conv_prompt(x=xs.view(B * T, -1), weight=dev["conv_weight"], output=out, window=window,
                    seq_starts=i32([T * r for r in range(B + 1)]), src_slots=slots, dst_slots=slots)
    y = torch.empty(B, H * 128, dtype=BF, device="cuda")
    dbg = torch.zeros(B, H, 1, 4, 128, dtype=BF, device="cuda")
    for t in range(T):
        dev["x"] = xs[:, t].contiguous()
        step_from_inputs(dev, y, dbg=dbg)()
        want = out.view(B, T, 3, H, 128)[:, t].transpose(1, 2)          # [B, H, 3, 128]
        assert torch.equal(dbg[:, :, 0, :3], want)
    assert torch.equal(window, dev["conv_state"])


def test_captured_calls_on_two_streams():
    """Graphs replayed with other starts, inputs and slots; a step on another stream."""
    d, out = make(100, 48, seed=5)
    starts, src, dst = i32([0, 30, 90]), i32([1, 0]), i32([3, 4])
    def call():
        kda_conv_prompt(x=d["x"], weight=d["weight"], bias=d["bias"], seq_starts=starts,
                        output=out[:, 16:64], window=d["window"], src_slots=src, dst_slots=dst)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    side = torch.cuda.Stream()
    y, win = torch.empty(1, 48, dtype=BF, device="cuda"), d["window"].clone()
    for seed, (s, a, b) in enumerate((([0, 30, 90], [1, 0], [3, 4]), ([5, 5, 99], [2, 3], [2, 6]))):
        d["x"].copy_(torch.randn(100, 48, generator=torch.Generator().manual_seed(seed)))
        starts.copy_(i32(s)), src.copy_(i32(a)), dst.copy_(i32(b))
        out.fill_(float("nan"))
        before = d["window"].clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            kda_conv_step(x=d["x"][:1], weight=d["weight"], slots=i32([1]), window=win, output=y)
        graph.replay()
        torch.cuda.synchronize()
        want, bound, last = mixref.conv(d["x"], d["weight"], s, d["bias"], before, a)
        mixref.inside(out[:, 16:64].cpu(), want, bound)
        for r, slot in enumerate(b):
            assert torch.equal(d["window"][slot].cpu().double(), last[r])


def test_rows_past_32_bit_offsets():
    """Rows whose offset in elements passes 2^31, and a window pool that does."""
    C, stride = 64, 1 << 15
    rows = (1 << 16) + 40
    x = torch.zeros(rows, stride, dtype=BF, device="cuda")
    out = torch.zeros(rows, stride, dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(1)
    x[-50:, :C] = torch.randn(50, C, generator=g).to(BF).cuda()
    d, _ = make(1, C, seed=2)
    window = torch.zeros((1 << 31) // (C * 3) + 3, C, 3, dtype=BF, device="cuda")
    n = window.shape[0]
    window[n - 1].copy_(d["window"][1])
    kda_conv_prompt(x=x[:, :C], weight=d["weight"], output=out[:, :C], seq_starts=i32([rows - 50, rows]),
                    window=window, src_slots=i32([n - 1]), dst_slots=i32([n - 2]))
    want, bound, last = mixref.conv(x[-50:, :C], d["weight"], [0, 50], None, window, [n - 1])
    mixref.inside(out[-50:, :C].cpu(), want, bound)
    assert torch.equal(window[n - 2].cpu().double(), last[0]) and int(torch.count_nonzero(out[:-50])) == 0


def test_binding_refuses():
    d, out = make(10, 16)
    good = dict(x=d["x"], weight=d["weight"], seq_starts=i32([0, 10]), output=out[:, :16])
    for bad, what in ((dict(x=d["x"].float()), TypeError), (dict(output=out[:, :24]), ValueError),
                      (dict(weight=d["weight"][:, :8]), ValueError), (dict(src_slots=i32([1])), ValueError),
                      (dict(seq_starts=i32([])), ValueError), (dict(x=d["x"].T), ValueError),
                      (dict(window=d["window"].half()), TypeError), (dict(x=d["x"][:, :15]), ValueError),
                      (dict(window=d["window"], dst_slots=i32([1, 2])), ValueError),
                      (dict(window=d["window"][:, :8], dst_slots=i32([1])), ValueError),
                      (dict(window=d["window"][:, :, :2].contiguous(), dst_slots=i32([1])), kl.KdaError),
                      (dict(stream=torch.cuda.Stream(0), bias=d["weight"][0, :8]), ValueError)):
        with pytest.raises(what):
            kda_conv_prompt(**{**good, **bad})
    assert torch.isnan(out).all()

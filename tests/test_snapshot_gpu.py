"""GPU tests of the snapshots (kda_snapshot_save, kda_snapshot_load): codes,
scales and values are exactly the definition's (tests/linref.py), for ordinary
pages and for ties, tiny, huge, zero and non-finite groups."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from linear_attention_recurrent_kda_gb300 import lib as kl
from linear_attention_recurrent_kda_gb300.api import (kda_lin_prompt, kda_lin_step,
                                                      kda_snapshot_load, kda_snapshot_save)
from tests import linref

pytestmark = pytest.mark.gpu
D = 128


def pools(n, H, bits):
    codes = torch.full((n, H, D, D * bits // 8), 85, device="cuda",
                       dtype=torch.int8 if bits == 8 else torch.uint8)
    scales = torch.full((n, H, D) if bits == 8 else (n, H, D, 4), -3.0, device="cuda")
    return codes, scales


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def same(a, b):
    """Equal bit by bit, any NaN equal to any other."""
    return np.array_equal(a, b, equal_nan=True) and \
        np.array_equal(np.signbit(a) & (a != 0), np.signbit(b) & (b != 0))


def check(pages, bits):
    """Pages [n, H, 128, 128] through save and load, against the definition."""
    n, H = pages.shape[:2]
    state = torch.zeros(2 * n + 1, H, D, D)
    state[1:n + 1] = torch.from_numpy(pages)
    state = state.cuda()
    codes, scales = pools(n + 1, H, bits)
    order = list(range(n, 0, -1))
    kda_snapshot_save(state=state, slots=i32(list(range(1, n + 1))), codes=codes, scales=scales,
                      snaps=i32(order))
    kda_snapshot_load(codes=codes, scales=scales, snaps=i32(order), state=state,
                      slots=i32(list(range(n + 1, 2 * n + 1))))
    torch.cuda.synchronize()
    want_c, want_s = linref.quantise(pages, bits)
    got_c, got_s = codes.cpu().numpy()[order], scales.cpu().numpy()[order]
    assert same(got_s.reshape(want_s.shape), want_s)
    assert np.array_equal(got_c, linref.pack(want_c, bits))
    got = state.cpu().numpy()
    assert same(got[n + 1:], linref.dequantise(want_c, want_s))
    assert np.array_equal(got[1:n + 1].view(np.uint32), pages.view(np.uint32))
    assert np.all(codes[0].cpu().numpy() == 85) and np.all(scales[0].cpu().numpy() == -3.0)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("n,H", [(1, 1), (5, 3), (40, 8)])
def test_random_pages(n, H, bits):
    rng = np.random.default_rng(n + bits)
    x = rng.standard_normal((n, H, D, D)) * np.exp(3 * rng.standard_normal((n, H, D, 1)))
    check(x.astype(np.float32), bits)


@pytest.mark.parametrize("bits", [8, 4])
def test_ties_and_their_neighbours(bits):
    """Elements at and next to the middle between two codes, under scales whose
    reciprocal is not exact."""
    rng = np.random.default_rng(9)
    top = 127 if bits == 8 else 7
    x = np.zeros((1, 2, D, D), np.float32)
    for h in range(2):
        for i in range(D):
            # even scales give middles that FP32 holds: a tie is a real tie
            scale = np.float32(rng.integers(1, 2 ** 12) * 2.0 ** rng.integers(-30, 30))
            c = rng.integers(-top, top, D).astype(np.float64)
            mid = ((c + 0.5) * float(scale)).astype(np.float32)
            up = rng.random(D) < 0.5
            x[0, h, i] = np.nextafter(mid, np.where(up, np.inf, -np.inf).astype(np.float32))
            keep = rng.random(D) < 0.4
            x[0, h, i, keep] = mid[keep]
            x[0, h, i, ::32] = np.float32(top) * scale
    check(x, bits)


@pytest.mark.parametrize("bits", [8, 4])
def test_groups_without_a_scale(bits):
    rng = np.random.default_rng(10)
    x = rng.standard_normal((2, 2, D, D)).astype(np.float32)
    x[0, 0, :8] = 0.0
    x[0, 0, 8:16] *= np.float32(2.0 ** -126)        # subnormal and below the flush
    x[0, 0, 16] = 2.0 ** -118
    x[0, 0, 17] = np.nextafter(np.float32(2.0 ** -118), np.float32(0))
    x[0, 0, 18] = np.finfo(np.float32).max
    x[0, 0, 19] *= np.float32(2.0 ** -117)
    x[0, 1, 3, 5] = np.nan
    x[0, 1, 4, 77] = np.inf
    x[1, 0, 9, 127] = -np.inf
    x[1, 1, :, ::3] = -0.0
    check(x, bits)


@pytest.mark.parametrize("bits", [8, 4])
def test_padding_and_flags(bits):
    rng = np.random.default_rng(11)
    pages = torch.from_numpy(rng.standard_normal((6, 2, D, D)).astype(np.float32)).cuda()
    codes, scales = pools(4, 2, bits)
    err = i32([0])
    kda_snapshot_save(state=pages, slots=i32([1, 0, 2, -1, 3]), codes=codes, scales=scales,
                      snaps=i32([2, 1, 0, 3, -7]), err=err)
    assert int(err) == 0
    for s in (0, 1, 3):
        assert torch.all(codes[s] == 85) and torch.all(scales[s] == -3.0)
    assert not torch.all(codes[2] == 85)
    before = codes.clone()
    kda_snapshot_save(state=pages, slots=i32([6, 1]), codes=codes, scales=scales,
                      snaps=i32([1, 4]), err=err)
    assert int(err) == kl.KDA_DEVERR_SLOT and torch.equal(before, codes)
    err.zero_()
    kept = pages.clone()
    kda_snapshot_load(codes=codes, scales=scales, snaps=i32([2, 4, 0, 2]), state=pages,
                      slots=i32([6, 1, 2, 0]), err=err)
    assert int(err) == kl.KDA_DEVERR_SLOT and torch.equal(kept, pages)


@pytest.mark.parametrize("bits", [8, 4])
def test_one_snapshot_into_several_slots_on_another_stream_and_in_a_graph(bits):
    rng = np.random.default_rng(12)
    state = torch.zeros(6, 3, D, D, device="cuda")
    state[1] = torch.from_numpy(rng.standard_normal((3, D, D)).astype(np.float32))
    codes, scales = pools(2, 3, bits)
    kw = dict(state=state, codes=codes, scales=scales)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    one, snaps, to = i32([1]), i32([1, 1, 1]), i32([3, 5, 2])
    s.wait_stream(torch.cuda.current_stream())
    kda_snapshot_save(**kw, slots=one, snaps=one, stream=s)
    kda_snapshot_load(**kw, snaps=snaps, slots=to, stream=s)
    s.synchronize()
    want = state[3].clone()
    assert not torch.equal(want, torch.zeros_like(want))
    assert torch.equal(want, state[5]) and torch.equal(want, state[2])
    assert torch.all(state[4] == 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda_snapshot_save(**kw, slots=one, snaps=one)
        kda_snapshot_load(**kw, snaps=snaps, slots=to)
    state[2:].zero_()
    codes.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, state[3]) and torch.equal(want, state[2])


def test_saving_what_was_read_back_changes_nothing():
    """8 bits: a page that is read back and saved again keeps its codes."""
    rng = np.random.default_rng(13)
    x = rng.standard_normal((1, 1, D, D)).astype(np.float32)
    c, s = linref.quantise(x, 8)
    c2, s2 = linref.quantise(linref.dequantise(c, s), 8)
    assert np.array_equal(c, c2)
    check(linref.dequantise(c, s), 8)


def test_snapshots_past_32_bit_offsets():
    H, n = 64, 2 ** 31 // (64 * D * D) + 2
    state = torch.zeros(n, H, D, D, device="cuda")
    state[n - 1] = torch.randn(H, D, D, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    codes = torch.zeros(n, H, D, D, dtype=torch.int8, device="cuda")
    scales = torch.zeros(n, H, D, device="cuda")
    kda_snapshot_save(state=state, slots=i32([n - 1]), codes=codes, scales=scales,
                      snaps=i32([n - 1]))
    kda_snapshot_load(codes=codes, scales=scales, snaps=i32([n - 1]), state=state,
                      slots=i32([n - 2]))
    c, s = linref.quantise(state[n - 1].cpu().numpy(), 8)
    assert same(state[n - 2].cpu().numpy(), linref.dequantise(c, s))
    assert torch.all(state[1] == 0) and torch.all(state[0] == 0)


@pytest.mark.parametrize("bits,path", [(8, 0), (4, 0), (8, 1), (8, 2)])
def test_prefix_cache_run(bits, path):
    """As a server uses them: a prefix is run once, its page kept as a snapshot,
    two requests start from the snapshot, run their own suffixes and decode.
    Everything after the snapshot is compared with the recurrence in 64 bits
    from the page as it is read back."""
    H, Hk, scale = 4, 2, 0.25
    g = torch.Generator().manual_seed(3 + bits + path)

    def rnd(n, heads):
        return torch.randn(n, heads * D, generator=g).div(4).to(torch.bfloat16)

    def part(n):
        return dict(q=rnd(n, Hk), k=rnd(n, Hk), v=rnd(n, H),
                    decay=-0.3 * torch.rand(n, H, generator=g))

    state = torch.zeros(6, H, D, D, device="cuda")
    codes, scales = pools(3, H, bits)

    def prompt(x, starts, src, dst):
        out = torch.zeros(x["v"].shape, dtype=torch.bfloat16, device="cuda")
        kda_lin_prompt(**{n: t.cuda() for n, t in x.items()}, seq_starts=i32(starts), output=out,
                       scale=scale, state=state, src_slots=None if src is None else i32(src),
                       dst_slots=i32(dst), max_seq=max(b - a for a, b in zip(starts, starts[1:])),
                       path=path)
        return out.cpu()

    prefix, suffix, token = part(300), part(150), part(2)
    prompt(prefix, [0, 300], None, [1])
    kda_snapshot_save(state=state, slots=i32([1]), codes=codes, scales=scales, snaps=i32([2]))
    kda_snapshot_load(codes=codes, scales=scales, snaps=i32([2, 2]), state=state,
                      slots=i32([3, 4]))
    first = state.cpu()
    c, s = linref.quantise(first[1].numpy(), bits)
    for slot in (3, 4):
        assert same(first[slot].numpy(), linref.dequantise(c, s))
    starts = [0, 21, 150]
    out = prompt(suffix, starts, [3, 4], [3, 4])
    ref, mag, S, M = linref.prompt(*(suffix[n] for n in ("q", "k", "v", "decay")), starts, scale,
                                   first, [3, 4])
    for r in range(2):
        a, b = starts[r], starts[r + 1]
        assert torch.all((out[a:b].double() - ref[a:b]).abs()
                         <= linref.out_bound(ref[a:b], mag[a:b], b - a, True))
    mid = state.cpu()
    for r in range(2):
        assert torch.all((mid[3 + r].double() - S[r]).abs()
                         <= linref.state_bound(M[r], starts[r + 1] - starts[r]))
    o = torch.zeros(2, H * D, dtype=torch.bfloat16, device="cuda")
    kda_lin_step(**{n: t.cuda() for n, t in token.items()}, slots=i32([3, 4]), state=state,
                 output=o, scale=scale)
    ref, mag, S, M = linref.prompt(*(token[n] for n in ("q", "k", "v", "decay")), [0, 1, 2], scale,
                                   mid, [3, 4])
    assert torch.all((o.cpu().double() - ref).abs() <= linref.out_bound(ref, mag, 1, False))
    end = state.cpu()
    for r in range(2):
        assert torch.all((end[3 + r].double() - S[r]).abs() <= 5 * linref.U32 * M[r])


def test_refusals_of_the_binding():
    state = torch.zeros(4, 2, D, D, device="cuda")
    codes, scales = pools(3, 2, 8)
    base = dict(state=state, slots=i32([1, 2]), codes=codes, scales=scales, snaps=i32([1, 2]))
    for kw, error in [
            (dict(state=state.double()), TypeError),
            (dict(state=state[:, :, :64].contiguous()), ValueError),
            (dict(state=state.transpose(2, 3)), ValueError),
            (dict(codes=codes.short()), TypeError),
            (dict(codes=codes[:, :1].contiguous()), ValueError),
            (dict(codes=codes.view(torch.uint8)), ValueError),
            (dict(codes=codes[:2].contiguous()), ValueError),
            (dict(scales=scales[:, :, :64].contiguous()), ValueError),
            (dict(slots=i32([1])), ValueError),
            (dict(snaps=base["snaps"].long()), TypeError),
            (dict(slots=i32([[1, 2]])), ValueError),
            (dict(scales=scales.cpu()), ValueError)]:
        for f in (kda_snapshot_save, kda_snapshot_load):
            with pytest.raises(error):
                f(**dict(base, **kw))
    torch.cuda.synchronize()
    assert torch.all(codes == 85) and torch.all(state == 0)

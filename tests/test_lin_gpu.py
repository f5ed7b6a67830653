"""GPU tests of the linear attention with one decay per head (kda_lin_prompt,
kda_lin_step) against the recurrence in 64 bits; bounds from tests/linref.py."""
from __future__ import annotations

import pytest
import torch

from linear_attention_recurrent_kda_gb300 import lib as kl
from linear_attention_recurrent_kda_gb300.api import KdaLinStep, kda_lin_prompt, kda_lin_step
from tests import linref

pytestmark = pytest.mark.gpu
D = 128
bf16 = torch.bfloat16


def rows(g, n, heads, unit=False):
    x = torch.randn(n, heads, D, generator=g)
    if unit:
        x = x / x.norm(dim=-1, keepdim=True)
    return x.view(n, heads * D).to(bf16)


def make(lens, H, Hk, *, per_token=True, slots=0, seed=1, behind=0, scale_g=1.0):
    """Inputs on the CPU; `behind` rows follow the last sequence."""
    g = torch.Generator().manual_seed(seed)
    n = sum(lens) + behind
    starts = [0]
    for x in lens:
        starts.append(starts[-1] + x)
    decay = -scale_g * torch.rand(*((n, H) if per_token else (H,)), generator=g)
    return dict(q=rows(g, n, Hk, True), k=rows(g, n, Hk, True), v=rows(g, n, H), decay=decay,
                starts=starts,
                state=torch.randn(slots, H, D, D, generator=g) * 0.3 if slots else None)


def launch(inp, *, src=None, dst=None, path=0, max_seq=None, stream=None, fill=float("nan"),
           scale=0.5, err=None, **over):
    """One call on device copies; returns (output, state) on the CPU."""
    dev = {n: inp[n].cuda() for n in ("q", "k", "v", "decay")}
    dev.update(over)
    state = inp["state"].cuda() if inp["state"] is not None else None
    out = torch.full((inp["v"].shape[0], inp["v"].shape[1]), fill, dtype=bf16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    kda_lin_prompt(**dev, seq_starts=torch.tensor(inp["starts"], **i32), output=out, scale=scale,
                   state=state, src_slots=None if src is None else torch.tensor(src, **i32),
                   dst_slots=None if dst is None else torch.tensor(dst, **i32), path=path,
                   max_seq=max_seq, stream=stream, err=err)
    torch.cuda.synchronize()
    return out.cpu(), None if state is None else state.cpu()


def verify(inp, got, path, src=None, dst=None, scale=0.5):
    out, state = got
    starts = inp["starts"]
    ref, mag, S, M = linref.prompt(inp["q"], inp["k"], inp["v"], inp["decay"], starts, scale,
                                   inp["state"], src)
    for r in range(len(starts) - 1):
        a, b = starts[r], starts[r + 1]
        bound = linref.out_bound(ref[a:b], mag[a:b], b - a, path != 1)
        off = (out[a:b].double() - ref[a:b]).abs()
        assert torch.all(off <= bound), (r, a, b, float((off / bound).max()))
        if dst is not None and dst[r] > 0:
            off = (state[dst[r]].double() - S[r]).abs()
            bound = linref.state_bound(M[r], b - a)
            assert torch.all(off <= bound), (r, float((off / bound.clamp_min(1e-30)).max()))
    # rows behind the last sequence and pages nobody writes stay as they were
    assert torch.all(torch.isnan(out[starts[-1]:]))
    if state is not None:
        written = {s for s in dst or [] if s > 0}
        for s in range(state.shape[0]):
            if s not in written:
                assert torch.equal(state[s], inp["state"][s]), s


PATHS = [1, 2]
LENS = [[1], [2, 1], [5, 0, 3], [127], [128], [129, 1], [31, 32, 33, 64, 65], [255, 256, 257],
        [400, 7, 0, 130]]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("lens", LENS, ids=lambda v: "-".join(map(str, v)))
@pytest.mark.parametrize("H,Hk,per_token", [(2, 2, True), (4, 1, False), (3, 3, True)])
def test_prompt(lens, H, Hk, per_token, path):
    B = len(lens)
    inp = make(lens, H, Hk, per_token=per_token, slots=2 * B + 2, seed=sum(lens) + H, behind=5)
    # every other sequence starts from a page, the last one's state is dropped
    src = [r + 1 if r % 2 == 0 else 0 for r in range(B)]
    dst = [B + 1 + r for r in range(B)]
    if B > 1:
        dst[-1] = 0
    verify(inp, launch(inp, src=src, dst=dst, path=path), path, src, dst)


@pytest.mark.parametrize("lens", [[1300], [1, 1536, 513, 512, 40], [600, 1024, 1025]],
                         ids=lambda v: "-".join(map(str, v)))
@pytest.mark.parametrize("H,Hk,per_token", [(2, 1, True), (1, 1, False)])
def test_long_sequences_in_segments(lens, H, Hk, per_token):
    """Few heads and long sequences: the chunked form splits them into segments."""
    B = len(lens)
    inp = make(lens, H, Hk, per_token=per_token, slots=2 * B + 1, seed=sum(lens), behind=3,
               scale_g=0.05)
    assert kl.prompt_workspace(kl.KdaLinPromptArgs(
        seqs=B, heads=H, qk_heads=Hk, tokens=sum(lens) + 3, max_seq=max(lens), q_stride=Hk * D,
        k_stride=Hk * D, v_stride=H * D, o_stride=H * D)) > 0
    src = [r + 1 if r % 2 == 0 else 0 for r in range(B)]
    dst = [r + 1 for r in range(B)]                     # in place, where carried
    verify(inp, launch(inp, src=src, dst=dst, max_seq=max(lens)), 2, src, dst)


@pytest.mark.parametrize("lens,max_seq", [([1500] + [7, 40, 0] * 27 + [1400, 300], 1500),
                                          ([60, 129] * 20, None)], ids=["mixed", "loose bound"])
def test_split_sequences_among_many(lens, max_seq):
    """Two split sequences among 81 short ones, and a bound on the lengths that
    would allow splits where there are none."""
    B = len(lens)
    inp = make(lens, 2, 2, slots=2 * B + 1, seed=24, scale_g=0.1)
    src = [r + 1 if r % 3 else 0 for r in range(B)]
    dst = [B + 1 + r for r in range(B)]
    verify(inp, launch(inp, src=src, dst=dst, max_seq=max_seq), 2, src, dst)


def test_segments_of_many_chunks():
    """Segments of 7 chunks (every buffer comes round), checked on two heads."""
    H, n, heads = 64, 8192 + 77, (5, 63)
    inp = make([n], H, H, slots=3, seed=16, scale_g=0.02)
    args = kl.KdaLinPromptArgs(seqs=1, heads=H, qk_heads=H, tokens=n, max_seq=n, q_stride=H * D,
                               k_stride=H * D, v_stride=H * D, o_stride=H * D)
    assert kl.prompt_workspace(args) > 0
    out, state = launch(inp, src=[2], dst=[2])
    for h in heads:
        sl = slice(h * D, h * D + D)
        ref, mag, S, M = linref.prompt(inp["q"][:, sl], inp["k"][:, sl], inp["v"][:, sl],
                                       inp["decay"][:, h:h + 1], [0, n], 0.5,
                                       inp["state"][:, h:h + 1], [2])
        off = (out[:, sl].double() - ref).abs()
        assert torch.all(off <= linref.out_bound(ref, mag, n, True))
        assert torch.all((state[2, h:h + 1].double() - S[0]).abs() <= linref.state_bound(M[0], n))


@pytest.mark.parametrize("path", PATHS)
def test_without_a_state(path):
    inp = make([3, 140], 2, 2, seed=5)
    verify(inp, launch(inp, path=path), path)


@pytest.mark.parametrize("path", PATHS)
def test_page_in_place_and_shared(path):
    """A sequence may write the page it starts from; two may start from one page."""
    inp = make([150, 33, 70], 2, 1, slots=5, seed=6)
    src, dst = [1, 4, 4], [1, 2, 3]
    verify(inp, launch(inp, src=src, dst=dst, path=path), path, src, dst)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("how", ["reset", "none", "strong", "mixed"])
def test_decays(path, how):
    """Decays of -inf (a reset), 0 (none) and far below the smallest factor."""
    inp = make([300, 40], 2, 2, slots=4, seed=7)
    g = inp["decay"]
    if how == "reset":
        g[torch.randperm(340, generator=torch.Generator().manual_seed(1))[:20], 0] = -float("inf")
        g[150:155] = -float("inf")
    elif how == "none":
        g.zero_()
    elif how == "strong":
        g.mul_(60.0)
    else:
        g[::7] *= 200.0
        g[::3] = 0.0
    src, dst = [1, 0], [2, 3]
    verify(inp, launch(inp, src=src, dst=dst, path=path), path, src, dst)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_outside_a_sequence_reach_nothing(path, bad):
    """Non-finite rows behind the last sequence, and of another sequence, leave
    the others' outputs and pages as they are without them."""
    inp = make([70, 130, 9], 2, 2, slots=5, seed=8, behind=140)
    src, dst = [1, 0, 0], [2, 3, 4]
    clean = launch(inp, src=src, dst=dst, path=path)
    dirty = {n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in inp.items()}
    for n in ("q", "k", "v", "decay"):
        dirty[n][209:] = bad
        dirty[n][70:200] = bad
    got = launch(dirty, src=src, dst=dst, path=path)
    for a, b in ((0, 70), (200, 209)):
        assert torch.equal(got[0][a:b], clean[0][a:b])
    assert torch.equal(got[1][2], clean[1][2]) and torch.equal(got[1][4], clean[1][4])
    assert torch.all(torch.isnan(got[0][209:]))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("strong", [False, True])
def test_non_finite_values_reach_no_earlier_token(path, bad, strong):
    """Infinities and NaN among a sequence's own values: the tokens before, the
    other columns, heads and sequences stay as they are without them, the column
    itself is non-finite from there on."""
    lens = [300, 128, 70, 5]
    inp = make(lens, 2, 1, slots=9, seed=31, scale_g=6.0 if strong else 0.3)
    src, dst = [1, 2, 0, 4], [5, 6, 7, 8]
    clean = launch(inp, src=src, dst=dst, path=path)
    # (token, column): ends of chunks, of 8, 32 and 64 columns, twice in one column
    places = [(127, 0), (128, 7), (255, 8), (130, 31), (250, 31), (299, 63), (0, 64), (260, 127),
              (150, 128 + 5), (300, 33), (427, 200), (428 + 33, 255), (428 + 69, 1), (498, 90)]
    dirty = dict(inp, v=inp["v"].clone())
    for t, col in places:
        dirty["v"][t, col] = bad
    got = launch(dirty, src=src, dst=dst, path=path)
    out, state = clean[0].clone(), clean[1].clone()
    gone = torch.zeros(out.shape, dtype=torch.bool)
    rows_gone = torch.zeros(state.shape[:3], dtype=torch.bool)
    for t, col in places:
        r = max(i for i in range(4) if inp["starts"][i] <= t)
        gone[t:inp["starts"][r + 1], col] = True
        rows_gone[dst[r], col // D, col % D] = True
    assert not torch.any(torch.isfinite(got[0][gone]))
    assert torch.equal(got[0][~gone], out[~gone])
    assert not torch.any(torch.isfinite(got[1][rows_gone]))
    assert torch.equal(got[1][~rows_gone], state[~rows_gone])


def test_non_finite_values_in_segments():
    """The same in a sequence that is split."""
    inp = make([1300], 1, 1, slots=2, seed=32, scale_g=0.05)
    clean = launch(inp, dst=[1], path=2)
    v = inp["v"].clone()
    v[700, 3], v[1290, 100] = float("nan"), float("inf")
    got = launch(dict(inp, v=v), dst=[1], path=2)
    gone = torch.zeros(v.shape, dtype=torch.bool)
    gone[700:, 3] = gone[1290:, 100] = True
    assert not torch.any(torch.isfinite(got[0][gone]))
    assert torch.equal(got[0][~gone], clean[0][~gone])
    assert not torch.any(torch.isfinite(got[1][1, 0, [3, 100]]))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("name", ["q", "k", "decay"])
def test_non_finite_inputs_reach_no_earlier_token(path, name):
    """A NaN query spoils its own token's outputs, a NaN key or decay its own
    and the later ones of its sequence and head."""
    inp = make([300, 20], 2, 2, slots=3, seed=33)
    clean = launch(inp, dst=[1, 2], path=path)
    x = inp[name].clone()
    x[170, 1 if name == "decay" else 200] = float("nan")
    got = launch(dict(inp, **{name: x}), dst=[1, 2], path=path)
    gone = torch.zeros(got[0].shape, dtype=torch.bool)
    gone[170:171 if name == "q" else 300, 128:] = True
    assert torch.all(torch.isnan(got[0][gone]))
    same = ~gone
    if path == 2 and name == "decay":
        # (the chunk's factors take another form beside a NaN: within the bound instead)
        same[128:170, 128:] = False
        ref, mag, _, _ = linref.prompt(inp["q"], inp["k"], inp["v"], inp["decay"], inp["starts"],
                                       0.5)
        at = (slice(128, 170), slice(128, 256))
        off = (got[0][at].double() - ref[at]).abs()
        assert torch.all(off <= linref.out_bound(ref[at], mag[at], 300, True))
    assert torch.equal(got[0][same], clean[0][same])


@pytest.mark.parametrize("path", PATHS)
def test_slices_of_wider_rows(path):
    """q, k and v as column slices of one projection, the output as a slice too."""
    inp = make([200, 37], 2, 2, slots=3, seed=9)
    x = torch.full((237, 3 * 256 + 40), float("nan"), dtype=bf16)
    for i, n in enumerate("qkv"):
        x[:, 8 + 256 * i:8 + 256 * (i + 1)] = inp[n]
    x = x.cuda()
    out = torch.full((237, 512), float("nan"), dtype=bf16, device="cuda")
    state = inp["state"].cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    kda_lin_prompt(q=x[:, 8:264], k=x[:, 264:520], v=x[:, 520:776], decay=inp["decay"].cuda(),
                   seq_starts=torch.tensor(inp["starts"], **i32), output=out[:, 128:384],
                   scale=0.5, state=state, dst_slots=torch.tensor([2, 1], **i32), path=path)
    torch.cuda.synchronize()
    verify(inp, (out[:, 128:384].cpu(), state.cpu()), path, None, [2, 1])
    assert torch.all(torch.isnan(out[:, :128])) and torch.all(torch.isnan(out[:, 384:]))


@pytest.mark.parametrize("path", PATHS)
def test_flagged_sequences_write_nothing(path):
    inp = make([40, 50, 60, 70], 2, 2, slots=6, seed=10)
    good = launch(inp, src=[1, 0, 0, 0], dst=[2, 3, 4, 5], path=path)

    def check(src, dst, starts, flag, bad, max_seq=None):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = launch(dict(inp, starts=starts), src=src, dst=dst, path=path, err=err,
                     max_seq=max_seq)
        assert int(err) == flag
        for r in range(4):
            a, b = inp["starts"][r], inp["starts"][r + 1]
            if r in bad:
                assert torch.all(torch.isnan(got[0][a:b])), r
                assert torch.equal(got[1][r + 2], inp["state"][r + 2])
            else:
                assert torch.equal(got[0][a:b], good[0][a:b]), r
                assert torch.equal(got[1][r + 2], good[1][r + 2])

    starts = inp["starts"]
    check([1, 6, 0, 0], [2, 3, 4, 5], starts, kl.KDA_DEVERR_SLOT, {1})
    check([1, 0, 0, 0], [2, 3, 99, 5], starts, kl.KDA_DEVERR_SLOT, {2})
    check([1, 0, 0, 0], [2, 3, 4, 5], starts[:4] + [221], kl.KDA_DEVERR_SEQ, {3})
    check([1, 0, 0, 0], [2, 3, 4, 5], [-1] + starts[1:], kl.KDA_DEVERR_SEQ, {0})
    check([1, 0, 0, 0], [2, 3, 4, 5], starts, kl.KDA_DEVERR_SEQ, {3}, max_seq=60)
    check([1, 0, 0, 0], [2, 3, 4, 5], [0, 40, 30, 150, 220], kl.KDA_DEVERR_SEQ, {1, 2},
          max_seq=70)


@pytest.mark.parametrize("path", PATHS)
def test_other_stream_and_graph(path):
    inp = make([260, 33], 2, 2, slots=5, seed=11)
    src, dst = [1, 0], [3, 4]
    want = launch(inp, src=src, dst=dst, path=path)
    s = torch.cuda.Stream()
    got = launch(inp, src=src, dst=dst, path=path, stream=s)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    dev = {n: inp[n].cuda() for n in ("q", "k", "v", "decay", "state")}
    i32 = dict(dtype=torch.int32, device="cuda")
    out = torch.zeros(293, 256, dtype=bf16, device="cuda")
    kw = dict(dev, seq_starts=torch.tensor(inp["starts"], **i32), output=out, scale=0.5,
              src_slots=torch.tensor(src, **i32), dst_slots=torch.tensor(dst, **i32), path=path)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda_lin_prompt(**kw)
    for _ in range(3):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want[0], out.cpu())
    assert torch.equal(want[1], dev["state"].cpu())


def on_device(inp, src=None, dst=None, **kw):
    """The arguments of one call, as device copies of its own."""
    i32 = dict(dtype=torch.int32, device="cuda")
    n, width = inp["v"].shape
    a = {x: inp[x].cuda() for x in ("q", "k", "v", "decay", "state")}
    return dict(a, seq_starts=torch.tensor(inp["starts"], **i32), scale=0.5,
                output=torch.zeros(n, width, dtype=bf16, device="cuda"),
                src_slots=None if src is None else torch.tensor(src, **i32),
                dst_slots=None if dst is None else torch.tensor(dst, **i32), **kw)


def test_split_calls_on_two_streams_and_in_two_graphs():
    """Calls that need a workspace, at the same time on two streams and replayed
    from two graphs in turn, do not share it."""
    inps = [make([1500, 200], 2, 2, slots=4, seed=20), make([1400], 2, 1, slots=4, seed=21)]
    wants = [launch(x, src=[1] * (len(x["starts"]) - 1), dst=[2, 3][:len(x["starts"]) - 1])
             for x in inps]

    def check(kws):
        torch.cuda.synchronize()
        for kw, want in zip(kws, wants):
            assert torch.equal(kw["output"].cpu(), want[0])
            assert torch.equal(kw["state"].cpu(), want[1])

    def fresh():
        return [on_device(x, [1] * (len(x["starts"]) - 1), [2, 3][:len(x["starts"]) - 1])
                for x in inps]

    kws, streams = fresh(), [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for kw, s in zip(kws, streams):
            kda_lin_prompt(**kw, stream=s)
    check(kws)
    kws, graphs = fresh(), [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for kw, graph in zip(kws, graphs):
        with torch.cuda.graph(graph):
            kda_lin_prompt(**kw)
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    check(kws)


@pytest.mark.parametrize("lens,H,Hk", [([700, 33, 128, 1, 500, 256], 32, 8), ([2600, 90], 8, 8)])
def test_relaunches_give_the_same_bits(lens, H, Hk):
    """300 launches in a row, whole sequences and split ones, decays mild and
    strong: every one has the first one's bits."""
    B = len(lens)
    inp = make(lens, H, Hk, slots=2 * B + 1, seed=23, scale_g=0.1)
    inp["decay"][:, ::3] *= 40.0                       # strong chunks in every third head
    kw = on_device(inp, [1 + r for r in range(B)], [B + 1 + r for r in range(B)], max_seq=max(lens))
    kda_lin_prompt(**kw)
    out, state = kw["output"].clone(), kw["state"].clone()
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        kw["output"].fill_(float("nan"))
        kw["state"][B + 1:].fill_(float("nan"))
        kda_lin_prompt(**kw)
        bad += (kw["output"] != out).sum() + (kw["state"] != state).sum()
    assert int(bad) == 0


@pytest.mark.parametrize("path", PATHS)
def test_rows_past_32_bit_offsets(path):
    """The last rows of tensors of more than 2^31 elements."""
    H, n = 64, 2 ** 31 // (64 * D) + 301
    inp = make([200, 61], H, H, seed=22)
    want = launch(inp, path=path)[0]
    big = {x: torch.zeros(n, H * D, dtype=bf16, device="cuda") for x in ("q", "k", "v", "output")}
    decay = torch.zeros(n, H, device="cuda")
    for x in ("q", "k", "v"):
        big[x][-261:] = inp[x].cuda()
    decay[-261:] = inp["decay"].cuda()
    kda_lin_prompt(**big, decay=decay, scale=0.5, path=path, max_seq=200,
                   seq_starts=torch.tensor([n - 261, n - 61, n], dtype=torch.int32, device="cuda"))
    assert torch.equal(big["output"][-261:].cpu(), want)
    assert not big["output"][:-261].any()


@pytest.mark.parametrize("B,H", [(200, 4), (700, 3), (900, 2), (1, 300)])
def test_many_units(B, H):
    """More units than SMs: dealt by length (up to 8 a CTA and 768 sequences) and
    in turn.  Sequences of the same rows and lengths give the same bits wherever
    they run."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(1, 140, (B,), generator=g).tolist()
    lens[::7] = [0] * len(lens[::7])
    lens[0] = 33
    base = make([140], H, 1, slots=2, seed=B)
    starts, rows = [0], []
    for x in lens:
        starts.append(starts[-1] + x)
        rows += list(range(x))
    at = torch.tensor(rows)
    inp = dict(base, **{x: base[x][at] for x in ("q", "k", "v", "decay")}, starts=starts)
    inp["state"] = torch.zeros(B + 2, H, D, D)
    inp["state"][1] = base["state"][1]
    out, state = launch(inp, src=[1] * B, dst=list(range(2, B + 2)), path=2, max_seq=140)
    first = {}
    for r, x in enumerate(lens):
        a, b = starts[r], starts[r + 1]
        if x not in first:
            one = {k: v[a:b] if k in ("q", "k", "v", "decay") else v for k, v in inp.items()}
            one.update(starts=[0, x], state=torch.cat([inp["state"][:2], inp["state"][:1]]))
            first[x] = launch(one, src=[1], dst=[2], path=2)
        assert torch.equal(out[a:b], first[x][0]), r
        assert torch.equal(state[r + 2], first[x][1][2]), r


# ------------------------------------------------------------------------- step

def step_ref(inp, state, slots, scale):
    """Values and magnitudes of one step per live request."""
    B = len(slots)
    return linref.prompt(inp["q"], inp["k"], inp["v"], inp["decay"], list(range(B + 1)), scale,
                         state, slots)


@pytest.mark.parametrize("B,H,Hk,per_token", [(1, 1, 1, True), (7, 2, 1, False), (33, 5, 5, True),
                                              (3, 64, 8, True)])
def test_step(B, H, Hk, per_token):
    inp = make([1] * B, H, Hk, per_token=per_token, slots=B + 3, seed=B)
    g = torch.Generator().manual_seed(B)
    slots = (torch.randperm(B + 2, generator=g)[:B] + 1).to(torch.int32)
    if B > 2:
        slots[1], slots[2] = 0, -4
    state = inp["state"].cuda()
    out = torch.full((B, H * D), float("nan"), dtype=bf16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = {n: inp[n].cuda() for n in ("q", "k", "v", "decay")}
    kda_lin_step(**kw, slots=slots.cuda(), state=state, output=out, scale=0.7, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    sl = slots.tolist()
    ref, mag, S, M = step_ref(inp, inp["state"], sl, 0.7)
    for r, s in enumerate(sl):
        if s <= 0:
            assert torch.all(out[r].cpu().view(torch.int16) == 0)
            continue
        off = (out[r].cpu().double() - ref[r]).abs()
        assert torch.all(off <= linref.out_bound(ref[r], mag[r], 1, False))
        off = (state[s].cpu().double() - S[r]).abs()
        assert torch.all(off <= 5 * linref.U32 * M[r])
    for s in set(range(B + 3)) - set(sl):
        assert torch.equal(state[s].cpu(), inp["state"][s])


def test_step_flags_a_slot_past_the_pool():
    inp = make([1] * 3, 2, 2, slots=4, seed=3)
    kw = {n: inp[n].cuda() for n in ("q", "k", "v", "decay", "state")}
    out = torch.full((3, 256), float("nan"), dtype=bf16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda_lin_step(**kw, slots=torch.tensor([1, 4, 2], dtype=torch.int32).cuda(), output=out,
                 scale=1.0, err=err)
    assert int(err) == kl.KDA_DEVERR_SLOT
    assert torch.all(out[1].view(torch.int16) == 0) and torch.isfinite(out).all()
    assert torch.equal(kw["state"][3].cpu(), inp["state"][3])


def test_steps_from_a_page_past_32_bit_offsets():
    """The last pages of a pool of more than 2^31 floats (prompt and step)."""
    H, slots = 64, 2 ** 31 // (64 * D * D) + 3
    state = torch.zeros(slots, H, D, D, device="cuda")
    inp = make([140], H, H, seed=4)
    kw = {n: inp[n].cuda() for n in ("q", "k", "v", "decay")}
    i32 = dict(dtype=torch.int32, device="cuda")
    out = torch.zeros(140, H * D, dtype=bf16, device="cuda")
    small = torch.zeros(3, H, D, D, device="cuda")
    for pool, last in ((state, slots - 1), (small, 2)):
        for path in PATHS:
            kda_lin_prompt(**kw, seq_starts=torch.tensor([0, 140], **i32), output=out, scale=1.0,
                           state=pool, dst_slots=torch.tensor([last - (path == 1)], **i32),
                           path=path)
        one = {n: t[:1] if t.dim() == 2 else t for n, t in kw.items()}
        o = torch.zeros(1, H * D, dtype=bf16, device="cuda")
        kda_lin_step(**one, slots=torch.tensor([last], **i32), state=pool, output=o, scale=1.0)
    assert torch.equal(state[slots - 2:], small[1:])


def test_prepared_step_repeats_and_replays():
    """KdaLinStep over changing contents, eagerly and from a graph: the same bits."""
    inp = make([1] * 6, 4, 2, slots=8, seed=12)
    kw = {n: inp[n].cuda() for n in ("q", "k", "v", "decay")}
    slots = torch.tensor([3, 1, 0, 7, 5, 2], dtype=torch.int32, device="cuda")
    res = []
    for mode in ("eager", "graph"):
        state, out = inp["state"].cuda(), torch.zeros(6, 512, dtype=bf16, device="cuda")
        x = {n: t.clone() for n, t in kw.items()}
        step = KdaLinStep(**x, slots=slots, state=state, output=out, scale=0.3)
        if mode == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        outs = []
        for t in range(4):
            for n in "qkv":
                x[n].copy_(kw[n].roll(t, 0))
            graph.replay() if mode == "graph" else step()
            outs.append(out.clone())
        torch.cuda.synchronize()
        res.append((torch.stack(outs), state))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


@pytest.mark.parametrize("path", PATHS)
def test_slow_decays_over_many_tokens(path):
    """A decay near 1, the same at every token, does not drift: the last page
    after 6000 tokens is within 2e-6 of the 64-bit recurrence (2-norm).  A token
    rounds the page twice, at random (6000 ** 0.5 * 2 ** -24 = 5e-6 if all of them
    stayed; with a decay of exp(-1e-3) the last 1000 do: 2e-6, times the share of
    a uniform rounding error, 3 ** -0.5); a factor rounded to FP32 would be off by
    up to 2 ** -25 every time, 3e-5."""
    n = 6000
    inp = make([n], 1, 1, slots=3, seed=25)
    inp["decay"] = torch.full((1,), -1e-3)
    _, state = launch(inp, src=[1], dst=[2], path=path)
    _, _, S, _ = linref.prompt(inp["q"], inp["k"], inp["v"], inp["decay"], [0, n], 0.5,
                               inp["state"], [1])
    assert float((state[2].double() - S[0]).norm() / S[0].norm()) < 2e-6


def test_prompt_recurrent_form_equals_steps_bitwise():
    """The recurrent prompt form is the step token by token: the same bits."""
    inp = make([11], 3, 3, slots=3, seed=13)
    out, state = launch(inp, src=[1], dst=[2], path=1)
    st = inp["state"].cuda()
    kw = {n: inp[n].cuda() for n in ("q", "k", "v", "decay")}
    for t in range(11):
        o = torch.zeros(1, 384, dtype=bf16, device="cuda")
        kda_lin_step(**{n: x[t:t + 1].contiguous() for n, x in kw.items()},
                     slots=torch.tensor([1], dtype=torch.int32, device="cuda"), state=st,
                     output=o, scale=0.5)
        assert torch.equal(o[0].cpu(), out[t])
    assert torch.equal(st[1].cpu(), state[2])


# --------------------------------------------------------------------- refusals

def test_refusals_of_the_binding():
    inp = make([40, 8], 4, 2, slots=3, seed=14)
    dev = {n: inp[n].cuda() for n in ("q", "k", "v", "decay", "state")}
    i32 = dict(dtype=torch.int32, device="cuda")
    base = dict(dev, seq_starts=torch.tensor(inp["starts"], **i32), scale=1.0,
                output=torch.full((48, 512), 7.0, dtype=bf16, device="cuda"),
                dst_slots=torch.tensor([1, 2], **i32))
    wide = torch.zeros(48, 600, dtype=bf16, device="cuda")
    for kw, error in [
            (dict(q=dev["q"].float()), TypeError),
            (dict(q=dev["q"][:, :128 + 64]), ValueError),
            (dict(k=dev["k"][:47]), ValueError),
            (dict(k=dev["k"][:, :128]), ValueError),
            (dict(v=torch.zeros(48, 3 * 128, dtype=bf16, device="cuda")), ValueError),
            (dict(v=wide.t()[:512].t()), None),                  # a slice of wider rows
            (dict(v=torch.zeros(48, 516, dtype=bf16, device="cuda")[:, :512]), ValueError),
            (dict(v=torch.zeros(512, 48, dtype=bf16, device="cuda").t()), ValueError),
            (dict(v=wide[:, 4:516]), kl.KDA_ERR_ALIGNMENT),
            (dict(output=dev["v"].cpu()), ValueError),
            (dict(decay=dev["decay"].double()), TypeError),
            (dict(decay=dev["decay"][:, :3].contiguous()), ValueError),
            (dict(decay=dev["decay"].t()), ValueError),
            (dict(seq_starts=base["seq_starts"].long()), TypeError),
            (dict(seq_starts=torch.zeros(2, 2, **i32)), ValueError),
            (dict(dst_slots=torch.tensor([1], **i32)), ValueError),
            (dict(state=None), ValueError),
            (dict(state=dev["state"][:, :2].contiguous()), ValueError),
            (dict(state=dev["state"].half()), TypeError),
            (dict(path=3), kl.KDA_ERR_PATH),
            (dict(err=torch.zeros(1, device="cuda")), TypeError)]:
        if error is None:
            kda_lin_prompt(**dict(base, **kw))
            base["output"].fill_(7.0)
        elif isinstance(error, int):
            with pytest.raises(kl.KdaError) as e:
                kda_lin_prompt(**dict(base, **kw))
            assert e.value.code == error
        else:
            with pytest.raises(error):
                kda_lin_prompt(**dict(base, **kw))
    torch.cuda.synchronize()
    assert torch.all(base["output"] == 7.0)


def test_workspace_of_the_caller():
    """The caller's workspace gives the same bits; one too small is refused."""
    inp = make([1400], 2, 2, slots=3, seed=15)
    want = launch(inp, dst=[2], max_seq=1400)
    need = kl.prompt_workspace(kl.KdaLinPromptArgs(
        seqs=1, heads=2, qk_heads=2, tokens=1400, max_seq=1400, q_stride=256, k_stride=256,
        v_stride=256, o_stride=256))
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")      # (NaN bits)
    got = launch(inp, dst=[2], max_seq=1400, workspace=ws)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1][2], got[1][2])
    with pytest.raises(kl.KdaError) as e:
        launch(inp, dst=[2], max_seq=1400, workspace=ws[:-1].clone())
    assert e.value.code == kl.KDA_ERR_WORKSPACE

"""How exact the chunked form's pages stay (kda_lin_prompt): relative errors in the
2-norm against the recurrence in 64 bits, chunk by chunk, with limits that come
from FP32's own rounding."""
from __future__ import annotations

import pytest
import torch

from linear_attention_recurrent_kda_gb300 import lib as kl
from linear_attention_recurrent_kda_gb300.api import kda_lin_prompt
from tests import linref

D = 128
U32 = linref.U32


def last_pages(k, v, decay, first):
    """Pages [H, 128, 128] after k [n, Hk * 128], v [n, H * 128] and decay [n, H] or
    [H] from `first`, in 64 bits: S' = e^b_C S + sum_j e^(b_C - b_j) v_j k_j^T."""
    n, H = v.shape[0], v.shape[1] // D
    S = first.double()
    for a in range(0, n, 128):
        b = min(a + 128, n)
        g = (decay[a:b] if decay.dim() == 2 else decay.expand(b - a, H)).double().T   # [H, C]
        behind = g.flip(1).cumsum(1).flip(1) - g
        kk = k[a:b].double().view(b - a, -1, D).transpose(0, 1)
        kk = kk.repeat_interleave(H // kk.shape[0], 0) * behind.exp()[..., None]
        vv = v[a:b].double().view(b - a, H, D).permute(1, 2, 0)
        S = g.sum(1).exp()[:, None, None] * S + vv @ kk
    return S


def test_the_reference_is_the_recurrence():
    g = torch.Generator().manual_seed(3)
    n, H = 300, 2
    k, v = torch.randn(n, D, generator=g), torch.randn(n, H * D, generator=g)
    S0 = torch.randn(2, H, D, D, generator=g)
    for decay in (-torch.rand(n, H, generator=g), -torch.rand(H, generator=g)):
        S = linref.prompt(k, k, v, decay, [0, n], 1.0, S0, [1])[2][0]
        assert torch.allclose(last_pages(k, v, decay, S0[1]), S, rtol=1e-12, atol=1e-12)


def prompt(n, H, Hk, decay, *, seed, first=0.0, split):
    """One sequence of n tokens through the chunked form; (got, inputs)."""
    g = torch.Generator("cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    k = randn(n, Hk, D)
    k = (k / k.norm(dim=-1, keepdim=True)).view(n, Hk * D).to(torch.bfloat16)
    v = randn(n, H * D).to(torch.bfloat16)
    state = randn(2, H, D, D) * first
    i32 = dict(dtype=torch.int32, device="cuda")
    need = kl.prompt_workspace(kl.KdaLinPromptArgs(
        seqs=1, heads=H, qk_heads=Hk, tokens=n, max_seq=n, q_stride=Hk * D, k_stride=Hk * D,
        v_stride=H * D, o_stride=H * D))
    assert (need > 0) == split
    S0 = state[1].clone()
    kda_lin_prompt(q=k, k=k, v=v, decay=decay.cuda(), seq_starts=torch.tensor([0, n], **i32),
                   output=torch.empty_like(v), scale=1.0, state=state,
                   src_slots=torch.tensor([1], **i32), dst_slots=torch.tensor([1], **i32), path=2)
    return state[1], (k, v, decay.cuda(), S0)


def errors(got, want):
    """Relative error of each head's page."""
    return (got.double() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)


@pytest.mark.gpu
@pytest.mark.parametrize("H,split", [(80, False), (8, True)])
def test_pages_of_very_slow_heads_do_not_drift(H, split):
    """256 chunks at decays of exp(-1e-6) to exp(-1e-5) a token, from a page that
    outweighs what is added.  A chunk's factor rounded to FP32 would be off by up to
    U32 / 2 the same way at every chunk, 256 of them 7.6e-6 (split: 64 segments,
    1.9e-6), and no two heads' factors round alike.  Without that the page rounds
    once a chunk (split: 4 chunks and 64 segments), at random, an rms of at most
    U32 / 3^0.5: twice the square root of their number of these, and the exponent's
    own error, 8 U32 of at most 0.33."""
    n = 256 * 128
    decay = -torch.logspace(-6, -5, H)
    got, inp = prompt(n, H, 8, decay, seed=50, first=64.0, split=split)
    roundings = 256 if not split else 4 + 64
    limit = (2 * (roundings / 3) ** 0.5 + 8 * 0.33) * U32
    off = errors(got, last_pages(*inp))
    assert float(off.max()) < limit, (float(off.max()), limit)


@pytest.mark.gpu
@pytest.mark.parametrize("low", [-float("inf"), -70.0])
def test_decays_behind_many_strong_ones_keep_their_digits(low):
    """One chunk whose 32-token blocks start with up to 28 resets (or decays of
    2^-100) and go on mildly.  v is the identity, q k of one sign and the first page
    zero: output (i, j) is the masked product P_ij alone, rounded to BF16 once, so it
    is within half a last place of the exact one.  The factor's own error is allowed
    8.5e-5 (a difference of sums within +-2048 in FP32, 2^-13, times ln 2) and 1e-5
    for the sums' terms and exp2, in half last places (2^-8 to 2^-9 of the value) at
    most 0.05; sums of up to 28 * 160 from one end would leave 7e-4."""
    n, H = 128, 12
    g = torch.Generator().manual_seed(51)
    q, k = (torch.rand(n, H * D, generator=g).add(0.1).to(torch.bfloat16) for _ in "qk")
    decay = -0.05 * torch.rand(n, H, generator=g)
    for h in range(H):
        for block in range(4):
            strong = int(torch.randint(8, 29, (1,), generator=g))
            decay[32 * block:32 * block + strong, h] = low
    v = torch.eye(n).repeat(1, H).to(torch.bfloat16)
    out = torch.empty(n, H * D, dtype=torch.bfloat16, device="cuda")
    kda_lin_prompt(q=q.cuda(), k=k.cuda(), v=v.cuda(), decay=decay.cuda(), output=out, scale=1.0,
                   seq_starts=torch.tensor([0, n], dtype=torch.int32, device="cuda"), path=2)
    got = out.cpu().double().view(n, H, D)
    worst = 0.0
    for h in range(H):
        sl = slice(h * D, h * D + D)
        w = torch.zeros(n, n, dtype=torch.float64)
        for i in range(n):
            for j in range(i + 1):
                w[i, j] = decay[j + 1:i + 1, h].double().sum().exp()
        want = (q[:, sl].double() @ k[:, sl].double().T) * w
        near = want >= 2.0 ** -90
        half = torch.exp2(torch.floor(torch.log2(want[near]))) * linref.U16
        worst = max(worst, float(((got[:, h] - want)[near].abs() / half).max()))
        assert torch.all(got[:, h][~near].abs() < 2.0 ** -89)
    assert worst < 1.05, worst


@pytest.mark.gpu
@pytest.mark.parametrize("path", [1, 2])
def test_one_reset_among_no_decays_leaves_nothing(path):
    """A single reset in a chunk without other decays, from a page of 2^100: the
    tokens from it on have the bits that they have from an empty page."""
    n, at = 200, 70
    g = torch.Generator().manual_seed(52)
    q, k, v = (torch.randn(n, D, generator=g).to(torch.bfloat16).cuda() for _ in "qkv")
    decay = torch.zeros(n, 1)
    decay[at] = -float("inf")
    i32 = dict(dtype=torch.int32, device="cuda")
    outs = []
    for first in (2.0 ** 100, 0.0):
        state = torch.full((2, 1, D, D), first, device="cuda")
        vv = v.clone()
        if first == 0.0:
            vv[:at] = 0
        out = torch.empty_like(v)
        kda_lin_prompt(q=q, k=k, v=vv, decay=decay.cuda(), output=out, scale=1.0, state=state,
                       seq_starts=torch.tensor([0, n], **i32), path=path,
                       src_slots=torch.tensor([1], **i32), dst_slots=torch.tensor([1], **i32))
        outs.append((out[at:], state[1]))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


PARTS_LIMIT = 6e-7


def test_two_parts_of_a_key_would_break_the_limit():
    """The limit of the next test lies between what a factor times a key leaves in two
    BF16 parts (each element off by up to 2^-18, evenly: an rms of about 2^-18 /
    3^0.5 * 0.75) and in three."""
    g = torch.Generator().manual_seed(53)
    k = torch.randn(128, D, generator=g).to(torch.bfloat16).float()
    v = torch.randn(128, D, generator=g).to(torch.bfloat16).double()
    w = torch.exp(-0.15 * torch.arange(127, -1, -1.0))
    full = w[:, None] * k
    for parts, fails in ((2, True), (3, False)):
        left, held = full.clone(), torch.zeros_like(full, dtype=torch.float64)
        for _ in range(parts):
            part = left.to(torch.bfloat16).float()
            held, left = held + part.double(), left - part
        want = v.T @ full.double()
        off = float((v.T @ held - want).norm() / want.norm())
        assert (off > 2 * PARTS_LIMIT) if fails else (off < PARTS_LIMIT / 8), (parts, off)


@pytest.mark.gpu
@pytest.mark.parametrize("first", [0.0, 1.0], ids=["empty", "carried"])
@pytest.mark.parametrize("rate", [0.01, 0.3, 3.0], ids=["slow", "mild", "strong"])
@pytest.mark.parametrize("n,H", [(128, 4), (77, 4), (40 * 128 - 5, 80)])
def test_pages_keep_the_digits_of_fp32(n, H, rate, first):
    """Whole sequences of one chunk and of 40.  Expected of a page, in the 2-norm:
    sums of 128 tokens in three parts on the tensor cores, 24 steps off by up to a
    last place each, 24^0.5 * 2 U32 / 3^0.5 = 3.4e-7; factors and exponents 1.3e-7; the
    page's own update in the 10 chunks that a slow page remembers 1.1e-7: 4e-7
    together.  Two parts of a factor times a key would leave 1.6e-6."""
    g = torch.Generator().manual_seed(n + H)
    decay = -rate * torch.rand(n, H, generator=g)
    got, inp = prompt(n, H, 4, decay, seed=54, first=first, split=False)
    off = errors(got, last_pages(*inp))
    assert float(off.max()) < PARTS_LIMIT, (float(off.max()), off)


@pytest.mark.gpu
@pytest.mark.parametrize("power", [-54, 50])
def test_magnitudes_that_the_one_factor_form_holds(power):
    """Keys and pages of 2^-54 and 2^50 in chunks whose decay, 2^-120, is near the limit of
    the form that takes factors of up to 2^60 both ways: products q k stay above the
    normal range's end (2^-54 / 16 * 2^-60 > 2^-126), sums below the largest number."""
    from tests.test_lin_gpu import launch, make, verify
    inp = make([300, 128], 2, 2, slots=4, seed=55)
    inp["k"] = (inp["k"].float() * 2.0 ** power).to(torch.bfloat16)
    inp["state"] = inp["state"] * 2.0 ** power
    inp["decay"] = -0.65 + 0.0 * inp["decay"]
    src, dst = [1, 0], [2, 3]
    verify(inp, launch(inp, src=src, dst=dst, path=2), 2, src, dst)

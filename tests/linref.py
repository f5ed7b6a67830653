"""Plain implementations in 64 bits of the linear attention with one decay per
head and of the snapshots, and the error bounds the GPU tests use.

``prompt`` runs the recurrence token by token.  Beside the values it carries
the same recurrence on magnitudes (|S0|, |v| |k|^T, |q|): the sums of the
magnitudes of all terms, against which rounding errors are measured."""
from __future__ import annotations

import numpy as np
import torch

D = 128
U32 = 2.0 ** -24        # half a last place, FP32
U16 = 2.0 ** -8         # half a last place, BF16


def prompt(q, k, v, decay, starts, scale, state=None, src=None):
    """q, k [tokens, Hk * 128], v [tokens, H * 128], decay [H] or [tokens, H];
    returns (out, out_mag) [tokens, H * 128] and (S, S_mag) [seqs, H, 128, 128],
    float64.  Rows of no sequence stay NaN."""
    q, k, v, g = (t.detach().cpu().double() for t in (q, k, v, decay))
    n, H = v.shape[0], v.shape[1] // D
    per = H // (q.shape[1] // D)
    out = torch.full((n, H * D), float("nan"), dtype=torch.float64)
    mag = out.clone()
    B = len(starts) - 1
    S = torch.zeros(B, H, D, D, dtype=torch.float64)
    if src is not None:
        for r, s in enumerate(src):
            if s > 0:
                S[r] = state[s].cpu().double()
    M = S.abs()
    for r in range(B):
        for t in range(starts[r], starts[r + 1]):
            d = torch.exp(g if g.dim() == 1 else g[t]).view(H, 1, 1)
            qt = q[t].view(-1, 1, D).repeat_interleave(per, 0)
            kt = k[t].view(-1, 1, D).repeat_interleave(per, 0)
            vt = v[t].view(H, D, 1)
            S[r] = d * S[r] + vt * kt
            M[r] = d * M[r] + vt.abs() * kt.abs()
            out[t] = (scale * (S[r] * qt).sum(-1)).view(-1)
            mag[t] = abs(scale) * (M[r] * qt.abs()).sum(-1).view(-1)
    return out, mag, S, M


def state_bound(M, tokens):
    """Bound on a page's error, per element, from the magnitudes M.

    Recurrent form: a token multiplies by a factor that is off by at most 2
    last places and rounds once: 5 U32 of the magnitudes a token.  Chunked
    form: a chunk's factors are powers of two of FP32 sums; an exponent of
    magnitude x carries at most 8 roundings of size x U32 and scales its term by
    2^-x, x 2^-x <= 0.54, so 8 U32, plus 4 U32 for exp2 and two products; the
    BF16 parts of a factor times a key leave 2^-24; a chunk's sum has at most
    3 * 128 terms, each addition off by at most a whole last place (2 U32);
    the page's own update rounds twice.  Per chunk: 800 U32, and a chunk's
    errors decay with it, so they add up over at most all chunks."""
    chunks = -(-max(tokens, 1) // 128)
    return max(5 * tokens, 800 * chunks) * U32 * M


def out_bound(ref, mag, tokens, chunked):
    """Bound on an output's error: half a BF16 last place of the result, the
    errors of the state (as above) and of a sum of 2 * 128 terms, and in the
    chunked form the rounding of the masked products q k and of the state to
    BF16, half a last place of every term each."""
    chunks = -(-max(tokens, 1) // 128)
    rel = (max(5 * tokens, 800 * chunks) + 600) * U32 + (U16 * (1 + U16) if chunked else 0.0)
    return U16 * ref.abs() + rel * (1 + U16) * mag


def quantise(x, bits):
    """Pages [..., 128, 128] FP32 -> (codes int8 [..., 128, 128], scales FP32
    [..., 128, groups]) by the definition, in 64 bits."""
    x = np.asarray(x, np.float32)
    top = 127 if bits == 8 else 7
    g = x.reshape(*x.shape[:-1], 1 if bits == 8 else 4, -1)
    with np.errstate(all="ignore"):
        m = np.abs(g).max(-1).astype(np.float64)
        scale = (m / top).astype(np.float32)
        scale[m < 2.0 ** -118] = 0.0
        bad = ~np.isfinite(g).all(-1)
        scale[bad] = np.nan
        ok = (scale > 0)[..., None]
        code = np.where(ok, np.rint(g.astype(np.float64) / np.where(ok, scale[..., None], 1)), 0)
    return code.astype(np.int8).reshape(x.shape), scale


def dequantise(codes, scale):
    g = codes.reshape(*codes.shape[:-1], scale.shape[-1], -1).astype(np.float32)
    return (g * scale[..., None]).reshape(codes.shape)


def pack(codes, bits):
    """Codes as they are stored."""
    if bits == 8:
        return codes
    c = codes.astype(np.int16)
    return ((c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4)).astype(np.uint8)

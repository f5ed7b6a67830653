"""Plain implementations in 64 bits of the short convolution, the selective scan and
the product with its epilogue, each with a bound of what FP32 arithmetic and the one
BF16 rounding may leave, derived here from the operations (a rounding to nearest is
off by half a last place; the approximate exp2, reciprocal and divide by 2^-22)."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24        # half a last place, FP32
U16 = 2.0 ** -8         # half a last place, BF16
APPROX = 2.0 ** -22     # approximate exp2, divide
TINY = 2.0 ** -130      # BF16's and FP32's smallest steps


def f64(t):
    return t.detach().cpu().double()


def _silu(y, err):
    """silu(y) and the bound of a value whose argument is off by `err`: the slope is
    below 1.1; exp2's argument y log2 e is rounded (|y| 2^-23 of the factor), exp2, the
    sum 1 + e and the divide follow."""
    out = y * torch.sigmoid(y)
    return out, 1.1 * err + out.abs() * (2 * APPROX + 2 * U32 + y.abs() * 2.0 ** -23)


def rounded(out, err):
    """The bound after the rounding to BF16."""
    return err * (1 + U16) + out.abs() * U16 + TINY


def conv(x, weight, starts, bias=None, window=None, src=None, silu=True):
    """x [rows, C]; weight [taps, C] or [parts, taps, C / parts].  Returns (out, bound) with
    NaN in rows of no sequence, and the last inputs [seqs, C, taps - 1]."""
    x, w = f64(x), f64(weight)
    if w.dim() == 3:
        w = torch.cat(list(w), 1)
    n, C = w.shape[0] - 1, x.shape[1]
    out = torch.full(x.shape, float("nan"), dtype=torch.float64)
    bound, last = out.clone(), torch.zeros(len(starts) - 1, C, n, dtype=torch.float64)
    b = torch.zeros(C, dtype=torch.float64) if bias is None else f64(bias)
    for r, (lo, hi) in enumerate(zip(starts[:-1], starts[1:])):
        first = torch.zeros(n, C, dtype=torch.float64)
        if src is not None and src[r] > 0:
            first = f64(window[src[r]])[:, :n].T
        full = torch.cat([first, x[lo:hi]])
        for t in range(hi - lo):
            terms = full[t:t + n + 1] * w
            y = b + terms.sum(0)
            # n + 1 fused steps, each rounds a partial sum
            err = (n + 1) * U32 * (b.abs() + terms.abs().sum(0))
            if silu:
                y, err = _silu(y, err)
            out[lo + t], bound[lo + t] = y, rounded(y, err)
        last[r] = full[full.shape[0] - n:].T
    return out, bound, last


def softplus(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def ssm(x, dt, a, b, c, starts, d=None, z=None, dt_bias=None, soft=True, state=None, src=None):
    """The recurrence token by token.  Returns (out, bound) [rows, C] with NaN in rows of no
    sequence, and (h, bound) [seqs, C, N].

    Bounds, beside the values: the step s is off by `ds` of itself (the sum raw + bias
    by half a place; softplus by exp2, its argument, a reciprocal refined once, a
    polynomial and their products: below 2^-20 with the slope s' <= s); the exponent
    s a log2 e by ds and three roundings; the decay f by that times its exponent, and
    by its own evaluation, 2^-22 of f (the approximate exp2; forms of f - 1 are nearer, and
    tests of slow states hold the drift to less); the addition s x b by ds and two
    roundings; three roundings of the sum itself."""
    x, dt, a, b, c = (f64(t) for t in (x, dt, a, b, c))
    rows, C = x.shape
    N = a.shape[1]
    G = b.shape[1] // N
    b, c = (t.view(rows, G, 1, N).expand(-1, -1, C // G, -1).reshape(rows, C, N) for t in (b, c))
    raw = dt if dt_bias is None else dt + f64(dt_bias)
    s = softplus(raw) if soft else raw
    ds = 2.0 ** -20 + raw.abs() * U32 if soft else U32 * torch.ones_like(raw)
    skip = None if d is None else f64(d)
    out = torch.full((rows, C), float("nan"), dtype=torch.float64)
    bound = out.clone()
    B = len(starts) - 1
    h = torch.zeros(B, C, N, dtype=torch.float64)
    if src is not None:
        for r, slot in enumerate(src):
            if slot > 0:
                h[r] = f64(state[slot])
    e = torch.zeros_like(h)
    for r in range(B):
        for t in range(starts[r], starts[r + 1]):
            g = s[t][:, None] * a
            f = torch.exp(g)
            df = f * g.abs() * (ds[t][:, None] + 3 * U32) + f * APPROX + TINY
            add = (s[t] * x[t])[:, None] * b[t]
            e[r] = f * e[r] + df * (h[r].abs() + e[r]) + add.abs() * (ds[t][:, None] + 2 * U32)
            h[r] = f * h[r] + add
            e[r] += 3 * U32 * (h[r].abs() + add.abs()) + TINY
            y = (c[t] * h[r]).sum(-1)
            err = (c[t].abs() * (e[r] + (N + 1) * U32 * (h[r].abs() + e[r]))).sum(-1)
            if skip is not None:
                y = y + skip * x[t]
                err = err + U32 * (y.abs() + (skip * x[t]).abs())
            if z is not None:
                g8 = f64(z[t])
                gate, dgate = _silu(g8, torch.zeros_like(g8))
                err = err * gate.abs() + (y.abs() + err) * (dgate + U32 * gate.abs())
                y = y * gate
            out[t], bound[t] = y, rounded(y, err)
    return out, bound, h, e


def linear(x, weight, bias=None, residual=None, act=None):
    """(out, bound): products of BF16 values are exact in FP32; each of the `inner`
    additions may drop a last place (2^-23) of the magnitudes summed."""
    x, w = f64(x), f64(weight)
    y = x @ w.T
    err = (x.shape[1] + 1) * 2.0 ** -23 * (x.abs() @ w.abs().T)
    if bias is not None:
        y = y + f64(bias)
        err = err + U32 * y.abs()
    if act == "silu":
        y, err = _silu(y, err)
    elif act == "gelu":
        # erfc's argument y / sqrt(2) is off by 2^-23 of itself: erfc, whose slope there
        # is below (1 + y^2) erfc / |y|, by (1 + y^2) 2^-23 of itself, itself by 2^-21
        out = y * 0.5 * torch.erfc(-y * 0.5 ** 0.5)
        err = 1.2 * err + out.abs() * ((1 + y * y) * 2.0 ** -23 + 2.0 ** -21 + 2 * U32)
        y = out
    elif act == "softplus":
        y, err = softplus(y), err + softplus(y) * (2.0 ** -20 + y.abs() * U32)
    if residual is not None:
        y = y + f64(residual)
        err = err + U32 * y.abs()
    return y, rounded(y, err)


def inside(got, want, bound, what=""):
    """Every value within its bound (NaN where the reference has none: not looked at)."""
    got, live = f64(got), ~torch.isnan(want)
    off = (got - want).abs()
    bad = live & ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((off / bound)[live].max()),
                           bad.nonzero()[:4].tolist())

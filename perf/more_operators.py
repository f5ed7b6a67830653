"""The operators of a selective-state-space layer as they are measured.

* ``conv``: the short causal depthwise convolution over ragged prompts, with SiLU;
  windows (the last inputs of a sequence) in and out; also what a KDA layer's
  prompt runs on its q, k and v;
* ``conv_step``: the same for one token per request, the window shifted in place;
* ``ssm``: the selective scan over ragged prompts.  Per channel, with N states,
  dt = softplus(raw + bias), h_n <- exp(dt A_n) h_n + dt x B_n,
  out = (sum_n C_n h_n + D x) silu(z); states in and out;
* ``ssm_step``: the same for one token per request, the state in place;
* ``linear``: act(x W^T + bias) + residual in one call, the layer's projections.

State is FP32 [slot, channel, N], windows BF16 or FP32 [slot, channel, width];
slot 0 is the null slot.
"""
import math
import random

import torch

own = False


def listed():
    return [
        # drafts of a few requests: latency
        dict(name="conv_drafts_b4_c2048", op="conv", seqs=4, channels=2048, parts=1, taps=4, width=3,
             shortest=1, longest=9, lengths=21, bias=True, silu=True, carried=True, wide=False),
        # q, k and v of a KDA layer of 32 heads, an ordinary prefill batch
        dict(name="conv_kda_b8_h32", op="conv", seqs=8, channels=12288, parts=3, taps=4, width=3,
             shortest=257, longest=2047, lengths=12, bias=False, silu=True, carried=False,
             wide=False),
        # a decode batch, an eighth of it padding, windows in 32 bits
        dict(name="conv_step_b256_c8192", op="conv_step", seqs=256, channels=8192, parts=1, taps=4,
             width=3, pad=32, bias=True, silu=True, wide=True),
        # drafts of a few requests: latency
        dict(name="ssm_drafts_b4_c1024", op="ssm", seqs=4, channels=1024, states=16, groups=1,
             shortest=1, longest=9, lengths=22, carried=True, gated=True, skip=True, softplus=True),
        # an ordinary prefill batch of ragged prompts
        dict(name="ssm_ragged_b8_c4096", op="ssm", seqs=8, channels=4096, states=16, groups=1,
             shortest=257, longest=2047, lengths=12, carried=True, gated=True, skip=True,
             softplus=True),
        # one long document
        dict(name="ssm_long_c4096", op="ssm", seqs=1, channels=4096, states=16, groups=1,
             shortest=32749, longest=32749, lengths=13, carried=False, gated=True, skip=True,
             softplus=True),
        # decode of a few requests: latency
        dict(name="ssm_step_b4_c1024", op="ssm_step", seqs=4, channels=1024, states=16, groups=1,
             pad=0, gated=True, skip=True, softplus=True),
        # the largest decode batch, an eighth of it padding
        dict(name="ssm_step_b256_c8192", op="ssm_step", seqs=256, channels=8192, states=16, groups=1,
             pad=32, gated=True, skip=True, softplus=True),
        # decode of a few requests: latency
        dict(name="linear_m4_k4096_n1024", op="linear", rows=4, inner=4096, outer=1024,
             act="silu", bias=True, residual=False),
        # a decode batch into a layer: the weights' bytes
        dict(name="linear_m61_k4096_n16384", op="linear", rows=61, inner=4096, outer=16384,
             act="none", bias=False, residual=False),
        # the low-rank step projection of a prefill batch: thin
        dict(name="linear_m9159_k256_n4096", op="linear", rows=9159, inner=256, outer=4096,
             act="none", bias=True, residual=False),
        # out of the layer into the residual stream, a prefill batch
        dict(name="linear_m9159_k4096_n7168", op="linear", rows=9159, inner=4096, outer=7168,
             act="gelu", bias=True, residual=True),
    ]


MOST_STATES = 32749 * 4096 * 16          # tokens x channels x states of the largest scan
MOST_ROWS = 9159 * 12288                 # tokens x channels of the largest convolution
MOST_PRODUCTS = 9159 * 4096 * 7168       # of the largest product


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "ssm", "ssm", "ssm_step", "linear", "linear"])

    def flag():
        return rng.random() < 0.5

    if op == "linear":
        inner, outer = 8 * _spread(rng, 1, 1024), _spread(rng, 1, 16384)
        return dict(op=op, rows=_spread(rng, 1, max(1, min(16384, MOST_PRODUCTS // (inner * outer)))),
                    inner=inner, outer=outer, act=rng.choice(["none", "silu", "gelu", "softplus"]),
                    bias=flag(), residual=flag())
    if op.startswith("conv"):
        parts, taps = rng.choice([1, 3]), rng.choice([2, 3, 4])
        case = dict(op=op, channels=8 * parts * _spread(rng, 8, 512), parts=parts, taps=taps,
                    width=taps - 1 + rng.choice([0, 0, 3]), bias=flag(), silu=rng.random() < 0.8,
                    wide=flag())
        most = MOST_ROWS // case["channels"]
    else:
        groups = rng.choice([1, 1, 2, 8])
        case = dict(op=op, channels=8 * groups * _spread(rng, 1 if groups > 1 else 8, 1024 // groups),
                    states=rng.choice([16, 16, 32, 64]), groups=groups, gated=rng.random() < 0.8,
                    skip=flag(), softplus=rng.random() < 0.8)
        most = MOST_STATES // (case["channels"] * case["states"])
    seqs = _spread(rng, 1, 256)
    if op.endswith("step"):
        return dict(case, seqs=seqs, pad=rng.choice([0, 0, seqs // 8]))
    longest = _spread(rng, 1, max(1, min(32749, most // seqs)))
    return dict(case, seqs=seqs, shortest=_spread(rng, 1, longest), longest=longest,
                lengths=rng.randrange(1 << 30), carried=flag())


def _lens(case):
    r = random.Random(case["lengths"])
    return [r.randint(case["shortest"], case["longest"]) for _ in range(case["seqs"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, bf = case["op"], torch.bfloat16

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def rows_of(rows, width):
        """BF16 rows, 16 bytes at least apart, of a width that need not be a multiple of 8."""
        return randn(rows, -(-width // 8) * 8).to(bf)[:, :width]

    s = dict(case)
    if op == "linear":
        M, K, N = case["rows"], case["inner"], case["outer"]
        s.update(x=randn(M, K).to(bf), weight=(randn(N, K) * K ** -0.5).to(bf),
                 bias_row=(randn(N) * 0.5).to(bf) if case["bias"] else None,
                 residual_rows=rows_of(M, N) if case["residual"] else None,
                 output=torch.zeros(M, -(-N // 8) * 8, dtype=bf, device="cuda")[:, :N])
        return s
    B, C = case["seqs"], case["channels"]
    step = op.endswith("step")
    lens = [1] * B if step else _lens(case)
    rows = sum(lens)
    s.update(lens=lens, output=torch.zeros(rows, C, dtype=bf, device="cuda"))
    slots = B if step else 2 * B
    at = torch.randperm(slots, generator=g, device="cuda").to(torch.int32) + 1
    if step:
        s["slots"] = at
        s["slots"][torch.randperm(B, generator=g, device="cuda")[:case["pad"]]] = 0
    else:
        s["seq_starts"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        s["src_slots"] = at[:B].contiguous() if case["carried"] else None
        s["dst_slots"] = at[B:].contiguous()
    if op.startswith("conv"):
        P, W = case["parts"], case["taps"]
        s["x"] = randn(rows, 2 * C).to(bf)[:, :C]        # beside the gate in one projection
        shape = (W, C) if P == 1 else (P, W, C // P)
        s["weight"] = (randn(*shape) * 0.5).to(bf)
        s["bias_row"] = (randn(C) * 0.5).to(bf) if case["bias"] else None
        s["window"] = randn(slots + 1, C, case["width"]).to(torch.float32 if case["wide"] else bf)
    else:
        N, G = case["states"], case["groups"]
        s["x"] = randn(rows, C).to(bf)
        z = randn(rows, 2 * C).to(bf)[:, C:]             # the other half of the projection
        s["z"] = z if case["gated"] else None
        bc = randn(rows, 2 * G * N).to(bf)               # side by side, as projected
        s["b"], s["c"] = bc[:, :G * N], bc[:, G * N:]
        s["a"] = -(torch.arange(N, device="cuda") + 1.0) * torch.exp(0.3 * randn(C, N))
        s["d"] = 1.0 + 0.1 * randn(C) if case["skip"] else None
        rate = torch.exp(rand(C) * math.log(100.0)) * 1e-3           # steps of 1e-3 to 1e-1
        if case["softplus"]:
            s["dt_bias"], s["dt"] = rate + torch.log(-torch.expm1(-rate)), randn(rows, C).to(bf)
        else:
            s["dt_bias"], s["dt"] = None, (rate * torch.exp(0.5 * randn(rows, C))).to(bf)
        s["state"] = randn(slots + 1, C, N) * 0.1
    if step and own:   # a decoding program prepares its step once, over its own buffers
        from linear_attention_recurrent_kda_gb300.api import KdaConvStep, KdaSsmStep
        if op == "conv_step":
            s["step"] = KdaConvStep(x=s["x"], weight=s["weight"], bias=s["bias_row"],
                                    slots=s["slots"], window=s["window"], output=s["output"],
                                    silu=s["silu"])
        else:
            s["step"] = KdaSsmStep(x=s["x"], dt=s["dt"], a=s["a"], b=s["b"], c=s["c"], d=s["d"],
                                   z=s["z"], dt_bias=s["dt_bias"], softplus=s["softplus"],
                                   slots=s["slots"], state=s["state"], output=s["output"])
    return s


def run(s):
    op = s["op"]
    if op == "linear":
        if own:
            from linear_attention_recurrent_kda_gb300.api import kda_linear
            kda_linear(x=s["x"], weight=s["weight"], output=s["output"], bias=s["bias_row"],
                       residual=s["residual_rows"], activation=s["act"])
        else:
            _plain_linear(s)
        return [s["output"]]
    if op == "conv":
        if own:
            from linear_attention_recurrent_kda_gb300.api import kda_conv_prompt
            kda_conv_prompt(x=s["x"], weight=s["weight"], bias=s["bias_row"],
                            seq_starts=s["seq_starts"], output=s["output"], silu=s["silu"],
                            window=s["window"], src_slots=s["src_slots"], dst_slots=s["dst_slots"])
        else:
            _plain_conv(s)
        return [s["output"], s["window"]]
    if op == "ssm":
        if own:
            from linear_attention_recurrent_kda_gb300.api import kda_ssm_prompt
            kda_ssm_prompt(x=s["x"], dt=s["dt"], a=s["a"], b=s["b"], c=s["c"], d=s["d"], z=s["z"],
                           dt_bias=s["dt_bias"], softplus=s["softplus"],
                           seq_starts=s["seq_starts"], output=s["output"], state=s["state"],
                           src_slots=s["src_slots"], dst_slots=s["dst_slots"],
                           max_seq=max(s["lens"]))
        else:
            _plain_ssm(s)
        return [s["output"], s["state"]]
    if own:
        s["step"]()
    elif op == "conv_step":
        _plain_conv_step(s)
    else:
        _plain_ssm_step(s)
    return [s["output"], s["window"] if op == "conv_step" else s["state"]]


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _softplus(x):
    return x.clamp_min(0.0) + torch.log1p(torch.exp(-x.abs()))


def _plain_linear(s):
    y = s["x"].float() @ s["weight"].float().T
    if s["bias_row"] is not None:
        y += s["bias_row"].float()
    if s["act"] == "silu":
        y = _silu(y)
    elif s["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * 0.5 ** 0.5))
    elif s["act"] == "softplus":
        y = _softplus(y)
    if s["residual_rows"] is not None:
        y += s["residual_rows"].float()
    s["output"].copy_(y)


def _taps(s):
    """FP32 [taps, channels]."""
    w = s["weight"].float()
    return w if w.dim() == 2 else w.transpose(0, 1).reshape(w.shape[1], -1)


def _plain_conv(s):
    dev, n = s["x"].device, s["taps"] - 1
    lens = torch.tensor(s["lens"], device=dev)
    rows, starts = s["x"].shape[0], s["seq_starts"].long()
    seq = torch.repeat_interleave(torch.arange(len(s["lens"]), device=dev), lens, output_size=rows)
    place = torch.arange(rows, device=dev) - starts[seq]
    x = s["x"].float()
    if s["src_slots"] is not None:
        before = s["window"][s["src_slots"].long()][..., :n].float()       # [seqs, channels, n]
    else:
        before = torch.zeros(len(s["lens"]), s["channels"], n, device=dev)

    def tap(back):     # the input `back` tokens before, of the sequence or its window
        inside = place >= back
        got = x[torch.where(inside, torch.arange(rows, device=dev) - back, 0)]
        early = before[seq, :, (n + place - back).clamp(0, n - 1)]
        return torch.where(inside[:, None], got, early)

    w = _taps(s)
    y = sum(w[j] * tap(n - j) for j in range(n + 1))
    if s["bias_row"] is not None:
        y = y + s["bias_row"].float()
    s["output"].copy_(_silu(y) if s["silu"] else y)
    both = torch.arange(n, device=dev) + lens[:, None]      # [seqs, n], into window + sequence
    late = x[(starts[:-1, None] + both - n).clamp(0, rows - 1)].transpose(1, 2)
    kept = before.gather(2, both.clamp_max(n - 1)[:, None, :].expand(-1, s["channels"], -1))
    s["window"][s["dst_slots"].long(), :, :n] = torch.where(
        (both >= n)[:, None, :], late, kept).to(s["window"].dtype)


def _plain_conv_step(s):
    n, at = s["taps"] - 1, s["slots"].long()
    live = s["slots"] > 0
    old = s["window"][at]
    full = torch.cat([old[..., :n].float(), s["x"].float()[..., None]], -1)
    y = (full * _taps(s).T).sum(-1)
    if s["bias_row"] is not None:
        y = y + s["bias_row"].float()
    y = _silu(y) if s["silu"] else y
    s["output"].copy_(torch.where(live[:, None], y, 0.0))
    new = torch.cat([full[..., 1:].to(old.dtype), old[..., n:]], -1)
    s["window"][at] = torch.where(live[:, None, None], new, s["window"][:1])


def _gates(s):
    """FP32 step sizes [rows, channels], decays and additions [rows, channels, states],
    and C spread over the channels."""
    C, N, G = s["channels"], s["states"], s["groups"]
    x, dt = s["x"].float(), s["dt"].float()
    if s["dt_bias"] is not None:
        dt = dt + s["dt_bias"]
    if s["softplus"]:
        dt = _softplus(dt)
    b, c = (s[k].float().view(-1, G, 1, N).expand(-1, G, C // G, N).reshape(-1, C, N) for k in "bc")
    return x, torch.exp(dt[..., None] * s["a"]), (dt * x)[..., None] * b, c


def _outputs(s, x, h, c):
    y = (h * c).sum(-1)
    if s["d"] is not None:
        y = y + s["d"] * x
    return y * _silu(s["z"].float()) if s["gated"] else y


def _plain_ssm(s):
    """Every token's state at once, by doubling: after the pass with a shift, `h` sums what
    the tokens up to twice that far back add, and `keep` is the decay over them."""
    dev = s["x"].device
    lens = torch.tensor(s["lens"], device=dev)
    starts = s["seq_starts"].long()[:-1]
    x, keep, h, c = _gates(s)
    if s["src_slots"] is not None:
        h[starts] += keep[starts] * s["state"][s["src_slots"].long()]
    keep[starts] = 0.0
    shift = 1
    while shift < max(s["lens"]):
        h[shift:] += keep[shift:] * h[:-shift]
        keep[shift:] *= keep[:-shift].clone()
        shift *= 2
    s["output"].copy_(_outputs(s, x, h, c))
    s["state"][s["dst_slots"].long()] = h[starts + lens - 1]


def _plain_ssm_step(s):
    at, live = s["slots"].long(), s["slots"] > 0
    x, keep, add, c = _gates(s)
    h = s["state"][at] * keep + add
    s["output"].copy_(torch.where(live[:, None], _outputs(s, x, h, c), 0.0))
    s["state"][at] = torch.where(live[:, None, None], h, s["state"][:1])


def exact(case, seed):
    s = prepare(case, seed)
    op, f8 = s["op"], torch.float64
    if op == "linear":
        y = torch.einsum("mk,nk->mn", s["x"].to(f8), s["weight"].to(f8))
        if s["bias"]:
            y = y + s["bias_row"].to(f8)
        if s["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif s["act"] == "gelu":
            y = y * 0.5 * torch.erfc(-y / math.sqrt(2.0))
        elif s["act"] == "softplus":
            y = torch.logaddexp(y, torch.zeros_like(y))
        return [y + s["residual_rows"].to(f8) if s["residual"] else y]
    step = op.endswith("step")
    slots = s["slots"].tolist() if step else None
    src = slots if step else (s["src_slots"].tolist() if s["carried"] else [0] * s["seqs"])
    dst = slots if step else s["dst_slots"].tolist()
    out = torch.zeros(s["output"].shape, dtype=f8, device="cuda")
    if op.startswith("conv"):
        n, pool = s["taps"] - 1, s["window"].to(f8)
        w = s["weight"].to(f8).view(s["parts"], n + 1, -1)
        row = 0
        for r, length in enumerate(s["lens"]):
            if not step or src[r] > 0:
                x = s["x"][row:row + length].to(f8).T
                first = pool[src[r], :, :n] if src[r] > 0 else torch.zeros_like(x[:, :1]).expand(-1, n)
                full = torch.cat([first, x], 1)                       # [channels, n + length]
                y = full.unfold(1, n + 1, 1).unflatten(0, (s["parts"], -1))
                y = torch.einsum("pclj,pjc->lpc", y, w).flatten(1)
                if s["bias"]:
                    y = y + s["bias_row"].to(f8)
                out[row:row + length] = y * torch.sigmoid(y) if s["silu"] else y
                pool[dst[r], :, :n] = full[:, -n:]
            row += length
        return [out, pool]
    # the recurrence, token by token, all live sequences at a time, longest first
    C, N, G = s["channels"], s["states"], s["groups"]
    dt = s["dt"].to(f8)
    if s["dt_bias"] is not None:
        dt = dt + s["dt_bias"].to(f8)
    if s["softplus"]:
        dt = torch.logaddexp(dt, torch.zeros_like(dt))
    pool = s["state"].to(f8)
    lens, A = s["lens"], s["a"].to(f8)
    order = sorted(range(len(lens)), key=lambda r: -lens[r])
    starts = [sum(lens[:r]) for r in range(len(lens))]
    first = torch.tensor([starts[r] for r in order], device="cuda")
    src, dst = (torch.tensor([v[r] for r in order], device="cuda") for v in (src, dst))
    h = pool[src] * (src > 0)[:, None, None]
    n = len(lens)
    for t in range(lens[order[0]]):
        while lens[order[n - 1]] <= t:
            n -= 1
        at = first[:n] + t
        d, x = dt[at], s["x"][at].to(f8)
        b, c = (s[k][at].to(f8).view(n, G, 1, N) for k in "bc")
        live = h[:n]
        live.mul_(torch.exp(d[..., None] * A))
        live.view(n, G, C // G, N).add_((d * x).view(n, G, -1, 1) * b)
        out[at] = (live.view(n, G, C // G, N) * c).sum(-1).view(n, C)
    if s["skip"]:
        out += s["d"].to(f8) * s["x"].to(f8)
    if s["gated"]:
        z = s["z"].to(f8)
        out *= z * torch.sigmoid(z)
    if step:
        out[first[src == 0]] = 0.0
        pool[dst[dst > 0]] = h[dst > 0]
    else:
        pool[dst] = h
    return [out, pool]


def work(case):
    if case["op"] == "linear":
        M, K, N = case["rows"], case["inner"], case["outer"]
        size = 2 * (M * K + N * K + M * N * (1 + case["residual"]) + N * case["bias"])
        return {"bytes": size, "flops": 2 * M * K * N}
    C, step = case["channels"], case["op"].endswith("step")
    live = case["seqs"] - case.get("pad", 0)
    rows = live if step else sum(_lens(case))
    moves = live * (1 + (step or case["carried"]))       # states or windows read and written
    if case["op"].startswith("conv"):
        size = 4 * rows * C + 2 * C * (case["taps"] + case["bias"])
        size += moves * C * (case["taps"] - 1) * (4 if case["wide"] else 2)
        return {"bytes": size, "flops": rows * C * 2 * case["taps"]}
    N, G = case["states"], case["groups"]
    size = rows * 2 * (C * (3 + case["gated"]) + 2 * G * N) + 4 * C * N
    size += 4 * C * (case["skip"] + case["softplus"]) + moves * C * N * 4
    return {"bytes": size, "flops": rows * C * (7 * N + 10)}

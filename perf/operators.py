"""The linear-attention and snapshot operators as they are measured.

Operators (state pages are FP32 [slot, head, 128 value rows, 128 keys]; slot 0
is the null slot):

* ``prompt``: linear attention with one decay per head over ragged prompts,
  S_t = exp(g_t) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t, pages in and out;
* ``step``: the same for one token per request, the page updated in place;
* ``fork``: a page quantised into a snapshot (8 or 4 bits) and read back into
  another slot, as a request is forked;
* ``load``: snapshots read back into pages.
"""
import random

import torch

own = False

D = 128            # keys and values of a page
CHUNK = 128        # tokens of a chunk in the plain form
SCALE = D ** -0.5


def listed():
    return [
        # drafts of a few requests checked by the prompt form: latency
        dict(name="prompt_drafts_b4_h8", op="prompt", seqs=4, heads=8, qk_heads=8, shortest=1,
             longest=9, lengths=11, per_token=True, carried=True),
        # an ordinary prefill batch of ragged prompts, data-dependent decay
        dict(name="prompt_ragged_b8_h32", op="prompt", seqs=8, heads=32, qk_heads=32,
             shortest=257, longest=2047, lengths=12, per_token=True, carried=True),
        # one long document, a fixed decay for each head
        dict(name="prompt_long_h32", op="prompt", seqs=1, heads=32, qk_heads=32, shortest=32749,
             longest=32749, lengths=13, per_token=False, carried=False),
        # many short suffixes behind cached prefixes: pages and tokens weigh alike
        dict(name="prompt_suffixes_b256_h32", op="prompt", seqs=256, heads=32, qk_heads=32,
             shortest=16, longest=256, lengths=14, per_token=True, carried=True),
        # groups of 8 heads share their queries and keys
        dict(name="prompt_shared_qk_b16_h64", op="prompt", seqs=16, heads=64, qk_heads=8,
             shortest=500, longest=1500, lengths=15, per_token=True, carried=False),
        # decode of a few requests: latency
        dict(name="step_b4_h8", op="step", seqs=4, heads=8, qk_heads=8, pad=0, per_token=True),
        # an ordinary decode batch, an eighth of it padding
        dict(name="step_b64_h32_pad8", op="step", seqs=64, heads=32, qk_heads=32, pad=8,
             per_token=True),
        # the largest decode batch, a fixed decay, shared queries and keys
        dict(name="step_b256_h32", op="step", seqs=256, heads=32, qk_heads=4, pad=0,
             per_token=False),
        # requests forked through 8-bit and 4-bit snapshots
        dict(name="fork_8bit_b64_h32", op="fork", seqs=64, heads=32, bits=8, pad=0),
        dict(name="fork_4bit_b5_h8", op="fork", seqs=5, heads=8, bits=4, pad=1),
        # prefix-cache hits: snapshots read back
        dict(name="load_8bit_b3_h8", op="load", seqs=3, heads=8, bits=8, pad=0),
        dict(name="load_4bit_b128_h64", op="load", seqs=128, heads=64, bits=4, pad=9),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "step", "fork", "load"])
    heads = rng.choice([8, 16, 24, 32, 64])
    if op == "prompt":
        seqs = _spread(rng, 1, 256)
        most = max(1, 1_000_000 // (seqs * heads))     # keeps tokens x heads below the largest case's
        longest = _spread(rng, min(4, most), min(most, 32000))
        shortest = _spread(rng, 1, longest)
        return dict(op=op, seqs=seqs, heads=heads, qk_heads=rng.choice([heads, heads, heads // 8]),
                    shortest=shortest, longest=longest, lengths=rng.randrange(1 << 30),
                    per_token=rng.random() < 0.6, carried=rng.random() < 0.5)
    seqs = _spread(rng, 1, 8192 // heads)
    pad = rng.choice([0, 0, seqs // 8])
    if op == "step":
        return dict(op=op, seqs=seqs, heads=heads, qk_heads=rng.choice([heads, heads, heads // 8]),
                    pad=pad, per_token=rng.random() < 0.6)
    return dict(op=op, seqs=seqs, heads=heads, bits=rng.choice([8, 4]), pad=pad)


def _lens(case):
    r = random.Random(case["lengths"])
    return [r.randint(case["shortest"], case["longest"]) for _ in range(case["seqs"])]


def _decays(g, case, rows):
    """Logarithms of the decays. Fixed: one rate for each head, from slow to fast.
    Per token: a rate for each head times a softplus of the token's own logit."""
    H = case["heads"]
    if not case["per_token"]:
        return -torch.exp2(-1.0 - 8.0 * torch.arange(H, device="cuda") / H)
    rate = torch.exp(torch.rand(H, generator=g, device="cuda") * 4.0 - 4.0)
    x = torch.randn(rows, H, generator=g, device="cuda")
    return -rate * torch.log1p(torch.exp(x))


def _unit(x, heads):
    """Rows of unit length in bf16, as the layer's norm leaves queries and keys."""
    x = x.view(x.shape[0], heads, D)
    return (x * x.square().sum(-1, keepdim=True).rsqrt()).to(torch.bfloat16).view(x.shape[0], -1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H = case["seqs"], case["heads"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] in ("prompt", "step"):
        Hk = case["qk_heads"]
        lens = _lens(case) if case["op"] == "prompt" else [1] * B
        rows = sum(lens)
        s = dict(op=case["op"], heads=H, lens=lens,
                 q=_unit(randn(rows, Hk * D), Hk), k=_unit(randn(rows, Hk * D), Hk),
                 v=randn(rows, H * D).to(torch.bfloat16), decay=_decays(g, case, rows),
                 output=torch.zeros(rows, H * D, dtype=torch.bfloat16, device="cuda"))
    else:
        s = dict(op=case["op"], heads=H, bits=case["bits"])
    if case["op"] == "prompt":
        starts = torch.tensor([0] + lens, device="cuda").cumsum(0)
        at = torch.randperm(2 * B, generator=g, device="cuda").to(torch.int32) + 1
        s.update(state=randn(2 * B + 1, H, D, D) * 0.1, seq_starts=starts.to(torch.int32),
                 src_slots=at[:B].contiguous() if case["carried"] else None,
                 dst_slots=at[B:].contiguous())
        return s
    if case["op"] == "step":
        s["state"] = randn(B + 1, H, D, D) * 0.1
        s["slots"] = torch.randperm(B, generator=g, device="cuda").to(torch.int32) + 1
        if case["pad"]:
            s["slots"][torch.randperm(B, generator=g, device="cuda")[:case["pad"]]] = 0
        if own:   # a decoding program prepares its step once, over its own buffers
            from linear_attention_recurrent_kda_gb300.api import KdaLinStep
            s["step"] = KdaLinStep(q=s["q"], k=s["k"], v=s["v"], decay=s["decay"],
                                   slots=s["slots"], state=s["state"], output=s["output"],
                                   scale=SCALE)
        return s
    bits = case["bits"]
    snaps = torch.randperm(B, generator=g, device="cuda").to(torch.int32) + 1
    if case["pad"]:
        snaps[torch.randperm(B, generator=g, device="cuda")[:case["pad"]]] = 0
    s["snaps"] = snaps
    # keys differ in how much of the state they hold, and so do heads
    spread = torch.exp(0.5 * randn(1, H, 1, D)) * 0.1
    if case["op"] == "fork":
        at = torch.randperm(2 * B, generator=g, device="cuda").to(torch.int32) + 1
        s.update(state=randn(2 * B + 1, H, D, D) * spread, src_slots=at[:B].contiguous(),
                 dst_slots=at[B:].contiguous(),
                 codes=torch.zeros(B + 1, H, D, D if bits == 8 else D // 2, device="cuda",
                                   dtype=torch.int8 if bits == 8 else torch.uint8),
                 scales=torch.zeros((B + 1, H, D) if bits == 8 else (B + 1, H, D, 4),
                                    device="cuda"))
        return s
    top = 127 if bits == 8 else 7
    codes = torch.randint(-top, top + 1, (B + 1, H, D, D), generator=g, device="cuda",
                          dtype=torch.int8)
    if bits == 4:
        codes = ((codes[..., 0::2] & 15) | ((codes[..., 1::2] & 15) << 4)).view(torch.uint8)
    scales = torch.rand((B + 1, H, D) if bits == 8 else (B + 1, H, D, 4), generator=g,
                        device="cuda") * 0.01
    s.update(state=torch.zeros(B + 1, H, D, D, device="cuda"), codes=codes, scales=scales,
             dst_slots=torch.randperm(B, generator=g, device="cuda").to(torch.int32) + 1)
    return s


def run(s):
    if s["op"] == "prompt":
        if own:
            from linear_attention_recurrent_kda_gb300.api import kda_lin_prompt
            kda_lin_prompt(q=s["q"], k=s["k"], v=s["v"], decay=s["decay"],
                           seq_starts=s["seq_starts"], output=s["output"], state=s["state"],
                           src_slots=s["src_slots"], dst_slots=s["dst_slots"], scale=SCALE,
                           max_seq=max(s["lens"]))
        else:
            _plain_prompt(s)
        return [s["output"], s["state"]]
    if s["op"] == "step":
        if own:
            s["step"]()
        else:
            _plain_step(s)
        return [s["output"], s["state"]]
    if own:
        from linear_attention_recurrent_kda_gb300.api import kda_snapshot_load, kda_snapshot_save
        if s["op"] == "fork":
            kda_snapshot_save(state=s["state"], slots=s["src_slots"], codes=s["codes"],
                              scales=s["scales"], snaps=s["snaps"])
        kda_snapshot_load(codes=s["codes"], scales=s["scales"], snaps=s["snaps"],
                          state=s["state"], slots=s["dst_slots"])
    else:
        if s["op"] == "fork":
            _plain_save(s)
        _plain_load(s)
    return [s["state"]]


def _plain_prompt(s):
    """All chunks at once: inside a chunk by the masked product, across chunks by
    the matrix of the decays from each chunk's end to each later one's."""
    dev, H, B = s["q"].device, s["heads"], len(s["lens"])
    lens = torch.tensor(s["lens"], device=dev)
    starts = s["seq_starts"].long()
    counts = (lens + CHUNK - 1) // CHUNK
    total = sum(-(-n // CHUNK) for n in s["lens"])
    seq = torch.repeat_interleave(torch.arange(B, device=dev), counts, output_size=total)
    ends = counts.cumsum(0)
    place = torch.arange(total, device=dev) - (ends - counts)[seq]
    at = place[:, None] * CHUNK + torch.arange(CHUNK, device=dev)
    live = at < lens[seq][:, None]
    row = torch.where(live, starts[seq][:, None] + at, 0)

    def chunks(x):  # [chunks, heads, CHUNK, D] in FP32, zeros behind a sequence's end
        x = x[row].float().view(total, CHUNK, -1, D).transpose(1, 2)
        return torch.where(live[:, None, :, None], x, 0.0).repeat_interleave(H // x.shape[1], 1)

    q, k, v = chunks(s["q"]), chunks(s["k"]), chunks(s["v"])
    g = s["decay"].double()
    g = g[row] if g.dim() == 2 else g.expand(total, CHUNK, H)
    b = torch.where(live[:, :, None], g, 0.0).cumsum(1).transpose(1, 2)   # [chunks, heads, CHUNK]
    seen = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    decay = torch.where(seen, b[..., :, None] - b[..., None, :], -torch.inf).exp().float()
    inside = (q @ k.transpose(-1, -2) * decay) @ v
    left = (b[..., -1:] - b).exp().float()
    add = (v * left[..., None]).transpose(-1, -2) @ k                     # [chunks, heads, D, D]
    cum = b[..., -1].cumsum(0)                                            # [chunks, heads]
    own_seq = (seq[:, None] == seq) & (place[:, None] >= place)
    across = torch.where(own_seq, (cum.T[:, :, None] - cum.T[:, None, :]), -torch.inf).exp().float()
    after = (across @ add.transpose(0, 1).reshape(H, total, D * D)).view(H, total, D, D)
    after = after.transpose(0, 1)
    if s["src_slots"] is not None:
        first = s["state"][s["src_slots"].long()]
        base = cum - b[..., -1]                                           # before the chunk
        since = (cum - base[(ends - counts)[seq]]).exp().float()
        after = after + first[seq] * since[..., None, None]
        before = torch.where((place > 0)[:, None, None, None], after.roll(1, 0), first[seq])
    else:
        before = torch.where((place > 0)[:, None, None, None], after.roll(1, 0), 0.0)
    outside = (q @ before.transpose(-1, -2)) * b.exp().float()[..., None]
    o = ((inside + outside) * SCALE).transpose(1, 2).reshape(total, CHUNK, H * D)
    s["output"][row[live]] = o[live].to(torch.bfloat16)
    s["state"][s["dst_slots"].long()] = after[ends - 1]


def _plain_step(s):
    H = s["heads"]
    B = s["slots"].shape[0]
    q, k = (s[n].float().view(B, -1, D).repeat_interleave(H * D // s[n].shape[1], 1) for n in "qk")
    v = s["v"].float().view(B, H, D)
    live = s["slots"] > 0
    at = s["slots"].long()
    page = s["state"][at] * s["decay"].exp().expand(B, H)[..., None, None]
    page = page + v[..., :, None] * k[..., None, :]
    o = (page @ q[..., None]).view(B, H * D) * SCALE
    s["output"].copy_(torch.where(live[:, None], o, 0.0))
    s["state"][at] = torch.where(live[:, None, None, None], page, s["state"][:1])


def _plain_save(s):
    live = s["snaps"] > 0
    x = s["state"][s["src_slots"].long()]
    top = 127 if s["bits"] == 8 else 7
    x = x.view(*x.shape[:3], D // 32 if s["bits"] == 4 else 1, -1)
    # divided in 64 bits: the scale's last bit decides codes next to a border
    scale = (x.abs().amax(-1, keepdim=True).double() / top).float()
    codes = torch.where(scale > 0, x.double() / scale, 0.0).round().to(torch.int8).view(*x.shape[:3], D)
    if s["bits"] == 4:
        codes = ((codes[..., 0::2] & 15) | ((codes[..., 1::2] & 15) << 4)).view(torch.uint8)
    at = s["snaps"].long()
    s["codes"][at] = torch.where(live[:, None, None, None], codes, s["codes"][:1])
    scale = scale.view(-1, *s["scales"].shape[1:])
    s["scales"][at] = torch.where(live.view(-1, *[1] * (scale.dim() - 1)), scale, s["scales"][:1])


def _plain_load(s):
    live = (s["snaps"] > 0)[:, None, None, None]
    at = s["snaps"].long()
    codes, scale = s["codes"][at], s["scales"][at]
    if s["bits"] == 4:
        codes = codes.view(torch.int8)
        codes = torch.stack([(codes << 4) >> 4, codes >> 4], -1)
    x = (codes.reshape(*codes.shape[:3], scale[0, 0, 0].numel(), -1).float()
         * scale.reshape(*codes.shape[:3], -1, 1)).view(*codes.shape[:3], D)
    to = s["dst_slots"].long()
    s["state"][to] = torch.where(live, x, s["state"][to])


def exact(case, seed):
    s = prepare(case, seed)
    pool = s["state"].double()
    if s["op"] == "load":
        codes = s["codes"].to(torch.int16)
        if s["bits"] == 4:
            low, high = codes % 16, codes // 16
            codes = torch.stack([low - 16 * (low > 7), high - 16 * (high > 7)], -1).flatten(-2)
        for r, snap in enumerate(s["snaps"].tolist()):
            if snap > 0:
                scale = s["scales"][snap].double().repeat_interleave(D if s["bits"] == 8 else 32, -1)
                pool[int(s["dst_slots"][r])] = codes[snap].double() * scale.view(-1, D, D)
        return [pool]
    if s["op"] == "fork":
        top, width = (127, D) if s["bits"] == 8 else (7, 32)
        for r, snap in enumerate(s["snaps"].tolist()):
            if snap > 0:
                x = pool[int(s["src_slots"][r])].unflatten(-1, (-1, width))
                # the scale is stored in 32 bits: part of the format
                scale = (x.abs().amax(-1, keepdim=True) / top).float().double()
                x = torch.round(x / scale.clamp_min(1e-300)) * scale
                pool[int(s["dst_slots"][r])] = x.flatten(-2)
        return [pool]
    # the recurrence, token by token, all live sequences at a time, longest first
    H, lens = s["heads"], s["lens"]
    per = H * D // s["q"].shape[1]
    order = sorted(range(len(lens)), key=lambda r: -lens[r])
    begin = [sum(lens[:r]) for r in range(len(lens))]
    begin = torch.tensor([begin[r] for r in order], device="cuda")
    order_t = torch.tensor(order, device="cuda")
    if s["op"] == "step":
        src, dst = s["slots"][order_t].long(), s["slots"][order_t].long()
    else:
        dst = s["dst_slots"][order_t].long()
        src = s["src_slots"][order_t].long() if s["src_slots"] is not None else torch.zeros_like(dst)
    out = torch.zeros(s["output"].shape, dtype=torch.float64, device="cuda")
    S = pool[src] * (src > 0)[:, None, None, None]
    n = len(lens)
    keep = s["decay"].double().exp()
    for t in range(lens[order[0]]):
        while lens[order[n - 1]] <= t:
            n -= 1
        at = begin[:n] + t
        q, k = (s[x][at].double().view(n, -1, 1, D).repeat_interleave(per, 1) for x in "qk")
        v = s["v"][at].double().view(n, H, D, 1)
        live = S[:n]
        live *= keep[at].view(n, H, 1, 1) if keep.dim() == 2 else keep.view(H, 1, 1)
        live.addcmul_(v, k)
        out[at] = ((live * q).sum(-1) * SCALE).view(n, H * D)
    if s["op"] == "step":
        out[begin[src == 0]] = 0.0
        pool[dst[dst > 0]] = S[dst > 0]
    else:
        pool[dst] = S
    return [out, pool]


def work(case):
    H = case["heads"]
    page, live = 4 * D * D, case["seqs"] - case.get("pad", 0)
    if case["op"] in ("prompt", "step"):
        rows = sum(_lens(case)) if case["op"] == "prompt" else live
        pages = (1 + (case["op"] == "step" or case["carried"])) * live
        size = rows * 2 * (2 * case["qk_heads"] + 2 * H) * D + pages * H * page
        size += 4 * (rows * H if case["per_token"] else H)
        return {"bytes": size, "flops": rows * H * 4 * D * D}
    kept = D * D * case["bits"] // 8 + 4 * D * (1 if case["bits"] == 8 else 4)
    moved = page + kept
    if case["op"] == "fork":
        return {"bytes": live * H * 2 * moved, "flops": live * H * 4 * D * D}
    return {"bytes": live * H * moved, "flops": live * H * D * D}

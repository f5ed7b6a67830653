"""Python binding of the KDA decode / verify C ABI (include/kda.h).

PyTorch is used only for device memory and streams: the functions here check
that every tensor is a contiguous CUDA tensor of the documented dtype and shape,
fill ``struct kda_args`` with raw pointers and call ``kda_decode`` /
``kda_verify`` in ``libkda_gb300.so``.  Nothing of the step is computed in
Python and there is no fallback path.

Method: vLLM API page
"vllm.models.kimi_k3.nvidia.specialized_decode.cutedsl.kda.wide" (KdaWide).
"""
from __future__ import annotations

from typing import Dict, Optional

import torch

from . import lib as _lib

DK = 128


def _check(name, t, dtype, shape=None, allow_none=False):
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _ptr(t):
    return None if t is None else t.data_ptr()


def _same_device(dev, **tensors):
    """Every given tensor (None skipped) lives on ``dev``: the kernel would
    otherwise dereference another GPU's pointer."""
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")


class KdaStep:
    """A prepared KDA step over fixed device tensors.

    Validates once, keeps the filled ``kda_args`` and launches with
    ``__call__(stream)``; reuse it across steps that read the same buffers
    (the tensors' contents may change between calls, their storage may not).

    ``sched``: the persistent kernel's scheduler words (int32 [2], zero before
    first use; ``kda_args.sched``).  By default the step allocates its own,
    so its launches balance the last items over the CTAs; pass a tensor to
    share one between steps launched in order on one stream, or
    ``balance=False`` for fixed contiguous ranges only (same bits).
    ``noalloc=True`` allocates nothing and calls ``kda_step_noalloc``, which
    uses the library's own words (launches through it must be ordered).
    """

    def __init__(self, *, x, conv_weight, conv_state, f_a, f_b, beta, a_log,
                 dt_bias, slots, state, output, gate, norm_weight,
                 lower_bound: float, scale: float, eps: float,
                 tokens: int = 1, accepted=None, conv_bias=None,
                 gate_mode: int = 0, record: bool = False, rec_u=None,
                 rec_kg=None, err=None, dbg=None, use_pdl: bool = False,
                 path: int = 0, sched=None, balance: bool = True,
                 noalloc: bool = False):
        bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
        T = int(tokens)
        if not 1 <= T <= 8:
            raise ValueError(f"tokens must be 1..8, got {T}")
        _check("a_log", a_log, f32)
        H = a_log.shape[0]
        dim = H * DK
        _check("output", output, bf)
        if output.dim() != 2 or output.shape[1] != dim or output.shape[0] % T:
            raise ValueError("output must be [batch*tokens, heads*128]")
        B = output.shape[0] // T
        _check("state", state, f32)
        if state.dim() != 4 or tuple(state.shape[1:]) != (H, DK, DK):
            raise ValueError("state must be [num_slots, heads, 128, 128]")
        num_slots = state.shape[0]
        if not isinstance(conv_state, torch.Tensor) or conv_state.dtype not in (bf, f32):
            raise TypeError("conv_state must be a bfloat16 or float32 tensor")
        _check("conv_state", conv_state, conv_state.dtype)
        if conv_state.dim() != 3 or tuple(conv_state.shape[:2]) != (num_slots, 3 * dim):
            raise ValueError("conv_state must be [num_slots, 3*heads*128, width]")
        W = conv_state.shape[2]
        _check("x", x, bf, (B * T, 3 * dim))
        _check("conv_weight", conv_weight, bf, (3, 4, dim))
        _check("conv_bias", conv_bias, bf, (3 * dim,), allow_none=True)
        _check("f_a", f_a, bf, (B * T, DK))
        _check("f_b", f_b, bf, (dim, DK))
        _check("beta", beta, bf, (B * T, H))
        _check("dt_bias", dt_bias, f32, (dim,))
        _check("gate", gate, bf, (B * T, dim))
        _check("norm_weight", norm_weight, bf, (DK,))
        _check("slots", slots, i32)
        if T == 1:
            if slots.numel() != B:
                raise ValueError("decode slots must be [batch]")
            slot_cols = 1
        else:
            if slots.dim() != 2 or slots.shape[0] != B:
                raise ValueError("verify slots must be [batch, >= tokens]")
            slot_cols = slots.shape[1]
            _check("accepted", accepted, i32, (B,))
        if record:
            _check("rec_u", rec_u, f32, (B, H, T, DK))
            _check("rec_kg", rec_kg, bf, (B, H, T, 2 * DK))
        _check("err", err, i32, allow_none=True)
        _check("dbg", dbg, bf, (B, H, T, 4, DK), allow_none=True)
        dev = output.device
        if noalloc:
            sched = None
        elif sched is None and balance:
            sched = torch.zeros(2, dtype=i32, device=dev)
        _check("sched", sched, i32, (2,), allow_none=True)
        _same_device(dev, x=x, conv_weight=conv_weight, conv_bias=conv_bias,
                     conv_state=conv_state, f_a=f_a, f_b=f_b, beta=beta, a_log=a_log,
                     dt_bias=dt_bias, slots=slots, state=state, gate=gate,
                     norm_weight=norm_weight, accepted=accepted if T > 1 else None,
                     rec_u=rec_u if record else None, rec_kg=rec_kg if record else None,
                     err=err, dbg=dbg, sched=sched)

        a = _lib.KdaArgs()
        a.batch, a.heads, a.tokens = B, H, T
        a.num_slots, a.conv_width, a.slot_cols = num_slots, W, slot_cols
        a.gate_mode, a.has_bias = int(gate_mode), int(conv_bias is not None)
        a.record, a.use_pdl = int(bool(record)), int(bool(use_pdl))
        a.x, a.conv_weight, a.conv_bias = _ptr(x), _ptr(conv_weight), _ptr(conv_bias)
        a.f_a, a.f_b, a.beta = _ptr(f_a), _ptr(f_b), _ptr(beta)
        a.gate, a.norm_weight = _ptr(gate), _ptr(norm_weight)
        a.a_log, a.dt_bias = _ptr(a_log), _ptr(dt_bias)
        a.slots, a.accepted = _ptr(slots), _ptr(accepted if T > 1 else None)
        a.conv_state, a.state, a.output = _ptr(conv_state), _ptr(state), _ptr(output)
        a.rec_u, a.rec_kg = _ptr(rec_u), _ptr(rec_kg)
        a.lower_bound, a.scale, a.eps = float(lower_bound), float(scale), float(eps)
        a.err, a.dbg = _ptr(err), _ptr(dbg)
        a.path = int(path)
        a.conv_f32 = int(conv_state.dtype == f32)
        a.sched = _ptr(sched)
        self.args = a
        self.entry = ("kda_step_noalloc" if noalloc else
                      "kda_decode" if T == 1 else "kda_verify")
        self.device = dev
        # keep the tensors alive as long as the prepared step
        self._keep = (x, conv_weight, conv_state, f_a, f_b, beta, a_log, dt_bias,
                      slots, state, output, gate, norm_weight, accepted,
                      conv_bias, rec_u, rec_kg, err, dbg, sched)

    def __call__(self, stream: Optional[torch.cuda.Stream] = None) -> None:
        # the library launches on the current device: make it the tensors' one
        with torch.cuda.device(self.device):
            s = stream if stream is not None else torch.cuda.current_stream(self.device)
            rc = _lib.call(self.entry, self.args, s.cuda_stream)
        if rc != _lib.KDA_SUCCESS:
            raise _lib.KdaError(rc, _lib.strerror(rc))


def kda_decode(stream: Optional[torch.cuda.Stream] = None, **kw) -> None:
    """One decode step (tokens = 1) on ``stream``; see ``KdaStep``."""
    if kw.get("tokens", 1) != 1:
        raise ValueError("kda_decode takes tokens = 1")
    KdaStep(**kw)(stream)


def kda_verify(stream: Optional[torch.cuda.Stream] = None, **kw) -> None:
    """One speculative-verify step (tokens 2..8, optional record mode)."""
    if kw.get("tokens", 1) < 2:
        raise ValueError("kda_verify takes tokens >= 2")
    KdaStep(**kw)(stream)


INPUT_KEYS = ("x", "conv_weight", "conv_bias", "conv_state", "f_a", "f_b", "beta",
              "a_log", "dt_bias", "slots", "accepted", "state", "gate",
              "norm_weight")


def step_from_inputs(dev_inputs: Dict[str, object], output: torch.Tensor, *,
                     rec_u=None, rec_kg=None, err=None, dbg=None,
                     use_pdl: bool = False, path: int = 0, sched=None,
                     balance: bool = True, noalloc: bool = False) -> KdaStep:
    """A ``KdaStep`` from a device copy of a seeded workload's input dict."""
    d = dev_inputs
    T = int(d["tokens"])
    return KdaStep(
        x=d["x"], conv_weight=d["conv_weight"], conv_state=d["conv_state"],
        f_a=d["f_a"], f_b=d["f_b"], beta=d["beta"], a_log=d["a_log"],
        dt_bias=d["dt_bias"], slots=d["slots"], state=d["state"], output=output,
        gate=d["gate"], norm_weight=d["norm_weight"],
        lower_bound=d["lower_bound"], scale=d["scale"], eps=d["eps"], tokens=T,
        accepted=d.get("accepted") if T > 1 else None,
        conv_bias=d.get("conv_bias") if d.get("has_bias") else None,
        gate_mode=int(d["gate_mode"]), record=bool(d["record"]), rec_u=rec_u,
        rec_kg=rec_kg, err=err, dbg=dbg, use_pdl=use_pdl, path=path, sched=sched,
        balance=balance, noalloc=noalloc)


def kda_recover(*, state, src_slots, dst_slots, accepted, rec_u, rec_kg, a_log,
                dt_bias, lower_bound: float, err=None, sched=None, balance: bool = True,
                stream: Optional[torch.cuda.Stream] = None) -> None:
    """Record replay (include/kda.h ``kda_recover``): rebuild the accepted
    state pages from checkpoint pages and a record-mode verify's records.
    ``sched``: scheduler words (int32 [2], zero); by default a fresh pair per
    call (``balance=False``: contiguous item ranges only, same bits)."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    _check("rec_u", rec_u, f32)
    if rec_u.dim() != 4 or rec_u.shape[3] != DK:
        raise ValueError("rec_u must be [batch, heads, tokens, 128]")
    B, H, T = rec_u.shape[:3]
    _check("rec_kg", rec_kg, bf, (B, H, T, 2 * DK))
    _check("state", state, f32)
    if state.dim() != 4 or tuple(state.shape[1:]) != (H, DK, DK):
        raise ValueError("state must be [num_slots, heads, 128, 128]")
    for n, t in (("src_slots", src_slots), ("dst_slots", dst_slots),
                 ("accepted", accepted)):
        _check(n, t, i32, (B,))
    _check("a_log", a_log, f32, (H,))
    _check("dt_bias", dt_bias, f32, (H * DK,))
    _check("err", err, i32, allow_none=True)
    if sched is None and balance:
        sched = torch.zeros(2, dtype=i32, device=state.device)
    _check("sched", sched, i32, (2,), allow_none=True)
    _same_device(state.device, src_slots=src_slots, dst_slots=dst_slots, accepted=accepted,
                 rec_u=rec_u, rec_kg=rec_kg, a_log=a_log, dt_bias=dt_bias, err=err,
                 sched=sched)
    a = _lib.KdaRecoverArgs()
    a.batch, a.heads, a.tokens, a.num_slots = B, H, T, state.shape[0]
    a.src_slots, a.dst_slots, a.accepted = (_ptr(src_slots), _ptr(dst_slots),
                                            _ptr(accepted))
    a.rec_u, a.rec_kg = _ptr(rec_u), _ptr(rec_kg)
    a.a_log, a.dt_bias = _ptr(a_log), _ptr(dt_bias)
    a.lower_bound = float(lower_bound)
    a.state, a.err = _ptr(state), _ptr(err)
    a.sched = _ptr(sched)
    with torch.cuda.device(state.device):
        s = stream if stream is not None else torch.cuda.current_stream(state.device)
        rc = _lib.call("kda_recover", a, s.cuda_stream)
    if rc != _lib.KDA_SUCCESS:
        raise _lib.KdaError(rc, _lib.strerror(rc))


def kda_oproj(*, partials, prefix, output, out_norm, blocks=None, norm=None,
              query=None, has_delta: bool = True, eps: float = 1e-6,
              out_eps: float = 1e-6,
              stream: Optional[torch.cuda.Stream] = None) -> None:
    """Output-projection consumer epilogue (include/kda.h ``kda_oproj``).

    ``partials`` bf16 [tp, tokens, hidden]; ``prefix`` bf16 [tokens, hidden]
    (replaced by the new prefix); ``output`` bf16 [tokens, hidden];
    ``out_norm`` bf16 [hidden]; ``blocks`` bf16 [tokens, nb, hidden] with
    ``norm``/``query`` bf16 [hidden], or None for no earlier blocks."""
    bf = torch.bfloat16
    _check("partials", partials, bf)
    if partials.dim() != 3:
        raise ValueError("partials must be [tp, tokens, hidden]")
    tp, T, D = partials.shape
    _check("prefix", prefix, bf, (T, D))
    _check("output", output, bf, (T, D))
    _check("out_norm", out_norm, bf, (D,))
    nb = 0
    if blocks is not None:
        _check("blocks", blocks, bf)
        if blocks.dim() != 3 or blocks.shape[0] != T or blocks.shape[2] != D:
            raise ValueError("blocks must be [tokens, nb, hidden]")
        nb = blocks.shape[1]
        _check("norm", norm, bf, (D,))
        _check("query", query, bf, (D,))
    _same_device(partials.device, prefix=prefix, output=output, out_norm=out_norm,
                 blocks=blocks if nb else None, norm=norm if nb else None,
                 query=query if nb else None)
    a = _lib.KdaOprojArgs()
    a.tp, a.tokens, a.hidden, a.nb = tp, T, D, nb
    a.has_delta = int(bool(has_delta))
    a.partials, a.prefix, a.output = _ptr(partials), _ptr(prefix), _ptr(output)
    a.out_norm = _ptr(out_norm)
    a.blocks = _ptr(blocks) if nb else None
    a.norm = _ptr(norm) if nb else None
    a.query = _ptr(query) if nb else None
    a.eps, a.out_eps = float(eps), float(out_eps)
    with torch.cuda.device(partials.device):
        s = stream if stream is not None else torch.cuda.current_stream(partials.device)
        rc = _lib.call("kda_oproj", a, s.cuda_stream)
    if rc != _lib.KDA_SUCCESS:
        raise _lib.KdaError(rc, _lib.strerror(rc))


# ------------------------------------ linear attention with one decay per head
#
# These calls are short, so their host side is too: one look at each tensor, and
# the general checks (with their messages) only where that look fails.

_Tensor, _BF16, _F32, _I32 = torch.Tensor, torch.bfloat16, torch.float32, torch.int32


def _want(name, t, dtype, shape, index):
    """The address of a contiguous CUDA tensor of this type, shape (None: any)
    and device."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.is_contiguous()
            and t.get_device() == index and (shape is None or t.shape == shape)):
        _check(name, t, dtype, shape)
        _same_device(torch.device("cuda", index), **{name: t})
    return t.data_ptr()


def _count(name, n):
    """A number of rows, slots or entries that the library's 32-bit field holds (ctypes
    would keep its low bits)."""
    if n >= 1 << 31:
        raise ValueError(f"{name}: {n} are more than the library counts (2^31 - 1)")
    return n


def _counts(**sizes):
    for name, n in sizes.items():
        _count(name, n)


def _maybe(name, t, dtype, shape, index):
    return None if t is None else _want(name, t, dtype, shape, index)


def _cuda_index(name, t):
    """Index of the CUDA device of a tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    return t.get_device()


def _rows(name, t, rows, width, index):
    """(address, row stride) of a BF16 CUDA tensor [rows, width] whose rows may be
    slices of wider rows: elements of a row adjacent, any row stride that the
    library takes."""
    if not (isinstance(t, _Tensor) and t.dtype is _BF16
            and t.get_device() == index and t.shape == (rows, width)):
        if _cuda_index(name, t) != index:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
        if t.dtype is not torch.bfloat16:
            raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
        raise ValueError(f"{name} must have shape {(rows, width)}, got {tuple(t.shape)}")
    step, one = t.stride()
    if one == 1 and rows > 1 and step >= width > 0 and not step & 7:
        return t.data_ptr(), step
    if not width:
        return t.data_ptr(), 0
    if rows <= 1:
        step = -(-width // 8) * 8
    if (one != 1 and width > 1) or step % 8 or step < width:
        raise ValueError(f"{name}: the elements of a row must be adjacent and rows a "
                         f"multiple of 8 elements apart, got strides {tuple(t.stride())}")
    return t.data_ptr(), step


def _lin_shape(q, v):
    """(device index, rows, heads, qk_heads) of linear-attention rows."""
    index = _cuda_index("v", v)
    _cuda_index("q", q)
    if v.dim() != 2 or q.dim() != 2 or v.shape[1] % DK or q.shape[1] % DK or not q.shape[1]:
        raise ValueError("q, k and v must be rows of whole heads of 128")
    rows, width = _count("v", v.shape[0]), v.shape[1]
    H, Hk = width // DK, q.shape[1] // DK
    if H % Hk:
        raise ValueError(f"{H} value heads are not a multiple of {Hk} query heads")
    return index, rows, H, Hk


def _decay(decay, rows, H, index):
    per_row = isinstance(decay, torch.Tensor) and decay.dim() == 2
    return _want("decay", decay, torch.float32, (rows, H) if per_row else (H,), index), int(per_row)


def _state(state, H, index):
    ptr = _want("state", state, torch.float32, None, index)
    if state.dim() != 4 or state.shape[1:] != (H, DK, DK):
        raise ValueError(f"state must be [num_slots, {H}, 128, 128], got {tuple(state.shape)}")
    return ptr, _count("state", state.shape[0])


def _run(entry, args, index, stream, *more):
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device_index != index:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, expected cuda:{index}")
    else:
        handle = stream.cuda_stream
    # the library launches on the current device: make it the tensors' one
    if torch._C._cuda_getDevice() == index:
        rc = _lib.call(entry, args, handle, *more)
    else:
        with torch.cuda.device(index):
            rc = _lib.call(entry, args, handle, *more)
    if rc != _lib.KDA_SUCCESS:
        raise _lib.KdaError(rc, _lib.strerror(rc))


def _path(path):
    """A form's number; -1, which the library refuses, for what its 32 bits do not hold."""
    return path if 0 <= path < 1 << 31 else -1


def _most(max_seq, rows):
    """The longest sequence's length (-1, which the library refuses, for all below 0)."""
    return rows if max_seq is None else max(-1, min(int(max_seq), rows))


def _done(rc):
    """Whether a call by the short way (csrc/kda_bind.cpp) was made; None leaves it, or
    what is to be said about it, to the checks below."""
    if rc:
        raise _lib.KdaError(rc, _lib.strerror(rc))
    return rc is not None


def kda_lin_prompt(*, q, k, v, decay, seq_starts, output, scale: float, state=None,
                   src_slots=None, dst_slots=None, max_seq: Optional[int] = None, err=None,
                   path: int = 0, workspace=None,
                   stream: Optional[torch.cuda.Stream] = None) -> None:
    """Linear attention with one decay per head over ragged prompts
    (include/kda.h ``kda_lin_prompt``).

    ``q``, ``k`` bf16 [tokens, qk_heads * 128], ``v``, ``output`` bf16 [tokens,
    heads * 128] (each may be a slice of wider rows); ``decay`` f32, the
    logarithm of the decay, [heads] or [tokens, heads]; ``seq_starts`` i32 [seqs
    + 1]; ``state`` f32 [num_slots, heads, 128, 128] with ``src_slots`` (the
    pages the sequences start from) and ``dst_slots`` (where their last states
    go), i32 [seqs] each or None.  ``max_seq``: no sequence is longer (default:
    ``tokens``; the tighter, the better the work is laid out).  ``workspace``: a
    CUDA uint8 tensor of at least ``lib.prompt_workspace`` bytes; by default
    allocated for the call, on the stream it runs on."""
    i32 = torch.int32
    index, rows, H, Hk = _lin_shape(q, v)
    qp, qs = _rows("q", q, rows, Hk * DK, index)
    kp, ks = _rows("k", k, rows, Hk * DK, index)
    vp, vs = _rows("v", v, rows, H * DK, index)
    op, os_ = _rows("output", output, rows, H * DK, index)
    dp, per_row = _decay(decay, rows, H, index)
    sp = _want("seq_starts", seq_starts, i32, None, index)
    if seq_starts.dim() != 1 or seq_starts.shape[0] < 1:
        raise ValueError("seq_starts must be [seqs + 1]")
    B = _count("seq_starts", seq_starts.shape[0] - 1)
    src = _maybe("src_slots", src_slots, i32, (B,), index)
    dst = _maybe("dst_slots", dst_slots, i32, (B,), index)
    if state is None:
        if src_slots is not None or dst_slots is not None:
            raise ValueError("state is required with src_slots or dst_slots")
        state_p, num_slots = None, 0
    else:
        state_p, num_slots = _state(state, H, index)
    a = _lib.KdaLinPromptArgs(
        B, H, Hk, rows, _most(max_seq, rows), num_slots, per_row,
        _path(int(path)), qs, ks, vs, os_, qp, kp, vp, dp, sp, src, dst, state_p, op, float(scale),
        _maybe("err", err, i32, None, index))
    if workspace is not None:
        a.workspace = _want("workspace", workspace, torch.uint8, None, index)
        a.workspace_bytes = workspace.numel()
    elif (need := _lib.prompt_workspace(a)) > 0:
        # from the pool of the stream that uses it: freed behind its kernels
        with torch.cuda.device(index), torch.cuda.stream(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=v.device)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), need
    _run("kda_lin_prompt", a, index, stream)


class KdaLinStep:
    """A prepared single-token step of linear attention with one decay per head
    (include/kda.h ``kda_lin_step``) over fixed device tensors.

    ``q``, ``k`` bf16 [batch, qk_heads * 128], ``v``, ``output`` bf16 [batch,
    heads * 128]; ``decay`` f32 [heads] or [batch, heads]; ``slots`` i32 [batch]
    (<= 0: padding); ``state`` f32 [num_slots, heads, 128, 128], updated in
    place.  Validates once and launches with ``__call__(stream)``; the tensors'
    contents may change between calls, their storage may not."""

    def __init__(self, *, q, k, v, decay, slots, state, output, scale: float, err=None):
        self.index, rows, H, Hk = index, rows, H, Hk = _lin_shape(q, v)
        qp, qs = _rows("q", q, rows, Hk * DK, index)
        kp, ks = _rows("k", k, rows, Hk * DK, index)
        vp, vs = _rows("v", v, rows, H * DK, index)
        op, os_ = _rows("output", output, rows, H * DK, index)
        dp, per_row = _decay(decay, rows, H, index)
        sp = _want("slots", slots, torch.int32, (rows,), index)
        state_p, num_slots = _state(state, H, index)
        self.args = _lib.KdaLinStepArgs(
            rows, H, Hk, num_slots, per_row, qs, ks, vs, os_, qp, kp, vp, dp, sp, state_p, op,
            float(scale), _maybe("err", err, torch.int32, None, index))
        # keep the tensors alive as long as the prepared step
        self._keep = (q, k, v, decay, slots, state, output, err)

    def __call__(self, stream: Optional[torch.cuda.Stream] = None) -> None:
        _run("kda_lin_step", self.args, self.index, stream)


def kda_lin_step(stream: Optional[torch.cuda.Stream] = None, **kw) -> None:
    """One single-token step on ``stream``; see ``KdaLinStep``."""
    KdaLinStep(**kw)(stream)


# ------------------------------------------------- snapshots of state pages

def _snapshot(entry, state, slots, codes, scales, snaps, err, stream):
    index = _cuda_index("state", state)
    if state.dim() != 4:
        raise ValueError("state must be [num_slots, heads, 128, 128]")
    num_slots, H = _count("state", state.shape[0]), state.shape[1]
    _want("state", state, torch.float32, (num_slots, H, DK, DK), index)
    if _cuda_index("codes", codes) == index and codes.dtype is torch.int8:
        bits, width, groups = 8, DK, (DK,)
    elif codes.dtype is torch.uint8:
        bits, width, groups = 4, DK // 2, (DK, 4)
    else:
        raise TypeError("codes must be an int8 (8 bits) or uint8 (4 bits) tensor")
    n = _count("codes", codes.shape[0]) if codes.dim() else 0
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be an int32 tensor [count]")
    i32, count = torch.int32, _count("slots", slots.shape[0])
    a = _lib.KdaSnapshotArgs(
        count, H, num_slots, n, bits, _want("slots", slots, i32, None, index),
        _want("snaps", snaps, i32, (count,), index), state.data_ptr(),
        _want("codes", codes, codes.dtype, (n, H, DK, width), index),
        _want("scales", scales, torch.float32, (n, H) + groups, index),
        _maybe("err", err, i32, None, index))
    _run(entry, a, index, stream)


def kda_snapshot_save(*, state, slots, codes, scales, snaps, err=None,
                      stream: Optional[torch.cuda.Stream] = None) -> None:
    """Keep the pages ``state[slots[i]]`` as snapshots ``snaps[i]`` in 8 or 4
    bits (include/kda.h ``kda_snapshot_save``).  The KDA step's convolution windows
    (``conv_state``) are not part of them: copy a slot's beside its snapshot.

    ``state`` f32 [num_slots, heads, 128, 128]; ``codes`` int8 [num_snaps, heads,
    128, 128] (8 bits) or uint8 [num_snaps, heads, 128, 64] (4 bits); ``scales``
    f32 [num_snaps, heads, 128] or [num_snaps, heads, 128, 4]; ``slots`` and
    ``snaps`` i32 [count], an entry with either <= 0 is skipped."""
    _snapshot("kda_snapshot_save", state, slots, codes, scales, snaps, err, stream)


def kda_snapshot_load(*, codes, scales, snaps, state, slots, err=None,
                      stream: Optional[torch.cuda.Stream] = None) -> None:
    """Read the snapshots ``snaps[i]`` back into ``state[slots[i]]``; see
    ``kda_snapshot_save``."""
    _snapshot("kda_snapshot_load", state, slots, codes, scales, snaps, err, stream)


# ------------------------------------------------------ short causal convolution

def _sequences(seq_starts, src_slots, dst_slots, index):
    """(count, addresses) of a prompt call's sequences."""
    sp, shape = _want("seq_starts", seq_starts, _I32, None, index), seq_starts.shape
    if len(shape) != 1 or shape[0] < 1:
        raise ValueError("seq_starts must be [seqs + 1]")
    B = _count("seq_starts", shape[0] - 1)
    return (B, sp, None if src_slots is None else _want("src_slots", src_slots, _I32, (B,), index),
            None if dst_slots is None else _want("dst_slots", dst_slots, _I32, (B,), index))


def _conv_shape(x, weight):
    """(device index, rows, channels, parts, taps)"""
    index = _cuda_index("x", x)
    _cuda_index("weight", weight)
    rows, of = x.shape, weight.shape
    if len(rows) != 2 or len(of) not in (2, 3):
        raise ValueError("x must be [tokens, channels], weight [taps, channels] or "
                         "[parts, taps, channels / parts]")
    parts, taps = (1, of[0]) if len(of) == 2 else of[:2]
    if parts * of[-1] != rows[1]:
        raise ValueError(f"weight {tuple(of)} is not of {rows[1]} channels")
    return index, _count("x", rows[0]), _count("channels", rows[1]), parts, taps


def _window(window, channels, index):
    """(address, slots, width, whether FP32) of a window pool."""
    dtype = window.dtype if isinstance(window, _Tensor) else None
    if dtype is not _BF16 and dtype is not _F32:
        raise TypeError("window must be a bfloat16 or float32 tensor")
    ptr, shape = _want("window", window, dtype, None, index), window.shape
    if len(shape) != 3 or shape[1] != channels:
        raise ValueError(f"window must be [num_slots, {channels}, width], got {tuple(shape)}")
    return ptr, _count("window", shape[0]), _count("window", shape[2]), int(dtype is _F32)


def kda_conv_prompt(*, x, weight, seq_starts, output, bias=None, window=None, src_slots=None,
                    dst_slots=None, silu: bool = True, err=None,
                    stream: Optional[torch.cuda.Stream] = None) -> None:
    """Short causal depthwise convolution over ragged prompts (include/kda.h
    ``kda_conv_prompt``).

    ``x``, ``output`` bf16 [tokens, channels] (each may be a slice of wider rows);
    ``weight`` bf16 [taps, channels], or [parts, taps, channels / parts] as the KDA
    step keeps it (``conv_weight``); ``bias`` bf16 [channels]; ``seq_starts`` i32
    [seqs + 1]; ``window`` bf16 or f32 [num_slots, channels, width] (the KDA step's
    ``conv_state``) with ``src_slots`` (the windows the sequences continue from) and
    ``dst_slots`` (where their last inputs go), i32 [seqs] each or None."""
    if _done((_lib._bind or _lib.bind()).conv_prompt(
            x, weight, seq_starts, output, bias, window, src_slots, dst_slots, bool(silu), err, stream)):
        return
    bf = torch.bfloat16
    index, rows, C, parts, taps = _conv_shape(x, weight)
    xp, xs = _rows("x", x, rows, C, index)
    op, os_ = _rows("output", output, rows, C, index)
    B, sp, src, dst = _sequences(seq_starts, src_slots, dst_slots, index)
    if window is None:
        if src_slots is not None or dst_slots is not None:
            raise ValueError("window is required with src_slots or dst_slots")
        wp, num_slots, width, f32 = None, 0, 0, 0
    else:
        wp, num_slots, width, f32 = _window(window, C, index)
    _run("kda_conv_prompt", _lib.KdaConvPromptArgs(
        B, C, parts, taps, rows, num_slots, width, f32, int(bool(silu)), xs, os_, xp,
        _want("weight", weight, bf, None, index), _maybe("bias", bias, bf, (C,), index), sp, src,
        dst, wp, op, _maybe("err", err, torch.int32, None, index)), index, stream)


class KdaConvStep:
    """A prepared single-token convolution (include/kda.h ``kda_conv_step``) over
    fixed device tensors.

    ``x``, ``output`` bf16 [batch, channels]; ``weight``, ``bias``, ``window`` as in
    ``kda_conv_prompt``, the window shifted in place; ``slots`` i32 [batch] (<= 0:
    padding).  Validates once and launches with ``__call__(stream)``; the tensors'
    contents may change between calls, their storage may not."""

    def __init__(self, *, x, weight, slots, window, output, bias=None, silu: bool = True, err=None):
        bf = torch.bfloat16
        self.index, rows, C, parts, taps = index, rows, C, parts, taps = _conv_shape(x, weight)
        xp, xs = _rows("x", x, rows, C, index)
        op, os_ = _rows("output", output, rows, C, index)
        wp, num_slots, width, f32 = _window(window, C, index)
        self.args = _lib.KdaConvStepArgs(
            rows, C, parts, taps, num_slots, width, f32, int(bool(silu)), xs, os_, xp,
            _want("weight", weight, bf, None, index), _maybe("bias", bias, bf, (C,), index),
            _want("slots", slots, torch.int32, (rows,), index), wp, op,
            _maybe("err", err, torch.int32, None, index))
        # keep the tensors alive as long as the prepared step
        self._keep = (x, weight, slots, window, output, bias, err)

    def __call__(self, stream: Optional[torch.cuda.Stream] = None) -> None:
        _run("kda_conv_step", self.args, self.index, stream)


def kda_conv_step(stream: Optional[torch.cuda.Stream] = None, **kw) -> None:
    """One single-token convolution on ``stream``; see ``KdaConvStep``."""
    KdaConvStep(**kw)(stream)


# ------------------------------------------------------- selective state-space scan

def _ssm_rows(x, dt, a, b, c, d, z, dt_bias, output):
    """What the scan's calls share: (device index, rows, channels, states, groups,
    strides and addresses in the structs' order)."""
    index = _cuda_index("x", x)
    _cuda_index("a", a)
    _cuda_index("b", b)
    if x.dim() != 2 or a.dim() != 2 or b.dim() != 2:
        raise ValueError("x must be [tokens, channels], a [channels, states], b and c "
                         "[tokens, groups * states]")
    (rows, C), N, wide = x.shape, a.shape[1], b.shape[1]
    if (rows | C | N | wide) >> 31:
        _counts(x=rows, channels=C, a=N, b=wide)
    ap = _want("a", a, _F32, (C, N), index)
    groups = wide // N if N else 0
    if not N or not groups or groups * N != wide:
        raise ValueError(f"b must be [tokens, groups * {N}], got {tuple(b.shape)}")
    (xp, xs), (tp, ts) = _rows("x", x, rows, C, index), _rows("dt", dt, rows, C, index)
    (bp, bs), (cp, cs) = _rows("b", b, rows, wide, index), _rows("c", c, rows, wide, index)
    zp, zs = (None, 0) if z is None else _rows("z", z, rows, C, index)
    op, os_ = _rows("output", output, rows, C, index)
    return (index, rows, C, N, groups, (xs, ts, bs, cs, zs, os_),
            (xp, tp, ap, bp, cp, _maybe("d", d, _F32, (C,), index), zp,
             _maybe("dt_bias", dt_bias, _F32, (C,), index)), op)


def _ssm_state(state, C, N, index):
    ptr, shape = _want("state", state, _F32, None, index), state.shape
    if len(shape) != 3 or shape[1] != C or shape[2] != N:
        raise ValueError(f"state must be [num_slots, {C}, {N}], got {tuple(shape)}")
    return ptr, _count("state", shape[0])


def kda_ssm_prompt(*, x, dt, a, b, c, seq_starts, output, d=None, z=None, dt_bias=None,
                   softplus: bool = True, state=None, src_slots=None, dst_slots=None,
                   max_seq: Optional[int] = None, err=None, path: int = 0, workspace=None,
                   stream: Optional[torch.cuda.Stream] = None) -> None:
    """Selective state-space scan over ragged prompts (include/kda.h
    ``kda_ssm_prompt``).

    ``x``, ``dt``, ``z``, ``output`` bf16 [tokens, channels], ``b``, ``c`` bf16
    [tokens, groups * states] (each may be a slice of wider rows); ``a`` f32
    [channels, states], the decays' rate (below 0); ``d``, ``dt_bias`` f32
    [channels]; ``seq_starts`` i32 [seqs + 1]; ``state`` f32 [num_slots, channels,
    states] with ``src_slots`` (the states the sequences start from) and
    ``dst_slots`` (where their last states go), i32 [seqs] each or None.
    ``max_seq``: no sequence is longer (default: ``tokens``; the tighter, the better
    the work is laid out).  ``workspace``: a CUDA uint8 tensor of at least
    ``lib.ssm_workspace`` bytes; by default allocated for the call, on the stream it
    runs on."""
    if workspace is None and _done((_lib._bind or _lib.bind()).ssm_prompt(
            x, dt, a, b, c, seq_starts, output, d, z, dt_bias, bool(softplus), state, src_slots,
            dst_slots, max_seq, err, path, stream)):
        return
    index, rows, C, N, G, strides, ptrs, op = _ssm_rows(x, dt, a, b, c, d, z, dt_bias, output)
    B, sp, src, dst = _sequences(seq_starts, src_slots, dst_slots, index)
    if state is None:
        if src_slots is not None or dst_slots is not None:
            raise ValueError("state is required with src_slots or dst_slots")
        state_p, num_slots = None, 0
    else:
        state_p, num_slots = _ssm_state(state, C, N, index)
    args = _lib.KdaSsmPromptArgs(
        B, C, N, G, rows, _most(max_seq, rows), num_slots,
        int(bool(softplus)), _path(int(path)), *strides, *ptrs, sp, src, dst, state_p, op,
        _maybe("err", err, torch.int32, None, index))
    if workspace is not None:
        args.workspace = _want("workspace", workspace, torch.uint8, None, index)
        args.workspace_bytes = workspace.numel()
    elif (need := _lib.ssm_workspace(args)) > 0:
        # from the pool of the stream that uses it: freed behind its kernels
        with torch.cuda.device(index), torch.cuda.stream(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        args.workspace, args.workspace_bytes = workspace.data_ptr(), need
    _run("kda_ssm_prompt", args, index, stream)


class KdaSsmStep:
    """A prepared single-token step of the selective scan (include/kda.h
    ``kda_ssm_step``) over fixed device tensors.

    Rows ``x``, ``dt``, ``z``, ``output`` bf16 [batch, channels], ``b``, ``c`` bf16
    [batch, groups * states]; ``a``, ``d``, ``dt_bias`` as in ``kda_ssm_prompt``;
    ``slots`` i32 [batch] (<= 0: padding); ``state`` f32 [num_slots, channels,
    states], updated in place.  Validates once and launches with
    ``__call__(stream)``; the tensors' contents may change between calls, their
    storage may not."""

    def __init__(self, *, x, dt, a, b, c, slots, state, output, d=None, z=None, dt_bias=None,
                 softplus: bool = True, err=None):
        self.index, rows, C, N, G, strides, ptrs, op = _ssm_rows(x, dt, a, b, c, d, z, dt_bias,
                                                                 output)
        state_p, num_slots = _ssm_state(state, C, N, self.index)
        self.args = _lib.KdaSsmStepArgs(
            rows, C, N, G, num_slots, int(bool(softplus)), *strides, *ptrs,
            _want("slots", slots, torch.int32, (rows,), self.index), state_p, op,
            _maybe("err", err, torch.int32, None, self.index))
        # keep the tensors alive as long as the prepared step
        self._keep = (x, dt, a, b, c, slots, state, output, d, z, dt_bias, err)

    def __call__(self, stream: Optional[torch.cuda.Stream] = None) -> None:
        _run("kda_ssm_step", self.args, self.index, stream)


def kda_ssm_step(stream: Optional[torch.cuda.Stream] = None, **kw) -> None:
    """One single-token step of the scan on ``stream``; see ``KdaSsmStep``."""
    KdaSsmStep(**kw)(stream)


# --------------------------------------------------------------------- projections

ACTIVATIONS = {None: 0, "none": 0, "silu": 1, "gelu": 2, "softplus": 3}


def kda_linear(*, x, weight, output, bias=None, residual=None, activation: Optional[str] = None,
               err=None, path: int = 0, stream: Optional[torch.cuda.Stream] = None) -> None:
    """output = act(x weight^T + bias) + residual (include/kda.h ``kda_linear``).

    ``x`` bf16 [rows, inner], ``weight`` bf16 [outer, inner], ``residual`` and
    ``output`` bf16 [rows, outer] (each may be a slice of wider rows; the residual may
    be the output itself); ``bias`` bf16 [outer]; ``activation`` None, "none",
    "silu", "gelu" (with erf) or "softplus".  ``path``: 0 = automatic, 1 = the form for few
    tiles, 2 = the form for many (``kda_linear_path``).  ``err`` takes
    ``lib.KDA_DEVERR_TIMEOUT`` where a wait on the chip ran out and the output is
    incomplete, which nothing else tells."""
    act = ACTIVATIONS.get(activation)
    if act is not None and path == 0 and _done((_lib._bind or _lib.bind()).linear(
            x, weight, output, bias, residual, act, err, stream)):
        return
    index = _cuda_index("x", x)
    _cuda_index("weight", weight)
    if x.ndim != 2 or weight.ndim != 2:
        raise ValueError("x must be [rows, inner], weight [outer, inner]")
    if act is None:
        raise ValueError(f"activation must be one of {sorted(map(str, ACTIVATIONS))}, "
                         f"got {activation!r}")
    (rows, K), N = x.shape, weight.shape[0]
    if (rows | K | N) >> 31:
        _counts(x=rows, inner=K, weight=N)
    (xp, xs), (wp, ws) = _rows("x", x, rows, K, index), _rows("weight", weight, N, K, index)
    op, os_ = _rows("output", output, rows, N, index)
    rp, rs = (None, 0) if residual is None else _rows("residual", residual, rows, N, index)
    _run("kda_linear_path", _lib.KdaLinearArgs(
        rows, K, N, act, xs, ws, rs, os_, xp, wp,
        None if bias is None else _want("bias", bias, _BF16, (N,), index), rp, op,
        None if err is None else _want("err", err, _I32, None, index)), index, stream, _path(path))

"""Host side of the linear-attention and snapshot calls, without a GPU: every
refusal of the C ABI, the workspace's size, the structs' mirrors, and the
64-bit references themselves (tests/linref.py) on small cases."""
from __future__ import annotations

import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

from linear_attention_recurrent_kda_gb300 import api
from linear_attention_recurrent_kda_gb300 import lib as kl
from tests import linref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20
STRUCTS = [("kda_lin_prompt_args", kl.KdaLinPromptArgs),
           ("kda_lin_step_args", kl.KdaLinStepArgs),
           ("kda_snapshot_args", kl.KdaSnapshotArgs)]


def fill(a, names, kw):
    for n in names:
        setattr(a, n, FAKE)
    for n, v in kw.items():
        setattr(a, n, v)
    return a


def prompt_args(**kw):
    a = kl.KdaLinPromptArgs()
    a.seqs, a.heads, a.qk_heads, a.tokens, a.max_seq, a.num_slots = 2, 4, 2, 300, 200, 5
    a.q_stride = a.k_stride = 256
    a.v_stride = a.o_stride = 512
    return fill(a, ("q", "k", "v", "decay", "seq_starts", "src_slots", "dst_slots", "state",
                    "output"), kw)


def step_args(**kw):
    a = kl.KdaLinStepArgs()
    a.batch, a.heads, a.qk_heads, a.num_slots = 2, 4, 2, 5
    a.q_stride = a.k_stride = 256
    a.v_stride = a.o_stride = 512
    return fill(a, ("q", "k", "v", "decay", "slots", "state", "output"), kw)


def snap_args(**kw):
    a = kl.KdaSnapshotArgs()
    a.count, a.heads, a.num_slots, a.num_snaps, a.bits = 2, 4, 5, 5, 8
    return fill(a, ("slots", "snaps", "state", "codes", "scales"), kw)


ROWS = [
    (dict(heads=-1), kl.KDA_ERR_SHAPE),
    (dict(qk_heads=0), kl.KDA_ERR_SHAPE),
    (dict(qk_heads=3), kl.KDA_ERR_SHAPE),
    (dict(decay_rows=2), kl.KDA_ERR_SHAPE),
    (dict(q_stride=248), kl.KDA_ERR_SHAPE),
    (dict(k_stride=260), kl.KDA_ERR_SHAPE),
    (dict(v_stride=504), kl.KDA_ERR_SHAPE),
    (dict(o_stride=-512), kl.KDA_ERR_SHAPE),
    (dict(v_stride=1 << 38), kl.KDA_ERR_SHAPE),
    (dict(heads=0), kl.KDA_SUCCESS),
    (dict(q=None), kl.KDA_ERR_NULL_POINTER),
    (dict(k=None), kl.KDA_ERR_NULL_POINTER),
    (dict(v=None), kl.KDA_ERR_NULL_POINTER),
    (dict(decay=None), kl.KDA_ERR_NULL_POINTER),
    (dict(output=None), kl.KDA_ERR_NULL_POINTER),
    (dict(state=None), kl.KDA_ERR_NULL_POINTER),
    (dict(q=FAKE + 8), kl.KDA_ERR_ALIGNMENT),
    (dict(v=FAKE + 2), kl.KDA_ERR_ALIGNMENT),
    (dict(state=FAKE + 4), kl.KDA_ERR_ALIGNMENT),
    (dict(decay=FAKE + 2), kl.KDA_ERR_ALIGNMENT),
    (dict(err=FAKE + 1), kl.KDA_ERR_ALIGNMENT),
]


@pytest.mark.parametrize("kw,code", ROWS + [
    (dict(seqs=-1), kl.KDA_ERR_SHAPE),
    (dict(tokens=-1), kl.KDA_ERR_SHAPE),
    (dict(max_seq=-1), kl.KDA_ERR_SHAPE),
    (dict(num_slots=0), kl.KDA_ERR_SHAPE),
    (dict(seqs=1 << 30), kl.KDA_ERR_SHAPE),
    (dict(path=3), kl.KDA_ERR_PATH),
    (dict(path=-1), kl.KDA_ERR_PATH),
    (dict(seqs=0), kl.KDA_SUCCESS),
    (dict(seq_starts=None), kl.KDA_ERR_NULL_POINTER),
    (dict(seq_starts=FAKE + 2), kl.KDA_ERR_ALIGNMENT),
    (dict(src_slots=FAKE + 2), kl.KDA_ERR_ALIGNMENT),
    (dict(dst_slots=FAKE + 2), kl.KDA_ERR_ALIGNMENT),
])
def test_prompt_refusals(kw, code):
    assert kl.call("kda_lin_prompt", prompt_args(**kw), 0) == code
    assert kl.load().kda_lin_prompt(None, None) == kl.KDA_ERR_NULL_ARGS


@pytest.mark.parametrize("kw,code", ROWS + [
    (dict(batch=-1), kl.KDA_ERR_SHAPE),
    (dict(batch=1 << 30), kl.KDA_ERR_SHAPE),
    (dict(num_slots=0), kl.KDA_ERR_SHAPE),
    (dict(batch=0), kl.KDA_SUCCESS),
    (dict(slots=None), kl.KDA_ERR_NULL_POINTER),
    (dict(slots=FAKE + 2), kl.KDA_ERR_ALIGNMENT),
])
def test_step_refusals(kw, code):
    assert kl.call("kda_lin_step", step_args(**kw), 0) == code
    assert kl.load().kda_lin_step(None, None) == kl.KDA_ERR_NULL_ARGS


@pytest.mark.parametrize("entry", ["kda_snapshot_save", "kda_snapshot_load"])
@pytest.mark.parametrize("kw,code", [
    (dict(count=-1), kl.KDA_ERR_SHAPE),
    (dict(heads=-1), kl.KDA_ERR_SHAPE),
    (dict(num_slots=0), kl.KDA_ERR_SHAPE),
    (dict(num_snaps=0), kl.KDA_ERR_SHAPE),
    (dict(bits=5), kl.KDA_ERR_SHAPE),
    (dict(count=1 << 30), kl.KDA_ERR_SHAPE),
    (dict(count=0), kl.KDA_SUCCESS),
    (dict(heads=0), kl.KDA_SUCCESS),
    (dict(slots=None), kl.KDA_ERR_NULL_POINTER),
    (dict(snaps=None), kl.KDA_ERR_NULL_POINTER),
    (dict(state=None), kl.KDA_ERR_NULL_POINTER),
    (dict(codes=None), kl.KDA_ERR_NULL_POINTER),
    (dict(scales=None), kl.KDA_ERR_NULL_POINTER),
    (dict(state=FAKE + 8), kl.KDA_ERR_ALIGNMENT),
    (dict(codes=FAKE + 4), kl.KDA_ERR_ALIGNMENT),
    (dict(scales=FAKE + 4), kl.KDA_ERR_ALIGNMENT),
    (dict(slots=FAKE + 2), kl.KDA_ERR_ALIGNMENT),
    (dict(err=FAKE + 2), kl.KDA_ERR_ALIGNMENT),
])
def test_snapshot_refusals(entry, kw, code):
    assert kl.call(entry, snap_args(**kw), 0) == code
    assert getattr(kl.load(), entry)(None, None) == kl.KDA_ERR_NULL_ARGS


def test_new_codes_have_texts():
    assert "workspace" in kl.strerror(kl.KDA_ERR_WORKSPACE)


def test_cpu_tensors_are_refused():
    x = torch.zeros(3, 128, dtype=torch.bfloat16)
    kw = dict(q=x, k=x, v=x, output=x, decay=torch.zeros(1), scale=1.0)
    with pytest.raises(ValueError, match="CUDA"):
        api.kda_lin_prompt(**kw, seq_starts=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        api.kda_lin_step(**kw, slots=torch.ones(3, dtype=torch.int32),
                         state=torch.zeros(2, 1, 128, 128))
    snap = dict(state=torch.zeros(2, 1, 128, 128), slots=torch.ones(1, dtype=torch.int32),
                snaps=torch.ones(1, dtype=torch.int32), scales=torch.zeros(2, 1, 128),
                codes=torch.zeros(2, 1, 128, 128, dtype=torch.int8))
    for f in (api.kda_snapshot_save, api.kda_snapshot_load):
        with pytest.raises(ValueError, match="CUDA"):
            f(**snap)


KINDS = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "float": ctypes.c_float}


def header_fields(name):
    text = open(os.path.join(ROOT, "include", "kda.h")).read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    m = re.search(r"typedef\s+struct\s+%s\s*\{(.*?)\}" % name, text, flags=re.S)
    out = []
    for decl in filter(None, (" ".join(d.split()) for d in m.group(1).split(";"))):
        base = re.match(r"(?:const\s+)?(\w+)", decl)
        for d in decl[base.end():].split(","):
            ptr = "*" in d
            out.append((d.replace("*", "").strip(), ctypes.c_void_p if ptr else
                        KINDS[base.group(1)]))
    return out


@pytest.mark.parametrize("name,cls", STRUCTS, ids=[s[0] for s in STRUCTS])
def test_mirrors_match_the_header(name, cls):
    assert [(n, t) for n, t in cls._fields_] == header_fields(name)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_offsets_match_the_c_compiler(tmp_path):
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "kda.h"', "int main(void) {"]
    for name, cls in STRUCTS:
        lines.append(f'  printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'  printf("{name} {f} %zu\\n", offsetof({name}, {f}));'
                  for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True, capture_output=True)
    got = {}
    for line in subprocess.run([str(exe)], check=True, capture_output=True,
                               text=True).stdout.splitlines():
        a, b, n = line.split()
        got[a, b] = int(n)
    for name, cls in STRUCTS:
        assert got[name, "size"] == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert got[name, f] == getattr(cls, f).offset, (name, f)


# --------------------------------------------------------- the references themselves

def test_recurrence_reference_is_the_masked_product():
    """o = (Q K^T o decays, lower triangle) V + decayed S0 q, for one sequence."""
    g = torch.Generator().manual_seed(1)
    n, H = 9, 2
    q, k, v = (torch.randn(n, H * 128, generator=g) for _ in range(3))
    decay = -torch.rand(n, H, generator=g)
    S0 = torch.randn(2, H, 128, 128, generator=g)
    out, mag, S, M = linref.prompt(q, k, v, decay, [0, n], 0.5, S0, [1])
    b = decay.double().cumsum(0)
    for h in range(H):
        sl = slice(128 * h, 128 * h + 128)
        w = torch.exp(b[:, None, h] - b[None, :, h]).tril()
        a = q[:, sl].double() @ k[:, sl].double().T * w
        o = a @ v[:, sl].double() + torch.exp(b[:, h:h + 1]) * (q[:, sl].double()
                                                                @ S0[1, h].double().T)
        assert torch.allclose(out[:, sl], 0.5 * o, rtol=1e-12, atol=1e-12)
    assert torch.all(mag >= out.abs()) and torch.all(M >= S.abs())


def test_quantiser_reference():
    x = np.zeros((1, 128), np.float32)
    x[0, :5] = [127.0, 0.5, 1.5, -2.5, 63.49]
    c, s = linref.quantise(x, 8)
    assert s[0, 0] == 1.0 and c[0, :5].tolist() == [127, 0, 2, -2, 63]
    c, s = linref.quantise(x, 4)
    assert s.shape == (1, 4) and s[0, 0] == np.float32(127 / 7) and c[0, 0] == 7
    packed = linref.pack(c, 4)
    low = packed.astype(np.int8) << 4 >> 4
    high = packed.astype(np.int8) >> 4
    assert np.array_equal(np.stack([low, high], -1).reshape(1, 128), c)
    rng = np.random.default_rng(0)
    x = rng.standard_normal((4, 128)).astype(np.float32)
    for bits, top in ((8, 127), (4, 7)):
        c, s = linref.quantise(x, bits)
        off = np.abs(linref.dequantise(c, s) - x).reshape(4, s.shape[-1], -1)
        assert np.all(off <= s[..., None] * (0.5 + 1e-6)) and np.abs(c).max() == top


def test_workspace_sizes():
    """None for whole sequences, some for split ones (pages of the segments and
    their decays), none for refused sizes; a missing or short one is refused."""
    assert kl.load().kda_lin_prompt_workspace(None) == -1
    assert kl.prompt_workspace(prompt_args()) == 0
    assert kl.prompt_workspace(prompt_args(heads=-1)) == 0
    split = dict(seqs=1, tokens=20000, max_seq=20000)
    need = kl.prompt_workspace(prompt_args(**split))
    assert need > 0 and need % ((128 * 128 + 1) * 4 * 4) == 0
    assert kl.prompt_workspace(prompt_args(path=1, **split)) == 0
    assert kl.prompt_workspace(prompt_args(**dict(split, max_seq=200))) == 0
    for kw in (dict(), dict(workspace=FAKE, workspace_bytes=need - 1),
               dict(workspace=FAKE + 128, workspace_bytes=need)):
        assert kl.call("kda_lin_prompt", prompt_args(**split, **kw), 0) == kl.KDA_ERR_WORKSPACE

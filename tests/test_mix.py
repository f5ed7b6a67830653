"""Host side of the convolution, scan and product calls, without a GPU: every refusal
of the C ABI, the structs' mirrors, the binding's checks, and the 64-bit references
(tests/mixref.py) on small cases."""
from __future__ import annotations

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from linear_attention_recurrent_kda_gb300 import api
from linear_attention_recurrent_kda_gb300 import lib as kl
from tests import mixref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20
STRUCTS = [("kda_conv_prompt_args", kl.KdaConvPromptArgs), ("kda_conv_step_args", kl.KdaConvStepArgs),
           ("kda_ssm_prompt_args", kl.KdaSsmPromptArgs), ("kda_ssm_step_args", kl.KdaSsmStepArgs),
           ("kda_linear_args", kl.KdaLinearArgs)]


def fill(cls, kw, pointers, **sizes):
    a = cls()
    for n in pointers:
        setattr(a, n, FAKE)
    for n, v in {**sizes, **kw}.items():
        setattr(a, n, v)
    return a


def conv_prompt(**kw):
    return fill(kl.KdaConvPromptArgs, kw,
                ("x", "weight", "bias", "seq_starts", "src_slots", "dst_slots", "window", "output"),
                seqs=2, channels=96, parts=3, taps=4, tokens=9, num_slots=5, width=3, x_stride=96,
                o_stride=104)


def conv_step(**kw):
    return fill(kl.KdaConvStepArgs, kw, ("x", "weight", "bias", "slots", "window", "output"),
                batch=2, channels=96, parts=3, taps=4, num_slots=5, width=3, x_stride=96, o_stride=104)


SSM = dict(channels=96, states=16, groups=2, num_slots=5, x_stride=96, dt_stride=96, b_stride=32,
           c_stride=40, z_stride=96, o_stride=96)
SSM_ROWS = ("x", "dt", "a", "b", "c", "d", "z", "dt_bias", "state", "output")


def ssm_prompt(**kw):
    return fill(kl.KdaSsmPromptArgs, kw, SSM_ROWS + ("seq_starts", "src_slots", "dst_slots"),
                seqs=2, tokens=9, max_seq=9, **SSM)


def ssm_step(**kw):
    return fill(kl.KdaSsmStepArgs, kw, SSM_ROWS + ("slots",), batch=2, **SSM)


def linear(**kw):
    return fill(kl.KdaLinearArgs, kw, ("x", "weight", "bias", "residual", "output"), rows=5, inner=72,
                outer=33, x_stride=72, w_stride=80, r_stride=40, o_stride=48)


S, P, A = kl.KDA_ERR_SHAPE, kl.KDA_ERR_NULL_POINTER, kl.KDA_ERR_ALIGNMENT
CONV = [(dict(channels=-8), S), (dict(parts=0), S), (dict(parts=5), S), (dict(channels=100), S),
        (dict(taps=1), S), (dict(taps=5), S), (dict(x_stride=88), S), (dict(x_stride=100), S),
        (dict(o_stride=1 << 38), S), (dict(width=2), kl.KDA_ERR_CONV_WIDTH), (dict(weight=None), P),
        (dict(x=None), P), (dict(output=None), P), (dict(window=None), P), (dict(x=FAKE + 8), A),
        (dict(weight=FAKE + 2), A), (dict(bias=FAKE + 2), A), (dict(window=FAKE + 4), A),
        (dict(output=FAKE + 2), A), (dict(err=FAKE + 2), A), (dict(channels=0), 0)]
SCAN = [(dict(channels=-16), S), (dict(groups=0), S), (dict(groups=5), S), (dict(channels=104), S),
        (dict(states=8), S), (dict(states=17), S), (dict(states=128), S), (dict(x_stride=88), S),
        (dict(dt_stride=97), S), (dict(b_stride=24), S), (dict(c_stride=36), S), (dict(z_stride=0), S),
        (dict(o_stride=-96), S), (dict(a=None), P), (dict(x=None), P), (dict(dt=None), P),
        (dict(b=None), P), (dict(c=None), P), (dict(state=None), P), (dict(output=None), P),
        (dict(x=FAKE + 2), A), (dict(dt=FAKE + 2), A), (dict(a=FAKE + 4), A), (dict(b=FAKE + 8), A),
        (dict(c=FAKE + 8), A), (dict(z=FAKE + 2), A), (dict(state=FAKE + 4), A), (dict(d=FAKE + 2), A),
        (dict(dt_bias=FAKE + 1), A), (dict(output=FAKE + 2), A), (dict(channels=0), 0)]
CALLS = [("kda_conv_prompt", conv_prompt, CONV + [
            (dict(seqs=-1), S), (dict(tokens=-1), S), (dict(num_slots=0), S), (dict(seq_starts=None), P),
            (dict(tokens=2 ** 31 - 255), S), (dict(src_slots=FAKE + 2), A), (dict(dst_slots=FAKE + 2), A), (dict(seq_starts=FAKE + 1), A),
            (dict(seqs=0), 0)]),
         ("kda_conv_step", conv_step, CONV + [
            (dict(batch=-1), S), (dict(num_slots=0), S), (dict(slots=None), P), (dict(slots=FAKE + 2), A),
            (dict(batch=0), 0)]),
         ("kda_ssm_prompt", ssm_prompt, SCAN + [
            (dict(seqs=-1), S), (dict(tokens=-1), S), (dict(tokens=2 ** 31 - 1), S), (dict(max_seq=-1), S), (dict(num_slots=0), S),
            (dict(path=3), kl.KDA_ERR_PATH), (dict(path=-1), kl.KDA_ERR_PATH),
            (dict(seq_starts=None), P), (dict(seq_starts=FAKE + 2), A), (dict(src_slots=FAKE + 1), A),
            (dict(dst_slots=FAKE + 2), A), (dict(seqs=0), 0)]),
         ("kda_ssm_step", ssm_step, SCAN + [
            (dict(batch=-1), S), (dict(num_slots=0), S), (dict(slots=None), P), (dict(slots=FAKE + 2), A),
            (dict(batch=0), 0)]),
         ("kda_linear", linear, [
            (dict(rows=-1), S), (dict(inner=0), S), (dict(outer=-1), S), (dict(rows=2 ** 31 - 1), S),
            (dict(outer=2 ** 31 - 200, r_stride=1 << 32, o_stride=1 << 32), S), (dict(x_stride=64), S),
            (dict(w_stride=73), S), (dict(r_stride=32), S), (dict(o_stride=36), S),
            (dict(activation=-1), kl.KDA_ERR_ACTIVATION), (dict(activation=4), kl.KDA_ERR_ACTIVATION),
            (dict(x=None), P), (dict(weight=None), P), (dict(output=None), P), (dict(x=FAKE + 8), A),
            (dict(weight=FAKE + 2), A), (dict(bias=FAKE + 2), A), (dict(residual=FAKE + 2), A),
            (dict(output=FAKE + 4), A), (dict(err=FAKE + 2), A), (dict(rows=0), 0), (dict(outer=0), 0)])]


@pytest.mark.parametrize("entry,make,kw,code", [(e, m, kw, code) for e, m, rows in CALLS
                                                for kw, code in rows])
def test_refusals(entry, make, kw, code):
    """Nothing of these is launched: the addresses are none."""
    assert getattr(kl.load(), entry)(make(**kw), None) == code


@pytest.mark.parametrize("entry", [e for e, _, _ in CALLS])
def test_null_args(entry):
    assert getattr(kl.load(), entry)(None, None) == kl.KDA_ERR_NULL_ARGS


def test_workspace_of_refused_and_missing_arguments():
    assert kl.load().kda_ssm_prompt_workspace(None) == -1
    assert kl.ssm_workspace(ssm_prompt(states=17)) == 0
    assert kl.ssm_workspace(ssm_prompt(path=1)) == 0
    assert kl.ssm_workspace(ssm_prompt(channels=0, tokens=4096, max_seq=4096)) == 0
    assert kl.ssm_workspace(ssm_prompt(seqs=0, tokens=4096, max_seq=4096, path=2)) >= 0
    most = ssm_prompt(seqs=(1 << 31) - 2, channels=8, tokens=1 << 20, max_seq=1 << 20, path=2)
    assert kl.ssm_workspace(most) >= 0


def test_error_text():
    assert "activation" in kl.strerror(kl.KDA_ERR_ACTIVATION)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_mirrors_match_the_header(tmp_path):
    text = re.sub(r"/\*.*?\*/", " ", open(os.path.join(ROOT, "include", "kda.h")).read(), flags=re.S)
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "kda.h"', "int main(void) {"]
    for name, cls in STRUCTS:
        body = re.search(r"typedef\s+struct\s+%s\s*\{(.*?)\}" % name, text, flags=re.S).group(1)
        fields = re.findall(r"\**\s*(\w+)\s*(?=[,;])", body)
        assert fields == [n for n, _ in cls._fields_], name
        lines.append(f'  printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'  printf("{name}.{n} %zu\\n", offsetof({name}, {n}));' for n in fields]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(line.split() for line in
               subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    for name, cls in STRUCTS:
        assert int(got[name]) == ctypes.sizeof(cls)
        for n, _ in cls._fields_:
            assert int(got[f"{name}.{n}"]) == getattr(cls, n).offset, (name, n)


BF = torch.bfloat16


@pytest.mark.parametrize("call", [
    lambda t: api.kda_conv_prompt(x=t, weight=t, seq_starts=t, output=t),
    lambda t: api.KdaConvStep(x=t, weight=t, slots=t, window=t, output=t),
    lambda t: api.kda_ssm_prompt(x=t, dt=t, a=t, b=t, c=t, seq_starts=t, output=t),
    lambda t: api.KdaSsmStep(x=t, dt=t, a=t, b=t, c=t, slots=t, state=t, output=t),
    lambda t: api.kda_linear(x=t, weight=t, output=t)])
def test_the_binding_takes_cuda_tensors_only(call):
    with pytest.raises(ValueError, match="CUDA"):
        call(torch.zeros(4, 8, dtype=BF))
    with pytest.raises(TypeError):
        call(None)


def test_reference_conv_against_a_library_convolution():
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(7, 24, generator=g).to(BF), torch.randn(3, 24, generator=g).to(BF)
    bias, pool = torch.randn(24, generator=g).to(BF), torch.randn(3, 24, 4, generator=g)
    out, _, last = mixref.conv(x, w, [0, 5, 5, 6], bias, pool, [2, 1, 0])
    full = torch.cat([pool[2, :, :2].double(), x[:5].double().T], 1)
    want = torch.nn.functional.conv1d(full[None], w.double().T[:, None], bias.double(), groups=24)[0].T
    assert torch.allclose(out[:5], torch.nn.functional.silu(want), rtol=1e-12, atol=1e-12)
    assert torch.equal(last[0], full[:, -2:]) and torch.equal(last[1], pool[1, :, :2].double())
    assert torch.equal(last[2], torch.stack([torch.zeros(24).double(), x[5].double()], 1))
    assert torch.isnan(out[6]).all()
    parts = w.view(3, 3, 8).transpose(0, 1).contiguous()
    assert torch.equal(mixref.conv(x, parts, [0, 5, 5, 6], bias, pool, [2, 1, 0])[0][:6], out[:6])


def test_reference_scan_in_closed_form():
    """One channel group, constant inputs: h after T tokens is a geometric sum."""
    T, C, N = 6, 8, 16
    x, dt = torch.full((T, C), 0.5, dtype=BF), torch.full((T, C), 0.25, dtype=BF)
    a = -torch.arange(1.0, N + 1).expand(C, N)
    b, c = torch.full((T, N), 2.0, dtype=BF), torch.ones(T, N, dtype=BF)
    out, _, h, _ = mixref.ssm(x, dt, a, b, c, [0, T], soft=False)
    f = torch.exp(0.25 * a.double())
    want = 0.25 * 0.5 * 2.0 * (1 - f ** T) / (1 - f)
    assert torch.allclose(h[0], want, rtol=1e-12)
    assert torch.allclose(out[-1], want.sum(-1), rtol=1e-12)


def test_reference_product_against_the_library():
    g = torch.Generator().manual_seed(2)
    x, w, b = (torch.randn(*s, generator=g).to(BF) for s in ((5, 16), (7, 16), (7,)))
    y = torch.nn.functional.linear(x.double(), w.double(), b.double())
    for act, f in ((None, lambda v: v), ("silu", torch.nn.functional.silu),
                   ("gelu", torch.nn.functional.gelu), ("softplus", torch.nn.functional.softplus)):
        assert torch.allclose(mixref.linear(x, w, b, act=act)[0], f(y), rtol=1e-12, atol=1e-14)


def test_the_short_way_leaves_what_it_does_not_take():
    """The extension module returns None for what the general checks have to answer, and
    they do."""
    bind = kl.bind()
    x, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(8, 8, dtype=torch.bfloat16)
    assert bind.linear(x, w, x, None, None, 0, None, None) is None           # no CUDA tensors
    assert bind.linear(None, w, x, None, None, 0, None, None) is None
    assert bind.linear(3, "w", [], None, None, 0, None, None) is None
    assert bind.conv_prompt(*[x] * 8, True, None, None) is None
    assert bind.conv_prompt(*[None] * 11) is None
    assert bind.ssm_prompt(*[x] * 14, None, None, 0, None) is None
    assert bind.ssm_prompt(*[None] * 18) is None
    for fn, n in ((bind.linear, 7), (bind.conv_prompt, 0), (bind.ssm_prompt, 19), (bind.setup, 3)):
        with pytest.raises(TypeError):
            fn(*[None] * n)
    with pytest.raises(ValueError, match="CUDA"):
        api.kda_linear(x=x, weight=w, output=x)
    with pytest.raises(TypeError):
        api.kda_linear(x=None, weight=w, output=x)

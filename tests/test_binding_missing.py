"""The library without its binding (the short way from Python): it is built and used all the
same, and says so once.  On the CPU."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from linear_attention_recurrent_kda_gb300 import api
from linear_attention_recurrent_kda_gb300 import build as kbuild
from linear_attention_recurrent_kda_gb300 import lib as kl

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A library of one source and a binding, both to be built in tmp_path."""
    (tmp_path / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(kbuild, "LIBS", ((str(tmp_path / "one.so"), [str(tmp_path / "one.cu")]),))
    monkeypatch.setattr(kbuild, "BIND_PATH", str(tmp_path / "bind.so"))
    return tmp_path


@pytest.mark.parametrize("command", [["g++", "/no/such/source.cpp"], ["/no/such/compiler"], None])
def test_the_libraries_are_built_where_the_binding_is_not(small, monkeypatch, command):
    def made(out):
        if command is None:
            raise RuntimeError("no headers")
        return command
    monkeypatch.setattr(kbuild, "_bind_command", made)
    with pytest.warns(RuntimeWarning, match="general"):
        kbuild.build()
    assert (small / "one.so").exists() and not (small / "bind.so").exists()


def test_each_build_has_files_of_its_own_until_they_are_whole(small, monkeypatch):
    names, replace = [], os.replace

    def noted(src, dst):
        assert os.path.dirname(src) == os.path.dirname(dst)
        names.append(src)
        replace(src, dst)
    monkeypatch.setattr(kbuild, "_bind_command", lambda out: ["cp", str(small / "one.cu"), out])
    monkeypatch.setattr(kbuild.os, "replace", noted)
    kbuild.build(force=True)
    kbuild.build(force=True)
    assert len(names) == len(set(names)) == 4
    assert sorted(os.listdir(small)) == ["bind.so", "one.cu", "one.so"]


@pytest.mark.parametrize("path", [None, "missing", "broken"])
def test_calls_take_the_general_way(tmp_path, monkeypatch, path):
    if path is not None:
        path = str(tmp_path / (path + ".so"))
        if "broken" in path:
            open(path, "w").write("no module")
    monkeypatch.setattr(kbuild, "BIND_PATH", path)
    monkeypatch.setattr(kbuild, "build", lambda *a, **k: None)
    monkeypatch.setattr(kl, "_bind", None)
    x = torch.zeros(8, 8, dtype=torch.bfloat16)
    with pytest.warns(RuntimeWarning, match="general"):
        with pytest.raises(ValueError, match="CUDA"):
            api.kda_linear(x=x, weight=x, output=x)
    for call in (lambda: api.kda_linear(x=x, weight=x, output=x),       # no second warning
                 lambda: api.kda_conv_prompt(x=x, weight=x, seq_starts=x, output=x),
                 lambda: api.kda_ssm_prompt(x=x, dt=x, a=x, b=x, c=x, seq_starts=x, output=x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_without_a_version_of_torch():
    code = ("import importlib.metadata as m\n"
            "def version(name): raise m.PackageNotFoundError(name)\n"
            "m.version = version\n"
            "from linear_attention_recurrent_kda_gb300 import build, lib\n"
            "assert build.BIND_PATH is None\n"
            "lib.load()\n"
            "import warnings\n"
            "with warnings.catch_warnings(record=True) as seen:\n"
            "    warnings.simplefilter('always')\n"
            "    assert lib.bind().linear(1, 2) is None\n"
            "assert len(seen) == 1\n")
    res = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr

"""The product in a form of the caller's choice, without a GPU: what is refused."""
from __future__ import annotations

import pytest

from linear_attention_recurrent_kda_gb300 import api
from linear_attention_recurrent_kda_gb300 import lib as kl
from tests.test_mix import FAKE, linear


@pytest.mark.parametrize("path,kw,code", [
    (-1, {}, kl.KDA_ERR_PATH), (3, {}, kl.KDA_ERR_PATH), (3, dict(rows=0), kl.KDA_ERR_PATH),
    (2, dict(outer=7), kl.KDA_ERR_SHAPE), (2, dict(rows=0), 0), (1, dict(outer=0), 0), (2, dict(outer=0), 0),
    (1, dict(inner=0), kl.KDA_ERR_SHAPE), (2, dict(x=None), kl.KDA_ERR_NULL_POINTER),
    (1, dict(activation=4), kl.KDA_ERR_ACTIVATION), (2, dict(x=FAKE + 8), kl.KDA_ERR_ALIGNMENT)])
def test_refusals(path, kw, code):
    assert kl.call("kda_linear_path", linear(**kw), None, path) == code


def test_null_args():
    assert kl.call("kda_linear_path", None, None, 1) == kl.KDA_ERR_NULL_ARGS


def test_paths_that_32_bits_do_not_hold():
    assert [api._path(p) for p in (0, 1, 2, 7, -3, 1 << 32, (1 << 32) + 2)] == [0, 1, 2, 7, -1, -1, -1]

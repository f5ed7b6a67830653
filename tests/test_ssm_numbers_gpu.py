"""Forms and lengths whose low 32 bits would be others are refused, not taken for those."""
from __future__ import annotations

import pytest
import torch

from linear_attention_recurrent_kda_gb300 import lib as kl
from linear_attention_recurrent_kda_gb300.api import kda_lin_prompt, kda_ssm_prompt
from tests.test_ssm_gpu import i32, make

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("workspace", [False, True])      # the short way from Python, or the general one
@pytest.mark.parametrize("kw,code", [
    (dict(path=1 << 32), kl.KDA_ERR_PATH), (dict(path=(1 << 32) + 2), kl.KDA_ERR_PATH),
    (dict(path=1 - (1 << 32)), kl.KDA_ERR_PATH), (dict(max_seq=9 - (1 << 32)), kl.KDA_ERR_SHAPE),
    (dict(max_seq=-1), kl.KDA_ERR_SHAPE)])
def test_numbers_beyond_32_bits(kw, code, workspace):
    T, C = 9, 16
    d, _ = make(T, C)
    out = torch.zeros(T, C, dtype=BF, device="cuda")
    if workspace:
        kw = dict(kw, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(kl.KdaError) as e:
        kda_ssm_prompt(**d, seq_starts=i32([0, T]), output=out, **kw)
    assert e.value.code == code
    kw.pop("workspace", None)
    x, decay = torch.zeros(T, 128, dtype=BF, device="cuda"), torch.zeros(1, device="cuda")
    with pytest.raises(kl.KdaError) as e:
        kda_lin_prompt(q=x, k=x, v=x, decay=decay, seq_starts=i32([0, T]), output=torch.zeros_like(x), scale=1.0, **kw)
    assert e.value.code == code
    torch.cuda.synchronize()
    assert (out == 0).all()


def test_lengths_above_the_rows_are_the_rows():
    T, C = 9, 16
    d, _ = make(T, C)
    outs = [torch.zeros(T, C, dtype=BF, device="cuda") for _ in range(2)]
    for out, most in zip(outs, (T, 1 << 40)):
        kda_ssm_prompt(**d, seq_starts=i32([0, T]), output=out, max_seq=most)
    assert torch.equal(*outs) and (outs[0] != 0).any()

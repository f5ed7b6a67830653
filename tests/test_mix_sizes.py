"""Sizes of the convolution's and the scan's calls that their kernels' 32-bit numbers do not
hold are refused, without a GPU."""
from __future__ import annotations

import pytest

from linear_attention_recurrent_kda_gb300 import lib as kl
from tests.test_mix import conv_prompt, ssm_prompt


@pytest.mark.parametrize("seqs", [2 ** 31 - 255, 2 ** 31 - 7, 2 ** 31 - 1])
def test_sequences_that_bisection_cannot_round_up(seqs):
    """(hi - lo + 7) / 8 with hi = seqs would be below 0."""
    assert kl.call("kda_conv_prompt", conv_prompt(seqs=seqs, channels=24, x_stride=24), None) == kl.KDA_ERR_SHAPE
    for path in (0, 1, 2):
        args = ssm_prompt(seqs=seqs, channels=16, tokens=1 << 20, max_seq=1 << 20, path=path)
        assert kl.call("kda_ssm_prompt", args, None) == kl.KDA_ERR_SHAPE
        assert kl.ssm_workspace(args) == 0

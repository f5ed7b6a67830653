"""Sizes of the convolution's and the scan's calls that their kernels' 32-bit numbers do not
hold are refused, without a GPU."""
from __future__ import annotations

import pytest

from linear_attention_recurrent_kda_gb300 import api
from linear_attention_recurrent_kda_gb300 import lib as kl
from tests.test_mix import conv_prompt, ssm_prompt, ssm_step


@pytest.mark.parametrize("seqs", [2 ** 31 - 255, 2 ** 31 - 7, 2 ** 31 - 1])
def test_sequences_that_bisection_cannot_round_up(seqs):
    """(hi - lo + 7) / 8 with hi = seqs would be below 0."""
    assert kl.call("kda_conv_prompt", conv_prompt(seqs=seqs, channels=24, x_stride=24), None) == kl.KDA_ERR_SHAPE
    for path in (0, 1, 2):
        args = ssm_prompt(seqs=seqs, channels=16, tokens=1 << 20, max_seq=1 << 20, path=path)
        assert kl.call("kda_ssm_prompt", args, None) == kl.KDA_ERR_SHAPE
        assert kl.ssm_workspace(args) == 0


@pytest.mark.parametrize("channels,states,groups", [(1 << 30, 16, 1), (1 << 28, 64, 1), (1 << 26, 64, 1 << 23),
                                                    ((1 << 27) - 8, 16, 1)])
def test_channels_times_states_that_32_bits_do_not_count(channels, states, groups):
    """The kernels number the states of a slot's channels and groups."""
    sizes = dict(channels=channels, states=states, groups=groups, batch=1)
    sizes.update({f"{n}_stride": channels for n in ("x", "dt", "z", "o")})
    sizes.update({f"{n}_stride": groups * states for n in "bc"})
    assert kl.call("kda_ssm_step", ssm_step(**sizes), None) == kl.KDA_ERR_SHAPE
    del sizes["batch"]
    assert kl.call("kda_ssm_prompt", ssm_prompt(**sizes), None) == kl.KDA_ERR_SHAPE


@pytest.mark.parametrize("path", [0, 1, 2])
@pytest.mark.parametrize("seqs,channels,states,groups", [(1 << 24, 1 << 20, 16, 1), (1 << 22, 8 << 12, 64, 1 << 12),
                                                         ((1 << 31) - 256, 1 << 26, 16, 1)])
def test_no_workspace_for_grids_that_are_refused(seqs, channels, states, groups, path):
    """More blocks of threads than a launch takes: refused before its workspace is asked for."""
    sizes = dict(seqs=seqs, channels=channels, states=states, groups=groups, tokens=1 << 14, max_seq=1 << 14)
    sizes.update({f"{n}_stride": channels for n in ("x", "dt", "z", "o")})
    sizes.update({f"{n}_stride": groups * states for n in "bc"})
    assert kl.ssm_workspace(ssm_prompt(path=path, **sizes)) == 0
    assert kl.call("kda_ssm_prompt", ssm_prompt(path=path, **sizes), None) == kl.KDA_ERR_SHAPE


def test_lengths_that_32_bits_do_not_hold():
    most = [api._most(n, 9) for n in (None, 0, 5, 9, 10, 1 << 40, -1, -5, 5 - (1 << 32))]
    assert most == [9, 0, 5, 9, 9, 9, -1, -1, -1]

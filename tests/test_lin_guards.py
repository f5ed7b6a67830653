"""Guards of the linear-attention and snapshot calls: the chunked form's wait that
runs out, sequences out of order, and sizes that the C structs cannot hold."""
from __future__ import annotations

import ctypes
import time

import pytest
import torch

from linear_attention_recurrent_kda_gb300 import lib as kl


def test_wait_selftest_refusals():
    fn = kl.load().kda_selftest_lin_wait_timeout
    assert fn(None, None) == kl.KDA_ERR_NULL_POINTER
    assert fn(ctypes.c_void_p((1 << 20) + 2), None) == kl.KDA_ERR_ALIGNMENT


@pytest.mark.gpu
def test_wait_of_the_chunked_form_runs_out_and_the_context_stays_usable():
    """2 s of wall clock (no more than 3 with the launch), the flag, and TMEM
    free again: the chunked form runs afterwards on every SM."""
    from tests.test_lin_gpu import launch, make, verify
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.time()
    rc = kl.load().kda_selftest_lin_wait_timeout(
        ctypes.c_void_p(err.data_ptr()),
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == kl.KDA_SUCCESS
    torch.cuda.synchronize()
    waited = time.time() - t0
    assert int(err) == kl.KDA_DEVERR_TIMEOUT
    assert 1.9 < waited < 3.0, waited
    inp = make([130] * 40, 4, 4, seed=40)
    verify(inp, launch(inp, path=2), 2)

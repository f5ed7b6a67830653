"""Guards of the linear-attention and snapshot calls: the chunked form's wait that
runs out, sequences out of order, and sizes that the C structs cannot hold."""
from __future__ import annotations

import ctypes
import os
import subprocess
import sys
import time

import pytest
import torch

from linear_attention_recurrent_kda_gb300 import lib as kl
from linear_attention_recurrent_kda_gb300.api import (kda_lin_prompt, kda_lin_step,
                                                      kda_snapshot_load, kda_snapshot_save)


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


@pytest.mark.gpu
def test_starts_out_of_order_beside_sequences_that_would_be_split():
    """Sequences that share rows would share pages of the workspace: none that
    would be split runs, and the others are as they are without them."""
    from tests.test_lin_gpu import launch, make, verify
    inp = make([3000, 1000, 100, 40], 2, 2, slots=9, seed=41)
    assert kl.prompt_workspace(kl.KdaLinPromptArgs(
        seqs=5, heads=2, qk_heads=2, tokens=4140, max_seq=3000, q_stride=256, k_stride=256,
        v_stride=256, o_stride=256)) > 0
    bad = dict(inp, starts=[0, 3000, 1000, 4000, 4100, 4140])
    src, dst = [1, 2, 3, 4, 0], [1, 5, 6, 7, 8]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, state = launch(bad, src=src, dst=dst, max_seq=3000, err=err)
    assert int(err) == kl.KDA_DEVERR_SEQ
    assert torch.all(torch.isnan(out[:4000]))
    for slot in (0, 1, 2, 3, 4, 5, 6):
        assert torch.equal(state[slot], inp["state"][slot])
    rest = {n: inp[n][4000:] for n in ("q", "k", "v", "decay")}
    rest.update(starts=[0, 100, 140], state=inp["state"])
    state[[1, 5, 6]] = inp["state"][[1, 5, 6]]
    verify(rest, (out[4000:], state), 2, [4, 0], [7, 8])
    # in order again, everything runs and nothing is flagged
    err.zero_()
    good = dict(inp, starts=[0, 3000, 3000, 4000, 4100, 4140])
    verify(good, launch(good, src=src, dst=dst, max_seq=3000, err=err), 2, src, dst)
    assert int(err) == 0


@pytest.mark.gpu
def test_counts_past_32_bits_are_refused():
    """2^32 + 1 entries are not 1 entry (the list is never read)."""
    many = torch.empty(2 ** 32 + 1, dtype=torch.int32, device="cuda")
    state = torch.full((2, 1, 128, 128), 3.0, device="cuda")
    codes = torch.full((2, 1, 128, 128), 85, dtype=torch.int8, device="cuda")
    scales = torch.full((2, 1, 128), -3.0, device="cuda")
    for f in (kda_snapshot_save, kda_snapshot_load):
        with pytest.raises(ValueError, match="2\\^31"):
            f(state=state, slots=many, codes=codes, scales=scales, snaps=many)
    x = torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        kda_lin_prompt(q=x, k=x, v=x, decay=torch.zeros(1, device="cuda"), seq_starts=many,
                       output=torch.empty_like(x), scale=1.0)
    torch.cuda.synchronize()
    assert torch.all(state == 3.0) and torch.all(codes == 85) and torch.all(scales == -3.0)


@pytest.mark.gpu
@pytest.mark.parametrize("per_token", [False, True])
def test_no_heads_are_a_no_op(per_token):
    """As in the C ABI, for several rows too."""
    q = torch.zeros(5, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(5, 0, dtype=torch.bfloat16, device="cuda")
    decay = torch.zeros((5, 0) if per_token else (0,), device="cuda")
    kw = dict(q=q, k=q, v=v, decay=decay, output=torch.empty_like(v), scale=1.0,
              state=torch.zeros(6, 0, 128, 128, device="cuda"))
    i32 = dict(dtype=torch.int32, device="cuda")
    kda_lin_prompt(**kw, seq_starts=torch.tensor([0, 2, 5], **i32),
                   dst_slots=torch.tensor([1, 2], **i32))
    kda_lin_step(**kw, slots=torch.arange(1, 6, **i32))
    torch.cuda.synchronize()


CHILD = r"""
import threading, torch
from linear_attention_recurrent_kda_gb300 import api
from tests.test_lin_gpu import make, on_device

def prompt(lens, path, seed):
    inp = make(lens, 4, 2, slots=2 * len(lens) + 1, seed=seed, scale_g=0.1)
    B = len(lens)
    kw = on_device(inp, list(range(1, B + 1)), list(range(B + 1, 2 * B + 1)), path=path)
    return (lambda s: api.kda_lin_prompt(**kw, stream=s)), [kw["output"], kw["state"]]

def step(seed):
    inp = make([1] * 6, 4, 4, slots=7, seed=seed)
    d = {n: inp[n].cuda() for n in ("q", "k", "v", "decay", "state")}
    out = torch.zeros(6, 512, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(1, 7, dtype=torch.int32, device="cuda")
    return (lambda s: api.kda_lin_step(s, **d, slots=slots, output=out, scale=0.5)), [out, d["state"]]

def fork(bits, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    state = torch.randn(9, 3, 128, 128, generator=g, device="cuda")
    codes = torch.zeros(5, 3, 128, 16 * bits, device="cuda",
                        dtype=torch.int8 if bits == 8 else torch.uint8)
    scales = torch.zeros((5, 3, 128) if bits == 8 else (5, 3, 128, 4), device="cuda")
    ids = torch.arange(1, 5, dtype=torch.int32, device="cuda")
    kw = dict(state=state, codes=codes, scales=scales, snaps=ids)
    def run(s):
        api.kda_snapshot_save(**kw, slots=ids, stream=s)
        api.kda_snapshot_load(**kw, slots=ids + 4, stream=s)
    return run, [state, codes, scales]

def jobs():
    return [prompt([1500, 40], 0, 1), prompt([1400], 2, 2), prompt([200, 30], 2, 3),
            prompt([9, 3], 1, 4), step(5), step(6), fork(8, 7), fork(4, 8)]

mine, failures = jobs(), []
torch.cuda.synchronize()
gate = threading.Barrier(len(mine))

def work(run):
    try:
        s = torch.cuda.Stream()
        gate.wait()
        with torch.cuda.stream(s):
            run(s)
    except Exception as e:
        failures.append(repr(e))

threads = [threading.Thread(target=work, args=(run,)) for run, _ in mine]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not failures, failures
for (_, got), (run, want) in zip(mine, jobs()):
    run(None)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
print("same bits")
"""


@pytest.mark.gpu
def test_first_calls_from_several_host_threads():
    """A fresh process whose first calls come from eight threads at once, each on its
    own stream: the bits of the same calls one after another."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", CHILD], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert res.returncode == 0, res.stderr[-3000:]
    assert "same bits" in res.stdout

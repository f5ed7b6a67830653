"""Snapshots of the KDA step's own pages: a request that has decoded is kept and
decodes on from another slot.  The snapshot holds the state pages; the convolution
window of the slot is the caller's to keep."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from linear_attention_recurrent_kda_gb300.api import (kda_snapshot_load, kda_snapshot_save,
                                                      step_from_inputs)
from linear_attention_recurrent_kda_gb300.workloads import Workload, make_inputs
from tests import linref
from tests.parity import compare, run_gpu, to_device

pytestmark = pytest.mark.gpu
B, H, SLOTS = 5, 3, 16


def workload(seed):
    return Workload("snap", batch=B, heads=H, tokens=1, num_slots=SLOTS, conv_width=3,
                    slot_layout="decode", pad=1, seed=seed)


@pytest.mark.parametrize("bits", [8, 4])
def test_a_decoded_request_goes_on_from_its_snapshot(bits):
    inp = make_inputs(workload(70))
    dev = to_device(inp)
    out = torch.empty(B, H * 128, dtype=torch.bfloat16, device="cuda")
    step_from_inputs(dev, out)()
    slots = inp["slots"].tolist()
    live = [s for s in slots if s > 0]
    spare = [s for s in range(1, SLOTS) if s not in live][:len(live)]
    i32 = dict(dtype=torch.int32, device="cuda")
    codes = torch.zeros(B + 1, H, 128, 128 * bits // 8, device="cuda",
                        dtype=torch.int8 if bits == 8 else torch.uint8)
    scales = torch.zeros((B + 1, H, 128) if bits == 8 else (B + 1, H, 128, 4), device="cuda")
    snaps = torch.arange(1, len(live) + 1, **i32)
    state = dev["state"]
    kda_snapshot_save(state=state, slots=torch.tensor(live, **i32), codes=codes, scales=scales,
                      snaps=snaps)
    kda_snapshot_load(codes=codes, scales=scales, snaps=snaps, state=state,
                      slots=torch.tensor(spare, **i32))
    dev["conv_state"][spare] = dev["conv_state"][live]
    kept = state[live].cpu().numpy()
    want = linref.dequantise(*linref.quantise(kept, bits))
    assert np.array_equal(state[spare].cpu().numpy(), want)
    # the next token, from the spare slots: against the oracle on the pages as read back
    move = dict(zip(live, spare))
    nxt = make_inputs(workload(71))
    for n in ("conv_weight", "conv_bias", "f_b", "a_log", "dt_bias", "norm_weight"):
        nxt[n] = inp[n]
    nxt.update(state=state.cpu(), conv_state=dev["conv_state"].cpu(),
               slots=torch.tensor([move.get(s, s) for s in slots], dtype=torch.int32))
    compare(nxt, run_gpu(nxt))

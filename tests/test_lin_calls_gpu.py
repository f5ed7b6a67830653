"""Calls of the linear attention that serving makes and the other tests do not: no
tokens at all, and one captured call whose sequences change between replays."""
from __future__ import annotations

import pytest
import torch

from linear_attention_recurrent_kda_gb300 import lib as kl
from linear_attention_recurrent_kda_gb300.api import kda_lin_prompt
from tests.test_lin_gpu import launch, make, on_device, verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("path", [0, 1, 2])
@pytest.mark.parametrize("per_token", [False, True])
def test_no_tokens_copy_the_first_states(path, per_token):
    inp = make([0, 0, 0], 2, 1, slots=6, per_token=per_token, seed=60)
    out, state = launch(inp, src=[1, 0, 2], dst=[3, 4, 2], path=path)
    assert out.shape[0] == 0
    want = inp["state"].clone()
    want[3], want[4] = want[1], 0.0
    assert torch.equal(state, want)


def test_no_sequences_are_a_no_op():
    inp = make([], 2, 1, slots=3, seed=61, behind=7)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, state = launch(inp, src=[], dst=[], err=err)
    assert torch.all(torch.isnan(out)) and torch.equal(state, inp["state"]) and int(err) == 0


@pytest.mark.parametrize("H,Hk,max_seq,split", [(2, 1, 1500, True), (2, 2, 700, False)])
def test_a_captured_call_takes_the_starts_of_its_replay(H, Hk, max_seq, split):
    """The plan goes by the rows, the heads and max_seq; where sequences start and
    end, and their slots, are read when the graph runs."""
    n, B = 2000, 4
    kw = dict(seqs=B, heads=H, qk_heads=Hk, tokens=n, max_seq=max_seq, q_stride=Hk * 128,
              k_stride=Hk * 128, v_stride=H * 128, o_stride=H * 128)
    assert (kl.prompt_workspace(kl.KdaLinPromptArgs(**kw)) > 0) == split
    inp = make([n], H, Hk, slots=10, seed=62, scale_g=0.1)
    inp["starts"] = [0] * (B + 1)
    a = on_device(inp, [0] * B, [0] * B, max_seq=max_seq, path=2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda_lin_prompt(**a)
    runs = [([0, 700, 700, 701, 1400], [1, 0, 3, 1], [5, 6, 3, 0]),
            ([3, 130, 640, 1300, 2000], [0, 2, 0, 4], [1, 2, 7, 8])]
    if split:
        runs += [([0, 1500, 1500, 1999, 2000], [1, 2, 0, 4], [5, 6, 7, 8]),
                 ([10, 11, 20, 1400, 1400], [0, 0, 2, 2], [4, 5, 2, 0])]
    for starts, src, dst in runs:
        for name, val in (("seq_starts", starts), ("src_slots", src), ("dst_slots", dst)):
            a[name].copy_(torch.tensor(val, dtype=torch.int32))
        a["state"].copy_(inp["state"])
        a["output"].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = a["output"].cpu(), a["state"].cpu()
        case = dict(inp, starts=starts)
        verify(case, got, 2, src, dst)
        assert torch.all(torch.isnan(got[0][:starts[0]]))
        again = launch(case, src=src, dst=dst, path=2, max_seq=max_seq)
        assert torch.equal(again[0].nan_to_num(9.0), got[0].nan_to_num(9.0))
        assert torch.equal(again[1], got[1])

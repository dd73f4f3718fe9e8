"""Rows read back from batches of many empty sequences: a row's sequence is found in a few steps, not one by one."""
import pytest
import torch

import online_softmax_fa2_gb300 as ofa
from paged_q8_helpers import q8_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def batch(B, at):
    """Three sequences with rows, at the places `at` of B, and their rows alone."""
    rows = [3, 1, 5]
    s = q8_inputs([1] * 3, [40, 17, 70], 1, 2, 64, 16, poison=False)
    bt = torch.full((B, s["bt"].shape[1]), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    n = torch.zeros(B, dtype=torch.int32)
    at = torch.tensor(at)
    bt[at.to(DEV)], lens[at.to(DEV)] = s["bt"], s["lens"]
    n[at] = torch.tensor(rows, dtype=torch.int32)
    cu = torch.cat([torch.zeros(1, dtype=torch.int32), n.cumsum(0).int()]).to(DEV)
    few = torch.tensor([0, 3, 4, 9], dtype=torch.int32, device=DEV)
    cache = (s["kp"], s["vp"], s["ks"], s["vs"])
    return (*cache, bt, lens, 9, cu), (*cache, s["bt"], s["lens"], 9, few)


@pytest.mark.parametrize("B,at", [(3, [0, 1, 2]), (40, [0, 1, 39]), (40, [5, 38, 39]), (65535, [0, 40000, 65534]), (65535, [65532, 65533, 65534])])
def test_rows_between_empty_sequences(B, at):
    many, alone = batch(B, at)
    ofa.device_error_flags()
    got, want = ofa.attn_paged_read_q8(*many), ofa.attn_paged_read_q8(*alone)
    assert ofa.device_error_flags() == 0
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_the_time_does_not_go_by_the_empty_ones():
    """65,000 empty sequences between two rows cost no more than a few loads."""
    def us(args):
        k, v = ofa.attn_paged_read_q8(*args)
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        best = 1e9
        for _ in range(20):
            e[0].record()
            ofa.attn_paged_read_q8(*args, k_out=k, v_out=v)
            e[1].record()
            torch.cuda.synchronize()
            best = min(best, e[0].elapsed_time(e[1]) * 1e3)
        return best

    many, alone = batch(65535, [0, 40000, 65534])
    assert us(many) < us(alone) + 500  # (one by one 2000 us)

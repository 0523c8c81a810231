"""GPU checks of the page operations: slot bytes and tables bit for bit against the oracle."""
import numpy as np
import pytest
import torch

from mixed_format_paged_mkv_b200.workloads import Workload

from harness import lib_pool, oracle_pool

pytestmark = pytest.mark.gpu


def compare_pages(lp, op, seqs):
    for s in seqs:
        t, ctx = lp.block_table(s)
        assert t == op.block_table(s) and ctx == op.ctx[s], s
        cols = lp.cfg.max_pages_per_seq
        row = lp.buffers[2].view(torch.int32)[s * cols:(s + 1) * cols].cpu().numpy()
        assert row[:len(t)].tolist() == t, s
        for p, e in enumerate(t):
            assert np.array_equal(lp.read_slot(e), op.slot_bytes(e)), f"seq {s} page {p} {e:#x}"
    lp.device_status()


@pytest.mark.parametrize("tq3_slots", [0, 7])
def test_copy_in_a_control_pool(tq3_slots):
    """The pages of a BF16 control pool are copied inside the first slab (its TQ3 slab may be
    empty)."""
    w = Workload("ctlcopy", 71, B=2, Hq=4, Hkv=2, D=64, q_len=1, window=16, ctx=(50, 33))
    shape = dict(w.pool_shape(), fp8_slots=24, tq3_slots=tq3_slots, max_seqs=4)
    w = w.scaled(slot_order=False)
    lp = lib_pool(w, shape=shape, bf16_control=True)
    op = oracle_pool(w, shape=shape, bf16_control=True)
    lp.copy(0, 2)
    op.seq_copy(0, 2)
    compare_pages(lp, op, range(4))

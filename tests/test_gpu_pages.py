"""GPU checks of the page operations: slot bytes and tables bit for bit against the oracle."""
import numpy as np
import pytest
import torch

from mixed_format_paged_mkv_b200 import Pool
from mixed_format_paged_mkv_b200.workloads import Workload, bf16_bits
from oracle import formats as F
from oracle import pool as P

from harness import lib_pool, oracle_pool, to_bf16_tensor
from test_branch_host import pools, random_step

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


def draw_kv(g, n, Hkv, D):
    bits = bf16_bits(g.standard_normal((2, n, Hkv, D), dtype=np.float32))
    return (tuple(to_bf16_tensor(b) for b in bits), tuple(F.bf16_bits_to_f64(b) for b in bits))


@pytest.mark.parametrize("seed,Hkv,D,control", [(0, 1, 64, False), (1, 2, 128, False), (2, 3, 256, False),
                                                (3, 2, 64, True), (4, 1, 256, True), (5, 4, 64, False)])
def test_random_streams_keep_every_page_bit_exact(seed, Hkv, D, control):
    rng = np.random.default_rng(7000 + seed)
    lp, op, n_seqs, max_pages, slots = pools(rng, Hkv, D, control=control)
    seen = set()
    for step in range(120):
        kind, err = random_step(rng, lp, op, n_seqs, max_pages, slots, kv=lambda n: draw_kv(rng, n, Hkv, D))
        if err is None:
            seen.add(kind)
        if step % 6 == 5 or kind in ("truncate", "compact"):
            compare_pages(lp, op, range(n_seqs))
    assert {"fork", "truncate", "free", "compact", "copy"} <= seen


def test_calls_of_many_launches():
    """Lists longer than one launch holds, pages larger than a CTA's piece."""
    Hkv, D, n = 5, 256, 1500
    lp = Pool(Hkv, D, n + 10, 9, 2 * n, 40)
    op = P.RefPool(Hkv, D, n + 10, 9, 2 * n, 40)
    g = np.random.default_rng(5)
    l, o = draw_kv(g, 100, Hkv, D)
    for p, kv in ((lp, l), (op, o)):
        p.append([0], [100], *kv)
        p.demote([0], 32)
        p.fork([0] * n, list(range(5, 5 + n)), [100 - i % 4 for i in range(n)])
        p.truncate(list(range(5, 5 + n)), [97 - i % 30 for i in range(n)])
        p.free(list(range(5, 5 + n, 40)) + [0])
        assert p.compact() > 1200
    compare_pages(lp, op, list(range(0, 40)) + list(range(n - 30, n + 10)))


def test_branches_decode_as_their_own_copies():
    """fork, append, truncate and demote on branches against deep copies: the same outputs."""
    Hkv, D, Hq = 2, 128, 8
    g = np.random.default_rng(6)
    lp = Pool(Hkv, D, 8, 60, 200, 200)
    (k, v), _ = draw_kv(g, 700, Hkv, D)
    lp.prefill([0], [700], k, v, window=64)
    lp.fork([0, 0], [1, 2], [700, 688])
    lp.copy(0, 3)
    lp.copy(0, 4)
    lp.truncate([4], [688])
    for i in range(3):
        (k, v), _ = draw_kv(g, 2 * 9, Hkv, D)
        for ids in ([1, 2], [3, 4]):
            lp.append(ids, [9, 9], k, v)
            lp.demote(ids, 32)
    lp.truncate([1, 2, 3, 4], [720, 700, 720, 700])
    q = torch.randn((4, 1, Hq, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    q[2:] = q[:2]
    for _ in range(2):
        for s in (1, 2, 3, 4):
            kd, vd = lp.materialise(s)
            ke, ve = lp.materialise({1: 3, 2: 4, 3: 1, 4: 2}[s])
            assert torch.equal(kd, ke) and torch.equal(vd, ve), s
        out = lp.decode([1, 2, 3, 4], q)
        assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])
        lp.free([0])
        lp.compact()
    lp.device_status()

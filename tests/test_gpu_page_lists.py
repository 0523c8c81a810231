"""GPU check of the page operations where a call's lists change from the small parameter block to the large
one: pages and tables bit for bit against the oracle on both sides."""
import numpy as np
import pytest

from mixed_format_paged_mkv_b200 import Pool
from oracle import pool as P

from test_gpu_pages import compare_pages, draw_kv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 110, 111, 112, 113])
def test_lists_around_the_small_block(n):
    Hkv, D = 2, 64
    lp, op = Pool(Hkv, D, n + 4, 6, 3 * n + 20, 8), P.RefPool(Hkv, D, n + 4, 6, 3 * n + 20, 8)
    l, o = draw_kv(np.random.default_rng(n), 60, Hkv, D)
    order = np.random.default_rng(8).permutation(3 * n + 20)         # (no runs of neighbouring slots)
    ids = list(range(2, 2 + n))
    for p, kv in ((lp, l), (op, o)):
        p.set_slot_order(0, order)
        p.append([0], [60], *kv)
        p.demote([0], 30)
        p.fork([0] * n, ids, [60 - i % 9 for i in range(n)])
    compare_pages(lp, op, range(n + 4))
    for p in (lp, op):
        p.truncate(ids, [50 - i % 3 if i % 2 else 33 + i % 10 for i in range(n)])
    compare_pages(lp, op, range(n + 4))
    for p in (lp, op):
        p.set_slot_order(0, order[::-1].copy())
        p.compact()
    compare_pages(lp, op, range(n + 4))
    for p in (lp, op):
        p.free(ids)
    compare_pages(lp, op, range(n + 4))
    assert lp.stats()[0] == 60

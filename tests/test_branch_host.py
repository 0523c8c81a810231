"""Host logic of fork, truncate, free and compact (CPU, host-only pools): random streams of all pool
operations against the oracle's pool, failed launches, and the argument contract."""
import ctypes

import numpy as np
import pytest

from mixed_format_paged_mkv_b200 import MkvError, Pool
from mixed_format_paged_mkv_b200.api import lib
from oracle import pool as P

from test_host_fuzz import both, state
from test_plan import check_cut


def random_step(rng, lp, op, n_seqs, max_pages, slots, kv=None):
    """One random operation on both pools; returns its name and the error (None: it succeeded).
    ``kv(rows)`` draws inputs for both (default: none, zeros)."""
    HKV, D = lp.Hkv, lp.D
    ids_all = list(range(n_seqs)) + [n_seqs]

    def some(most=4):
        ids = [int(x) for x in rng.choice(ids_all, size=int(rng.integers(1, most + 1)))]
        return ids if rng.random() < 0.15 else (sorted(set(i for i in ids if i < n_seqs)) or [0])

    def rows(n):
        if kv is None:
            z = np.zeros((n, HKV, D))
            return (None, None), (z, z)
        return kv(n)

    kind = rng.choice(["append", "append", "append", "protect", "demote", "demote", "prefill", "copy",
                       "reset", "order", "fork", "fork", "fork", "truncate", "truncate", "free", "compact"])
    if kind == "append":
        ids = some(3)
        counts = [int(rng.integers(0, 40)) for _ in ids]
        l, o = rows(sum(counts))
        r = both(lambda: lp.append(ids, counts, *l), lambda: op.append(ids, counts, *o))
    elif kind == "protect":
        s, page = int(rng.integers(0, n_seqs)), int(rng.integers(-1, max_pages + 1))
        flag = int(rng.integers(0, 2))
        r = both(lambda: lp.set_protected(s, page, flag), lambda: op.set_protected(s, page, flag))
    elif kind == "demote":
        ids, W = some(n_seqs), int(rng.choice([0, 16, 40, 64]))
        r = both(lambda: lp.demote(ids, W), lambda: op.demote(ids, W))
        assert r[2] or r[0] == len(r[1])
    elif kind == "prefill":
        ids = some(2)
        counts, W = [int(rng.integers(0, 80)) for _ in ids], int(rng.choice([0, 16, 64]))
        l, o = rows(sum(counts))
        r = both(lambda: lp.prefill(ids, counts, *l, window=W), lambda: op.prefill(ids, counts, *o, W))
    elif kind == "copy":
        s, d = (int(x) for x in rng.integers(0, n_seqs, size=2))
        r = both(lambda: lp.copy(s, d), lambda: op.seq_copy(s, d))
    elif kind == "reset":
        s = int(rng.integers(0, n_seqs))
        r = both(lambda: lp.reset(s), lambda: op.seq_reset(s))
    elif kind == "order":
        fmt = int(rng.integers(0, 2))
        order = rng.permutation(slots[fmt]).tolist()
        r = both(lambda: lp.set_slot_order(fmt, order), lambda: op.set_slot_order(fmt, order))
    elif kind == "fork":
        empty = [s for s in range(n_seqs) if not op.ctx[s]]
        full = [s for s in range(n_seqs) if op.ctx[s]] or [0]
        k = int(rng.integers(0, 4))
        src = [int(rng.choice(full)) for _ in range(k)]
        dst = [int(x) for x in rng.permutation(empty)[:k]] if len(empty) >= k else some(3)[:k]
        src = src[:len(dst)]
        at = None if rng.random() < 0.4 else [int(rng.integers(-1 if rng.random() < 0.05 else 0, op.ctx[s] + 1))
                                              if rng.random() < 0.5 else op.ctx[s] // 16 * 16 for s in src]
        if rng.random() < 0.05 and dst:
            dst[0] = int(rng.choice(ids_all))
        r = both(lambda: lp.fork(src, dst, at), lambda: op.fork(src, dst, at))
    elif kind == "truncate":
        ids = some(3)
        cut = [max(0, (op.ctx[s] if s < n_seqs else 3) - int(rng.integers(-1 if rng.random() < 0.1 else 0, 40)))
               for s in ids]
        r = both(lambda: lp.truncate(ids, cut), lambda: op.truncate(ids, cut))
    elif kind == "free":
        ids = some(2)
        r = both(lambda: lp.free(ids), lambda: op.free(ids))
    else:
        r = both(lambda: lp.compact(), lambda: op.compact())
        assert r[0] == r[1]
        for f in (0, 1):  # the slots in use are the first ones of the order
            a = op.alloc[f]
            held = a.n - len(a.free)
            assert all(a.rank[s] >= held for s in a.free)
    return str(kind), r[2]


def pools(rng, HKV, D, control=False, **kw):
    n_seqs, max_pages = int(rng.integers(3, 8)), int(rng.integers(3, 12))
    slots = int(rng.integers(6, 4 * max_pages)), int(rng.integers(0, 3 * max_pages))
    sink = int(rng.integers(0, 3))
    lp = Pool(HKV, D, n_seqs, max_pages, *slots, sink_pages=sink, bf16_control=control, **kw)
    op = P.RefPool(HKV, D, n_seqs, max_pages, *slots, sink_pages=sink, bf16_control=control)
    return lp, op, n_seqs, max_pages, slots


@pytest.mark.parametrize("seed", range(12))
def test_random_streams_match_the_oracle(seed):
    rng = np.random.default_rng(4000 + seed)
    lp, op, n_seqs, max_pages, slots = pools(rng, 1, 64, control=seed % 4 == 3, host_only=True)
    seen = {}
    for step in range(300):
        kind, err = random_step(rng, lp, op, n_seqs, max_pages, slots)
        seen.setdefault(kind, set()).add(err)
        state(lp, op, n_seqs)
        if step % 10 == 9:
            live = [q for q in range(n_seqs) if op.ctx[q] > 0]
            if live:
                check_cut(lp, live, *lp.decode_plan(live, 1, 1), 1)
    assert all(None in seen[k] for k in ("fork", "truncate", "free", "compact")), seen


def test_shared_pages_count_once_and_live_as_long_as_a_holder():
    p = Pool(1, 64, 5, 8, 16, 16, host_only=True)
    p.append([0], [100])                          # 7 pages, the last with 4 tokens
    p.fork([0, 0], [1, 2], [100, 96])
    t0, t1, t2 = (p.block_table(s)[0] for s in (0, 1, 2))
    assert t1[:6] == t0[:6] == t2 and t1[6] == 7 and p.block_table(2)[1] == 96
    live, n8, n3, bpt = p.stats()
    assert (live, n8, n3) == (296, 8, 0) and bpt == pytest.approx(8 * 2064 / 296)
    p.reset(0)
    assert p.stats()[1] == 7 and p.block_table(1)[0] == t1
    assert p.demote([1, 2], 0) == 5 + 5           # converted once for both holders
    assert p.stats()[1:3] == (2, 5)
    assert p.block_table(1)[0][1:6] == p.block_table(2)[0][1:6]
    p.fork([2], [3], [32])
    assert p.demote([3], 0) == 0
    p.free([1, 2])
    assert p.stats()[1:3] == (1, 1)
    p.free([3, 4])
    assert p.stats()[:3] == (0, 0, 0)


def test_demoting_one_holder_leaves_the_others_page():
    p = Pool(1, 64, 3, 8, 16, 16, sink_pages=0, host_only=True)
    p.append([0], [48])
    p.fork([0], [1])
    assert p.demote([1], 0) == 3
    assert p.block_table(0)[0] == [0, 1, 2] and p.stats()[1:3] == (3, 3)
    p.reset(0)
    assert p.stats()[1:3] == (0, 3)


def small():
    p = Pool(1, 64, 3000, 40, 40000, 20000, host_only=True)
    p.set_slot_order(0, np.random.default_rng(1).permutation(40000))   # (no runs of neighbouring slots)
    p.append([0, 1], [500, 77])
    p.demote([0], 48)
    return p


def many(p, n=1400):
    """More branches than one launch holds, each with a partial page of its own."""
    return [0] * n, list(range(10, 10 + n)), [500 - 1] * n


CALLS = {
    "fork": lambda p: p.fork(*many(p)),
    "truncate": lambda p: p.truncate(list(range(10, 1410)), [470 + i % 29 for i in range(1400)]),
    "free": lambda p: p.free(list(range(10, 1410))),
    "compact": lambda p: p.compact(),
}


def tables(p, seqs=range(0, 1420)):
    return [p.block_table(s) for s in seqs], p.stats()


def build(name):
    p = small()
    if name != "fork":
        p.fork(*many(p))
    if name == "compact":
        p.free(list(range(10, 1410, 9)) + [1])
        p.append([1], [1])
        p.set_slot_order(0, list(range(40000))[::-1])
    return p


@pytest.mark.parametrize("name", list(CALLS))
def test_failed_launch(name):
    """fork leaves the pool as it was; the other calls have done a leading part, and the same call
    again does the rest: the pool then equals one that never failed, up to the slots' numbers."""
    twin = build(name)
    CALLS[name](twin)
    failures = 0
    for k in range(64):
        p = build(name)
        before = tables(p)
        p.test_fail_launch(k)
        try:
            CALLS[name](p)
            p.test_fail_launch(-1)
            break
        except MkvError as e:
            assert e.name == "CUDA"
        failures += 1
        if name == "fork" or k == 0:
            assert tables(p) == before
        elif name in ("free", "truncate"):
            want = tables(twin, range(10, 1410))[0]
            got = tables(p, range(10, 1410))[0]
            undone = before[0][10:1410]
            done = [g[1] == w[1] for g, w in zip(got, want)]
            first = done.index(False)
            assert first > 0 and got[first + 30:] == undone[first + 30:]
        if name == "compact":  # the lengths, formats and sharing never change
            assert [t[1] for t in tables(p)[0]] == [t[1] for t in before[0]] and p.stats() == before[1]
        CALLS[name](p)
        assert p.stats() == twin.stats()
        assert [t[1] for t in tables(p)[0]] == [t[1] for t in tables(twin)[0]]
        if name != "truncate":
            assert tables(p) == tables(twin)
    assert failures >= 2


def test_null_pool_and_lists():
    L = lib()
    seqs = (ctypes.c_int32 * 1)(0)
    n = ctypes.c_int32(7)
    assert L.mkv_seq_fork(None, seqs, seqs, None, 1, None) == -1
    assert L.mkv_seq_truncate(None, seqs, seqs, 1, None) == -1
    assert L.mkv_seq_free(None, seqs, 1, None) == -1
    assert L.mkv_pool_compact(None, ctypes.byref(n), None) == -1 and n.value == 0
    p = Pool(1, 64, 2, 4, 4, 4, host_only=True)
    assert L.mkv_seq_fork(p.handle, None, seqs, None, 1, None) == -1
    assert L.mkv_seq_fork(p.handle, seqs, seqs, None, -1, None) == -1
    assert L.mkv_seq_truncate(p.handle, seqs, None, 1, None) == -1
    assert L.mkv_seq_free(p.handle, None, 1, None) == -1
    assert L.mkv_pool_compact(p.handle, None, None) == 0
    p.fork([], [])
    p.truncate([], [])
    p.free([])


@pytest.mark.parametrize("call,name", [
    (lambda p: p.fork([0], [0]), "INVALID_ARG"),                # a source as destination
    (lambda p: p.fork([0], [1]), "INVALID_ARG"),                # not empty
    (lambda p: p.fork([0, 0], [2, 2]), "INVALID_ARG"),
    (lambda p: p.fork([0, 2], [2, 3]), "INVALID_ARG"),          # destination and source
    (lambda p: p.fork([0], [9]), "BAD_SEQ"),
    (lambda p: p.fork([9, 0], [0, 0]), "BAD_SEQ"),              # reported before the other errors
    (lambda p: p.fork([0], [2], [501]), "INVALID_ARG"),
    (lambda p: p.fork([0], [2], [-1]), "INVALID_ARG"),
    (lambda p: p.fork([0], [2], [39]), "UNSUPPORTED"),          # inside a TQ3 page
    (lambda p: p.fork([0, 0], [2, 3]), "OUT_OF_PAGES"),         # one free slot, two partial pages
    (lambda p: p.truncate([0, 0], [3, 3]), "INVALID_ARG"),
    (lambda p: p.truncate([0], [501]), "INVALID_ARG"),
    (lambda p: p.truncate([0], [-1]), "INVALID_ARG"),
    (lambda p: p.truncate([0], [39]), "UNSUPPORTED"),
    (lambda p: p.truncate([-1], [3]), "BAD_SEQ"),
    (lambda p: p.free([0, 0]), "INVALID_ARG"),
    (lambda p: p.free([0, 4]), "BAD_SEQ"),
])
def test_refusals_change_nothing(call, name):
    p = Pool(1, 64, 4, 40, 33, 60, host_only=True)
    p.append([0], [500])
    p.demote([0], 48)
    p.append([1], [16 * 26 + 5])
    assert p.stats()[1] == 32
    before = [p.block_table(s) for s in range(4)], p.stats()
    with pytest.raises(MkvError) as e:
        call(p)
    assert e.value.name == name
    assert ([p.block_table(s) for s in range(4)], p.stats()) == before


def test_truncate_needs_a_slot_for_a_shared_page():
    p = Pool(1, 64, 3, 8, 3, 0, host_only=True)
    p.append([0], [48])
    p.fork([0], [1])
    with pytest.raises(MkvError) as e:
        p.truncate([1], [40])
    assert e.value.name == "OUT_OF_PAGES"
    p.truncate([1], [32])
    p.truncate([0], [40])                        # its own page now: cut where it is
    assert p.block_table(0) == ([0, 1, 2], 40) and p.block_table(1) == ([0, 1], 32)
    p.truncate([0, 1], [0, 0])
    assert p.stats()[:3] == (0, 0, 0)


def test_binding_checks_lengths():
    p = Pool(1, 64, 3, 8, 3, 0, host_only=True)
    with pytest.raises(ValueError):
        p.fork([0], [1, 2])
    with pytest.raises(ValueError):
        p.fork([0], [1], [1, 2])
    with pytest.raises(ValueError):
        p.truncate([0], [1, 2])

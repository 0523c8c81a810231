"""Up to which size a truncate, free or compact is one launch, hence all or nothing (CPU): one device
operation for the largest such list, two for one sequence more."""
import pytest

from mixed_format_paged_mkv_b200 import MkvError, Pool

PAGES, ROWS = 850, 960      # pages cut or moved, table rows of a launch


def branches(n):
    """n branches of a sequence of 16 + 9 tokens, each with a partial page of its own."""
    p = Pool(1, 64, 2000, 4, 2000, 0, host_only=True)
    p.append([0], [25])
    ids = list(range(1, n + 1))
    p.fork([0] * n, ids)
    return p, ids


def state(p):
    return [p.block_table(s) for s in range(p.cfg.max_seqs)], p.stats()


def operations(p, call):
    """Device operations that the call issues: the injected failure that it no longer reaches."""
    before = state(p)
    p.test_fail_launch(0)
    with pytest.raises(MkvError):
        call(p)
    assert state(p) == before                       # nothing was issued yet
    p.test_fail_launch(1)
    try:
        call(p)
    except MkvError as e:
        assert e.name == "CUDA"
        return 2
    p.test_fail_launch(-1)
    return 1


@pytest.mark.parametrize("cut,drop,launches", [
    (PAGES, 0, 1), (PAGES + 1, 0, 2),               # ends inside a page
    (0, ROWS, 1), (0, ROWS + 1, 2),                 # the last page given up
    (PAGES, ROWS - PAGES, 1), (PAGES + 1, 9, 2),
    (PAGES, ROWS, 1), (PAGES, ROWS + 1, 2),         # (a sequence cut in its last page changes no entry)
])
@pytest.mark.parametrize("cuts_first", [True, False])
def test_truncate(cut, drop, launches, cuts_first):
    p, ids = branches(cut + drop)
    at = [20] * cut + [16] * drop if cuts_first else [16] * drop + [20] * cut
    assert operations(p, lambda p: p.truncate(ids, at)) == launches
    done = [p.block_table(s)[1] != 25 for s in ids]
    assert all(done) if launches == 1 else any(done) and not all(done)


@pytest.mark.parametrize("n,launches", [(ROWS, 1), (ROWS + 1, 2)])
def test_free(n, launches):
    p, ids = branches(n)
    assert operations(p, lambda p: p.free(ids)) == launches


@pytest.mark.parametrize("n,launches", [(PAGES, 1), (PAGES + 1, 2)])
def test_compact(n, launches):
    p = Pool(1, 64, 2200, 2, 4400, 0, host_only=True)
    p.append(list(range(2 * n)), [1] * (2 * n))
    p.free(list(range(0, 2 * n, 2)))
    order = [s for s in range(0, 2 * n, 2)] + [s for s in range(2 * n - 1, 0, -2)]   # the free ones first
    order += [s for s in range(2 * n, 4400)]
    p.set_slot_order(0, order)
    p.test_fail_launch(1)
    try:
        assert p.compact() == n and launches == 1
    except MkvError:
        assert launches == 2

"""The lists of sequences, lengths and axes that the binding takes: whole numbers that fit 32 bits, in
any container; anything else is refused before it can cut or free another part (CPU)."""
import numpy as np
import pytest
import torch

from mixed_format_paged_mkv_b200 import Pool
from mixed_format_paged_mkv_b200.api import _i32_list


def pool():
    p = Pool(1, 64, 4, 8, 16, 0, host_only=True)
    p.append([0, 1], [100, 50])
    return p


BAD = [[3.9], [3.0], np.array([3.9]), np.array([3.0], np.float32), np.array([2 ** 32 + 5]), [2 ** 32 + 5],
       np.array([-2 ** 31 - 1]), np.array([2 ** 63 + 1], np.uint64), [None], ["3"], np.array(["3"]),
       np.array([True]), None, torch.tensor([3.9]), torch.tensor([2 ** 32 + 5]), [np.float64(3.0)],
       [2 ** 80]]


@pytest.mark.parametrize("bad", BAD, ids=repr)
@pytest.mark.parametrize("call", ["truncate", "truncate_ids", "free", "fork", "fork_at"])
def test_refused_and_nothing_changed(call, bad):
    p = pool()
    before = [p.block_table(s) for s in range(4)], p.stats()
    with pytest.raises(ValueError):
        if call == "truncate":
            p.truncate([0], bad)
        elif call == "truncate_ids":
            p.truncate(bad, [3])
        elif call == "free":
            p.free(bad)
        elif call == "fork":
            p.fork(bad, [2])
        elif bad is None:                            # (the default: whole sources)
            raise ValueError
        else:
            p.fork([0], [2], bad)
    assert ([p.block_table(s) for s in range(4)], p.stats()) == before


@pytest.mark.parametrize("good", [[3, 2], (3, 2), np.array([3, 2]), np.array([3, 2], np.uint8), np.array([3, 2], np.int16),
                                  [np.int64(3), np.uint8(2)], torch.tensor([3, 2]), range(3, 1, -1),
                                  np.array([3, 9, 2, 9])[::2], [torch.tensor(3), 2], [[3], [2]],
                                  np.array([[3, 2]])], ids=repr)
def test_containers(good):
    p = pool()
    p.truncate([0, 1], good)
    assert [p.block_table(s)[1] for s in (0, 1)] == [3, 2]


@pytest.mark.parametrize("empty", [[], (), np.array([]), np.zeros(0, np.int64), range(0)], ids=repr)
def test_empty(empty):
    p = pool()
    p.free(empty)
    p.truncate(empty, empty)
    p.fork(empty, empty, empty)
    assert p.stats()[0] == 150


def test_one_number():
    p = pool()
    p.truncate(0, 7)
    p.free(np.int64(1))
    assert [p.block_table(s)[1] for s in (0, 1)] == [7, 0]


def test_limits():
    for x in (2 ** 31 - 1, -2 ** 31):
        for xs in ([x], np.array([x])):
            assert list(_i32_list(xs)[2]) == [x]

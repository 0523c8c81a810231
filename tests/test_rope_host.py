"""The argument contract of mkv_rope, called through ctypes on the CPU: every refusal comes before any
device call, and a call that passes them all is refused last because a host-only pool has no device."""
import ctypes

import pytest

from mixed_format_paged_mkv_b200 import Pool
from mixed_format_paged_mkv_b200.api import lib

INVALID_ARG = -1
HKV, D, HQ, ROWS = 2, 64, 4, 5
QB, KB = ROWS * HQ * D * 2, ROWS * HKV * D * 2


@pytest.fixture(scope="module")
def pool():
    return Pool(HKV, D, 1, 1, 1, 1, host_only=True)


def call(pool, rows=ROWS, pos=0x900000, axes=1, inv=0x910000, nf=32, axis=None, hq=HQ, qi=0x100000, qo=0x200000,
         ki=0x300000, ko=0x400000, qis=HQ * D, qos=HQ * D, kis=HKV * D, kos=HKV * D):
    P = ctypes.c_void_p
    a = None if axis is None else (ctypes.c_int32 * len(axis))(*axis)
    rc = lib().mkv_rope(pool.handle if pool else None, rows, P(pos), axes, P(inv), nf, a, 0, P(qi), qis, P(qo), qos,
                        hq, P(ki), kis, P(ko), kos, None)
    return rc, lib().mkv_last_error().decode()


S = (HQ + HKV) * D + 6   # a fused row


@pytest.mark.parametrize("kw,word", [
    (dict(rows=-1), "rows"), (dict(rows=1 << 31), "rows"),
    (dict(hq=3), "multiple"), (dict(hq=0), "multiple"),
    (dict(axes=0), "n_axes"), (dict(axes=129), "n_axes"),
    (dict(nf=0), "n_freq"), (dict(nf=33), "n_freq"), (dict(nf=1 << 30), "n_freq"),
    (dict(axis=[0] * 31 + [1]), "axis 1 of frequency 31"), (dict(axes=2, axis=[-1] + [0] * 31), "axis -1"),
    (dict(pos=0), "NULL"), (dict(inv=0), "NULL"), (dict(qi=0), "NULL"), (dict(ko=0), "NULL"),
    (dict(pos=0x900002), "4-byte"), (dict(inv=0x910001), "4-byte"),
    (dict(qis=HQ * D - 1), "q_in: row stride"), (dict(kos=0), "k_out: row stride"),
    (dict(kis=1 << 38), "k_in: row stride"),
    (dict(qi=0x100001), "2-byte"),
    (dict(qo=0x100002), "q_out overlaps q_in"), (dict(qo=0x100000, qos=HQ * D + 8), "q_out overlaps q_in"),
    (dict(qo=0x300000 + KB - 2), "q_out overlaps k_in"), (dict(ko=0x200000 + QB - 2), "k_out overlaps q_out"),
    (dict(ko=0x100000), "k_out overlaps q_in"),
    (dict(qo=0x900000), "q_out overlaps positions"), (dict(ko=0x910000 + 32 * 4 - 4), "k_out overlaps inv_freq"),
    # parts of one fused array: apart, then one element into the other
    (dict(qi=0x100000, qo=0x100000, qis=S, qos=S, ki=0x100000 + 2 * HQ * D, ko=0x100000 + 2 * HQ * D, kis=S, kos=S),
     "host-only"),
    (dict(qi=0x100000, qo=0x100000, qis=S, qos=S, ki=0x100000 + 2 * HQ * D - 2, ko=0x100000 + 2 * HQ * D - 2, kis=S,
          kos=S), "overlaps"),
    (dict(qo=0x100000, ko=0x300000), "host-only"),          # in place
    (dict(qo=0x100000 + QB), "host-only"),
    (dict(), "host-only"), (dict(nf=1, qi=0x100002), "host-only"),
])
def test_refusals(pool, kw, word):
    rc, msg = call(pool, **kw)
    assert rc == INVALID_ARG and word in msg, (rc, msg)


def test_null_pool_and_no_rows(pool):
    assert call(None)[0] == INVALID_ARG
    assert call(pool, rows=0, pos=0, inv=0, qi=0, qo=0, ki=0, ko=0)[0] == 0


def test_binding_refuses_host_only_pools(pool):
    with pytest.raises(ValueError, match="host-only"):
        pool.rope(None, None, None, None)

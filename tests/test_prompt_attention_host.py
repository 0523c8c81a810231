"""The argument contract of mkv_prompt_attention, called through ctypes on the CPU: every refusal
comes before any device call, and a call that passes them all is refused last because a host-only
pool has no device."""
import ctypes

import pytest

from mixed_format_paged_mkv_b200 import Pool
from mixed_format_paged_mkv_b200.api import lib

INVALID_ARG, UNSUPPORTED = -1, -10
HKV, D = 2, 64


def call(pool, lens=(5,), hq=4, scale=0.1, q=0x10000, k=0x20000, v=0x30000, out=0x40000, qs=None, ks=None, vs=None,
         n=None):
    arr = (ctypes.c_int32 * max(len(lens), 1))(*lens)
    P = ctypes.c_void_p
    rc = lib().mkv_prompt_attention(pool.handle, arr if lens else None, len(lens) if n is None else n, P(q),
                                    hq * D if qs is None else qs, P(k), HKV * D if ks is None else ks, P(v),
                                    HKV * D if vs is None else vs, hq, scale, P(out), None)
    return rc, lib().mkv_last_error().decode()


@pytest.fixture(scope="module")
def pool():
    return Pool(HKV, D, 1, 1, 1, 1, host_only=True)


def test_null_pool():
    assert lib().mkv_prompt_attention(None, None, 0, None, 0, None, 0, None, 0, 4, 0.1, None, None) == INVALID_ARG


@pytest.mark.parametrize("kw,code,word", [
    (dict(n=-1), INVALID_ARG, "prompt list"),
    (dict(lens=(), n=2), INVALID_ARG, "prompt list"),
    (dict(lens=(3, -1)), INVALID_ARG, "negative"),
    (dict(hq=3), INVALID_ARG, "multiple"),
    (dict(hq=0), INVALID_ARG, "multiple"),
    (dict(hq=-2), INVALID_ARG, "multiple"),
    (dict(hq=2 * 129), UNSUPPORTED, "not built"),
    (dict(scale=float("nan")), INVALID_ARG, "sm_scale"),
    (dict(scale=float("inf")), INVALID_ARG, "sm_scale"),
    (dict(scale=-0.5), INVALID_ARG, "sm_scale"),
    (dict(scale=65537.0), INVALID_ARG, "sm_scale"),
    (dict(scale=1e30), INVALID_ARG, "sm_scale"),
    (dict(scale=65536.0), INVALID_ARG, "host-only"),
    (dict(lens=(1 << 30, 1 << 30)), INVALID_ARG, "too many"),
    (dict(q=0), INVALID_ARG, "NULL"),
    (dict(k=0), INVALID_ARG, "NULL"),
    (dict(v=0), INVALID_ARG, "NULL"),
    (dict(out=0), INVALID_ARG, "NULL"),
    (dict(q=0x10008), INVALID_ARG, "q must be 16"),
    (dict(v=0x30002), INVALID_ARG, "v must be 16"),
    (dict(out=0x40008), INVALID_ARG, "out must be 16"),
    (dict(qs=4 * D - 8), INVALID_ARG, "q: row stride"),
    (dict(ks=2 * D + 4), INVALID_ARG, "k: row stride"),
    (dict(vs=0), INVALID_ARG, "v: row stride"),
    (dict(vs=-2 * D), INVALID_ARG, "v: row stride"),
    (dict(vs=1 << 38), INVALID_ARG, "v: row stride"),
    (dict(out=0x10000), INVALID_ARG, "overlaps q"),
    (dict(out=0x20000 + 5 * 2 * HKV * D - 16), INVALID_ARG, "overlaps k"),
    (dict(out=0x30000 - 5 * 2 * 4 * D + 16), INVALID_ARG, "overlaps v"),
    (dict(), INVALID_ARG, "host-only"),                     # nothing else is wrong
    (dict(qs=4 * D + 8, hq=4), INVALID_ARG, "host-only"),
    (dict(out=0x20000 + 5 * 2 * HKV * D), INVALID_ARG, "host-only"),
])
def test_refusals(pool, kw, code, word):
    rc, msg = call(pool, **kw)
    assert rc == code and word in msg, (rc, msg)


def test_no_tokens_is_no_work(pool):
    assert call(pool, lens=(), n=0, q=0, k=0, v=0, out=0)[0] == 0
    assert call(pool, lens=(0, 0), q=0, k=0, v=0, out=0)[0] == 0


def test_binding_refuses_host_only_pools_and_host_tensors(pool):
    torch = pytest.importorskip("torch")
    x = torch.zeros((5, HKV, D), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="host-only"):
        pool.prompt_attention(x, x, x, (5,))

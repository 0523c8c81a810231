"""On which device and stream the pool's calls run (CPU, a runtime that writes its calls down): all of
them on the device of the pool's buffers, whichever is current, and without a given stream on that
device's current one."""
import ctypes

import pytest
import torch

from mixed_format_paged_mkv_b200 import api

from fake_runtime import build, device_pool, log


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return build(tmp_path_factory.mktemp("fake"))


class FakeStream:
    def __init__(self, value):
        self.cuda_stream = value


@pytest.fixture
def pool(lib, monkeypatch):
    """A pool on device 1 while device 0 is current; the current stream of device d is 4096 + d."""
    monkeypatch.setattr(api, "_lib", lib)
    monkeypatch.setattr(api, "_dev_ptr", lambda t, *_: ctypes.c_void_p(t.data_ptr()))
    monkeypatch.setattr(api, "_rows_ptr", lambda t, heads, dim, *_: (t.data_ptr(), heads * dim, t.shape[0]))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 4096 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: FakeStream(4096 + (d or 0)))
    lib.fake_devices(0, 1)
    log(lib)
    p = device_pool(lib, 1)
    yield p
    p.close()


def rows(n, heads):
    return torch.zeros((n, heads, 64), dtype=torch.bfloat16)


def q(n, heads=4):
    return torch.zeros((n, 1, heads, 64), dtype=torch.bfloat16)


def decode(p, **kw):
    ws = torch.zeros(p.workspace_bytes([0], 1, 4) + 256, dtype=torch.uint8)
    p.decode([0], q(1), out=torch.zeros((1, 1, 4, 64)), workspace=ws[-ws.data_ptr() % 256:], **kw)


def noalloc(p):
    seqs, x, out = (ctypes.c_int32 * 1)(0), q(1), torch.zeros((1, 1, 4, 64))
    api._check(api.lib().mkv_decode_attention_noalloc(p.handle, seqs, 1, 1, x.data_ptr(), 4, 0.1, out.data_ptr(),
                                                      4096 + 1), "noalloc")


def rope(p, **kw):
    pos, inv = torch.zeros(64, dtype=torch.int32), torch.zeros(32)   # (4-byte addresses apart from q and k)
    kw = dict(q_out=rows(64, 4), k_out=rows(64, 2), **kw)
    p.rope(rows(64, 4), rows(64, 2), pos, inv, **kw)


CALLS = {
    "append": lambda p, **kw: p.append([0], [100], rows(100, 2), rows(100, 2), **kw),
    "demote": lambda p, **kw: p.demote([0], 16, **kw),
    "prefill": lambda p, **kw: p.prefill([1], [90], rows(90, 2), rows(90, 2), window=16, **kw),
    "workspace": lambda p: p.workspace_bytes([0], 1, 4),
    "plan": lambda p: p.decode_plan([0], 1, 4),
    "decode": decode,
    "noalloc": noalloc,
    "materialise": lambda p, **kw: p.materialise(0, torch.zeros((128, 2, 64)), torch.zeros((128, 2, 64)), **kw),
    "copy": lambda p, **kw: p.copy(0, 2, **kw),
    "fork": lambda p, **kw: p.fork([0], [3], **kw),
    "truncate": lambda p, **kw: p.truncate([3], [50], **kw),
    "free": lambda p, **kw: p.free([3], **kw),
    "compact": lambda p, **kw: p.compact(**kw),
    "prompt_attention": lambda p, **kw: p.prompt_attention(rows(9, 4), rows(9, 2), rows(9, 2), [9], out=rows(9, 4), **kw),
    "rope": rope,
    "read_slot": lambda p, **kw: p.read_slot(p.block_table(0)[0][0], **kw),
    "reset": lambda p, **kw: p.reset(0, **kw),
    "device_status": lambda p, **kw: p.device_status(**kw),
    "selftest_wait": lambda p, **kw: p.selftest_wait(**kw),
}
STREAMLESS = {"workspace", "plan", "noalloc"}


def prepared(p, name):
    """The pool's sequences as the call needs them; earlier calls' log is dropped."""
    if name != "append":
        CALLS["append"](p)
    if name in ("truncate", "free", "compact"):
        CALLS["fork"](p)
    if name == "compact":
        p.copy(0, 2)
        p.free([0, 3])
    log(api.lib())


@pytest.mark.parametrize("name", list(CALLS))
def test_calls_run_on_the_pools_device_and_its_current_stream(pool, lib, name):
    prepared(pool, name)
    pool.timing()                                   # (decode records events too)
    CALLS[name](pool)
    calls = log(lib)
    assert calls and {d for _, d, _ in calls} == {1}, calls
    assert lib.fake_current_device() == 0           # as the caller left it
    streams = {s for what, _, s in calls if what not in ("occupancy", "scratch", "event_create", "memcpy", "memset")}
    assert streams <= {4097}, calls


@pytest.mark.parametrize("name", sorted(set(CALLS) - STREAMLESS))
def test_a_given_stream_is_used(pool, lib, name, monkeypatch):
    class Scope:                                    # (torch.cuda.stream needs a device)
        def __init__(self, stream):
            pass
        def __enter__(self):
            return self
        def __exit__(self, *_):
            return False
    monkeypatch.setattr(torch.cuda, "stream", Scope)
    prepared(pool, name)
    CALLS[name](pool, stream=FakeStream(77))
    calls = log(lib)
    streams = {s for what, _, s in calls if what not in ("occupancy", "event_create", "memcpy", "memset")}
    assert {d for _, d, _ in calls} == {1} and streams == {77}, calls


def test_the_pool_is_set_up_on_its_device(pool, lib):
    calls = log(lib)
    assert len(calls) == 3 and {d for _, d, _ in calls} == {1}, calls


def test_the_cut_is_planned_for_the_pools_device(pool):
    """(148 SMs on a real one; the fake device 1 has 101)"""
    pool.append([0], [1000], rows(1000, 2), rows(1000, 2))
    assert pool.decode_plan([0], 1, 4)[1] == 101

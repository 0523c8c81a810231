"""A call that runs out of host memory reports it through the C ABI, throws nothing, and leaves the pool
as it was (CPU).  The library's host side is built with an allocator that fails from the n-th
allocation on, for every n until the call succeeds; the same call again then gives the tables of a
pool that never failed.  Each call runs in a process of its own, because an exception that leaves a C
entry ends it."""
import ctypes
import os
import subprocess
import sys
import traceback

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [p for p in (ROOT, os.path.join(ROOT, "tests")) if p not in sys.path]

from mixed_format_paged_mkv_b200 import MkvError, Pool, api  # noqa: E402

import fake_runtime  # noqa: E402

SEQS = 12


def host_pool():
    """Sequence 0 holds TQ3 and FP8 pages, 1 to 4 are branches of it, 5 an append of its own."""
    p = Pool(1, 64, SEQS, 400, 1200, 900, host_only=True)
    p.set_slot_order(0, np.random.default_rng(1).permutation(1200))
    p.append([0], [1600 + 5])
    p.fork([0, 0], [1, 2])
    p.demote([0], 800)
    p.fork([0, 0], [3, 4], [1600, 1603])
    p.append([5], [77])
    return p


def state(p):
    return [p.block_table(s) for s in range(SEQS)], p.stats()


def seqs(*ids):
    return (ctypes.c_int32 * len(ids))(*ids)


def decode(p, n):
    out = ctypes.c_size_t()
    api._check(api.lib().mkv_decode_workspace_bytes(p.handle, seqs(0), 1, 1, 4, ctypes.byref(out)), "workspace")
    api._check(api.lib().mkv_decode_attention(p.handle, seqs(0), 1, 1, 0x100, 4, 0.1, 0x100, 0x100, 1 << 30, None), "decode")


def prompt(p, n):
    api._check(api.lib().mkv_prompt_attention(p.handle, seqs(5, 9, 3), 3, 0x10000, 256, 0x20000, 128, 0x30000, 128, 4,
                                              0.1, 0x40000, None), "prompt")


def timed_decode(p, n):
    p.timing()
    decode(p, n)
    p.timing_read()


def create(p, n):
    Pool(1, 64, 4, 8, 16, 16, host_only=True).close()


CALLS = {
    "append": lambda p, n: p.append([0, 5, 6], [300, 1, 40]),
    "demote": lambda p, n: p.demote([1], 16),
    "demote_shared": lambda p, n: p.demote([0, 1, 2, 3, 5], 16),
    "prefill": lambda p, n: p.prefill([6, 7], [900, 33], window=64),
    "copy": lambda p, n: p.copy(3, 6),
    "fork": lambda p, n: p.fork([0, 5, 0, 1], [6, 7, 8, 9], [1605, 70, 1604, 1600]),
    "truncate": lambda p, n: p.truncate([1, 2, 4, 5], [900, 901, 1601, 3]),
    "free": lambda p, n: p.free([1, 4, 0]),
    "compact": lambda p, n: p.compact(),
    "reset": lambda p, n: p.reset(1),
    "slot_order": lambda p, n: p.set_slot_order(1, list(range(900))[::-1]),
    "plan": lambda p, n: p.decode_plan([0, 1, 5], 1, 4),
    "create": create,
    "decode": decode,
    "timed_decode": timed_decode,
    "prompt": prompt,
}
ON_A_DEVICE = {"decode", "timed_decode", "prompt"}
NO_ALLOCATION = {"reset"}


def build(lib, name):
    if name in ON_A_DEVICE:
        p = fake_runtime.device_pool(lib, 0, Hkv=2)
        kv = ctypes.c_void_p(0x1000)
        api._check(lib.mkv_append_kv(p.handle, seqs(0), seqs(900), 1, kv, kv, None), "append")
        return p
    p = host_pool()
    if name == "compact":
        p.free([1, 2, 5])
        p.set_slot_order(0, list(range(1200))[::-1])
    return p


def check(lib, name):
    call, look = CALLS[name], (lambda p: p.launch_count() * 0) if name in ON_A_DEVICE else state
    twin = build(lib, name)
    before = look(twin)
    call(twin, 0)
    after, follow_up = look(twin), None
    if name not in ON_A_DEVICE:                      # the free slots are the same too
        twin.append([10], [100])
        follow_up = state(twin)
    for n in range(1000):
        p = build(lib, name)
        lib.fake_allocations(n)
        try:
            call(p, n)
            failed = False
        except MkvError as e:
            failed = True
            assert e.name == "INVALID_ARG" and "out of host memory" in str(e), (n, str(e))
        lib.fake_allocations(-1)
        if failed:
            assert look(p) == before or name == "compact", (name, n)
            call(p, n)
        assert look(p) == after, (name, n)
        if follow_up:
            p.append([10], [100])
            assert state(p) == follow_up, (name, n)
        if not failed:
            break
    assert n > 0 or name in NO_ALLOCATION, name
    print("failures", n)


@pytest.fixture(scope="module")
def results(tmp_path_factory):
    """{call: (exit status, what it printed)}"""
    folder = tmp_path_factory.mktemp("fake")
    fake_runtime.build(folder)
    subprocess.run([sys.executable, __file__, str(folder)], check=True, timeout=600)
    return {name: (int((folder / f"{name}.status").read_text()), (folder / f"{name}.log").read_text()) for name in CALLS}


@pytest.mark.parametrize("name", list(CALLS))
def test_out_of_host_memory(results, name):
    status, text = results[name]
    assert status == 0, (status, text[-2000:])


def main(folder):
    api._lib = fake_runtime.load(os.path.join(folder, "libmkv_fake.so"))
    Pool(1, 64, 4, 8, 16, 16, host_only=True).append([0], [1])   # (the binding's imports, once for all)
    for name in CALLS:
        pid = os.fork()
        if pid == 0:
            log = os.open(os.path.join(folder, f"{name}.log"), os.O_WRONLY | os.O_CREAT)
            os.dup2(log, 1), os.dup2(log, 2)
            status = 1
            try:
                check(api._lib, name)
                status = 0
            except BaseException:
                traceback.print_exc()
            sys.stdout.flush(), sys.stderr.flush()
            os._exit(status)
        with open(os.path.join(folder, f"{name}.status"), "w") as f:
            f.write(str(os.waitpid(pid, 0)[1]))


if __name__ == "__main__":
    main(sys.argv[1])

"""The library's host side linked against a CUDA runtime that only writes down its calls
(fake_runtime.cpp), loaded through the binding's own signatures."""
import ctypes
import os
import subprocess

import numpy as np

from mixed_format_paged_mkv_b200 import Pool, api
from mixed_format_paged_mkv_b200._build import CSRC, INCLUDE, _nvcc

HERE = os.path.dirname(os.path.abspath(__file__))


def build(folder):
    out = os.path.join(str(folder), "libmkv_fake.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-fvisibility=hidden", "-Wl,-Bsymbolic",
                    f"-I{INCLUDE}", f"-I{CSRC}", f"-I{cuda}", os.path.join(CSRC, "pool.cpp"),
                    os.path.join(HERE, "fake_runtime.cpp"), "-o", out], check=True)
    return load(out)


def load(path):
    lib = ctypes.CDLL(path)
    for name, (res, args) in api.SIGNATURES.items():
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    lib.fake_log.restype = ctypes.c_char_p
    lib.fake_allocations.argtypes = [ctypes.c_long]
    lib.fake_allocations_left.restype = ctypes.c_long
    return lib


def log(lib):
    """[(call, device that was current, stream)] since the last look."""
    rows = [line.split() for line in lib.fake_log().decode().splitlines()]
    return [(name, int(device), int(stream)) for name, device, stream in rows]


def device_pool(lib, device, Hkv=2, D=64, seqs=8, pages=64, fp8=200, tq3=200):
    """A pool whose buffers (host memory that nothing reads) lie on a device of the fake runtime;
    ``api.lib()`` has to return ``lib`` already."""
    p = object.__new__(Pool)
    p.cfg = api.PoolConfig(Hkv, D, 16, seqs, pages, fp8, tq3, 1, 0)
    p.bf16_control, p.host_only, p.Hkv, p.D, p.device_index = False, False, Hkv, D, device
    sizes = [ctypes.c_size_t() for _ in range(4)]
    assert lib.mkv_pool_required_bytes(ctypes.byref(p.cfg), *[ctypes.byref(s) for s in sizes]) == 0
    p.buffers = [np.zeros(s.value + 256, np.uint8) for s in sizes]
    ptrs = [ctypes.c_void_p((b.ctypes.data + 255) // 256 * 256) for b in p.buffers]
    p.handle = ctypes.c_void_p()
    assert lib.mkv_pool_create(ctypes.byref(p.cfg), *ptrs, ctypes.byref(p.handle)) == 0
    return p

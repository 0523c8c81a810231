"""Python binding of ``libmkv.so`` (the C ABI in ``include/mkv.h``): argument marshalling only.

PyTorch supplies device memory and the current CUDA stream; every step of append, demotion
and decode runs in the library's kernels.  There is no fallback: if the library is missing or
a call fails, an exception is raised.
"""
from __future__ import annotations

import array
import ctypes
import math
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmkv.so")

FMT_FP8, FMT_TQ3, FMT_BF16 = 0, 1, 2
POOL_HOST_ONLY, POOL_BF16_CONTROL = 1, 2
ERRORS = {0: "OK", -1: "INVALID_ARG", -2: "BAD_SEQ", -3: "OUT_OF_PAGES", -4: "EMPTY_CONTEXT",
          -5: "PAGE_NOT_FULL", -6: "WORKSPACE_TOO_SMALL", -7: "CUDA", -8: "DEVICE_CHECK",
          -9: "DEVICE_TIMEOUT", -10: "UNSUPPORTED"}

# exported symbol -> (restype, argtypes)
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_I32P = ctypes.POINTER(ctypes.c_int32)
_SZP = ctypes.POINTER(ctypes.c_size_t)


class PoolConfig(ctypes.Structure):
    _fields_ = [("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_seqs", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("fp8_slots", ctypes.c_int32),
                ("tq3_slots", ctypes.c_int32), ("sink_pages", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


SIGNATURES = {
    "mkv_pool_required_bytes": (ctypes.c_int, [ctypes.POINTER(PoolConfig), _SZP, _SZP, _SZP, _SZP]),
    "mkv_pool_create": (ctypes.c_int, [ctypes.POINTER(PoolConfig), _P, _P, _P, _P,
                                       ctypes.POINTER(_P)]),
    "mkv_pool_destroy": (None, [_P]),
    "mkv_pool_set_slot_order": (ctypes.c_int, [_P, _I32, _I32P, _I32]),
    "mkv_append_kv": (ctypes.c_int, [_P, _I32P, _I32P, _I32, _P, _P, _P]),
    "mkv_set_protected": (ctypes.c_int, [_P, _I32, _I32, _I32]),
    "mkv_demote_pages": (ctypes.c_int, [_P, _I32P, _I32, _I32, _I32P, _P]),
    "mkv_decode_workspace_bytes": (ctypes.c_int, [_P, _I32P, _I32, _I32, _I32, _SZP]),
    "mkv_decode_plan": (ctypes.c_int, [_P, _I32P, _I32, _I32, _I32, _I32P, _I32, _I32P, _I32P]),
    "mkv_decode_attention": (ctypes.c_int, [_P, _I32P, _I32, _I32, _P, _I32, ctypes.c_float,
                                            _P, _P, ctypes.c_size_t, _P]),
    "mkv_decode_attention_noalloc": (ctypes.c_int, [_P, _I32P, _I32, _I32, _P, _I32,
                                                    ctypes.c_float, _P, _P]),
    "mkv_seq_reset": (ctypes.c_int, [_P, _I32, _P]),
    "mkv_seq_copy": (ctypes.c_int, [_P, _I32, _I32, _P]),
    "mkv_seq_fork": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P]),
    "mkv_seq_truncate": (ctypes.c_int, [_P, _P, _P, _I32, _P]),
    "mkv_seq_free": (ctypes.c_int, [_P, _P, _I32, _P]),
    "mkv_pool_compact": (ctypes.c_int, [_P, _I32P, _P]),
    "mkv_materialise_kv": (ctypes.c_int, [_P, _I32, _P, _P, ctypes.c_int64, _P]),
    "mkv_prefill_kv": (ctypes.c_int, [_P, _I32P, _I32P, _I32, _P, _P, _I32, _P]),
    "mkv_rope": (ctypes.c_int, [_P, _I64, _P, _I32, _P, _I32, _P, _I32, _P, _I64, _P, _I64, _I32,
                                _P, _I64, _P, _I64, _P]),
    "mkv_prompt_attention": (ctypes.c_int, [_P, _P, _I32, _P, _I64, _P, _I64, _P, _I64, _I32,
                                            ctypes.c_float, _P, _P]),
    "mkv_selftest_wait": (ctypes.c_int, [_P, ctypes.c_int64, _P]),
    "mkv_selftest_tc_logits": (ctypes.c_int, [_P, _P, _P, _P, _P]),
    "mkv_get_block_table": (ctypes.c_int, [_P, _I32, _I32P, _I32, _I32P, _I32P]),
    "mkv_slot_bytes": (ctypes.c_int, [_P, _I32, _SZP]),
    "mkv_read_slot": (ctypes.c_int, [_P, _I32, _P, ctypes.c_size_t, _P]),
    "mkv_pool_stats": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_int64), _I32P, _I32P,
                                      ctypes.POINTER(ctypes.c_double)]),
    "mkv_get_device_status": (ctypes.c_int, [_P, _P]),
    "mkv_timing_enable": (ctypes.c_int, [_P, _I32]),
    "mkv_timing_read": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_double),
                                       ctypes.POINTER(ctypes.c_double),
                                       ctypes.POINTER(ctypes.c_int64)]),
    "mkv_launch_count": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_int64)]),
    "mkv_test_fail_launch": (ctypes.c_int, [_P, _I32]),
    "mkv_set_decode_kernels": (ctypes.c_int, [_P, _I32]),
    "mkv_set_decode_sms": (ctypes.c_int, [_P, _I32]),
    "mkv_last_error": (ctypes.c_char_p, []),
}

_lib = None


class MkvError(RuntimeError):
    def __init__(self, code: int, fn: str, msg: str):
        super().__init__(f"{fn} -> {ERRORS.get(code, code)}: {msg}")
        self.code = code
        self.name = ERRORS.get(code, str(code))


def lib():
    """Load libmkv.so (built in-tree by ``_build.py``); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run "
                               "`python -m mixed_format_paged_mkv_b200._build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(rc: int, fn: str):
    if rc != 0:
        raise MkvError(rc, fn, lib().mkv_last_error().decode())


def _i32_array(xs):
    a = np.ascontiguousarray(np.asarray(xs, dtype=np.int32))
    return a, a.ctypes.data_as(_I32P)


def _dev_ptr(t, dtype, name, device):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device >= 0 and t.get_device() != device:  # (a host-only pool has none)
        raise ValueError(f"{name} is on {t.device}, the pool on cuda:{device}")
    return ctypes.c_void_p(t.data_ptr())


def _rows_ptr(t, heads, dim, name, device):
    """Address, row stride (elements) and rows of a bf16 [rows, heads, dim] tensor whose rows are
    contiguous but may be further apart, such as a part of a fused projection's output."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the pool on cuda:{device}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be [rows, {heads}, {dim}]")
    if shape[0] and (stride[2] != 1 or (heads > 1 and stride[1] != dim)):
        raise ValueError(f"{name}: each row must be contiguous")
    return t.data_ptr(), stride[0] if shape[0] > 1 else heads * dim, shape[0]


def _empty_like(t, shape, stream, dtype=None, returned=True):
    """A new tensor of t's device (and type) from the memory of the stream that will write it: memory of
    another stream could be given out there again, or still be in use there, while this one's kernels
    work on it.  What the caller gets is also held for the caller's current stream, which usually reads
    it: given up, its memory waits for both."""
    import torch
    if stream is None:
        return t.new_empty(shape) if dtype is None else t.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        new = t.new_empty(shape, dtype=dtype or t.dtype)
    if returned:
        new.record_stream(torch.cuda.current_stream(t.device))
    return new


def _i32_list(xs):
    """(address, length, owner) of a list's int32 values on the host; the owner keeps them alive.
    Anything but whole numbers that fit is refused: a converted one would cut or free another part."""
    if isinstance(xs, (list, tuple)):
        try:
            a = array.array("i", xs)
            return a.buffer_info()[0], len(a), a
        except (TypeError, OverflowError):  # nested lists or no integers: numpy tells them apart
            pass
    a = np.asarray(xs)
    if a.size and (a.dtype.kind not in "iu" or a.max() > 2 ** 31 - 1 or a.min() < -2 ** 31):
        raise ValueError(f"{xs!r} must hold whole numbers that fit int32")
    a = np.ascontiguousarray(a, dtype=np.int32).reshape(-1)
    return a.ctypes.data, a.size, a


class Pool:
    """A mixed-format paged KV cache over device buffers owned by this object (torch)."""

    def __init__(self, num_kv_heads, head_dim, max_seqs, max_pages_per_seq, fp8_slots,
                 tq3_slots, sink_pages=1, device=None, host_only=False, bf16_control=False):
        flags = (POOL_HOST_ONLY if host_only else 0) | (POOL_BF16_CONTROL if bf16_control else 0)
        self.cfg = PoolConfig(num_kv_heads, head_dim, 16, max_seqs, max_pages_per_seq,
                              fp8_slots, tq3_slots, sink_pages, flags)
        self.bf16_control = bf16_control
        self.Hkv, self.D = num_kv_heads, head_dim
        self.host_only = host_only
        self.device_index = -1
        L = lib()
        sizes = [ctypes.c_size_t() for _ in range(4)]
        _check(L.mkv_pool_required_bytes(ctypes.byref(self.cfg), *[ctypes.byref(s) for s in sizes]),
               "mkv_pool_required_bytes")
        self.bytes = [s.value for s in sizes]
        handle = ctypes.c_void_p()
        if host_only:
            self.buffers = None
            ptrs = [None, None, None, None]
        else:
            import torch
            dev = torch.device(device or "cuda")
            self.buffers = [torch.empty(max(b, 256), dtype=torch.uint8, device=dev)
                            for b in self.bytes]
            ptrs = [ctypes.c_void_p(b.data_ptr()) for b in self.buffers]
            self.device_index = self.buffers[0].get_device()
        _check(L.mkv_pool_create(ctypes.byref(self.cfg), *ptrs, ctypes.byref(handle)),
               "mkv_pool_create")
        self.handle = handle

    # ------------------------------------------------------------------ lifecycle
    def close(self):
        if getattr(self, "handle", None) and self.handle.value:
            lib().mkv_pool_destroy(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------------ calls
    def set_slot_order(self, fmt, order):
        a, p = _i32_array(order)
        _check(lib().mkv_pool_set_slot_order(self.handle, fmt, p, a.size), "mkv_pool_set_slot_order")

    def append(self, seq_ids, n_new, k=None, v=None, stream=None):
        import torch
        s, sp = _i32_array(seq_ids)
        n, np_ = _i32_array(n_new)
        if self.host_only:
            kp = vp = None
            st = None
        else:
            kp = _dev_ptr(k, torch.bfloat16, "k", self.device_index)
            vp = _dev_ptr(v, torch.bfloat16, "v", self.device_index)
            rows = int(n.sum())
            if tuple(k.shape) != (rows, self.Hkv, self.D) or tuple(v.shape) != (rows, self.Hkv, self.D):
                raise ValueError(f"k, v must be [{rows}, {self.Hkv}, {self.D}]")
            st = self._stream(stream)
        _check(lib().mkv_append_kv(self.handle, sp, np_, s.size, kp, vp, st), "mkv_append_kv")

    def prefill(self, seq_ids, n_tokens, k=None, v=None, window=0, stream=None):
        """First tokens of empty sequences; full pages the anchor policy would demote at once
        are packed to TQ3 straight from bf16 (mkv_prefill_kv)."""
        import torch
        s, sp = _i32_array(seq_ids)
        n, np_ = _i32_array(n_tokens)
        if self.host_only:
            kp = vp = None
            st = None
        else:
            kp = _dev_ptr(k, torch.bfloat16, "k", self.device_index)
            vp = _dev_ptr(v, torch.bfloat16, "v", self.device_index)
            rows = int(n.sum())
            if tuple(k.shape) != (rows, self.Hkv, self.D) or tuple(v.shape) != (rows, self.Hkv, self.D):
                raise ValueError(f"k, v must be [{rows}, {self.Hkv}, {self.D}]")
            st = self._stream(stream)
        _check(lib().mkv_prefill_kv(self.handle, sp, np_, s.size, kp, vp, int(window), st),
               "mkv_prefill_kv")

    def selftest_wait(self, limit_ns=1_000_000, stream=None):
        """Launch the bounded-wait self-test; the next device_status() raises DEVICE_TIMEOUT."""
        st = self._stream(stream)
        _check(lib().mkv_selftest_wait(self.handle, int(limit_ns), st), "mkv_selftest_wait")

    def selftest_tc_logits(self, a, q, stream=None):
        """fp32 [128, 8] = a [128, 256] . q [8, 256]^T (f16 device tensors) through tensor memory
        and tcgen05.mma (mkv_selftest_tc_logits)."""
        import torch
        if tuple(a.shape) != (128, 256) or tuple(q.shape) != (8, 256):
            raise ValueError("a must be [128, 256] and q [8, 256]")
        d = _empty_like(a, (128, 8), stream, torch.float32)
        dev = self.device_index
        _check(lib().mkv_selftest_tc_logits(self.handle, _dev_ptr(a, torch.float16, "a", dev),
                                            _dev_ptr(q, torch.float16, "q", dev),
                                            _dev_ptr(d, torch.float32, "d", dev), self._stream(stream)),
               "mkv_selftest_tc_logits")
        return d

    def set_protected(self, seq, page, flag=True):
        _check(lib().mkv_set_protected(self.handle, seq, page, 1 if flag else 0), "mkv_set_protected")

    def demote(self, seq_ids, window_tokens, stream=None):
        s, sp = _i32_array(seq_ids)
        n = ctypes.c_int32(0)
        st = self._stream(stream)
        _check(lib().mkv_demote_pages(self.handle, sp, s.size, window_tokens, ctypes.byref(n), st),
               "mkv_demote_pages")
        return n.value

    def workspace_bytes(self, seq_ids, q_len, num_q_heads):
        s, sp = _i32_array(seq_ids)
        b = ctypes.c_size_t()
        _check(lib().mkv_decode_workspace_bytes(self.handle, sp, s.size, q_len, num_q_heads,
                                                ctypes.byref(b)), "mkv_decode_workspace_bytes")
        return b.value

    def decode_plan(self, seq_ids, q_len, num_q_heads):
        """The work units a decode call would cut (mkv_decode_plan): int32 [units, 6] rows of
        (call position, format, first logical page, end logical page, pages of that format, CTA),
        CTA by CTA, and the CTA budget of one wave."""
        s, sp = _i32_array(seq_ids)
        n, wave = ctypes.c_int32(), ctypes.c_int32()
        _check(lib().mkv_decode_plan(self.handle, sp, s.size, q_len, num_q_heads, None, 0,
                                     ctypes.byref(n), ctypes.byref(wave)), "mkv_decode_plan")
        u = np.zeros((max(n.value, 1), 6), dtype=np.int32)
        _check(lib().mkv_decode_plan(self.handle, sp, s.size, q_len, num_q_heads,
                                     u.ctypes.data_as(_I32P), n.value, ctypes.byref(n), None),
               "mkv_decode_plan")
        return u[:n.value], wave.value

    def decode(self, seq_ids, q, sm_scale=None, out=None, workspace=None, stream=None):
        """q: bf16 [n, q_len, Hq, D] on the device -> fp32 [n, q_len, Hq, D]."""
        import torch
        s, sp = _i32_array(seq_ids)
        n, q_len, Hq, D = q.shape
        if n != s.size or D != self.D:
            raise ValueError("q must be [len(seq_ids), q_len, Hq, head_dim]")
        qp = _dev_ptr(q, torch.bfloat16, "q", self.device_index)
        if out is None:
            out = _empty_like(q, (n, q_len, Hq, D), stream, torch.float32)
        op = _dev_ptr(out, torch.float32, "out", self.device_index)
        if workspace is None:   # the library checks a caller-given workspace's size itself
            workspace = _empty_like(q, (self.workspace_bytes(s, q_len, Hq),), stream, torch.uint8, returned=False)
        wp = _dev_ptr(workspace, torch.uint8, "workspace", self.device_index)
        scale = 1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale)
        _check(lib().mkv_decode_attention(self.handle, sp, s.size, q_len, qp, Hq,
                                          ctypes.c_float(scale), op, wp, workspace.numel(),
                                          self._stream(stream)), "mkv_decode_attention")
        return out

    def _stream(self, stream):
        """The given stream (of the pool's device), or the current one of the pool's device."""
        import torch
        if self.host_only:
            return None
        if stream is not None:
            return stream.cuda_stream
        return torch._C._cuda_getCurrentRawStream(self.device_index)

    def rope(self, q, k, positions, inv_freq, axes=None, interleaved=False, q_out=None, k_out=None,
             stream=None):
        """Rotate q bf16 [rows, Hq, D] and k bf16 [rows, Hkv, D] (rows may be strided) by
        ``positions`` (int32 [rows] or [n_axes, rows]) times ``inv_freq`` (fp32 [n_freq]); ``axes``
        lists the axis of each frequency (default: axis 0 for all of them).  Pairs are channels n_freq apart, or
        neighbours when ``interleaved``.  Returns (q_out, k_out): new tensors unless given; the
        inputs themselves for a rotation in place (mkv_rope)."""
        import torch
        if self.host_only:
            raise ValueError("host-only pools have no device")
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be [rows, Hq, head_dim]")
        Hq, Hkv, D, dev = q.shape[1], self.Hkv, self.D, self.device_index
        qp, qs, rows = _rows_ptr(q, Hq, D, "q", dev)
        kp, ks, k_rows = _rows_ptr(k, Hkv, D, "k", dev)
        if q_out is None:
            q_out = _empty_like(q, (rows, Hq, D), stream)
            qo, qos, q_rows = q_out.data_ptr(), Hq * D, rows
        else:
            qo, qos, q_rows = _rows_ptr(q_out, Hq, D, "q_out", dev)
        if k_out is None:
            k_out = _empty_like(k, (rows, Hkv, D), stream)
            ko, kos, o_rows = k_out.data_ptr(), Hkv * D, rows
        else:
            ko, kos, o_rows = _rows_ptr(k_out, Hkv, D, "k_out", dev)
        if k_rows != rows or q_rows != rows or o_rows != rows:
            raise ValueError(f"q, k and the outputs must all have {rows} rows")
        pp = _dev_ptr(positions, torch.int32, "positions", dev)
        fp = _dev_ptr(inv_freq, torch.float32, "inv_freq", dev)
        n_axes = positions.shape[0] if positions.dim() == 2 else 1
        if positions.dim() not in (1, 2) or positions.shape[-1] != rows or inv_freq.dim() != 1:
            raise ValueError(f"positions must be [{rows}] or [n_axes, {rows}], inv_freq [n_freq]")
        n_freq = inv_freq.shape[0]
        a = None
        if axes is not None:
            a, n, keep = _i32_list(axes)
            if n != n_freq:
                raise ValueError("axes must list an axis per frequency")
        _check(lib().mkv_rope(self.handle, rows, pp, n_axes, fp, n_freq, a, 1 if interleaved else 0,
                              qp, qs, qo, qos, Hq, kp, ks, ko, kos, self._stream(stream)), "mkv_rope")
        return q_out, k_out

    def prompt_attention(self, q, k, v, n_tokens, sm_scale=None, out=None, stream=None):
        """Causal attention over packed prompts of ``n_tokens`` tokens each: q bf16 [rows, Hq, D],
        k and v bf16 [rows, Hkv, D] (rows may be strided) -> bf16 [rows, Hq, D].  Rows beyond
        sum(n_tokens) are ignored, and in a given ``out`` left as they were
        (mkv_prompt_attention)."""
        import torch
        if self.host_only:
            raise ValueError("host-only pools have no device")
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be [rows, Hq, head_dim]")
        n, count, lens = _i32_list(n_tokens)
        Hq, D, dev = q.shape[1], self.D, self.device_index
        rows = int(sum(lens))  # (the library refuses a negative count)
        qp, qs, q_rows = _rows_ptr(q, Hq, D, "q", dev)
        kp, ks, k_rows = _rows_ptr(k, self.Hkv, D, "k", dev)
        vp, vs, v_rows = _rows_ptr(v, self.Hkv, D, "v", dev)
        if q_rows < rows or k_rows < rows or v_rows < rows:
            raise ValueError(f"q, k and v must have the {rows} rows of n_tokens")
        if out is None:
            out = _empty_like(q, (q_rows, Hq, D), stream)
            op = out.data_ptr()
        else:
            op, _, o_rows = _rows_ptr(out, Hq, D, "out", dev)
            if o_rows < rows or not out.is_contiguous():
                raise ValueError(f"out must be contiguous with the {rows} rows of n_tokens")
        scale = D ** -0.5 if sm_scale is None else float(sm_scale)
        _check(lib().mkv_prompt_attention(self.handle, n, count, qp, qs, kp, ks, vp, vs, Hq, scale, op,
                                          self._stream(stream)), "mkv_prompt_attention")
        return out

    def reset(self, seq, stream=None):
        st = self._stream(stream)
        _check(lib().mkv_seq_reset(self.handle, seq, st), "mkv_seq_reset")

    def copy(self, src, dst, stream=None):
        st = self._stream(stream)
        _check(lib().mkv_seq_copy(self.handle, src, dst, st), "mkv_seq_copy")

    def fork(self, src_ids, dst_ids, n_tokens=None, stream=None):
        """Give each empty sequence of ``dst_ids`` the first tokens (default: all) of its source,
        sharing full pages copy-on-write (mkv_seq_fork)."""
        s, ns, _s = _i32_list(src_ids)
        d, nd, _d = _i32_list(dst_ids)
        n, nn, _n = (None, ns, None) if n_tokens is None else _i32_list(n_tokens)
        if nd != ns or nn != ns:
            raise ValueError("src_ids, dst_ids and n_tokens must have the same length")
        st = self._stream(stream)
        _check(lib().mkv_seq_fork(self.handle, s, d, n, ns, st), "mkv_seq_fork")

    def truncate(self, seq_ids, n_tokens, stream=None):
        """Roll sequences back to their first ``n_tokens`` tokens (mkv_seq_truncate)."""
        s, ns, _s = _i32_list(seq_ids)
        n, nn, _n = _i32_list(n_tokens)
        if nn != ns:
            raise ValueError("seq_ids and n_tokens must have the same length")
        st = self._stream(stream)
        _check(lib().mkv_seq_truncate(self.handle, s, n, ns, st), "mkv_seq_truncate")

    def free(self, seq_ids, stream=None):
        """Free every page of several sequences (mkv_seq_free)."""
        s, ns, _s = _i32_list(seq_ids)
        st = self._stream(stream)
        _check(lib().mkv_seq_free(self.handle, s, ns, st), "mkv_seq_free")

    def compact(self, stream=None):
        """Move pages so that the slots in use are the first ones of each slab's order; returns
        the number of pages moved (mkv_pool_compact)."""
        n = ctypes.c_int32(0)
        st = self._stream(stream)
        _check(lib().mkv_pool_compact(self.handle, ctypes.byref(n), st), "mkv_pool_compact")
        return n.value

    def materialise(self, seq, k_out=None, v_out=None, stream=None):
        """Dense fp32 dequantised K and V of a sequence, [ctx, Hkv, D] each (a debugging and
        quality-control path; decode never uses it)."""
        if self.host_only:  # the library rejects it (no device pages)
            _check(lib().mkv_materialise_kv(self.handle, seq, None, None, 0, None),
                   "mkv_materialise_kv")
        import torch
        _, ctx = self.block_table(seq)
        shape = (ctx, self.Hkv, self.D)
        k_out = _empty_like(self.buffers[0], shape, stream, torch.float32) if k_out is None else k_out
        v_out = _empty_like(self.buffers[0], shape, stream, torch.float32) if v_out is None else v_out
        kp = _dev_ptr(k_out, torch.float32, "k_out", self.device_index)
        vp = _dev_ptr(v_out, torch.float32, "v_out", self.device_index)
        cap = min(k_out.numel(), v_out.numel()) // (self.Hkv * self.D)
        _check(lib().mkv_materialise_kv(self.handle, seq, kp, vp, cap, self._stream(stream)),
               "mkv_materialise_kv")
        return k_out, v_out

    def block_table(self, seq):
        n = ctypes.c_int32()
        ctx = ctypes.c_int32()
        _check(lib().mkv_get_block_table(self.handle, seq, None, 0, ctypes.byref(n), ctypes.byref(ctx)),
               "mkv_get_block_table")
        a = np.zeros(max(n.value, 1), dtype=np.int32)
        _check(lib().mkv_get_block_table(self.handle, seq, a.ctypes.data_as(_I32P), n.value, None, None),
               "mkv_get_block_table")
        return a[:n.value].tolist(), ctx.value

    def slot_bytes(self, fmt):
        b = ctypes.c_size_t()
        _check(lib().mkv_slot_bytes(self.handle, fmt, ctypes.byref(b)), "mkv_slot_bytes")
        return b.value

    def read_slot(self, entry, stream=None):
        nb = self.slot_bytes((entry >> 30) & 3)  # format tag (a BF16 entry is negative)
        buf = np.zeros(nb, dtype=np.uint8)
        _check(lib().mkv_read_slot(self.handle, entry, buf.ctypes.data_as(_P), nb,
                                   self._stream(stream)), "mkv_read_slot")
        return buf

    def stats(self):
        live = ctypes.c_int64()
        n8 = ctypes.c_int32()
        n3 = ctypes.c_int32()
        bpt = ctypes.c_double()
        _check(lib().mkv_pool_stats(self.handle, ctypes.byref(live), ctypes.byref(n8),
                                    ctypes.byref(n3), ctypes.byref(bpt)), "mkv_pool_stats")
        return live.value, n8.value, n3.value, bpt.value

    def device_status(self, stream=None):
        """Raise MkvError if a kernel flagged an invalid entry/input or a timed-out wait."""
        _check(lib().mkv_get_device_status(self.handle, self._stream(stream)), "mkv_get_device_status")

    def timing(self, enable=True):
        _check(lib().mkv_timing_enable(self.handle, 1 if enable else 0), "mkv_timing_enable")

    def timing_read(self):
        """{'partial_ms', 'merge_ms': summed device time of each decode kernel, 'calls'}."""
        v = [ctypes.c_double(), ctypes.c_double()]
        n = ctypes.c_int64()
        _check(lib().mkv_timing_read(self.handle, ctypes.byref(v[0]), ctypes.byref(v[1]),
                                     ctypes.byref(n)), "mkv_timing_read")
        return dict(partial_ms=v[0].value, merge_ms=v[1].value, calls=n.value)

    def set_decode_kernels(self, fused):
        """Decode with one fused partial grid (True), a grid per page format (False) or the
        automatic per-call choice (None, the default)."""
        mode = 2 if fused is None else (1 if fused else 0)
        _check(lib().mkv_set_decode_kernels(self.handle, mode), "mkv_set_decode_kernels")

    def set_decode_sms(self, sms):
        """Plan later decode calls for at most ``sms`` SMs (0: all of the device's)."""
        _check(lib().mkv_set_decode_sms(self.handle, int(sms)), "mkv_set_decode_sms")

    def test_fail_launch(self, after):
        """Make the device operation after the next ``after`` ones fail (test hook; -1: off)."""
        _check(lib().mkv_test_fail_launch(self.handle, int(after)), "mkv_test_fail_launch")

    def launch_count(self):
        n = ctypes.c_int64()
        _check(lib().mkv_launch_count(self.handle, ctypes.byref(n)), "mkv_launch_count")
        return n.value

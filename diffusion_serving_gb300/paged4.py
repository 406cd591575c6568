"""Python binding of the 4-bit paged cache (include/kvc_paged4.h): argument marshalling only.

``PagedKVCache4`` is used as ``paged.PagedKVCache`` is, with one pool of 4-bit records in the place of two of 16-bit pages:

    cache = paged4.PagedKVCache4(batch, 32, 8, 128, torch.bfloat16, page_size=16, n_pages=4096, max_pages=256)
    cache.block_table[b, :n] = pages          # the caller's allotment
    cache.kv_len += new                       # tokens of each row, the new ones included
    q = cache.append(k, v, rope=table, q=q)
    out = cache.attend(q)
    k_held, v_held = cache.read(n)            # what is held of each row's last slots
    assert cache.get_error() == 0
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

from . import kvc, paged
from .kvc import CODE_DTYPE, ERR_ARG, ERR_DEVICE, OK, KvcError
from .paged import _current_stream, _dense, kvc_paged_config, kvc_rope_axes, make_config

HEADER_PATH = os.path.join(os.path.dirname(kvc.HEADER_PATH), "kvc_paged4.h")


def _bind():
    P, I32, I64, U32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t
    cfgp = ctypes.POINTER(kvc_paged_config)
    sig = {
        "kvc_paged4_page_bytes": (SZ, [cfgp]),
        "kvc_paged4_workspace_bytes": (SZ, [cfgp]),
        "kvc_paged4_create": (ctypes.c_int, [cfgp, P, P, P, P, P, ctypes.POINTER(P)]),
        "kvc_paged4_append": (ctypes.c_int, [P, P, P, I64, P, I64, P, I32, P, P, I32, ctypes.POINTER(kvc_rope_axes), P, U32, P]),
        "kvc_paged4_read": (ctypes.c_int, [P, P, P, I32, P, P]),
        "kvc_paged4_attend": (ctypes.c_int, [P, P, P, P, I32, P, I32, U32, P]),
        "kvc_paged4_get_error": (ctypes.c_int, [P, P, ctypes.POINTER(I32)]),
        "kvc_paged4_debug_stall_waits": (ctypes.c_int, [P, ctypes.c_uint64]),
        "kvc_paged4_destroy": (ctypes.c_int, [P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(kvc._lib, name)
        fn.restype, fn.argtypes = res, args


_bind()
_lib = kvc._lib


def header_functions() -> list[str]:
    """Names of the functions include/kvc_paged4.h declares."""
    with open(HEADER_PATH) as f:
        return re.findall(r"^(?:int|size_t)\s+(kvc_paged4_\w+)\s*\(", f.read(), flags=re.M)


def kvc_paged4_page_bytes(cfg: kvc_paged_config) -> int:
    return _lib.kvc_paged4_page_bytes(ctypes.byref(cfg))


def kvc_paged4_workspace_bytes(cfg: kvc_paged_config) -> int:
    return _lib.kvc_paged4_workspace_bytes(ctypes.byref(cfg))


def kvc_paged4_create(cfg, pages, table, kv_len, workspace, stream=None) -> int:
    h = ctypes.c_void_p()
    kvc._check(_lib.kvc_paged4_create(ctypes.byref(cfg), kvc._ptr(pages), kvc._ptr(table), kvc._ptr(kv_len),
                                      kvc._ptr(workspace), kvc._stream(stream), ctypes.byref(h)), "kvc_paged4_create")
    return h.value


def kvc_paged4_get_error(h: int, stream=None) -> int:
    """The device error bits (0 if none), cleared."""
    bits = ctypes.c_int32(0)
    rc = _lib.kvc_paged4_get_error(h, kvc._stream(stream), ctypes.byref(bits))
    if rc not in (OK, ERR_DEVICE):
        raise KvcError(rc, "kvc_paged4_get_error")
    return bits.value


def kvc_paged4_debug_stall_waits(h: int, ns: int) -> None:
    kvc._check(_lib.kvc_paged4_debug_stall_waits(h, ns), "kvc_paged4_debug_stall_waits")


def kvc_paged4_destroy(h: int) -> None:
    kvc._check(_lib.kvc_paged4_destroy(h), "kvc_paged4_destroy")


class PagedKVCache4(paged.PagedKVCache):
    """A paged cache held in 4 bits: a pool of records, each row's page numbers and length, and a handle over them.

    ``pages`` uint8 [n_pages, kv_heads, page_size * (head_dim + head_dim / 16)] (the records' layout: include/kvc_paged4.h),
    ``block_table`` and ``kv_len`` may be given.  ``dtype`` (float16 or bfloat16) is that of queries, keys, values and
    outputs.  Token rows, ``stream`` and lifetimes are as ``paged.PagedKVCache`` has them.  There is no attention over a
    shared prefix or selected pages."""

    def __init__(self, batch, heads, kv_heads, head_dim, dtype, *, page_size, n_pages, max_pages, max_tokens=0,
                 softmax_scale=0.0, pages=None, block_table=None, kv_len=None, device="cuda", stream=None):
        self.cfg = make_config(batch, heads, kv_heads, head_dim, dtype, page_size=page_size, n_pages=n_pages,
                               max_pages=max_pages, max_tokens=max_tokens, softmax_scale=softmax_scale)
        self.handle = None
        wb = kvc_paged4_workspace_bytes(self.cfg)
        if wb == 0:
            raise KvcError(ERR_ARG, "kvc_paged4_workspace_bytes")
        self.dtype = CODE_DTYPE[self.cfg.dtype]
        self.batch, self.heads, self.kv_heads, self.head_dim = batch, heads, kv_heads, head_dim
        device = torch.device(device)
        if device.index is None:
            device = torch.device(device.type, torch.cuda.current_device())
        self.device, self._index = device, device.index
        self._own, self._streams = [], {_current_stream(self._index)}    # buffers allotted here, streams they may be used on

        def own(what, t, shape, dt, fill=None):
            if t is not None:
                return _dense(what, t, shape, dt, device)
            t = torch.empty(shape, dtype=dt, device=device) if fill is None else torch.full(shape, fill, dtype=dt, device=device)
            self._own.append(t)
            return t

        record = kvc_paged4_page_bytes(self.cfg) // kv_heads
        self.pages = own("pages", pages, (n_pages, kv_heads, record), torch.uint8)
        self.block_table = own("block_table", block_table, (batch, max_pages), torch.int32, -1)
        self.kv_len = own("kv_len", kv_len, (batch,), torch.int32, 0)
        self.workspace = own("workspace", None, (wb,), torch.uint8)
        h, current = self._stream(stream), torch.cuda.current_stream(device)
        other = None if h == current.cuda_stream else kvc._stream_of(h, device)
        if other is not None:                              # (what was allotted and filled above)
            other.wait_stream(current)
        with torch.cuda.device(device):
            self.handle = kvc_paged4_create(self.cfg, self.pages, self.block_table, self.kv_len, self.workspace, h)
        if other is not None:                              # (the workspace's zeros)
            current.wait_stream(other)

    def append(self, k, v, *, cu_new=None, rope=None, half=False, q=None, q_out=None, positions=None, axes=None, stream=None):
        """As ``paged.PagedKVCache.append``; keys (once turned and rounded) and values are held in 4 bits."""
        args, q_out = self._append_args(k, v, cu_new, rope, half, q, q_out, positions, axes, stream)
        if positions is None:
            args = (*args[:10], None, None, *args[10:])
        self._call("kvc_paged4_append", _lib.kvc_paged4_append, *args)
        return q_out

    def read(self, n_tokens, *, cu=None, k_out=None, v_out=None, stream=None):
        """(k, v), [n_tokens, kv_heads, head_dim] each: what is held of each row's last slots, ``n_tokens`` in all: as many of
        every row, or row b's ``cu[b + 1] - cu[b]``."""
        shape = (n_tokens, self.kv_heads, self.head_dim)
        if cu is None and n_tokens % self.batch:
            raise ValueError(f"kvc: read takes as many tokens of each of {self.batch} rows, or cu; got {n_tokens}")
        out = []
        for what, t in (("k_out", k_out), ("v_out", v_out)):
            if t is None:
                t = kvc._empty(shape, self.dtype, self.device, stream)
            elif t.dtype is not self.dtype or t.numel() != n_tokens * self.kv_heads * self.head_dim or \
                    self._tokens(what, t, self.kv_heads) != n_tokens or not t.is_contiguous():
                raise ValueError(f"kvc: {what} must be a dense {list(shape)} {self.dtype} on {self.device}")
            out.append(t)
        self._call("kvc_paged4_read", _lib.kvc_paged4_read, out[0].data_ptr(), out[1].data_ptr(), n_tokens, self._cu(cu),
                   self._stream(stream))
        return out[0], out[1]

    def attend(self, q, *, cu_q=None, max_q=None, out=None, lse=None, flags=0, stream=None):
        """As ``paged.PagedKVCache.attend``, over the values held (flags: CAUSAL alone)."""
        n, out, lse, lse_ptr = self._q(q, out, lse, stream)
        self._call("kvc_paged4_attend", _lib.kvc_paged4_attend, q.data_ptr(), out.data_ptr(), lse_ptr, n, self._cu(cu_q),
                   n if max_q is None else max_q, flags, self._stream(stream))
        return out if lse is None else (out, lse)

    def attend_shared(self, *args, **kw):
        raise KvcError(kvc.ERR_UNSUPPORTED, "attend_shared of a 4-bit cache")

    def attend_sparse(self, *args, **kw):
        raise KvcError(kvc.ERR_UNSUPPORTED, "attend_sparse of a 4-bit cache")

    def get_error(self, stream=None) -> int:
        with torch.cuda.device(self.device):
            return kvc_paged4_get_error(self.handle, self._stream(stream))

    def close(self):
        if self.handle:
            kvc_paged4_destroy(self.handle)
            self.handle = None

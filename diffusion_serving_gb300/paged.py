"""Python binding of the paged cache (include/kvc_paged.h): argument marshalling only.

The functions carry the C names and take torch tensors and torch CUDA streams, as those of
``kvc`` do, and raise ``kvc.KvcError`` on a non-zero return code.  ``PagedKVCache`` bundles a
handle with its buffers:

    cache = paged.PagedKVCache(batch, 32, 8, 128, torch.bfloat16, page_size=16, n_pages=4096, max_pages=256)
    cache.block_table[b, :n] = pages          # the caller's allotment
    cache.kv_len += new                       # tokens of each row, the new ones included
    cache.append(k, v, rope=table, q=q, q_out=q)
    out = cache.attend(q)
    assert cache.get_error() == 0
"""
from __future__ import annotations

import ctypes
import functools
import os
import re

import torch

from . import kvc
from .kvc import (BF16, CAUSAL, CODE_DTYPE, DEV_BAD_CUSEQ, DEV_BAD_KVLEN, DEV_BAD_POS, DEV_TIMEOUT,  # noqa: F401
                  DTYPE_CODE, ERR_ARG, ERR_CUDA, ERR_DEVICE, ERR_RANGE, ERR_UNSUPPORTED, F16, F32, KERNEL_SIMT, OK,
                  KvcError)

HEADER_PATH = os.path.join(os.path.dirname(kvc.HEADER_PATH), "kvc_paged.h")
AXES_HEADER_PATH = os.path.join(os.path.dirname(kvc.HEADER_PATH), "kvc_rope_axes.h")
DEV_BAD_PAGE = 128
ROPE_HALF = 1


class kvc_paged_config(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float)]


class kvc_rope_axes(ctypes.Structure):
    _fields_ = [("n_axes", ctypes.c_int32), ("pair_axis", ctypes.c_uint8 * 64)]
    pairs = None                                           # rope_axes: how many were given; else all of a head's are meant


def rope_axes(pair_axis, n_axes=None) -> kvc_rope_axes:
    """Which axis (0 .. n_axes - 1, at most 4 of them) each of a head's D/2 rotated pairs goes by: [0] * 16 + [1] * 24 +
    [2] * 24 for sections of time, height and width side by side in heads of 128.  Made once, given to each ``append``."""
    pair_axis = [int(x) for x in pair_axis]
    n = max(pair_axis, default=0) + 1 if n_axes is None else int(n_axes)
    if not 1 <= len(pair_axis) <= 64 or not 1 <= n <= 4 or min(pair_axis) < 0 or max(pair_axis) >= n:
        raise ValueError(f"kvc: rope_axes takes an axis from 0 to {n - 1} (at most 4 axes) for each of up to 64 pairs")
    a = kvc_rope_axes(n_axes=n)
    a.pair_axis[:len(pair_axis)] = pair_axis
    a.pairs = len(pair_axis)
    return a


def _bind():
    P, I32, I64, U32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t
    cfgp = ctypes.POINTER(kvc_paged_config)
    sig = {
        "kvc_paged_workspace_bytes": (SZ, [cfgp]),
        "kvc_paged_create": (ctypes.c_int, [cfgp, P, P, P, P, P, P, P, ctypes.POINTER(P)]),
        "kvc_paged_append": (ctypes.c_int, [P, P, P, I64, P, I64, P, I32, P, P, I32, U32, P]),
        "kvc_paged_append_axes": (ctypes.c_int, [P, P, P, I64, P, I64, P, I32, P, P, I32, ctypes.POINTER(kvc_rope_axes), P,
                                                 U32, P]),
        "kvc_paged_attend": (ctypes.c_int, [P, P, P, P, I32, P, I32, U32, P]),
        "kvc_paged_attend_shared": (ctypes.c_int, [P, P, P, P, I32, P, I32, P, I32, P, U32, P]),
        "kvc_paged_attend_sparse": (ctypes.c_int, [P, P, P, P, I32, I32, I32, P, U32, P]),
        "kvc_paged_get_error": (ctypes.c_int, [P, P, ctypes.POINTER(I32)]),
        "kvc_paged_debug_stall_waits": (ctypes.c_int, [P, ctypes.c_uint64]),
        "kvc_paged_destroy": (ctypes.c_int, [P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(kvc._lib, name)
        fn.restype, fn.argtypes = res, args


_bind()
_lib = kvc._lib


def header_functions() -> list[str]:
    """Names of the functions include/kvc_paged.h declares."""
    with open(HEADER_PATH) as f:
        return re.findall(r"^\s*(?:const\s+)?\w+\**\s+\**(kvc_\w+)\s*\(", f.read(), flags=re.M)


def make_config(batch, heads, kv_heads, head_dim, dtype, *, page_size, n_pages, max_pages, max_tokens=0,
                softmax_scale=0.0) -> kvc_paged_config:
    d = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return kvc_paged_config(batch, heads, kv_heads, head_dim, page_size, n_pages, max_pages, max_tokens or batch, d,
                            softmax_scale)


def kvc_paged_workspace_bytes(cfg: kvc_paged_config) -> int:
    return _lib.kvc_paged_workspace_bytes(ctypes.byref(cfg))


def kvc_paged_create(cfg, k_pages, v_pages, bounds, table, kv_len, workspace, stream=None) -> int:
    h = ctypes.c_void_p()
    kvc._check(_lib.kvc_paged_create(ctypes.byref(cfg), kvc._ptr(k_pages), kvc._ptr(v_pages), kvc._ptr(bounds),
                                     kvc._ptr(table), kvc._ptr(kv_len), kvc._ptr(workspace), kvc._stream(stream),
                                     ctypes.byref(h)), "kvc_paged_create")
    return h.value


def kvc_paged_get_error(h: int, stream=None) -> int:
    """The device error bits (0 if none), cleared."""
    bits = ctypes.c_int32(0)
    rc = _lib.kvc_paged_get_error(h, kvc._stream(stream), ctypes.byref(bits))
    if rc not in (OK, ERR_DEVICE):
        raise KvcError(rc, "kvc_paged_get_error")
    return bits.value


def kvc_paged_debug_stall_waits(h: int, ns: int) -> None:
    kvc._check(_lib.kvc_paged_debug_stall_waits(h, ns), "kvc_paged_debug_stall_waits")


def kvc_paged_destroy(h: int) -> None:
    kvc._check(_lib.kvc_paged_destroy(h), "kvc_paged_destroy")


def _dense(what, t, shape, dtype, device):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"kvc: {what} must be a dense {list(shape)} {dtype} on {device}, got {list(t.shape)} {t.dtype} "
                         f"on {t.device}" + ("" if t.is_contiguous() else ", strided"))
    return t


# The current stream's handle without a Stream object around it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current_stream(index):
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


class PagedKVCache:
    """A paged cache: pools of pages, each row's page numbers and length, and a handle over them.

    ``k_pages`` / ``v_pages`` [n_pages, page_size, kv_heads, head_dim], ``block_table`` int32 [batch,
    max_pages], ``kv_len`` int32 [batch] and ``bounds`` [n_pages, kv_heads, 2, head_dim] (True: allot
    one; needed by ``attend_sparse``) may be given, so that layers, or handles on different streams,
    share them.  Token rows of a call are packed ([total, heads, head_dim] with ``cu`` int32 [batch + 1]) or
    even ([batch, n, heads, head_dim], or [batch * n, ...]).

    ``stream`` is where a call runs (None: the current stream).  The caller orders streams: what a call reads is ready
    there, and results are waited for before they are read on another.  Results that a call allots itself are safe to
    use on that stream and on the one that was current; the cache's own buffers are kept from reuse until the
    calls made so far are done, whichever streams they ran on.  Buffers passed in are the caller's to keep."""

    def __init__(self, batch, heads, kv_heads, head_dim, dtype, *, page_size, n_pages, max_pages, max_tokens=0,
                 bounds=None, softmax_scale=0.0, k_pages=None, v_pages=None, block_table=None, kv_len=None,
                 device="cuda", stream=None):
        self.cfg = make_config(batch, heads, kv_heads, head_dim, dtype, page_size=page_size, n_pages=n_pages,
                               max_pages=max_pages, max_tokens=max_tokens, softmax_scale=softmax_scale)
        self.handle = None
        wb = kvc_paged_workspace_bytes(self.cfg)
        if wb == 0:
            raise KvcError(ERR_ARG, "kvc_paged_workspace_bytes")
        self.dtype = CODE_DTYPE[self.cfg.dtype]
        self.batch, self.heads, self.kv_heads, self.head_dim = batch, heads, kv_heads, head_dim
        device = torch.device(device)
        if device.index is None:
            device = torch.device(device.type, torch.cuda.current_device())
        self.device, self._index = device, device.index
        pool = (n_pages, page_size, kv_heads, head_dim)

        self._own, self._streams = [], {_current_stream(self._index)}    # buffers allotted here, streams they may be used on

        def own(what, t, shape, dt, fill=None):
            if t is not None:
                return _dense(what, t, shape, dt, device)
            t = torch.empty(shape, dtype=dt, device=device) if fill is None else torch.full(shape, fill, dtype=dt, device=device)
            self._own.append(t)
            return t

        self.k_pages = own("k_pages", k_pages, pool, self.dtype)
        self.v_pages = own("v_pages", v_pages, pool, self.dtype)
        self.block_table = own("block_table", block_table, (batch, max_pages), torch.int32, -1)
        self.kv_len = own("kv_len", kv_len, (batch,), torch.int32, 0)
        self.bounds = None
        if bounds is not None and bounds is not False:
            self.bounds = own("bounds", None if bounds is True else bounds, (n_pages, kv_heads, 2, head_dim), self.dtype, 0)
        self.workspace = own("workspace", None, (wb,), torch.uint8)
        h, current = self._stream(stream), torch.cuda.current_stream(device)
        other = None if h == current.cuda_stream else kvc._stream_of(h, device)
        if other is not None:                              # (what was allotted and filled above)
            other.wait_stream(current)
        with torch.cuda.device(device):
            self.handle = kvc_paged_create(self.cfg, self.k_pages, self.v_pages, self.bounds, self.block_table,
                                           self.kv_len, self.workspace, h)
        if other is not None:                              # (the workspace's zeros)
            current.wait_stream(other)

    # -- arguments ----------------------------------------------------------------------
    # (A decode step's kernels take some ten microseconds, and what these checks take comes on top of each
    # call: they look at each property once, and build messages only when one is wrong.)
    def _stream(self, stream):
        """The stream's handle; without one, the current stream of the cache's device."""
        h = _current_stream(self._index) if stream is None else stream if isinstance(stream, int) else stream.cuda_stream
        if h not in self._streams:
            s = kvc._stream_of(h, self.device)
            for t in self._own:
                t.record_stream(s)
            self._streams.add(h)
        return h

    def _call(self, what, fn, *args):
        rc = fn(self.handle, *args)
        if rc == ERR_ARG and torch.cuda.current_device() != self._index:
            with torch.cuda.device(self.device):       # (refused before anything was enqueued)
                rc = fn(self.handle, *args)
        if rc != OK:
            raise KvcError(rc, what)

    def _tokens(self, what, t, heads):
        """The number of token rows of ``t``: [total, heads, D] or [batch, n, heads, D]."""
        shape = t.shape
        if t.dtype is self.dtype and t.get_device() == self._index:
            if len(shape) == 3:
                n, h, d = shape
                if h == heads and d == self.head_dim:
                    return n
            elif len(shape) == 4:
                b, n, h, d = shape
                if h == heads and d == self.head_dim and b == self.batch:
                    return b * n
        raise ValueError(f"kvc: {what} must be [tokens, {heads}, {self.head_dim}] or [{self.batch}, n, {heads}, "
                         f"{self.head_dim}] {self.dtype} on {self.device}, got {list(shape)} {t.dtype} on {t.device}")

    def _rows(self, what, t, heads):
        """(token rows, elements from one to the next) of ``t``, whose rows are dense and evenly apart.  (The stride of a
        dimension of size 1 means nothing.)"""
        shape, s = t.shape, t.stride()
        if t.dtype is self.dtype and t.get_device() == self._index:
            if len(shape) == 3:
                n, h, d = shape
                row, head, one = s
                if h == heads and d == self.head_dim and one == 1 and (head == d or h == 1):
                    return n, row if n > 1 else h * d
            elif len(shape) == 4:
                b, m, h, d = shape
                batch, row, head, one = s
                if h == heads and d == self.head_dim and b == self.batch and one == 1 and (head == d or h == 1):
                    if m == 1:
                        return b, batch if b > 1 else h * d
                    if b == 1 or batch == m * row:
                        return b * m, row
        self._tokens(what, t, heads)                       # (says what else is wrong)
        raise ValueError(f"kvc: {what}: a token's heads must be dense and its tokens evenly apart, got strides {list(s)}")

    def _cu(self, cu):
        if cu is None:
            return None
        if cu.dtype is not torch.int32 or cu.numel() != self.batch + 1 or cu.get_device() != self._index or not cu.is_contiguous():
            raise ValueError(f"kvc: row offsets must be a dense int32 [{self.batch + 1}] on {self.device}")
        return cu.data_ptr()

    def _q(self, q, out, lse, stream):
        n = self._tokens("q", q, self.heads)
        if not q.is_contiguous():
            raise ValueError("kvc: q must be dense")
        shape = q.shape
        if out is None:
            out = kvc._empty(shape, q.dtype, q.device, stream)
        elif out.dtype is not self.dtype or out.shape != shape or out.get_device() != self._index or not out.is_contiguous():
            raise ValueError(f"kvc: out must match q ({list(shape)} {q.dtype} on {q.device}, dense)")
        if lse is None:
            return n, out, None, None
        if lse is True:
            lse = kvc._empty(shape[:-1], torch.float32, q.device, stream)
        else:
            rows = lse.shape
            if lse.dtype is not torch.float32 or len(rows) != len(shape) - 1 or rows[0] != shape[0] or \
                    rows[-1] != self.heads or lse.numel() != n * self.heads or lse.get_device() != self._index or \
                    not lse.is_contiguous():
                raise ValueError(f"kvc: lse must be a dense float32 {list(shape[:-1])}")
        return n, out, lse, lse.data_ptr()

    # -- calls --------------------------------------------------------------------------
    def append(self, k, v, *, cu_new=None, rope=None, half=False, q=None, q_out=None, positions=None, axes=None,
               stream=None):
        """Store the new tokens' keys, turned by ``rope`` [positions, D/2, 2] fp32 at their positions
        (``half``: pairs D/2 apart), and values; ``kv_len`` counts them already.  With ``q`` the queries
        of the same tokens are turned into ``q_out`` (returned; allotted when None).

        Tokens' positions are their slots, or ``positions``, int32 [tokens, axes] or [batch, n, axes]: several axes with
        ``axes`` (``rope_axes``: which of them each pair goes by), one without."""
        args, q_out = self._append_args(k, v, cu_new, rope, half, q, q_out, positions, axes, stream)
        if positions is None:
            self._call("kvc_paged_append", _lib.kvc_paged_append, *args)
        else:
            self._call("kvc_paged_append_axes", _lib.kvc_paged_append_axes, *args)
        return q_out

    def _append_args(self, k, v, cu_new, rope, half, q, q_out, positions, axes, stream):
        n, stride = self._rows("k", k, self.kv_heads)
        if v.shape != k.shape or v.stride() != k.stride() or v.dtype is not self.dtype or v.get_device() != self._index:
            nv, vstride = self._rows("v", v, self.kv_heads)
            if n != nv or stride != vstride:
                raise ValueError(f"kvc: k and v must have the same rows and strides ({n}, {stride} and {nv}, {vstride})")
        n_pos, rp = 0, None
        if rope is not None:
            s = rope.shape
            if rope.dtype is not torch.float32 or len(s) != 3 or 2 * s[1] != self.head_dim or s[2] != 2 or \
                    rope.get_device() != self._index or not rope.is_contiguous():
                raise ValueError(f"kvc: rope must be a dense float32 [positions, {self.head_dim // 2}, 2] on {self.device}")
            n_pos, rp = s[0], rope.data_ptr()
        qp = op = None
        q_stride = 0
        if q is not None:
            nq, q_stride = self._rows("q", q, self.heads)
            if nq != n:
                raise ValueError(f"kvc: q has {nq} tokens, k {n}")
            if q_out is None:
                q_out = kvc._empty(q.shape, q.dtype, q.device, stream)
            elif q_out.dtype is not self.dtype or q_out.shape != q.shape or q_out.get_device() != self._index or \
                    not q_out.is_contiguous():
                raise ValueError("kvc: q_out must be dense and match q")
            qp, op = q.data_ptr(), q_out.data_ptr()
        elif q_out is not None:
            raise ValueError("kvc: q_out without q")
        where = ()
        if positions is not None:
            where = self._positions(positions, axes, n, rope)
        elif axes is not None:
            raise ValueError("kvc: axes without positions")
        return (k.data_ptr(), v.data_ptr(), stride, qp, q_stride, op, n, self._cu(cu_new), rp, n_pos, *where,
                ROPE_HALF if half else 0, self._stream(stream)), q_out

    def _positions(self, positions, axes, n, rope):
        if axes is None:
            axes = self._one_axis
        elif not isinstance(axes, kvc_rope_axes):
            raise ValueError(f"kvc: axes are made by rope_axes, got {type(axes).__name__}")
        if axes.pairs not in (None, self.head_dim // 2):
            raise ValueError(f"kvc: axes must name an axis for each of the {self.head_dim // 2} pairs of a head, got {axes.pairs}")
        s = positions.shape
        if positions.dtype is not torch.int32 or positions.get_device() != self._index or not positions.is_contiguous() or \
                not (len(s) == 2 and s[0] == n or len(s) == 3 and s[0] == self.batch and s[0] * s[1] == n) or \
                s[-1] != axes.n_axes:
            raise ValueError(f"kvc: positions must be a dense int32 [{n}, {axes.n_axes}] (or [{self.batch}, n, {axes.n_axes}]) "
                             f"on {self.device}, got {list(s)} {positions.dtype} on {positions.device}")
        if rope is None:
            raise ValueError("kvc: positions without rope")
        return axes, positions.data_ptr()

    @functools.cached_property
    def _one_axis(self):
        return rope_axes([0] * (self.head_dim // 2))

    def attend(self, q, *, cu_q=None, max_q=None, out=None, lse=None, flags=0, stream=None):
        """Attention of every token over its row's slots.  ``max_q``: most tokens of a row (with ``cu_q``; None: as many as
        the call has in all, which is right but runs packed single tokens in the chunks' kernel: give it).
        ``lse``: a buffer, or True for a new one; then (out, lse) is returned."""
        n, out, lse, lse_ptr = self._q(q, out, lse, stream)
        self._call("kvc_paged_attend", _lib.kvc_paged_attend, q.data_ptr(), out.data_ptr(),
                   lse_ptr, n, self._cu(cu_q), n if max_q is None else max_q, flags,
                   self._stream(stream))
        return out if lse is None else (out, lse)

    def attend_shared(self, q, prefix_pages, prefix_len, *, cu_q=None, max_q=None, out=None, lse=None, flags=0,
                      stream=None):
        """``attend`` for rows whose first ``prefix_len`` (int32 [1], on the device) slots are those of
        ``prefix_pages`` (int32): they are read once for all rows."""
        n, out, lse, lse_ptr = self._q(q, out, lse, stream)
        for what, t in (("prefix_pages", prefix_pages), ("prefix_len", prefix_len)):
            if t.dtype is not torch.int32 or t.get_device() != self._index or not t.is_contiguous():
                raise ValueError(f"kvc: {what} must be a dense int32 tensor on {self.device}")
        if prefix_len.numel() != 1:
            raise ValueError("kvc: prefix_len holds one length")
        self._call("kvc_paged_attend_shared", _lib.kvc_paged_attend_shared, q.data_ptr(), out.data_ptr(),
                   lse_ptr, n, self._cu(cu_q), n if max_q is None else max_q,
                   prefix_pages.data_ptr(), prefix_pages.numel(), prefix_len.data_ptr(), flags, self._stream(stream))
        return out if lse is None else (out, lse)

    def attend_sparse(self, q, n_select, *, first=1, recent=1, out=None, lse=None, selected=None, flags=0, stream=None):
        """Attention of one token per row over ``n_select`` pages per kv head: the ``first`` and the newest
        ``recent`` ones, and those whose bounds promise the largest scores.  Returns (out, lse, selected), or
        (out, selected) without ``lse``; selected int32 [batch, kv_heads, n_select], -1 behind the last."""
        n, out, lse, lse_ptr = self._q(q, out, lse, stream)
        if n != self.batch:
            raise ValueError(f"kvc: attend_sparse takes one token per row ({self.batch}), got {n}")
        shape = (self.batch, self.kv_heads, n_select)
        if selected is None:
            selected = kvc._empty(shape, torch.int32, self.device, stream)
        elif selected.dtype is not torch.int32 or selected.shape != shape or selected.get_device() != self._index or \
                not selected.is_contiguous():
            raise ValueError(f"kvc: selected must be a dense int32 {list(shape)}")
        self._call("kvc_paged_attend_sparse", _lib.kvc_paged_attend_sparse, q.data_ptr(), out.data_ptr(),
                   lse_ptr, n_select, first, recent, selected.data_ptr(), flags,
                   self._stream(stream))
        return (out, selected) if lse is None else (out, lse, selected)

    def get_error(self, stream=None) -> int:
        with torch.cuda.device(self.device):
            return kvc_paged_get_error(self.handle, self._stream(stream))

    def close(self):
        if self.handle:
            kvc_paged_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

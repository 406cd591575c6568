"""The paged cache's C ABI and binding without a GPU: exports, sizes, refusals before any device work."""
import ctypes
import subprocess

import pytest
import torch

from diffusion_serving_gb300 import kvc, paged


def cfg(**kw):
    base = dict(batch=4, heads=32, kv_heads=8, head_dim=128, dtype=kvc.BF16, page_size=16, n_pages=64, max_pages=8)
    base.update(kw)
    return paged.make_config(base.pop("batch"), base.pop("heads"), base.pop("kv_heads"), base.pop("head_dim"),
                             base.pop("dtype"), **base)


def test_header_and_exports():
    names = paged.header_functions()
    assert len(names) == 9
    out = subprocess.run(["nm", "-D", "--defined-only", kvc.LIB_PATH], capture_output=True, text=True).stdout
    assert set(names) <= {line.split()[-1] for line in out.splitlines() if line.strip()}
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-x", "c", paged.HEADER_PATH],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert ctypes.sizeof(paged.kvc_paged_config) == 40


@pytest.mark.parametrize("bad", [dict(batch=0), dict(batch=1025), dict(heads=30), dict(head_dim=96), dict(page_size=8),
                                 dict(page_size=48), dict(n_pages=0), dict(max_pages=0), dict(max_pages=2 ** 27),
                                 dict(dtype=9), dict(softmax_scale=-1.0), dict(softmax_scale=float("nan")),
                                 dict(max_tokens=-1)])
def test_bad_configs_are_refused(bad):
    c = cfg(**bad)
    assert paged.kvc_paged_workspace_bytes(c) == 0
    h = ctypes.c_void_p()
    rc = kvc._lib.kvc_paged_create(ctypes.byref(c), 256, 256, None, 256, 256, 256, None, ctypes.byref(h))
    assert rc in (kvc.ERR_ARG, kvc.ERR_UNSUPPORTED) and h.value is None


def test_bad_pointers_are_refused():
    c = cfg()
    h = ctypes.c_void_p()
    good = [256, 256, None, 256, 256, 256]
    for i, x in ((0, None), (1, None), (3, None), (4, None), (5, None), (0, 8), (1, 8), (2, 8), (3, 2), (4, 2), (5, 128)):
        p = list(good)
        p[i] = x
        assert kvc._lib.kvc_paged_create(ctypes.byref(c), *p, None, ctypes.byref(h)) == kvc.ERR_ARG
    assert kvc._lib.kvc_paged_create(ctypes.byref(c), *good, None, None) == kvc.ERR_ARG
    L = kvc._lib
    assert L.kvc_paged_append(None, 16, 16, 1024, None, 0, None, 4, None, None, 0, 0, None) == kvc.ERR_ARG
    assert L.kvc_paged_attend(None, 16, 16, None, 4, None, 1, 0, None) == kvc.ERR_ARG
    assert L.kvc_paged_attend_shared(None, 16, 16, None, 4, None, 1, 16, 1, 16, 0, None) == kvc.ERR_ARG
    assert L.kvc_paged_attend_sparse(None, 16, 16, None, 2, 1, 1, 16, 0, None) == kvc.ERR_ARG
    assert L.kvc_paged_get_error(None, None, None) == kvc.ERR_ARG
    assert L.kvc_paged_debug_stall_waits(None, 0) == kvc.ERR_ARG
    assert L.kvc_paged_destroy(None) == kvc.OK


class Fake(paged.PagedKVCache):
    """The binding's checks alone: tensors on the CPU, calls recorded."""

    def __init__(self, dtype=torch.bfloat16):
        self.batch, self.heads, self.kv_heads, self.head_dim, self.dtype = 2, 8, 2, 64, dtype
        self.device, self._index, self.handle, self.calls = torch.device("cpu"), -1, None, []

    def _stream(self, stream):
        return None

    def _call(self, what, fn, *args):
        self.calls.append((what, args))


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_tensors_that_do_not_fit():
    f = Fake()
    q, cu = t(6, 8, 64), torch.tensor([0, 2, 6], dtype=torch.int32)
    bad = [
        lambda: f.attend(t(6, 8, 32)), lambda: f.attend(t(6, 4, 64)), lambda: f.attend(t(6, 8, 64, dtype=torch.float16)),
        lambda: f.attend(t(3, 2, 8, 64)), lambda: f.attend(t(12, 8, 64)[::2]), lambda: f.attend(q, out=t(6, 8, 64, dtype=torch.float32)),
        lambda: f.attend(q, lse=t(6, 8)), lambda: f.attend(q, cu_q=cu.long()), lambda: f.attend(q, cu_q=cu[:2]),
        lambda: f.append(t(6, 2, 64), t(5, 2, 64)), lambda: f.append(t(6, 2, 64), t(6, 2, 64), q=t(5, 8, 64)),
        lambda: f.append(t(6, 2, 64), t(6, 2, 64), q_out=q), lambda: f.append(t(6, 64, 2).transpose(1, 2), t(6, 2, 64)),
        lambda: f.append(t(6, 2, 64), t(6, 3, 64)[:, :2]), lambda: f.append(t(6, 2, 64), t(6, 2, 64), rope=t(9, 32, 2)),
        lambda: f.append(t(6, 2, 64), t(6, 2, 64), rope=t(9, 64, 2, dtype=torch.float32)),
        lambda: f.append(t(2, 4, 2, 64)[:, :3], t(2, 4, 2, 64)[:, :3]),
        lambda: f.attend_shared(q, cu.long(), cu[:1]), lambda: f.attend_shared(q, cu, cu),
        lambda: f.attend_sparse(q, 4), lambda: f.attend_sparse(t(2, 8, 64), 4, selected=torch.zeros(2, 2, 5, dtype=torch.int32)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
        assert not f.calls, i


def test_binding_passes_strided_rows_of_a_joint_projection():
    f = Fake()
    joint = t(6, 12, 64)
    f.append(joint[:, 8:10], joint[:, 10:], q=joint[:, :8], rope=t(9, 32, 2, dtype=torch.float32))
    _, a = f.calls[-1]
    assert a[2] == 12 * 64 and a[4] == 12 * 64 and a[6] == 6 and a[0] - a[3] == 8 * 64 * 2
    f.append(t(2, 3, 2, 64), t(2, 3, 2, 64))
    assert f.calls[-1][1][2] == 128 and f.calls[-1][1][6] == 6
    f.append(t(1, 2, 64), t(1, 2, 64))
    assert f.calls[-1][1][2] == 128

"""The 4-bit cache's C ABI, binding and sources without a GPU: exports, sizes, refusals before any device work, exactness of the
arithmetic that codes become values by."""
import ctypes
import glob
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from diffusion_serving_gb300 import kvc, paged, paged4
from tests import paged4_ref as ref4
from tests.test_kernel_source import CSRC, block_from, code
from tests.test_paged_abi import cfg, t

PAGED4 = sorted(glob.glob(os.path.join(CSRC, "k_paged4_*.cu")) + glob.glob(os.path.join(CSRC, "paged4_*")))


def test_header_and_exports():
    names = paged4.header_functions()
    assert len(names) == 9
    out = subprocess.run(["nm", "-D", "--defined-only", kvc.LIB_PATH], capture_output=True, text=True).stdout
    assert set(names) <= {line.split()[-1] for line in out.splitlines() if line.strip()}
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-x", "c", paged4.HEADER_PATH],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_page_bytes(dim, page):
    c = cfg(head_dim=dim, page_size=page)
    assert paged4.kvc_paged4_page_bytes(c) == 8 * page * (dim + dim // 16)
    assert paged4.kvc_paged4_workspace_bytes(c) > 0


@pytest.mark.parametrize("bad", [dict(batch=0), dict(batch=1025), dict(heads=30), dict(head_dim=96), dict(page_size=8),
                                 dict(n_pages=0), dict(max_pages=0), dict(max_pages=2 ** 27), dict(dtype=9), dict(dtype=kvc.F32),
                                 dict(softmax_scale=-1.0), dict(softmax_scale=float("nan")), dict(max_tokens=-1)])
def test_bad_configs_are_refused(bad):
    c = cfg(**bad)
    assert paged4.kvc_paged4_page_bytes(c) == 0 and paged4.kvc_paged4_workspace_bytes(c) == 0
    h = ctypes.c_void_p()
    rc = kvc._lib.kvc_paged4_create(ctypes.byref(c), 256, 256, 256, 256, None, ctypes.byref(h))
    assert rc in (kvc.ERR_ARG, kvc.ERR_UNSUPPORTED) and h.value is None
    assert rc == kvc.ERR_UNSUPPORTED or "dtype" not in bad or bad["dtype"] != kvc.F32


def test_bad_pointers_are_refused():
    c, h, L = cfg(), ctypes.c_void_p(), kvc._lib
    good = [256, 256, 256, 256]
    for i, x in ((0, None), (1, None), (2, None), (3, None), (0, 8), (1, 2), (2, 2), (3, 128)):
        p = list(good)
        p[i] = x
        assert L.kvc_paged4_create(ctypes.byref(c), *p, None, ctypes.byref(h)) == kvc.ERR_ARG
    assert L.kvc_paged4_create(ctypes.byref(c), *good, None, None) == kvc.ERR_ARG
    assert L.kvc_paged4_append(None, 16, 16, 1024, None, 0, None, 4, None, None, 0, None, None, 0, None) == kvc.ERR_ARG
    assert L.kvc_paged4_read(None, 16, 16, 4, None, None) == kvc.ERR_ARG
    assert L.kvc_paged4_attend(None, 16, 16, None, 4, None, 1, 0, None) == kvc.ERR_ARG
    assert L.kvc_paged4_get_error(None, None, None) == kvc.ERR_ARG
    assert L.kvc_paged4_debug_stall_waits(None, 0) == kvc.ERR_ARG
    assert L.kvc_paged4_destroy(None) == kvc.OK


class Fake(paged4.PagedKVCache4):
    """The binding's checks alone: tensors on the CPU, calls recorded."""

    def __init__(self, dtype=torch.bfloat16):
        self.batch, self.heads, self.kv_heads, self.head_dim, self.dtype = 2, 8, 2, 64, dtype
        self.device, self._index, self.handle, self.calls = torch.device("cpu"), -1, None, []

    def _stream(self, stream):
        return None

    def _call(self, what, fn, *args):
        self.calls.append((what, args))


def test_binding_refuses_tensors_that_do_not_fit():
    f = Fake()
    q, k, cu = t(6, 8, 64), t(6, 2, 64), torch.tensor([0, 2, 6], dtype=torch.int32)
    rope = t(9, 32, 2, dtype=torch.float32)
    pos = torch.zeros(6, 3, dtype=torch.int32)
    bad = [
        lambda: f.attend(t(6, 8, 32)), lambda: f.attend(t(6, 8, 64, dtype=torch.float16)), lambda: f.attend(t(12, 8, 64)[::2]),
        lambda: f.attend(q, out=t(6, 8, 64, dtype=torch.float32)), lambda: f.attend(q, lse=t(6, 8)), lambda: f.attend(q, cu_q=cu.long()),
        lambda: f.append(k, t(5, 2, 64)), lambda: f.append(k, k, q=t(5, 8, 64)), lambda: f.append(k, k, q_out=q),
        lambda: f.append(k, k, rope=t(9, 32, 2)), lambda: f.append(k, k, rope=rope, positions=pos),
        lambda: f.append(k, k, positions=pos[:, :1].contiguous()), lambda: f.append(k, k, rope=rope, axes=paged.rope_axes([0] * 32)),
        lambda: f.read(7), lambda: f.read(6, k_out=t(6, 2, 32)), lambda: f.read(6, v_out=t(6, 2, 64, dtype=torch.float16)),
        lambda: f.read(6, k_out=t(4, 2, 64)), lambda: f.read(6, k_out=t(12, 2, 64)[::2]), lambda: f.read(6, cu=cu[:2], k_out=k, v_out=k),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
        assert not f.calls, i


def test_binding_passes_what_the_c_entry_takes():
    f = Fake()
    joint = t(6, 12, 64)
    f.append(joint[:, 8:10], joint[:, 10:], q=joint[:, :8], rope=t(9, 32, 2, dtype=torch.float32))
    what, a = f.calls[-1]
    assert what == "kvc_paged4_append" and len(a) == 14 and a[2] == 12 * 64 and a[6] == 6 and a[9] == 9 and a[10] is None and a[11] is None
    pos = torch.zeros(2, 3, 1, dtype=torch.int32)
    f.append(t(2, 3, 2, 64), t(2, 3, 2, 64), rope=t(9, 32, 2, dtype=torch.float32), positions=pos, half=True)
    what, a = f.calls[-1]
    assert len(a) == 14 and a[11] == pos.data_ptr() and a[12] == paged.ROPE_HALF
    ko, vo = t(2, 3, 2, 64), t(6, 2, 64)
    assert f.read(6, k_out=ko, v_out=vo)[0] is ko
    assert f.calls[-1][1][:3] == (ko.data_ptr(), vo.data_ptr(), 6)
    with pytest.raises(kvc.KvcError):
        f.attend_shared(t(6, 8, 64), None, None)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_every_held_value_is_exact_in_16_bits(dtype):
    s = torch.from_numpy(ref4.E4M3)[:, None]
    c = torch.arange(16, dtype=torch.float64)
    x = (c - 8) * s
    assert torch.equal(x.to(dtype).double(), x)


def half_pairs(text, name):
    return [int(x, 16) for x in re.search(name, text).groups()]


def test_codes_become_values_without_rounding():
    """The constants of paged4_internal.h: a code under an exponent, times the scale, less the offset's product, each exact in
    the type, for all codes and scales."""
    text = code(os.path.join(CSRC, "paged4_internal.h"))
    s = torch.from_numpy(ref4.E4M3)
    types = re.findall(r"kMask = 0x(\w+)u, kBase = 0x(\w+)u, kOff = 0x(\w+)u;\s*static constexpr int kAt = (\d)", text)
    fast = re.search(r"return \{s, pg4_mul\(s, 0x(\w+)u, t\), pg4_mul\(s, 0x(\w+)u, t\)\};", text)
    base16 = types[0][1]
    cases = [(torch.float16, *types[0], 1.0), (torch.bfloat16, *types[1], 1.0),
             (torch.float16, "000F000F", base16, fast.group(1), "0", 1 / 16), (torch.float16, "00F000F0", base16, fast.group(2), "4", 1.0)]
    for dtype, mask, base, off, at, factor in cases:
        mask, base, off, at = int(mask, 16), int(base, 16), int(off, 16), int(at)
        for x in (mask, base, off):
            assert x & 0xFFFF == x >> 16
        assert mask & 0xFFFF == 15 << at
        as_type = lambda b: torch.tensor(np.array(b, dtype=np.uint16).astype(np.int16)).view(dtype).double()  # noqa: E731
        x = as_type([(base & 0xFFFF) | c << at for c in range(16)])
        o = as_type([off & 0xFFFF])[0] * s                           # the offset's product
        assert torch.equal(o.to(dtype).double(), o) and torch.isfinite(o).all()
        y = x[None] * s[:, None] + o[:, None]                        # (exact in 64 bits)
        want = (torch.arange(16, dtype=torch.float64) - 8)[None] * s[:, None] * factor
        assert torch.equal(y, want) and torch.equal(y.to(dtype).double(), y)


def test_nothing_is_read_through_the_read_only_path():
    """As the 16-bit kernels (every kernel may live while the one before it still writes)."""
    assert len(PAGED4) == 5
    for path in PAGED4:
        text, name = code(path), os.path.basename(path)
        assert "__ldg" not in text and ".nc" not in text, name
        assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", text), name
        for m in re.finditer(r"__global__", text):
            body = block_from(text, m.start())
            assert body.index("kvc_pdl_wait();") < body.index("kvc_pdl_release();"), name


def test_a_stage_belongs_to_one_set_and_one_producer():
    """The streaming kernel's rings: producers and sets of consumers that step over one another's tiles see every phase of the
    barriers that they wait on only if the stages are a multiple of both."""
    text = code(os.path.join(CSRC, "k_paged4_decode.cu"))
    sets = [int(x) for x in re.search(r"kSets = R == 8 \? (\d) : (\d);", text).groups()]
    producers = int(re.search(r"kProducers = (\d);", text).group(1))
    stages = [int(x) for x in re.search(r"kStages = D == 128 \? (\d+) : (\d+);", text).groups()]
    for s in stages:
        assert s % producers == 0 and all(s % x == 0 for x in sets) and s >= 2 * producers

"""Refusals of the append with several axes, before any device work (no GPU)."""
import ctypes
import subprocess

import pytest
import torch

from diffusion_serving_gb300 import kvc, paged
from tests.test_paged_abi import Fake, t


def test_header_compiles_as_c_and_matches_the_binding():
    text = open(paged.AXES_HEADER_PATH).read()
    assert "int kvc_paged_append_axes(" in text
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-x", "c", paged.AXES_HEADER_PATH],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert ctypes.sizeof(paged.kvc_rope_axes) == 68 and hasattr(kvc._lib, "kvc_paged_append_axes")


def test_null_handle_is_refused():
    axes = paged.rope_axes([0] * 64)
    assert kvc._lib.kvc_paged_append_axes(None, 16, 16, 1024, None, 0, None, 4, None, 16, 9, ctypes.byref(axes), 16, 0,
                                          None) == kvc.ERR_ARG


@pytest.mark.parametrize("bad", [[], [0] * 65, [0, 4], [0, -1], [5]])
def test_rope_axes_refuses(bad):
    with pytest.raises(ValueError):
        paged.rope_axes(bad)


def test_rope_axes_counts_axes():
    assert paged.rope_axes([0, 2]).n_axes == 3 and paged.rope_axes([0, 0], 4).n_axes == 4
    with pytest.raises(ValueError):
        paged.rope_axes([0, 1], 1)
    with pytest.raises(ValueError):
        paged.rope_axes([0], 5)


def test_binding_refuses_positions_that_do_not_fit():
    f = Fake()
    k, rope = t(6, 2, 64), t(9, 32, 2, dtype=torch.float32)
    axes = paged.rope_axes([j % 3 for j in range(32)])
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    bad = [dict(positions=i32(6, 2), axes=axes), dict(positions=i32(5, 3), axes=axes), dict(positions=i32(6, 3).long(), axes=axes),
           dict(positions=i32(3, 6).t(), axes=axes), dict(positions=i32(18), axes=axes), dict(positions=i32(3, 2, 3), axes=axes),
           dict(axes=axes), dict(positions=i32(6, 3)), dict(positions=i32(6, 3), axes=paged.rope_axes([0, 1, 2] * 10)),
           dict(positions=i32(6, 3), axes=axes, rope=None)]
    for i, kw in enumerate(bad):
        with pytest.raises(ValueError):
            f.append(k, k, **{"rope": rope, **kw})
        assert not f.calls, i


def test_binding_passes_positions():
    f = Fake()
    k, rope = t(6, 2, 64), t(9, 32, 2, dtype=torch.float32)
    axes = paged.rope_axes([j % 3 for j in range(32)])
    for pos in (torch.zeros(6, 3, dtype=torch.int32), torch.zeros(2, 3, 3, dtype=torch.int32)):
        f.append(k, k, rope=rope, positions=pos, axes=axes, half=True)
        what, a = f.calls[-1]
        assert what == "kvc_paged_append_axes" and a[6] == 6 and a[9] == 9 and a[11] == pos.data_ptr() and a[12] == paged.ROPE_HALF
    f.append(k, k, rope=rope, positions=torch.zeros(6, 1, dtype=torch.int32))
    assert f.calls[-1][0] == "kvc_paged_append_axes"
    f.append(k, k, rope=rope)
    assert f.calls[-1][0] == "kvc_paged_append"

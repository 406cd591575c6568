"""What the binding takes for axes (no GPU): a structure from rope_axes, a copy of one, or one filled in by hand."""
import copy
import ctypes

import pytest
import torch

from diffusion_serving_gb300 import kvc, paged
from tests.test_paged4_abi import Fake as Fake4
from tests.test_paged_abi import Fake, t


@pytest.mark.parametrize("fake", [Fake, Fake4])
def test_structures_filled_in_by_hand_and_copies(fake):
    f = fake()
    k, rope, pos = t(6, 2, 64), t(9, 32, 2, dtype=torch.float32), torch.zeros(6, 3, dtype=torch.int32)
    made = paged.rope_axes([j % 3 for j in range(32)])
    byhand = paged.kvc_rope_axes(n_axes=3)
    byhand.pair_axis[:32] = [j % 3 for j in range(32)]
    for axes in (made, byhand, copy.copy(made), copy.deepcopy(byhand)):
        f.append(k, k, rope=rope, positions=pos, axes=axes)
        assert f.calls[-1][1][10] is axes and bytes(axes) == bytes(made)


def test_the_c_entry_gets_the_structure_itself():
    """ctypes hands a structure on by its address where the argument is declared as a pointer to one."""
    for fn, at in ((kvc._lib.kvc_paged_append_axes, 11), (kvc._lib.kvc_paged4_append, 11)):
        made = paged.rope_axes([0, 1])
        arg = fn.argtypes[at].from_param(made)
        assert fn.argtypes[at] is ctypes.POINTER(paged.kvc_rope_axes) and f"{ctypes.addressof(made):#x}" in repr(arg)


@pytest.mark.parametrize("bad", [[j % 3 for j in range(32)], 3, None])
def test_anything_else_is_refused(bad):
    f = Fake()
    with pytest.raises(ValueError):
        f.append(t(6, 2, 64), t(6, 2, 64), rope=t(9, 32, 2, dtype=torch.float32), positions=torch.zeros(6, 3, dtype=torch.int32),
                 axes=bad)
    assert not f.calls

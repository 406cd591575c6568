"""Static checks of the paged cache's CUDA sources (no GPU)."""
import glob
import os
import re

from tests.test_kernel_source import CSRC, block_from, code

PAGED = sorted(glob.glob(os.path.join(CSRC, "k_paged_*.cu")) + glob.glob(os.path.join(CSRC, "paged_*")))


def test_nothing_is_read_through_the_read_only_path():
    """Every kernel is launched as a programmatic dependent, so it lives while the kernel before it still writes what it
    will read (queries, page numbers, selections, keys and bounds).  ld.global.nc, which __ldg makes, and which the compiler may make
    of loads through const __restrict__ pointers, is defined only for data that nobody writes during the kernel's life."""
    assert len(PAGED) >= 10
    for path in PAGED:
        text, name = code(path), os.path.basename(path)
        assert "__ldg" not in text and ".nc" not in text, name
        assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", text), name


def test_the_coherent_loads_stay_behind_the_wait():
    """An asm without `volatile` may be moved across another one, and so ahead of kvc_pdl_wait()."""
    text = code(os.path.join(CSRC, "paged_internal.h"))
    loads = re.findall(r"asm\s*(volatile)?\s*\(\s*\"ld\.global", text)
    assert loads and all(loads)


def test_every_kernel_waits_before_it_releases():
    """A kernel that let its dependents start before its own wait would let them run next to what precedes it."""
    for path in PAGED:
        text = code(path)
        for m in re.finditer(r"__global__", text):
            body = block_from(text, m.start())
            assert "kvc_pdl_wait();" in body and "kvc_pdl_release();" in body, os.path.basename(path)
            assert body.index("kvc_pdl_wait();") < body.index("kvc_pdl_release();"), os.path.basename(path)

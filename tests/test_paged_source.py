"""Static checks of the paged cache's CUDA sources (no GPU)."""
import glob
import os
import random
import re
import subprocess

from diffusion_serving_gb300.build import nvcc
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


PROGRAM = r"""
#include <stdio.h>
#include "paged_internal.h"
// every line of the input: most items tiles grid min_tiles whole; out: padded per stride
int main() {
  int most, grid, min_tiles, whole;
  long long items, tiles;
  for (; scanf("%d %lld %lld %d %d %d", &most, &items, &tiles, &grid, &min_tiles, &whole) == 6;) {
    int per = -1, stride = -1;
    const bool padded = pg_padded(most, items, tiles, grid, min_tiles, whole, &per, &stride);
    printf("%d %d %d\n", padded, per, stride);
  }
}
"""


def test_a_padded_line_stays_within_32_bits(tmp_path):
    """The work split's arithmetic on the host: items are padded to equal stretches only where all of them fit the 32 bits
    that places on the line are counted in.  (152 rows of 0.8 to 1 times 2^30 slots, 64 to a tile, are 2.04e9 tiles, which fit,
    but 2.55e9 when each is padded to the longest.)"""
    src = tmp_path / "split.cu"
    src.write_text(PROGRAM)
    exe = tmp_path / "split"
    r = subprocess.run([nvcc(), "-std=c++17", "--expt-relaxed-constexpr", "-I", CSRC, "-o", str(exe), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    rng = random.Random(5)
    cases = [(2 ** 24, 152, 2 ** 24 + 151 * 13421773, 152, 8, 8), (2 ** 24, 304, 304 * 7000000, 304, 1, 1)]
    for _ in range(4000):
        grid, min_tiles, whole = rng.choice([(152, 8, 8), (152, 4, 4), (304, 1, 1), (152, 1, 1), (152, 2, 8)])
        items = rng.randint(1, grid + 20)
        most = int(2 ** rng.uniform(0, 24))
        cases.append((most, items, max(most, int(most * items * rng.uniform(0.5, 1.0))), grid, min_tiles, whole))
    out = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True).stdout
    rows = [tuple(map(int, line.split())) for line in out.splitlines()]
    assert len(rows) == len(cases)
    assert rows[0][0] == 0 and 0 < sum(p for p, _, _ in rows) < len(rows)
    for (most, items, tiles, grid, min_tiles, whole), (padded, per, stride) in zip(cases, rows):
        alike = items <= grid and (most <= max(whole, 2 * min_tiles) or most * items * 4 <= 5 * tiles)
        if padded:
            assert alike and stride >= most and stride % per == 0 and items * stride <= 2 ** 31 - 1 - 65536
            assert items * (stride // per) <= grid or most <= whole or per == min_tiles
        elif alike:
            assert items * most * 2 > 2 ** 31 - 65536      # refused for its length alone

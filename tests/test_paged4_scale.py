"""The 4-bit append's scale, max |x| / 7, on the host (no GPU): the kernel's steps in exact arithmetic, for every magnitude of both
16-bit types."""
import os
import re
from fractions import Fraction

import pytest
import torch

from tests.test_kernel_source import CSRC, block_from, code


def fp32(x: Fraction) -> Fraction:
    """x rounded to fp32, to nearest, ties to even (x of normal magnitude or 0)."""
    if x == 0:
        return x
    a = abs(x)
    e = a.numerator.bit_length() - a.denominator.bit_length()
    if a < Fraction(2) ** e:
        e -= 1
    ulp = Fraction(2) ** (e - 23)
    return round(x / ulp) * ulp                           # (round takes a tie to the even neighbour)


def test_rounding_helper():
    for x, want in ((Fraction(1, 3), torch.tensor(1 / 3).item()), (Fraction(2 ** 24 + 1), 2.0 ** 24), (Fraction(2 ** 24 + 3), 2.0 ** 24 + 4),
                    (Fraction(-5, 7), -torch.tensor(5 / 7).item())):
        assert fp32(x) == Fraction(want)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_the_quotient_is_the_rounded_one(dtype):
    body = block_from(code(os.path.join(CSRC, "k_paged4_append.cu")), code(os.path.join(CSRC, "k_paged4_append.cu")).index("scale_bits(float top)"))
    assert re.search(r"kInv = 1\.f / 7\.f;\s*const float q0 = x \* kInv, q = __fmaf_rn\(__fmaf_rn\(-7\.f, q0, x\), kInv, q0\);", body)
    x = torch.arange(1, 0x7C00 if dtype == torch.float16 else 0x7F80, dtype=torch.int16).view(dtype).double()
    x = x[(x <= 4096) & (x >= 2.0 ** -12)]                # (below: e4m3's least step is 2^-9, so 7 2^-10 and less become 0)
    inv = fp32(Fraction(1, 7))
    for v in x.tolist():
        v = Fraction(v)
        q0 = fp32(v * inv)
        rest = v - 7 * q0
        assert fp32(rest) == rest
        assert fp32(rest * inv + q0) == fp32(v / 7)

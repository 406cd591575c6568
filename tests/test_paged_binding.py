"""The paged cache's binding: layouts that mean the same tokens are passed alike (no GPU needed)."""
import pytest
import torch

from tests.test_paged_abi import Fake, t


def strides(f):
    """(kv_stride, q_stride, tokens) of the last append."""
    _, a = f.calls[-1]
    return a[2], a[4], a[6]


def test_single_tokens_whatever_the_token_dimensions_stride():
    """[B, 1, H, D]: the stride of a dimension of size 1 is arbitrary, in torch's own results too."""
    f = Fake()
    k, v, q = (t(2, h, 1, 64).transpose(1, 2) for h in (2, 2, 8))     # what is left of [B, H, 1, D]
    assert k.stride() == (128, 64, 64, 1) and k.is_contiguous()
    f.append(k, v, q=q, rope=t(9, 32, 2, dtype=torch.float32))
    assert strides(f) == (2 * 64, 8 * 64, 2)
    joint = t(2, 12, 64)
    f.append(joint[:, 8:10].unsqueeze(1), joint[:, 10:].unsqueeze(1), q=joint[:, :8].unsqueeze(1),
             rope=t(9, 32, 2, dtype=torch.float32))
    assert strides(f) == (12 * 64, 12 * 64, 2)
    odd = torch.as_strided(t(4096), (2, 1, 2, 64), (128, 3, 64, 1))
    f.append(odd, odd)
    assert strides(f)[0] == 128


def test_one_token_in_all():
    """Its strides mean nothing: a slice and a dense tensor go together."""
    f = Fake()
    f.batch = 1
    joint = t(1, 1, 12, 64)
    for k, v in ((joint[0, :, 8:10], t(1, 2, 64)), (joint[:, :, 8:10], t(1, 1, 2, 64)),
                 (torch.as_strided(t(4096), (1, 2, 64), (131, 64, 1)), t(1, 2, 64))):
        f.append(k, v, q=t(1, 8, 64), rope=t(9, 32, 2, dtype=torch.float32))
        assert strides(f) == (2 * 64, 8 * 64, 1)


def test_one_row_of_several_tokens():
    """[1, n, H, D]: the batch's stride means nothing."""
    f = Fake()
    f.batch = 1
    joint = t(5, 12, 64)
    k = torch.as_strided(joint, (1, 5, 2, 64), (7, 12 * 64, 64, 1), 8 * 64)
    f.append(k, joint[:, 10:].unsqueeze(0))
    assert strides(f)[0] == 12 * 64 and strides(f)[2] == 5


def test_one_head_has_no_stride():
    f = Fake()
    f.kv_heads = 1
    k = t(6, 5, 64)[:, 2:3]
    f.append(k, k)
    assert strides(f)[0] == 5 * 64


@pytest.mark.parametrize("make", [
    lambda: t(2, 4, 2, 64)[:, :3],                                     # rows with a gap between them
    lambda: t(2, 3, 4, 64)[:, :, ::2],                                 # heads apart
    lambda: t(2, 2, 3, 64).transpose(1, 2),                            # heads outside tokens
    lambda: t(2, 3, 2, 128)[..., ::2],
])
def test_tokens_that_are_not_evenly_apart_are_refused(make):
    f = Fake()
    with pytest.raises(ValueError):
        f.append(make(), make())
    assert not f.calls

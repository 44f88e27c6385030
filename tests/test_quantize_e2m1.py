"""The 4-bit quantiser without a GPU: ties, and weights that are not numbers."""
import math

import pytest
import torch

from combine_ep_get_03_gb300 import moe

VALUE = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6])


def exponent(s, n, c):
    return int(s[0, n // 128, c // 4, 16 * (n % 32) + 4 * (n % 128 // 32) + c % 4])


def codes_of(q, N, K):
    return torch.stack((q & 15, q >> 4), -1).view(N, K).long()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float64])
@pytest.mark.parametrize("power", [-120, -3, 0, 40])
def test_ties_go_to_the_even_code(dtype, power):
    """Half way between two values the one whose last bit is 0; a bf16 weight has
    eight bits, so that ties are common, and rounding them all down would shift the weights to zero."""
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    even = [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
    near = 1 + 2.0 ** -7
    w = torch.zeros((1, 1, 128), dtype=torch.float64)
    w[0, 0, :7], w[0, 0, 7:14] = torch.tensor(ties, dtype=torch.float64), -torch.tensor(ties, dtype=torch.float64)
    w[0, 0, 14:21], w[0, 0, 21:28] = w[0, 0, :7] * near, w[0, 0, :7] / near
    w[0, 0, 28] = 6.0
    q, s = moe.quantize_e2m1((w * 2.0 ** power).to(dtype))
    assert exponent(s, 0, 0) == power + 127
    c = codes_of(q, 1, 128)[0]
    v = VALUE[c & 7] * (1 - 2 * (c >> 3))
    assert v[:7].tolist() == even and v[7:14].tolist() == [-x for x in even]
    assert v[14:21].tolist() == [0.5, 1, 1.5, 2, 3, 4, 6] and v[21:28].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4]
    assert v[28] == 6 and (v[29:] == 0).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_weights_that_are_not_finite_stay_visible(bad):
    """32 channels with such a weight get the exponent that stands for NaN (the 8-bit
    weights' block becomes NaN too); the others keep their codes."""
    torch.manual_seed(1)
    w = torch.randn(1, 130, 256)
    q, s = moe.quantize_e2m1(w)
    w2 = w.clone()
    w2[0, 129, 70] = bad
    q2, s2 = moe.quantize_e2m1(w2)
    assert exponent(s2, 129, 2) == 255 and exponent(s, 129, 2) < 255
    codes, codes2 = codes_of(q[0], 130, 256), codes_of(q2[0], 130, 256)
    rest = torch.ones(130, 256, dtype=torch.bool)
    rest[129, 64:96] = False
    assert torch.equal(codes[rest], codes2[rest])
    assert (s != s2).sum() == 1 and (s2 == 255).sum() == 1

"""The ends of the experts' and the gate's ranges: large gates, rows whose scales
lie far apart, tiny gradients, experts that hardly any token looks at, and row
buffers beyond 2^31 elements.  Bounds as derived in test_gpu_experts.py unless a
test derives its own."""
import math

import pytest
import torch

from combine_ep_get_03_gb300 import ep
from test_gpu_experts import DEV, U24, Rows, check8, gen, silu64, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("weighted", [False, True])
def test_swiglu_backward_of_large_gates(weighted):
    """Gates up to 2^40 of either sign.  With t = e^-g, s = 1 / (1 + t) is off by
    (1 - s) (2 |g| + 8) u24 + 4 u24 of itself, so 1 + g (1 - s) by
    |g| (1 - s) (2 |g| + 12) u24 + 4 min(|g|, 18) u24 at most: from g = 18 on,
    1 + t rounds to 1, and s and 1 - s are 1 and 0 exactly.  Below g = -128 s is
    0 in fp32 and every gradient below the smallest code."""
    exps = list(range(-8, 41, 2))
    F, n = 128 * len(exps), 24
    r = Rows([n], "em")
    pq, ps, p = r.fp8(2 * F, 1)
    for i, e in enumerate(exps):
        r._scales(ps)[:n, i] *= 2.0 ** e
        p[:, 128 * i:128 * (i + 1)] *= 2.0 ** e
    da = torch.randn((n, F), generator=gen(2), device=DEV).bfloat16()
    rw = torch.randn(n, generator=gen(3), device=DEV) if weighted else None
    drw = torch.empty(n, device=DEV) if weighted else None
    dp, dps = r.out8(2 * F)
    ep.ep_grouped_swiglu_backward(da, pq, ps, dp, dps, row_weights=rw, grad_row_weights=drw, **r.args())
    g, u = p.chunk(2, 1)
    d = da.double()
    wd = d * rw.double()[:, None] if weighted else d
    s, rest = torch.sigmoid(g), torch.sigmoid(-g)  # rest = 1 - s
    ref = torch.cat([wd * u * s * (1 + g * rest), wd * silu64(g)], 1)
    a = g.abs()
    near = a.clamp_max(128.0)
    eg = (wd * u).abs() * s * (1 + a.clamp_max(18.0) + a * rest) * (16 + 2 * near) * U24
    eu = (wd * silu64(g)).abs() * (16 + 2 * near) * U24
    v, sc = r.read8(dp, dps)
    check8(v, sc, ref, torch.cat([eg, eu], 1), "gradient")
    far = g > 2.0 ** 24
    assert far.any() and (v[:, :F][far & (wd * u).abs().gt(0.1)] != 0).all(), "the gate's gradient is d u there, not 0"
    if weighted:
        terms = (d * silu64(g) * u).abs()
        within(drw.double(), (d * silu64(g) * u).sum(1), (terms * (F / 32 + 24 + 2 * near) * U24).sum(1), "row weights")

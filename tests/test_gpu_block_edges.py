"""The norms around a block at the ends of what their calls accept: widths whose
stages fill shared memory, calls that need no input, as many tokens as an int
counts, weights that are not finite beside padding tokens."""
import math

import pytest
import torch

import test_gpu_block as block
from combine_ep_get_03_gb300 import ep
from test_gpu_block import Norms, TYPES

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


# Four stages of 5592 channels and three of 7456 take 223 680 bytes where all (bf16) or
# two (fp32) of the residual-typed rows are there: more than a block has beside its barriers.
@pytest.mark.parametrize("H", [5592, 7456, 5584, 7464])
@pytest.mark.parametrize("gate", ["none", "token"])
@pytest.mark.parametrize("res,wt", TYPES)
def test_norm_backward_where_stages_fill_shared_memory(H, gate, res, wt):
    for T in (3, 320):
        block.test_norm_backward(dict(T=T, H=H, post=True, pre=True, gate=gate), res, wt)
    c = Norms(320, H, res, wt, True, True, gate)
    new, _, rstd = c.forward()
    ws = torch.empty(ep.ep_block_norm_workspace_bytes(H), dtype=torch.uint8, device=DEV)

    def grads(y, dnew, dx):
        dres, dy = torch.empty_like(new), None if y is None else torch.empty_like(c.y)
        dpre = None if dx is None else torch.empty(H, device=DEV)
        ep.ep_block_norm_backward(new, y, rstd, dnew, dx, dres, dy, ws, grad_pre_weight=dpre, **c.how)
        return [t for t in (dres, dy, dpre) if t is not None]

    # an input left out counts as zeros: the same bits
    for y in (None, c.y):
        for dnew, dx in ((None, c.dx), (c.dnew, None)):
            zeros = [torch.zeros_like(t) if g is None else g for t, g in ((c.dnew, dnew), (c.dx, dx))]
            for a, b in zip(grads(y, dnew, dx), grads(y, *zeros)):
                assert torch.equal(a, b)


@pytest.mark.parametrize("H", [264, 2048, 7168, 8200])
@pytest.mark.parametrize("gate", ["none", "vector", "token"])
def test_norm_backward_that_needs_no_input(H, gate):
    """No gradient given, nothing of y needed: zeros, whatever the gate."""
    for res, wt in TYPES:
        c = Norms(33, H, res, wt, False, True, gate, masked=True)
        dres, dy = torch.full_like(c.residual, 7.0), torch.full_like(c.y, 7.0)
        how = dict(pre_weight=c.pre, gate=c.gate, token_mask=c.mask)
        ep.ep_block_norm_backward(None, None, None, None, None, dres, None, None, **how)
        assert (dres == 0).all()
        dres.fill_(7.0)
        ep.ep_block_norm_backward(None, None, None, None, None, dres, dy, None, **how)
        assert (dres == 0).all() and (dy == 0).all()


def test_norm_of_as_many_tokens_as_an_int_counts():
    """2^31 - 1 rows of eight channels, of which the first and the last are not
    zeros: the bits of those rows in a small call."""
    T, H, few = 2 ** 31 - 1, 8, 1000
    torch.cuda.empty_cache()
    n = lambda s: torch.randn((2 * few, H), generator=block.gen(s), device=DEV).bfloat16()  # noqa: E731
    pre = 1 + 0.1 * torch.randn(H, generator=block.gen(3), device=DEV)

    def spread(rows):
        big = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
        big[:few], big[-few:] = rows[:few], rows[few:]
        return big

    ends = lambda t: torch.cat((t[:few], t[-few:]))  # noqa: E731

    def run(h, dx):
        x, rstd = torch.empty_like(h), torch.empty((2, h.shape[0]), device=DEV)
        ep.ep_block_norm_forward(h, None, None, x, rstd=rstd, pre_weight=pre)
        # x's memory takes the gradient
        first = ends(x)
        ep.ep_block_norm_backward(h, None, rstd, None, dx, x, None, None, pre_weight=pre)
        assert not x[few:few + 10000].any() and not x[-few - 10000:-few].any() or h.shape[0] == 2 * few
        return first, ends(rstd[1]), ends(x)

    h, dx = n(1), n(2)
    want = run(h, dx)
    got = run(spread(h), spread(dx))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("H", [64, 2048, 8200])
@pytest.mark.parametrize("gate", ["none", "vector", "token"])
def test_padding_beside_weights_that_are_not_finite(H, gate):
    """A padding token's results are 0 whatever the weights are."""
    for res, wt in TYPES:
        c = Norms(60, H, res, wt, True, True, gate, masked=True)
        c.post[3], c.post[4], c.pre[5], c.pre[6] = math.inf, math.nan, -math.inf, math.nan
        if gate == "vector":
            c.gate[7] = math.inf
        off = ~c.on
        new, x, rstd = c.forward()
        assert (new[off] == 0).all() and (x[off] == 0).all() and (rstd[:, off] == 0).all()
        assert not new[c.on][:, 3:5].isfinite().any() and not x[c.on][:, 3:7].isfinite().any()
        dres, dy = torch.empty_like(new), torch.empty_like(c.y)
        ep.ep_block_norm_backward(new, c.y, rstd, c.dnew, c.dx, dres, dy, None, **c.how)
        assert (dres[off] == 0).all() and (dy[off] == 0).all()
        x2 = torch.empty_like(x)
        ep.ep_block_norm_forward(c.residual, None, None, x2, pre_weight=c.pre, token_mask=c.mask)
        assert (x2[off] == 0).all()

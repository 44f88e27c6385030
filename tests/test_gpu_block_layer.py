"""The layer of experts and the block around it: what a call's result has to be bit
for bit."""
import pytest
import torch

from combine_ep_get_03_gb300 import ep
from test_gpu_block import Layout

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("H,scale", [(512, 1.0), (2048, 1e-2), (640, 1e-6)])
def test_combine_gradient_in_e4m3_bit_for_bit(H, scale):
    """Codes and scales are the definition's in fp32: v = w grad_out rounded, a = the
    largest |v| of 128 channels or 1e-4, scale a / 448, codes of v (448 / a), each
    division rounded once.  (A product of two bf16 numbers often lies midway between
    codes, so 448 times a reciprocal differs from 448 / a there.)  The gradient
    without y and without the weights' has the same bits, and writes no other row."""
    l = Layout(2, 300, 12, 4, H, 16, seed=15)
    l.g = (l.g.float() * scale).bfloat16()
    t, j, row = l.entries()
    v = (l.w[t, j, None] * l.g[t].float()).view(len(row), H // 128, 128)
    a = v.abs().amax(2).clamp_min(1e-4)
    s = a / torch.full_like(a, 448.0)
    codes = (v * (torch.full_like(a, 448.0) / a)[..., None]).view(-1, H).to(torch.float8_e4m3fn).view(torch.uint8)
    ld = (l.rows + 3) // 4 * 4 + 4
    for y, dw in ((l.y, torch.empty_like(l.w)), (None, None)):
        dy = torch.full((l.rows, H), 0x5A, dtype=torch.uint8, device=DEV)
        ds = torch.full((H // 128, ld), 7.25, device=DEV)
        l.h.em_combine_weighted_backward(l.g, y, l.w, ep.EP_FP8_E4M3, dy, ds, grad_topk_weights=dw)
        assert torch.equal(ds.t()[row], s) and torch.equal(dy[row], codes)
        assert (dy[~l.live] == 0x5A).all() and (ds.t()[:l.rows][~l.live] == 7.25).all() and (ds[:, l.rows:] == 7.25).all()
    assert l.h.get_device_status() == ep.EP_OK
    l.h.close()

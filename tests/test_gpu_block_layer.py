"""The layer of experts and the block around it: what a call's result has to be bit
for bit, how the block routes, and backward passes around replayed graphs."""
import math

import pytest
import torch

from combine_ep_get_03_gb300 import ep
from combine_ep_get_03_gb300 import moe
from test_gpu_block import Layout
from test_gpu_experts import gen

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


def block_and_weights(router, weigh=False, T=256, R=2, k=1, E=8, H=256, F=128):
    torch.manual_seed(3)
    layer = moe.MoELayer(R, E, k, H, F, T // R, weigh_in_combine=weigh, expert_alignment=16)
    w1 = moe.ExpertWeights(torch.randn((E, 2 * F, H), device=DEV) / H ** 0.5)
    w2 = moe.ExpertWeights(torch.randn((E, H, F), device=DEV) / F ** 0.5)
    pre = 1 + 0.1 * torch.randn(H, device=DEV)
    return moe.MoEBlock(layer, pre, router), w1, w2


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_routing_of_experts_close_together(dtype):
    """Experts in pairs whose logits differ by about a thousandth of themselves: a bf16
    logit has 8 bits and would tie them, fp32's error (256 products) is far below."""
    T, E, H = 256, 8, 256
    g = gen(21)
    base = torch.randn((E // 2, 1, H), generator=g, device=DEV)
    router = (base + 2.0 ** -10 * torch.randn((E // 2, 2, H), generator=g, device=DEV) * (dtype is torch.float32)).reshape(E, H)
    if dtype is torch.bfloat16:  # one channel of the second of a pair a step of bf16 away
        router = router.bfloat16()
        router[1::2, 0] = (router[1::2, 0].view(torch.int16) + 1).view(torch.bfloat16)
    block, w1, w2 = block_and_weights(router)
    h = torch.randn((T, H), generator=g, device=DEV)
    out, _, saved = block.forward(h, w1, w2)
    x, idx = saved[1], saved[5][2][:, 0]
    logits = x.double() @ router.double().t()
    top = logits.topk(2, 1)
    err = (H + 4) * 2.0 ** -24 * (x.double().abs() @ router.double().abs().t()).amax(1)
    clear = top.values[:, 0] - top.values[:, 1] > 2 * err
    assert clear.sum() > T // 8 and torch.equal(idx[clear], top.indices[clear, 0])
    # gradients of the router's type, and of the stream
    grads = block.backward(torch.randn((T, H), generator=g, device=DEV), torch.ones(1, device=DEV), saved, w1, w2)
    assert grads["router"].dtype is dtype and grads["router"].isfinite().all() and grads["h"].isfinite().all()
    dec = block.decode(h.clone(), w1, w2)
    assert ((dec - out).norm() / (out - h).norm()).item() < 3 * math.sqrt(4) * 0.026
    block.layer.check()
    block.layer.close()


def test_gradients_of_an_fp32_router():
    """Against 64 bits, from the layer's own gradient of the logits: the balance
    loss alone, so that nothing but the router's products rounds."""
    T, E, H = 256, 8, 256
    router = torch.randn((E, H), generator=gen(22), device=DEV) / 16
    block, w1, w2 = block_and_weights(router, k=2)
    h = torch.randn((T, H), generator=gen(23), device=DEV)
    _, _, saved = block.forward(h, w1, w2)
    zero = torch.zeros((T, H), device=DEV)
    grads = block.backward(zero, torch.full((1,), 100.0, device=DEV), saved, w1, w2)
    x, idx = saved[1].double(), saved[5][2]
    hd = h.double().requires_grad_(True)
    rd = router.double().requires_grad_(True)
    xd = hd * (hd.square().mean(1, keepdim=True) + 1e-6).rsqrt() * block.pre.double()
    p = torch.softmax(xd @ rd.t(), 1).mean(0)
    count = torch.bincount(idx.reshape(-1), minlength=E)
    (100.0 * 1e-2 * E / (2 * T) * (count * p).sum()).backward()
    rel = lambda a, b: ((a.double() - b).norm() / b.norm()).item()  # noqa: E731
    # x in bf16 on the one side, x's gradient on the other: half a step of 2^-8 at most each
    assert rel(grads["router"], rd.grad) < 2.0 ** -8
    assert rel(grads["h"], hd.grad) < 2.0 ** -7
    block.layer.close()


@pytest.mark.parametrize("weigh", [False, True])
def test_backward_around_a_replayed_forward(weigh):
    """A captured forward makes the handle's layout anew whenever it is replayed,
    which the host does not see: a backward behind it has the bits of one that
    directly follows its forward."""
    T, E, H = 64, 8, 256
    block, w1, w2 = block_and_weights(None, weigh, T, k=2)
    layer = block.layer
    batch = lambda s: (torch.randn((T, H), generator=gen(s), device=DEV).bfloat16(),  # noqa: E731
                       torch.randn((T, E), generator=gen(s + 50), device=DEV))
    (x, logits), (x2, logits2), (go, _) = batch(1), batch(2), batch(3)
    gl = torch.ones(1, device=DEV)
    out, _, saved = layer.forward(x, logits, w1, w2)
    want = layer.backward(go, gl, saved, w1, w2)
    out2, _, saved2 = layer.forward(x2, logits2, w1, w2)
    want2 = layer.backward(go, gl, saved2, w1, w2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured, _, kept = layer.forward(x2, logits2, w1, w2)
    out, _, saved = layer.forward(x, logits, w1, w2)
    graph.replay()
    got = layer.backward(go, gl, saved, w1, w2)
    graph.replay()
    got2 = layer.backward(go, gl, kept, w1, w2)
    layer.check()
    assert torch.equal(captured, out2)
    for a, b in zip(got + got2, want + want2):
        assert torch.equal(a, b)
    # a captured step of both passes, an eager forward before each replay
    step = torch.cuda.CUDAGraph()
    with torch.cuda.graph(step):
        _, _, kept = layer.forward(x2, logits2, w1, w2)
        both = layer.backward(go, gl, kept, w1, w2)
    for _ in range(2):
        _, _, saved = layer.forward(x, logits, w1, w2)
        step.replay()
        for a, b in zip(both + layer.backward(go, gl, saved, w1, w2), want2 + want):
            assert torch.equal(a, b)
    layer.check()
    layer.close()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_token(dtype):
    """A block of one token, trained and decoded: its row is the row of a batch that
    holds it (the router's product may sum in another order)."""
    router = (torch.randn((8, 256), generator=gen(31), device=DEV) / 16).to(dtype)
    block, w1, w2 = block_and_weights(router, T=64, R=1, k=2)
    h = torch.randn((64, 256), generator=gen(32), device=DEV)
    many, _, saved = block.forward(h, w1, w2)
    one, _, single = block.forward(h[5:6].clone(), w1, w2)
    dec = block.decode(h[5:6].clone(), w1, w2)
    assert torch.equal(saved[5][2][5], single[5][2][0])
    # the routing weights differ by fp32 roundings, which may move an e4m3 code by a step
    rel = lambda a, b: ((a - b).norm() / (b - h[5]).norm()).item()  # noqa: E731
    assert rel(one[0], many[5]) < 2.0 ** -4 and rel(dec[0], many[5]) < 3 * math.sqrt(4) * 0.026
    grads = block.backward(torch.ones((1, 256), device=DEV), torch.ones(1, device=DEV), single, w1, w2)
    assert all(t is None or t.isfinite().all() for t in grads.values())
    assert grads["router"].dtype is dtype and grads["h"].shape == (1, 256)
    block.layer.check()
    block.layer.close()

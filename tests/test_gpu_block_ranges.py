"""The weighted combine, the norms and the 4-bit products where sizes and orders
go to their ends: tensors beyond 2^31 elements, no tokens, calls side by side in
two streams, a decode step replayed from a graph."""
import math

import pytest
import torch

from combine_ep_get_03_gb300 import ep
from combine_ep_get_03_gb300 import moe

from test_gpu_block import BF, Layout, Norms, U24
from test_gpu_experts import Rows, gen, within
from test_gpu_experts_w4 import weights4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_norms_beyond_2_31_elements():
    """The last rows of [300 000, 8 192], against the same rows alone."""
    T, H, last = 300000, 8192, 400
    g = gen(1)
    n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    post, pre, gate = 1 + 0.1 * n(H), 1 + 0.1 * n(H), n(H)
    big = [torch.zeros((T, H), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    small = [n(last, H).bfloat16() for _ in range(2)]
    for a, b in zip(big, small):
        a[-last:] = b
    assert big[0].numel() > 2 ** 31
    how = dict(post_weight=post, pre_weight=pre, gate=gate)

    def both(residual, y):
        new, x = torch.empty_like(residual), torch.empty_like(y)
        rstd = torch.empty((2, residual.shape[0]), device=DEV)
        ep.ep_block_norm_forward(residual, y, new, x, rstd=rstd, **how)
        dres, dy = torch.empty_like(new), torch.empty_like(y)
        sums = [torch.empty(H, device=DEV) for _ in range(3)]
        ws = torch.empty(ep.ep_block_norm_workspace_bytes(H), dtype=torch.uint8, device=DEV)
        ep.ep_block_norm_backward(new, y, rstd, residual, x, dres, dy, ws, grad_post_weight=sums[0],
                                  grad_pre_weight=sums[1], grad_gate=sums[2], **how)
        return (new, x, dres, dy), sums

    (rows, sums), (want, want_sums) = both(*big), both(*small)
    for a, b in zip(rows, want):
        assert torch.equal(a[-last:], b) and not a[:1000].any()
    for a, b in zip(sums, want_sums):  # the same terms, zeros among them, in another order
        within(a.double(), b.double(), 1e-4 * b.double().abs().mean() + 1e-4 * b.double().abs(), "sums")


def test_combine_beyond_2_31_elements():
    T, k, H = 40000, 8, 7168
    l = Layout(1, T, 8, k, H, 1, seed=2, masked=0.0)
    assert l.y.numel() > 2 ** 31
    t = torch.arange(T - 50, T, device=DEV)
    out = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    l.h.em_combine_weighted(l.y, l.w, out)
    v = l.w[t][..., None].double() * l.y[l.row[t]].double()
    within(out[t].double(), v.sum(1), v.sum(1).abs() * BF + (k + 1) * U24 * v.abs().sum(1), "combine")
    dy, dw = torch.empty_like(l.y), torch.empty_like(l.w)
    l.h.em_combine_weighted_backward(l.g, l.y, l.w, ep.EP_BF16, dy, grad_topk_weights=dw)
    ref = l.w[t][..., None].double() * l.g[t][:, None].double()
    within(dy[l.row[t]].double(), ref, (BF + 2 * U24) * ref.abs(), "rows' gradient")
    terms = l.g[t][:, None].double() * l.y[l.row[t]].double()
    within(dw[t].double(), terms.sum(2), (H / 32 + 16) * U24 * terms.abs().sum(2), "weights' gradient")
    assert l.h.get_device_status() == ep.EP_OK
    l.h.close()


def block_of(weigh, post=True, gate=None, T=32, R=2, k=2, E=8, H=256, F=128, seed=3):
    torch.manual_seed(seed)
    layer = moe.MoELayer(R, E, k, H, F, max(T // R, 1), weigh_in_combine=weigh, expert_alignment=16)
    W1, W2 = torch.randn((E, 2 * F, H), device=DEV) / H ** 0.5, torch.randn((E, H, F), device=DEV) / F ** 0.5
    router = torch.randn((E, H), device=DEV).bfloat16()
    block = moe.MoEBlock(layer, 1 + 0.1 * torch.randn(H, device=DEV), router, gate=gate,
                         post=1 + 0.1 * torch.randn(H, device=DEV) if post else None)
    return block, W1, W2


@pytest.mark.parametrize("weigh", [False, True])
def test_block_without_tokens(weigh):
    block, W1, W2 = block_of(weigh, gate=torch.ones(256, device=DEV))
    w1, w2 = moe.ExpertWeights(W1), moe.ExpertWeights(W2)
    h = torch.empty((0, 256), device=DEV)
    out, loss, saved = block.forward(h, w1, w2)
    grads = block.backward(torch.empty_like(h), torch.ones(1, device=DEV), saved, w1, w2)
    block.layer.check()
    assert out.shape == (0, 256) and loss.item() == 0 and grads["h"].shape == (0, 256)
    for name in ("pre", "post", "gate", "w1", "w2", "router"):
        assert (grads[name] == 0).all(), name
    block.layer.close()


@pytest.mark.parametrize("four", [False, True])
def test_decode_from_a_graph(four):
    """A block's decode step captured once, replayed on new tokens: the eager bits."""
    block, W1, W2 = block_of(False)
    w1, w2 = (moe.ExpertWeights4(W1), moe.ExpertWeights4(W2)) if four else (moe.ExpertWeights(W1), moe.ExpertWeights(W2))
    h = torch.randn((32, 256), device=DEV)
    block.decode(h.clone(), w1, w2)
    torch.cuda.synchronize()
    graph, static = torch.cuda.CUDAGraph(), h.clone()
    with torch.cuda.graph(graph):
        block.decode(static, w1, w2)
    for seed in (5, 6, 7):
        new = torch.randn((32, 256), generator=gen(seed), device=DEV)
        want = block.decode(new.clone(), w1, w2).clone()
        static.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(static, want)
    block.layer.check()
    block.layer.close()


def test_calls_side_by_side_in_two_streams():
    """Calls that share nothing but their inputs, at the same time: the bits of
    one after the other."""
    r = Rows([3, 0, 40, 17, 100, 64], "em", 8)
    xq, xs, _ = r.fp8(1024, 11)
    q, s, _ = weights4(6, 512, 1024, 12)
    c = Norms(500, 2048, torch.float32, torch.bfloat16, True, True, "vector")
    new, x, rstd = c.forward()
    want = r.out16(512)
    ep.ep_grouped_matmul_w4(xq, xs, q, s, want, **r.args())

    def grads(ws):
        out = [torch.empty_like(c.residual), torch.empty_like(c.y)] + [torch.empty(2048, device=DEV) for _ in range(3)]
        ep.ep_block_norm_backward(new, c.y, rstd, c.dnew, c.dx, out[0], out[1], ws, grad_post_weight=out[2],
                                  grad_pre_weight=out[3], grad_gate=out[4], **c.how)
        return out

    size = ep.ep_block_norm_workspace_bytes(2048)
    first = grads(torch.empty(size, dtype=torch.uint8, device=DEV))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in streams]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for st, ws in zip(streams, spaces):
            with torch.cuda.stream(st):
                out = r.out16(512)
                ep.ep_grouped_matmul_w4(xq, xs, q, s, out, **r.args())
                got.append((out, grads(ws), c.forward()))
    torch.cuda.synchronize()
    for out, g, f in got:
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        assert all(torch.equal(a, b) for a, b in zip(g, first))
        assert all(torch.equal(a, b) for a, b in zip(f, (new, x, rstd)))


def test_rows_do_not_depend_on_their_company():
    """A token's row of a 4-bit product has the same bits alone and in a batch
    of any size, whichever tile width the launch takes."""
    K, N = 1024, 512
    q, s, _ = weights4(2, N, K, 21)
    base = Rows([200, 1], "em")
    xq, xs, _ = base.fp8(K, 22)
    want = base.out16(N)
    ep.ep_grouped_matmul_w4(xq, xs, q, s, want, **base.args())
    for n in (1, 16, 30, 45, 64, 112, 113, 199):
        out = base.out16(N)
        count = torch.tensor([n, 0], dtype=torch.int32, device=DEV)
        ep.ep_grouped_matmul_w4(xq, xs, q, s, out, count, base.offset)
        assert torch.equal(out[:n], want[:n]) and (out[n:] == -5.5).all(), n


def test_special_values_do_not_cross_tokens_in_the_combine():
    l = Layout(1, 16, 4, 2, 256, 1, seed=9, masked=0.0)
    l.y[l.row[3, 0], 5] = math.inf
    l.y[l.row[4, 1], 7] = math.nan
    out = torch.empty((16, 256), dtype=torch.bfloat16, device=DEV)
    l.h.em_combine_weighted(l.y, l.w, out)
    bad = torch.zeros((16, 256), dtype=torch.bool, device=DEV)
    bad[3, 5] = bad[4, 7] = True
    assert out[~bad].isfinite().all() and not out[bad].isfinite().any()
    l.h.close()

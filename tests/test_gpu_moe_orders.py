"""The layer's calls in the orders that training and serving make of them:
decodes between a forward and its backward, several forwards before their
backwards.  Each backward's results are those of a backward that directly
follows its forward, bit for bit: the routing, the rows' places and every sum's
order depend on the forward's own inputs alone."""
import math

import pytest
import torch

from combine_ep_get_03_gb300 import ep
from combine_ep_get_03_gb300 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
R, E, k, H, F, tpr = 4, 16, 4, 256, 256, 32


@pytest.fixture(scope="module")
def weights():
    g = torch.Generator(device=DEV).manual_seed(5)
    w1 = torch.randn((E, 2 * F, H), generator=g, device=DEV) / math.sqrt(H)
    w2 = torch.randn((E, H, F), generator=g, device=DEV) / math.sqrt(F)
    return moe.ExpertWeights(w1), moe.ExpertWeights(w2)


@pytest.fixture
def layer():
    m = moe.MoELayer(R, E, k, H, F, tpr, score=ep.EP_GATE_SIGMOID, loss_coef=0.5, expert_alignment=16)
    yield m
    m.close()


def batch(seed, T=R * tpr):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    return dict(x=rand(T, H).bfloat16(), logits=rand(T, E) + 2 * rand(E), go=rand(T, H).bfloat16(),
                gl=torch.full((1,), 3.0, device=DEV))


def forward(layer, b, weights):
    return layer.forward(b["x"], b["logits"], *weights)


def backward(layer, b, saved, weights):
    return layer.backward(b["go"], b["gl"], saved, *weights)


def straight(layer, b, weights):
    out, loss, saved = forward(layer, b, weights)
    return out, loss, backward(layer, b, saved, weights)


def same(got, want):
    for name, a, b in zip(("x", "logits", "w1", "w2"), got, want):
        assert b.isfinite().all() and torch.equal(a, b), name


def test_decode_between_forward_and_backward(layer, weights):
    a, d = batch(1), batch(2, R)
    want_out, _, want = straight(layer, a, weights)
    want_dec = layer.decode(d["x"], d["logits"], *weights)
    out, _, saved = forward(layer, a, weights)
    dec = layer.decode(d["x"], d["logits"], *weights)
    same(backward(layer, a, saved, weights), want)
    assert torch.equal(out, want_out) and torch.equal(dec, want_dec)
    layer.check()


@pytest.mark.parametrize("sizes", [(R * tpr, R * tpr), (R * tpr, R * 3), (R, R * tpr)])
@pytest.mark.parametrize("order", [(0, 1), (1, 0), (0, 1, 0)])
def test_forwards_before_their_backwards(layer, weights, sizes, order):
    """Two micro-batches in flight, of one size and of two; a backward may also
    be repeated."""
    b = [batch(11, sizes[0]), batch(12, sizes[1])]
    want = [straight(layer, one, weights) for one in b]
    runs = [forward(layer, one, weights) for one in b]
    for i in order:
        same(backward(layer, b[i], runs[i][2], weights), want[i][2])
    for i in (0, 1):
        assert torch.equal(runs[i][0], want[i][0]) and torch.equal(runs[i][1], want[i][1])
    layer.check()


def test_layout_made_outside_the_layer(layer, weights):
    """The handle is the layer's own attribute: a layout made on it directly is
    not taken for the forward's."""
    a = batch(21)
    _, _, want = straight(layer, a, weights)
    _, _, saved = forward(layer, a, weights)
    other = torch.randn((R * tpr, E), device=DEV).topk(k).indices
    rows = R * tpr * k
    layer.h.em_layout_and_dispatch(other, a["x"], None, ep.EP_BF16, 1,
                                   torch.empty((rows, H), dtype=torch.bfloat16, device=DEV))
    same(backward(layer, a, saved, weights), want)


def test_backward_is_linear_in_its_gradients(layer, weights):
    """Both gradients times 2^10: every result is 2^10 times what it was, bit for
    bit, since no 128 channels are at the quantisation's floor here.  That is how
    small gradients are scaled up."""
    a = batch(31)
    _, _, saved = forward(layer, a, weights)
    one = backward(layer, a, saved, weights)
    big = layer.backward((a["go"].float() * 1024).bfloat16(), a["gl"] * 1024, saved, *weights)
    for x, y in zip(big, one):
        assert torch.equal(x, y * 1024)


def test_no_tokens_and_one_token_per_rank(layer, weights):
    """A micro-batch without tokens has gradients of zero; one of a token for each
    rank agrees with itself inside a larger batch's buffers."""
    empty = batch(41, 0)
    out, loss, saved = forward(layer, empty, weights)
    gx, gl, gw1, gw2 = backward(layer, empty, saved, weights)
    assert out.shape == (0, H) and gx.shape == (0, H) and gl.shape == (0, E) and loss.item() == 0.0
    assert not gw1.any() and not gw2.any()
    assert layer.decode(empty["x"], empty["logits"], *weights).shape == (0, H)
    few = batch(42, R)
    _, _, want = straight(layer, few, weights)
    forward(layer, batch(43), weights)
    same(straight(layer, few, weights)[2], want)
    layer.check()

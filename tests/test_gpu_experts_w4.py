"""The experts' products on 4-bit weights on the GPU, against plain 64-bit forms.

The bounds are those of the 8-bit products: e2m1 times a power of two is exact,
so a block of 128 products in the tensor core and one fused multiply-add per
block are all that rounds.
"""
import math

import pytest
import torch

from combine_ep_get_03_gb300 import ep
from combine_ep_get_03_gb300 import moe

from test_gpu_experts import LAYOUTS, Rows, U24, check8, gen, product64, silu64, sum_err, within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
VALUES = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)

WIDTHS = LAYOUTS + [([1, 16, 17, 15], "em", 1, 2), ([48, 49, 33, 32], "ll", 1, 3), ([112, 113, 16, 0, 224, 225], "em", 8, 1),
                    ([785, 3], "em", 1, 0), ([16] * 9, "ll", 1, 0), ([64, 8], "em", 1, 0)]


def unpack(q, s, N, K):
    """Weights in 64 bits from codes and exponents, by index."""
    n, k = torch.arange(N, device=DEV)[:, None], torch.arange(K, device=DEV)[None]
    code = (q[:, n, k // 2].long() >> (4 * (k % 2))) & 15
    b = s[:, n // 128, k // 128, 16 * (n % 32) + 4 * (n % 128 // 32) + k % 128 // 32]
    return VALUES.to(DEV)[code] * torch.exp2(b.double() - 127)


def weights4(E, N, K, seed):
    q, s = moe.quantize_e2m1(torch.randn((E, N, K), generator=gen(seed), device=DEV) / math.sqrt(K))
    return q, s, unpack(q, s, N, K)


@pytest.mark.parametrize("counts,layout,align,slack", WIDTHS)
@pytest.mark.parametrize("N,K", [(8, 128), (136, 256), (256, 128), (1000, 640), (520, 384)])
def test_product(counts, layout, align, slack, N, K):
    r = Rows(counts, layout, align, slack)
    xq, xs, x = r.fp8(K, 1)
    q, s, w = weights4(len(counts), N, K, 2)
    out = r.out16(N)
    ep.ep_grouped_matmul_w4(xq, xs, q, s, out, **r.args())
    y, mag = product64(r, x, w)
    within(r.read16(out), y, y.abs() * 2.0 ** -8 + sum_err(K) * mag + 1e-38, "product")


@pytest.mark.parametrize("counts,layout,align,slack", WIDTHS)
@pytest.mark.parametrize("F,K,weighted", [(128, 128, True), (384, 256, False), (256, 1152, True)])
def test_product_swiglu(counts, layout, align, slack, F, K, weighted):
    r = Rows(counts, layout, align, slack)
    xq, xs, x = r.fp8(K, 11)
    q, s, w = weights4(len(counts), 2 * F, K, 12)
    rw = None
    if weighted:
        rw = torch.full((r.rows,), math.nan, device=DEV)
        rw[r.live] = torch.randn(len(r.live), generator=gen(13), device=DEV)
        rw[r.live[:1]] = 0.0
    act, acts = r.out8(F)
    ep.ep_grouped_matmul_w4_swiglu(xq, xs, q, s, act, acts, row_weights=rw, **r.args())
    y, mag = product64(r, x, w)
    err = sum_err(K) * mag
    g, u = y.chunk(2, 1)
    eg, eu = err.chunk(2, 1)
    wt = rw[r.live].double()[:, None] if weighted else 1.0
    a = silu64(g) * u * wt
    # |silu'| <= 1.1; the activation itself in fp32 with a fast exponential and division
    ea = ((1.1 * eg) * u.abs() + (silu64(g).abs() + 1.1 * eg) * eu) * (wt.abs() if weighted else 1.0) + \
        (16 + 2 * g.abs()) * U24 * a.abs()
    v, sc = r.read8(act, acts)
    check8(v, sc, a, ea, "activations")


def test_long_contraction_many_tiles_any_sms():
    r = Rows([500, 0, 700, 260], "em", 1)
    xq, xs, x = r.fp8(7168, 3)
    q, s, w = weights4(4, 2056, 7168, 4)
    out = r.out16(2056)
    ep.ep_grouped_matmul_w4(xq, xs, q, s, out, **r.args())
    y, mag = product64(r, x, w)
    within(r.read16(out), y, y.abs() * 2.0 ** -8 + sum_err(7168) * mag, "product")
    for sms in (1, 2, 7, 100):
        again = r.out16(2056)
        ep.ep_grouped_matmul_w4(xq, xs, q, s, again, num_sms=sms, **r.args())
        assert torch.equal(again.view(torch.int16), out.view(torch.int16)), sms


@pytest.mark.parametrize("rows", [1, 20, 40, 100])
def test_every_code_and_exponents_apart(rows):
    """All 256 bytes of codes; exponents of neighbouring 32 channels and rows far
    apart; rows' scales far apart.  What is summed spans more than fp32: the
    bound is relative to the largest terms."""
    N, K = 256, 512
    r = Rows([rows], "em")
    sig = torch.exp2(torch.linspace(-30, 30, rows, device=DEV))
    xq, xs, x = r.fp8(K, 5)
    xs[:, :rows] *= sig
    x = x * sig.double()[:, None]
    q = torch.randint(0, 256, (1, N, K // 2), generator=gen(6), device=DEV, dtype=torch.int32).to(torch.uint8)
    s = torch.randint(127 - 30, 127 + 30, (1, 2, 4, 512), generator=gen(7), device=DEV, dtype=torch.int32).to(torch.uint8)
    out = r.out16(N)
    ep.ep_grouped_matmul_w4(xq, xs, q, s, out, **r.args())
    y, mag = product64(r, x, unpack(q, s, N, K))
    within(r.read16(out), y, y.abs() * 2.0 ** -8 + sum_err(K) * mag, "product")


@pytest.mark.parametrize("low,sig", [(2, 100), (230, -110)])
def test_exponents_at_both_ends(low, sig):
    """Exponents near 2^-125 and 2^103, the rows' scales at the other end."""
    N, K = 128, 256
    r = Rows([40], "em")
    xq, xs, x = r.fp8(K, 45)
    xs[:, :40] *= 2.0 ** sig
    x = x * 2.0 ** sig
    q = torch.randint(0, 256, (1, N, K // 2), generator=gen(46), device=DEV, dtype=torch.int32).to(torch.uint8)
    s = torch.randint(low, low + 8, (1, 1, 2, 512), generator=gen(47), device=DEV, dtype=torch.int32).to(torch.uint8)
    out = r.out16(N)
    ep.ep_grouped_matmul_w4(xq, xs, q, s, out, **r.args())
    y, mag = product64(r, x, unpack(q, s, N, K))
    # products below fp32's smallest normal number may count as 0: 256 of them, times the row's scale
    tiny = 256 * 2.0 ** -126 * xs[:, :40].max().item()
    within(r.read16(out), y, y.abs() * 2.0 ** -8 + sum_err(K) * mag + tiny, "product")


def test_special_scales_and_values_stay_in_their_rows():
    """A NaN exponent ruins its weight row only, a NaN code or an infinite scale
    of x its token only."""
    N, K = 256, 256
    r = Rows([30], "em")
    xq, xs, x = r.fp8(K, 8)
    q, s, w = weights4(1, N, K, 9)
    s[0, 0, 1, 16 * (5 % 32) + 2] = 255  # row 5, channels 192..223
    q[0, 5] = 0x22
    xq.view(torch.uint8)[7, 3] = 0x7F
    xs[1, 9] = math.inf
    out = r.out16(N)
    ep.ep_grouped_matmul_w4(xq, xs, q, s, out, **r.args())
    got = r.read16(out)
    y, mag = product64(r, x, w)
    keep = torch.tensor([i for i in range(30) if i not in (7, 9)], device=DEV)
    cols = torch.tensor([i for i in range(N) if i != 5], device=DEV)
    within(got[keep][:, cols], y[keep][:, cols], y[keep][:, cols].abs() * 2.0 ** -8 + sum_err(K) * mag[keep][:, cols], "product")
    assert got[:, 5].isnan().all() and got[7].isnan().all() and not got[9].isfinite().any()


def test_groups_that_do_not_fit_are_cut():
    E, N, K = 3, 128, 128
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    r = Rows([40, 30, 20], "em", 1)
    xq, xs, x = r.fp8(K, 21)
    q, s, w = weights4(E, N, K, 22)
    y, mag = product64(r, x, w)
    out = r.out16(N)
    count = torch.tensor([40, 30, 2000], dtype=torch.int32, device=DEV)
    ep.ep_grouped_matmul_w4(xq, xs, q, s, out, count, r.offset, device_status=st)
    assert st.item() == ep.EP_ERR_CAPACITY
    within(out.double(), y, y.abs() * 2.0 ** -8 + sum_err(K) * mag, "product")
    # overlapping groups whose tiles are more than the buffers have: no fault, reported
    st.zero_()
    many = torch.full((64,), 90, dtype=torch.int32, device=DEV)
    q64, s64 = q[:1].expand(64, -1, -1).contiguous(), s[:1].expand(64, -1, -1, -1).contiguous()
    ep.ep_grouped_matmul_w4(xq, xs, q64, s64, out, many, torch.zeros(64, dtype=torch.int32, device=DEV), device_status=st)
    ep.ep_grouped_matmul_w4(xq, xs, q64, s64, out, many * -1, torch.full((64,), -5, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()


def test_4096_groups():
    E, N, K = 4096, 128, 128
    counts = [0] * E
    for e, c in ((0, 3), (77, 20), (4095, 130)):
        counts[e] = c
    r = Rows(counts, "em", 4)
    xq, xs, x = r.fp8(K, 31)
    q, s, w = weights4(2, N, K, 32)
    pick = torch.arange(E, device=DEV) % 2
    q, s, w = q[pick].contiguous(), s[pick].contiguous(), w[pick]
    out = r.out16(N)
    ep.ep_grouped_matmul_w4(xq, xs, q, s, out, **r.args())
    y, mag = product64(r, x, w)
    within(r.read16(out), y, y.abs() * 2.0 ** -8 + sum_err(K) * mag, "product")


# As many stages as fit are five where tiles have 17 to 64 tokens, and with 16 where
# there are thousands of groups: every block of k has to wait for its own fill.
@pytest.mark.parametrize("counts,layout,K", [([33, 0, 7, 20, 1, 16], "ll", 6272), ([30, 2, 11, 5], "em", 1152), ([64, 9, 50], "em", 1408),
                                             ([3] * 2500, "em", 640)])
def test_stages_in_odd_numbers_and_many_launches(counts, layout, K):
    E, F = len(counts), 256
    r = Rows(counts, layout, 1, 3)
    xq, xs, x = r.fp8(K, 41)
    some = min(E, 6)
    q, s, w = weights4(some, 2 * F, K, 42)
    if some < E:
        pick = torch.arange(E, device=DEV) % some
        q, s, w = q[pick], s[pick], w[pick]
    out, (act, acts) = r.out16(2 * F), r.out8(F)
    ep.ep_grouped_matmul_w4(xq, xs, q, s, out, **r.args())
    y, mag = product64(r, x, w)
    within(r.read16(out), y, y.abs() * 2.0 ** -8 + sum_err(K) * mag, "product")
    ep.ep_grouped_matmul_w4_swiglu(xq, xs, q, s, act, acts, **r.args())
    first = out.clone(), act.clone(), acts.clone()
    for _ in range(200):
        ep.ep_grouped_matmul_w4(xq, xs, q, s, out, **r.args())
        ep.ep_grouped_matmul_w4_swiglu(xq, xs, q, s, act, acts, **r.args())
    for a, b in zip(first, (out, act, acts)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_reads_64_bit_offsets():
    """Live rows past 2^31 elements of x and out, weights past 2^31 codes."""
    M, E, K, N = 45000, 8, 7168, 7168
    x = torch.empty((E, M, K), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    xs = torch.empty((E, M, K // 128), device=DEV)
    out = torch.empty((E, M, N), dtype=torch.bfloat16, device=DEV)
    r = Rows([5], "em")
    xq, sc, xd = r.fp8(K, 41)
    x[E - 1, :5], xs[E - 1, :5] = xq, sc[:, :5].t()
    count = torch.tensor([0] * (E - 1) + [5], dtype=torch.int32, device=DEV)
    q, s, w = weights4(1, N, K, 42)
    big = torch.zeros((90, N, K // 2), dtype=torch.uint8, device=DEV)
    big[89] = q[0]
    scales = torch.zeros((90,) + s.shape[1:], dtype=torch.uint8, device=DEV)
    scales[89] = s[0]
    assert x.numel() > 2 ** 31 and big.numel() > 2 ** 31
    y, mag = xd @ w[0].t(), xd.abs() @ w[0].abs().t()
    ep.ep_grouped_matmul_w4(x, xs, big[90 - E:], scales[90 - E:], out, count)
    within(out[E - 1, :5].double(), y, y.abs() * 2.0 ** -8 + sum_err(K) * mag, "product")
    r = Rows([0] * 89 + [5], "em")
    out2 = r.out16(N)
    ep.ep_grouped_matmul_w4(xq, sc, big, scales, out2, r.count, r.offset)
    within(r.read16(out2), y, y.abs() * 2.0 ** -8 + sum_err(K) * mag, "product")


def test_streams_graphs_and_dependent_chains():
    """First and second product back to back, their input refilled between:
    eager, on another stream and replayed from a graph the same bits."""
    E, H, F = 6, 512, 256
    r = Rows([3, 0, 40, 17, 1, 64], "ll", 1, 4)
    xq, xs, _ = r.fp8(H, 51)
    q1, s1, _ = weights4(E, 2 * F, H, 52)
    q2, s2, _ = weights4(E, H, F, 53)
    (act, acts), y = r.out8(F), r.out16(H)

    def step():
        ep.ep_grouped_matmul_w4_swiglu(xq, xs, q1, s1, act, acts, **r.args())
        ep.ep_grouped_matmul_w4(act, acts, q2, s2, y, **r.args())

    step()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(54, 58):
        new, ns, _ = r.fp8(H, seed)
        xq.copy_(new), xs.copy_(ns)
        step()
        torch.cuda.synchronize()
        want = r.read16(y).clone()
        y.fill_(-5.5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r.read16(y), want)
        y.fill_(-5.5)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(3):
                step()
        side.synchronize()
        assert torch.equal(r.read16(y), want)


def test_binding_refusals():
    r = Rows([5, 3], "em", 4)
    xq, xs, _ = r.fp8(256, 61)
    q, s, _ = weights4(2, 128, 256, 62)
    ok = dict(x=xq, x_scales=xs, w=q, w_scales=s, out=r.out16(128), group_count=r.count, group_offset=r.offset)
    ep.ep_grouped_matmul_w4(**ok)
    for bad in (dict(w=q[:1]), dict(w=q[:, :, :64].contiguous()), dict(w=q.view(torch.int8)), dict(w=q.transpose(1, 2)),
                dict(w_scales=s[:, :, :1].contiguous()), dict(w_scales=s.view(2, 1, 1024)), dict(w_scales=None), dict(x=xq.float()),
                dict(out=r.out16(256)), dict(w=torch.empty(q.numel() + 16, dtype=torch.uint8, device=DEV)[16:].view(q.shape))):
        with pytest.raises((ValueError, TypeError, ep.EPError)):
            ep.ep_grouped_matmul_w4(**{**ok, **bad})
    act, acts = r.out8(128)
    with pytest.raises(ValueError):  # weights of half the width
        ep.ep_grouped_matmul_w4_swiglu(xq, xs, q, s, act, acts, r.count, r.offset)


def test_layer_decodes_and_prefills_with_4_bit_weights():
    """Against the layer in 64 bits on the dequantised weights: e4m3 rounds a
    factor by 0.026 in the root mean square, twice in a row."""
    torch.manual_seed(7)
    R, E, k, H, F, tpr = 2, 8, 2, 256, 128, 40
    T = R * tpr
    w1 = moe.ExpertWeights4(torch.randn((E, 2 * F, H), device=DEV) / H ** 0.5)
    w2 = moe.ExpertWeights4(torch.randn((E, H, F), device=DEV) / F ** 0.5)
    W1, W2 = unpack(w1.q, w1.s, 2 * F, H), unpack(w2.q, w2.s, H, F)
    x, logits = torch.randn((T, H), device=DEV).bfloat16(), torch.randn((T, E), device=DEV)
    for weigh in (False, True):
        layer = moe.MoELayer(R, E, k, H, F, tpr, weigh_in_combine=weigh)
        out, _, saved = layer.forward(x, logits, w1, w2)
        dec = layer.decode(x, logits, w1, w2)
        layer.check()
        assert saved is None
        idx = logits.topk(k, 1).indices
        wt = torch.softmax(logits.double().gather(1, idx), 1)
        ref = torch.zeros((T, H), dtype=torch.float64, device=DEV)
        for e in range(E):
            t, j = (idx == e).nonzero(as_tuple=True)
            a, b = (x[t].double() @ W1[e].t()).chunk(2, 1)
            ref = ref.index_add(0, t, (silu64(a) * b * wt[t, j][:, None]) @ W2[e].t())
        for got in (out, dec):
            assert ((got.double() - ref).norm() / ref.norm()).item() < 3 * math.sqrt(4) * 0.026
        layer.close()

"""The ends of the experts' and the gate's ranges: large gates, rows whose scales
lie far apart, tiny gradients, experts that hardly any token looks at, and row
buffers beyond 2^31 elements.  Bounds as derived in test_gpu_experts.py unless a
test derives its own."""
import math

import pytest
import torch

from combine_ep_get_03_gb300 import ep
from test_gpu_experts import (DEV, F8, U24, Rows, check8, gen, quantize, run_gate, silu64, sum_err, weights,
                              within)

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


def weight_grad(r, y, x):
    dw = torch.full((len(r.counts), y[0].shape[-1], x[0].shape[-1]), math.nan, dtype=torch.bfloat16, device=DEV)
    ep.ep_grouped_weight_grad(*y, *x, dw, **r.args())
    return dw


def scale_rows(r, scales, values, factor):
    """Multiplies the live rows' scales (and, in 64 bits, their values)."""
    r._scales(scales)[r.live] *= factor[:, None].float()
    return values * factor[:, None]


def test_weight_grad_rounds_each_factor_once():
    """Scales that f16 rounds by almost 2^-11 of themselves: a factor is code *
    scale rounded once, not the code times a rounded scale, which would be off
    by 2^-10 on every term.  Against the sum of such factors in 64 bits only the
    fp32 sum's error and half a unit of the bf16 result (8 bits) remain."""
    n = 64
    r = Rows([n], "em")
    yq, ys, _ = r.fp8(256, 31)
    xq, xs, _ = r.fp8(384, 32)
    j = torch.randint(0, 6, (n, 1), generator=gen(33), device=DEV)
    s = (1 + 2.0 ** -11 - 2.0 ** -20) * torch.exp2(-j.double())
    factors = []
    for q, scales in ((yq, ys), (xq, xs)):
        q.view(torch.uint8)[r.live] &= 0x7F  # all terms of one sign
        r._scales(scales)[r.live] = s.float().expand(-1, scales.shape[0])
        e = 2.0 ** (math.floor(math.log2(s.max().item())) - 6)
        factors.append((q[r.live].double() * s / e).half().double() * e)
    ref = factors[0].t() @ factors[1]
    dw = weight_grad(r, (yq, ys), (xq, xs))
    half_unit = torch.exp2(torch.floor(torch.log2(ref)) - 8)
    within(dw[0].double(), ref, half_unit + ref * 2 * n * U24, "weight gradient")


@pytest.mark.parametrize("spread", [12, 24, 30, 36])
def test_weight_grad_of_opposed_row_scales(spread):
    """Row scales over 2^spread in either operand and opposed in the two, so
    that every row's products are alike: a factor is off by 2^-11 of itself and
    2^-39 of the largest possible in its channels."""
    n = 96
    r = Rows([n, 5], "em")
    up = torch.exp2(torch.linspace(0, spread, n, device=DEV).round().double())
    up = torch.cat([up, torch.ones(5, dtype=torch.float64, device=DEV)])
    yq, ys, y = r.fp8(256, 34)
    xq, xs, x = r.fp8(128, 35)
    y, x = scale_rows(r, ys, y, up), scale_rows(r, xs, x, 1 / up)
    dw = weight_grad(r, (yq, ys), (xq, xs))
    for e, at in r.spans():
        ref, mag = y[at].t() @ x[at], y[at].abs().t() @ x[at].abs()
        lost = []
        for t, scales in ((y, ys), (x, xs)):
            top = r._scales(scales)[r.live][at].double().amax(0) * 448.0
            lost.append((top * 2.0 ** -39).repeat_interleave(128)[None, :].expand(len(t[at]), -1))
        bound = ref.abs() * 2.0 ** -8 + mag * (2.0 ** -10 * (1 + 2.0 ** -11) + 2 * n * U24)
        bound += 1.001 * (lost[0].t() @ x[at].abs() + y[at].abs().t() @ lost[1] + lost[0].t() @ lost[1])
        within(dw[e].double(), ref, bound, f"weight gradient of expert {e}")


@pytest.mark.parametrize("ey,ex", [(-100, 60), (-110, 0), (0, -110), (100, -90), (-70, 100), (116, -116), (60, 60)])
def test_weight_grad_of_tiny_and_huge_scales(ey, ex):
    """Scales anywhere in fp32's normal range (2^-8 of the factor here, or more):
    powers of two change nothing but the result's own exponent."""
    r = Rows([70, 0, 3], "em", 4)
    yq, ys, y = r.fp8(256, 36)
    xq, xs, x = r.fp8(384, 37)
    plain = weight_grad(r, (yq, ys), (xq, xs))
    n = len(r.live)
    scale_rows(r, ys, y, torch.full((n,), 2.0 ** ey, dtype=torch.float64, device=DEV))
    scale_rows(r, xs, x, torch.full((n,), 2.0 ** ex, dtype=torch.float64, device=DEV))
    dw = weight_grad(r, (yq, ys), (xq, xs))
    want = plain.double() * 2.0 ** (ey + ex)
    assert torch.equal(dw, torch.where(want.abs() < 2.0 ** 127, want, want.sign() * math.inf).bfloat16())


def test_weight_grad_beside_an_infinite_row():
    """A row of infinite scale makes its terms infinite, of the codes' signs;
    the other rows stay finite beside it."""
    n = 40
    r = Rows([n], "em")
    yq, ys, _ = r.fp8(128, 38)
    xq, xs, _ = r.fp8(128, 39)
    for q in (yq, xq):
        q.view(torch.uint8)[7] = torch.where(torch.arange(128, device=DEV) % 3 == 0, 0x38, 0xB8).to(torch.uint8)  # 1, -1
    ys[0, :n] *= 2.0 ** 30
    ys[0, 7] = math.inf
    dw = weight_grad(r, (yq, ys), (xq, xs))
    want = yq.double()[7][:, None] * xq.double()[7][None, :] * math.inf
    assert torch.equal(dw[0].double(), want)


@pytest.mark.parametrize("T", [16, 17, 300, 4096, 40000])
@pytest.mark.parametrize("sms", [0, 1, 7])
@pytest.mark.parametrize("score", [ep.EP_GATE_SOFTMAX, ep.EP_GATE_SIGMOID])
def test_gate_mean_probability_of_a_cold_expert(T, sms, score):
    """An expert that every token gives about 1e-14: its mean comes out to fp32's
    rounding and half a step of 2^-(63 - ceil(log2 T)) for every block that adds."""
    E, k = 64, 4
    l = torch.randn((T, E), generator=gen(41), device=DEV)
    l[:, 9] -= 28.0
    o = run_gate(l, k, score=score, num_sms=sms)
    l64 = l.double()
    s = torch.exp(l64) if score == ep.EP_GATE_SOFTMAX else torch.sigmoid(l64)
    prob = (s / s.sum(1, keepdim=True)).mean(0)
    step = 2.0 ** -(63 - math.ceil(math.log2(T)))
    blocks = min(-(-T // 16), 2 * (sms or 152))
    # exponentials to 2^-21 and (|l| + 4) u24, sums over E and over the tokens of a warp
    tol = (E / 32 + 64 + 40 + T / (16 * blocks)) * U24
    within(o["prob"].double(), prob, tol * prob + 0.5 * step * blocks / T, "mean probabilities")


def test_swiglu_backward_of_tiny_gradients():
    """As the header says: steps of 1e-4 / 448 / 512 for 128 channels below 1e-4,
    0 below half a step, and every bit back when the gradient is scaled up."""
    F, n = 256, 20
    r = Rows([n], "em")
    pq, ps, p = r.fp8(2 * F, 51)
    d = torch.randn((n, F), generator=gen(52), device=DEV).bfloat16()
    g, u = p.chunk(2, 1)
    sg = torch.sigmoid(g)
    slope = torch.cat([u * sg * (1 + g * (1 - sg)), silu64(g)], 1)
    rel = torch.cat([u.abs() * sg * (1 + g.abs() + silu64(g).abs()), silu64(g).abs()], 1) * (16 + 2 * g.abs().repeat(1, 2)) * U24
    for e in (-27, -3):
        da = (d.double() * 2.0 ** e).bfloat16()
        dp, dps = r.out8(2 * F)
        ep.ep_grouped_swiglu_backward(da, pq, ps, dp, dps, **r.args())
        v, sc = r.read8(dp, dps)
        da2 = da.double().repeat(1, 2)
        check8(v, sc, da2 * slope, da2.abs() * rel, "gradient")
        if e == -27:  # the floor's scale everywhere
            assert (sc == sc.flatten()[0]).all() and (v != 0).any()
            assert (v[(da2 * slope).abs() < 2.1e-10] == 0).all()
        else:  # no group at the floor
            assert (sc > 1.01e-4 / 448).all()


def test_swiglu_and_its_backward_read_64_bit_offsets():
    """The only live rows lie past 2^31 elements of x, of both outputs and of the
    gradients."""
    M, G, K, F, n = 45000, 8, 6016, 6144, 5
    f8 = lambda w: torch.empty((G, M, w), dtype=torch.uint8, device=DEV)  # noqa: E731
    f32 = lambda w: torch.empty((G, M, w), device=DEV)  # noqa: E731
    x, xs, act, acts, pre, pres = f8(K), f32(K // 128), f8(F), f32(F // 128), f8(2 * F), f32(2 * F // 128)
    assert min(x.numel(), act.numel()) > 2 ** 31
    q, s = quantize(torch.randn((n, K), generator=gen(61), device=DEV))
    x[G - 1, :n], xs[G - 1, :n] = q.view(torch.uint8), s
    count = torch.tensor([0] * (G - 1) + [n], dtype=torch.int32, device=DEV)
    wq, ws, w = weights(1, 2 * F, K, 62)
    w8 = wq.view(torch.uint8).expand(G, -1, -1).contiguous()
    ep.ep_grouped_matmul_swiglu(x, xs, w8, ws.expand(G, -1, -1).contiguous(), act, acts, count, pre=pre, pre_scales=pres)
    del w8
    xd = q.double() * s.double().repeat_interleave(128, 1)
    y, err = xd @ w[0].t(), sum_err(K) * (xd.abs() @ w[0].abs().t())
    read = lambda t, sc: t[G - 1, :n].view(F8).double() * sc[G - 1, :n].double().repeat_interleave(128, 1)  # noqa: E731
    check8(read(pre, pres), pres[G - 1, :n].double(), y, err, "pre-activations")
    g, u = y.chunk(2, 1)
    eg, eu = err.chunk(2, 1)
    a = silu64(g) * u
    ea = 1.1 * eg * u.abs() + (silu64(g).abs() + 1.1 * eg) * eu + (16 + 2 * g.abs()) * U24 * a.abs()
    check8(read(act, acts), acts[G - 1, :n].double(), a, ea, "activations")

    del x, xs, act, acts
    da = torch.empty((G, M, F), dtype=torch.bfloat16, device=DEV)
    da[G - 1, :n] = torch.randn((n, F), generator=gen(63), device=DEV).bfloat16()
    dp, dps = f8(2 * F), f32(2 * F // 128)
    ep.ep_grouped_swiglu_backward(da, pre, pres, dp, dps, count)
    g, u = read(pre, pres).chunk(2, 1)
    d, sg = da[G - 1, :n].double(), torch.sigmoid(g)
    mag = torch.cat([(d * u).abs() * sg * (1 + g.abs() + silu64(g).abs()), (d * silu64(g)).abs()], 1)
    check8(read(dp, dps), dps[G - 1, :n].double(), torch.cat([d * u * sg * (1 + g * (1 - sg)), d * silu64(g)], 1),
           mag * (16 + 2 * g.abs().repeat(1, 2)) * U24, "gradient")


def test_weight_grad_and_product_of_weights_beyond_2_31_elements():
    """The last group's weights, and their gradient, lie past 2^31 elements."""
    G, N, K, n = 66, 4096, 8192, 70
    r = Rows([0] * (G - 1) + [n], "em")
    yq, ys, y = r.fp8(N, 64, sigma=1e-2)
    xq, xs, x = r.fp8(K, 65)
    dw = torch.full((G, N, K), math.nan, dtype=torch.bfloat16, device=DEV)
    assert (G - 1) * N * K > 2 ** 31
    ep.ep_grouped_weight_grad(yq, ys, xq, xs, dw, **r.args())
    ref, mag = y.t() @ x, y.abs().t() @ x.abs()
    within(dw[G - 1].double(), ref, ref.abs() * 2.0 ** -8 + mag * 2.0 ** -8.9, "weight gradient")
    assert all((dw[e] == 0).all() for e in range(G - 1))
    del dw
    w8 = torch.empty((G, N, K), dtype=torch.uint8, device=DEV)
    wq, ws, w = weights(1, N, K, 66)
    w8[G - 1] = wq[0].view(torch.uint8)
    scales = torch.empty((G, N // 128, K // 128), device=DEV)
    scales[G - 1] = ws[0]
    out = r.out16(N)
    ep.ep_grouped_matmul(xq, xs, w8, scales, out, **r.args())
    p, pmag = x @ w[0].t(), x.abs() @ w[0].abs().t()
    within(r.read16(out), p, p.abs() * 2.0 ** -8 + sum_err(K) * pmag, "product")


def test_weight_grad_of_rows_beyond_2_31_elements():
    M, G, N, K, n = 1400000, 4, 128, 512, 90
    y, x = (torch.empty((G, M, w), dtype=torch.uint8, device=DEV) for w in (N, K))
    ys, xs = (torch.empty((G, M, w // 128), device=DEV) for w in (N, K))
    assert (G - 1) * M * K > 2 ** 31
    vals = []
    for q, s, w in ((y, ys, N), (x, xs, K)):
        c, sc = quantize(torch.randn((n, w), generator=gen(w), device=DEV))
        q[G - 1, :n], s[G - 1, :n] = c.view(torch.uint8), sc
        vals.append(c.double() * sc.double().repeat_interleave(128, 1))
    dw = torch.empty((G, N, K), dtype=torch.bfloat16, device=DEV)
    ep.ep_grouped_weight_grad(y, ys, x, xs, dw, torch.tensor([0] * (G - 1) + [n], dtype=torch.int32, device=DEV))
    ref, mag = vals[0].t() @ vals[1], vals[0].abs().t() @ vals[1].abs()
    within(dw[G - 1].double(), ref, ref.abs() * 2.0 ** -8 + mag * 2.0 ** -8.9, "weight gradient")
    assert (dw[:G - 1] == 0).all()


def test_gate_reads_64_bit_offsets():
    """The only unmasked tokens lie past 2^31 logits."""
    T, E, k, n = 560000, 4000, 5, 6
    l = torch.empty((T, E), dtype=torch.bfloat16, device=DEV)
    assert (T - n) * E > 2 ** 31
    l[T - n:] = torch.randn((n, E), generator=gen(67), device=DEV).bfloat16()
    mask = torch.zeros(T, dtype=torch.bool, device=DEV)
    mask[T - n:] = True
    o = run_gate(l, k, mask=mask)
    tail = l[T - n:].contiguous()
    small = run_gate(tail, k)
    assert torch.equal(o["idx"][T - n:], small["idx"]) and torch.equal(o["w"][T - n:], small["w"])
    assert (o["idx"][:T - n] == -1).all() and torch.equal(o["count"], small["count"])
    dw = torch.randn((T, k), generator=gen(68), device=DEV)
    one = torch.ones(1, device=DEV)
    grad, want = torch.full_like(l, 7.0), torch.empty_like(tail)
    ep.ep_gate_backward(l, o["idx"], o["count"], dw, one, grad, loss_coef=0.5, token_mask=mask)
    ep.ep_gate_backward(tail, small["idx"], small["count"], dw[T - n:].contiguous(), one, want, loss_coef=0.5)
    assert torch.equal(grad[T - n:], want) and not grad[:T - n].any()

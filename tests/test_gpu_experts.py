"""The gate, the experts' products, the activation's backward and the weight
gradient on the GPU, against plain 64-bit forms of their definitions.

Tolerances, derived from the arithmetic (u24 = 2^-24, fp32's unit roundoff):
* bf16 results: half a unit in the last place, 2^-8 of the value at most, plus
  the fp32 sum's error, at most (2 * 128 + K/128 + 4) u24 times the sum of the
  terms' magnitudes (a block of 128 products inside the tensor core, taken at
  two roundings each, then one fused multiply-add per block).
* e4m3 results, compared as code * scale: half a step, 2^-4 of the value (2^-10
  of the group's scale below e4m3's normal range), plus the relative error of
  what was rounded; scales: that relative error alone.
* weight gradient: each operand carries a scale and a product rounded to 11
  bits, (1 + 2^-11)^4 - 1 < 2^-8.9 of the terms' magnitudes, plus the bf16
  rounding.
* gate: exponentials to 2^-21, a sum over E and a division.
"""
import math

import numpy as np
import pytest
import torch

from combine_ep_get_03_gb300 import ep
from combine_ep_get_03_gb300 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn
U24 = 2.0 ** -24


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def quantize(v):
    """fp32 [rows, width] -> codes, scales [rows, width/128]."""
    b = v.float().unflatten(-1, (-1, 128))
    a = b.abs().amax(-1, keepdim=True).clamp_min(1e-4)
    return (b * (448.0 / a)).flatten(-2).to(F8), (a / 448.0).squeeze(-1)


class Rows:
    """Groups of rows in one of the two layouts.  Rows of no group hold NaN
    codes and scales, outputs a sentinel that must survive."""

    def __init__(self, counts, layout, align=1, slack=0):
        self.counts, self.layout = list(counts), layout
        E = len(counts)
        if layout == "em":
            start = np.concatenate([[0], np.cumsum([-(-c // align) * align for c in counts])])
            self.start, self.rows = start[:-1], int(start[-1]) + slack
            self.offset = torch.tensor(start, dtype=torch.int32, device=DEV)
            self.lead = (self.rows,)
        else:
            M = max(max(counts), 1) + slack
            self.start, self.rows = np.arange(E) * M, E * M
            self.offset = None
            self.lead = (E, M)
        self.count = torch.tensor(self.counts, dtype=torch.int32, device=DEV)
        live = np.concatenate([s + np.arange(c) for s, c in zip(self.start, self.counts)]).astype(np.int64)
        self.live = torch.from_numpy(live).to(DEV)
        dead = np.ones(self.rows, bool)
        dead[live] = False
        self.dead = torch.from_numpy(dead.nonzero()[0]).to(DEV)

    def spans(self):
        at = 0
        for e, c in enumerate(self.counts):
            yield e, slice(at, at + c)
            at += c

    def args(self, **kw):
        return dict(group_count=self.count, group_offset=self.offset, **kw)

    def scale_shape(self, g):
        return (g, (self.rows + 3) // 4 * 4 + 4) if self.layout == "em" else self.lead + (g,)

    def fp8(self, width, seed, sigma=1.0, row_sigma=None):
        """(codes, scales) buffers and the live rows' values in 64 bits."""
        v = torch.randn((len(self.live), width), generator=gen(seed), device=DEV) * sigma
        if row_sigma is not None:
            v *= row_sigma[:, None]
        q, s = quantize(v)
        data = torch.full((self.rows, width), 0x7F, dtype=torch.uint8, device=DEV)
        data[self.live] = q.view(torch.uint8)
        scales = torch.full(self.scale_shape(width // 128), math.nan, device=DEV)
        self._scales(scales)[self.live] = s
        return data.view(F8).view(self.lead + (width,)), scales, q.double() * s.double().repeat_interleave(128, 1)

    def _scales(self, t):
        return t.t()[:self.rows] if self.layout == "em" else t.view(self.rows, -1)

    def out8(self, width):
        return (torch.full(self.lead + (width,), 0x5A, dtype=torch.uint8, device=DEV).view(F8),
                torch.full(self.scale_shape(width // 128), 7.25, device=DEV))

    def read8(self, q, s):
        """Live rows of an output pair: values and scales; the rest must be untouched."""
        raw = q.view(torch.uint8).view(self.rows, -1)
        sc = self._scales(s)
        assert (raw[self.dead] == 0x5A).all() and (sc[self.dead] == 7.25).all(), "rows outside the groups were written"
        s = sc[self.live].double()
        return raw[self.live].view(F8).double() * s.repeat_interleave(128, 1), s

    def out16(self, width):
        return torch.full(self.lead + (width,), -5.5, dtype=torch.bfloat16, device=DEV)

    def read16(self, t):
        t = t.view(self.rows, -1)
        assert (t[self.dead] == -5.5).all(), "rows outside the groups were written"
        return t[self.live].double()


def weights(E, N, K, seed):
    q, s = moe.quantize_blocks(torch.randn((E, N, K), generator=gen(seed), device=DEV) / math.sqrt(K))
    full = q.double() * s.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)
    return q, s, full


def within(got, ref, bound, what):
    over = (got - ref).abs() - bound
    assert not got.isnan().any() and (over <= 0).all(), f"{what}: over the bound by {over.max().item():.3g}"


def check8(got, scales, exact, err, what):
    """got = code * scale against exact values whose own error is at most err."""
    amax = (exact.abs() + err).unflatten(-1, (-1, 128)).amax(-1).clamp_min(1e-4)
    group_err = err.unflatten(-1, (-1, 128)).amax(-1)
    s = exact.abs().unflatten(-1, (-1, 128)).amax(-1).clamp_min(1e-4) / 448.0
    within(scales, s, group_err / 448.0 + 4 * U24 * amax / 448.0, what + " scales")
    step = torch.maximum(exact.abs() * 2.0 ** -4, (scales * 2.0 ** -10).repeat_interleave(128, 1))
    within(got, exact, step * (1 + 1e-6) + 2 * err + 8 * U24 * exact.abs(), what)


def product64(rows, x, w):
    """The products of every live row and the sums of their terms' magnitudes."""
    y = torch.empty((x.shape[0], w.shape[1]), dtype=torch.float64, device=DEV)
    mag = torch.empty_like(y)
    for e, at in rows.spans():
        y[at] = x[at] @ w[e].t()
        mag[at] = x[at].abs() @ w[e].abs().t()
    return y, mag


def sum_err(K):
    return (2 * 128 + K / 128 + 4) * U24


LAYOUTS = [
    # counts, layout, alignment, slack
    ([1], "em", 1, 0), ([1], "ll", 1, 0), ([0, 0, 5, 0], "em", 4, 3), ([0, 3, 0, 0], "ll", 1, 2),
    ([127, 128, 129, 0, 1], "em", 1, 5), ([127, 128, 129, 0, 1], "ll", 1, 3), ([300, 2, 64], "em", 128, 0),
    ([256, 257, 31], "em", 16, 0), ([0], "em", 1, 7), ([0, 0], "ll", 1, 4)]


@pytest.mark.parametrize("counts,layout,align,slack", LAYOUTS)
@pytest.mark.parametrize("N,K", [(8, 128), (136, 256), (256, 128), (1000, 384)])
def test_product(counts, layout, align, slack, N, K):
    r = Rows(counts, layout, align, slack)
    xq, xs, x = r.fp8(K, 1)
    q, s, w = weights(len(counts), N, K, 2)
    out = r.out16(N)
    ep.ep_grouped_matmul(xq, xs, q, s, out, **r.args())
    y, mag = product64(r, x, w)
    within(r.read16(out), y, y.abs() * 2.0 ** -8 + sum_err(K) * mag + 1e-38, "product")


def test_product_long_contraction_and_many_tiles():
    r = Rows([500, 0, 700, 260], "em", 1)
    xq, xs, x = r.fp8(7168, 3)
    q, s, w = weights(4, 2056, 7168, 4)
    out = r.out16(2056)
    ep.ep_grouped_matmul(xq, xs, q, s, out, **r.args())
    y, mag = product64(r, x, w)
    within(r.read16(out), y, y.abs() * 2.0 ** -8 + sum_err(7168) * mag, "product")
    # the same bits on any number of SMs
    for sms in (1, 2, 7, 100):
        again = r.out16(2056)
        ep.ep_grouped_matmul(xq, xs, q, s, again, num_sms=sms, **r.args())
        assert torch.equal(again.view(torch.int16), out.view(torch.int16)), sms


def test_product_rows_of_extreme_scales():
    """Rows 2^-60 to 2^60 apart in one tile, and infinities and NaN in a row of
    their own: no row changes another."""
    r = Rows([64], "em")
    sig = torch.exp2(torch.linspace(-60, 60, 64, device=DEV))
    xq, xs, x = r.fp8(256, 5)
    xs[:, :64] *= sig
    x = x * sig.double()[:, None]
    q, s, w = weights(1, 256, 256, 6)
    xq.view(torch.uint8)[7, 3] = 0x7F  # NaN code
    xs[1, 9] = math.inf
    out = r.out16(256)
    ep.ep_grouped_matmul(xq, xs, q, s, out, **r.args())
    got = r.read16(out)
    y, mag = product64(r, x, w)
    keep = [i for i in range(64) if i not in (7, 9)]
    within(got[keep], y[keep], y[keep].abs() * 2.0 ** -8 + sum_err(256) * mag[keep], "product")
    assert got[7].isnan().all() and not got[9].isfinite().any()


def test_product_reads_64_bit_offsets():
    """The only live rows lie past 2^31 elements of x and of out."""
    M, E, K, N = 45000, 8, 7168, 7168
    x = torch.empty((E, M, K), dtype=torch.uint8, device=DEV).view(F8)
    xs = torch.empty((E, M, K // 128), device=DEV)
    out = torch.empty((E, M, N), dtype=torch.bfloat16, device=DEV)
    assert x.numel() > 2 ** 31 and out.numel() > 2 ** 31
    v = torch.randn((5, K), generator=gen(7), device=DEV)
    q, s = quantize(v)
    x[E - 1, :5], xs[E - 1, :5] = q, s
    count = torch.tensor([0] * (E - 1) + [5], dtype=torch.int32, device=DEV)
    wq, ws = moe.quantize_blocks(torch.randn((1, N, K), generator=gen(8), device=DEV) / math.sqrt(K))
    wq8 = wq.view(torch.uint8).expand(E, N, K).contiguous().view(F8)
    ep.ep_grouped_matmul(x, xs, wq8, ws.expand(E, -1, -1).contiguous(), out, count)
    w = wq[0].double() * ws[0].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    xd = q.double() * s.double().repeat_interleave(128, 1)
    y, mag = xd @ w.t(), xd.abs() @ w.abs().t()
    within(out[E - 1, :5].double(), y, y.abs() * 2.0 ** -8 + sum_err(K) * mag, "product")


def silu64(g):
    return g * torch.sigmoid(g)


@pytest.mark.parametrize("counts,layout,align,slack", LAYOUTS)
@pytest.mark.parametrize("F,K,weighted,keep", [(128, 128, True, True), (384, 256, False, True), (256, 384, True, False)])
def test_product_swiglu(counts, layout, align, slack, F, K, weighted, keep):
    r = Rows(counts, layout, align, slack)
    xq, xs, x = r.fp8(K, 11)
    q, s, w = weights(len(counts), 2 * F, K, 12)
    rw = None
    if weighted:
        rw = torch.full((r.rows,), math.nan, device=DEV)
        rw[r.live] = torch.randn(len(r.live), generator=gen(13), device=DEV)
        rw[r.live[:1]] = 0.0
    act, acts = r.out8(F)
    pre, pres = r.out8(2 * F) if keep else (None, None)
    ep.ep_grouped_matmul_swiglu(xq, xs, q, s, act, acts, row_weights=rw, pre=pre, pre_scales=pres, **r.args())
    y, mag = product64(r, x, w)
    err = sum_err(K) * mag
    if keep:
        v, sc = r.read8(pre, pres)
        check8(v, sc, y, err, "pre-activations")
    g, u = y.chunk(2, 1)
    eg, eu = err.chunk(2, 1)
    wt = rw[r.live].double()[:, None] if weighted else 1.0
    a = silu64(g) * u * wt
    # |silu'| <= 1.1; the activation itself in fp32 with a fast exponential and division
    ea = ((1.1 * eg) * u.abs() + (silu64(g).abs() + 1.1 * eg) * eu) * (wt.abs() if weighted else 1.0) + \
        (16 + 2 * g.abs()) * U24 * a.abs()
    v, sc = r.read8(act, acts)
    check8(v, sc, a, ea, "activations")


@pytest.mark.parametrize("counts,layout,align,slack", LAYOUTS)
@pytest.mark.parametrize("F,weighted", [(128, True), (640, False), (1536, True)])
def test_swiglu_backward(counts, layout, align, slack, F, weighted):
    r = Rows(counts, layout, align, slack)
    pq, ps, p = r.fp8(2 * F, 21, sigma=2.0)
    n = len(r.live)
    da = torch.full((r.rows, F), math.nan, dtype=torch.bfloat16, device=DEV)
    da[r.live] = (torch.randn((n, F), generator=gen(22), device=DEV) * 1e-2).bfloat16()
    rw = drw = None
    if weighted:
        rw = torch.full((r.rows,), math.nan, device=DEV)
        rw[r.live] = torch.randn(n, generator=gen(23), device=DEV)
        drw = torch.full((r.rows,), -9.0, device=DEV)
    dp, dps = r.out8(2 * F)
    ep.ep_grouped_swiglu_backward(da.view(r.lead + (F,)), pq, ps, dp, dps, row_weights=rw, grad_row_weights=drw,
                                  **r.args())
    g, u = (t.clone().requires_grad_(True) for t in p.chunk(2, 1))
    wt = (rw[r.live].double() if weighted else torch.ones(n, dtype=torch.float64, device=DEV)).requires_grad_(True)
    d = da[r.live].double()
    (silu64(g) * u * wt[:, None] * d).sum().backward()
    ref = torch.cat([g.grad, u.grad], 1)
    # the factors of each gradient are off by a few roundings and the exponential's (|g| + 4) u24; in
    # s (1 + g - silu) the bracket may cancel, so its terms' magnitudes count
    gd, ud = g.detach(), u.detach()
    sg = torch.sigmoid(gd)
    dw = (d * wt.detach()[:, None]).abs()
    eg = dw * ud.abs() * sg * (1 + gd.abs() + silu64(gd).abs()) * (16 + 2 * gd.abs()) * U24
    eu = dw * silu64(gd).abs() * (16 + 2 * gd.abs()) * U24
    v, sc = r.read8(dp, dps)
    check8(v, sc, ref, torch.cat([eg, eu], 1), "gradient")
    if weighted:
        assert (drw[r.dead] == -9.0).all()
        terms = (d * silu64(gd) * ud).abs()
        within(drw[r.live].double(), wt.grad, ((F / 32 + 24) * U24 * terms + terms * 2 * gd.abs() * U24).sum(1) + 1e-30,
               "row weights")


def test_swiglu_backward_against_differences():
    """(f(p + h v) - f(p - h v)) / 2h of f(p, w) = sum d w silu(gate) up, in 64
    bits, against the gradients' inner products with v: e4m3 rounds the
    gradient, independently for every channel, by 2^-4 at most."""
    F, n, h = 512, 40, 1e-4
    r = Rows([n], "em")
    pq, ps, p = r.fp8(2 * F, 25)
    da = (torch.randn((n, F), generator=gen(26), device=DEV)).bfloat16()
    rw = torch.randn(n, generator=gen(27), device=DEV)
    dp, dps = r.out8(2 * F)
    drw = torch.empty(n, device=DEV)
    ep.ep_grouped_swiglu_backward(da, pq, ps, dp, dps, row_weights=rw, grad_row_weights=drw, **r.args())
    grad, sc = r.read8(dp, dps)
    f = lambda p, w: (silu64(p[:, :F]) * p[:, F:] * da.double() * w[:, None]).sum()  # noqa: E731
    v = torch.randn((n, 2 * F), generator=gen(28), device=DEV).double()
    num = (f(p + h * v, rw.double()) - f(p - h * v, rw.double())) / (2 * h)
    bound = (grad.abs() * 2.0 ** -4 + (sc * 2.0 ** -10).repeat_interleave(128, 1)) * v.abs()
    # independent roundings: five times their root sum of squares, and h^2 f''' / 6
    assert abs((grad * v).sum() - num) <= 5 * bound.square().sum().sqrt() + 1e-4 * num.abs() + 1e-4
    vw = torch.randn(n, generator=gen(29), device=DEV).double()
    num = (f(p, rw.double() + h * vw) - f(p, rw.double() - h * vw)) / (2 * h)
    assert abs((drw.double() * vw).sum() - num) <= 1e-4 * (drw.double() * vw).abs().sum()


@pytest.mark.parametrize("counts,layout,align,slack", LAYOUTS)
@pytest.mark.parametrize("N,K", [(128, 128), (256, 256), (384, 640)])
def test_weight_grad(counts, layout, align, slack, N, K):
    r = Rows(counts, layout, align, slack)
    yq, ys, y = r.fp8(N, 31, sigma=1e-2)
    xq, xs, x = r.fp8(K, 32)
    dw = torch.full((len(counts), N, K), math.nan, dtype=torch.bfloat16, device=DEV)
    ep.ep_grouped_weight_grad(yq, ys, xq, xs, dw, **r.args())
    for e, at in r.spans():
        ref, mag = y[at].t() @ x[at], y[at].abs().t() @ x[at].abs()
        within(dw[e].double(), ref, ref.abs() * 2.0 ** -8 + mag * 2.0 ** -8.9, f"weight gradient of expert {e}")
        if r.counts[e] == 0:
            assert (dw[e] == 0).all()


def test_weight_grad_many_rows_and_sms():
    r = Rows([1000, 0, 65, 3000], "em", 1)
    yq, ys, y = r.fp8(640, 33, sigma=1e-2)
    xq, xs, x = r.fp8(1152, 34)
    dw = torch.empty((4, 640, 1152), dtype=torch.bfloat16, device=DEV)
    ep.ep_grouped_weight_grad(yq, ys, xq, xs, dw, **r.args())
    for e, at in r.spans():
        ref, mag = y[at].t() @ x[at], y[at].abs().t() @ x[at].abs()
        within(dw[e].double(), ref, ref.abs() * 2.0 ** -8 + mag * 2.0 ** -8.9, f"expert {e}")
    for sms in (1, 2, 5, 90):
        again = torch.empty_like(dw)
        ep.ep_grouped_weight_grad(yq, ys, xq, xs, again, num_sms=sms, **r.args())
        assert torch.equal(again.view(torch.int16), dw.view(torch.int16)), sms


def test_weight_grad_rows_of_different_sizes():
    """Row scales over 2^-16 of the largest, in either operand and opposed in
    the two (products alike), keep the bound: their codes and scales stay in
    f16's normal range.  A NaN row shows in the whole group and in no other."""
    n = 96
    r = Rows([n, n], "em")
    up = torch.exp2(torch.linspace(0, 15, n, device=DEV)).repeat(2)
    yq, ys, y = r.fp8(128, 35, row_sigma=up)
    xq, xs, x = r.fp8(128, 36, row_sigma=1.0 / up)
    dw = torch.empty((2, 128, 128), dtype=torch.bfloat16, device=DEV)
    ep.ep_grouped_weight_grad(yq, ys, xq, xs, dw, **r.args())
    for e, at in r.spans():
        ref, mag = y[at].t() @ x[at], y[at].abs().t() @ x[at].abs()
        # a code below 2^-2 of a row 2^-15 of the largest is subnormal in f16: 2^-25 of 2^-15 * 64 = 2^-9 at most
        within(dw[e].double(), ref, ref.abs() * 2.0 ** -8 + mag * 2.0 ** -7.9, f"expert {e}")
    ys[0, n + 3] = math.nan
    ep.ep_grouped_weight_grad(yq, ys, xq, xs, dw, **r.args())
    assert dw[0].isfinite().all() and dw[1].isnan().all()


def test_weight_grad_against_the_product():
    """<dw, V> is the derivative of <dy, x w^T> along V, and the product is
    linear in w: the two kernels agree on random directions."""
    r = Rows([200, 31], "ll", slack=9)
    yq, ys, y = r.fp8(256, 37)
    xq, xs, x = r.fp8(384, 38)
    dw = torch.empty((2, 256, 384), dtype=torch.bfloat16, device=DEV)
    ep.ep_grouped_weight_grad(yq, ys, xq, xs, dw, **r.args())
    q, s, v = weights(2, 256, 384, 39)
    out = r.out16(256)
    ep.ep_grouped_matmul(xq, xs, q, s, out, **r.args())
    left = (dw.double() * v).sum()
    right = (r.read16(out) * y).sum()
    spread = ((r.read16(out) * y).square().sum().sqrt() + (dw.double() * v).square().sum().sqrt()) * 2.0 ** -8
    assert abs(left - right) <= 5 * spread


def test_groups_that_do_not_fit_are_cut():
    """Counts over the slots, offsets past the buffer, negative counts: only
    rows that exist are touched, and the status says so."""
    K = N = 128
    q, s, w = weights(3, N, K, 41)
    for offset, count, want in (([0, 5, 14, 99], [3, 9, 4], [3, 9, 2]), ([0, -4, 200, 0], [16, 2, 5], [16, 0, 0]),
                                ([0, 4, 8, 12], [-3, 4, 4], [0, 4, 4])):
        x = torch.randn((16, K), generator=gen(42), device=DEV)
        xq, sc = quantize(x)
        xs = torch.zeros((1, 16), device=DEV)
        xs[0] = sc[:, 0]
        out = torch.full((16, N), -5.5, dtype=torch.bfloat16, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        ep.ep_grouped_matmul(xq, xs, q, s, out, torch.tensor(count, dtype=torch.int32, device=DEV),
                             group_offset=torch.tensor(offset, dtype=torch.int32, device=DEV), device_status=status)
        ref = torch.full((16, N), -5.5, dtype=torch.float64, device=DEV)
        xd = xq.double() * sc.double()
        for e, n in enumerate(want):
            if n:
                ref[offset[e]:offset[e] + n] = xd[offset[e]:offset[e] + n] @ w[e].t()
        within(out.double(), ref, ref.abs() * 2.0 ** -8 + 1e-3, "cut groups")
        cut = any(n != max(c, 0) for n, c in zip(want, count))
        assert int(status) == (ep.EP_ERR_CAPACITY if cut else ep.EP_OK)
    # low latency: more rows counted than slots
    r = Rows([5, 5], "ll")
    xq, xs, x = r.fp8(K, 43)
    over = torch.tensor([9, 5], dtype=torch.int32, device=DEV)
    q, s, w = weights(2, N, K, 44)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = r.out16(N)
    ep.ep_grouped_matmul(xq, xs, q, s, out, over, device_status=status)
    y, mag = product64(r, x, w)
    within(r.read16(out), y, y.abs() * 2.0 ** -8 + sum_err(K) * mag, "product")
    assert int(status) == ep.EP_ERR_CAPACITY
    for call in (lambda st: ep.ep_grouped_weight_grad(xq, xs, xq, xs, torch.empty((2, K, K), dtype=torch.bfloat16,
                                                                                   device=DEV), over, device_status=st),
                 lambda st: ep.ep_grouped_swiglu_backward(torch.zeros((2, 5, 128), dtype=torch.bfloat16, device=DEV),
                                                          *r.fp8(256, 45)[:2], *r.out8(256), over, device_status=st)):
        status.zero_()
        call(status)
        assert int(status) == ep.EP_ERR_CAPACITY


# ------------------------------------------------------------------ gate


def gate64(l, k, groups, keep, score, coef, on):
    """The gate's definition in 64 bits (l fp64 [T, E] with gradients)."""
    T, E = l.shape
    lm = l.detach().masked_fill(l.detach().isnan(), -math.inf)
    order = lm
    if groups > 1:
        best = lm.view(T, groups, -1).amax(2)
        rank = best.argsort(dim=1, descending=True, stable=True).argsort(dim=1)
        order = lm.masked_fill((rank >= keep).repeat_interleave(E // groups, 1), -math.inf)
    val, idx = torch.sort(order, dim=1, descending=True, stable=True)
    idx = torch.where((val > -math.inf) & on[:, None], idx, -torch.ones_like(idx))[:, :k]
    chosen = idx >= 0
    if score == ep.EP_GATE_SOFTMAX:
        p = torch.softmax(l, 1)
        raw = l.gather(1, idx.clamp_min(0)).masked_fill(~chosen, -math.inf)
        w = torch.where(chosen, torch.softmax(raw.masked_fill(~chosen.any(1, keepdim=True), 0.0), 1), 0.0)
    else:
        # log-sigmoid differences, so that tiny sigmoids keep their ratios
        ls = torch.nn.functional.logsigmoid(l)
        p = torch.softmax(ls, 1)
        raw = ls.gather(1, idx.clamp_min(0)).masked_fill(~chosen, -math.inf)
        w = torch.where(chosen, torch.softmax(raw.masked_fill(~chosen.any(1, keepdim=True), 0.0), 1), 0.0)
    none = ~(l.detach() > -math.inf).any(1)
    p = torch.where((on & ~none)[:, None], p, 0.0)
    V = int(on.sum())
    count = torch.bincount(idx[chosen].reshape(-1), minlength=E)
    prob = p.sum(0) / max(V, 1)
    loss = coef * E / (k * max(V, 1)) * (count * prob).sum()
    return idx, w, count, V, prob, loss


def run_gate(l, k, groups=1, keep=1, score=ep.EP_GATE_SOFTMAX, coef=0.5, mask=None, idt=torch.int64, ws=None, **kw):
    T, E = l.shape
    o = dict(idx=torch.full((T, k), -7, dtype=idt, device=DEV), w=torch.full((T, k), -7.0, device=DEV),
             count=torch.full((E + 1,), -7, dtype=torch.int32, device=DEV), prob=torch.full((E,), -7.0, device=DEV),
             loss=torch.full((1,), -7.0, device=DEV))
    ws = torch.zeros(ep.ep_gate_workspace_bytes(E), dtype=torch.uint8, device=DEV) if ws is None else ws
    ep.ep_gate_forward(l, o["idx"], o["w"], o["count"], o["prob"], o["loss"], ws, score=score, num_groups=groups,
                       topk_groups=keep, loss_coef=coef, token_mask=mask, **kw)
    assert not ws.any(), "the workspace is left zeroed"
    return o


GATES = [
    # T, E, k, groups, keep
    (1, 256, 8, 1, 1), (1, 1, 1, 1, 1), (5, 8, 8, 1, 1), (33, 60, 5, 4, 2), (200, 256, 8, 8, 4), (17, 160, 6, 8, 3),
    (70, 100, 32, 1, 1), (40, 384, 7, 3, 2), (1000, 64, 2, 64, 9), (9, 512, 32, 16, 2), (50, 1000, 9, 1, 1),
    (20, 2048, 4, 32, 5), (3, 4096, 31, 1, 1), (7, 4096, 8, 64, 4), (3000, 33, 3, 1, 1)]


@pytest.mark.parametrize("T,E,k,groups,keep", GATES)
@pytest.mark.parametrize("score", [ep.EP_GATE_SOFTMAX, ep.EP_GATE_SIGMOID])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate(T, E, k, groups, keep, score, dtype):
    g = gen(T * 7 + E)
    l = (torch.randn((T, E), generator=g, device=DEV) * 2).to(dtype)
    mask = torch.rand(T, generator=g, device=DEV) < 0.8
    if T == 1:
        mask[:] = True
    l[~mask] = math.nan
    idt = torch.int32 if k % 2 else torch.int64
    o = run_gate(l, k, groups, keep, score, mask=mask, idt=idt)
    l64 = torch.where(mask[:, None], l, torch.zeros_like(l)).double().requires_grad_(True)
    idx, w, count, V, prob, loss = gate64(l64, k, groups, keep, score, 0.5, mask)
    assert torch.equal(o["idx"].long(), idx)
    assert o["count"].tolist() == count.tolist() + [V]
    tol = (E / 32 + 64) * U24
    within(o["w"].double(), w.detach(), 64 * U24 * w.detach() + 1e-30, "weights")
    within(o["prob"].double(), prob.detach(), tol * prob.detach() + 2.0 ** -33, "mean probabilities")
    within(o["loss"].double(), loss.detach(), tol * loss.detach(), "loss")
    # backward, of both outputs and of each alone
    dw = torch.randn((T, k), generator=g, device=DEV)
    dl = torch.full((1,), 3.0, device=DEV)
    # a row's probabilities sum to one, so counts less their mean have the same
    # gradient, without the reference's own rounding where they cancel
    off_mean = 0.5 * E / (k * max(V, 1)) * ((count - k * V / E) * prob).sum()
    for use_w, use_l in ((True, True), (True, False), (False, True)):
        grad = torch.full((T, E), -7.0, dtype=dtype, device=DEV)
        ep.ep_gate_backward(l, o["idx"], o["count"], dw if use_w else None, dl if use_l else None, grad, score=score,
                            loss_coef=0.5, token_mask=mask)
        total = ((w * dw.double()).sum() if use_w else 0.0) + (off_mean * 3.0 if use_l else 0.0)
        ref, = torch.autograd.grad(total, l64, retain_graph=True)
        ref = torch.where(mask[:, None], ref, 0.0)
        # terms that cancel: w (|dw| + sum w |dw|) and coef p (|c - mean| + sum p |c - mean|)
        mag = torch.zeros_like(ref)
        if use_w:
            a = w.detach() * (dw.double().abs() + (w.detach() * dw.double().abs()).sum(1, keepdim=True))
            mag.scatter_add_(1, idx.clamp_min(0), torch.where(idx >= 0, a, 0.0))
        if use_l:
            lm = l64.detach()
            p = torch.softmax(lm if score == ep.EP_GATE_SOFTMAX else torch.nn.functional.logsigmoid(lm), 1)
            c = (count - k * V / E).double().abs()
            mag += 3.0 * 0.5 * E / (k * max(V, 1) ** 2) * p * (c + (p * c).sum(1, keepdim=True))
        bound = 2 * tol * mag + (ref.abs() * 2.0 ** -8 if dtype == torch.bfloat16 else 0.0) + 1e-37
        within(grad.double(), ref, bound, "gradient")


def test_gate_gradient_against_differences():
    """Central differences of coef-weighted loss and weights along a direction,
    the choice and the counts held (h far below the gaps that decide it)."""
    T, E, k = 64, 32, 4
    l = torch.randn((T, E), generator=gen(51), device=DEV)
    dw = torch.randn((T, k), generator=gen(52), device=DEV)
    one = torch.ones(1, device=DEV)
    for score in (ep.EP_GATE_SOFTMAX, ep.EP_GATE_SIGMOID):
        o = run_gate(l, k, score=score)
        grad = torch.empty_like(l)
        ep.ep_gate_backward(l, o["idx"], o["count"], dw, one, grad, score=score, loss_coef=0.5)
        v = torch.randn((T, E), generator=gen(53), device=DEV).double()
        c = o["count"][:E].double()

        def f(z):
            s = torch.exp(z) if score == ep.EP_GATE_SOFTMAX else torch.sigmoid(z)
            w = s.gather(1, o["idx"])
            w = w / w.sum(1, keepdim=True)
            p = s / s.sum(1, keepdim=True)
            return (w * dw.double()).sum() + 0.5 * E / (k * T) * (c * p.mean(0)).sum()

        h = 1e-5
        num = (f(l.double() + h * v) - f(l.double() - h * v)) / (2 * h)
        assert abs((grad.double() * v).sum() - num) <= 1e-5 * (grad.double() * v).abs().sum() + 1e-7


def test_gate_ties_empty_rows_and_special_values():
    inf, nan = math.inf, math.nan
    rows = [[1.0, 1.0, 1.0, 1.0, 1.0, 1.0], [0.0, -0.0, 0.0, -0.0, -1.0, -1.0], [-inf] * 6,
            [-inf, 2.0, -inf, -inf, -inf, -inf], [-1e30, -3e38, -inf, -2e38, -3.4e38, -inf],
            [3.4e38, -3.4e38, 0.0, 1e-45, -1e-45, 1.0], [-200.0, -200.0, -300.0, -201.0, -inf, -400.0],
            [1.0, 1.0 + 2.0 ** -23, 1.0 - 2.0 ** -24, 1.0, 1.0 + 2.0 ** -22, 0.5]]
    l = torch.tensor(rows, device=DEV)
    want = [[0, 1, 2], [0, 1, 2], [-1, -1, -1], [1, -1, -1], [0, 3, 1], [0, 5, 3], [0, 1, 3], [4, 1, 0]]
    on = torch.ones(len(rows), dtype=torch.bool, device=DEV)
    for score in (ep.EP_GATE_SOFTMAX, ep.EP_GATE_SIGMOID):
        o = run_gate(l, 3, score=score)
        assert o["idx"].tolist() == want
        _, w, count, V, prob, loss = gate64(l.double(), 3, 1, 1, score, 0.5, on)
        within(o["w"].double(), w, 64 * U24 * w + 1e-37, "weights")
        assert o["count"].tolist() == count.tolist() + [len(rows)]
        within(o["prob"].double(), prob, 1e-5 * prob + 2.0 ** -33, "probabilities")
        grad = torch.full_like(l, nan)
        ep.ep_gate_backward(l, o["idx"], o["count"], torch.ones((len(rows), 3), device=DEV), torch.ones(1, device=DEV),
                            grad, score=score, loss_coef=0.5)
        assert grad.isfinite().all() and (grad[2] == 0).all()
    # a NaN or +inf logit: chosen as its order says, and the loss says that p is not a number
    l[1, 2], l[3, 0] = nan, inf
    o = run_gate(l, 3)
    assert o["idx"][1].tolist() == [0, 1, 3] and o["idx"][3].tolist() == [0, 1, -1]
    assert o["loss"].isnan().all() and o["prob"].isnan().all()
    again = run_gate(l[4:].contiguous(), 3)
    assert again["loss"].isfinite().all()


def test_gate_all_tokens_masked_and_no_tokens():
    l = torch.full((5, 16), math.nan, device=DEV)
    off = torch.zeros(5, dtype=torch.bool, device=DEV)
    o = run_gate(l, 4, mask=off)
    assert (o["idx"] == -1).all() and (o["w"] == 0).all() and (o["count"] == 0).all()
    assert (o["prob"] == 0).all() and o["loss"].item() == 0.0
    grad = torch.full_like(l, math.nan)
    ep.ep_gate_backward(l, o["idx"], o["count"], torch.ones((5, 4), device=DEV), torch.ones(1, device=DEV), grad,
                        loss_coef=0.5, token_mask=off)
    assert (grad == 0).all()
    o = run_gate(torch.empty((0, 16), device=DEV), 4)
    assert (o["count"] == 0).all() and o["loss"].item() == 0.0
    ep.ep_gate_backward(torch.empty((0, 16), device=DEV), o["idx"], o["count"], None, None,
                        torch.empty((0, 16), device=DEV))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_strided_rows(dtype):
    """Rows inside a wider table, 16-byte aligned and not."""
    wide = torch.randn((50, 77), generator=gen(61), device=DEV).to(dtype)
    for first in (0, 3, 8):
        l = wide[:, first:first + 64]
        o, d = run_gate(l, 6), run_gate(l.contiguous(), 6)
        assert all(torch.equal(o[n], d[n]) for n in o)
        dw, one = torch.randn((50, 6), generator=gen(62), device=DEV), torch.ones(1, device=DEV)
        g1 = torch.full((50, 90), -7.0, dtype=dtype, device=DEV)
        g2 = torch.empty((50, 64), dtype=dtype, device=DEV)
        ep.ep_gate_backward(l, o["idx"], o["count"], dw, one, g1[:, first:first + 64], loss_coef=0.5)
        ep.ep_gate_backward(l.contiguous(), o["idx"], o["count"], dw, one, g2, loss_coef=0.5)
        assert torch.equal(g1[:, first:first + 64], g2)
        assert (g1[:, :first] == -7.0).all() and (g1[:, first + 64:] == -7.0).all()


def test_gate_same_bits_on_any_number_of_sms():
    """The choice and counts; P and the loss add in one fixed-point grid, but a
    block's own fp32 sum depends on which tokens it has."""
    l = torch.randn((5000, 256), generator=gen(63), device=DEV)
    ws = torch.zeros(ep.ep_gate_workspace_bytes(256), dtype=torch.uint8, device=DEV)
    first = run_gate(l, 8, 8, 4, ws=ws)
    for _ in range(3):
        again = run_gate(l, 8, 8, 4, ws=ws)
        assert all(torch.equal(first[n], again[n]) for n in first)
    for sms in (1, 3, 50):
        o = run_gate(l, 8, 8, 4, ws=ws, num_sms=sms)
        assert all(torch.equal(first[n], o[n]) for n in ("idx", "w", "count"))
        within(o["prob"].double(), first["prob"].double(), 2e-6 * first["prob"].double(), "probabilities")


# ------------------------------------------------------------------ use


def test_streams_and_graphs():
    """Every call runs on the stream it is given, and a captured sequence gives
    new results for new inputs."""
    r = Rows([40, 0, 90], "em", 16)
    xq, xs, _ = r.fp8(256, 71)
    q, s, _ = weights(3, 512, 256, 72)
    act, acts = r.out8(256)
    pre, pres = r.out8(512)
    dw = torch.empty((3, 256, 256), dtype=torch.bfloat16, device=DEV)
    l = torch.randn((64, 32), generator=gen(73), device=DEV)
    ws = torch.zeros(ep.ep_gate_workspace_bytes(32), dtype=torch.uint8, device=DEV)
    idx, w = torch.empty((64, 4), dtype=torch.int64, device=DEV), torch.empty((64, 4), device=DEV)
    count, prob, loss = torch.empty(33, dtype=torch.int32, device=DEV), torch.empty(32, device=DEV), torch.empty(1, device=DEV)
    grad = torch.empty_like(l)

    def work():
        ep.ep_gate_forward(l, idx, w, count, prob, loss, ws, loss_coef=0.5)
        ep.ep_gate_backward(l, idx, count, w, loss, grad, loss_coef=0.5)
        ep.ep_grouped_matmul_swiglu(xq, xs, q, s, act, acts, pre=pre, pre_scales=pres, **r.args())
        ep.ep_grouped_weight_grad(act, acts, xq, xs, dw, **r.args())

    results = (idx, w, count, loss, grad, act.view(torch.uint8), acts, pre.view(torch.uint8), dw)
    work()
    torch.cuda.synchronize()
    want = [t.clone() for t in results]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, results))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, results))
    l.mul_(-1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(want[0], idx)


def test_em_groups_and_weights_of_a_handle():
    R, E, k, H, tpr, align = 4, 16, 3, 256, 24, 8
    T = R * tpr
    with ep.Handle(R, E, k, H, tpr) as h:
        off, cnt = (torch.full((n,), -9, dtype=torch.int32, device=DEV) for n in (E + 1, E))
        with pytest.raises(ep.EPError):
            h.em_get_groups(off, cnt)
        with pytest.raises(RuntimeError):
            h.em_combine_weights(torch.zeros(4, device=DEV), torch.zeros((T, k), device=DEV))
        idx = torch.randn((T, E), generator=gen(81), device=DEV).topk(k).indices
        idx[::7, 1] = -1
        w = torch.rand((T, k), generator=gen(82), device=DEV)
        x = torch.randn((T, H), generator=gen(83), device=DEV).bfloat16()
        rows = T * k + E * (align - 1)
        recv, rw = torch.empty((rows, H), dtype=torch.bfloat16, device=DEV), torch.empty(rows, device=DEV)
        h.em_layout_and_dispatch(idx, x, w, ep.EP_BF16, align, recv, recv_weights=rw)
        h.em_get_groups(off, cnt)
        counts, offsets, _ = h.em_get_layout()
        assert off.tolist() == offsets.tolist() and cnt.tolist() == counts.tolist()
        back = torch.full((T, k), -9.0, device=DEV)
        h.em_combine_weights(rw, back)
        assert torch.equal(back, torch.where(idx >= 0, w, torch.zeros_like(w)))
        assert h.get_device_status() == ep.EP_OK
        # a vector that ends before the layout does
        used = int(offsets[-2]) + 1
        h.em_combine_weights(rw[:used].contiguous(), back)
        assert h.get_device_status() == ep.EP_ERR_CAPACITY


@pytest.mark.parametrize("score,groups,keep,masked", [(ep.EP_GATE_SOFTMAX, 1, 1, False), (ep.EP_GATE_SIGMOID, 4, 2, True)])
def test_moe_layer(score, groups, keep, masked):
    """The layer's forward, backward and decode against 64-bit autograd through
    the unquantised layer.  Each e4m3 rounding costs about 2.6 % rms: four of
    them lie before the output (x, w1, act, w2), at most eight before a
    gradient; bars of 3 times their root sum of squares."""
    torch.manual_seed(3)
    R, E, k, H, F, tpr = 4, 16, 4, 512, 384, 32
    T = R * tpr
    layer = moe.MoELayer(R, E, k, H, F, tpr, score=score, num_groups=groups, topk_groups=keep, loss_coef=0.5,
                         expert_alignment=16)
    W1, W2 = torch.randn((E, 2 * F, H), device=DEV) / H ** 0.5, torch.randn((E, H, F), device=DEV) / F ** 0.5
    w1, w2 = moe.ExpertWeights(W1), moe.ExpertWeights(W2)
    x = torch.randn((T, H), device=DEV).bfloat16()
    logits = torch.randn((T, E), device=DEV)
    mask = torch.rand(T, device=DEV) < 0.9 if masked else None
    go = (torch.randn((T, H), device=DEV)).bfloat16()
    out, loss, saved = layer.forward(x, logits, w1, w2, mask)
    gx, gl, gw1, gw2 = layer.backward(go, torch.ones(1, device=DEV), saved, w1, w2)
    dec = layer.decode(x, logits, w1, w2, mask)
    layer.check()

    on = torch.ones(T, dtype=torch.bool, device=DEV) if mask is None else mask
    xd, ld, W1d, W2d = (t.double().requires_grad_(True) for t in (x, logits, W1, W2))
    idx, w, count, V, prob, l64 = gate64(ld, k, groups, keep, score, 0.5, on)
    ref = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        y = xd[t] @ W1d[e].t()
        ref = ref.index_add(0, t, (silu64(y[:, :F]) * y[:, F:] * w[t, j][:, None]) @ W2d[e].t())
    ((ref * go.double()).sum() + l64).backward()
    rel = lambda a, b: ((a.double() - b).norm() / b.norm()).item()  # noqa: E731
    fwd_bar, bwd_bar = 3 * math.sqrt(4) * 0.026, 3 * math.sqrt(8) * 0.026
    assert rel(loss, l64.detach()[None]) < 1e-5
    assert rel(out, ref.detach()) < fwd_bar and rel(dec, ref.detach()) < fwd_bar
    for name, a, b in (("x", gx, xd), ("logits", gl, ld), ("w1", gw1, W1d), ("w2", gw2, W2d)):
        assert rel(a, b.grad) < bwd_bar, name
    layer.close()


def test_binding_refusals():
    r = Rows([5, 3], "em", 4)
    xq, xs, _ = r.fp8(256, 91)
    q, s, _ = weights(2, 128, 256, 92)
    out = r.out16(128)
    ok = dict(x=xq, x_scales=xs, w=q, w_scales=s, out=out, group_count=r.count, group_offset=r.offset)
    ep.ep_grouped_matmul(**ok)
    cpu = torch.empty(4)
    for bad in (dict(x=xq[:, :192]), dict(x=xq.float()), dict(x=cpu), dict(x=None), dict(x_scales=xs[:1]),
                dict(x_scales=xs[:, :4].contiguous()), dict(x_scales=xs.double()), dict(x_scales=xs.t()), dict(w=q[:1]),
                dict(w=q[:, :, :128].contiguous()), dict(w_scales=s[:, :, :1].contiguous()), dict(w_scales=None),
                dict(out=out[:4]), dict(out=out.float()), dict(out=out.t()), dict(group_count=r.count.long()),
                dict(group_count=r.count[:1].contiguous()), dict(group_count=None), dict(group_offset=None),
                dict(group_offset=r.offset[:1].contiguous()), dict(group_offset=cpu.int()),
                dict(device_status=torch.zeros(0, dtype=torch.int32, device=DEV)),
                dict(device_status=torch.zeros(1, device=DEV))):
        with pytest.raises((ValueError, TypeError)):
            ep.ep_grouped_matmul(**{**ok, **bad})
    with pytest.raises(ep.EPError):  # N not a multiple of 8: the library's own refusal
        ep.ep_grouped_matmul(xq, xs, q[:, :4].contiguous(), s, out[:, :4].contiguous(), r.count, r.offset)
    act, acts = r.out8(128)
    with pytest.raises(ValueError):  # weights of half the width
        ep.ep_grouped_matmul_swiglu(xq, xs, q, s, act, acts, r.count, r.offset)
    l = torch.randn((6, 16), device=DEV)
    good = dict(logits=l, topk_idx=torch.empty((6, 2), dtype=torch.int64, device=DEV),
                topk_weights=torch.empty((6, 2), device=DEV), expert_count=torch.empty(17, dtype=torch.int32, device=DEV),
                expert_prob=torch.empty(16, device=DEV), loss=torch.empty(1, device=DEV),
                workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))
    ep.ep_gate_forward(**good)
    for bad in (dict(logits=l.double()), dict(logits=l.t()), dict(logits=l[0]), dict(logits=l.cpu()),
                dict(topk_idx=good["topk_idx"][:5]), dict(topk_idx=good["topk_idx"].float()),
                dict(topk_weights=torch.empty((6, 1), device=DEV)), dict(expert_count=good["expert_count"][:16]),
                dict(expert_prob=torch.empty(15, device=DEV)), dict(loss=torch.empty(0, device=DEV)), dict(loss=None),
                dict(workspace=torch.zeros(100, dtype=torch.uint8, device=DEV)), dict(workspace=None),
                dict(token_mask=torch.ones(5, dtype=torch.bool, device=DEV)), dict(token_mask=torch.ones(6, device=DEV))):
        with pytest.raises((ValueError, TypeError)):
            ep.ep_gate_forward(**{**good, **bad})
    for bad in (dict(num_groups=3), dict(topk_groups=2), dict(score=5)):
        with pytest.raises(ep.EPError):
            ep.ep_gate_forward(**{**good, **bad})

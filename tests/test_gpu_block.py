"""The weighted expert-major combine with its gradient and the norms around a
block with theirs, on the GPU, against plain 64-bit forms of their definitions.

Tolerances, derived from the arithmetic (u24 = 2^-24, fp32's unit roundoff):
* bf16 results: half a step, 2^-8 of the value at most, plus the fp32 error of
  what was rounded.
* a sum of n fp32 terms, taken by 32 lanes or more and joined in at most 16
  steps: (n / 32 + 16) u24 times the sum of the terms' magnitudes; a sum over T
  tokens: (T + 16) u24.
* norms: rstd carries half its sum's relative error, and 4 u24 for the mean, the
  root and the rounding.
* e4m3 results as in the experts' tests: half a step, 2^-4 of the value.
"""
import math

import pytest
import torch

from combine_ep_get_03_gb300 import ep
from combine_ep_get_03_gb300 import moe

from test_gpu_experts import check8, gen, within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U24 = 2.0 ** -24
BF = 2.0 ** -8


# ------------------------------------------------------------------ combine

class Layout:
    """A handle with an expert-major layout, and the same layout in torch."""

    def __init__(self, R, T, E, k, H, align, seed, masked=0.1, repeat=False, bits=64):
        g = gen(seed)
        self.idx = torch.stack([torch.randperm(E, generator=g, device=DEV)[:k] for _ in range(T)]) if T else \
            torch.empty((0, k), dtype=torch.int64, device=DEV)
        if repeat and T:
            self.idx[0] = 1 % E  # one expert, k times
        if T:
            self.idx[torch.rand((T, k), generator=g, device=DEV) < masked] = -1
            if masked and T > 2:
                self.idx[1] = -1  # a token sent nowhere
        self.h = ep.Handle(R, E, k, H, max(T // R, 1))
        self.h.set_topk_idx_bits(bits)
        self.T, self.k, self.H = T, k, H
        flat = self.idx.reshape(-1)
        count = torch.bincount(flat[flat >= 0], minlength=E)
        start = torch.cat([count.new_zeros(1), ((count + align - 1) // align * align).cumsum(0)])
        self.rows = int(start[-1]) + 3
        self.row = torch.full_like(flat, -1)
        for e in range(E):
            at = (flat == e).nonzero().squeeze(1)
            self.row[at] = start[e] + torch.arange(len(at), device=DEV)
        self.row = self.row.view(T, k)
        x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
        self.h.em_layout_and_dispatch(self.idx if bits == 64 else self.idx.int(), x, None, ep.EP_BF16, align,
                                      torch.empty((self.rows, H), dtype=torch.bfloat16, device=DEV))
        self.live = torch.zeros(self.rows, dtype=torch.bool, device=DEV)
        self.live[self.row[self.row >= 0]] = True
        self.y = torch.full((self.rows, H), math.nan, dtype=torch.bfloat16, device=DEV)
        self.y[self.live] = torch.randn((int(self.live.sum()), H), generator=g, device=DEV).bfloat16()
        self.w = torch.randn((T, k), generator=g, device=DEV)
        self.w[self.row < 0] = math.nan  # of no entry: not used
        self.g = torch.randn((T, H), generator=g, device=DEV).bfloat16()

    def entries(self):
        t, j = (self.row >= 0).nonzero(as_tuple=True)
        return t, j, self.row[t, j]

    def combine64(self):
        t, j, row = self.entries()
        v = self.w[t, j, None].double() * self.y[row].double()
        z = torch.zeros((self.T, self.H), dtype=torch.float64, device=DEV)
        return z.index_add(0, t, v), z.index_add(0, t, v.abs())


LAYOUTS = [dict(R=1, T=1, E=1, k=1, H=128, align=1, masked=0.0), dict(R=4, T=4, E=8, k=8, H=256, align=4),
           dict(R=2, T=74, E=6, k=3, H=384, align=1, repeat=True), dict(R=8, T=200, E=64, k=8, H=2048, align=16),
           dict(R=1, T=33, E=40, k=32, H=640, align=128), dict(R=2, T=10, E=4, k=2, H=7168, align=8, bits=32),
           dict(R=4, T=64, E=8, k=2, H=1280, align=1, masked=1.0)]


@pytest.mark.parametrize("lay", LAYOUTS)
def test_combine_weighted(lay):
    l = Layout(seed=1, **lay)
    out = torch.full((l.T, l.H), math.nan, dtype=torch.bfloat16, device=DEV)
    l.h.em_combine_weighted(l.y, l.w, out)
    ref, mag = l.combine64()
    within(out.double(), ref, ref.abs() * BF + (l.k + 1) * U24 * mag, "combine")
    # weights of one are the unweighted combine, bit for bit
    a, b = torch.empty_like(out), torch.empty_like(out)
    l.h.em_combine_weighted(l.y, torch.ones_like(l.w), a)
    l.h.em_combine(l.y, b)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert l.h.get_device_status() == ep.EP_OK
    l.h.close()


@pytest.mark.parametrize("lay", LAYOUTS)
@pytest.mark.parametrize("fp8", [False, True])
def test_combine_weighted_backward(lay, fp8):
    l = Layout(seed=2, **lay)
    t, j, row = l.entries()
    ref = l.w[t, j, None].double() * l.g[t].double()
    dw = torch.full((l.T, l.k), math.nan, device=DEV)
    dead = ~l.live
    if fp8:
        dy = torch.full((l.rows, l.H), 0x5A, dtype=torch.uint8, device=DEV)
        ds = torch.full((l.H // 128, (l.rows + 3) // 4 * 4 + 4), 7.25, device=DEV)
        l.h.em_combine_weighted_backward(l.g, l.y, l.w, ep.EP_FP8_E4M3, dy, ds, grad_topk_weights=dw)
        assert (dy[dead] == 0x5A).all() and (ds.t()[:l.rows][dead] == 7.25).all() and (ds[:, l.rows:] == 7.25).all()
        s = ds.t()[row].double()
        v = dy[row].view(torch.float8_e4m3fn).double() * s.repeat_interleave(128, 1)
        check8(v, s, ref, U24 * ref.abs(), "rows' gradient")
    else:
        dy = torch.full((l.rows, l.H), -5.5, dtype=torch.bfloat16, device=DEV)
        l.h.em_combine_weighted_backward(l.g, l.y, l.w, ep.EP_BF16, dy, grad_topk_weights=dw)
        assert (dy[dead] == -5.5).all()
        within(dy[row].double(), ref, (BF + 2 * U24) * ref.abs(), "rows' gradient")
    terms = l.g[t].double() * l.y[row].double()
    want, err = torch.zeros((l.T, l.k), dtype=torch.float64, device=DEV), torch.zeros((l.T, l.k), dtype=torch.float64, device=DEV)
    want[t, j], err[t, j] = terms.sum(1), (l.H / 32 + 16) * U24 * terms.abs().sum(1)
    within(dw.double(), want, err, "weights' gradient")  # 0, exactly, where masked
    # either alone gives the same bits
    only = torch.empty_like(dw)
    l.h.em_combine_weighted_backward(l.g, l.y, None, ep.EP_BF16, grad_topk_weights=only)
    assert torch.equal(only, dw)
    alone = torch.empty_like(dy)
    scales = torch.empty_like(ds) if fp8 else None
    l.h.em_combine_weighted_backward(l.g, None, l.w, ep.EP_FP8_E4M3 if fp8 else ep.EP_BF16, alone, scales)
    assert torch.equal(alone[row].view(torch.uint8), dy[row].view(torch.uint8))
    assert l.h.get_device_status() == ep.EP_OK
    l.h.close()


def test_combine_weighted_gradient_against_differences():
    """The combine is linear in y and in w: f(y + d) - f(y), f = <grad_out, out>,
    is <grad_y, d> up to the bf16 roundings of both outputs and of grad_y."""
    l = Layout(2, 60, 12, 4, 512, 4, seed=3)
    t, j, row = l.entries()
    out = [torch.empty((l.T, l.H), dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    dy, dw = torch.zeros_like(l.y), torch.empty_like(l.w)
    l.h.em_combine_weighted_backward(l.g, l.y, l.w, ep.EP_BF16, dy, grad_topk_weights=dw)
    y2 = l.y.clone()
    y2[row] = torch.randn((len(row), l.H), generator=gen(4), device=DEV).bfloat16()
    w2 = torch.where(l.row >= 0, torch.randn_like(l.w), l.w)
    l.h.em_combine_weighted(l.y, l.w, out[0])
    l.h.em_combine_weighted(y2, l.w, out[1])
    l.h.em_combine_weighted(l.y, w2, out[2])
    g = l.g.double()
    noise = lambda a: (g * a.double()).square().sum().sqrt() * BF  # noqa: E731  independent roundings
    d = (y2[row].double() - l.y[row].double())
    num = (g * (out[1].double() - out[0].double())).sum()
    assert abs((dy[row].double() * d).sum() - num) <= 5 * (noise(out[0]) + noise(out[1]) + (dy[row].double() * d).square().sum().sqrt() * BF)
    num = (g * (out[2].double() - out[0].double())).sum()
    dwd = dw[t, j].double() * (w2 - l.w)[t, j].double()
    assert abs(dwd.sum() - num) <= 5 * (noise(out[0]) + noise(out[2])) + 1e-5 * dwd.abs().sum()
    l.h.close()


def test_combine_weighted_rows_past_the_buffer():
    l = Layout(1, 40, 4, 2, 256, 1, seed=5, masked=0.0)
    cut = l.rows // 2
    y = l.y[:cut].contiguous()
    out = torch.empty((l.T, l.H), dtype=torch.bfloat16, device=DEV)
    l.h.em_combine_weighted(y, l.w, out)
    assert l.h.get_device_status() == ep.EP_ERR_CAPACITY
    whole = l.row.clone()
    l.row[l.row >= cut] = -1
    ref, mag = l.combine64()
    within(out.double(), ref, ref.abs() * BF + 3 * U24 * mag, "combine")
    buf = torch.full((cut + 5, l.H), -5.5, dtype=torch.bfloat16, device=DEV)
    dw = torch.empty_like(l.w)
    l.h.em_combine_weighted_backward(l.g, y, l.w, ep.EP_BF16, buf[:cut], grad_topk_weights=dw)
    assert l.h.get_device_status() == ep.EP_ERR_CAPACITY
    assert (buf[cut:] == -5.5).all() and (dw[whole >= cut] == 0).all() and (dw[whole < cut] != 0).all()
    l.h.close()


def test_combine_weighted_refusals():
    h = ep.Handle(1, 4, 2, 256, 8)
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    w = torch.empty((8, 2), device=DEV)
    with pytest.raises(RuntimeError):
        h.em_combine_weighted(e(16, 256), w, e(8, 256))
    with pytest.raises(RuntimeError):
        h.em_combine_weighted_backward(e(8, 256), e(16, 256), w, ep.EP_BF16, e(16, 256))
    assert ep.lib().ep_em_combine_weighted(h.ptr, e(16, 256).data_ptr(), 16, w.data_ptr(), e(8, 256).data_ptr(), 0,
                                           None) == ep.EP_ERR_STATE
    l = Layout(1, 8, 4, 2, 256, 1, seed=6)
    f8, sc = torch.empty((l.rows, 256), dtype=torch.uint8, device=DEV), torch.empty((2, (l.rows + 3) // 4 * 4), device=DEV)
    for bad in (dict(y=l.y[:, :128]), dict(topk_weights=w[:4]), dict(out=e(7, 256)), dict(y=l.y.float()),
                dict(topk_weights=w.double()), dict(topk_weights=None)):
        with pytest.raises((ValueError, ep.EPError)):
            l.h.em_combine_weighted(**{**dict(y=l.y, topk_weights=l.w, out=e(8, 256)), **bad})
    ok = dict(grad_out=l.g, y=l.y, topk_weights=l.w, dtype=ep.EP_FP8_E4M3, grad_y=f8, grad_y_scales=sc)
    l.h.em_combine_weighted_backward(**ok)
    for bad in (dict(grad_out=l.g[:4]), dict(grad_y=f8[:, :128]), dict(grad_y=f8[:4]), dict(grad_y_scales=None),
                dict(grad_y_scales=sc[:1]), dict(grad_y_scales=sc[:, :4]), dict(dtype=7), dict(topk_weights=None),
                dict(grad_y=None, y=None), dict(grad_y=None), dict(y=None, grad_topk_weights=l.w.clone()),
                dict(dtype=ep.EP_BF16), dict(grad_topk_weights=w[:3]),
                dict(grad_y_scales=torch.empty((2, l.rows + (l.rows + 1) % 2), device=DEV))):
        with pytest.raises((ValueError, ep.EPError)):
            l.h.em_combine_weighted_backward(**{**ok, **bad})
    l.h.close()
    h.close()


def test_combine_weighted_without_tokens():
    l = Layout(2, 0, 4, 2, 256, 8, seed=7)
    out = torch.empty((0, 256), dtype=torch.bfloat16, device=DEV)
    l.h.em_combine_weighted(l.y, l.w, out)
    l.h.em_combine_weighted_backward(l.g, l.y, l.w, ep.EP_BF16, torch.empty_like(l.y), grad_topk_weights=l.w)
    assert l.h.get_device_status() == ep.EP_OK
    l.h.close()


# ------------------------------------------------------------------ norms

class Norms:
    """A case's tensors; a padding token's rows hold NaN."""

    def __init__(self, T, H, res, wt, post, pre, gate, masked=False, scale=0.5, seed=11, sigma=1.0):
        g = gen(seed)
        n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        self.T, self.H, self.res = T, H, res
        self.residual, self.y = (2 * sigma * n(T, H)).to(res), (0.7 * sigma * n(T, H)).bfloat16()
        self.post = (1 + 0.3 * n(H)).to(wt) if post else None
        self.pre = (1 + 0.3 * n(H)).to(wt) if pre else None
        self.gate = {"none": None, "vector": (n(H)).to(wt), "token": n(T, H).bfloat16()}[gate]
        self.dx, self.dnew = n(T, H).bfloat16(), n(T, H).to(res)
        self.mask = None
        if masked:
            self.mask = torch.rand(T, generator=g, device=DEV) < 0.7
            for t in (self.residual, self.y, self.dx, self.dnew) + ((self.gate,) if gate == "token" else ()):
                t[~self.mask] = math.nan
        self.how = dict(post_weight=self.post, pre_weight=self.pre, gate=self.gate, residual_scale=scale,
                        token_mask=self.mask)
        self.scale = scale
        self.on = torch.ones(T, dtype=torch.bool, device=DEV) if self.mask is None else self.mask

    def d(self, t):
        return None if t is None else (t[self.on] if t.dim() == 2 else t).double()

    def forward(self, eps=1e-6, **kw):
        new = torch.full((self.T, self.H), math.nan, dtype=self.res, device=DEV)
        x = torch.full((self.T, self.H), math.nan, dtype=torch.bfloat16, device=DEV) if self.pre is not None else None
        rstd = torch.full((2, self.T), -3.0, device=DEV)
        ep.ep_block_norm_forward(self.residual, self.y, new, x, rstd=rstd, eps=eps, **self.how, **kw)
        return new, x, rstd


CASES = [dict(T=1, H=8, post=True, pre=True, gate="none"), dict(T=3, H=16, post=True, pre=True, gate="vector"),
         dict(T=5, H=136, post=False, pre=True, gate="token"), dict(T=700, H=256, post=True, pre=True, gate="token", masked=True),
         dict(T=153, H=1032, post=True, pre=False, gate="vector", masked=True), dict(T=33, H=2056, post=False, pre=False, gate="none"),
         dict(T=40, H=2560, post=True, pre=True, gate="none", masked=True), dict(T=20, H=4104, post=False, pre=True, gate="none"),
         dict(T=305, H=7168, post=True, pre=True, gate="vector"), dict(T=9, H=8192, post=True, pre=True, gate="token"),
         dict(T=10, H=8200, post=True, pre=True, gate="token", masked=True), dict(T=6, H=16384, post=True, pre=True, gate="vector"),
         dict(T=700, H=8200, post=True, pre=False, gate="none"), dict(T=700, H=12296, post=False, pre=True, gate="vector", masked=True),
         dict(T=7, H=12288, post=False, pre=False, gate="token"), dict(T=2, H=520, post=False, pre=False, gate="vector"),
         dict(T=700, H=2048, post=True, pre=True, gate="token", masked=True), dict(T=310, H=4096, post=True, pre=True, gate="vector"),
         dict(T=170, H=3848, post=True, pre=True, gate="token"), dict(T=911, H=1280, post=False, pre=True, gate="vector", masked=True)]
TYPES = [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16)]


def half_step(t, v):
    return v.abs() * (BF if t is torch.bfloat16 else U24)


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("res,wt", TYPES)
def test_norm_forward(case, res, wt):
    c = Norms(res=res, wt=wt, **case)
    new, x, rstd = c.forward()
    H, eps = c.H, 1e-6
    es = ((H / 32 + 16) / 2 + 4) * U24  # of rstd
    on = c.on
    r, y, gate = c.d(c.residual), c.d(c.y), c.d(c.gate)
    n = y
    if c.post is not None:
        r1 = (y.square().mean(1) + eps).rsqrt()
        n = y * r1[:, None] * c.d(c.post)
        within(rstd[0][on].double(), r1, es * r1, "rstd of y")
        assert (rstd[0][~on] == 0).all()
    else:
        assert (rstd[0] == -3.0).all()
    if gate is not None:
        n = n * gate
    n = n * c.scale
    h = r + n
    eh = (es + 6 * U24) * n.abs() + U24 * h.abs()
    within(new[on].double(), h, half_step(res, h) + eh, "new residual")
    assert (new[~on] == 0).all()
    if c.pre is None:
        assert (rstd[1] == -3.0).all()
        return
    r2 = (h.square().mean(1) + eps).rsqrt()
    e2 = es + (h.abs() * eh).sum(1) / h.square().sum(1)
    within(rstd[1][on].double(), r2, e2 * r2, "rstd of the residual")
    ref = h * r2[:, None] * c.d(c.pre)
    within(x[on].double(), ref, (BF + e2[:, None] + 4 * U24) * ref.abs() + eh * r2[:, None] * c.d(c.pre).abs(), "x")
    assert (x[~on] == 0).all() and (rstd[1][~on] == 0).all()


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("res,wt", TYPES)
def test_norm_backward(case, res, wt):
    c = Norms(res=res, wt=wt, **case)
    new, _, rstd = c.forward()
    T, H, on, a = c.T, c.H, c.on, c.scale
    if c.mask is not None:
        new[~on] = math.nan  # not read: it is 0 where the forward pass wrote it
    ws = torch.full((ep.ep_block_norm_workspace_bytes(H),), 0xFF, dtype=torch.uint8, device=DEV)
    nan = lambda *s, dt=torch.float32: torch.full(s, math.nan, dtype=dt, device=DEV)  # noqa: E731
    token = case["gate"] == "token"
    dres, dy = nan(T, H, dt=res), nan(T, H, dt=torch.bfloat16)
    dpost, dpre = nan(H) if c.post is not None else None, nan(H) if c.pre is not None else None
    dgate = None if c.gate is None else nan(T, H, dt=torch.bfloat16) if token else nan(H)
    dx = c.dx if c.pre is not None else None
    call = lambda dres, dy, dpost, dpre, dgate, **kw: ep.ep_block_norm_backward(  # noqa: E731
        new, c.y, rstd, c.dnew, dx, dres, dy, ws, grad_post_weight=dpost, grad_pre_weight=dpre, grad_gate=dgate, **c.how, **kw)
    call(dres, dy, dpost, dpre, dgate)

    # the formulas, and the sums of their terms' magnitudes for the errors
    n1 = (H / 32 + 24) * U24
    gh, h, y = c.d(c.dnew), c.d(new), c.d(c.y)
    eg = 4 * U24 * gh.abs()
    hn = torch.zeros_like(gh)
    ag = gh.abs()  # magnitudes inside m2's sum
    if c.pre is not None:
        r2, w = rstd[1][on].double()[:, None], c.d(c.pre)
        hn, ax = h * r2, c.d(c.dx) * w
        m1, am = (ax * hn).mean(1, keepdim=True), (ax * hn).abs().mean(1, keepdim=True)
        eg = eg + r2 * (8 * U24 * ax.abs() + hn.abs() * (8 * U24 * m1.abs() + n1 * am))
        ag = ag + r2 * (ax.abs() + hn.abs() * am)
        gh = gh + r2 * (ax - hn * m1)
        terms = c.d(c.dx) * hn
        within(dpre.double(), terms.sum(0), (T + 16) * U24 * terms.abs().sum(0), "pre")
    within(dres[on].double(), gh, half_step(res, gh) + eg, "residual")
    r1 = rstd[0][on].double()[:, None] if c.post is not None else 1.0
    yn, gate = y * r1, c.d(c.gate) if c.gate is not None else 1.0
    post = c.d(c.post) if c.post is not None else 1.0
    s, es = a * gh * yn, a * (eg * yn.abs()) + 8 * U24 * (a * gh * yn).abs()
    if c.gate is not None:
        if token:
            ref = s * post
            within(dgate[on].double(), ref, BF * ref.abs() + es * (post.abs() if c.post is not None else 1.0), "gate")
            assert (dgate[~on] == 0).all()
        else:
            p = post.abs() if c.post is not None else 1.0
            within(dgate.double(), (s * post).sum(0), ((T + 16) * U24 * s.abs().sum(0) + es.sum(0)) * p, "gate")
    ga = gate.abs() if c.gate is not None else 1.0
    if c.post is not None:
        within(dpost.double(), (s * gate).sum(0), ((T + 16) * U24 * (s * gate).abs().sum(0) + (es * ga).sum(0)), "post")
    q = a * gate * post
    qa = abs(a) * ga * (post.abs() if c.post is not None else 1.0)
    ref, err = q * gh, qa * eg + 8 * U24 * (q * gh).abs()
    if c.post is not None:
        m2 = (q * gh * yn).mean(1, keepdim=True)
        em = n1 * (qa * yn.abs() * ag).mean(1, keepdim=True) + (qa * yn.abs() * eg).mean(1, keepdim=True)
        ref = r1 * (ref - yn * m2)
        err = r1 * (err + yn.abs() * (em + 8 * U24 * m2.abs()) + 8 * U24 * (q * gh).abs())
    within(dy[on].double(), ref, BF * ref.abs() + err + 1e-30, "y")
    assert (dy[~on] == 0).all() and (dres[~on] == 0).all()

    # in place, each gradient alone, and again: the same bits
    inplace = c.dnew.clone()
    ep.ep_block_norm_backward(new, c.y, rstd, inplace, dx, inplace, None, ws, **c.how)
    assert torch.equal(inplace, dres)
    for k, t in enumerate((dres, dy, dpost, dpre, dgate)):
        if t is not None:
            one = torch.empty_like(t)
            call(*(one if i == k else None for i in range(5)))
            assert torch.equal(one, t), k


def test_norm_without_a_block_behind():
    """y None: x is the norm of the residual; its backward has no block side."""
    c = Norms(50, 640, torch.float32, torch.float32, False, True, "none", masked=True)
    x, rstd = torch.empty((50, 640), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 50), device=DEV)
    ep.ep_block_norm_forward(c.residual, None, None, x, rstd=rstd, pre_weight=c.pre, token_mask=c.mask)
    h = c.d(c.residual)
    r2 = (h.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    ref = h * r2 * c.d(c.pre)
    within(x[c.on].double(), ref, (BF + 40 * U24) * ref.abs(), "x")
    dres, dpre = torch.empty_like(c.residual), torch.empty(640, device=DEV)
    ws = torch.empty(ep.ep_block_norm_workspace_bytes(640), dtype=torch.uint8, device=DEV)
    ep.ep_block_norm_backward(c.residual, None, rstd, None, c.dx, dres, None, ws, pre_weight=c.pre, grad_pre_weight=dpre,
                              token_mask=c.mask)
    hv, wv = h.clone().requires_grad_(True), c.d(c.pre).requires_grad_(True)
    (hv * (hv.square().mean(1, keepdim=True) + 1e-6).rsqrt() * wv * c.d(c.dx)).sum().backward()
    mag = r2 * (c.d(c.dx) * c.d(c.pre)).abs().amax(1, keepdim=True) * 8
    within(dres[c.on].double(), hv.grad, 100 * U24 * mag, "residual")
    within(dpre.double(), wv.grad, 100 * U24 * (c.d(c.dx) * h * r2).abs().sum(0), "pre")


def test_norm_gradient_against_differences():
    """Central differences of the definition in 64 bits, along random directions
    of every input, against the gradients' inner products with them."""
    c = Norms(60, 512, torch.float32, torch.float32, True, True, "token", scale=0.7)
    new, _, rstd = c.forward()
    T, H = 60, 512
    grads = dict(residual=torch.empty_like(c.residual), y=torch.empty_like(c.y), gate=torch.empty_like(c.gate),
                 post=torch.empty(H, device=DEV), pre=torch.empty(H, device=DEV))
    ws = torch.empty(ep.ep_block_norm_workspace_bytes(H), dtype=torch.uint8, device=DEV)
    ep.ep_block_norm_backward(new, c.y, rstd, c.dnew, c.dx, grads["residual"], grads["y"], ws, grad_gate=grads["gate"],
                              grad_post_weight=grads["post"], grad_pre_weight=grads["pre"], **c.how)
    at = dict(residual=c.d(c.residual), y=c.d(c.y), gate=c.d(c.gate), post=c.d(c.post), pre=c.d(c.pre))

    def f(v):
        h = v["residual"] + 0.7 * v["gate"] * v["post"] * v["y"] * (v["y"].square().mean(1, keepdim=True) + 1e-6).rsqrt()
        x = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * v["pre"]
        return (h * c.dnew.double()).sum() + (x * c.dx.double()).sum()

    for name, g in grads.items():
        d = torch.randn(g.shape, generator=gen(41), device=DEV).double()
        s = 1e-4
        num = (f({**at, name: at[name] + s * d}) - f({**at, name: at[name] - s * d})) / (2 * s)
        terms = g.double() * d
        # bf16 gradients: independent roundings, five times their root sum of squares; fp32 sums 1e-4
        assert abs(terms.sum() - num) <= 5 * BF * terms.square().sum().sqrt() * (g.dtype is torch.bfloat16) + 1e-4 * terms.abs().sum(), name


def test_norm_special_rows():
    """Zeros, tiny and huge rows, and infinities: each row for itself."""
    c = Norms(8, 256, torch.float32, torch.float32, True, True, "none", scale=1.0)
    c.residual[1:3], c.y[1] = 0, 0
    c.y[2] *= 2.0 ** -60
    c.y[3] *= 2.0 ** 50
    c.residual[4, 7] = math.inf
    c.y[5, 9] = math.nan
    c.residual[6] = -c.residual[6].abs()
    new, x, rstd = c.forward()
    ok = [0, 1, 2, 3, 6, 7]
    y, r = c.y.double(), c.residual.double()
    h = r + y * (y.square().mean(1, keepdim=True) + 1e-6).rsqrt() * c.post.double()
    ref = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * c.pre.double()
    within(new[ok].double(), h[ok], 40 * U24 * (h - r).abs()[ok] + 2 * U24 * h[ok].abs(), "h")
    within(x[ok].double(), ref[ok], (BF + 80 * U24) * ref[ok].abs() + 80 * U24, "x")
    assert (x[1] == 0).all() and (new[1] == 0).all()
    assert x[5].isnan().all() and new[5].isnan().all() and new[4, 7] == math.inf


def test_norm_in_place_no_tokens_and_sms():
    c = Norms(100, 1536, torch.bfloat16, torch.float32, True, True, "vector")
    new, x, rstd = c.forward()
    for sms in (1, 2, 64):
        again = c.forward(num_sms=sms)
        assert torch.equal(new, again[0]) and torch.equal(x, again[1]) and torch.equal(rstd, again[2])
    h = c.residual.clone()
    x2 = torch.empty_like(x)
    ep.ep_block_norm_forward(h, c.y, h, x2, **c.how)
    assert torch.equal(h, new) and torch.equal(x2, x)
    e = lambda dt: torch.empty((0, 1536), dtype=dt, device=DEV)  # noqa: E731
    ep.ep_block_norm_forward(e(torch.bfloat16), e(torch.bfloat16), e(torch.bfloat16), e(torch.bfloat16),
                             post_weight=c.post, pre_weight=c.pre)
    sums = [torch.full((1536,), math.nan, device=DEV) for _ in range(3)]
    ws = torch.empty(ep.ep_block_norm_workspace_bytes(1536), dtype=torch.uint8, device=DEV)
    ep.ep_block_norm_backward(e(torch.bfloat16), e(torch.bfloat16), torch.empty((2, 0), device=DEV), e(torch.bfloat16),
                              e(torch.bfloat16), e(torch.bfloat16), e(torch.bfloat16), ws, post_weight=c.post,
                              pre_weight=c.pre, gate=c.gate, grad_post_weight=sums[0], grad_pre_weight=sums[1],
                              grad_gate=sums[2])
    assert all((s == 0).all() for s in sums)


def test_norm_refusals():
    c = Norms(10, 64, torch.float32, torch.float32, True, True, "vector")
    x, new = torch.empty((10, 64), dtype=torch.bfloat16, device=DEV), torch.empty_like(c.residual)
    ok = dict(residual=c.residual, y=c.y, new_residual=new, x=x, post_weight=c.post, pre_weight=c.pre, gate=c.gate)
    ep.ep_block_norm_forward(**ok)
    for bad in (dict(residual=c.residual.double()), dict(residual=c.residual[0]), dict(residual=c.residual.t()), dict(y=c.y.float()),
                dict(y=c.y[:9]), dict(y=None), dict(new_residual=None), dict(new_residual=new.bfloat16()), dict(x=None),
                dict(pre_weight=None), dict(x=x[:, :32]), dict(post_weight=c.post[:32]), dict(post_weight=c.post.bfloat16()),
                dict(gate=c.gate[:8]), dict(gate=torch.empty((9, 64), dtype=torch.bfloat16, device=DEV)),
                dict(gate=torch.empty((10, 64), device=DEV)), dict(rstd=torch.empty(19, device=DEV)), dict(y=c.y.cpu()),
                dict(token_mask=torch.ones(9, dtype=torch.bool, device=DEV)), dict(residual=None)):
        with pytest.raises((ValueError, TypeError, AttributeError, ep.EPError)):
            ep.ep_block_norm_forward(**{**ok, **bad})
    with pytest.raises(ep.EPError):  # 12 channels: the library's own refusal
        ep.ep_block_norm_forward(c.residual[:, :12].contiguous(), None, None, x[:, :12].contiguous(), pre_weight=c.pre[:12].contiguous())
    rstd, ws = torch.zeros((2, 10), device=DEV), torch.empty(ep.ep_block_norm_workspace_bytes(64), dtype=torch.uint8, device=DEV)
    back = dict(new_residual=new, y=c.y, rstd=rstd, grad_new_residual=c.dnew, grad_x=c.dx, grad_residual=new.clone(),
                grad_y=torch.empty_like(c.y), workspace=ws, post_weight=c.post, pre_weight=c.pre, gate=c.gate,
                grad_post_weight=torch.empty(64, device=DEV), grad_pre_weight=torch.empty(64, device=DEV),
                grad_gate=torch.empty(64, device=DEV))
    ep.ep_block_norm_backward(**back)
    for bad in (dict(new_residual=None), dict(y=None), dict(rstd=None), dict(grad_x=None), dict(workspace=None),
                dict(workspace=ws[:-1]), dict(post_weight=None), dict(pre_weight=None), dict(gate=None),
                dict(grad_residual=new.bfloat16()), dict(grad_y=new), dict(grad_gate=torch.empty((10, 64), device=DEV, dtype=torch.bfloat16)),
                dict(grad_post_weight=torch.empty(63, device=DEV)), dict(grad_new_residual=c.dnew[:5])):
        with pytest.raises((ValueError, TypeError, ep.EPError)):
            ep.ep_block_norm_backward(**{**back, **bad})


# ------------------------------------------------------------------ together

def rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("res,gate,masked", [(torch.float32, "vector", False), (torch.bfloat16, "none", True),
                                             (torch.float32, "token", True)])
@pytest.mark.parametrize("weigh", [False, True])
def test_moe_block(res, gate, masked, weigh):
    """Forward, backward and decode of a block against autograd in 64 bits, on
    the routing that the block chose.  e4m3 rounds a factor by 0.026 in the root
    mean square: four such factors in a row forward, eight backward."""
    torch.manual_seed(5)
    R, E, k, H, F, tpr = 2, 8, 2, 256, 128, 48
    T = R * tpr
    layer = moe.MoELayer(R, E, k, H, F, tpr, loss_coef=0.5, expert_alignment=16, weigh_in_combine=weigh)
    W1, W2 = torch.randn((E, 2 * F, H), device=DEV) / H ** 0.5, torch.randn((E, H, F), device=DEV) / F ** 0.5
    w1, w2 = moe.ExpertWeights(W1), moe.ExpertWeights(W2)
    pre, post = 1 + 0.1 * torch.randn(H, device=DEV), 1 + 0.1 * torch.randn(H, device=DEV)
    router = (torch.randn((E, H), device=DEV) * 2 / H ** 0.5).bfloat16()
    g = {"none": None, "vector": torch.randn(H, device=DEV), "token": torch.randn((T, H), device=DEV).bfloat16()}[gate]
    h = torch.randn((T, H), device=DEV).to(res)
    mask = torch.rand(T, device=DEV) < 0.9 if masked else None
    block = moe.MoEBlock(layer, pre, router, post=post, gate=g, residual_scale=0.7)
    go = torch.randn((T, H), device=DEV).to(res)
    out, loss, saved = block.forward(h, w1, w2, mask)
    # another forward and a decode in between
    block.forward(h.flip(0).contiguous(), w1, w2, mask)
    dec = block.decode(h.clone(), w1, w2, mask)
    grads = block.backward(go, torch.ones(1, device=DEV), saved, w1, w2)
    layer.check()

    on = torch.ones(T, dtype=torch.bool, device=DEV) if mask is None else mask
    idx = saved[5][2]
    leaf = lambda t: None if t is None else t.double().requires_grad_(True)  # noqa: E731
    hd, pred, postd, gd, rd, W1d, W2d = (leaf(t) for t in (h, pre, post, g, router, W1, W2))
    norm = lambda v: v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
    x = norm(hd) * pred
    logits = x @ rd.t()
    w = torch.softmax(logits.gather(1, idx.clamp_min(0)), 1)
    p = torch.softmax(logits, 1)[on].mean(0)
    count = torch.bincount(idx[on].reshape(-1), minlength=E)
    l64 = 0.5 * E / (k * int(on.sum())) * (count * p).sum()
    y = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        a, b = (x[t] @ W1d[e].t()).chunk(2, 1)
        y = y.index_add(0, t, (a * torch.sigmoid(a) * b * w[t, j][:, None]) @ W2d[e].t())
    new = (hd + 0.7 * (1.0 if gd is None else gd) * norm(y + (~on[:, None])) * postd)[on]
    ((new * go.double()[on]).sum() + l64).backward()
    fwd_bar, bwd_bar = 3 * math.sqrt(4) * 0.026, 3 * math.sqrt(8) * 0.026
    assert rel(loss, l64.detach()[None]) < 1e-2  # logits in bf16
    # what the block adds, relative to itself
    assert rel(out[on].double() - h[on].double(), (new - hd[on]).detach()) < fwd_bar
    assert rel(dec[on].double() - h[on].double(), (new - hd[on]).detach()) < fwd_bar
    assert (out[~on] == 0).all() and (dec[~on] == 0).all() and (grads["h"][~on] == 0).all()
    ref = dict(h=hd.grad, pre=pred.grad, post=postd.grad, router=rd.grad, w1=W1d.grad, w2=W2d.grad)
    if g is not None:
        ref["gate"] = gd.grad
    for name, b in ref.items():
        a = grads[name]
        a, b = (a[on], b[on]) if name == "h" else (a, b)
        assert rel(a, b) < bwd_bar, (name, rel(a, b))
    layer.close()


def test_weights_in_experts_or_in_combine_agree():
    """The two places of the routing weights give the same layer up to e4m3's
    roundings, and the same gradients."""
    torch.manual_seed(6)
    R, E, k, H, F, tpr = 2, 8, 2, 256, 128, 64
    T = R * tpr
    W1, W2 = torch.randn((E, 2 * F, H), device=DEV) / H ** 0.5, torch.randn((E, H, F), device=DEV) / F ** 0.5
    w1, w2 = moe.ExpertWeights(W1), moe.ExpertWeights(W2)
    x, logits = torch.randn((T, H), device=DEV).bfloat16(), torch.randn((T, E), device=DEV)
    go = torch.randn((T, H), device=DEV).bfloat16()
    got = []
    for weigh in (False, True):
        layer = moe.MoELayer(R, E, k, H, F, tpr, weigh_in_combine=weigh)
        out, loss, saved = layer.forward(x, logits, w1, w2)
        got.append((out, loss) + layer.backward(go, torch.ones(1, device=DEV), saved, w1, w2))
        layer.check()
        layer.close()
    for a, b in zip(*got):
        assert rel(a, b.double()) < 3 * math.sqrt(8) * 0.026


def test_streams_and_graphs():
    """A norm, the combine and their gradients captured once and replayed on new
    inputs give what the eager calls give, also on another stream."""
    l = Layout(2, 64, 8, 2, 512, 4, seed=8, masked=0.0)
    c = Norms(64, 512, torch.float32, torch.float32, True, True, "vector")
    ws = torch.empty(ep.ep_block_norm_workspace_bytes(512), dtype=torch.uint8, device=DEV)
    bufs = dict(out=torch.empty((64, 512), dtype=torch.bfloat16, device=DEV), dw=torch.empty_like(l.w), dy=torch.empty_like(l.y),
                new=torch.empty_like(c.residual), x=torch.empty_like(c.y), rstd=torch.empty((2, 64), device=DEV),
                dres=torch.empty_like(c.residual), dyn=torch.empty_like(c.y), dpost=torch.empty(512, device=DEV),
                dpre=torch.empty(512, device=DEV), dgate=torch.empty(512, device=DEV))

    def step(b):
        l.h.em_combine_weighted(l.y, l.w, b["out"])
        ep.ep_block_norm_forward(c.residual, b["out"], b["new"], b["x"], rstd=b["rstd"], **c.how)
        ep.ep_block_norm_backward(b["new"], b["out"], b["rstd"], c.dnew, b["x"], b["dres"], b["dyn"], ws,
                                  grad_post_weight=b["dpost"], grad_pre_weight=b["dpre"], grad_gate=b["dgate"], **c.how)
        l.h.em_combine_weighted_backward(b["dyn"], l.y, l.w, ep.EP_BF16, b["dy"], grad_topk_weights=b["dw"])

    step(bufs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(bufs)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(bufs)
    for seed in (1, 2, 3):
        for t in (c.residual, c.dnew, l.w):
            t.copy_(torch.randn(t.shape, generator=gen(seed), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in bufs.items()}
        step(bufs)
        torch.cuda.synchronize()
        _, _, row = l.entries()
        for k in bufs:
            a, b = (got[k][row], bufs[k][row]) if k == "dy" else (got[k], bufs[k])
            assert torch.equal(a, b), k
    assert l.h.get_device_status() == ep.EP_OK
    l.h.close()

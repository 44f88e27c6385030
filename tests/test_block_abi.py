"""The weighted combine's, the norms' and the 4-bit products' entry points
without a GPU: every argument error is refused before any CUDA call."""
import ctypes

import pytest

from combine_ep_get_03_gb300 import build as cuda_build
from combine_ep_get_03_gb300 import ep
from test_experts_abi import BAD_GROUPS, BAD_ROWS, P, groups, rows8

BAD = ep.EP_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return ep.lib()


def test_struct_is_the_headers():
    class Norm(ctypes.Structure):
        _fields_ = [("post", ctypes.c_void_p), ("pre", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                    ("mask", ctypes.c_void_p), ("tokens", ctypes.c_int), ("hidden", ctypes.c_int),
                    ("per_token", ctypes.c_int), ("residual", ctypes.c_int), ("weight", ctypes.c_int),
                    ("eps", ctypes.c_float), ("scale", ctypes.c_float)]

    assert ep._BLOCK_NORM.size == ctypes.sizeof(Norm)
    n = Norm.from_buffer_copy(ep._BLOCK_NORM.pack(1, 2, 3, 4, 5, 6, 7, 8, 9, 0.5, 0.25))
    assert (n.post, n.pre, n.gate, n.mask, n.tokens, n.hidden, n.per_token, n.residual, n.weight, n.eps, n.scale) == (
        1, 2, 3, 4, 5, 6, 7, 8, 9, 0.5, 0.25)


def test_combine_refuses_a_null_handle(lib):
    assert lib.ep_em_combine_weighted(None, P, 4, P, P, 0, None) == BAD
    assert lib.ep_em_combine_weighted_backward(None, P, P, 4, P, ep.EP_BF16, P, None, 0, P, 0, None) == BAD


def norm(post=P, pre=P, gate=P, mask=0, T=4, H=64, per_token=0, res=0, weight=1, eps=1e-6, scale=1.0):
    return ep._BLOCK_NORM.pack(post, pre, gate, mask, T, H, per_token, res, weight, eps, scale)


BAD_NORMS = [None, norm(T=-1), norm(H=0), norm(H=4), norm(H=12), norm(H=16392), norm(H=-8), norm(res=2), norm(res=-1),
             norm(weight=2), norm(post=P + 8), norm(pre=P + 4), norm(gate=P + 2)]


def test_norm_forward_refusals(lib):
    call = lambda n=norm(), r=P, y=P, new=P, x=P, rstd=P: lib.ep_block_norm_forward(n, r, y, new, x, rstd, 0, None)  # noqa: E731
    for n in BAD_NORMS:
        assert call(n=n) == BAD
    for kw in (dict(r=None), dict(new=None), dict(x=None), dict(y=None), dict(r=P + 8), dict(y=P + 2), dict(new=P + 8),
               dict(x=P + 4), dict(rstd=P + 2), dict(n=norm(pre=0)), dict(n=norm(post=0), y=None),
               dict(n=norm(gate=0), y=None), dict(n=norm(post=0, gate=0, pre=0), y=None, x=None)):
        assert call(**kw) == BAD, kw
    assert call(n=norm(T=0), r=None, y=None, new=None, x=None) == ep.EP_OK


def test_norm_workspace_bytes(lib):
    n = ctypes.c_int64()
    assert lib.ep_block_norm_workspace_bytes(7168, ctypes.byref(n)) == ep.EP_OK and n.value == 256 * 2 * 4 * 7168
    for H in (0, -8, 4, 20, 16392):
        assert lib.ep_block_norm_workspace_bytes(H, ctypes.byref(n)) == BAD
    assert lib.ep_block_norm_workspace_bytes(64, None) == BAD


def test_norm_backward_refusals(lib):
    ok = dict(n=norm(), new=P, y=P, rstd=P, gnew=P, gx=P, gr=P, gy=P, gg=P, gpost=P, gpre=P, ws=P)
    call = lambda **kw: (lambda a: lib.ep_block_norm_backward(  # noqa: E731
        a["n"], a["new"], a["y"], a["rstd"], a["gnew"], a["gx"], a["gr"], a["gy"], a["gg"], a["gpost"], a["gpre"],
        a["ws"], 0, None))({**ok, **kw})
    for n in BAD_NORMS:
        assert call(n=n) == BAD
    for kw in (dict(new=None), dict(y=None), dict(rstd=None), dict(gx=None), dict(ws=None), dict(n=norm(gate=0)),
               dict(n=norm(post=0)), dict(n=norm(pre=0)), dict(rstd=P + 2),
               dict(n=norm(post=0), gpost=None, gy=None, y=None), dict(gpre=None, n=norm(pre=0), gx=P)):
        assert call(**kw) == BAD, kw
    for k in ok:
        if k not in ("n", "rstd"):
            assert call(**{k: P + 8}) == BAD, k
    # nothing asked for is nothing done
    assert call(gr=None, gy=None, gg=None, gpost=None, gpre=None) == ep.EP_OK


def test_w4_refusals(lib):
    call = lambda g=groups(), x=rows8(), w=P, s=P, N=256, K=256, out=P: lib.ep_grouped_matmul_w4(  # noqa: E731
        g, x, w, s, N, K, out, 0, None)
    for g in BAD_GROUPS:
        assert call(g=g) == BAD
    for x in BAD_ROWS:
        assert call(x=x) == BAD
    for kw in (dict(w=None), dict(w=P + 16), dict(s=None), dict(s=P + 8), dict(N=0), dict(N=4), dict(N=260), dict(K=0),
               dict(K=64), dict(K=200), dict(out=None), dict(out=P + 8), dict(N=1 << 30),
               dict(g=groups(rows=(1 << 31) - 1), N=1 << 20)):
        assert call(**kw) == BAD, kw
    assert call(g=groups(rows=0), x=None, out=None) == ep.EP_OK


def test_w4_swiglu_refusals(lib):
    call = lambda g=groups(), x=rows8(), w=P, s=P, F=256, K=256, rw=None, act=rows8(): (  # noqa: E731
        lib.ep_grouped_matmul_w4_swiglu(g, x, w, s, F, K, rw, act, 0, None))
    for g in BAD_GROUPS:
        assert call(g=g) == BAD
    for r in BAD_ROWS:
        assert call(x=r) == BAD and call(act=r) == BAD
    for kw in (dict(w=None), dict(w=P + 16), dict(s=None), dict(s=P + 4), dict(F=0), dict(F=64), dict(F=192),
               dict(K=100), dict(rw=P + 2), dict(F=1 << 29), dict(F=1 << 30)):
        assert call(**kw) == BAD, kw
    assert call(g=groups(rows=0), x=None, act=None) == ep.EP_OK


def test_quantize_e2m1_on_the_cpu():
    """Nearest codes, exponents of the largest magnitude, the scales' places."""
    import torch

    from combine_ep_get_03_gb300 import moe

    torch.manual_seed(0)
    w = torch.randn(2, 136, 256) * torch.exp2(torch.randint(-8, 8, (2, 136, 1)).float())
    w[0, 3, 32:64] = 0
    w[1, 7, :4] = torch.tensor([6.0, 0.25, -1.25, -7.9]) * 2 ** 10
    w[1, 7, 4:32] = 2.0 ** 11
    q, s = moe.quantize_e2m1(w)
    assert q.shape == (2, 136, 128) and s.shape == (2, 2, 2, 512)
    value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6])
    codes = torch.stack((q & 15, q >> 4), -1).view(2, 136, 256).long()
    v = value[codes & 7] * (1 - 2 * (codes >> 3))
    nat = torch.empty(2, 136, 8)
    for n in range(136):
        for c in range(8):
            nat[:, n, c] = s[:, n // 128, c // 4, 16 * (n % 32) + 4 * (n % 128 // 32) + c % 4].float()
    got = v * torch.exp2(nat - 127).repeat_interleave(32, 2)
    step = torch.exp2(nat - 127).repeat_interleave(32, 2)
    # at most half the widest gap (4 to 6), and 2 beyond 6 where the maximum lies in [6, 8)
    assert ((got - w).abs() <= step * torch.where((w / step).abs() > 6, 2.0, 1.0)).all()
    small = (w / step).abs() <= 2
    assert ((got - w).abs()[small] <= step[small] * 0.25).all()
    assert got[1, 7, 0] == 6 * 2 ** 10 and got[1, 7, 3] == -6 * 2 ** 10 and (got[0, 3, 32:64] == 0).all()

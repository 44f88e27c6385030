"""Groups as the device may hold them: counts that overlap, and as many groups
as the header allows.  Bounds as derived in test_gpu_experts.py."""
import pytest
import torch

from combine_ep_get_03_gb300 import ep
from test_gpu_experts import DEV, Rows, check8, gen, product64, quantize, silu64, sum_err, weights, within

pytestmark = pytest.mark.gpu


def test_overlapping_groups_end_and_are_reported():
    """Every group claims the whole buffer: far more tiles than rows.  The calls
    end after the tiles that groups side by side could have, report it, and
    touch no row past the claimed ones."""
    G, n, spare, K, N = 64, 1024, 32, 128, 512
    rows = n + spare
    v = torch.randn((rows, K), generator=gen(1), device=DEV)
    xq, sc = quantize(v)
    xs = sc.t().contiguous()
    q, s, _ = weights(G, N, K, 2)
    count = torch.full((G,), n, dtype=torch.int32, device=DEV)
    offset = torch.zeros(G, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((rows, N), -5.5, dtype=torch.bfloat16, device=DEV)
    ep.ep_grouped_matmul(xq, xs, q, s, out, count, group_offset=offset, device_status=status)
    assert int(status) == ep.EP_ERR_CAPACITY and (out[n:] == -5.5).all()
    status.zero_()
    act = torch.full((rows, N // 2), 0x5A, dtype=torch.uint8, device=DEV)
    act_s = torch.full((N // 256, rows), 7.25, device=DEV)
    ep.ep_grouped_matmul_swiglu(xq, xs, q, s, act, act_s, count, group_offset=offset, device_status=status)
    assert int(status) == ep.EP_ERR_CAPACITY and (act[n:] == 0x5A).all() and (act_s[:, n:] == 7.25).all()
    status.zero_()
    pre, pre_s = torch.zeros((rows, N), dtype=torch.uint8, device=DEV), torch.ones((N // 128, rows), device=DEV)
    dp = torch.full((rows, N), 0x5A, dtype=torch.uint8, device=DEV)
    dps = torch.full((N // 128, rows), 7.25, device=DEV)
    ep.ep_grouped_swiglu_backward(torch.zeros((rows, N // 2), dtype=torch.bfloat16, device=DEV), pre, pre_s, dp, dps,
                                  count, group_offset=offset, device_status=status)
    assert int(status) == ep.EP_ERR_CAPACITY and (dp[n:] == 0x5A).all() and (dps[:, n:] == 7.25).all()


def test_full_groups_side_by_side_are_not_overlapping():
    """As many tiles as rows / 128 + groups allow, with no slack: every group
    ends in a partial tile."""
    for counts in ([1, 1, 1, 125], [129, 127], [1] * 128, [128], [1]):
        r = Rows(counts, "em")
        xq, xs, x = r.fp8(128, 3)
        q, s, w = weights(len(counts), 64, 128, 4)
        out = r.out16(64)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        ep.ep_grouped_matmul(xq, xs, q, s, out, **r.args(device_status=status))
        y, mag = product64(r, x, w)
        within(r.read16(out), y, y.abs() * 2.0 ** -8 + sum_err(128) * mag, "product")
        assert int(status) == ep.EP_OK


@pytest.mark.parametrize("layout", ["em", "ll"])
@pytest.mark.parametrize("G", [2718, 2719, 4096])
def test_as_many_groups_as_the_header_allows(G, layout):
    """Up to 4096 groups, most of them small, some empty, the last one not."""
    N = K = 128
    counts = torch.randint(0, 4, (G,), generator=torch.Generator().manual_seed(G)).tolist()
    counts[5], counts[-1] = 70, 2
    r = Rows(counts, layout, 1)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = r.args(device_status=status)
    xq, xs, x = r.fp8(K, 5)
    yq, ys, y = r.fp8(N, 6, sigma=1e-2)

    dw = torch.full((G, N, K), float("nan"), dtype=torch.bfloat16, device=DEV)
    ep.ep_grouped_weight_grad(yq, ys, xq, xs, dw, **args)
    group = torch.repeat_interleave(torch.arange(G, device=DEV), r.count)
    slot = torch.cat([torch.arange(c) for c in counts]).to(DEV)
    py, px = (torch.zeros((G, max(counts), N), dtype=torch.float64, device=DEV) for _ in range(2))
    py[group, slot], px[group, slot] = y, x
    ref, mag = py.transpose(1, 2) @ px, py.abs().transpose(1, 2) @ px.abs()
    within(dw.double(), ref, ref.abs() * 2.0 ** -8 + mag * 2.0 ** -8.9, "weight gradient")

    q, s, w = weights(G, 2 * N, K, 7)
    out = r.out16(2 * N)
    ep.ep_grouped_matmul(xq, xs, q, s, out, **args)
    p, pmag = product64(r, x, w)
    within(r.read16(out), p, p.abs() * 2.0 ** -8 + sum_err(K) * pmag, "product")

    act, acts = r.out8(N)
    ep.ep_grouped_matmul_swiglu(xq, xs, q, s, act, acts, **args)
    (g, u), (eg, eu) = p.chunk(2, 1), (sum_err(K) * pmag).chunk(2, 1)
    a = silu64(g) * u
    ea = (1.1 * eg) * u.abs() + (silu64(g).abs() + 1.1 * eg) * eu + (16 + 2 * g.abs()) * 2.0 ** -24 * a.abs()
    check8(*r.read8(act, acts), a, ea, "activations")

    pq, ps, pre = r.fp8(2 * N, 8, sigma=2.0)
    d = torch.zeros((r.rows, N), dtype=torch.bfloat16, device=DEV)
    d[r.live] = torch.randn((len(r.live), N), generator=gen(9), device=DEV).bfloat16()
    dp, dps = r.out8(2 * N)
    ep.ep_grouped_swiglu_backward(d.view(r.lead + (N,)), pq, ps, dp, dps, **args)
    (g, u), d = pre.chunk(2, 1), d[r.live].double()
    sg = torch.sigmoid(g)
    grad = torch.cat([d * u * sg * (1 + g * (1 - sg)), d * silu64(g)], 1)
    eg = torch.cat([(d * u).abs() * sg * (1 + g.abs() + silu64(g).abs()), (d * silu64(g)).abs()], 1)
    check8(*r.read8(dp, dps), grad, eg * (16 + 2 * g.abs().repeat(1, 2)) * 2.0 ** -24, "gradient")
    assert int(status) == ep.EP_OK


@pytest.mark.parametrize("lead", [(0,), (3, 0)])
def test_buffers_without_rows(lead):
    """No rows at all: nothing to write, and weight gradients of zero."""
    G, N, K = 3, 128, 256
    f8 = lambda w: torch.empty(lead + (w,), dtype=torch.uint8, device=DEV)  # noqa: E731
    f32 = lambda w: torch.empty((w // 128, 4) if len(lead) == 1 else lead + (w // 128,), device=DEV)  # noqa: E731
    bf = lambda w: torch.empty(lead + (w,), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    zero = torch.zeros(G, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = dict(group_count=zero, group_offset=zero if len(lead) == 1 else None, device_status=status)
    q, s, _ = weights(G, 2 * N, K, 1)
    ep.ep_grouped_matmul(f8(K), f32(K), q, s, bf(2 * N), **args)
    ep.ep_grouped_matmul_swiglu(f8(K), f32(K), q, s, f8(N), f32(N), pre=f8(2 * N), pre_scales=f32(2 * N), **args)
    ep.ep_grouped_swiglu_backward(bf(N), f8(2 * N), f32(2 * N), f8(2 * N), f32(2 * N), **args)
    dw = torch.full((G, N, K), float("nan"), dtype=torch.bfloat16, device=DEV)
    ep.ep_grouped_weight_grad(f8(N), f32(N), f8(K), f32(K), dw, **args)
    assert not dw.any() and int(status) == ep.EP_OK

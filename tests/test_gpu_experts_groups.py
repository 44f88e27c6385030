"""Groups as the device may hold them: counts that overlap, and as many groups
as the header allows.  Bounds as derived in test_gpu_experts.py."""
import pytest
import torch

from combine_ep_get_03_gb300 import ep
from test_gpu_experts import DEV, Rows, gen, product64, quantize, sum_err, weights, within

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

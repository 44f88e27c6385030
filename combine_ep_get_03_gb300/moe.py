"""A Mixture-of-Experts layer of this library's calls, forward, backward and
decode: gate -> dispatch -> experts -> combine.

``python -m combine_ep_get_03_gb300.moe`` runs one training step and one decode
step of a small layer on synthetic data and prints what they took.

Training: the gate routes (``ep_gate_forward``); the expert-major dispatch sends
each token's row to its experts in e4m3; the first product applies SwiGLU and
the routing weights in its epilogue and keeps the pre-activations in 8 bits;
the second product's rows are combined.  The backward pass dispatches the
output's gradient through the same layout and uses the 8-bit rows as they are
kept: the dispatched x, the activations and the pre-activations.

Decode: the low-latency dispatch, the same products on its [E, M, width] slots,
and the combine that applies the routing weights.
"""
from __future__ import annotations

import torch

from . import ep

E4M3_MAX = 448.0


def quantize_blocks(w: torch.Tensor):
    """[E, N, K] weights -> e4m3 codes and one fp32 scale for every 128 x 128 block."""
    E, N, K = w.shape
    nb = (N + 127) // 128
    q = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device=w.device)
    s = torch.empty((E, nb, K // 128), dtype=torch.float32, device=w.device)
    for e in range(E):
        b = torch.zeros((nb * 128, K), dtype=torch.float32, device=w.device)
        b[:N] = w[e]
        b = b.view(nb, 128, K // 128, 128)
        a = b.abs().amax((1, 3)).clamp_min(1e-4)
        s[e] = a / E4M3_MAX
        q[e] = (b * (E4M3_MAX / a)[:, None, :, None]).view(nb * 128, K)[:N].to(torch.float8_e4m3fn)
    return q, s


class ExpertWeights:
    """One projection's experts, [E, N, K], in e4m3; transposed too where the
    backward pass needs them (the same codes: a block's scale is its
    transpose's)."""

    def __init__(self, w: torch.Tensor, training: bool = True):
        self.q, self.s = quantize_blocks(w)
        self.qt = self.st = None
        if training:
            self.qt = self.q.view(torch.uint8).transpose(1, 2).contiguous().view(torch.float8_e4m3fn)
            self.st = self.s.transpose(1, 2).contiguous()


class MoELayer:
    """hidden and ffn are multiples of 128.  Every output is a tensor of its
    own, and what forward saves is all that its backward needs: other forwards
    and decodes may come between, and backward calls in any order.  The handle
    and the gate's workspace are the layer's, so its calls go to one stream at a
    time."""

    def __init__(self, num_ranks, num_experts, num_topk, hidden, ffn, max_tokens_per_rank, score=ep.EP_GATE_SOFTMAX,
                 num_groups=1, topk_groups=1, loss_coef=1e-2, expert_alignment=128, device="cuda"):
        self.R, self.E, self.k, self.H, self.F = num_ranks, num_experts, num_topk, hidden, ffn
        self.gate = dict(score=score, loss_coef=loss_coef)
        self.limit = dict(num_groups=num_groups, topk_groups=topk_groups)
        self.align = expert_alignment
        self.dev = torch.device(device)
        self.h = ep.Handle(num_ranks, num_experts, num_topk, hidden, max_tokens_per_rank)
        rows, _ = ep.ep_get_buffer_size_hint(num_ranks, num_experts, num_topk, hidden, max_tokens_per_rank,
                                             ep.EP_FP8_E4M3, ep.EP_LAYOUT_EXPERT_MAJOR, expert_alignment)
        self.rows, self.ld = rows, (rows + 3) // 4 * 4
        self.workspace = torch.zeros(ep.ep_gate_workspace_bytes(num_experts), dtype=torch.uint8, device=self.dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.dev)

    def close(self):
        self.h.close()

    def _fp8(self, width):
        return (torch.empty((self.rows, width), dtype=torch.float8_e4m3fn, device=self.dev),
                torch.empty((width // 128, self.ld), dtype=torch.float32, device=self.dev))

    def _f32(self, *shape):
        return torch.empty(shape, dtype=torch.float32, device=self.dev)

    def _bf16(self, *shape):
        return torch.empty(shape, dtype=torch.bfloat16, device=self.dev)

    def _i32(self, n):
        return torch.empty(n, dtype=torch.int32, device=self.dev)

    def route(self, logits, token_mask=None):
        """Gate of logits [T, E]: (topk_idx, topk_weights, expert_count, loss)."""
        T = logits.shape[0]
        idx = torch.empty((T, self.k), dtype=torch.int64, device=self.dev)
        w, prob, loss = self._f32(T, self.k), self._f32(self.E), self._f32(1)
        count = self._i32(self.E + 1)
        ep.ep_gate_forward(logits, idx, w, count, prob, loss, self.workspace, token_mask=token_mask, **self.gate,
                           **self.limit)
        return idx, w, count, loss

    def forward(self, x, logits, w1: ExpertWeights, w2: ExpertWeights, token_mask=None):
        """x bf16 [T, H], logits [T, E]; w1 [E, 2F, H] (gate rows, then up rows),
        w2 [E, H, F].  -> (out bf16 [T, H], balance loss [1], saved)."""
        T = x.shape[0]
        idx, w, count, loss = self.route(logits, token_mask)
        xq, xs = self._fp8(self.H)
        row_w = self._f32(self.rows)
        # no tokens, no weights: an empty tensor has no address to give with recv_weights
        self.h.em_layout_and_dispatch(idx, x, w, ep.EP_FP8_E4M3, self.align, xq, xs, recv_weights=row_w if T else None)
        offset, rows = self._i32(self.E + 1), self._i32(self.E)
        self.h.em_get_groups(offset, rows)
        groups = dict(group_count=rows, group_offset=offset, device_status=self.status)
        act, act_s = self._fp8(self.F)
        pre, pre_s = self._fp8(2 * self.F)
        ep.ep_grouped_matmul_swiglu(xq, xs, w1.q, w1.s, act, act_s, row_weights=row_w, pre=pre, pre_scales=pre_s,
                                    **groups)
        y = self._bf16(self.rows, self.H)
        ep.ep_grouped_matmul(act, act_s, w2.q, w2.s, y, **groups)
        out = self._bf16(T, self.H)
        self.h.em_combine(y, out)
        return out, loss, (logits, token_mask, idx, count, self.h.em_layouts, groups, xq, xs, row_w, act, act_s, pre,
                           pre_s)

    def backward(self, grad_out, grad_loss, saved, w1: ExpertWeights, w2: ExpertWeights):
        """-> (grad_x bf16 [T, H], grad_logits, grad_w1, grad_w2 bf16).

        Gradients travel in e4m3 with a scale for 128 channels, whose largest
        magnitude counts as 1e-4 at least: below that they lose bits, and below
        2e-10 they are 0.  Every result is linear in (grad_out, grad_loss), so
        where a mean over many tokens makes gradients that small, scale both up
        by a power of two (the loss, before its backward) and the results down."""
        logits, token_mask, idx, count, layout, groups, xq, xs, row_w, act, act_s, pre, pre_s = saved
        T = grad_out.shape[0]
        gy, gy_s = self._fp8(self.H)
        if self.h.em_layouts == layout:
            self.h.em_dispatch(grad_out, None, ep.EP_FP8_E4M3, gy, gy_s)
        else:  # another forward came between: the same ids give the same rows again
            self.h.em_layout_and_dispatch(idx, grad_out, None, ep.EP_FP8_E4M3, self.align, gy, gy_s)
        grad_w2 = self._bf16(self.E, self.H, self.F)
        ep.ep_grouped_weight_grad(gy, gy_s, act, act_s, grad_w2, **groups)
        grad_act = self._bf16(self.rows, self.F)
        ep.ep_grouped_matmul(gy, gy_s, w2.qt, w2.st, grad_act, **groups)
        gp, gp_s = self._fp8(2 * self.F)
        grad_row_w = self._f32(self.rows)
        ep.ep_grouped_swiglu_backward(grad_act, pre, pre_s, gp, gp_s, row_weights=row_w,
                                      grad_row_weights=grad_row_w, **groups)
        grad_w1 = self._bf16(self.E, 2 * self.F, self.H)
        ep.ep_grouped_weight_grad(gp, gp_s, xq, xs, grad_w1, **groups)
        grad_rows = self._bf16(self.rows, self.H)
        ep.ep_grouped_matmul(gp, gp_s, w1.qt, w1.st, grad_rows, **groups)
        grad_x = self._bf16(T, self.H)
        self.h.em_combine(grad_rows, grad_x)
        grad_w = self._f32(T, self.k)
        self.h.em_combine_weights(grad_row_w, grad_w)
        grad_logits = torch.empty_like(logits)
        ep.ep_gate_backward(logits, idx, count, grad_w, grad_loss, grad_logits, token_mask=token_mask, **self.gate)
        return grad_x, grad_logits, grad_w1, grad_w2

    def decode(self, x, logits, w1: ExpertWeights, w2: ExpertWeights, token_mask=None):
        """The low-latency path: x bf16 [T, H], logits [T, E] -> out bf16 [T, H]."""
        T, M, E = x.shape[0], self.h.M, self.E
        idx, w, _, _ = self.route(logits, token_mask)
        f8 = lambda width: torch.empty((E, M, width), dtype=torch.float8_e4m3fn, device=self.dev)  # noqa: E731
        xq, xs = f8(self.H), self._f32(E, M, self.H // 128)
        count = self._i32(E)
        self.h.low_latency_dispatch(x, idx, ep.EP_FP8_E4M3, xq, xs, recv_count=count)
        act, act_s = f8(self.F), self._f32(E, M, self.F // 128)
        ep.ep_grouped_matmul_swiglu(xq, xs, w1.q, w1.s, act, act_s, count, device_status=self.status)
        y = self._bf16(E, M, self.H)
        ep.ep_grouped_matmul(act, act_s, w2.q, w2.s, y, count, device_status=self.status)
        out = self._bf16(T, self.H)
        self.h.low_latency_combine(y, w, out)
        return out

    def check(self):
        """Synchronise and raise what the device found, if anything."""
        st = self.h.get_device_status()
        st = st if st != ep.EP_OK else int(self.status.item())
        if st != ep.EP_OK:
            self.status.zero_()
            raise ep.EPError(st, "MoELayer")


def main():
    torch.manual_seed(0)
    R, E, k, H, F, tpr = 8, 32, 8, 1024, 512, 64
    T = R * tpr
    dev = "cuda"
    layer = MoELayer(R, E, k, H, F, tpr, score=ep.EP_GATE_SIGMOID, num_groups=8, topk_groups=4)
    w1 = ExpertWeights(torch.randn((E, 2 * F, H), device=dev) / H ** 0.5)
    w2 = ExpertWeights(torch.randn((E, H, F), device=dev) / F ** 0.5)
    x = torch.randn((T, H), device=dev).bfloat16()
    logits = torch.randn((T, E), device=dev)
    grad_out, grad_loss = (torch.randn((T, H), device=dev) * 1e-2).bfloat16(), torch.ones(1, device=dev)

    def timed(fn):
        fn()
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        out = fn()
        b.record()
        torch.cuda.synchronize()
        return out, a.elapsed_time(b) * 1e3

    (out, loss, saved), fwd = timed(lambda: layer.forward(x, logits, w1, w2))
    grads, bwd = timed(lambda: layer.backward(grad_out, grad_loss, saved, w1, w2))
    dec, ll = timed(lambda: layer.decode(x[:R], logits[:R], w1, w2))
    layer.check()
    print(f"training step: balance loss {loss.item():.5f}, |out| {out.float().norm().item():.3f}, "
          f"|grad x| {grads[0].float().norm().item():.4f}, |grad w1| {grads[2].float().norm().item():.3f}; "
          f"forward {fwd:.0f} us, backward {bwd:.0f} us")
    print(f"decode of {R} tokens: |out| {dec.float().norm().item():.3f}; {ll:.0f} us")
    layer.close()


if __name__ == "__main__":
    main()

"""A Mixture-of-Experts layer of this library's calls, forward, backward and
decode: gate -> dispatch -> experts -> combine, and the block of a model around
it: norm -> router -> layer -> norm, gate and residual sum.

``python -m combine_ep_get_03_gb300.moe`` runs one training step and one decode
step of a small block on synthetic data and prints what they took.

Training: the gate routes (``ep_gate_forward``); the expert-major dispatch sends
each token's row to its experts in e4m3; the first product applies SwiGLU and
the routing weights in its epilogue and keeps the pre-activations in 8 bits;
the second product's rows are combined.  The backward pass dispatches the
output's gradient through the same layout and uses the 8-bit rows as they are
kept: the dispatched x, the activations and the pre-activations.  Or the
combine applies the routing weights (``weigh_in_combine``): their gradient then
comes from the experts' bf16 results instead of the 8-bit activations.

Decode: the low-latency dispatch, the same products on its [E, M, width] slots,
and the combine that applies the routing weights.  Its weights, and those of a
forward pass that no backward follows, may have 4 bits (``ExpertWeights4``).
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


# Half way between 0, 0.5, 1, 1.5, 2, 3, 4, 6, the borders to even codes an fp32 step
# lower: a weight on a border goes to the even code.
_STEP = 2.0 ** -24
_E2M1_BORDERS = (0.25, 0.75 - _STEP, 1.25, 1.75 - 2 * _STEP, 2.5, 3.5 - 4 * _STEP, 5.0)


def quantize_e2m1(w: torch.Tensor):
    """[E, N, K] weights -> 4-bit codes [E, N, K/2] and the exponents of every 32
    channels [E, ceil(N/128), K/128, 512], as ``ep_grouped_matmul_w4`` takes them.

    The largest magnitude of 32 channels lies in [4, 8) steps of 2^exponent; what
    is above 6 becomes 6, the rest rounds to the nearest value, ties to even codes.
    32 channels with a weight that is not finite get the exponent of NaN."""
    E, N, K = w.shape
    nb, kb = (N + 127) // 128, K // 128
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((E, nb, kb, 512), dtype=torch.uint8, device=w.device)
    borders = torch.tensor(_E2M1_BORDERS, device=w.device)
    for e in range(E):
        b = w[e].float().view(N, K // 32, 32)
        # exponents 2^-127 .. 2^127; 32 zeros take the smallest, and stay zeros
        x = (torch.frexp(b.abs().amax(2)).exponent - 3).clamp(-127, 127)
        x = torch.where(b.abs().amax(2) > 0, x, torch.full_like(x, -127))
        t = torch.ldexp(b.double(), -x[..., None])
        c = torch.bucketize(t.abs().float(), borders, out_int32=True).to(torch.uint8) | ((t < 0).to(torch.uint8) << 3)
        c = c.view(N, K // 2, 2)
        codes[e] = c[..., 0] | (c[..., 1] << 4)
        s = torch.full((nb * 128, K // 32), 127, dtype=torch.uint8, device=w.device)
        s[:N] = torch.where(b.isfinite().all(2), x + 127, 255).to(torch.uint8)
        scales[e] = s.view(nb, 4, 32, kb, 4).permute(0, 3, 2, 1, 4).reshape(nb, kb, 512)
    return codes, scales


class ExpertWeights4:
    """One projection's experts, [E, N, K], in 4 bits: for serving."""

    def __init__(self, w: torch.Tensor):
        self.q, self.s = quantize_e2m1(w)


class MoELayer:
    """hidden and ffn are multiples of 128.  Every output is a tensor of its
    own, and what forward saves is all that its backward needs: other forwards
    and decodes may come between, replayed from a graph too, and backward calls in
    any order.  The handle and the gate's workspace are the layer's, so its calls
    go to one stream at a time."""

    def __init__(self, num_ranks, num_experts, num_topk, hidden, ffn, max_tokens_per_rank, score=ep.EP_GATE_SOFTMAX,
                 num_groups=1, topk_groups=1, loss_coef=1e-2, expert_alignment=128, device="cuda",
                 weigh_in_combine=False):
        self.R, self.E, self.k, self.H, self.F = num_ranks, num_experts, num_topk, hidden, ffn
        self.gate = dict(score=score, loss_coef=loss_coef)
        self.limit = dict(num_groups=num_groups, topk_groups=topk_groups)
        self.align = expert_alignment
        self.weigh_in_combine = weigh_in_combine
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
        w2 [E, H, F].  -> (out bf16 [T, H], balance loss [1], saved).  With
        4-bit weights nothing is saved: no backward follows."""
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
        four = isinstance(w1, ExpertWeights4)
        pre, pre_s = (None, None) if four else self._fp8(2 * self.F)
        in_experts = None if self.weigh_in_combine else row_w
        y = self._bf16(self.rows, self.H)
        if four:
            ep.ep_grouped_matmul_w4_swiglu(xq, xs, w1.q, w1.s, act, act_s, row_weights=in_experts, **groups)
            ep.ep_grouped_matmul_w4(act, act_s, w2.q, w2.s, y, **groups)
        else:
            ep.ep_grouped_matmul_swiglu(xq, xs, w1.q, w1.s, act, act_s, row_weights=in_experts, pre=pre, pre_scales=pre_s,
                                        **groups)
            ep.ep_grouped_matmul(act, act_s, w2.q, w2.s, y, **groups)
        out = self._bf16(T, self.H)
        if self.weigh_in_combine:
            self.h.em_combine_weighted(y, w, out)
        else:
            self.h.em_combine(y, out)
        if four:
            return out, loss, None
        return out, loss, (logits, token_mask, idx, count, self.h.em_layouts, groups, xq, xs, row_w, act, act_s, pre,
                           pre_s, (w, y) if self.weigh_in_combine else None)

    def backward(self, grad_out, grad_loss, saved, w1: ExpertWeights, w2: ExpertWeights):
        """-> (grad_x bf16 [T, H], grad_logits, grad_w1, grad_w2 bf16).

        Gradients travel in e4m3 with a scale for 128 channels, whose largest
        magnitude counts as 1e-4 at least: below that they lose bits, and below
        2e-10 they are 0.  Every result is linear in (grad_out, grad_loss), so
        where a mean over many tokens makes gradients that small, scale both up
        by a power of two (the loss, before its backward) and the results down."""
        logits, token_mask, idx, count, layout, groups, xq, xs, row_w, act, act_s, pre, pre_s, weighed = saved
        T = grad_out.shape[0]
        gy, gy_s = self._fp8(self.H)
        grad_w = self._f32(T, self.k)
        # another forward came, or may have been replayed, between: the same ids give the same rows again
        if self.h.em_captured or self.h.em_layouts != layout:
            self.h.em_layout_and_dispatch(idx, grad_out, None, ep.EP_FP8_E4M3, self.align, gy, gy_s)
        elif not weighed:
            self.h.em_dispatch(grad_out, None, ep.EP_FP8_E4M3, gy, gy_s)
        if weighed:
            w, y = weighed
            self.h.em_combine_weighted_backward(grad_out, y, w, ep.EP_FP8_E4M3, gy, gy_s, grad_topk_weights=grad_w)
        grad_w2 = self._bf16(self.E, self.H, self.F)
        ep.ep_grouped_weight_grad(gy, gy_s, act, act_s, grad_w2, **groups)
        grad_act = self._bf16(self.rows, self.F)
        ep.ep_grouped_matmul(gy, gy_s, w2.qt, w2.st, grad_act, **groups)
        gp, gp_s = self._fp8(2 * self.F)
        grad_row_w = None if weighed else self._f32(self.rows)
        ep.ep_grouped_swiglu_backward(grad_act, pre, pre_s, gp, gp_s, row_weights=None if weighed else row_w,
                                      grad_row_weights=grad_row_w, **groups)
        grad_w1 = self._bf16(self.E, 2 * self.F, self.H)
        ep.ep_grouped_weight_grad(gp, gp_s, xq, xs, grad_w1, **groups)
        grad_rows = self._bf16(self.rows, self.H)
        ep.ep_grouped_matmul(gp, gp_s, w1.qt, w1.st, grad_rows, **groups)
        grad_x = self._bf16(T, self.H)
        self.h.em_combine(grad_rows, grad_x)
        if not weighed:
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
        four = isinstance(w1, ExpertWeights4)
        first, second = ((ep.ep_grouped_matmul_w4_swiglu, ep.ep_grouped_matmul_w4) if four else
                         (ep.ep_grouped_matmul_swiglu, ep.ep_grouped_matmul))
        first(xq, xs, w1.q, w1.s, act, act_s, count, device_status=self.status)
        y = self._bf16(E, M, self.H)
        second(act, act_s, w2.q, w2.s, y, count, device_status=self.status)
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


class MoEBlock:
    """The block of a model around a layer of experts, on the residual stream h
    [T, H] (fp32 or bf16):

        x = norm(h) pre;  y = layer(x) routed by x @ router.T
        h' = h + residual_scale * gate * (norm(y) * post)

    pre and post [H] (post may be None: no norm behind), gate [H], [T, H] bf16 or
    None, router [E, H] bf16 or fp32.  The logits are fp32 for both: of two experts
    close together a bf16 logit, of 8 bits, would make a tie.  What forward saves is
    complete, as the layer's.

    The norm in front and what is behind are two calls, so that a block stands
    alone: h is written and read between two blocks, and the next norm takes it as it
    was rounded.  ``ep_block_norm_forward`` does both at once, with the next block's
    pre."""

    def __init__(self, layer: MoELayer, pre, router, post=None, gate=None, residual_scale=1.0, eps=1e-6):
        self.layer, self.pre, self.post, self.gate, self.router = layer, pre, post, gate, router
        self.scale, self.eps = residual_scale, eps
        self.workspace = torch.empty(ep.ep_block_norm_workspace_bytes(layer.H), dtype=torch.uint8, device=layer.dev)

    def _front(self, h, token_mask, rstd=None):
        x = self.layer._bf16(*h.shape)
        ep.ep_block_norm_forward(h, None, None, x, rstd=rstd, pre_weight=self.pre, eps=self.eps, token_mask=token_mask)
        if self.router.dtype is torch.float32:
            return x, x.float() @ self.router.t()
        return x, torch.mm(x, self.router.t(), out_dtype=torch.float32)

    def _behind(self, h, y, out, token_mask, rstd=None):
        ep.ep_block_norm_forward(h, y, out, None, rstd=rstd, post_weight=self.post, gate=self.gate, eps=self.eps,
                                 residual_scale=self.scale, token_mask=token_mask)

    def forward(self, h, w1, w2, token_mask=None):
        """-> (h' , balance loss [1], saved); padding tokens' rows of h' are 0."""
        rstd = self.layer._f32(2, h.shape[0])
        x, logits = self._front(h, token_mask, rstd)
        y, loss, saved = self.layer.forward(x, logits, w1, w2, token_mask)
        out = torch.empty_like(h)
        self._behind(h, y, out, token_mask, rstd)
        return out, loss, (h, x, y, rstd, token_mask, saved)

    def backward(self, grad_h, grad_loss, saved, w1: ExpertWeights, w2: ExpertWeights):
        """Gradients from those of h' and of the balance loss: a dict of h, pre,
        post, gate (where there is one), router, w1 and w2."""
        h, x, y, rstd, mask, inner = saved
        f32 = lambda on: self.layer._f32(self.layer.H) if on else None  # noqa: E731
        per_token = self.gate is not None and self.gate.dim() == 2
        grad_post = f32(self.post is not None)
        grad_gate = torch.empty_like(self.gate) if per_token else f32(self.gate is not None)
        grad_y = self.layer._bf16(*y.shape)
        ep.ep_block_norm_backward(None, y, rstd, grad_h, None, None, grad_y, self.workspace, post_weight=self.post,
                                  gate=self.gate, grad_post_weight=grad_post, grad_gate=grad_gate,
                                  residual_scale=self.scale, token_mask=mask)
        grad_x, grad_logits, grad_w1, grad_w2 = self.layer.backward(grad_y, grad_loss, inner, w1, w2)
        if self.router.dtype is torch.float32:
            grad_router = grad_logits.t() @ x.float()
            grad_x = torch.addmm(grad_x.float(), grad_logits, self.router).bfloat16()
        else:  # the products take the logits' gradient in bf16; their sums are fp32
            grad_logits = grad_logits.bfloat16()
            grad_router = grad_logits.t() @ x
            grad_x = torch.addmm(grad_x, grad_logits, self.router)
        grad, grad_pre = torch.empty_like(h), f32(True)
        ep.ep_block_norm_backward(h, None, rstd, grad_h, grad_x, grad, None, self.workspace, pre_weight=self.pre,
                                  grad_pre_weight=grad_pre, token_mask=mask)
        return dict(h=grad, pre=grad_pre, post=grad_post, gate=grad_gate, router=grad_router, w1=grad_w1, w2=grad_w2)

    def decode(self, h, w1, w2, token_mask=None):
        """One step for tokens h [T, H], in place."""
        x, logits = self._front(h, token_mask)
        self._behind(h, self.layer.decode(x, logits, w1, w2, token_mask), h, token_mask)
        return h


def main():
    torch.manual_seed(0)
    R, E, k, H, F, tpr = 8, 32, 8, 1024, 512, 64
    T = R * tpr
    dev = "cuda"
    layer = MoELayer(R, E, k, H, F, tpr, score=ep.EP_GATE_SIGMOID, num_groups=8, topk_groups=4)
    W1, W2 = torch.randn((E, 2 * F, H), device=dev) / H ** 0.5, torch.randn((E, H, F), device=dev) / F ** 0.5
    w1, w2 = ExpertWeights(W1), ExpertWeights(W2)
    w1_4, w2_4 = ExpertWeights4(W1), ExpertWeights4(W2)
    norm = lambda: torch.ones(H, device=dev)  # noqa: E731
    block = MoEBlock(layer, norm(), (torch.randn((E, H), device=dev) / H ** 0.5).bfloat16(), post=norm())
    h = torch.randn((T, H), device=dev)
    grad_h, grad_loss = torch.randn((T, H), device=dev) * 1e-2, torch.ones(1, device=dev)

    def timed(fn):
        fn()
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        out = fn()
        b.record()
        torch.cuda.synchronize()
        return out, a.elapsed_time(b) * 1e3

    (out, loss, saved), fwd = timed(lambda: block.forward(h, w1, w2))
    grads, bwd = timed(lambda: block.backward(grad_h, grad_loss, saved, w1, w2))
    dec, ll = timed(lambda: block.decode(h[:R].clone(), w1, w2))
    dec4, ll4 = timed(lambda: block.decode(h[:R].clone(), w1_4, w2_4))
    layer.check()
    print(f"training step: balance loss {loss.item():.5f}, |h'| {out.norm().item():.3f}, "
          f"|grad h| {grads['h'].norm().item():.4f}, |grad w1| {grads['w1'].float().norm().item():.3f}; "
          f"forward {fwd:.0f} us, backward {bwd:.0f} us")
    print(f"decode of {R} tokens: |h'| {dec.norm().item():.3f}; {ll:.0f} us; 4-bit weights {dec4.norm().item():.3f}; "
          f"{ll4:.0f} us")
    layer.close()


if __name__ == "__main__":
    main()

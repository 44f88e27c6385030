"""Cases of the operators that turn a Mixture-of-Experts layer into a block of a
model: the combine that applies the routing weights to expert-major rows, with
its gradient; the norms before and after a block with its gate and residual
scale, with their gradients; and the experts' products on 4-bit weights (e2m1
codes, a power-of-two scale for every 32 channels), which serving uses.

A case is one call at one size.  Expert-major rows (``em``) are packed by
expert, each group starting at a multiple of ``align`` rows; low-latency rows
(``ll``) are ``cap`` slots for every expert.  Rows between groups hold what an
uninitialised buffer may hold, NaN among it; no operator reads them into a
result or writes them.
"""
import math

import torch

own = False

DEV = "cuda:0"
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of the eight codes; bit 3 is the sign


def listed():
    return [
        # a few tokens per rank, eight rows each, weights applied on the way back: latency is all there is
        dict(name="combine_few_tokens", op="combine", backward=False, R=8, T=16, E=64, k=8, H=2048, align=1, masked=0.0,
             skew=0.0),
        # the training batch of the benchmark (8 192 tokens, hidden 7168, top-8)
        dict(name="combine_train", op="combine", backward=False, R=8, T=8192, E=256, k=8, H=7168, align=128, masked=0.02,
             skew=0.5),
        # its gradient, rows in e4m3 as the experts' products take them
        dict(name="combine_grad_fp8", op="combine", backward=True, R=8, T=8192, E=256, k=8, H=7168, align=128,
             masked=0.02, skew=0.5, dtype="fp8"),
        # the gradient of a small odd batch in bf16, groups packed without alignment, masked entries
        dict(name="combine_grad_bf16", op="combine", backward=True, R=4, T=1036, E=60, k=4, H=2048, align=1, masked=0.1,
             skew=1.0, dtype="bf16"),
        # one token in a decode step: the norm behind the block, the residual sum, the norm before the next
        dict(name="norms_one_token", op="norms", backward=False, T=1, H=7168, residual="bf16", weights="bf16", post=True,
             pre=True, gate="vector", scale=0.5, masked=0.0),
        # prefill: a long prompt with the residual stream kept in fp32
        dict(name="norms_prefill", op="norms", backward=False, T=16384, H=7168, residual="fp32", weights="bf16",
             post=True, pre=True, gate="none", scale=1.0, masked=0.0),
        # gradients of a training batch: a gate for every channel
        dict(name="norms_grad_train", op="norms", backward=True, T=8192, H=7168, residual="bf16", weights="fp32",
             post=True, pre=True, gate="vector", scale=0.5, masked=0.0),
        # ... and of an odd, padded one whose gate comes with every token
        dict(name="norms_grad_gated", op="norms", backward=True, T=4099, H=2048, residual="fp32", weights="fp32",
             post=True, pre=True, gate="token", scale=1.0, masked=0.05),
        # decode, one token: eight experts' 4-bit weights are streamed for one row each
        dict(name="w4_one_token", op="w4", layout="ll", T=1, cap=128, E=32, k=8, K=7168, N=4096, skew=0.0),
        # decode, a batch: every expert's weights are streamed for a few tens of rows
        dict(name="w4_decode", op="w4", layout="ll", T=128, cap=128, E=32, k=8, K=2048, N=7168, skew=0.0),
        # first product of a decode step with the activation in its epilogue, odd batch
        dict(name="w4_swiglu_decode", op="w4_swiglu", layout="ll", T=77, cap=128, E=32, k=8, K=7168, F=2048, skew=0.0,
             weighted=False),
        # the same in a prefill: uneven experts, routing weights applied
        dict(name="w4_swiglu_prefill", op="w4_swiglu", layout="em", T=2048, align=128, E=32, k=8, K=7168, F=2048,
             skew=0.5, weighted=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["combine", "norms", "w4", "w4_swiglu"])
    if op == "combine":
        R = rng.choice([1, 2, 4, 8])
        E = R * rng.choice([4, 8, 15, 32])
        H = 128 * _log_int(rng, 1, 56)
        T = R * _log_int(rng, 1, 2048)
        k = rng.randint(1, 8)
        while k > E or T * k * H > 8192 * 8 * 7168:
            T, k = max(R, T // (2 * R) * R), min(k, E)
        c = dict(op=op, backward=rng.random() < 0.6, R=R, T=T, E=E, k=k, H=H, align=rng.choice([1, 4, 16, 128]),
                 masked=rng.choice([0.0, 0.02, 0.3]), skew=rng.choice([0.0, 0.5, 1.0]))
        if c["backward"]:
            c["dtype"] = rng.choice(["bf16", "fp8"])
        return c
    if op == "norms":
        T, H = _log_int(rng, 1, 16384), 8 * _log_int(rng, 8, 1024)
        return dict(op=op, backward=rng.random() < 0.6, T=min(T, 16384 * 7168 // H // 2), H=H,
                    residual=rng.choice(["bf16", "fp32"]), weights=rng.choice(["bf16", "fp32"]),
                    post=rng.random() < 0.7, pre=rng.random() < 0.8, gate=rng.choice(["none", "vector", "token"]),
                    scale=rng.choice([1.0, 0.5, 0.22]), masked=rng.choice([0.0, 0.0, 0.1]))
    E = rng.choice([4, 7, 16, 24, 32])
    c = dict(op=op, layout=rng.choice(["em", "ll"]), T=_log_int(rng, 1, 1024), E=E, k=rng.randint(1, min(8, E)),
             K=128 * _log_int(rng, 1, 56), skew=rng.choice([0.0, 0.5, 1.0]))
    if c["layout"] == "em":
        c["align"] = rng.choice([1, 4, 16, 128])
    else:
        c["T"] = min(c["T"], 512)
        c["cap"] = c["T"] + rng.randint(0, 64)
    if op == "w4":
        return dict(c, N=8 * _log_int(rng, 2, 512))
    return dict(c, F=128 * _log_int(rng, 1, 16), weighted=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _routing(case, g):
    """A seeded top-k routing; masked entries are -1."""
    E, T, k = case["E"], case["T"], case["k"]
    logits = torch.randn((T, E), generator=g, device=DEV)
    bias = torch.arange(1, E + 1, device=DEV, dtype=torch.float32).reciprocal() * 4.0 * case["skew"]
    logits += bias[torch.randperm(E, generator=g, device=DEV)]
    idx = logits.topk(k, dim=1).indices
    if case.get("masked"):
        idx[torch.rand((T, k), generator=g, device=DEV) < case["masked"]] = -1
    return idx


def _groups(case, idx):
    """Counts, group starts, and the row of every entry (-1: masked): the entries of an expert in (token, k) order."""
    E, T, k = case["E"], case["T"], case["k"]
    flat = idx.reshape(-1)
    live = flat >= 0
    count = torch.bincount(flat[live], minlength=E)
    if case.get("layout", "em") == "em":
        al = case["align"]
        end = torch.cumsum((count + al - 1) // al * al, 0)
        offset = torch.cat([end.new_zeros(1), end])
        start, rows = offset[:-1], T * k + E * (al - 1)
    else:
        start, rows, offset = torch.arange(E, device=DEV) * case["cap"], E * case["cap"], None
    order = torch.sort(torch.where(live, flat, torch.full_like(flat, E)), stable=True).indices[:int(live.sum())]
    expert = flat[order]
    before = torch.cat([count.new_zeros(1), torch.cumsum(count, 0)])
    slot = torch.arange(len(order), device=DEV) - before[expert]
    row_of = torch.full_like(flat, -1)
    row_of[order] = start[expert] + slot
    return dict(count=count.int(), offset=None if offset is None else offset.int(), rows=rows, most=int(count.max()),
                row_of=row_of.view(T, k), live_rows=start[expert] + slot, expert=expert, slot=slot)


def _quantize_rows(v):
    """e4m3 codes and one scale for every 128 channels of a row, as dispatch quantises."""
    v = v.float().unflatten(-1, (-1, 128))
    a = v.abs().amax(-1, keepdim=True).clamp_min(1e-4)
    return (v * (F8_MAX / a)).flatten(-2).to(F8), (a / F8_MAX).squeeze(-1)


def _row_buffer(case, rows, width, dtype):
    lead = (rows,) if case.get("layout", "em") == "em" else (case["E"], case["cap"])
    return torch.zeros(lead + (width,), dtype=dtype, device=DEV)


def _scale_buffer(case, rows, groups):
    if case.get("layout", "em") == "em":
        return torch.zeros((groups, (rows + 3) // 4 * 4), dtype=torch.float32, device=DEV)
    return torch.zeros((case["E"], case["cap"], groups), dtype=torch.float32, device=DEV)


def _fp8_rows(case, gr, g, width):
    """Dispatched rows: live rows of N(0, 1) in e4m3, NaN codes and scales elsewhere."""
    n = gr["live_rows"].numel()
    q, s = _quantize_rows(torch.randn((n, width), generator=g, device=DEV).bfloat16())
    data = torch.full((gr["rows"], width), 0x7F, dtype=torch.uint8, device=DEV)
    data[gr["live_rows"]] = q.view(torch.uint8)
    scales = torch.full((gr["rows"], width // 128), math.nan, device=DEV)
    scales[gr["live_rows"]] = s
    if case["layout"] == "em":
        out = torch.full_like(_scale_buffer(case, gr["rows"], width // 128), math.nan)
        out[:, :gr["rows"]] = scales.t()
        return data.view(F8), out
    return data.view(F8).view(case["E"], case["cap"], width), scales.view(case["E"], case["cap"], -1)


def _weights4(g, E, N, K):
    """Weights [E, N, K] of sigma 1/sqrt(K) in e2m1, two codes a byte (the even channel in the low bits), with an
    8-bit exponent for every 32 channels: the scales of 128 rows and 128 channels are 512 bytes together, byte
    16 (n % 32) + 4 (n % 128 / 32) + k % 128 / 32."""
    Nb, Kb = (N + 127) // 128, K // 128
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((E, Nb, Kb, 512), dtype=torch.uint8, device=DEV)
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    for e in range(E):
        w = (torch.randn((N, K), generator=g, device=DEV) / math.sqrt(K)).view(N, K // 32, 32)
        exponent = torch.frexp(w.abs().amax(2)).exponent - 3  # the largest magnitude lies in [4, 8) steps
        t = w * torch.exp2(-exponent.float())[..., None]
        c = torch.bucketize(t.abs(), border, out_int32=True).to(torch.uint8) | ((t < 0).to(torch.uint8) << 3)
        c = c.view(N, K // 2, 2)
        codes[e] = c[..., 0] | (c[..., 1] << 4)
        s = torch.full((Nb * 128, K // 32), 127, dtype=torch.uint8, device=DEV)
        s[:N] = (exponent + 127).to(torch.uint8)
        scales[e] = s.view(Nb, 4, 32, Kb, 4).permute(0, 3, 2, 1, 4).reshape(Nb, Kb, 512)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return dict(combine=_prepare_combine, norms=_prepare_norms, w4=_prepare_w4, w4_swiglu=_prepare_w4)[case["op"]](case, g)


def _prepare_combine(case, g):
    T, k, H = case["T"], case["k"], case["H"]
    idx = _routing(case, g)
    st = dict(case=case, idx=idx, **_groups(case, idx))
    w = torch.rand((T, k), generator=g, device=DEV) + 0.05
    st["weights"] = w / w.sum(1, keepdim=True)
    st["y"] = torch.full((st["rows"], H), math.nan, dtype=torch.bfloat16, device=DEV)
    st["y"][st["live_rows"]] = torch.randn((st["live_rows"].numel(), H), generator=g, device=DEV).bfloat16()
    if case["backward"]:
        st["dout"] = (torch.randn((T, H), generator=g, device=DEV) * 1e-2).bfloat16()
        f8 = case["dtype"] == "fp8"
        st["dy"] = _row_buffer(case, st["rows"], H, F8 if f8 else torch.bfloat16)
        st["dy_scales"] = _scale_buffer(case, st["rows"], H // 128) if f8 else None
        st["dweights"] = torch.zeros((T, k), device=DEV)
    else:
        st["out"] = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    if own:  # the handle holds the layout of the dispatch that the rows came from
        from combine_ep_get_03_gb300 import ep

        st["handle"] = ep.Handle(case["R"], case["E"], k, H, T // case["R"])
        x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
        st["handle"].em_layout_and_dispatch(idx, x, None, ep.EP_BF16, case["align"],
                                            torch.empty((st["rows"], H), dtype=torch.bfloat16, device=DEV))
    return st


def _prepare_norms(case, g):
    T, H = case["T"], case["H"]
    rdt = torch.float32 if case["residual"] == "fp32" else torch.bfloat16
    wdt = torch.float32 if case["weights"] == "fp32" else torch.bfloat16
    n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    st = dict(case=case, eps=1e-6, mask=None)
    if case["masked"]:
        st["mask"] = torch.rand(T, generator=g, device=DEV) >= case["masked"]
    st["post"] = (1 + 0.1 * n(H)).to(wdt) if case["post"] else None
    st["pre"] = (1 + 0.1 * n(H)).to(wdt) if case["pre"] else None
    st["gate"] = (dict(vector=(0.3 + 0.1 * n(H)).to(wdt)) if case["gate"] == "vector" else
                  dict(token=n(T, H).bfloat16()) if case["gate"] == "token" else dict(none=None))[case["gate"]]
    st["residual"] = (2 * n(T, H)).to(rdt)
    st["y"] = (0.7 * n(T, H)).bfloat16()
    if st["mask"] is not None:
        for t in (st["residual"], st["y"]):
            t[~st["mask"]] = math.nan  # a padding token's rows mean nothing
    if not case["backward"]:
        st["new_residual"] = torch.zeros((T, H), dtype=rdt, device=DEV)
        st["x"] = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV) if case["pre"] else None
        st["rstd"] = torch.zeros((2, T), device=DEV)
        return st
    # what the forward pass left
    out = _norms_plain(st)
    st["new_residual"], st["rstd"] = out["new_residual"], out["rstd"]
    st["dx"] = (n(T, H) * 1e-2).bfloat16() if case["pre"] else None
    st["dnew"] = (n(T, H) * 1e-2).to(rdt)
    if st["mask"] is not None:
        st["dnew"][~st["mask"]] = math.nan
    st["dresidual"] = torch.zeros((T, H), dtype=rdt, device=DEV)
    st["dy"] = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    zeros = lambda on: torch.zeros(H, device=DEV) if on else None  # noqa: E731
    st["dpost"], st["dpre"] = zeros(case["post"]), zeros(case["pre"])
    st["dgate"] = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV) if case["gate"] == "token" else zeros(case["gate"] == "vector")
    st["workspace"] = torch.zeros(256 * 3 * 4 * H, dtype=torch.uint8, device=DEV)
    return st


def _prepare_w4(case, g):
    st = dict(case=case, **_groups(case, _routing(case, g)))
    K = case["K"]
    st["x"], st["x_scales"] = _fp8_rows(case, st, g, K)
    if case["op"] == "w4":
        st["w"], st["w_scales"] = _weights4(g, case["E"], case["N"], K)
        st["out"] = _row_buffer(case, st["rows"], case["N"], torch.bfloat16)
        return st
    F = case["F"]
    st["w"], st["w_scales"] = _weights4(g, case["E"], 2 * F, K)
    st["row_weights"] = None
    if case["weighted"]:
        st["row_weights"] = torch.full((st["rows"],), math.nan, device=DEV)
        st["row_weights"][st["live_rows"]] = torch.rand(st["live_rows"].numel(), generator=g, device=DEV) * 0.5
    st["act"], st["act_scales"] = _row_buffer(case, st["rows"], F, F8), _scale_buffer(case, st["rows"], F // 128)
    return st


# ------------------------------------------------------------------ the operators

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    from combine_ep_get_03_gb300 import ep

    c = st["case"]
    if c["op"] == "combine":
        h = st["handle"]
        if not c["backward"]:
            h.em_combine_weighted(st["y"], st["weights"], st["out"])
            return st["out"]
        h.em_combine_weighted_backward(st["dout"], st["y"], st["weights"],
                                       ep.EP_FP8_E4M3 if c["dtype"] == "fp8" else ep.EP_BF16, st["dy"], st["dy_scales"],
                                       grad_topk_weights=st["dweights"])
        out = dict(dy=st["dy"], dweights=st["dweights"])
        return dict(out, dy_scales=st["dy_scales"]) if c["dtype"] == "fp8" else out
    if c["op"] == "norms":
        how = dict(post_weight=st["post"], pre_weight=st["pre"], gate=st["gate"], eps=st["eps"],
                   residual_scale=c["scale"], token_mask=st["mask"])
        if not c["backward"]:
            ep.ep_block_norm_forward(st["residual"], st["y"], st["new_residual"], st["x"], rstd=st["rstd"], **how)
            out = dict(new_residual=st["new_residual"], rstd=st["rstd"])
            return dict(out, x=st["x"]) if c["pre"] else out
        ep.ep_block_norm_backward(st["new_residual"], st["y"], st["rstd"], st["dnew"], st["dx"], st["dresidual"], st["dy"],
                                  st["workspace"], grad_post_weight=st["dpost"], grad_pre_weight=st["dpre"],
                                  grad_gate=st["dgate"], **{k: v for k, v in how.items() if k != "eps"})
        return {k: st[k] for k in ("dresidual", "dy", "dpost", "dpre", "dgate") if st[k] is not None}
    if c["op"] == "w4":
        ep.ep_grouped_matmul_w4(st["x"], st["x_scales"], st["w"], st["w_scales"], st["out"], st["count"],
                                group_offset=st["offset"])
        return st["out"]
    ep.ep_grouped_matmul_w4_swiglu(st["x"], st["x_scales"], st["w"], st["w_scales"], st["act"], st["act_scales"],
                                   st["count"], group_offset=st["offset"], row_weights=st["row_weights"])
    return dict(act=st["act"], act_scales=st["act_scales"])


# -- plain forms

def _run_plain(st):
    c = st["case"]
    if c["op"] == "combine":
        return _combine_grad_plain(st) if c["backward"] else _combine_plain(st)
    if c["op"] == "norms":
        return _norms_grad_plain(st) if c["backward"] else _norms_plain(st)
    return _w4_plain(st)


def _combine_plain(st):
    live = (st["row_of"] >= 0)[..., None]
    rows = st["y"][st["row_of"].clamp_min(0).reshape(-1)].view(st["row_of"].shape + (-1,))
    v = torch.where(live, rows.float() * st["weights"][..., None], torch.zeros((), device=DEV))
    return v.sum(1).bfloat16()


def _combine_grad_plain(st):
    c = st["case"]
    T, k = st["row_of"].shape
    entry = (st["row_of"].reshape(-1) >= 0).nonzero().squeeze(1)
    row = st["row_of"].reshape(-1)[entry]
    g = st["dout"].float()[entry // k]
    v = g * st["weights"].reshape(-1)[entry, None]
    dweights = torch.zeros(T * k, device=DEV)
    dweights[entry] = (g * st["y"][row].float()).sum(1)
    dy = torch.zeros_like(st["dy"])
    if c["dtype"] == "bf16":
        dy[row] = v.bfloat16()
        return dict(dy=dy, dweights=dweights.view(T, k))
    q, s = _quantize_rows(v)
    dy.view(torch.uint8)[row] = q.view(torch.uint8)
    scales = torch.zeros_like(st["dy_scales"])
    scales.t()[row] = s
    return dict(dy=dy, dy_scales=scales, dweights=dweights.view(T, k))


def _norms_plain(st):
    """h = residual + scale gate norm(y) post and x = norm(h) pre, norm(v) = v / sqrt(mean(v^2) + eps); 0 on padding."""
    c = st["case"]
    on = None if st["mask"] is None else st["mask"][:, None]
    clean = lambda t: t.float() if on is None else torch.where(on, t.float(), torch.zeros((), device=DEV))  # noqa: E731
    y, h = clean(st["y"]), clean(st["residual"])
    rstd = torch.zeros((2, c["T"]), device=DEV)
    if c["post"]:
        r = torch.rsqrt((y * y).mean(1) + st["eps"])
        rstd[0] = r if on is None else r * on[:, 0]
        y = y * r[:, None] * st["post"].float()
    if st["gate"] is not None:
        y = y * st["gate"].float()
    h = h + c["scale"] * clean(y)
    out = dict(new_residual=h.to(st["residual"].dtype), rstd=rstd)
    if c["pre"]:
        r = torch.rsqrt((h * h).mean(1) + st["eps"])
        rstd[1] = r if on is None else r * on[:, 0]
        out["x"] = (h * r[:, None] * st["pre"].float()).bfloat16()
    return out


def _norms_grad_plain(st):
    c = st["case"]
    on = None if st["mask"] is None else st["mask"][:, None]
    clean = lambda t: t.float() if on is None else torch.where(on, t.float(), torch.zeros((), device=DEV))  # noqa: E731
    h, y, gh = clean(st["new_residual"]), clean(st["y"]), clean(st["dnew"])
    out = dict()
    if c["pre"]:
        r, gx = st["rstd"][1][:, None], clean(st["dx"])
        hn, a = h * r, gx * st["pre"].float()
        out["dpre"] = (gx * hn).sum(0)
        gh = gh + r * (a - hn * (a * hn).mean(1, keepdim=True))
    out["dresidual"] = gh.to(st["residual"].dtype)
    gn = c["scale"] * gh
    r = st["rstd"][0][:, None] if c["post"] else torch.ones((), device=DEV)
    yn = y * r
    n = yn * st["post"].float() if c["post"] else yn
    if c["gate"] == "token":
        out["dgate"] = (gn * n).bfloat16()
    elif c["gate"] == "vector":
        out["dgate"] = (gn * n).sum(0)
    if st["gate"] is not None:
        gn = gn * st["gate"].float()
    if c["post"]:
        out["dpost"] = (gn * yn).sum(0)
        b = gn * st["post"].float()
        gn = r * (b - yn * (b * yn).mean(1, keepdim=True))
    out["dy"] = gn.bfloat16()
    return out


def _rows_to_table(st, v):
    """Live rows in an [expert][slot] table, zeros elsewhere."""
    t = v.new_zeros((st["case"]["E"], st["most"], v.shape[1]))
    t[st["expert"], st["slot"]] = v
    return t


def _w4_plain(st):
    c = st["case"]
    E, K, rows = c["E"], c["K"], st["live_rows"]
    q = st["x"].view(torch.uint8).view(st["rows"], K)[rows].view(F8).float()
    s = st["x_scales"].t()[rows] if c["layout"] == "em" else st["x_scales"].view(st["rows"], -1)[rows]
    x = (q.unflatten(-1, (-1, 128)) * s[..., None]).flatten(-2)
    N = st["w"].shape[1]
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    w = torch.stack((value[(st["w"] & 15).int()], value[(st["w"] >> 4).int()]), -1).view(E, N, K // 32, 32)
    blocks = st["w_scales"].view(E, (N + 127) // 128, K // 128, 32, 4, 4).permute(0, 1, 4, 3, 2, 5)
    w *= (blocks.reshape(E, -1, K // 32)[:, :N].int() << 23).view(torch.float32)[..., None]  # 2^(b - 127)
    y = torch.bmm(_rows_to_table(st, x), w.view(E, N, K).transpose(1, 2))[st["expert"], st["slot"]]
    if c["op"] == "w4":
        out = torch.zeros_like(st["out"])
        out.view(-1, N)[rows] = y.bfloat16()
        return out
    gate, up = y.chunk(2, 1)
    a = gate / (1 + torch.exp(-gate)) * up
    if c["weighted"]:
        a = a * st["row_weights"][rows, None]
    q, s = _quantize_rows(a)
    act, scales = torch.zeros_like(st["act"]), torch.zeros_like(st["act_scales"])
    act.view(torch.uint8).view(-1, c["F"])[rows] = q.view(torch.uint8)
    (scales.t() if c["layout"] == "em" else scales.view(st["rows"], -1))[rows] = s
    return dict(act=act, act_scales=scales)


# ------------------------------------------------------------------ work and exact values

def work(case):
    op, T = case["op"], case["T"]
    if op == "combine":
        H, entries = case["H"], T * case["k"] * (1 - case["masked"])
        b = entries * 2 * H + T * case["k"] * 12 + T * 2 * H
        if not case["backward"]:
            return dict(bytes=b, flops=2 * entries * H)
        return dict(bytes=b + entries * (2 * H if case["dtype"] == "bf16" else H + H // 32) + T * case["k"] * 4,
                    flops=3 * entries * H)
    if op == "norms":
        n, r = T * (1 - case["masked"]) * case["H"], 4 if case["residual"] == "fp32" else 2
        each = 2 * r + 2 + (2 if case["gate"] == "token" else 0) + (2 if case["pre"] else 0)
        if case["backward"]:  # the new residual is read, the output's gradient written
            each += 2 + (r if case["pre"] else 0) + (2 if case["gate"] == "token" else 0)
            if case["gate"] == "none" and not case["post"]:
                each -= 2  # nothing needs y
        return dict(bytes=n * each + 8 * T, flops=n * (25 if case["backward"] else 9))
    rows, E = T * case["k"], case["E"]
    live = E * (1 - (1 - case["k"] / E) ** T)  # experts that get a row
    K, N = case["K"], case["N"] if op == "w4" else 2 * case["F"]
    b = rows * (K + K // 32) + live * N * (K // 2 + K // 32) + 8 * E
    b += rows * 2 * N if op == "w4" else rows * (case["F"] + case["F"] // 32) + (4 * rows if case["weighted"] else 0)
    return dict(bytes=b, flops=2 * rows * N * K)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "combine":
        return _combine_exact(st)
    if case["op"] == "norms":
        return _norms_grad_exact(st) if case["backward"] else _norms_exact(st)
    return _w4_exact(st)


def _combine_exact(st):
    """Entry by entry of a token: column j of the routing at a time."""
    c = st["case"]
    T, k = st["row_of"].shape
    if not c["backward"]:
        out = torch.zeros((T, c["H"]), dtype=torch.float64, device=DEV)
        for j in range(k):
            on = (st["row_of"][:, j] >= 0).nonzero().squeeze(1)
            out[on] += st["weights"][on, j, None].double() * st["y"][st["row_of"][on, j]].double()
        return out
    dy = torch.zeros(st["dy"].shape, dtype=torch.float64, device=DEV)
    scales = None if st["dy_scales"] is None else torch.zeros(st["dy_scales"].shape, dtype=torch.float64, device=DEV)
    dw = torch.zeros((T, k), dtype=torch.float64, device=DEV)
    for j in range(k):
        on = (st["row_of"][:, j] >= 0).nonzero().squeeze(1)
        row, g = st["row_of"][on, j], st["dout"][on].double()
        dw[on, j] = torch.einsum("th,th->t", g, st["y"][row].double())
        g = g * st["weights"][on, j, None].double()
        if scales is not None:
            a = g.reshape(len(on), -1, 128).abs().amax(2).clamp_min(1e-4)
            scales[:, row] = (a / 448.0).t()
            g = g * (448.0 / a).repeat_interleave(128, 1)
        dy[row] = g
    out = dict(dy=dy, dweights=dw)
    return out if scales is None else dict(out, dy_scales=scales)


def _norms_function(st, residual, y, gate, post, pre):
    """One operator as a function of 64-bit tensors of the unmasked rows."""
    n = y if post is None else y / (y.pow(2).mean(1, keepdim=True) + st["eps"]).sqrt() * post
    h = residual + st["case"]["scale"] * (n if gate is None else n * gate)
    return h, None if pre is None else h / (h.pow(2).mean(1, keepdim=True) + st["eps"]).sqrt() * pre


def _unmasked(st):
    return torch.arange(st["case"]["T"], device=DEV) if st["mask"] is None else st["mask"].nonzero().squeeze(1)


def _d(t, rows=None):
    return None if t is None else (t if rows is None or t.dim() == 1 else t[rows]).double()


def _norms_exact(st):
    on = _unmasked(st)
    r, y = _d(st["residual"], on), _d(st["y"], on)
    h, x = _norms_function(st, r, y, _d(st["gate"], on), _d(st["post"]), _d(st["pre"]))
    full = lambda t: torch.zeros((st["case"]["T"],) + t.shape[1:], dtype=torch.float64, device=DEV).index_copy_(0, on, t)  # noqa: E731
    one = lambda t, have: full(t.pow(2).mean(1).add(st["eps"]).pow(-0.5)) if have else torch.zeros(st["case"]["T"], dtype=torch.float64, device=DEV)  # noqa: E731
    out = dict(new_residual=full(h), rstd=torch.stack((one(y, st["post"] is not None), one(h, st["pre"] is not None))))
    return out if x is None else dict(out, x=full(x))


def _norms_grad_exact(st):
    """From the definition's Jacobians: a norm's output v r w has d(v)/d(v') = r (1 - v v' r^2 / H) w, where r is what
    the forward pass left."""
    c, on = st["case"], _unmasked(st)
    H = c["H"]
    full = lambda t: torch.zeros((c["T"], H), dtype=torch.float64, device=DEV).index_copy_(0, on, t)  # noqa: E731
    d, h, y = _d(st["dnew"], on), _d(st["new_residual"], on), _d(st["y"], on)
    out = dict()
    if c["pre"]:
        r, gx, w = _d(st["rstd"][1])[on, None], _d(st["dx"], on), _d(st["pre"])
        out["dpre"] = torch.einsum("th,th->h", gx, h * r)
        d = d + r * gx * w - r.pow(3) / H * h * torch.einsum("th,th,h->t", gx, h, w)[:, None]
    out["dresidual"] = full(d)
    gate, post = _d(st["gate"], on), _d(st["post"])
    up = d * c["scale"]
    r = _d(st["rstd"][0])[on, None] if c["post"] else 1.0
    n = y * r * (1.0 if post is None else post)
    if c["gate"] == "token":
        out["dgate"] = full(up * n)
    elif c["gate"] == "vector":
        out["dgate"] = torch.einsum("th,th->h", up, n)
    if gate is not None:
        up = up * gate
    if c["post"]:
        out["dpost"] = torch.einsum("th,th->h", up, y * r)
        up = r * up * post - r.pow(3) / H * y * torch.einsum("th,th,h->t", up, y, post)[:, None]
    out["dy"] = full(up)
    return out


def _w4_exact(st):
    """Expert by expert, the weights from their bits."""
    c = st["case"]
    K, rows = c["K"], st["rows"]
    start = st["offset"].tolist() if c["layout"] == "em" else [e * c["cap"] for e in range(c["E"])]
    N = st["w"].shape[1]
    n = torch.arange(N, device=DEV)[:, None]
    k = torch.arange(K, device=DEV)[None, :]
    y = torch.zeros((rows, N), dtype=torch.float64, device=DEV)
    live = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for e, many in enumerate(st["count"].tolist()):
        if not many:
            continue
        code = (st["w"][e][n, k // 2] >> (4 * (k % 2)).to(torch.uint8)).int() & 15
        m, ex = code & 1, (code >> 1) & 3
        v = torch.where(ex > 0, (1 + m.double() / 2) * torch.exp2(ex.double() - 1), m.double() / 2)
        at = (n % 32) * 16 + n % 128 // 32 * 4 + k % 128 // 32
        b = st["w_scales"][e][n // 128, k // 128, at].int() - 127
        w = torch.where(code > 7, -v, v) * torch.exp2(b.double())
        own_rows = slice(start[e], start[e] + many)
        live[own_rows] = True
        x = st["x"].view(rows, K)[own_rows].double()
        s = st["x_scales"][:, own_rows].t() if c["layout"] == "em" else st["x_scales"].view(rows, -1)[own_rows]
        y[own_rows] = (x * s.double().repeat_interleave(128, 1)) @ w.t()
    if c["op"] == "w4":
        return y.view(st["out"].shape)
    F = c["F"]
    a = y[:, :F] * torch.sigmoid(y[:, :F]) * y[:, F:]
    if c["weighted"]:
        a = a * torch.where(live, st["row_weights"], torch.zeros((), device=DEV))[:, None].double()
    most = a.view(rows, -1, 128).abs().amax(2).clamp_min(1e-4)
    act = a * (448.0 / most).repeat_interleave(128, 1)
    scales = torch.zeros(st["act_scales"].shape, dtype=torch.float64, device=DEV)
    if c["layout"] == "em":
        scales[:, :rows] = torch.where(live, (most / 448.0).t(), 0.0)
    else:
        scales.view(rows, -1)[:] = torch.where(live[:, None], most / 448.0, 0.0)
    return dict(act=act.view(st["act"].shape), act_scales=scales)

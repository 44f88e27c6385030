"""Cases of the operators around dispatch and combine: the gate with its balance
loss, the experts' FP8 products, the SwiGLU between them with its activations
kept in 8 bits, and the products' weight gradient.

A case is one call (or a forward and its backward) at one size.  Group layouts
are those that dispatch leaves: expert-major rows (``em``: groups packed, each
starting at a multiple of ``align`` rows, scales group-major) or low-latency
slots (``ll``: ``cap`` rows for every expert, scales row-major).  Rows between
groups hold what an uninitialised buffer may hold, NaN codes among it; no
operator reads them into a result or writes them.
"""
import math

import torch

own = False

DEV = "cuda:0"
F8 = torch.float8_e4m3fn
F8_MAX = 448.0


def listed():
    return [
        # one token's routing in a decode step: latency is all there is
        dict(name="gate_one_token", op="gate", T=1, E=256, k=8, groups=1, keep=1, score="softmax", dtype="fp32",
             masked=0.0, backward=False),
        # a training micro-batch of the benchmark's group-limited, skewed gate, some padding tokens, both directions
        dict(name="gate_group_limited", op="gate", T=8192, E=256, k=8, groups=8, keep=4, score="sigmoid", dtype="fp32",
             masked=0.02, backward=True),
        # the large-EP training batch, router logits left in bf16 (ties are common), both directions
        dict(name="gate_large_bf16", op="gate", T=32768, E=256, k=8, groups=1, keep=1, score="softmax", dtype="bf16",
             masked=0.0, backward=True),
        # decode, one token: eight experts' weights are streamed for one row each
        dict(name="product_one_token", op="product", layout="ll", T=1, cap=128, E=32, k=8, K=7168, N=4096, skew=0.0),
        # decode, a batch: every expert's weights are streamed for a few tens of rows
        dict(name="product_decode", op="product", layout="ll", T=128, cap=128, E=32, k=8, K=2048, N=7168, skew=0.0),
        # prefill: a rank's experts, about a thousand rows each, uneven
        dict(name="product_prefill", op="product", layout="em", T=4096, align=128, E=32, k=8, K=7168, N=4096, skew=1.0),
        # first product of a decode step with the activation in its epilogue, odd batch
        dict(name="swiglu_decode", op="swiglu", layout="ll", T=77, cap=128, E=32, k=8, K=7168, F=2048, skew=0.0,
             weighted=False, keep8=False),
        # first product of a training step: routing weights applied, the pre-activations kept in 8 bits
        dict(name="swiglu_train", op="swiglu", layout="em", T=1024, align=128, E=32, k=8, K=7168, F=2048, skew=0.5,
             weighted=True, keep8=True),
        # the activation's backward from the 8-bit checkpoint: a small ragged batch
        dict(name="swiglu_backward_small", op="swiglu_backward", layout="em", T=130, align=16, E=16, k=2, F=512,
             skew=1.0, weighted=True),
        # ... and a training batch
        dict(name="swiglu_backward_train", op="swiglu_backward", layout="em", T=4096, align=128, E=32, k=8, F=2048,
             skew=0.5, weighted=True),
        # weight gradient of small experts, groups packed without alignment
        dict(name="weight_grad_small", op="weight_grad", layout="em", T=500, align=1, E=16, k=2, K=512, N=1024, skew=1.0),
        # weight gradient of the training step's first product
        dict(name="weight_grad_train", op="weight_grad", layout="em", T=2048, align=128, E=16, k=8, K=7168, N=2048,
             skew=0.5),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_groups(rng):
    E = rng.choice([4, 7, 16, 24, 32])
    c = dict(layout=rng.choice(["em", "ll"]), T=_log_int(rng, 1, 2048), E=E, k=rng.randint(1, min(8, E)),
             skew=rng.choice([0.0, 0.5, 1.0]))
    if c["layout"] == "em":
        c["align"] = rng.choice([1, 4, 16, 128])
    else:
        c["T"] = min(c["T"], 512)
        c["cap"] = c["T"] + rng.randint(0, 64)
    return c


def draw(rng):
    op = rng.choice(["gate", "product", "swiglu", "swiglu_backward", "weight_grad"])
    if op == "gate":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256, 384])
        k = rng.randint(1, 8)
        groups = rng.choice([g for g in (1, 4, 8) if E % g == 0])
        keep = rng.randint(1, groups)
        while keep * (E // groups) < k:
            keep += 1
        return dict(op=op, T=_log_int(rng, 1, 32768), E=E, k=k, groups=groups, keep=keep,
                    score=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["fp32", "bf16"]),
                    masked=rng.choice([0.0, 0.1, 0.5]), backward=rng.random() < 0.7)
    c = _draw_groups(rng)
    c["op"] = op
    K, F = 128 * _log_int(rng, 1, 56), 128 * _log_int(rng, 1, 16)
    if op == "product":
        return dict(c, K=K, N=8 * _log_int(rng, 2, 512))
    if op == "swiglu":
        return dict(c, K=K, F=F, weighted=rng.random() < 0.5, keep8=rng.random() < 0.5)
    if op == "swiglu_backward":
        return dict(c, F=F, weighted=rng.random() < 0.5)
    return dict(c, K=K, N=128 * _log_int(rng, 1, 16))


# ------------------------------------------------------------------ inputs

def _quantize_rows(x):
    """e4m3 codes and one scale for every 128 channels of a row (bf16 in, as dispatch quantises)."""
    v = x.float().unflatten(-1, (-1, 128))
    a = v.abs().amax(-1, keepdim=True).clamp_min(1e-4)
    return (v * (F8_MAX / a)).flatten(-2).to(F8), (a / F8_MAX).squeeze(-1)


def _weights(g, E, N, K):
    """e4m3 weights [E, N, K] of sigma 1/sqrt(K) with one scale for every 128 x 128 block."""
    Nb, Kb = (N + 127) // 128, K // 128
    q = torch.empty((E, N, K), dtype=F8, device=DEV)
    s = torch.empty((E, Nb, Kb), dtype=torch.float32, device=DEV)
    for e in range(E):
        w = torch.randn((Nb * 128, K), generator=g, device=DEV) / math.sqrt(K)
        w[N:] = 0
        b = w.view(Nb, 128, Kb, 128)
        a = b.abs().amax((1, 3)).clamp_min(1e-4)
        s[e] = a / F8_MAX
        q[e] = (b * (F8_MAX / a)[:, None, :, None]).view(Nb * 128, K)[:N].to(F8)
    return q, s


def _groups(case, g):
    """A seeded top-k routing and the rows that each expert receives."""
    E, T, k = case["E"], case["T"], case["k"]
    logits = torch.randn((T, E), generator=g, device=DEV)
    bias = torch.arange(1, E + 1, device=DEV, dtype=torch.float32).reciprocal() * 4.0 * case["skew"]
    logits += bias[torch.randperm(E, generator=g, device=DEV)]
    idx = logits.topk(k, dim=1).indices
    count = torch.bincount(idx.reshape(-1), minlength=E)
    if case["layout"] == "em":
        al = case["align"]
        end = torch.cumsum((count + al - 1) // al * al, 0)
        offset = torch.cat([end.new_zeros(1), end])
        rows = T * k + E * (al - 1)
        start = offset[:-1]
    else:
        rows, offset = E * case["cap"], None
        start = torch.arange(E, device=DEV) * case["cap"]
    # the rows that hold an entry, and their place in a [group][slot] table
    most = int(count.max())
    slot = torch.arange(most, device=DEV)
    live = (slot[None, :] < count[:, None]).reshape(-1).nonzero().squeeze(1)
    table = (start[:, None] + slot[None, :]).reshape(-1)
    return dict(count=count.int(), offset=None if offset is None else offset.int(), rows=rows, most=most,
                live_rows=table[live], live_pos=live)


def _row_buffer(case, gr, width, dtype):
    lead = (gr["rows"],) if case["layout"] == "em" else (case["E"], case["cap"])
    return torch.zeros(lead + (width,), dtype=dtype, device=DEV)


def _scale_buffer(case, gr, groups):
    if case["layout"] == "em":
        return torch.zeros((groups, (gr["rows"] + 3) // 4 * 4), dtype=torch.float32, device=DEV)
    return torch.zeros((case["E"], case["cap"], groups), dtype=torch.float32, device=DEV)


def _fp8_rows(case, gr, g, width, sigma=1.0):
    """Dispatched rows: live rows of N(0, sigma) in e4m3, NaN codes and scales elsewhere."""
    n = gr["live_rows"].numel()
    q, s = _quantize_rows((torch.randn((n, width), generator=g, device=DEV) * sigma).bfloat16())
    data = torch.full((gr["rows"], width), 0x7F, dtype=torch.uint8, device=DEV)
    data[gr["live_rows"]] = q.view(torch.uint8)
    scales = torch.full((gr["rows"], width // 128), math.nan, device=DEV)
    scales[gr["live_rows"]] = s
    if case["layout"] == "em":
        out = torch.full_like(_scale_buffer(case, gr, width // 128), math.nan)
        out[:, :gr["rows"]] = scales.t()
        return data.view(F8), out
    return data.view(F8).view(case["E"], case["cap"], width), scales.view(case["E"], case["cap"], -1)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, st = case["op"], dict(case=case)
    if op == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        logits = torch.randn((T, E), generator=g, device=DEV)
        logits += torch.linspace(2.0, 0.0, E, device=DEV)[torch.randperm(E, generator=g, device=DEV)]
        st["mask"] = torch.rand(T, generator=g, device=DEV) >= case["masked"] if case["masked"] else None
        if st["mask"] is not None:
            logits[~st["mask"]] = math.nan  # a padding token's logits mean nothing
        st.update(logits=logits.to(dt), dweights=torch.randn((T, k), generator=g, device=DEV) * 1e-2,
                  dloss=torch.ones(1, device=DEV), coef=1e-2,
                  idx=torch.empty((T, k), dtype=torch.int64, device=DEV), weights=torch.empty((T, k), device=DEV),
                  count=torch.empty(E + 1, dtype=torch.int32, device=DEV), prob=torch.empty(E, device=DEV),
                  loss=torch.empty(1, device=DEV), dlogits=torch.empty((T, E), dtype=dt, device=DEV),
                  workspace=torch.zeros(2 << 20, dtype=torch.uint8, device=DEV))
        return st
    gr = _groups(case, g)
    st.update(gr)
    if op in ("product", "swiglu"):
        st["x"], st["x_scales"] = _fp8_rows(case, gr, g, case["K"])
        st["w"], st["w_scales"] = _weights(g, case["E"], case["N"] if op == "product" else 2 * case["F"], case["K"])
    if op in ("swiglu", "swiglu_backward"):
        st["row_weights"] = None
        if case["weighted"]:
            st["row_weights"] = torch.full((gr["rows"],), math.nan, device=DEV)
            st["row_weights"][gr["live_rows"]] = torch.rand(gr["live_rows"].numel(), generator=g, device=DEV) * 0.5
    if op == "product":
        st["out"] = _row_buffer(case, gr, case["N"], torch.bfloat16)
    elif op == "swiglu":
        F = case["F"]
        st["act"], st["act_scales"] = _row_buffer(case, gr, F, F8), _scale_buffer(case, gr, F // 128)
        st["pre"] = _row_buffer(case, gr, 2 * F, F8) if case["keep8"] else None
        st["pre_scales"] = _scale_buffer(case, gr, 2 * F // 128) if case["keep8"] else None
    elif op == "swiglu_backward":
        F = case["F"]
        st["pre"], st["pre_scales"] = _fp8_rows(case, gr, g, 2 * F)
        da = torch.full((gr["rows"], F), math.nan, dtype=torch.bfloat16, device=DEV)
        da[gr["live_rows"]] = (torch.randn((gr["live_rows"].numel(), F), generator=g, device=DEV) * 1e-2).bfloat16()
        st["dact"] = da if case["layout"] == "em" else da.view(case["E"], case["cap"], F)
        st["dpre"], st["dpre_scales"] = _row_buffer(case, gr, 2 * F, F8), _scale_buffer(case, gr, 2 * F // 128)
        st["drow_weights"] = torch.zeros(gr["rows"], device=DEV) if case["weighted"] else None
    elif op == "weight_grad":
        st["x"], st["x_scales"] = _fp8_rows(case, gr, g, case["K"])
        st["dy"], st["dy_scales"] = _fp8_rows(case, gr, g, case["N"], 1e-2)
        st["dw"] = torch.zeros((case["E"], case["N"], case["K"]), dtype=torch.bfloat16, device=DEV)
    return st


# ------------------------------------------------------------------ the operators

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    from combine_ep_get_03_gb300 import ep

    c = st["case"]
    op = c["op"]
    if op == "gate":
        score = ep.EP_GATE_SOFTMAX if c["score"] == "softmax" else ep.EP_GATE_SIGMOID
        ep.ep_gate_forward(st["logits"], st["idx"], st["weights"], st["count"], st["prob"], st["loss"],
                           st["workspace"], score=score, num_groups=c["groups"], topk_groups=c["keep"],
                           loss_coef=st["coef"], token_mask=st["mask"])
        out = dict(idx=st["idx"], weights=st["weights"], count=st["count"], prob=st["prob"], loss=st["loss"])
        if c["backward"]:
            ep.ep_gate_backward(st["logits"], st["idx"], st["count"], st["dweights"], st["dloss"], st["dlogits"],
                                score=score, loss_coef=st["coef"], token_mask=st["mask"])
            out["dlogits"] = st["dlogits"]
        return out
    if op == "product":
        ep.ep_grouped_matmul(st["x"], st["x_scales"], st["w"], st["w_scales"], st["out"], st["count"],
                             group_offset=st["offset"])
        return st["out"]
    if op == "swiglu":
        ep.ep_grouped_matmul_swiglu(st["x"], st["x_scales"], st["w"], st["w_scales"], st["act"], st["act_scales"],
                                    st["count"], group_offset=st["offset"], row_weights=st["row_weights"],
                                    pre=st["pre"], pre_scales=st["pre_scales"])
        out = dict(act=st["act"], act_scales=st["act_scales"])
        if c["keep8"]:
            out.update(pre=st["pre"], pre_scales=st["pre_scales"])
        return out
    if op == "swiglu_backward":
        ep.ep_grouped_swiglu_backward(st["dact"], st["pre"], st["pre_scales"], st["dpre"], st["dpre_scales"],
                                      st["count"], group_offset=st["offset"], row_weights=st["row_weights"],
                                      grad_row_weights=st["drow_weights"])
        out = dict(dpre=st["dpre"], dpre_scales=st["dpre_scales"])
        if c["weighted"]:
            out["drow_weights"] = st["drow_weights"]
        return out
    ep.ep_grouped_weight_grad(st["dy"], st["dy_scales"], st["x"], st["x_scales"], st["dw"], st["count"],
                              group_offset=st["offset"])
    return st["dw"]


# -- plain forms

def _live(st, data, scales):
    """The live rows of an e4m3 row buffer as 32-bit values."""
    q = data.view(torch.uint8).view(st["rows"], -1)[st["live_rows"]].view(F8).float()
    s = scales.t()[st["live_rows"]] if st["case"]["layout"] == "em" else scales.view(st["rows"], -1)[st["live_rows"]]
    return (q.unflatten(-1, (-1, 128)) * s[..., None]).flatten(-2)


def _padded(st, v):
    """Live rows in a [group][slot] table, zeros elsewhere."""
    t = v.new_zeros((st["case"]["E"] * st["most"], v.shape[1]))
    t[st["live_pos"]] = v
    return t.view(st["case"]["E"], st["most"], -1)


def _dequantized_weights(st):
    w = st["w"].float()
    s = st["w_scales"].repeat_interleave(128, 1)[:, :w.shape[1]]
    return (w.unflatten(-1, (-1, 128)) * s[..., None]).flatten(-2)


def _store(like, rows, v):
    o = torch.zeros_like(like)
    if like.dtype == F8:
        o.view(torch.uint8).view(-1, like.shape[-1])[rows] = v.view(torch.uint8)
    else:
        o.view(-1, like.shape[-1])[rows] = v
    return o


def _store_scales(st, like, v):
    o = torch.zeros_like(like)
    if st["case"]["layout"] == "em":
        o.t()[st["live_rows"]] = v
    else:
        o.view(st["rows"], -1)[st["live_rows"]] = v
    return o


def _product(st):
    y = torch.bmm(_padded(st, _live(st, st["x"], st["x_scales"])), _dequantized_weights(st).transpose(1, 2))
    return y.view(-1, y.shape[-1])[st["live_pos"]]


def _run_plain(st):
    c = st["case"]
    op = c["op"]
    if op == "gate":
        return _gate_plain(st)
    if op == "product":
        return _store(st["out"], st["live_rows"], _product(st).bfloat16())
    if op == "swiglu":
        y = _product(st)
        gate, up = y.chunk(2, 1)
        a = gate / (1 + torch.exp(-gate)) * up
        if c["weighted"]:
            a = a * st["row_weights"][st["live_rows"], None]
        q, s = _quantize_rows(a)
        out = dict(act=_store(st["act"], st["live_rows"], q), act_scales=_store_scales(st, st["act_scales"], s))
        if c["keep8"]:
            q, s = _quantize_rows(y)
            out.update(pre=_store(st["pre"], st["live_rows"], q), pre_scales=_store_scales(st, st["pre_scales"], s))
        return out
    if op == "swiglu_backward":
        gate, up = _live(st, st["pre"], st["pre_scales"]).chunk(2, 1)
        da = st["dact"].view(st["rows"], -1)[st["live_rows"]].float()
        sig = 1 / (1 + torch.exp(-gate))
        dw = da * (st["row_weights"][st["live_rows"], None] if c["weighted"] else 1.0)
        d = torch.cat([dw * up * sig * (1 + gate * (1 - sig)), dw * gate * sig], 1)
        q, s = _quantize_rows(d)
        out = dict(dpre=_store(st["dpre"], st["live_rows"], q), dpre_scales=_store_scales(st, st["dpre_scales"], s))
        if c["weighted"]:
            out["drow_weights"] = torch.zeros_like(st["drow_weights"])
            out["drow_weights"][st["live_rows"]] = (da * gate * sig * up).sum(1)
        return out
    dy, x = _padded(st, _live(st, st["dy"], st["dy_scales"])), _padded(st, _live(st, st["x"], st["x_scales"]))
    return torch.bmm(dy.transpose(1, 2), x).bfloat16()


def _gate_plain(st):
    c = st["case"]
    T, E, k, coef = c["T"], c["E"], c["k"], st["coef"]
    mask = st["mask"]
    l = st["logits"].float()
    if mask is not None:
        l = torch.where(mask[:, None], l, torch.zeros_like(l))
    choice = l
    if c["groups"] > 1:
        top = l.view(T, c["groups"], -1).amax(2)
        kept = torch.sort(top, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        allowed = torch.zeros_like(top, dtype=torch.bool).scatter(1, kept, True)
        choice = torch.where(allowed.repeat_interleave(E // c["groups"], 1), l, torch.full_like(l, -math.inf))
    idx = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    if c["score"] == "softmax":
        s = torch.exp(l - l.amax(1, keepdim=True))
        r = torch.ones_like(s)
    else:
        s = 1 / (1 + torch.exp(-l))
        r = 1 - s
    chosen = s.gather(1, idx)
    w = chosen / chosen.sum(1, keepdim=True)
    p = s / s.sum(1, keepdim=True)
    on = torch.ones((T, 1), device=DEV) if mask is None else mask[:, None].float()
    live = on.sum()
    many = live.clamp_min(1)
    count = torch.zeros(E, device=DEV).scatter_add(0, idx.reshape(-1), on.expand(T, k).reshape(-1))
    prob = (p * on).sum(0) / many
    loss = coef * E / (k * many) * (count * prob).sum()
    out = dict(idx=torch.where(on > 0, idx, -torch.ones_like(idx)), weights=w * on,
               count=torch.cat([count, live[None]]).int(), prob=prob, loss=loss[None])
    if c["backward"]:
        dw = st["dweights"]
        d = p * r * (count - (p * count).sum(1, keepdim=True)) * (st["dloss"] * coef * E / (k * many * many))
        d = d.scatter_add(1, idx, w * r.gather(1, idx) * (dw - (w * dw).sum(1, keepdim=True)))
        out["dlogits"] = (d * on).to(st["logits"].dtype)
    return out


# ------------------------------------------------------------------ work and exact values

def work(case):
    op = case["op"]
    if op == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        sz = 4 if case["dtype"] == "fp32" else 2
        b = T * E * sz + T * k * 12 + 8 * E + 8 + (T if case["masked"] else 0)
        f = 4 * T * E
        if case["backward"]:
            b += 2 * T * E * sz + T * k * 12 + 4 * E
            f += 8 * T * E
        return dict(bytes=b, flops=f)
    rows, E = case["T"] * case["k"], case["E"]
    live = E * (1 - (1 - case["k"] / E) ** case["T"])  # experts that get a row
    if op in ("product", "swiglu"):
        K, N = case["K"], case["N"] if op == "product" else 2 * case["F"]
        b = rows * (K + K // 32) + live * (N * K + 4 * ((N + 127) // 128) * (K // 128)) + 8 * E
        if op == "product":
            b += rows * 2 * N
        else:
            F = case["F"]
            b += rows * (F + F // 32) + (rows * 2 * (F + F // 32) if case["keep8"] else 0) + (4 * rows if case["weighted"] else 0)
        return dict(bytes=b, flops=2 * rows * N * K)
    if op == "swiglu_backward":
        F = case["F"]
        return dict(bytes=rows * (2 * F + 4 * (F + F // 32) + (8 if case["weighted"] else 0)) + 8 * E, flops=16 * rows * F)
    K, N = case["K"], case["N"]
    return dict(bytes=rows * (N + K + (N + K) // 32) + E * N * K * 2 + 8 * E, flops=2 * rows * N * K)


def _group_rows(st):
    """(expert, its live rows as a slice of the row buffer) of every group, from its definition."""
    count = st["count"].tolist()
    start = st["offset"].tolist() if st["offset"] is not None else [e * st["case"]["cap"] for e in range(len(count))]
    return [(e, slice(start[e], start[e] + n)) for e, n in enumerate(count) if n]


def _rows64(st, data, scales, rows):
    q = data.reshape(st["rows"], data.shape[-1])[rows].to(torch.float64)
    s = scales[:, rows].t() if st["offset"] is not None else scales.reshape(st["rows"], -1)[rows]
    return q * s.double().repeat_interleave(128, 1)


def _put64(st, tensors, rows, v):
    """128-channel groups of v: codes before rounding, and scales."""
    codes, scales = tensors
    a = v.reshape(v.shape[0], -1, 128).abs().amax(2).clamp_min(1e-4)
    codes.view(st["rows"], -1)[rows] = v * (448.0 / a).repeat_interleave(128, 1)
    if st["offset"] is not None:
        scales[:, rows] = (a / 448.0).t()
    else:
        scales.view(st["rows"], -1)[rows] = a / 448.0


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "gate":
        return _gate_exact(st)
    if op == "weight_grad":
        dw = torch.zeros(st["dw"].shape, dtype=torch.float64, device=DEV)
        for e, rows in _group_rows(st):
            dw[e] = _rows64(st, st["dy"], st["dy_scales"], rows).t() @ _rows64(st, st["x"], st["x_scales"], rows)
        return dw
    f64 = lambda t: torch.zeros(t.shape, dtype=torch.float64, device=DEV)  # noqa: E731
    if op == "swiglu_backward":
        d, dr = (f64(st["dpre"]), f64(st["dpre_scales"])), f64(st["drow_weights"]) if case["weighted"] else None
        for e, rows in _group_rows(st):
            v = _rows64(st, st["pre"], st["pre_scales"], rows)
            g, u = v[:, :case["F"]], v[:, case["F"]:]
            da = st["dact"].reshape(st["rows"], -1)[rows].double()
            sg = torch.sigmoid(g)
            if case["weighted"]:
                dr[rows] = (da * u * g * sg).sum(1)
                da = da * st["row_weights"][rows, None].double()
            _put64(st, d, rows, torch.cat([da * u * (sg + g * sg * (1 - sg)), da * g * sg], 1))
        out = dict(dpre=d[0], dpre_scales=d[1])
        return dict(out, drow_weights=dr) if case["weighted"] else out
    out = f64(st["out"]) if op == "product" else None
    act = (f64(st["act"]), f64(st["act_scales"])) if op == "swiglu" else None
    pre = (f64(st["pre"]), f64(st["pre_scales"])) if op == "swiglu" and case["keep8"] else None
    for e, rows in _group_rows(st):
        n = st["w"].shape[1]
        w = st["w"][e].double() * st["w_scales"][e].double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
        y = _rows64(st, st["x"], st["x_scales"], rows) @ w.t()
        if op == "product":
            out.view(st["rows"], -1)[rows] = y
            continue
        if pre is not None:
            _put64(st, pre, rows, y)
        a = y[:, :case["F"]] * torch.sigmoid(y[:, :case["F"]]) * y[:, case["F"]:]
        if case["weighted"]:
            a = a * st["row_weights"][rows, None].double()
        _put64(st, act, rows, a)
    if op == "product":
        return out
    res = dict(act=act[0], act_scales=act[1])
    if pre is not None:
        res.update(pre=pre[0], pre_scales=pre[1])
    return res


def _gate_exact(st):
    """The gate by autograd in 64 bits, on the choice that a stable ordering makes."""
    c = st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    on = torch.ones(T, dtype=torch.bool, device=DEV) if st["mask"] is None else st["mask"]
    l = st["logits"][on].double().requires_grad_(True)
    with torch.no_grad():
        order = l
        if c["groups"] > 1:
            best = l.reshape(len(l), c["groups"], -1).max(2).values
            rank = best.argsort(dim=1, descending=True, stable=True).argsort(dim=1)
            order = l.masked_fill((rank >= c["keep"]).repeat_interleave(E // c["groups"], 1), -math.inf)
        idx = order.argsort(dim=1, descending=True, stable=True)[:, :k]
        count = torch.bincount(idx.reshape(-1), minlength=E).double()
    many = max(len(l), 1)
    if c["score"] == "softmax":
        w, p = torch.softmax(l.gather(1, idx), 1), torch.softmax(l, 1)
    else:
        s = torch.sigmoid(l)
        w, p = s.gather(1, idx), s / s.sum(1, keepdim=True)
        w = w / w.sum(1, keepdim=True)
    prob = p.sum(0) / many
    loss = st["coef"] * E / (k * many) * (count * prob).sum()
    weights = torch.zeros((T, k), dtype=torch.float64, device=DEV)
    weights[on] = w.detach()
    out = dict(idx=None, weights=weights, count=None, prob=prob.detach(), loss=loss.detach()[None])
    if c["backward"]:
        d = torch.zeros((T, E), dtype=torch.float64, device=DEV)
        if len(l):
            (loss * st["dloss"].double() + (w * st["dweights"][on].double()).sum()).sum().backward()
            d[on] = l.grad
        out["dlogits"] = d
    return out

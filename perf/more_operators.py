"""Workloads of a trainer's large arrays: the cross entropy of the LM head and its gradient without
the logits, RMSNorm with the residual's addition and 8-bit outputs, and activations kept in 8 bits
with the backward passes that read them.

``run`` computes a case in plain torch operations, or (``own`` true) by the calls a user makes of
libbiv.  Shapes are those of the decoders this repository configures: hidden 256, 2048 and 4096,
MLP widths 688 and 6144, vocabularies 4096, 131072 and 151936, up to 16 sequences of 1024 tokens.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 128                      # elements per scale of an 8-bit row
IGNORE = -100
PIECE = 16384                    # vocabulary columns that the plain forms hold at a time
EPS = 1e-6


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # a few rows of the tiny decoder, summed to a mean: latency only
        dict(name="loss_13x4096", op="loss", T=13, V=4096, K=256, masked=False, weighted=False,
             z=0.0, reduce="mean"),
        # a trainer's micro-batch, prompts ignored, weighted tokens, with the z-loss
        dict(name="loss_4096x151936", op="loss", T=4096, V=151936, K=2048, masked=True,
             weighted=True, z=1e-4, reduce="sum"),
        # the gradient of a few rows of the tiny decoder
        dict(name="grad_13x4096", op="grad", T=13, V=4096, K=256, masked=False, kind="ce", z=0.0,
             dh="bf16", dw="bf16"),
        # one short answer at the full vocabulary: the weights are read, their gradient is written
        dict(name="grad_200x151936", op="grad", T=200, V=151936, K=2048, masked=False,
             kind="policy", z=0.0, dh="bf16", dw="bf16"),
        # a trainer's micro-batch, prompts ignored, the z-loss in the gradient
        dict(name="grad_4096x151936", op="grad", T=4096, V=151936, K=2048, masked=True, kind="ce",
             z=1e-4, dh="bf16", dw="bf16"),
        # a vocabulary of no even size, policy gradient, FP32 gradients for an accumulating trainer
        dict(name="grad_1000x32003_f32", op="grad", T=1000, V=32003, K=2048, masked=True,
             kind="policy", z=0.0, dh="f32", dw="f32"),
        # a decode step's rows before an FP8 matrix product: latency only
        dict(name="norm_16x2048", op="norm", rows=16, d=2048, pad=0, y=False, keep=False),
        # a prefill's rows in training: FP8 input of the product, bf16 beside it, a kept 8-bit copy
        dict(name="norm_16384x4096_keep", op="norm", rows=16384, d=4096, pad=0, y=True, keep=True),
        # backward of a norm on an odd count of the tiny decoder's rows, FP32 gradients
        dict(name="norm_back_301x256", op="norm_back", rows=301, d=256, dtype="f32", res=False),
        # backward of a norm from its kept rows, with the residual's gradient added
        dict(name="norm_back_16384x2048", op="norm_back", rows=16384, d=2048, dtype="bf16", res=True),
        # the MLP's activation of a micro-batch, its input kept in 8 bits
        dict(name="silu_keep_8192x6144", op="silu", rows=8192, I=6144, pad=0),
        # its backward, which also gives the activation again for the product's weight gradient
        dict(name="silu_back_8191x6144", op="silu_back", rows=8191, I=6144, dtype="bf16", y=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "grad", "grad", "norm", "norm_back", "silu", "silu_back"])
    if op in ("loss", "grad"):
        V = rng.choice([4096, 131072, 151936, _log_int(rng, 2, 200000)])
        K = rng.choice([256, 2048, 8 * _log_int(rng, 1, 512)])
        T = _log_int(rng, 1, min(8192, max(2, 4096 * 151936 * 2048 // (V * K) - 1)))
        c = dict(op=op, T=T, V=V, K=K, masked=rng.random() < 0.6, z=rng.choice([0.0, 1e-4]))
        if op == "loss":
            return dict(c, weighted=rng.random() < 0.5, reduce=rng.choice(["mean", "sum"]))
        return dict(c, kind=rng.choice(["ce", "policy"]), dh=rng.choice(["bf16", "bf16", "f32"]),
                    dw=rng.choice(["bf16", "bf16", "f32"]))
    if op in ("norm", "norm_back"):
        d = rng.choice([256, 2048, 4096, 16 * _log_int(rng, 1, 512)])
        rows = _log_int(rng, 1, min(32768, 16384 * 4096 // d))
        if op == "norm":
            return dict(op=op, rows=rows, d=d, pad=rng.choice([0, 0, 64]), y=rng.random() < 0.5,
                        keep=rng.random() < 0.5)
        return dict(op=op, rows=rows, d=d, dtype=rng.choice(["f32", "bf16"]), res=rng.random() < 0.5)
    I = rng.choice([688, 6144, 16 * _log_int(rng, 1, 512)])  # noqa: E741
    rows = _log_int(rng, 1, min(32768, 8192 * 6144 // I))
    if op == "silu":
        return dict(op=op, rows=rows, I=I, pad=rng.choice([0, 0, 64]))
    return dict(op=op, rows=rows, I=I, dtype=rng.choice(["f32", "bf16"]), y=rng.random() < 0.5)


def _live(case):
    """Which rows count: of every sequence of up to 1024 tokens, those behind its prompt."""
    T = case["T"]
    L = min(T, 1024)
    skip = L // 4 if case["masked"] else 0
    return [t % L >= skip for t in range(T)]


def _size(s):
    return 4 if s == "f32" else 2


def work(case):
    op = case["op"]
    if op in ("loss", "grad"):
        n, V, K = sum(_live(case)), case["V"], case["K"]
        if op == "loss":
            return {"bytes": 2 * K * (n + V) + 24 * case["T"], "flops": 2.0 * n * V * K}
        return {"bytes": 2 * K * (n + V) + K * (case["T"] * _size(case["dh"]) + V * _size(case["dw"]))
                + 16 * case["T"], "flops": 6.0 * n * V * K}
    rows = case["rows"]
    if op in ("norm", "norm_back"):
        n = rows * case["d"]
        s = 4 * rows * ((case["d"] + GROUP - 1) // GROUP)
        if op == "norm":
            return {"bytes": 7 * n + s + 2 * case["d"] + (2 * n if case["y"] else 0)
                    + ((n + s + 4 * rows) if case["keep"] else 0), "flops": 12.0 * n}
        return {"bytes": n * (1 + _size(case["dtype"]) * (3 if case["res"] else 2)) + s + 4 * rows
                + 6 * case["d"], "flops": 12.0 * n}
    n = rows * case["I"]
    s = 4 * rows * ((case["I"] + GROUP - 1) // GROUP)
    if op == "silu":
        return {"bytes": n * (4 + 2 + 2) + 2 * s, "flops": 16.0 * n}
    return {"bytes": n * (2 + 3 * _size(case["dtype"]) + (2 if case["y"] else 0)) + 2 * s, "flops": 16.0 * n}


# ---------------------------------------------------------------- prepare --
def _dtype(s):
    return torch.float32 if s == "f32" else torch.bfloat16


def _empty(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device=DEV)


def _rows(rows, width, pad, dtype=torch.bfloat16):
    """Rows of `width`, `pad` elements between them."""
    return _empty(rows, width + pad, dtype=dtype)[:, :width]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=gen)  # noqa: E731
    uni = lambda *s: torch.rand(*s, device=DEV, generator=gen)   # noqa: E731
    st = {"case": case}
    return {"loss": _prepare_head, "grad": _prepare_head, "norm": _prepare_norm,
            "norm_back": _prepare_norm_back, "silu": _prepare_silu,
            "silu_back": _prepare_silu_back}[case["op"]](st, case, gen, rnd, uni)


def _prepare_head(st, c, gen, rnd, uni):
    T, V, K = c["T"], c["V"], c["K"]
    h = rnd(T, K).bfloat16()
    W = _empty(V, K, dtype=torch.bfloat16)
    for a in range(0, V, PIECE):
        W[a:a + PIECE] = rnd(min(PIECE, V - a), K) * (2.5 / math.sqrt(K))
    live = torch.tensor(_live(c), device=DEV)
    target = torch.empty(T, dtype=torch.int64, device=DEV)
    lse = torch.empty(T, device=DEV)
    for a in range(0, T, 512):                   # targets sampled from the model itself
        z = (h[a:a + 512] @ W.t()).float()
        lse[a:a + 512] = z.logsumexp(1)
        e = torch.empty_like(z).exponential_(1.0, generator=gen)
        target[a:a + 512] = (z - e.log_()).argmax(1)
    st.update(h=h, W=W, live=live, target=target.int())
    if c["op"] == "loss":
        st["target"] = torch.where(live, st["target"], IGNORE)
        st["weight"] = 0.5 + uni(T) if c["weighted"] else None
        st["norm"] = float(max(1, T // 2))
        st["out"] = {"lp": _empty(T), "lse": _empty(T), "dlp": _empty(T)}
        if c["z"]:
            st["out"]["dlse"] = _empty(T)
        st["stats"] = _empty(4)
        st["parts"] = _loss_parts(st["stats"])
        if own:
            from invariant_forward_bitwise_gb300 import biv
            st["ws"] = _empty(biv.biv_lm_head_loss_workspace(T, V), dtype=torch.uint8)
        return st
    n = float(max(1, int(live.sum())))
    st["lse"] = lse
    st["dlp"] = live * (rnd(T) if c["kind"] == "policy" else -torch.ones(T, device=DEV)) / n
    st["dlse"] = live * (2 * c["z"] / n) * lse if c["z"] else None
    st["dh"], st["dW"] = _empty(T, K, dtype=_dtype(c["dh"])), _empty(V, K, dtype=_dtype(c["dw"]))
    if own:
        from invariant_forward_bitwise_gb300 import biv
        st["ws"] = _empty(biv.biv_lm_head_backward_workspace(T, V, K, st["dh"].dtype, st["dW"].dtype),
                          dtype=torch.uint8)
    return st


def _hidden(rnd, rows, d):
    """Rows of a residual stream: a few channels are far larger than the rest."""
    x = rnd(rows, d) * 1.5
    x[:, ::97] *= 20
    return x


def _codes(x):
    """Rows in 8 bits: e4m3 codes and a scale amax / 448 per 128 elements (1 where amax is 0)."""
    rows, d = x.shape
    g = (d + GROUP - 1) // GROUP
    p = torch.nn.functional.pad(x, (0, g * GROUP - d)).view(rows, g, GROUP)
    a = p.abs().amax(2)
    s = torch.where(a > 0, a / 448, torch.ones_like(a))
    q = (p / s[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(rows, g * GROUP)[:, :d]
    return q.contiguous().view(torch.uint8), s


def _values(codes, scales):
    """What 8-bit rows stand for, in 32 bits."""
    d = codes.shape[1]
    return codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(GROUP, 1)[:, :d]


def _groups(d):
    return (d + GROUP - 1) // GROUP


def _prepare_norm(st, c, gen, rnd, uni):
    rows, d = c["rows"], c["d"]
    st["x"], st["res"] = _rows(rows, d, c["pad"]), _rows(rows, d, c["pad"])
    st["x"].copy_(rnd(rows, d) * 0.5)
    st["res"].copy_(_hidden(rnd, rows, d))
    st["w"] = (1 + 0.2 * rnd(d)).bfloat16()
    st["out"] = {"res": _empty(rows, d, dtype=torch.bfloat16), "codes": _empty(rows, d, dtype=torch.uint8),
                 "scales": _empty(rows, _groups(d))}
    if c["y"]:
        st["out"]["y"] = _empty(rows, d, dtype=torch.bfloat16)
    if c["keep"]:
        st["out"] |= {"keep": _empty(rows, d, dtype=torch.uint8), "keep_scales": _empty(rows, _groups(d)),
                      "inv": _empty(rows)}
    return st


def _prepare_norm_back(st, c, gen, rnd, uni):
    rows, d = c["rows"], c["d"]
    x = _hidden(rnd, rows, d)
    st["keep"], st["keep_scales"] = _codes(x)
    st["inv"] = torch.rsqrt(x.square().mean(1) + EPS)
    st["w"] = (1 + 0.2 * rnd(d)).bfloat16()
    size = torch.exp(rnd(rows, 1))
    st["dy"] = (1e-3 * size * rnd(rows, d)).to(_dtype(c["dtype"]))
    st["dres"] = (1e-3 * size * rnd(rows, d)).to(_dtype(c["dtype"])) if c["res"] else None
    st["dx"], st["dw"] = _empty(rows, d, dtype=_dtype(c["dtype"])), _empty(d)
    if own:
        from invariant_forward_bitwise_gb300 import biv
        st["ws"] = _empty(biv.biv_rmsnorm_backward_fp8_workspace(rows, d), dtype=torch.uint8)
    return st


def _prepare_silu(st, c, gen, rnd, uni):
    rows, I = c["rows"], c["I"]  # noqa: E741
    st["gu"] = _rows(rows, 2 * I, c["pad"])
    st["gu"].copy_(rnd(rows, 2 * I) * torch.exp(0.5 * rnd(rows, 1)))
    st["out"] = {"y": _empty(rows, I, dtype=torch.bfloat16), "keep": _empty(rows, 2 * I, dtype=torch.uint8),
                 "keep_scales": _empty(rows, 2 * _groups(I))}
    return st


def _prepare_silu_back(st, c, gen, rnd, uni):
    rows, I = c["rows"], c["I"]  # noqa: E741
    size = torch.exp(0.5 * rnd(rows, 1))
    (qg, sg), (qu, su) = _codes(rnd(rows, I) * size), _codes(rnd(rows, I) * size)
    st["keep"], st["keep_scales"] = torch.cat([qg, qu], 1), torch.cat([sg, su], 1)
    st["dy"] = (1e-3 * size * rnd(rows, I)).to(_dtype(c["dtype"]))
    st["dgu"] = _empty(rows, 2 * I, dtype=_dtype(c["dtype"]))
    st["y"] = _empty(rows, I, dtype=torch.bfloat16) if c["y"] else None
    return st


# -------------------------------------------------------------------- run --
def run(st):
    f = _OWN if own else _PLAIN
    return f[st["case"]["op"]](st)


def _loss_parts(stats):
    return dict(zip(("loss", "nll", "lse2", "count"), stats.split(1)))


def _as_values(out):
    """8-bit arrays as the e4m3 values of their codes (their scales stand beside them)."""
    return {k: v.view(torch.float8_e4m3fn) if v.dtype is torch.uint8 else v for k, v in out.items()}


def _own_loss(st):
    from invariant_forward_bitwise_gb300 import biv
    c, o = st["case"], st["out"]
    biv.biv_lm_head_loss(
        st["h"], st["W"], st["target"], o["lp"], o["lse"], st["stats"], st["ws"], weight=st["weight"],
        dlp=o["dlp"], dlse=o.get("dlse"), z_coef=c["z"],
        reduce=biv.LOSS_TOKEN_MEAN if c["reduce"] == "mean" else biv.LOSS_SUM, norm=st["norm"],
        ignore_index=IGNORE)
    return {**o, **st["parts"]}


def _own_grad(st):
    from invariant_forward_bitwise_gb300 import biv
    biv.biv_lm_head_backward(st["h"], st["W"], st["target"], st["lse"], st["dlp"], st["dh"], st["dW"],
                             st["ws"], dlse=st["dlse"])
    return {"dh": st["dh"], "dW": st["dW"]}


def _own_norm(st):
    from invariant_forward_bitwise_gb300 import biv
    o = st["out"]
    biv.biv_add_rmsnorm_fp8(st["x"], st["res"], st["w"], EPS, residual_out=o["res"], y=o.get("y"),
                            codes=o["codes"], scales=o["scales"], keep=o.get("keep"),
                            keep_scales=o.get("keep_scales"), inv=o.get("inv"))
    return _as_values(o)


def _own_norm_back(st):
    from invariant_forward_bitwise_gb300 import biv
    biv.biv_rmsnorm_backward_fp8(st["keep"], st["keep_scales"], st["inv"], st["w"], st["dy"], st["dx"],
                                 st["dw"], st["ws"], dres=st["dres"])
    return {"dx": st["dx"], "dw": st["dw"]}


def _own_silu(st):
    from invariant_forward_bitwise_gb300 import biv
    o = st["out"]
    biv.biv_silu_mul_keep_fp8(st["gu"], o["y"], o["keep"], o["keep_scales"])
    return _as_values(o)


def _own_silu_back(st):
    from invariant_forward_bitwise_gb300 import biv
    biv.biv_silu_mul_backward_fp8(st["keep"], st["keep_scales"], st["dy"], st["dgu"], y=st["y"])
    return {"dgu": st["dgu"]} if st["y"] is None else {"dgu": st["dgu"], "y": st["y"]}


def _pieces(W):
    """(first column, piece of the weights in 32 bits) over the vocabulary."""
    for a in range(0, W.shape[0], PIECE):
        yield a, W[a:a + PIECE].float()


def _plain_loss(st):
    c, T = st["case"], st["case"]["T"]
    h = st["h"].float()
    t = st["target"].long()
    on = t != IGNORE
    m = torch.full((T,), -math.inf, device=DEV)
    s, zt = torch.zeros(T, device=DEV), torch.zeros(T, device=DEV)
    for a, w in _pieces(st["W"]):                # a running maximum and sum over the pieces
        z = h @ w.t()
        new = torch.maximum(m, z.amax(1))
        s = s * (m - new).exp() + (z - new[:, None]).exp().sum(1)
        m = new
        here = (t >= a) & (t < a + w.shape[0])
        zt = torch.where(here, z.gather(1, (t - a).clamp(0, w.shape[0] - 1)[:, None])[:, 0], zt)
    lse = m + s.log()
    lp = zt - lse
    zero = torch.zeros((), device=DEV)
    wt = torch.where(on, st["weight"] if c["weighted"] else torch.ones((), device=DEV), zero)
    count = wt.double().sum()
    share = wt / (count if c["reduce"] == "mean" else torch.tensor(st["norm"], device=DEV)).float()
    share = torch.where(on, share, zero)
    lp, lse = torch.where(on, lp, zero), torch.where(on, lse, zero)
    nll, sq = (share * -lp).double().sum(), (share * lse * lse).double().sum()
    stats = torch.stack([nll + c["z"] * sq, nll, sq, count]).float()
    out = {"lp": lp, "lse": lse, "dlp": -share}
    if c["z"]:
        out["dlse"] = 2 * c["z"] * share * lse
    return {**out, **_loss_parts(stats)}


def _plain_grad(st):
    c = st["case"]
    h, t = st["h"].float(), st["target"].long()
    dh, dW = torch.zeros_like(h), torch.empty_like(st["dW"])
    scale = -st["dlp"] if st["dlse"] is None else st["dlse"] - st["dlp"]
    for a, w in _pieces(st["W"]):
        dz = (h @ w.t() - st["lse"][:, None]).exp() * scale[:, None]
        here = (t >= a) & (t < a + w.shape[0])
        dz.scatter_add_(1, (t - a).clamp(0, w.shape[0] - 1)[:, None], (st["dlp"] * here)[:, None])
        dh += dz @ w
        dW[a:a + w.shape[0]] = dz.t() @ h
    return {"dh": dh.to(_dtype(c["dh"])), "dW": dW}


def _plain_norm(st):
    c = st["case"]
    r = (st["x"].float() + st["res"].float()).bfloat16()
    x = r.float()
    inv = 1 / (x.square().mean(1) + EPS).sqrt()
    y = x * inv[:, None] * st["w"].float()
    q, s = _codes(y)
    out = {"res": r, "codes": q, "scales": s}
    if c["y"]:
        out["y"] = y.bfloat16()
    if c["keep"]:
        kq, ks = _codes(x)
        out |= {"keep": kq, "keep_scales": ks, "inv": inv}
    return _as_values(out)


def _plain_norm_back(st):
    x = _values(st["keep"], st["keep_scales"])
    inv, dy = st["inv"][:, None], st["dy"].float()
    g = dy * st["w"].float()
    dx = inv * g - x * (inv ** 3 * (g * x).mean(1, keepdim=True))
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    return {"dx": dx.to(st["dx"].dtype), "dw": (dy * (x * inv)).sum(0, dtype=torch.float64).float()}


def _plain_silu(st):
    g, u = st["gu"].float().split(st["case"]["I"], 1)
    y = (g / (1 + (-g).exp()) * u).bfloat16()
    (qg, sg), (qu, su) = _codes(g), _codes(u)
    return _as_values({"y": y, "keep": torch.cat([qg, qu], 1), "keep_scales": torch.cat([sg, su], 1)})


def _plain_silu_back(st):
    I, n = st["case"]["I"], _groups(st["case"]["I"])  # noqa: E741
    g = _values(st["keep"][:, :I].contiguous(), st["keep_scales"][:, :n])
    u = _values(st["keep"][:, I:].contiguous(), st["keep_scales"][:, n:])
    s, dy = 1 / (1 + (-g).exp()), st["dy"].float()
    out = {"dgu": torch.cat([dy * u * (s * (1 + g * (1 - s))), dy * (g * s)], 1).to(st["dgu"].dtype)}
    if st["y"] is not None:
        out["y"] = (g * s * u).bfloat16()
    return out


_OWN = {"loss": _own_loss, "grad": _own_grad, "norm": _own_norm, "norm_back": _own_norm_back,
        "silu": _own_silu, "silu_back": _own_silu_back}
_PLAIN = {"loss": _plain_loss, "grad": _plain_grad, "norm": _plain_norm, "norm_back": _plain_norm_back,
          "silu": _plain_silu, "silu_back": _plain_silu_back}


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    st = prepare(case, seed)
    return {"loss": _exact_loss, "grad": _exact_grad, "norm": _exact_norm, "norm_back": _exact_norm_back,
            "silu": _exact_silu, "silu_back": _exact_silu_back}[case["op"]](st, case)


F64 = torch.float64


def _exact_loss(st, c):
    """Row blocks of whole logits; the coefficients by differentiating the loss."""
    T = c["T"]
    keep = torch.nonzero(st["target"] != IGNORE)[:, 0]
    weight = torch.ones(T, dtype=F64, device=DEV) if st["weight"] is None else st["weight"].to(F64)
    total = weight[keep].sum()
    over = total if c["reduce"] == "mean" else st["norm"]
    out = {k: torch.zeros(T, dtype=F64, device=DEV) for k in st["out"]}
    sums = torch.zeros(4, dtype=F64, device=DEV)
    sums[3] = total
    W = st["W"].to(F64).t()
    for r in keep.split(1024):
        logits = st["h"][r].to(F64) @ W
        lse = torch.logsumexp(logits, 1).requires_grad_(True)
        lp = (logits[torch.arange(r.numel(), device=DEV), st["target"][r].long()] - lse.detach()).requires_grad_(True)
        part = weight[r] / over
        nll, sq = -(part * lp).sum(), (part * lse ** 2).sum()
        (nll + c["z"] * sq).backward()
        sums[:3] += torch.stack([nll + c["z"] * sq, nll, sq]).detach()
        out["lp"][r], out["lse"][r], out["dlp"][r] = lp.detach(), lse.detach(), lp.grad
        if c["z"]:
            out["dlse"][r] = lse.grad
    return {**out, **_loss_parts(sums)}


def _exact_grad(st, c):
    T, V, K = c["T"], c["V"], c["K"]
    dh = torch.zeros(T, K, dtype=F64, device=DEV)
    dW = torch.zeros(V, K, dtype=F64, device=DEV)
    W = st["W"].to(F64)
    for a in range(0, T, 1024):
        rows = slice(a, min(T, a + 1024))
        h = st["h"][rows].to(F64)
        p = torch.exp(torch.addmm(-st["lse"][rows].to(F64)[:, None], h, W.t()))
        dlp = st["dlp"][rows].to(F64)
        dlse = torch.zeros_like(dlp) if st["dlse"] is None else st["dlse"][rows].to(F64)
        p *= (dlse - dlp)[:, None]
        p[torch.arange(p.shape[0], device=DEV), st["target"][rows].long()] += dlp
        dh[rows] = p @ W
        dW.addmm_(p.t(), h)
    return {"dh": dh, "dW": dW}


def _exact_codes(x):
    """What the codes stand for before they are rounded, x / s, and the scales s."""
    a = torch.stack([p.abs().amax(1) for p in x.split(GROUP, 1)], 1)
    s = torch.where(a == 0, torch.ones_like(a), a / 448)
    return torch.cat([p / s[:, i:i + 1] for i, p in enumerate(x.split(GROUP, 1))], 1), s


def _exact_norm(st, c):
    r = st["x"].to(F64).add(st["res"].to(F64)).bfloat16()
    x = r.to(F64)
    inv = torch.rsqrt(torch.linalg.vector_norm(x, dim=1) ** 2 / c["d"] + EPS)
    y = torch.einsum("rd,r,d->rd", x, inv, st["w"].to(F64))
    out = {"res": r, "y": y, "inv": inv}
    out["codes"], out["scales"] = _exact_codes(y)
    out["keep"], out["keep_scales"] = _exact_codes(x)
    return {k: out[k] for k in st["out"]}


def _exact_values(codes, scales):
    out = codes.view(torch.float8_e4m3fn).to(F64)
    for i, part in enumerate(out.split(GROUP, 1)):
        part *= scales[:, i:i + 1].to(F64)
    return out


def _exact_norm_back(st, c):
    unit = _exact_values(st["keep"], st["keep_scales"]) * st["inv"].to(F64)[:, None]
    dy = st["dy"].to(F64)
    g = dy * st["w"].to(F64)
    along = torch.einsum("rd,rd->r", g, unit) / c["d"]
    dx = st["inv"].to(F64)[:, None] * (g - along[:, None] * unit)
    if st["dres"] is not None:
        dx += st["dres"].to(F64)
    return {"dx": dx, "dw": torch.einsum("rd,rd->d", dy, unit)}


def _exact_silu(st, c):
    g, u = st["gu"].to(F64).chunk(2, 1)
    (qg, sg), (qu, su) = _exact_codes(g), _exact_codes(u)
    return {"y": torch.nn.functional.silu(g) * u, "keep": torch.cat([qg, qu], 1),
            "keep_scales": torch.cat([sg, su], 1)}


def _exact_silu_back(st, c):
    n = _groups(c["I"])
    gate = _exact_values(st["keep"][:, :c["I"]].contiguous(), st["keep_scales"][:, :n]).requires_grad_(True)
    up = _exact_values(st["keep"][:, c["I"]:].contiguous(), st["keep_scales"][:, n:]).requires_grad_(True)
    y = torch.nn.functional.silu(gate) * up
    y.backward(st["dy"].to(F64))
    out = {"dgu": torch.cat([gate.grad, up.grad], 1)}
    if st["y"] is not None:
        out["y"] = y.detach()
    return out

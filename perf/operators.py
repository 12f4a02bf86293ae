"""Workloads of the trainer-end operators: the clipped policy loss (from per-token logprobs, and
from logits) with its gradient, and the AdamW step over many tensors with its gradient-norm clip.

``run`` computes a case in plain torch operations, or (``own`` true) by the calls a user makes of
libbiv.  Shapes are those of a group-relative policy-optimisation step on the decoders this
repository configures: 64 prompts x 8 responses of 128 to 1024 tokens, vocabularies 4096, 131072
and 151936, weight shapes of the 2-layer tiny decoder and of the hidden-2048 decoder.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128                      # elements per scale of an 8-bit state
M32 = 0xFFFFFFFF


# ------------------------------------------------------------------ cases --
def listed():
    tok = dict(op="tokens", clip_lo=0.2, clip_hi=0.28)
    log = dict(op="logits", clip_lo=0.2, clip_hi=0.2, pad=0)
    return [
        # one prompt's group of 8 short answers, token mean, no KL: latency only
        dict(name="tokens_8x150", nseq=8, max_len=150, kl=0.0, dual=0.0, reduce="token",
             adv="seq", masked=False, **tok),
        # a whole rollout of 512 responses, KL to a reference, dual clip, per-sequence means
        dict(name="tokens_512x1024", nseq=512, max_len=1024, kl=0.04, dual=3.0, reduce="seq",
             adv="seq", masked=True, **tok),
        # a few rows of the tiny decoder
        dict(name="logits_13x4096", nseq=3, T=13, V=4096, z="f32", dz="f32", kl=0.04, ent=0.0,
             temp=1.0, reduce="token", adv="seq", masked=True, **log),
        # one short response at the full vocabulary, bf16 gradient for the GEMMs that follow
        dict(name="logits_64x151936", nseq=2, T=64, V=151936, z="f32", dz="bf16", kl=0.0, ent=0.0,
             temp=1.0, reduce="token", adv="seq", masked=False, **log),
        # a trainer micro-batch, FP32 logits and gradient, KL and entropy terms
        dict(name="logits_4096x151936", nseq=7, T=4096, V=151936, z="f32", dz="f32", kl=0.02,
             ent=0.001, temp=1.0, reduce="seq", adv="tok", masked=True, **log),
        # the hybrid's vocabulary with bf16 logits, sampled at a temperature, an odd row count
        dict(name="logits_2037x131072_bf16", nseq=5, T=2037, V=131072, z="bf16", dz="bf16",
             kl=0.02, ent=0.0, temp=0.8, reduce="sum", adv="seq", masked=True, **log),
        # a vocabulary of no even size, rows packed without padding (no row is 16-byte aligned)
        dict(name="logits_1000x32003", nseq=4, T=1000, V=32003, z="f32", dz="f32", kl=0.0,
             ent=0.01, temp=1.0, reduce="token", adv="tok", masked=True, **log),
        # every weight of the 2-layer tiny decoder, FP32 master and states, clipped by the norm
        dict(name="adamw_tiny", op="adamw", shapes="tiny", layers=2, state="f32", param="master",
             grad="f32", rounding="nearest", clip=1.0, wd=0.1),
        # eight layers and the embedding of the hidden-2048 decoder: bf16 weights with an FP32 master
        dict(name="adamw_8L_f32", op="adamw", shapes="dense", layers=8, state="f32", param="master",
             grad="f32", rounding="nearest", clip=1.0, wd=0.1),
        # the same weights with 8-bit states, bf16 weights without a master, stochastic rounding
        dict(name="adamw_8L_8bit", op="adamw", shapes="dense", layers=8, state="e4m3", param="bf16",
             grad="bf16", rounding="stochastic", clip=0.0, wd=0.1),
        # one layer, 8-bit states beside an FP32 master
        dict(name="adamw_1L_8bit_master", op="adamw", shapes="layer", layers=1, state="e4m3",
             param="master", grad="f32", rounding="nearest", clip=1.0, wd=0.0),
        # 300 tensors of odd sizes (norm gains, biases, adapters), FP32 weights
        dict(name="adamw_300_odd", op="adamw", shapes="odd", layers=300, state="e4m3", param="f32",
             grad="f32", rounding="nearest", clip=0.5, wd=0.01),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tokens", "logits", "logits", "adamw", "adamw"])
    if op == "tokens":
        return dict(op=op, nseq=_log_int(rng, 1, 512), max_len=_log_int(rng, 1, 1024),
                    kl=rng.choice([0.0, 0.01, 0.04]), dual=rng.choice([0.0, 3.0]),
                    reduce=rng.choice(["token", "seq", "sum"]), adv=rng.choice(["seq", "tok"]),
                    masked=rng.random() < 0.7, clip_lo=rng.choice([0.1, 0.2]),
                    clip_hi=rng.choice([0.2, 0.28]))
    if op == "logits":
        V = rng.choice([4096, 131072, 151936, _log_int(rng, 2, 200000)])
        z, dz = rng.choice([("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
        T = _log_int(rng, 1, min(8192, max(2, 4096 * 151936 // (V + 8))))
        return dict(op=op, nseq=rng.randint(1, min(T, 16)), T=T, V=V, z=z, dz=dz,
                    kl=rng.choice([0.0, 0.02]), ent=rng.choice([0.0, 0.001, 0.01]),
                    temp=rng.choice([1.0, 0.8, 1.3]), reduce=rng.choice(["token", "seq", "sum"]),
                    adv=rng.choice(["seq", "tok"]), masked=rng.random() < 0.7, clip_lo=0.2,
                    clip_hi=rng.choice([0.2, 0.28]), pad=rng.choice([0, 1, 8]))
    shapes = rng.choice(["tiny", "layer", "dense", "odd"])
    layers = {"tiny": rng.randint(1, 2), "layer": rng.randint(1, 4), "dense": rng.randint(1, 6),
              "odd": _log_int(rng, 1, 400)}[shapes]
    return dict(op="adamw", shapes=shapes, layers=layers, state=rng.choice(["f32", "e4m3"]),
                param=rng.choice(["master", "bf16", "f32"]), grad=rng.choice(["f32", "bf16"]),
                rounding=rng.choice(["nearest", "stochastic"]), clip=rng.choice([0.0, 0.5, 1.0]),
                wd=rng.choice([0.0, 0.01, 0.1]))


def _sizes(case):
    """Element counts of the case's tensors, and which of them decay (matrices do, gains do not)."""
    d, inter, width, q, vocab, L = ((256, 688, 512, 256, 4096, case["layers"]) if case["shapes"] == "tiny"
                                    else (2048, 6144, 4096, 2048, 151936, case["layers"]))
    if case["shapes"] == "odd":
        n = [1 + (i * 7919 * 7919 + 104729 * i) % (3 ** (2 + i % 9)) for i in range(L)]
        return n, [i % 3 == 0 for i in range(L)]
    sizes, decay = [], []
    if case["shapes"] != "layer":
        sizes += [vocab * d, d]
        decay += [True, False]
    if case["shapes"] == "tiny":
        sizes, decay = sizes + [vocab * d], decay + [True]
    for _ in range(L):
        sizes += [width * d, d * q, 2 * inter * d, d * inter, d, d]
        decay += [True, True, True, True, False, False]
    return sizes, decay


def _lengths(case):
    """Sequence lengths: between an eighth of the longest and the longest, the last one full."""
    n, top = case["nseq"], case["max_len"]
    lo = max(1, top // 8)
    return [lo + (i * 40503 + 12345 * i * i) % (top - lo + 1) for i in range(n - 1)] + [top]


def work(case):
    if case["op"] == "tokens":
        T = sum(_lengths(case))
        per = 12 + (4 if case["kl"] else 0) + (4 if case["adv"] == "tok" else 0) + (1 if case["masked"] else 0)
        return {"bytes": per * T + 4 * case["nseq"], "flops": 20.0 * T}
    if case["op"] == "logits":
        by = {"f32": 4, "bf16": 2}
        n = case["T"] * case["V"]
        return {"bytes": n * (by[case["z"]] + by[case["dz"]]) + 28 * case["T"], "flops": 16.0 * n}
    n = float(sum(_sizes(case)[0]))
    g = 4 if case["grad"] == "f32" else 2
    p = {"master": 4 + 4 + 2, "bf16": 2 + 2, "f32": 4 + 4}[case["param"]]
    s = 16 if case["state"] == "f32" else 4 + 16.0 / BLOCK
    return {"bytes": n * (g + p + s), "flops": 16.0 * n}


# ---------------------------------------------------------------- prepare --
def _dtype(s):
    return torch.float32 if s == "f32" else torch.bfloat16


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    return _prepare_adamw(case, seed, gen) if case["op"] == "adamw" else _prepare_loss(case, gen)


def _prepare_loss(case, gen):
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=gen)  # noqa: E731
    uni = lambda *s: torch.rand(*s, device=DEV, generator=gen)   # noqa: E731
    if case["op"] == "tokens":
        lens = _lengths(case)
        T = sum(lens)
    else:
        T, n = case["T"], case["nseq"]
        tail = 1 if T > 2 * n else 0             # a row behind the last sequence (padding)
        cuts = sorted((i * (T - tail)) // n for i in range(n + 1))
        lens = [b - a for a, b in zip(cuts, cuts[1:])]
    st = {"case": case, "T": T}
    start = [0]
    for x in lens:
        start.append(start[-1] + x)
    st["seq_start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
    if case["op"] == "tokens":
        st["lp"] = -torch.empty(T, device=DEV).exponential_(1.2, generator=gen)
    else:
        V, ld = case["V"], case["V"] + case["pad"]
        z = torch.empty(T, ld, device=DEV, dtype=_dtype(case["z"]))
        lp = torch.empty(T, device=DEV)
        target = torch.empty(T, dtype=torch.int32, device=DEV)
        for a in range(0, T, 512):               # targets sampled from the policy itself
            b = min(T, a + 512)
            x = rnd(b - a, V) * 2.5
            z[a:b, :V] = x
            x = z[a:b, :V].float() / case["temp"]
            e = torch.empty_like(x).exponential_(1.0, generator=gen)
            target[a:b] = (x - e.log_()).argmax(1)
            lp[a:b] = x.gather(1, target[a:b, None].long())[:, 0] - x.logsumexp(1)
        st["logits"], st["target"], st["lp"] = z[:, :V], target, lp
        st["dz"] = torch.zeros(T, ld, device=DEV, dtype=_dtype(case["dz"]))[:, :V]
        st["lp_out"], st["ent_out"] = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    # the behaviour policy lags behind by an update or two, the reference further
    st["old_lp"] = st["lp"] + 0.15 * rnd(T) * (uni(T) < 0.8)
    st["ref_lp"] = st["lp"] + 0.3 * rnd(T) if case["kl"] else None
    st["adv"] = rnd(T if case["adv"] == "tok" else len(lens))
    st["mask"] = None
    if case["masked"]:
        st["mask"] = (uni(T) < 0.97).to(torch.uint8)
        if len(lens) > 1:
            st["mask"][start[0]:start[1]] = 0    # an answer that was cut: none of it counts
    st["dlp"] = torch.empty(T, device=DEV)
    st["stats"] = torch.empty(8, device=DEV)
    st["parts"] = _parts(st["stats"])
    st["norm"] = float(max(1, T // 2))
    if own:
        from invariant_forward_bitwise_gb300 import biv
        st["ws"] = torch.empty(biv.biv_policy_loss_workspace(T, len(lens)), dtype=torch.uint8, device=DEV)
    return st


def _prepare_adamw(case, seed, gen):
    sizes, decay = _sizes(case)
    offs, total = [], 0
    for n in sizes:                              # tensors start on a block of their flat buffer
        offs.append(total)
        total += (n + BLOCK - 1) // BLOCK * BLOCK
    inside = torch.ones(total, dtype=torch.bool, device=DEV)
    for n, o, nxt in zip(sizes, offs, offs[1:] + [total]):
        inside[o + n:nxt] = False
    rnd = lambda std: (torch.randn(total, device=DEV, generator=gen) * std).mul_(inside)  # noqa: E731
    st = {"case": case, "seed": int(seed) & 0x7FFFFFFF, "inside": inside}
    w = rnd(0.02)
    st["w"] = w.to(torch.bfloat16) if case["param"] == "bf16" else w
    st["p"] = w.to(torch.bfloat16) if case["param"] == "master" else None
    # gradients of differing size from row to row, as a loss gives them
    size = torch.exp(torch.randn(total // BLOCK, 1, device=DEV, generator=gen)).expand(-1, BLOCK).reshape(-1)
    st["g"] = (rnd(1e-3) * size).to(_dtype(case["grad"]))
    m = rnd(3e-4) * size
    v = (rnd(1e-3) * size) ** 2 + (1e-4 * size * inside) ** 2
    st["decay"] = torch.zeros(total, dtype=torch.bool, device=DEV)
    for n, o, d in zip(sizes, offs, decay):
        st["decay"][o:o + n] = d
    if case["state"] == "f32":
        st["m"], st["v"] = m, v
    else:
        for k, x in (("m", m), ("v", v.sqrt())):
            x = x.view(-1, BLOCK)
            s = x.abs().amax(1).clamp_min(2.0 ** -100) / 448
            st[k] = (x / s[:, None]).to(torch.float8_e4m3fn).view(-1)
            st[k + "s"] = s
    st["lr"] = torch.tensor([1e-5 if case["param"] == "master" else 1e-3], device=DEV)
    st["step"] = torch.tensor([11, 0], dtype=torch.int32, device=DEV)
    st["betas"], st["eps"] = (0.9, 0.999), 1e-8
    if own:
        from invariant_forward_bitwise_gb300.optim import AdamW
        cut = lambda t: [t[o:o + n] for n, o in zip(sizes, offs)]  # noqa: E731
        nb = lambda t: [t[o // BLOCK:o // BLOCK + (n + BLOCK - 1) // BLOCK]  # noqa: E731
                        for n, o in zip(sizes, offs)]
        e8 = case["state"] == "e4m3"
        st["opt"] = AdamW(
            params=cut(st["p"] if case["param"] == "master" else st["w"]), grads=cut(st["g"]),
            master=cut(st["w"]) if case["param"] == "master" else None,
            exp_avg=cut(st["m"]), exp_avg_sq=cut(st["v"]),
            exp_avg_scale=nb(st["ms"]) if e8 else None, exp_avg_sq_scale=nb(st["vs"]) if e8 else None,
            lr=st["lr"], betas=st["betas"], eps=st["eps"], step=st["step"],
            weight_decay=[case["wd"] if d else 0.0 for d in decay], max_norm=case["clip"],
            rounding=case["rounding"], seed=st["seed"])
    return st


# -------------------------------------------------------------------- run --
def run(st):
    op = st["case"]["op"]
    if own:
        return _own_adamw(st) if op == "adamw" else _own_loss(st)
    return _plain_adamw(st) if op == "adamw" else _plain_loss(st)


def _parts(stats):
    """The loss with its two terms, the entropy, the diagnostics and the count of tokens, each by itself."""
    return dict(zip(("loss", "entropy_mean", "diag", "count"), stats.split([3, 1, 3, 1])))


def _own_loss(st):
    from invariant_forward_bitwise_gb300 import biv
    c = st["case"]
    d = biv.policy_desc(
        st["seq_start"], st["adv"], st["stats"], st["ws"], T=st["T"], mask=st["mask"],
        old_lp=st["old_lp"], ref_lp=st["ref_lp"], clip_lo=c["clip_lo"], clip_hi=c["clip_hi"],
        dual_clip=c.get("dual", 0.0), kl_coef=c["kl"], ent_coef=c.get("ent", 0.0),
        reduce={"token": biv.LOSS_TOKEN_MEAN, "seq": biv.LOSS_SEQ_MEAN, "sum": biv.LOSS_SUM}[c["reduce"]],
        norm=st["norm"])
    if c["op"] == "tokens":
        biv.biv_policy_loss(d, st["lp"], st["dlp"])
        return {**st["parts"], "dlp": st["dlp"]}
    biv.biv_policy_loss_logits(d, st["logits"], st["target"], st["lp_out"], st["ent_out"], st["dz"],
                               inv_temp=1.0 / c["temp"])
    return {**st["parts"], "lp": st["lp_out"], "entropy": st["ent_out"], "dz": st["dz"]}


def _own_adamw(st):
    st["opt"].step()
    return _adamw_outputs(st, st["opt"].norm)


def _adamw_outputs(st, norm):
    out = {"w": st["w"], "m": st["m"], "v": st["v"], "step": st["step"][:1]}
    if st["p"] is not None:
        out["p"] = st["p"]
    if st["case"]["state"] == "e4m3":
        out |= {"ms": st["ms"], "vs": st["vs"]}
    if st["case"]["clip"]:
        out["norm"] = norm[:1]
    return out


def _plain_loss(st):
    c, T = st["case"], st["T"]
    gamma = c.get("ent", 0.0)
    counted, seq = _counted(st)
    if c["op"] == "tokens":
        lp, H = st["lp"], None
    else:
        x = st["logits"].float() * (1.0 / c["temp"])
        m = x.amax(1, keepdim=True)
        e = (x - m).exp()
        s = e.sum(1, keepdim=True)
        hit = st["target"].long().clamp(0, c["V"] - 1)[:, None]
        lp = ((x.gather(1, hit) - m) - s.log())[:, 0]
        p = e.div_(s)
        H = s.log()[:, 0] - (p * (x - m)).sum(1)
    A = st["adv"] if c["adv"] == "tok" else st["adv"][seq]
    lens = torch.zeros(c["nseq"], device=DEV).index_add_(0, seq, counted.float())
    N = lens.sum()
    if c["reduce"] == "token":
        w = counted / N.clamp_min(1)
    elif c["reduce"] == "seq":
        w = counted / (lens.clamp_min(1)[seq] * (lens > 0).sum().clamp_min(1))
    else:
        w = counted / st["norm"]
    zero = torch.zeros((), device=DEV)
    gap = lp - st["old_lp"]
    r = gap.clamp(-20, 20).exp()
    u, cl = -A * r, -A * r.clamp(1 - c["clip_lo"], 1 + c["clip_hi"])
    pg, live = torch.maximum(u, cl), u >= cl
    if c.get("dual", 0.0):
        top = -A * c["dual"]
        over = (A < 0) & (pg > top)
        pg, live = torch.where(over, top, pg), live & ~over
    dlp = torch.where(live & (gap.abs() < 20), -A * r, zero)
    kl = torch.zeros(T, device=DEV)
    if c["kl"]:
        far = st["ref_lp"] - lp
        q = far.clamp(-20, 20)
        kl = q.exp() - q - 1
        dlp = dlp + c["kl"] * torch.where(far.abs() < 20, 1 - q.exp(), zero)
    keep = lambda t: torch.where(counted, t, zero)  # noqa: E731
    dlp = keep(w * dlp)
    ent = H if H is not None else torch.zeros(T, device=DEV)
    n1 = N.clamp_min(1)
    lin = gap.clamp(-20, 20)
    sums = [keep(w * (pg + c["kl"] * kl - gamma * ent)), keep(w * pg), keep(w * kl), keep(w * ent)]
    stats = [t.double().sum() for t in sums]
    stats += [keep((~live).float()).sum() / n1, keep(r - 1 - lin).double().sum() / n1,
              keep(gap.abs()).amax(), N]
    stats = torch.stack([t.float() for t in stats])
    if c["op"] == "tokens":
        return {**_parts(stats), "dlp": dlp}
    it = 1.0 / c["temp"]
    dz = p * (-it * dlp)[:, None]
    if gamma:
        logp = (x - m) - s.log()
        dz = dz + p * (logp + H[:, None]) * (it * gamma * w)[:, None]
    dz.scatter_add_(1, hit, (it * dlp)[:, None])
    dz = torch.where(counted[:, None], dz, zero)
    return {**_parts(stats), "lp": keep(lp), "entropy": keep(H), "dz": dz.to(_dtype(c["dz"]))}


def _counted(st):
    """Which rows count, and each row's sequence (rows of no sequence: clamped, and not counted)."""
    start, T = st["seq_start"].long(), st["T"]
    row = torch.arange(T, device=DEV)
    seq = torch.searchsorted(start, row, right=True) - 1
    n = start.numel() - 1
    counted = (seq >= 0) & (seq < n)
    if st["mask"] is not None:
        counted = counted & (st["mask"] != 0)
    return counted, seq.clamp(0, n - 1)


def _mix(x):
    """A 32-bit integer hash (xor-shifts and two odd multipliers; bijective)."""
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & M32
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & M32
    return x ^ (x >> 16)


def _random_bits(total, seed, step):
    """Two words of random bits per element: for the states, and for the parameter."""
    i = torch.arange(total, device=DEV)
    key = _mix((seed + step.long() * 0x9E3779B9) & M32)
    h = _mix((((i & M32) ^ key) + (i >> 32) * 0x85EBCA6B) & M32)
    return h, _mix(h ^ 0x9E3779B9)


def _to_e4m3(x, bits):
    """Blocks of 128 as (e4m3 values, scales); bits: 16 random bits an element, or None (nearest)."""
    x = x.view(-1, BLOCK)
    a = x.abs().amax(1, keepdim=True).clamp_min(2.0 ** -100)
    y = x.abs() * (448 / a)
    if bits is not None:
        b = bits.view(-1, BLOCK)
        big = ((y.view(torch.int32) + (b << 4).int()) & ~0xFFFFF).view(torch.float32)
        small = (y * 512 + b.float() / 65536).floor() / 512
        y = torch.where(y < 2.0 ** -6, small, big)
    return torch.copysign(y.clamp_max(448), x).to(torch.float8_e4m3fn), (a / 448).view(-1)


def _plain_adamw(st):
    c = st["case"]
    b1, b2 = st["betas"]
    norm = coef = None
    g = st["g"].float()
    if c["clip"]:
        norm = g.double().square().sum().sqrt().float()
        coef = (c["clip"] / (norm + 1e-6)).clamp_max(1)
        g = g * coef
    st["step"][0] += 1
    t = st["step"][0].double()
    bc1, rbc2 = (1 - b1 ** t).float(), (1 / (1 - b2 ** t).sqrt()).float()
    w = st["w"].float()
    if c["state"] == "f32":
        m, v = st["m"], st["v"]
    else:
        m = (st["m"].float().view(-1, BLOCK) * st["ms"][:, None]).view(-1)
        v = (st["v"].float().view(-1, BLOCK) * st["vs"][:, None]).view(-1).square()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    r = v.sqrt()
    lr = st["lr"]
    w = w * torch.where(st["decay"], 1 - lr * c["wd"], torch.ones((), device=DEV))
    w = w - (lr / bc1) * m / (r * rbc2 + st["eps"])
    hs = hp = None
    if c["rounding"] == "stochastic" and (c["state"] == "e4m3" or c["param"] == "bf16"):
        hs, hp = _random_bits(w.numel(), st["seed"], st["step"][0])
    if c["param"] == "bf16":
        if hp is not None:
            w = ((w.view(torch.int32) + (hp & 0xFFFF).int()) & ~0xFFFF).view(torch.float32)
        st["w"].copy_(w)
    else:
        st["w"].copy_(w)
        if st["p"] is not None:
            st["p"].copy_(w)
    if c["state"] == "f32":
        st["m"].copy_(m)
        st["v"].copy_(v)
    else:
        q, s = _to_e4m3(m, None if hs is None else hs & 0xFFFF)
        st["m"].copy_(q.view(-1))
        st["ms"].copy_(s)
        q, s = _to_e4m3(r, None if hs is None else hs >> 16)
        q = torch.where((r.view(-1, BLOCK) > 0) & (q.float() == 0), 2.0 ** -9, q.float())
        st["v"].copy_(q.view(-1).to(torch.float8_e4m3fn))
        st["vs"].copy_(s)
    return _adamw_outputs(st, None if norm is None else norm.view(1))


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    st = prepare(case, seed)
    return _exact_adamw(st) if case["op"] == "adamw" else _exact_loss(st)


def _exact_loss(st):
    """The loss written as a sum over sequences in 64 bits; its gradient by differentiation."""
    c = st["case"]
    f = torch.float64
    start = st["seq_start"].tolist()
    T = st["T"]
    ok = torch.zeros(T, dtype=torch.bool, device=DEV)
    A = torch.zeros(T, dtype=f, device=DEV)
    w = torch.zeros(T, dtype=f, device=DEV)
    spans = [(a, b) for a, b in zip(start, start[1:])]
    mask = torch.ones(T, dtype=torch.bool, device=DEV) if st["mask"] is None else st["mask"].bool()
    ok[start[0]:start[-1]] = True
    ok &= mask
    have = [int(x) for x in torch.stack([mask[a:b].sum() for a, b in spans]).tolist()]
    live = sum(1 for n in have if n)
    for s, (a, b) in enumerate(spans):
        A[a:b] = st["adv"][a:b] if c["adv"] == "tok" else st["adv"][s]
        if have[s]:
            w[a:b] = {"token": 1.0 / sum(have), "seq": 1.0 / (have[s] * live), "sum": 1.0 / st["norm"]}[c["reduce"]]
    it = 1.0 / c.get("temp", 1.0)
    stats = torch.zeros(8, dtype=f, device=DEV)
    outs = {"lp": torch.zeros(T, dtype=f, device=DEV), "entropy": torch.zeros(T, dtype=f, device=DEV)}
    grad = torch.zeros(T, dtype=f, device=DEV) if c["op"] == "tokens" else \
        torch.zeros(T, c["V"], dtype=f, device=DEV)
    step = T if c["op"] == "tokens" else max(1, (1 << 27) // c["V"])
    for a in range(0, T, step):
        rows = torch.nonzero(ok[a:a + step])[:, 0] + a
        if not rows.numel():
            continue
        if c["op"] == "tokens":
            leaf = st["lp"][rows].to(f).requires_grad_(True)
            lp, H = leaf, torch.zeros_like(leaf)
        else:
            leaf = st["logits"][rows].to(f).requires_grad_(True)
            logp = torch.log_softmax(leaf * it, 1)
            lp = logp.gather(1, st["target"][rows].long()[:, None])[:, 0]
            H = -(logp.exp() * logp).sum(1)
        gap = lp - st["old_lp"][rows].to(f)
        ratio = torch.exp(gap.clamp(-20, 20))
        Ar = A[rows]
        bounded = torch.minimum(torch.maximum(ratio, torch.tensor(1.0 - c["clip_lo"], dtype=f, device=DEV)),
                                torch.tensor(1.0 + c["clip_hi"], dtype=f, device=DEV))
        gain = torch.minimum(ratio * Ar, bounded * Ar)
        cut = ratio * Ar > bounded * Ar
        if c.get("dual", 0.0):
            floor = c["dual"] * Ar
            low = (Ar < 0) & (gain < floor)
            gain, cut = torch.where(low, floor, gain), cut | low
        kl = torch.zeros_like(gap)
        if c["kl"]:
            away = (st["ref_lp"][rows].to(f) - lp).clamp(-20, 20)
            kl = torch.expm1(away) - away
        wr = w[rows]
        loss = (wr * (c["kl"] * kl - gain - c.get("ent", 0.0) * H)).sum()
        loss.backward()
        grad[rows] = leaf.grad
        with torch.no_grad():
            flat = gap.clamp(-20, 20)
            stats[0] += loss
            stats[1] -= (wr * gain).sum()
            stats[2] += (wr * kl).sum()
            stats[3] += (wr * H).sum()
            stats[4] += cut.sum()
            stats[5] += (torch.expm1(flat) - flat).sum()
            stats[6] = torch.maximum(stats[6], gap.abs().amax())
            outs["lp"][rows], outs["entropy"][rows] = lp.detach(), H.detach()
    n = max(1, sum(have))
    stats[4] /= n
    stats[5] /= n
    stats[7] = sum(have)
    if c["op"] == "tokens":
        return {**_parts(stats), "dlp": grad}
    return {**_parts(stats), **outs, "dz": grad}


def _exact_adamw(st):
    c = st["case"]
    f = torch.float64
    b1, b2 = st["betas"]
    t = int(st["step"][0]) + 1
    g = st["g"].to(f)
    out = {"step": torch.tensor([t], dtype=torch.int32)}
    if c["clip"]:
        norm = torch.linalg.vector_norm(g)
        out["norm"] = norm.view(1)
        g = g * min(1.0, c["clip"] / (float(norm) + 1e-6))
    m, v = st["m"].float().to(f), st["v"].float().to(f)
    if c["state"] == "e4m3":
        m = m * st["ms"].to(f).repeat_interleave(BLOCK)
        v = (v * st["vs"].to(f).repeat_interleave(BLOCK)) ** 2
    m = torch.lerp(g, m, b1)
    v = torch.lerp(g * g, v, b2)
    lr = float(st["lr"])
    w = st["w"].to(f)
    w = w - lr * c["wd"] * w * st["decay"]
    w = w - lr * (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + st["eps"])
    up = None
    if c["rounding"] == "stochastic":
        i = torch.arange(w.numel(), device=DEV)
        key = _mix(torch.tensor((st["seed"] + t * 0x9E3779B9) & M32, device=DEV))
        up = _mix(i ^ key)
    if c["param"] == "bf16" and up is not None:
        w = _on_grid(w, _mix(up ^ 0x9E3779B9) & 0xFFFF, 8, -126)
    out["w"] = w
    if st["p"] is not None:
        out["p"] = w
    if c["state"] == "f32":
        return {**out, "m": m, "v": v}
    for k, x, bits in (("m", m, None if up is None else up & 0xFFFF),
                       ("v", v.sqrt(), None if up is None else up >> 16)):
        s = torch.clamp(x.abs().view(-1, BLOCK).amax(1), min=2.0 ** -100) / 448
        q = _on_grid(x / s.repeat_interleave(BLOCK), bits, 4, -6)
        if k == "v":
            q = torch.where((x > 0) & (q == 0), torch.full_like(q, 2.0 ** -9), q)
        out[k], out[k + "s"] = q.clamp(-448, 448), s
    return out


def _on_grid(x, bits, digits, low):
    """x on the grid of `digits` significant binary digits, exponents from `low` up: to the nearest
    (ties to even), or up with a chance equal to the part cut off (bits: 16 random bits)."""
    e = torch.frexp(x)[1] - 1
    step = torch.ldexp(torch.ones_like(x), torch.clamp(e, min=low) - (digits - 1))
    k = x.abs() / step
    k = torch.round(k) if bits is None else torch.floor(k + bits.to(x.dtype) / 65536)
    return torch.copysign(k * step, x)

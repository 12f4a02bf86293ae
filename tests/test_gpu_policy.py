"""The clipped policy loss against the float64 oracle, from logprobs and from
logits: sizes from one row and one logit up, odd sizes and strides, masks that
leave a row, a sequence or everything empty, padded targets and rows, NaN and
infinities in rows that do not count, in-place gradients, other streams,
captured replays, and the same bits for a row in any batch.

Tolerances.  p = 2^y / S: y = fma(x, c, -M) with |x c| up to Y is off by half
an ulp (Y 2^-24) plus c's rounding (Y 2^-24), ex2.approx by 2^-22, S by the
depth of its sums (32 + 5 + 8 + 5 additions, 50 2^-24) and 2^-22; at Y <= 96
(|logits| <= 60, temperature >= 0.8) that is ln2 192 2^-24 + 2^-21 + 50 2^-24
< 1.2e-5 relative.  lp and H are off by that (absolute, times H's mean |log p|
for H), lp - old by lp's rounding too, so r and dlp by < 3e-5 relative.  A
bf16 result adds half a step, 2^-8."""
import math

import numpy as np
import pytest
import torch

import synth
from oracle import trainer as tr
from oracle.codecs import bf16_to_f32

pytestmark = pytest.mark.gpu
REL = 3e-5
GAPS = np.array([-25.0, -0.9, -0.3, -0.1, 0.0, 0.05, 0.1, 0.4, 1.5, 21.0])   # none near ln(1 +- clip)
REDUCE = {"token": 0, "seq": 1, "sum": 2}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def B():
    from invariant_forward_bitwise_gb300 import biv, build
    build.build()
    biv.load()
    return biv


def f64(t):
    t = t.detach().cpu()
    if t.dtype == torch.bfloat16:
        return bf16_to_f32(t.contiguous().view(torch.int16).numpy().view(np.uint16)).astype(np.float64)
    return t.numpy().astype(np.float64)


def bits(t):
    return t.detach().contiguous().view(-1).view(torch.uint8).cpu().numpy()


def same(a, b):
    return np.array_equal(bits(a), bits(b))


def dev(x, dt=np.float32):
    return torch.from_numpy(np.ascontiguousarray(x).astype(dt)).cuda()


def workspace(B, T, nseq):
    return torch.full((B.biv_policy_loss_workspace(T, nseq),), 0xA5, dtype=torch.uint8, device="cuda")


STARTS = {"one": lambda T: [0, T], "many": lambda T: sorted({0, T // 7, T // 3, T // 2, T}),
          "empty": lambda T: [0, 0, T // 2, T // 2, T], "inner": lambda T: [T // 5, T // 2, max(T // 2, T - 2)],
          "none": lambda T: [0], "rows": lambda T: list(range(T + 1))}


def rows_case(g, lp, start, kw):
    """What goes with T logprobs: the sampling and reference policies' at known
    distances, advantages, a mask; and the weights they amount to."""
    T, n = len(lp), len(start) - 1
    c = dict(T=T, start=start, kw=kw, lp=lp)
    c["old"] = (lp - g.choice(GAPS, T)).astype(np.float32)
    c["ref"] = (lp + g.choice([-30.0, -0.5, -0.01, 0.0, 0.2, 3.0, 22.0], T)).astype(np.float32)
    c["adv"] = g.standard_normal(T if kw.get("per_row") else n).astype(np.float32)
    c["mask"] = None
    if kw.get("mask", True):
        c["mask"] = ((g.random(T) < 0.85) * g.integers(1, 256, T)).astype(np.uint8)
    c["w"], seq = tr.row_weights(T, start, c["mask"], kw.get("reduce", "token"), 3.0)
    A = c["adv"] if kw.get("per_row") else np.append(c["adv"], 0)[np.where(seq >= 0, seq, n)]
    c["A"] = A.astype(np.float64)
    return c


def oracle_loss(c, H=None, lp=None):
    kw = c["kw"]
    beta = kw.get("beta", 0.0)
    return tr.policy_loss(c["lp"] if lp is None else lp, c["w"], c["A"],
                          None if kw.get("no_old") else c["old"].astype(np.float64),
                          c["ref"].astype(np.float64) if beta else None, 0.2, 0.28, kw.get("dual", 0.0), beta,
                          kw.get("gamma", 0.0), H)


def sizes(c, H=None):
    """The sizes of what is summed, for the tolerances: (stats [4], dlp [T])."""
    kw, lp, w, aA = c["kw"], c["lp"], c["w"], np.abs(c["A"])
    r = np.ones_like(lp) if kw.get("no_old") else np.exp(np.clip(lp - c["old"], -20, 20))
    beta = kw.get("beta", 0.0)
    e = np.clip(c["ref"] - lp, -20, 20) if beta else np.zeros_like(lp)
    pg, kl = aA * (r + 2), np.exp(e) + np.abs(e) + 1
    h = np.abs(H) + 1 if H is not None else np.zeros_like(lp)
    stats = [np.sum(w * x) for x in (pg + beta * kl + kw.get("gamma", 0.0) * h, pg, kl, h)]
    return np.array(stats), w * (aA * r + beta * (np.exp(e) + 1))


def check_stats(got, ref, scale):
    """Sums to REL of the sum of their terms' sizes; shares, largest gap and count."""
    assert np.all(np.abs(got[:4] - ref[:4]) <= REL * scale), (got, ref, scale)
    assert abs(got[4] - ref[4]) <= 1e-6 and got[7] == ref[7]
    assert abs(got[5] - ref[5]) <= REL * (abs(ref[5]) + 1)
    assert abs(got[6] - ref[6]) <= REL * (1 + ref[6])


def desc(B, c, stats, ws):
    kw = c["kw"]
    beta = kw.get("beta", 0.0)
    keep = [dev(c["start"], np.int32), dev(c["adv"]), None if c["mask"] is None else dev(c["mask"], np.uint8),
            None if kw.get("no_old") else dev(c["old"]), dev(c["ref"]) if beta else None, stats, ws]
    d = B.policy_desc(keep[0], keep[1], stats, ws, T=c["T"], mask=keep[2], old_lp=keep[3], ref_lp=keep[4],
                      clip_lo=0.2, clip_hi=0.28, dual_clip=kw.get("dual", 0.0), kl_coef=beta,
                      ent_coef=kw.get("gamma", 0.0), reduce=REDUCE[kw.get("reduce", "token")], norm=3.0)
    d.keep = keep                                   # the tensors live as long as the descriptor
    return d


@pytest.mark.parametrize("T,starts,kw", [
    (1, "one", dict(mask=False)), (1, "empty", dict(reduce="seq")), (5, "rows", dict(reduce="seq")),
    (31, "many", dict(reduce="sum", dual=3.0)), (1024, "inner", dict(beta=0.1, per_row=True)),
    (1025, "many", dict(reduce="seq", beta=0.1, dual=1.2)), (4099, "empty", dict(no_old=True)),
    (2000, "rows", dict(beta=0.02, reduce="seq")), (9000, "rows", dict(beta=0.02)), (70001, "many", dict(reduce="seq", per_row=True, beta=0.5)),
    (7, "none", dict(per_row=True)), (7, "none", dict()), (6000, "many", dict(mask=False, reduce="seq")),
    (5003, "none", dict(per_row=True)), (140000, "one", dict(reduce="seq"))])
def test_policy_loss(B, T, starts, kw):
    g = synth.rng(T)
    lp = (-g.exponential(1.0, T)).astype(np.float32).astype(np.float64)
    c = rows_case(g, lp, STARTS[starts](T), kw)
    want, want_dlp = oracle_loss(c)
    # rows that do not count hold NaN
    junk = dev(lp)
    junk[torch.from_numpy(c["w"] == 0).cuda()] = float("nan")
    stats = torch.full((8,), float("nan"), device="cuda")
    d = desc(B, c, stats, workspace(B, T, len(c["start"]) - 1))
    dlp = torch.full((T + 3,), 7.0, device="cuda")
    B.biv_policy_loss(d, junk, dlp[:T])
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    scale, size = sizes(c)
    check_stats(f64(stats), want, scale)
    got = f64(dlp)
    assert np.all(np.abs(got[:T] - want_dlp) <= REL * size) and np.all(got[T:] == 7.0)
    assert np.all(got[:T][c["w"] == 0] == 0)
    # again on a used workspace, and statistics alone on another stream: the same bits
    s2, d2 = torch.empty(8, device="cuda"), torch.empty(T, device="cuda")
    d.stats = s2.data_ptr()
    B.biv_policy_loss(d, junk, d2)
    torch.cuda.synchronize()
    assert same(s2, stats) and same(d2, dlp[:T])
    s2.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.biv_policy_loss(d, junk, None, stream=side)
    side.synchronize()
    assert same(s2, stats)


def logits_case(T, V, pad, col, zt, dzt, starts, kw):
    g = synth.rng(1000 * T + V)
    it = kw.get("it", 1.0)
    ld = V + pad + col
    zb = torch.from_numpy((g.standard_normal((T, ld)) * 3).astype(np.float32)).clamp_(-60, 60)
    if V >= 16:
        zb[:, col + 5] = -math.inf                 # a forbidden token
        zb[::2, col + V - 1] = 9.0
    zb = zb.to(TYPES[zt]).cuda()
    z = zb[:, col:col + V]
    target = g.integers(0, V, T)
    target[target == 5] = 0
    target[0] = V - 1
    zz = f64(z)
    lp, H, p, logp = tr.token_logprobs(zz, target, it)
    c = rows_case(g, lp, STARTS[starts](T), kw)
    junk = torch.from_numpy(c["w"] == 0).cuda()
    zb[junk] = float("nan")                        # rows that do not count are not read
    tgt = dev(target, np.int32)
    tgt[junk] = -100
    return c | dict(V=V, it=it, zb=zb, z=z, zz=zz, target=target, tgt=tgt, H=H, p=p, logp=logp, col=col, ld=ld,
                    dzt=dzt)


def run_logits(B, c, dz="new", z=None):
    T, V = c["T"], c["V"]
    stats = torch.full((8,), float("nan"), device="cuda")
    d = desc(B, c, stats, workspace(B, T, len(c["start"]) - 1))
    lp, ent = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    buf = None
    if isinstance(dz, str):
        buf = torch.full((T, c["ld"]), 7.0, dtype=TYPES[c["dzt"]], device="cuda")
        dz = buf[:, c["col"]:c["col"] + V]
    B.biv_policy_loss_logits(d, c["z"] if z is None else z, c["tgt"], lp, ent, dz, inv_temp=c["it"])
    return dict(stats=stats, lp=lp, ent=ent, dz=dz, buf=buf, desc=d)


def dz_size(c):
    """The sizes of the terms of each element of dz."""
    _, dlp = sizes(c, c["H"])
    hit = np.zeros_like(c["p"])
    hit[np.arange(c["T"]), c["target"]] = 1
    logp = np.where(c["p"] > 0, np.abs(np.where(c["p"] > 0, c["logp"], 0)), 0)
    gamma = c["kw"].get("gamma", 0.0)
    return c["it"] * (dlp[:, None] * (hit + c["p"]) +
                      gamma * c["w"][:, None] * c["p"] * (logp + c["H"][:, None] + 1))


@pytest.mark.parametrize("T,V,pad,col,zt,dzt,starts,kw", [
    # T, V, row padding, first column, logits, gradient, starts, options
    (1, 1, 0, 0, "f32", "f32", "one", dict(mask=False)),
    (3, 2, 1, 0, "bf16", "f32", "one", dict()),
    (2, 3, 0, 1, "f32", "bf16", "one", dict(gamma=0.1)),
    (9, 7, 0, 0, "bf16", "bf16", "many", dict(it=1.25)),
    (13, 33, 2, 3, "f32", "f32", "inner", dict(beta=0.1, gamma=0.05)),
    (6, 1023, 0, 0, "f32", "f32", "one", dict(gamma=0.05)),
    (7, 1024, 3, 1, "f32", "f32", "many", dict(gamma=0.05)),     # whole groups, no row aligned
    (7, 2048, 1, 5, "bf16", "bf16", "many", dict(gamma=0.05)),
    (5, 1025, 0, 0, "bf16", "f32", "empty", dict(dual=1.5)),
    (40, 4096, 0, 0, "f32", "f32", "many", dict(beta=0.1)),
    (4, 4096, 8, 0, "bf16", "bf16", "rows", dict(it=0.8, reduce="seq")),
    (11, 32003, 0, 0, "f32", "f32", "many", dict(gamma=0.01, it=1.25)),
    (3, 50257, 3, 0, "bf16", "bf16", "one", dict(beta=0.02)),
    (170, 40963, 5, 0, "f32", "bf16", "many", dict(gamma=0.01, reduce="sum")),  # more rows than fit at once
    (9, 5000, 1, 1, "f32", "f32", "many", dict(gamma=0.01)),      # every offset from 16 bytes in turn
    (9, 5000, 1, 1, "f32", "bf16", "many", dict(gamma=0.01)),
    (9, 9000, 1, 3, "bf16", "bf16", "many", dict(gamma=0.01)),
    (9, 9000, 1, 1, "bf16", "f32", "many", dict(gamma=0.01)),
    (2, 151936, 0, 0, "f32", "f32", "one", dict(gamma=0.01, beta=0.02)),
    (45, 151936, 0, 0, "f32", "bf16", "many", dict(reduce="seq")),
    (2, 262144, 0, 0, "f32", "f32", "one", dict()),
    (1, 262143, 1, 1, "bf16", "f32", "one", dict(mask=False, gamma=0.01))])
def test_policy_loss_logits(B, T, V, pad, col, zt, dzt, starts, kw):
    c = logits_case(T, V, pad, col, zt, dzt, starts, kw)
    o = run_logits(B, c)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    on = c["w"] > 0
    want, dlp = oracle_loss(c, c["H"])
    dz = tr.policy_dz(c["zz"], c["target"], dlp, c["w"], kw.get("gamma", 0.0), c["it"])
    check_stats(f64(o["stats"]), want, sizes(c, c["H"])[0])
    for got, exp in ((o["lp"], c["lp"]), (o["ent"], c["H"])):
        got = f64(got)
        assert np.all(np.abs(got - exp)[on] <= REL * (1 + np.abs(exp[on]))) and np.all(got[~on] == 0)
    half = 2.0 ** -8 if dzt == "bf16" else 2.0 ** -24
    got = f64(o["dz"])
    # results below 2^-126 flush to zero; a p that small is off by no more than it
    assert np.all(np.abs(got - dz) <= (REL + half) * dz_size(c) + 1e-37)
    assert np.all(got[~on] == 0)
    outside = o["buf"].float().cpu().numpy()
    assert np.all(outside[:, :col] == 7.0) and np.all(outside[:, col + V:] == 7.0)
    # a second run, on another stream: the same bits
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2 = run_logits(B, c)
    side.synchronize()
    for k in ("stats", "lp", "ent", "dz"):
        assert same(o2[k], o[k]), k
    # no gradient asked for: the same values; and the gradient over the logits themselves
    o3 = run_logits(B, c, dz=None)
    torch.cuda.synchronize()
    for k in ("stats", "lp", "ent"):
        assert same(o3[k], o[k]), k
    if zt == dzt:
        zb = c["zb"].clone()
        zi = zb[:, col:col + V]
        o4 = run_logits(B, c, dz=zi, z=zi)
        torch.cuda.synchronize()
        for k in ("stats", "lp", "ent", "dz"):
            assert same(o4[k], o[k]), k
        assert same(zb[:, :col], c["zb"][:, :col]) and same(zb[:, col + V:], c["zb"][:, col + V:])


@pytest.mark.parametrize("V,zt", [(4096, "f32"), (32003, "f32"), (131072, "bf16")])
def test_a_row_has_the_same_bits_in_any_batch(B, V, zt):
    """Rows spread over more or fewer CTAs, at another alignment, among other
    rows: lp, entropy and (weights equal) dz keep their bits."""
    c = logits_case(90, V, 0, 0, zt, zt, "one", dict(mask=False, gamma=0.01, reduce="sum"))
    o = run_logits(B, c)
    for rows in (slice(4, 5), slice(10, 13), slice(0, 60)):
        n = rows.stop - rows.start
        buf = torch.empty(n, V + 3, dtype=c["zb"].dtype, device="cuda")
        z = buf[:, 1:V + 1]
        z.copy_(c["z"][rows])
        part = c | dict(T=n, start=[0, n], z=z, tgt=c["tgt"][rows].contiguous(), old=c["old"][rows],
                        ref=c["ref"][rows])
        q = run_logits(B, part)
        torch.cuda.synchronize()
        for k in ("lp", "ent", "dz"):
            assert same(q[k], o[k][rows]), (k, rows)


def test_logits_gradient_by_differences(B):
    """The kernel's dz along random directions against central differences of
    the oracle's loss (step 2^-12: truncation 2^-24 f''' / 6)."""
    c = logits_case(6, 300, 0, 0, "f32", "f32", "many", dict(mask=False, beta=0.1, gamma=0.05, per_row=True))
    c["zb"][:, 5] = -1.0
    c["zz"] = f64(c["z"])
    lp, c["H"], c["p"], c["logp"] = tr.token_logprobs(c["zz"], c["target"])
    c["lp"], c["old"], c["ref"] = lp, (lp - 0.05).astype(np.float32), (lp + 0.2).astype(np.float32)
    dz = f64(run_logits(B, c)["dz"])
    g = synth.rng(8)

    def loss(zz):
        a, H, _, _ = tr.token_logprobs(zz, c["target"])
        return oracle_loss(c, H, a)[0][0]
    for _ in range(4):
        u, h = g.standard_normal(c["zz"].shape), 2.0 ** -12
        fd = (loss(c["zz"] + h * u) - loss(c["zz"] - h * u)) / (2 * h)
        assert abs(fd - np.sum(dz * u)) <= REL * np.sum(dz_size(c) * np.abs(u)) + 1e-6


def test_bad_targets_bad_starts_and_nothing_left(B):
    c = logits_case(8, 100, 0, 0, "f32", "f32", "one", dict(mask=False))
    c["tgt"][3] = 100
    o = run_logits(B, c)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 2 and math.isnan(o["lp"][3].item()) and math.isnan(o["stats"][0].item())
    assert B.biv_poll_error() == 0 and not torch.isnan(o["lp"][torch.arange(8) != 3]).any()
    # every row masked: zeros, though logits and targets are rubbish
    c["mask"], c["zb"][:] = np.zeros(8, np.uint8), float("inf")
    o = run_logits(B, c)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    assert not any(bool(o[k].any()) for k in ("stats", "lp", "ent", "dz"))
    # a row of -inf alone has no distribution
    c = logits_case(4, 40, 0, 0, "f32", "f32", "one", dict(mask=False))
    c["zb"][2] = -math.inf
    o = run_logits(B, c)
    torch.cuda.synchronize()
    assert math.isnan(o["lp"][2].item()) and not torch.isnan(o["lp"][[0, 1, 3]]).any()
    # starts that leave [0, T] or go back are reported
    for start in ([0, 5], [-1, 4], [0, 3, 2, 4]):
        ws, stats = workspace(B, 4, len(start) - 1), torch.zeros(8, device="cuda")
        st, adv = dev(start, np.int32), torch.ones(len(start) - 1, device="cuda")
        d = B.policy_desc(st, adv, stats, ws, T=4)
        B.biv_policy_loss(d, torch.zeros(4, device="cuda"), torch.empty(4, device="cuda"))
        assert B.biv_poll_error() == 2 and B.biv_poll_error() == 0


@pytest.mark.parametrize("T,V,starts", [
    (130, 300, "many"), (300, 300, "empty"), (2000, 9000, "many"), (1500, 5000, "rows"), (4096, 2100, "inner"),
    (5000, 300, "rows"), (40, 5000, "none")])
def test_sums_are_those_of_the_logprobs(B, T, V, starts):
    """However the sums of a call from logits are taken (by its last CTA, by a
    kernel behind it): the bits that its lp alone give."""
    c = logits_case(T, V, 0, 0, "f32", "bf16", starts, dict(beta=0.05, reduce="seq"))
    o = run_logits(B, c)
    stats = torch.full((8,), float("nan"), device="cuda")
    d = desc(B, c, stats, workspace(B, T, len(c["start"]) - 1))
    B.biv_policy_loss(d, o["lp"])
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    keep = [0, 1, 2, 4, 5, 6, 7]
    assert same(stats[keep], o["stats"][keep])
    check_stats(f64(o["stats"]), oracle_loss(c, c["H"])[0], sizes(c, c["H"])[0])


def test_masks_of_any_alignment(B):
    """Counts of sequences that start and end at any byte, masks of any byte values."""
    g = synth.rng(77)
    T = 5000
    for off in range(0, 20, 3):
        start = np.sort(np.concatenate([[0, T], g.integers(0, T + 1, 29), 100 + np.arange(20)])).astype(np.int32)
        mask = (g.random(T) < 0.5) * g.integers(1, 256, T)
        buf = torch.full((T + 40,), 255, dtype=torch.uint8, device="cuda")
        buf[off:off + T] = dev(mask, np.uint8)
        n = len(start) - 1
        stats, dlp = torch.empty(8, device="cuda"), torch.empty(T, device="cuda")
        d = B.policy_desc(dev(start, np.int32), torch.ones(n, device="cuda"), stats, workspace(B, T, n), T=T,
                          mask=buf[off:off + T], reduce=1)
        B.biv_policy_loss(d, torch.zeros(T, device="cuda"), dlp)
        torch.cuda.synchronize()
        w, _ = tr.row_weights(T, start, mask, "seq", 1.0)
        assert stats[7] == np.count_nonzero(w)
        assert np.all(np.abs(f64(dlp) + w) <= 3 * 2.0 ** -24 * w)


def test_no_rows_and_temporaries(B):
    """No row at all: statistics of zeros; a descriptor keeps the tensors that only
    it was given."""
    z = lambda *n: torch.zeros(*n, device="cuda")  # noqa: E731
    ws = workspace(B, 0, 2)
    for call in ("lp", "logits"):
        stats = torch.full((8,), float("nan"), device="cuda")
        d = B.policy_desc(torch.zeros(3, dtype=torch.int32, device="cuda"), z(2), stats, ws, T=0)
        if call == "lp":
            B.biv_policy_loss(d, z(0), z(0))
        else:
            B.biv_policy_loss_logits(d, z(0, 5), torch.zeros(0, dtype=torch.int32, device="cuda"), z(0), z(0), z(0, 5))
        torch.cuda.synchronize()
        assert torch.all(stats == 0)
    T, stats = 600, torch.empty(8, device="cuda")
    d = B.policy_desc(torch.tensor([0, T], dtype=torch.int32, device="cuda"), z(1) + 2.0, stats, workspace(B, T, 1),
                      T=T, mask=(torch.arange(T, device="cuda") % 2 == 0), old_lp=z(T) - 1.0)
    junk = [torch.full((n,), 7.0, device="cuda") for n in (1, 1, 2, T, T, 4 * T) for _ in range(4)]
    dlp = torch.empty(T, device="cuda")
    B.biv_policy_loss(d, z(T) - 1.0, dlp)
    torch.cuda.synchronize()
    assert stats[7] == T // 2 and torch.all(dlp[::2] == -2.0 / (T // 2)) and torch.all(dlp[1::2] == 0) and junk


def test_captured_policy_loss(B):
    """A replay reads new inputs and gives the bits of an eager call."""
    c = logits_case(37, 5000, 0, 0, "f32", "bf16", "many", dict(gamma=0.01, beta=0.02))
    o = run_logits(B, c)
    torch.cuda.synchronize()
    outs = [o["stats"], o["lp"], o["ent"], o["dz"]]
    want = [x.clone() for x in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.biv_policy_loss_logits(o["desc"], c["z"], c["tgt"], o["lp"], o["ent"], o["dz"], inv_temp=1.0)
    for x in outs:
        x.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(want, outs))
    c["z"].copy_(torch.where(torch.isnan(c["z"]), c["z"], c["z"] * 0.5))
    g.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in outs]
    o2 = run_logits(B, c)
    torch.cuda.synchronize()
    assert all(same(a, o2[k]) for a, k in zip(got, ("stats", "lp", "ent", "dz")))
    assert not same(got[1], want[1])


def test_first_call_of_a_shape_inside_a_capture(B):
    c = logits_case(5, 777, 0, 0, "bf16", "f32", "many", dict(gamma=0.01))
    stats = torch.empty(8, device="cuda")
    d = desc(B, c, stats, workspace(B, 5, len(c["start"]) - 1))
    lp, ent, dz = torch.empty(5, device="cuda"), torch.empty(5, device="cuda"), torch.empty(5, 777, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.biv_policy_loss_logits(d, c["z"], c["tgt"], lp, ent, dz)
    g.replay()
    o = run_logits(B, c)
    torch.cuda.synchronize()
    assert same(dz, o["dz"]) and same(stats, o["stats"]) and same(lp, o["lp"])


def test_offsets_beyond_32_bits(B):
    """33000 rows of 131072 bf16 logits (more than 2^32 of them), gradient in
    place: the first and last rows as in a small call."""
    T, V = 33000, 131072
    c = logits_case(6, V, 0, 0, "bf16", "bf16", "one", dict(mask=False, reduce="sum"))
    small = run_logits(B, c)
    big = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 2, T - 3, T - 2, T - 1]
    for i, r in enumerate(rows):
        big[r] = c["z"][i]
    wide = dict(c, T=T, start=[0, T], V=V)
    idx = np.zeros(T, np.int64)
    for i, r in enumerate(rows):
        idx[r] = i
    wide["old"], wide["ref"] = c["old"][idx], c["ref"][idx]
    wide["tgt"] = c["tgt"][torch.from_numpy(idx).cuda()].contiguous()
    wide["mask"] = np.zeros(T, np.uint8)
    wide["mask"][rows] = 1
    o = run_logits(B, wide, dz=big, z=big)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    for i, r in enumerate(rows):
        assert same(big[r], small["dz"][i]) and same(o["lp"][r:r + 1], small["lp"][i:i + 1]), r
    assert not bool(big[5000].any()) and not bool(big[T - 4].any())


def test_binding_refuses(B):
    start, adv = dev([0, 4], np.int32), torch.ones(1, device="cuda")
    ws, stats, x = workspace(B, 4, 1), torch.zeros(8, device="cuda"), torch.zeros(4, device="cuda")
    good = dict(seq_start=start, adv=adv, stats=stats, workspace=ws, T=4)
    B.policy_desc(**good)
    for kw in (dict(seq_start=start.long()), dict(seq_start=start.cpu()), dict(adv=torch.ones(3, device="cuda")),
               dict(adv=adv.double()), dict(mask=torch.ones(3, dtype=torch.uint8, device="cuda")),
               dict(mask=torch.ones(4, device="cuda")), dict(old_lp=x[::2]), dict(ref_lp=x.half()),
               dict(stats=stats[:7]), dict(seq_start=start[:0])):
        with pytest.raises(ValueError):
            B.policy_desc(**(good | kw))
    d = B.policy_desc(**good)
    for lp, dlp in ((x[:3], None), (x.cpu(), None), (x, x.double()), (torch.zeros(8, device="cuda")[::2], None)):
        with pytest.raises(ValueError):
            B.biv_policy_loss(d, lp, dlp)
    z = torch.zeros(4, 10, device="cuda")
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    y = torch.zeros(4, device="cuda")
    for kw in (dict(logits=z.half()), dict(logits=z[:3]), dict(logits=z.t().contiguous().t()), dict(target=t.long()),
               dict(dz=z.double()), dict(dz=torch.zeros(4, 9, device="cuda")),
               dict(dz=torch.zeros(60, device="cuda").as_strided((4, 10), (8, 1)))):
        a = dict(logits=z, target=t, lp=x, entropy=y, dz=None) | kw
        with pytest.raises((ValueError, B.BivError)):
            B.biv_policy_loss_logits(d, **a)


@pytest.mark.parametrize("zt", ["f32", "bf16"])
@pytest.mark.parametrize("low", [-math.inf, "lowest", -1e31])
def test_masked_logits(B, zt, low):
    """Whole groups and single logits masked by -inf or by a low value, in rows
    of which a few logits are left, down to one: p = 0 there, and the rest as
    if the masked ones were not in the row."""
    T, V = 5, 3000
    c = logits_case(T, V, 0, 0, zt, zt, "one", dict(mask=False, gamma=0.05, beta=0.1))
    low = torch.finfo(TYPES[zt]).min if low == "lowest" else low
    z = c["z"]
    keep = [list(range(V)), list(range(0, V, 7)), list(range(1024, 2048)), [2500, 2999], [17]]
    for t, k in enumerate(keep):
        on = torch.zeros(V, dtype=torch.bool, device="cuda")
        on[torch.tensor(k, device="cuda")] = True
        z[t] = torch.where(on, torch.nan_to_num(z[t], neginf=-2.0), torch.full_like(z[t], low))
        c["target"][t] = k[-1]
    c["tgt"] = dev(c["target"], np.int32)
    c["zz"] = np.where(f64(z) <= -1e30, -np.inf, f64(z))
    with np.errstate(all="ignore"):
        c["lp"], c["H"], c["p"], c["logp"] = tr.token_logprobs(c["zz"], c["target"])
    c["old"], c["ref"] = (c["lp"] - 0.05).astype(np.float32), (c["lp"] + 0.2).astype(np.float32)
    o = run_logits(B, c)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    want, dlp = oracle_loss(c, c["H"])
    with np.errstate(all="ignore"):
        dz = tr.policy_dz(c["zz"], c["target"], dlp, c["w"], 0.05)
    got = f64(o["dz"])
    half = 2.0 ** -8 if zt == "bf16" else 2.0 ** -24
    assert np.all(np.abs(got - dz) <= (REL + half) * dz_size(c) + 1e-37)
    assert np.all(got[f64(z) <= -1e30] == 0)
    assert np.all(np.abs(f64(o["lp"]) - c["lp"]) <= REL * (1 + np.abs(c["lp"])))
    assert np.all(np.abs(f64(o["ent"]) - c["H"]) <= REL * (1 + c["H"]))
    check_stats(f64(o["stats"]), want, sizes(c, c["H"])[0])


@pytest.mark.parametrize("size", [1e3, 1e5, 1e7, -1e7])
@pytest.mark.parametrize("it", [1.0, 1.25, 0.77])
def test_large_logits(B, size, it):
    """Rows of logits far from 0.  The products of such logits and 1 / temperature
    (and of their largest) are rounded, by |size it| 2^-24 each, and so are
    exponents to base 2."""
    g = synth.rng(int(abs(size)))
    T, V = 9, 5000
    z = (size + g.standard_normal((T, V)) * 3).astype(np.float32)
    target = g.integers(0, V, T)
    c = dict(T=T, start=[0, T], kw=dict(no_old=True), adv=np.ones(1), mask=None, V=V, it=it, z=dev(z),
             tgt=dev(target, np.int32), col=0, ld=V, dzt="f32", ref=None)
    o = run_logits(B, c)
    torch.cuda.synchronize()
    lp, H, _, _ = tr.token_logprobs(z.astype(np.float64), target, float(np.float32(it)))
    # x and max x, half a step each; the exponents to base 2, half a step of the
    # largest times ln 2, in the sum and its entropy
    off = 2 * abs(size) * it * 2.0 ** -24 + abs(size) * it * 2.0 ** -24
    assert np.all(np.abs(f64(o["lp"]) - lp) <= off + REL * (1 + np.abs(lp)))


@pytest.mark.parametrize("zt", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_bad_logit_spoils_its_row_only(B, zt, bad):
    c = logits_case(4, 2500, 0, 0, zt, zt, "one", dict(mask=False, gamma=0.05))
    clean = run_logits(B, c)
    c["z"][2, :] = -math.inf
    c["z"][2, 1700] = bad                          # the rest of its group masked
    o = run_logits(B, c)
    torch.cuda.synchronize()
    rows = [0, 1, 3]
    assert math.isnan(o["lp"][2].item()) and math.isnan(o["stats"][0].item())
    assert all(same(o[k][rows], clean[k][rows]) for k in ("lp", "ent", "dz"))


@pytest.mark.parametrize("zt,dzt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("pad,col", [(0, 0), (1, 1), (400, 8)])
def test_a_bad_target_leaves_everything_else(B, zt, dzt, pad, col):
    """Targets from V on, up to and past the end of the row's last group of logits
    (2048 here), and negative ones: the other rows, the padding around dz and what
    lies behind its last row keep their bits."""
    T, V = 7, 1104                                  # (rows of whole 16 bytes, of either type)
    c = logits_case(T, V, pad, col, zt, dzt, "one", dict(mask=False, gamma=0.05, reduce="sum"))
    clean = run_logits(B, c)
    same_type = zt == dzt
    for bad in (V, V + 1, V + col + pad, 2047, 2048, 2 ** 31 - 1, -1, -2 ** 31):
        for row in (0, 3, T - 1):
            b = c | dict(tgt=c["tgt"].clone())
            b["tgt"][row] = bad
            buf = torch.full((T + 2, c["ld"]), 7.0, dtype=TYPES[dzt], device="cuda")
            runs = [(run_logits(B, b, dz=buf[:T, col:col + V]), buf)]
            if same_type:                           # the gradient over the logits
                over = buf.clone()
                over[:T] = c["zb"]
                z = over[:T, col:col + V]
                runs.append((run_logits(B, b, dz=z, z=z), over))
            torch.cuda.synchronize()
            assert B.biv_poll_error() == 2
            keep = torch.arange(T, device="cuda") != row
            for i, (o, mem) in enumerate(runs):
                assert math.isnan(o["lp"][row].item()) and same(o["ent"], clean["ent"])
                assert same(o["lp"][keep], clean["lp"][keep]) and same(o["dz"][keep], clean["dz"][keep])
                around = c["zb"] if i else buf[:0].new_full((T, c["ld"]), 7.0)
                assert same(mem[:T, :col], around[:, :col]) and same(mem[:T, col + V:], around[:, col + V:])
                assert bool((mem[T:] == 7.0).all())


@pytest.mark.parametrize("zt", ["f32", "bf16"])
@pytest.mark.parametrize("low", [-math.inf, "lowest", -1e31])
@pytest.mark.parametrize("old", ["none", "own", "other"])
def test_a_masked_target_has_no_gradient(B, zt, low, old):
    """A target whose logit is masked: dz is 0 there and what the entropy term alone
    gives elsewhere, whatever the old and reference logprobs are; so is dlp from a
    logprob of -inf.
    Other rows keep their bits."""
    T, V, row = 5, 1200, 2
    kw = dict(mask=False, gamma=0.05, reduce="sum", no_old=old == "none", beta=0.1 if old == "other" else 0.0)
    c = logits_case(T, V, 0, 0, zt, "f32", "one", kw)
    clean = run_logits(B, c)
    c["ref"][row] = -math.inf                       # (the reference masks it too)
    t = int(c["target"][row])
    c["zb"][row, t] = torch.finfo(c["zb"].dtype).min if low == "lowest" else low
    if old == "own":
        first = run_logits(B, c)
        torch.cuda.synchronize()
        # (an old logprob of -inf has no difference from -inf: the lowest value in its place)
        c["old"] = np.maximum(first["lp"].cpu().numpy(), -3e38)
    o = run_logits(B, c)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    zz = f64(c["z"])
    zz[row, t] = -math.inf
    _, H, p, logp = tr.token_logprobs(zz, np.where(np.arange(T) == row, t, c["target"]))
    dlp = np.zeros(T)
    want = tr.policy_dz(zz, c["target"], dlp, c["w"], 0.05)[row]
    size = 0.05 * c["w"][row] * p[row] * (np.abs(np.where(p[row] > 0, logp[row], 0)) + H[row] + 1)
    got = f64(o["dz"])[row]
    assert float(o["lp"][row]) < -1e28 and got[t] == 0.0
    assert np.all(np.abs(got - want) <= (REL + 2.0 ** -24) * size + 1e-37)
    keep = torch.arange(T, device="cuda") != row
    if old != "own":
        assert same(o["dz"][keep], clean["dz"][keep]) and same(o["lp"][keep], clean["lp"][keep])
    # from logprobs
    lp = o["lp"].clone()
    if old != "own":
        lp[row] = -math.inf
        d = desc(B, c | dict(kw=kw | dict(gamma=0.0)), torch.empty(8, device="cuda"), workspace(B, T, 1))
        out = torch.empty(T, device="cuda")
        B.biv_policy_loss(d, lp, out)
        torch.cuda.synchronize()
        assert float(out[row]) == 0.0 and bool(torch.isfinite(out).all())


@pytest.mark.parametrize("per_row", [True, False, None])
def test_as_many_rows_as_sequences(B, per_row):
    """Four rows in four sequences, two of them empty: the caller says whether the
    four advantages are the rows' or the sequences' (None: the sequences')."""
    T, start = 4, [0, 0, 0, 2, 4]
    adv = np.array([1.0, 2.0, 3.0, 4.0], np.float32)
    stats, dlp = torch.empty(8, device="cuda"), torch.empty(T, device="cuda")
    make = lambda a, n, **kw: B.policy_desc(dev(start, np.int32), dev(a), stats, workspace(B, n, 4), T=n, **kw)  # noqa: E731
    d = make(adv, T, adv_per_row=per_row)
    B.biv_policy_loss(d, torch.full((T,), -1.0, device="cuda"), dlp)
    torch.cuda.synchronize()
    A = adv if per_row else adv[[2, 2, 3, 3]]
    assert np.all(np.abs(f64(dlp) + A / 4) <= 2.0 ** -23 * A)
    for a, n, kw in ((adv, 5, dict(adv_per_row=True)), (np.ones(5), 5, dict(adv_per_row=False)),
                     (np.ones(3), 5, {})):
        with pytest.raises(ValueError):
            make(a, n, **kw)


@pytest.mark.parametrize("T,nseq", [(600_001, 5), (1_100_003, 1024), (1_100_003, 1025), (1_100_003, 3)])
def test_large_batches(B, T, nseq):
    """Beyond 524288 rows, by either way of counting: weights, gradient and sums."""
    g = synth.rng(nseq)
    start = np.sort(np.concatenate([[3, T - 7], g.integers(3, T - 7, nseq - 1)]))
    mask, adv = (g.random(T) < 0.9).astype(np.uint8), g.standard_normal(nseq).astype(np.float32)
    stats, dlp = torch.empty(8, device="cuda"), torch.full((T,), 7.0, device="cuda")
    d = B.policy_desc(dev(start, np.int32), dev(adv), stats, workspace(B, T, nseq), T=T, mask=dev(mask, np.uint8),
                      reduce=B.LOSS_SEQ_MEAN)
    B.biv_policy_loss(d, torch.full((T,), -1.0, device="cuda"), dlp)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    seq = np.searchsorted(start, np.arange(T), side="right") - 1
    on = (seq >= 0) & (seq < nseq) & (mask != 0)
    n = np.bincount(seq[on], minlength=nseq)
    w = np.where(on, 1.0 / (np.sum(n > 0) * np.maximum(n, 1))[np.clip(seq, 0, nseq - 1)], 0)
    want = -w * adv.astype(np.float64)[np.clip(seq, 0, nseq - 1)]
    # the weight's product and reciprocal, and its product with A: three roundings
    assert np.all(np.abs(f64(dlp) - want) <= 3.1 * 2.0 ** -24 * np.abs(want))
    got = f64(stats)
    assert got[7] == on.sum() and got[4] == got[5] == got[6] == 0
    # (blocks of 1024 rows, then 32 lanes over at most 34 blocks each: 4 + 5 + 8 + 34 + 5 additions)
    assert abs(got[0] - want.sum()) <= 60 * 2.0 ** -24 * np.abs(want).sum()

"""Cross entropy of the LM head and its gradient without logits, against 64 bits.

Tolerances, per element, with |.| sums over the terms of the product at hand:
 - z = h.W has K products summed in FP32 in some order, each addition off by at
   most 2^-23 of the running sum (a truncating adder): dz <= K 2^-23 (|h|.|W|);
   p = exp(z - lse) then has a relative error of e^(dz + 2^-20) - 1, where 2^-20
   covers the difference's, expf's and the factor's roundings;
 - the p terms of dz enter as bf16 (2^-8 each) or as two bf16 parts (2^-16);
 - the products' sums: (terms + 64) 2^-23 of the sum of magnitudes;
 - the output's own rounding: 2^-8 (bf16) or 2^-24 (FP32)."""
import ctypes as C

import pytest
import torch

gpu = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(scope="module")
def B():
    from invariant_forward_bitwise_gb300 import biv, build
    build.build()
    biv.load()
    return biv


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def padded(rows, cols, pad, dtype=torch.bfloat16):
    """A matrix with `pad` columns of a marker behind its rows."""
    full = torch.full((rows, cols + pad), 7.0, dtype=dtype, device="cuda")
    return full, full[:, :cols]


class Case:
    def __init__(self, T, V, K, seed=0, live=None, z=0.0, policy=True, targets=None, pad=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.T, self.V, self.K = T, V, K
        self.h = padded(T, K, pad)[1].copy_(rnd(T, K))
        self.W = padded(V, K, pad)[1].copy_(rnd(V, K) * (2.0 / K ** 0.5))
        self.target = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
        if targets is not None:
            self.target.fill_(targets)
        self.live = torch.ones(T, dtype=torch.bool, device="cuda") if live is None else live
        self.logits = self.h.to(F64) @ self.W.to(F64).t()
        self.lse64 = torch.logsumexp(self.logits, 1)
        self.lse = self.lse64.float()
        self.dlp = (rnd(T) if policy else -torch.ones(T, device="cuda")) / T * self.live
        self.dlse = (2 * z * self.lse / T) * self.live if z else None

    def run(self, B, dh_t=torch.bfloat16, dw_t=torch.bfloat16, accumulate=None, want=(True, True), pad=0, **kw):
        dh_full, dh = padded(self.T, self.K, pad, dh_t)
        dw_full, dW = padded(self.V, self.K, pad, dw_t)
        if accumulate is not None:
            dW.copy_(accumulate)
        ws = torch.empty(B.biv_lm_head_backward_workspace(self.T, self.V, self.K, dh_t, dw_t), dtype=torch.uint8,
                         device="cuda")
        ws.fill_(255)      # NaN everywhere: no initial value is needed
        B.biv_lm_head_backward(self.h, self.W, self.target, self.lse, self.dlp, dh if want[0] else None,
                               dW if want[1] else None, ws, dlse=self.dlse, accumulate=accumulate is not None, **kw)
        if pad:
            torch.cuda.synchronize()
            assert bool((dh_full[:, self.K:] == 7).all()) and bool((dw_full[:, self.K:] == 7).all())
        return dh, dW

    def check(self, dh, dW, before=None):
        """Both gradients against 64 bits."""
        on = self.live[:, None]
        h = torch.where(on, self.h.to(F64), 0.0)
        W = self.W.to(F64)
        p = torch.where(on, torch.exp(self.logits - self.lse.to(F64)[:, None]), 0.0)
        cp = (0 if self.dlse is None else self.dlse.to(F64)) - self.dlp.to(F64)
        pz = p * cp[:, None]
        hot = torch.zeros_like(pz)
        hot[torch.arange(self.T, device="cuda"), self.target.long().clamp(0, self.V - 1)] = self.dlp.to(F64) * self.live
        dz_err = self.K * 2.0 ** -23 * (h.abs() @ W.abs().t())
        p_err = torch.expm1(dz_err + 2.0 ** -20)
        for out, left, right, terms, add in (
                (dh, lambda m: m, W, self.V, None), (dW, lambda m: m.t(), h, self.T, before)):
            if out is None:
                continue
            out_eps, in_eps = (2.0 ** -8, 2.0 ** -8) if out.dtype == torch.bfloat16 else (2.0 ** -24, 2.0 ** -16)
            want = left(pz + hot) @ right + (0 if add is None else add.to(F64))
            size = left(pz.abs() + hot.abs()) @ right.abs() + (0 if add is None else add.to(F64).abs())
            tol = left(pz.abs() * (in_eps + p_err)) @ right.abs() + (terms + 64) * 2.0 ** -23 * size
            # (the target's p cancels against 1 in FP32: its error is p's, counted above)
            tol = tol * (1 + out_eps) + out_eps * want.abs() + 1e-38
            off = (out.to(F64) - want).abs()
            assert bool((off <= tol).all()), (float((off / tol).max()), out.shape, out.dtype)


SIZES = [
    (1, 1, 8), (1, 2, 8), (3, 7, 16), (13, 4096, 256), (127, 255, 64), (128, 256, 128), (129, 257, 136),
    (255, 513, 72), (256, 8191, 64), (257, 8192, 128), (300, 8193, 248), (64, 16400, 264), (40, 20011, 688),
    (700, 3000, 520), (1, 30000, 2048), (513, 9000, 256),
]


@gpu
@pytest.mark.parametrize("T,V,K", SIZES)
@pytest.mark.parametrize("dh_t,dw_t", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
def test_gradient_against_64_bits(B, T, V, K, dh_t, dw_t):
    t = {"bf16": torch.bfloat16, "f32": torch.float32}
    c = Case(T, V, K, seed=T + V, z=1e-3 if T % 2 else 0.0)
    dh, dW = c.run(B, t[dh_t], t[dw_t])
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    c.check(dh, dW)


@gpu
@pytest.mark.parametrize("pad", [0, 8, 72])
def test_strided_rows_and_what_lies_between(B, pad):
    live = torch.arange(200, device="cuda") % 3 != 0
    c = Case(200, 1000, 136, live=live, z=1e-3, pad=pad)
    for t in (torch.bfloat16, torch.float32):
        c.check(*c.run(B, t, t, pad=pad))


@gpu
def test_unaligned_gradient_rows(B):
    """Gradients whose rows start anywhere: elements are stored one by one."""
    c = Case(70, 300, 72)
    ws = torch.empty(B.biv_lm_head_backward_workspace(70, 300, 72), dtype=torch.uint8, device="cuda")
    full = torch.full((300 * 73 + 1,), 7.0, dtype=torch.bfloat16, device="cuda")
    dW = full[1:].view(300, 73)[:, :72]
    dh = torch.full((70, 75), 7.0, dtype=torch.bfloat16, device="cuda")[:, 1:73]
    B.biv_lm_head_backward(c.h, c.W, c.target, c.lse, c.dlp, dh, dW, ws)
    c.check(dh, dW)
    assert float(full[0]) == 7.0 and bool((full[1:].view(300, 73)[:, 72] == 7).all())


@gpu
@pytest.mark.parametrize("which", ["none", "first", "last", "scattered"])
def test_rows_that_do_not_count(B, which):
    """Their dh is zero, and NaN or infinities in their h, lse or target change nothing."""
    T, V, K = 300, 777, 200
    live = torch.zeros(T, dtype=torch.bool, device="cuda")
    if which == "first":
        live[:17] = True
    elif which == "last":
        live[-1] = True
    elif which == "scattered":
        live[torch.arange(0, T, 7)] = True
    c = Case(T, V, K, live=live, z=1e-3)
    dh, dW = c.run(B)
    clean = [dh.clone(), dW.clone()]
    c.check(dh, dW)
    assert bool((dh[~live] == 0).all())
    c.h[~live] = float("nan")
    c.lse[~live] = float("inf")
    c.target[~live] = -100
    dh, dW = c.run(B)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    assert same(clean[0], dh) and same(clean[1], dW)


@gpu
def test_bad_target_is_reported_and_left_out(B):
    c = Case(50, 300, 64)
    c.target[7], c.target[9] = 300, -1
    dh, dW = c.run(B)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 2
    c.live = torch.ones(50, dtype=torch.bool, device="cuda")
    c.live[7] = c.live[9] = False
    c.dlp = c.dlp * c.live
    c.check(dh, dW)
    assert bool((dh[[7, 9]] == 0).all())


@gpu
def test_a_row_with_nan_stays_alone_in_dh(B):
    c = Case(40, 500, 64)
    clean, _ = c.run(B)
    clean = clean.clone()
    c.h[3, 5] = float("nan")
    dh, dW = c.run(B)
    assert bool(dh[3].isnan().all()) and bool(dW.isnan().all(0)[5])
    keep = torch.arange(40, device="cuda") != 3
    assert same(clean[keep], dh[keep])


@gpu
@pytest.mark.parametrize("low", [-3.3e38, -float("inf")])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
def test_weights_whose_logits_are_minus_infinity(B, low, t):
    """A vocabulary row that no h can reach has p = 0: its gradient is zero and the
    others' are as without it, in the rows behind the counted ones of a tile too."""
    c = Case(70, 300, 64)
    c.h.copy_(c.h.abs() + 1)
    c.W[5] = low
    c.target[c.target == 5] = 6
    keep = torch.arange(300, device="cuda") != 5
    c.logits = c.h.to(F64) @ torch.where(keep[:, None], c.W.to(F64), 0.0).t()
    c.logits[:, 5] = -1e4
    c.lse = torch.logsumexp(c.logits, 1).float()
    dh, dW = c.run(B, t, t)
    assert bool((dW[5] == 0).all())
    c.W[5] = 0                                     # (check multiplies it by p = 0)
    c.check(dh if low > -float("inf") else None, dW)


@gpu
def test_every_row_has_the_same_target(B):
    c = Case(600, 900, 256, targets=450)
    for t in (torch.bfloat16, torch.float32):
        c.check(*c.run(B, t, t))


@gpu
def test_targets_at_the_ends(B):
    for tg in (0, 8191, 8192, 8200):
        c = Case(30, 8201, 64, targets=tg)
        c.check(*c.run(B, torch.float32, torch.float32))


@gpu
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
def test_accumulate_and_single_outputs(B, t):
    c = Case(100, 600, 136)
    dh, dW = c.run(B, t, t)
    base = (torch.randn(600, 136, device="cuda") * 0.01).to(t)
    _, more = c.run(B, t, t, accumulate=base)
    c.check(None, more, before=base)
    only, _ = c.run(B, t, t, want=(True, False))
    _, wonly = c.run(B, t, t, want=(False, True))
    assert same(only, dh) and same(wonly, dW)
    untouched, _ = c.run(B, t, t, want=(False, True))
    assert bool((untouched == 7).all())


@gpu
def test_accumulate_without_counted_rows(B):
    c = Case(20, 300, 64, live=torch.zeros(20, dtype=torch.bool, device="cuda"))
    base = torch.randn(300, 64, device="cuda").bfloat16()
    dh, dW = c.run(B, accumulate=base)
    assert same(dW, base) and bool((dh == 0).all())
    dh, dW = c.run(B)
    assert bool((dW == 0).all())


@gpu
def test_no_rows(B):
    e = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    W = torch.randn(300, 64, device="cuda").bfloat16()
    h, tg, dW = e(0, 64, t=torch.bfloat16), e(0, t=torch.int32), torch.ones(300, 64, device="cuda")
    ws, stats = e(B.biv_lm_head_loss_workspace(0, 300), t=torch.uint8), e(4)
    B.biv_lm_head_backward(h, W, tg, e(0), e(0), None, dW, e(0, t=torch.uint8), accumulate=True)
    assert bool((dW == 1).all())
    B.biv_lm_head_backward(h, W, tg, e(0), e(0), None, dW, e(0, t=torch.uint8))
    B.biv_lm_head_loss(h, W, tg, e(0), e(0), stats, ws)
    assert bool((dW == 0).all()) and stats.tolist() == [0, 0, 0, 0]


@gpu
def test_a_rows_dh_does_not_depend_on_the_batch(B):
    """Alone, among others, and in the batch size at which chunks are added up as they come."""
    T, V, K = 8300, 20000, 2048          # 3 chunks; more partials than are held side by side
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(T, K, device="cuda", generator=g).bfloat16()
    W = (torch.randn(V, K, device="cuda", generator=g) * 0.04).bfloat16()
    target = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
    lse = torch.cat([(x @ W.t()).float().logsumexp(1) for x in h.split(2048)])
    dlp = torch.randn(T, device="cuda", generator=g)
    for t in (torch.bfloat16, torch.float32):
        outs = []
        for rows in (slice(0, T), slice(4000, 4300), slice(4100, 4101)):
            n = rows.stop - rows.start
            dh = torch.empty(n, K, dtype=t, device="cuda")
            ws = torch.empty(B.biv_lm_head_backward_workspace(n, V, K, t, torch.bfloat16), dtype=torch.uint8,
                             device="cuda")
            B.biv_lm_head_backward(h[rows], W, target[rows], lse[rows], dlp[rows], dh, None, ws)
            outs.append(dh)
        assert same(outs[0][4000:4300], outs[1]) and same(outs[1][100:101], outs[2])
        if t is torch.float32:           # that large batch itself, on a sample of rows
            pick = torch.arange(5, T, 577, device="cuda")
            z = h[pick].to(F64) @ W.to(F64).t()
            dz = -dlp[pick].to(F64)[:, None] * torch.exp(z - lse[pick].to(F64)[:, None])
            dz[torch.arange(pick.numel(), device="cuda"), target[pick].long()] += dlp[pick].to(F64)
            want = dz @ W.to(F64)
            assert float((outs[0][pick].to(F64) - want).norm() / want.norm()) < 1e-4


@gpu
def test_many_rows_dw(B):
    """Several row tiles and column pieces at once, the gradient of the weights."""
    T, V, K = 3100, 9000, 512
    c = Case(T, V, K, live=torch.arange(T, device="cuda") % 5 != 0)
    c.check(*c.run(B))


@gpu
@pytest.mark.parametrize("T", [1023, 1024, 1025, 2048, 5000])
@pytest.mark.parametrize("which", ["all", "few", "ties", "none", "one run"])
def test_order_of_many_rows(B, T, which):
    """Rows sorted by target in runs: targets on every side of every run, ties across
    runs, runs without a counted row."""
    t = torch.arange(T, device="cuda")
    live = {"few": t % 97 == 5, "none": t < 0, "one run": (t >= 1000) & (t < 1030)}.get(which, t >= 0)
    c = Case(T, 600, 64, seed=T, live=live, z=1e-3)
    if which == "ties":
        c.target.copy_((t * 7919 % 5 * 100).int())
    c.target[~live] = 600
    dh, dW = c.run(B, torch.float32, torch.float32)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    c.check(dh, dW)
    again = c.run(B, torch.float32, torch.float32)
    assert same(again[0], dh) and same(again[1], dW)


@gpu
@pytest.mark.parametrize("T", [64, 65, 200, 1300])
@pytest.mark.parametrize("V", [2, 3, 40])
def test_targets_that_many_rows_share(B, T, V):
    """Sums over 8 and 64 rows of one target, their ends, and single rows beside them."""
    c = Case(T, V, 136, seed=V, live=torch.arange(T, device="cuda") % 11 != 3)
    c.target.copy_((c.target.float() / V).square().mul(V).int())      # low ones are frequent
    for t in (torch.bfloat16, torch.float32):
        c.check(*c.run(B, t, t))
    _, dW = c.run(B, want=(False, True))
    again = c.run(B, want=(False, True))[1]
    assert same(dW, again)


@gpu
def test_bad_targets_among_many_rows(B):
    c = Case(1500, 300, 64)
    c.target[7], c.target[1300] = 300, -1
    dh, dW = c.run(B)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 2
    c.live = torch.ones(1500, dtype=torch.bool, device="cuda")
    c.live[7] = c.live[1300] = False
    c.dlp = c.dlp * c.live
    c.check(dh, dW)


@gpu
def test_offsets_beyond_32_bits(B):
    """More than 2^31 elements of W and dW."""
    T, V, K = 3, 140000, 16384
    g = torch.Generator(device="cuda").manual_seed(2)
    h = torch.randn(T, K, device="cuda", generator=g).bfloat16()
    W = torch.empty(V, K, dtype=torch.bfloat16, device="cuda")
    for a in range(0, V, 8192):
        W[a:a + 8192] = torch.randn(min(8192, V - a), K, device="cuda", generator=g) * 0.01
    target = torch.tensor([0, V - 1, V - 1], dtype=torch.int32, device="cuda")
    dlp = torch.tensor([1.0, -0.5, 0.25], device="cuda")
    z = torch.cat([h.to(F64) @ W[a:a + 8192].to(F64).t() for a in range(0, V, 8192)], 1)
    lse = z.logsumexp(1)
    dh, dW = torch.empty_like(h), torch.empty_like(W)
    ws = torch.empty(B.biv_lm_head_backward_workspace(T, V, K), dtype=torch.uint8, device="cuda")
    B.biv_lm_head_backward(h, W, target, lse.float(), dlp, dh, dW, ws)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    dz = -torch.exp(z - lse[:, None]) * dlp.to(F64)[:, None]
    dz[torch.arange(3, device="cuda"), target.long()] += dlp.to(F64)
    for v in (0, 1, 131071, 131072, V - 2, V - 1):
        want = dz[:, v] @ h.to(F64)
        tol = 2.0 ** -7 * (dz[:, v].abs() @ h.to(F64).abs())
        assert bool(((dW[v].to(F64) - want).abs() <= tol).all()), v
    want = sum(dz[:, a:a + 8192] @ W[a:a + 8192].to(F64) for a in range(0, V, 8192))
    assert float((dh.to(F64) - want).norm() / want.norm()) < 2.0 ** -8
    lp, l2, stats = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty(4, device="cuda")
    fws = torch.empty(B.biv_lm_head_loss_workspace(T, V), dtype=torch.uint8, device="cuda")
    B.biv_lm_head_loss(h, W, target, lp, l2, stats, fws)
    assert float((l2.to(F64) - lse).abs().max()) < 1e-4


@gpu
def test_a_graph_and_two_streams_repeat_the_bits(B):
    cs = [Case(300, 9000, 256, seed=s, live=torch.arange(300, device="cuda") % 4 != s) for s in (0, 1)]
    eager = [[x.clone() for x in c.run(B)] for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    outs, wss = [], []
    for c, s in zip(cs, streams):
        dh, dW = torch.empty(300, 256, dtype=torch.bfloat16, device="cuda"), torch.empty_like(c.W)
        ws = torch.empty(B.biv_lm_head_backward_workspace(300, 9000, 256), dtype=torch.uint8, device="cuda")
        outs.append((dh, dW))
        wss.append(ws)
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s, o, w in zip(cs, streams, outs, wss):
            B.biv_lm_head_backward(c.h, c.W, c.target, c.lse, c.dlp, *o, w, stream=s)
    torch.cuda.synchronize()
    for e, o in zip(eager, outs):
        assert same(e[0], o[0]) and same(e[1], o[1])
    c, (dh, dW), ws = cs[0], outs[0], wss[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.biv_lm_head_backward(c.h, c.W, c.target, c.lse, c.dlp, dh, dW, ws)
    # replayed on other inputs in the same places, another number of counted rows among them
    for k in (1, 0):
        for a, b in ((c.h, cs[k].h), (c.W, cs[k].W), (c.target, cs[k].target), (c.lse, cs[k].lse),
                     (c.dlp, cs[k].dlp)):
            if k == 1 and not hasattr(c, "first"):
                c.first = True
                kept = [t.clone() for t in (c.h, c.W, c.target, c.lse, c.dlp)]
            a.copy_(b if k else kept.pop(0))
        g.replay()
        torch.cuda.synchronize()
        assert same(dh, eager[k][0]) and same(dW, eager[k][1])


@gpu
def test_a_captured_gradient_of_many_rows_on_other_inputs(B):
    """Sorted runs and sums over equal targets: one graph, replayed with other targets
    and another number of counted rows, while a second stream runs a call of its own."""
    T, V, K = 1500, 700, 136
    cs = [Case(T, V, K, seed=s, live=torch.arange(T, device="cuda") % 7 > 2 * s) for s in (0, 1, 2)]
    cs[1].target.copy_(cs[1].target % 4)
    for c in cs:
        c.h[~c.live] = 0
    f32 = torch.float32
    eager = [[x.clone() for x in c.run(B, f32, f32)] for c in cs]
    new = lambda: (torch.empty(T, K, device="cuda"), torch.empty(V, K, device="cuda"),  # noqa: E731
                   torch.empty(B.biv_lm_head_backward_workspace(T, V, K, f32, f32), dtype=torch.uint8, device="cuda"))
    (dh, dW, ws), other = new(), new()
    at = [t.clone() for t in (cs[0].h, cs[0].W, cs[0].target, cs[0].lse, cs[0].dlp)]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        B.biv_lm_head_backward(*at, dh, dW, ws)
    side = torch.cuda.Stream()
    for k in (1, 0, 2, 1):
        for t, v in zip(at, (cs[k].h, cs[k].W, cs[k].target, cs[k].lse, cs[k].dlp)):
            t.copy_(v)
        torch.cuda.synchronize()
        g.replay()
        c = cs[2 - k]
        B.biv_lm_head_backward(c.h, c.W, c.target, c.lse, c.dlp, *other, stream=side)
        torch.cuda.synchronize()
        assert same(dh, eager[k][0]) and same(dW, eager[k][1])
        assert same(other[0], eager[2 - k][0]) and same(other[1], eager[2 - k][1])
    assert B.biv_poll_error() == 0


@gpu
@pytest.mark.parametrize("T,V,K,hot,dh,dw", [
    (300, 32768, 256, False, True, False),      # dh's products of 64 stages and two parts
    (16384, 600, 256, False, False, True),      # dW's of 256 stages and two parts
    (1000, 32003, 2048, True, True, True),      # a ring shorter than the chunks, partials side by side
    (2100, 50000, 2048, True, True, True),      # and partials added up as they come
])
def test_fp32_gradients_have_fp32_quality(B, T, V, K, hot, dh, dw):
    """2-norm of the error against 64 bits, relative to the gradient's.  Its parts:
     - hi + lo of dz: a bf16 rounding is off by at most 2^-8 of the value, 2^-8 / sqrt(3) *
       0.735 = 1.7e-3 of it in the mean square over mantissas; the second one by as much of
       the first one's rest: 2.7e-6, of terms of random signs, so of their sums too;
     - an accumulator truncates at each of the 48 steps of its 12 stages: by 0.72 * 2^-24 =
       4.3e-8 of the running sum in the mean, 48 / 2 * 4.3e-8 = 1.0e-6 where the sum grows
       steadily, and 48 / sqrt(12) * 4.3e-8 = 0.6e-6 more for its wandering;
     - logits of size 0.5 from such sums, their difference from lse (of up to 11: 2^-21 at
       most, 2.7e-7 in the mean square) and expf: 1e-6.
    Added up 5.3e-6.  One bf16 part leaves 1.7e-3 of the p terms; accumulators over all
    stages lose 1.7e-7 a stage, 9e-6 and more in the first two cases, whose dz is of p alone."""
    g = torch.Generator(device="cuda").manual_seed(T)
    h = torch.randn(T, K, device="cuda", generator=g).bfloat16()
    W = (torch.randn(V, K, device="cuda", generator=g) * (0.5 / K ** 0.5)).bfloat16()
    target = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
    a = torch.randn(T, device="cuda", generator=g) / T
    dlp, dlse = (a if hot else torch.zeros_like(a)), torch.randn(T, device="cuda", generator=g) / T
    h64, W64 = h.to(F64), W.to(F64)
    dz = h64 @ W64.t()
    lse = torch.logsumexp(dz, 1).float()
    dz.sub_(lse.to(F64)[:, None]).exp_().mul_((dlse.to(F64) - dlp.to(F64))[:, None])
    dz[torch.arange(T, device="cuda"), target.long()] += dlp.to(F64)
    gh, gw = torch.empty(T, K, device="cuda"), torch.empty(V, K, device="cuda")
    ws = torch.empty(B.biv_lm_head_backward_workspace(T, V, K, torch.float32, torch.float32), dtype=torch.uint8,
                     device="cuda").fill_(255)
    B.biv_lm_head_backward(h, W, target, lse, dlp, gh, gw, ws, dlse=dlse)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    for on, got, left, right in ((dh, gh, dz, W64), (dw, gw, dz.t(), h64)):
        if on:
            want = left @ right
            assert float((got.to(F64) - want).norm() / want.norm()) <= 5.3e-6

# ---------------------------------------------------------------- forward --
@gpu
@pytest.mark.parametrize("T,V,K", [(1, 1, 8), (13, 4096, 256), (130, 1001, 72), (300, 20011, 688), (5, 30000, 2048)])
@pytest.mark.parametrize("mean", [True, False])
@pytest.mark.parametrize("weighted", [True, False])
def test_loss_against_64_bits(B, T, V, K, mean, weighted):
    live = torch.arange(T, device="cuda") % 3 != 1
    c = Case(T, V, K, live=live, seed=5)
    g = torch.Generator(device="cuda").manual_seed(9)
    weight = 0.5 + torch.rand(T, device="cuda", generator=g) if weighted else None
    target = torch.where(live, c.target, -100)
    if weighted and T > 5:
        weight[3] = 0.0                       # a weight of 0 is as good as an ignored target
    c.h[~live] = float("nan")
    lp, lse, dlp, dlse = (torch.full((T,), 5.0, device="cuda") for _ in range(4))
    stats = torch.empty(4, device="cuda")
    ws = torch.empty(B.biv_lm_head_loss_workspace(T, V), dtype=torch.uint8, device="cuda").fill_(255)
    zc = 1e-2
    B.biv_lm_head_loss(c.h, c.W, target, lp, lse, stats, ws, weight=weight, dlp=dlp, dlse=dlse, z_coef=zc,
                       reduce=B.LOSS_TOKEN_MEAN if mean else B.LOSS_SUM, norm=17.0)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    w = (torch.ones(T, device="cuda") if weight is None else weight).to(F64) * live
    on = w != 0
    want_lse = torch.where(on, c.lse64, 0.0)
    zt = c.logits.gather(1, c.target.long()[:, None])[:, 0]
    want_lp = torch.where(on, zt - c.lse64, 0.0)
    # the logits' error (K products), then sums of V positive terms and a few roundings of lse
    h = torch.where(live[:, None], c.h.to(F64), 0.0)
    tol = (K + 8) * 2.0 ** -23 * (h.abs() @ c.W.to(F64).abs().t()).amax(1) + 2.0 ** -19 * (1 + want_lse.abs())
    assert bool(((lse.to(F64) - want_lse).abs() <= tol).all())
    assert bool(((lp.to(F64) - want_lp).abs() <= 2 * tol).all())
    assert bool((lp[~on] == 0).all()) and bool((lse[~on] == 0).all())
    share = w / (w.sum() if mean else 17.0)
    assert torch.allclose(dlp.to(F64), -share, rtol=2.0 ** -22, atol=0)
    assert torch.allclose(dlse.to(F64), 2 * zc * share * lse.to(F64), rtol=2.0 ** -21, atol=0)
    nll, sq = -(share * lp.to(F64)).sum(), (share * lse.to(F64) ** 2).sum()
    want = torch.stack([nll + zc * sq, nll, sq, w.sum()])
    assert torch.allclose(stats.to(F64), want, rtol=2.0 ** -20, atol=1e-30)


@gpu
def test_logprobs_are_those_of_the_fused_head(B):
    for T, V, K in ((300, 4096, 256), (33, 30000, 2048)):
        c = Case(T, V, K)
        lp, lse, ref = (torch.empty(T, device="cuda") for _ in range(3))
        ws = torch.empty(B.biv_lm_head_loss_workspace(T, V), dtype=torch.uint8, device="cuda")
        B.biv_lm_head_loss(c.h, c.W, c.target, lp, lse, torch.empty(4, device="cuda"), ws)
        B.biv_lm_head_logprob(c.h, c.W, c.target, ref, ws)
        assert same(lp, ref)
        one, l1 = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
        B.biv_lm_head_loss(c.h[7:8], c.W, c.target[7:8], one, l1, torch.empty(4, device="cuda"), ws)
        assert same(one, lp[7:8]) and same(l1, lse[7:8])


@gpu
@pytest.mark.parametrize("which", ["prompts", "tail", "one", "none", "all", "weights"])
def test_row_tiles_that_do_not_count(B, which):
    """A product large enough that 128-row tiles without counted rows are left out."""
    T, V, K = 1111, 36000, 2048
    g = torch.Generator(device="cuda").manual_seed(3)
    h = torch.randn(T, K, device="cuda", generator=g).bfloat16()
    W = (torch.randn(V, K, device="cuda", generator=g) * 0.04).bfloat16()
    target = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
    row = torch.arange(T, device="cuda")
    on = {"prompts": row % 500 >= 300, "tail": row < 385, "one": row == 1110, "none": row < 0, "all": row >= 0,
          "weights": (row // 128) % 2 == 1}[which]
    weight = torch.where(on, 0.5 + torch.rand(T, device="cuda", generator=g), 0.0) if which == "weights" else None
    if weight is None:
        target = torch.where(on, target, -100)
    ws = torch.empty(B.biv_lm_head_loss_workspace(T, V), dtype=torch.uint8, device="cuda")
    ref = torch.empty(T, device="cuda")
    B.biv_lm_head_logprob(h, W, target.clamp_min(0), ref, ws)
    h[~on] = float("nan")
    ws.fill_(255)
    lp, lse, dlp, dlse = (torch.full((T,), 5.0, device="cuda") for _ in range(4))
    stats = torch.empty(4, device="cuda")
    B.biv_lm_head_loss(h, W, target, lp, lse, stats, ws, weight=weight, dlp=dlp, dlse=dlse, z_coef=0.5)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    assert same(lp, torch.where(on, ref, 0.0)) and bool((lse[~on] == 0).all()) and bool((lse[on] > 0).all())
    w = (on if weight is None else weight).to(F64)
    share = w / max(float(w.sum()), 1e-30)
    # (each a handful of FP32 roundings of values computed in 64 bits)
    assert torch.allclose(dlp.to(F64), -share, rtol=2.0 ** -22, atol=0)
    assert torch.allclose(dlse.to(F64), share * lse.to(F64), rtol=2.0 ** -21, atol=0)
    nll, sq = -(share * lp.to(F64)).sum(), (share * lse.to(F64) ** 2).sum()
    want = torch.stack([nll + 0.5 * sq, nll, sq, w.sum()])
    assert torch.allclose(stats.to(F64), want, rtol=2.0 ** -20, atol=0)


@gpu
def test_a_captured_loss_on_other_masks(B):
    """The tiles that are left out follow the targets of each replay."""
    T, V, K = 1111, 36000, 2048
    g = torch.Generator(device="cuda").manual_seed(3)
    h = torch.randn(T, K, device="cuda", generator=g).bfloat16()
    W = (torch.randn(V, K, device="cuda", generator=g) * 0.04).bfloat16()
    target = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
    row = torch.arange(T, device="cuda")
    masks = [row >= 0, row % 500 >= 300, row < 0, row == 1110]
    out = lambda: [torch.empty(T, device="cuda") for _ in range(3)] + [torch.empty(4, device="cuda")]  # noqa: E731
    ws = torch.empty(B.biv_lm_head_loss_workspace(T, V), dtype=torch.uint8, device="cuda")
    eager, got, at = [], out(), target.clone()
    for m in masks:
        o = out()
        B.biv_lm_head_loss(h, W, torch.where(m, target, -100), *o[:2], o[3], ws, dlp=o[2])
        eager.append(o)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        B.biv_lm_head_loss(h, W, at, *got[:2], got[3], ws, dlp=got[2])
    for k in (1, 3, 0, 2, 0):
        at.copy_(torch.where(masks[k], target, -100))
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, eager[k]))
    assert B.biv_poll_error() == 0


@gpu
def test_few_rows_have_the_bits_of_many(B):
    """At most 32 rows take one kernel for all sums: lp and lse are those of a larger call."""
    T, V, K = 70, 9001, 256
    c = Case(T, V, K)
    out = [torch.empty(T, device="cuda") for _ in range(2)]
    ws = torch.empty(B.biv_lm_head_loss_workspace(T, V), dtype=torch.uint8, device="cuda")
    stats = torch.empty(4, device="cuda")
    B.biv_lm_head_loss(c.h, c.W, c.target, *out, stats, ws)
    for n in (1, 31, 32, 33):
        few = [torch.empty(n, device="cuda") for _ in range(3)]
        B.biv_lm_head_loss(c.h[5:5 + n], c.W, c.target[5:5 + n], *few[:2], stats, ws, dlp=few[2])
        assert all(same(a, b[5:5 + n]) for a, b in zip(few, out))
        assert torch.allclose(few[2].to(F64), torch.full((n,), -1 / n, device="cuda", dtype=F64), rtol=2.0 ** -23)
        assert torch.allclose(stats[1].to(F64), -few[0].to(F64).mean(), rtol=2.0 ** -22) and float(stats[3]) == n


@gpu
def test_loss_bad_target(B):
    c = Case(20, 300, 64)
    c.target[4] = 300
    lp, lse, dlp, stats = (torch.empty(n, device="cuda") for n in (20, 20, 20, 4))
    ws = torch.empty(B.biv_lm_head_loss_workspace(20, 300), dtype=torch.uint8, device="cuda")
    B.biv_lm_head_loss(c.h, c.W, c.target, lp, lse, stats, ws, dlp=dlp)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 2 and bool(lp[4].isnan()) and bool(stats[0].isnan())
    assert not bool(lp[:4].isnan().any()) and not bool(lp[5:].isnan().any())


@gpu
def test_differences_of_the_loss(B):
    """The gradient of loss(h, W) along a direction, against a difference of 64-bit losses."""
    T, V, K = 60, 700, 64
    c = Case(T, V, K, policy=False)
    target = c.target.clone()
    target[::5] = -100
    lp, lse, dlp, dlse, stats = (torch.empty(n, device="cuda") for n in (T, T, T, T, 4))
    ws = torch.empty(B.biv_lm_head_loss_workspace(T, V), dtype=torch.uint8, device="cuda")
    zc = 0.05
    B.biv_lm_head_loss(c.h, c.W, target, lp, lse, stats, ws, dlp=dlp, dlse=dlse, z_coef=zc)
    dh, dW = torch.empty(T, K, device="cuda"), torch.empty(V, K, device="cuda")
    bws = torch.empty(B.biv_lm_head_backward_workspace(T, V, K, torch.float32, torch.float32), dtype=torch.uint8,
                      device="cuda")
    B.biv_lm_head_backward(c.h, c.W, target, lse, dlp, dh, dW, bws, dlse=dlse)

    def loss(h, W):
        z = h @ W.t()
        on = target >= 0
        l = torch.logsumexp(z, 1)  # noqa: E741
        p = z.gather(1, target.long().clamp_min(0)[:, None])[:, 0] - l
        return ((-p + zc * l ** 2) * on).sum() / on.sum()

    g = torch.Generator(device="cuda").manual_seed(3)
    a = torch.randn(T, K, device="cuda", generator=g, dtype=F64)
    b = torch.randn(V, K, device="cuda", generator=g, dtype=F64) * 0.1
    e = 1e-5
    h, W = c.h.to(F64), c.W.to(F64)
    diff = (loss(h + e * a, W + e * b) - loss(h - e * a, W - e * b)) / (2 * e)
    got = (dh.to(F64) * a).sum() + (dW.to(F64) * b).sum()
    # (the difference is off by O(e^2) and 1e-16 / e; the gradients by 2^-15 of their terms)
    size = (dh.to(F64) * a).abs().sum() + (dW.to(F64) * b).abs().sum()
    assert abs(float(diff - got)) <= 2.0 ** -15 * float(size) + 1e-8
    assert abs(float(loss(h, W)) - float(stats[0])) <= 1e-5 * abs(float(stats[0]))


# ----------------------------------------------------------- on the host ----
def test_refusals_on_the_host(B):
    lib = B.load()
    n = C.c_size_t(0)
    INV, WS = B.BIV_ERR_INVALID, B.BIV_ERR_WORKSPACE
    for T, V, K, ht, wt in ((-1, 8, 8, 0, 0), (4, 0, 8, 0, 0), (4, 8, 12, 0, 0), (4, 8, 8, 2, 0), (4, 8, 8, 0, 2),
                            ((1 << 20) + 1, 8, 8, 0, 0), (4, 1 << 24, 8, 0, 0)):
        assert lib.biv_lm_head_backward_workspace(T, V, K, ht, wt, C.byref(n)) == INV
    assert lib.biv_lm_head_backward_workspace(4, 8, 8, 0, 0, None) == INV
    assert lib.biv_lm_head_backward_workspace(4, 8, 8, 0, 0, C.byref(n)) == B.BIV_OK and n.value > 0
    need = n.value
    p = 0x10000000                       # never dereferenced: nothing is launched

    def grad(**kw):
        d = B.LmGradDesc(4, 8, 8, p, 8, p, 8, p, p, p, None, p, 8, 0, p, 8, 0, 0, p, need)
        for k, v in kw.items():
            setattr(d, k, v)
        return lib.biv_lm_head_backward(C.byref(d), None)

    assert lib.biv_lm_head_backward(None, None) == INV
    for bad in (dict(T=-1), dict(K=12), dict(h=None), dict(W=None), dict(target=None), dict(lse=None),
                dict(dlp=None), dict(h=p + 2), dict(ldh=7), dict(ldw=12), dict(lddh=7), dict(lddw=7),
                dict(dh_dtype=2), dict(accumulate=2), dict(dW=p + 1), dict(dh=p + 1), dict(workspace=p + 16)):
        assert grad(**bad) == INV, bad
    assert grad(workspace=None) == WS and grad(workspace_bytes=need - 1) == WS
    assert grad(dh=None, dW=None) == B.BIV_OK

    assert lib.biv_lm_head_loss_workspace(4, 8, C.byref(n)) == B.BIV_OK
    lneed = n.value

    def loss(**kw):
        d = B.LmLossDesc(4, 8, 8, p, 8, p, 8, p, None, -100, 0.0, 0, 1.0, p, p, None, None, p, p, lneed)
        for k, v in kw.items():
            setattr(d, k, v)
        return lib.biv_lm_head_loss(C.byref(d), None)

    nan = float("nan")
    for bad in (dict(T=-1), dict(V=0), dict(K=12), dict(h=None), dict(target=None), dict(lp=None), dict(lse=None),
                dict(stats=None), dict(reduce=1), dict(reduce=2, norm=0.0), dict(reduce=2, norm=nan),
                dict(z_coef=-1.0), dict(z_coef=nan), dict(workspace=p + 8), dict(ldh=4)):
        assert loss(**bad) == INV, bad
    assert loss(workspace=None) == WS and loss(workspace_bytes=lneed - 1) == WS


@gpu
def test_refusals_of_the_binding(B):
    c = Case(8, 100, 64)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    dh, dW = torch.empty(8, 64, device="cuda"), torch.empty(100, 64, device="cuda")
    ok = dict(h=c.h, W=c.W, target=c.target, lse=c.lse, dlp=c.dlp, dh=dh, dW=dW, workspace=ws)
    for bad in (dict(h=c.h.float()), dict(h=c.h[:, :32]), dict(h=c.h.t()), dict(W=c.W.cpu()),
                dict(target=c.target.long()), dict(target=c.target[:4]), dict(lse=c.lse[:4]),
                dict(dlp=c.dlp.double()), dict(dh=dh[:4]), dict(dh=dh.half()), dict(dW=dW[:, :32]),
                dict(dlse=c.lse[:4]), dict(T=9)):
        with pytest.raises(ValueError):
            B.biv_lm_head_backward(**{**ok, **bad})
    with pytest.raises(B.BivError):
        B.biv_lm_head_backward(**{**ok, "workspace": ws[:64]})

"""RMSNorm with 8-bit outputs, and activations kept in 8 bits with their backward.

Forward outputs are compared bit for bit: with biv_add_rmsnorm, biv_silu_mul and
biv_act_quant_fp8 where they define them, and with the stated FP32 operations in
torch.  Backward passes are compared with 64 bits: an FP32 result of n operations
on a sum of magnitudes S is off by at most n 2^-24 S, expf by 2^-22 of its value,
an output in bf16 by another 2^-8 of itself."""
import ctypes as C

import pytest
import torch

gpu = pytest.mark.gpu
F64 = torch.float64
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def B():
    from invariant_forward_bitwise_gb300 import biv, build
    build.build()
    biv.load()
    return biv


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def rows_of(rows, width, pad, dtype=torch.bfloat16):
    return torch.full((rows, width + pad), 7.0, dtype=dtype, device="cuda")[:, :width]


def stream(rows, d, seed=0, spread=True):
    """Rows with a few large channels, an all-zero group, and groups of very small and large size."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, d, device="cuda", generator=g)
    x[:, ::37] *= 30
    if spread and rows > 2:
        x[1, :128] = 0
        x[2, :128] *= 2.0 ** -70
        x[rows - 1, :16] *= 2.0 ** 40
    return x


def groups(d):
    return (d + 127) // 128


def quantised(x):
    """The stated rule in FP32: codes and scales."""
    rows, d = x.shape
    n = groups(d)
    p = torch.nn.functional.pad(x, (0, n * 128 - d)).view(rows, n, 128)
    a = p.abs().amax(2)
    # (by a tensor: torch multiplies by the reciprocal of a number)
    s = torch.where(a == 0, torch.ones_like(a), a / torch.full_like(a, 448))
    q = (p / s[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(rows, n * 128)[:, :d]
    return q.contiguous().view(torch.uint8), s


def values(codes, scales, t=F64):
    d = codes.shape[1]
    return codes.view(torch.float8_e4m3fn).to(t) * scales.to(t).repeat_interleave(128, 1)[:, :d]


def u8(*s):
    return torch.full(s, 255, dtype=torch.uint8, device="cuda")


def f32(*s):
    return torch.full(s, 7.0, device="cuda")


SHAPES = [(1, 16), (3, 128), (5, 144), (17, 256), (9, 272), (33, 688), (16, 2048), (7, 2064), (4, 4096), (3, 6160),
          (3, 8192), (301, 256), (1000, 1024)]


@gpu
@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("pad", [0, 8])
def test_add_rmsnorm_bits(B, rows, d, pad):
    x, r = rows_of(rows, d, pad), rows_of(rows, d, pad)
    x.copy_(stream(rows, d, 1) * 0.3)
    r.copy_(stream(rows, d, 2))
    w = (1 + 0.2 * torch.randn(d, device="cuda")).bfloat16()
    # biv_add_rmsnorm in place, and its r' quantised
    ref_r, ref_y = rows_of(rows, d, pad), rows_of(rows, d, pad)
    ref_r.copy_(r)
    B.biv_add_rmsnorm(x, ref_r, w, ref_y, EPS)
    ref_k, ref_ks = u8(rows, d), f32(rows, groups(d))
    B.biv_act_quant_fp8(ref_r, ref_k, ref_ks)
    y, out = rows_of(rows, d, pad), rows_of(rows, d, pad)
    codes, scales, keep, ks, inv = u8(rows, d), f32(rows, groups(d)), u8(rows, d), f32(rows, groups(d)), f32(rows)
    before = r.clone()
    B.biv_add_rmsnorm_fp8(x, r, w, EPS, residual_out=out, y=y, codes=codes, scales=scales, keep=keep,
                          keep_scales=ks, inv=inv)
    assert same(r, before) and same(out, ref_r) and same(y, ref_y)
    assert same(keep, ref_k) and same(ks, ref_ks)
    v = (ref_r.float() * inv[:, None]) * w.float()
    want, want_s = quantised(v)
    assert same(scales, want_s) and same(codes, want)
    mean = ref_r.to(F64).square().mean(1)
    # (d products and sums in FP32, then a division, a root and a reciprocal)
    assert torch.allclose(inv.to(F64), 1 / (mean + EPS).sqrt(), rtol=(d + 8) * 2.0 ** -24, atol=0)
    # in place, without y, without what the backward needs: the same bits
    c2, s2 = u8(rows, d), f32(rows, groups(d))
    B.biv_add_rmsnorm_fp8(x, r, w, EPS, codes=c2, scales=s2)
    assert same(r, ref_r) and same(c2, codes) and same(s2, scales)
    # no residual: r' is x
    B.biv_add_rmsnorm(x, None, w, ref_y, EPS)
    y2, k2, ks2 = rows_of(rows, d, pad), u8(rows, d), f32(rows, groups(d))
    B.biv_add_rmsnorm_fp8(x, None, w, EPS, y=y2, keep=k2, keep_scales=ks2)
    B.biv_act_quant_fp8(x, ref_k, ref_ks)
    assert same(y2, ref_y) and same(k2, ref_k) and same(ks2, ref_ks)
    if pad:
        for t in (out, y, y2):
            assert bool((t.as_strided((rows, d + pad), (d + pad, 1))[:, d:] == 7).all())


@gpu
def test_quotients_are_those_of_a_division(B):
    """Every bf16 magnitude against many scales: the codes of an IEEE division."""
    bits = torch.arange(1, 0x7F80, device="cuda", dtype=torch.int32)
    mags = (bits << 16).view(torch.float32)                    # all positive finite bf16 values
    rows = []
    g = torch.Generator(device="cuda").manual_seed(4)
    for top in torch.randint(1, 0x7F80, (300,), device="cuda", generator=g).tolist():
        lo = max(0, top - 127 * 12)                            # from 2^-12 of the group's largest up
        pick = torch.linspace(lo, top - 1, 128, device="cuda").round().long()
        rows.append(mags[pick])
    x = torch.stack(rows).bfloat16()
    x[:, ::2] *= -1
    codes, scales = u8(300, 128), f32(300, 1)
    B.biv_add_rmsnorm_fp8(x, None, torch.ones(128, device="cuda").bfloat16(), EPS,
                          y=torch.empty_like(x), keep=codes, keep_scales=scales)
    want, ws = quantised(x.float())
    assert same(scales, ws) and same(codes, want)


@gpu
@pytest.mark.parametrize("exponent", [-50, 0, 50])
def test_every_pair_of_mantissas(B, exponent):
    """Kept codes of all 128 mantissas of a group's largest value times all bf16
    values down to 2^-13 of it: an IEEE division's.  (Scaling both by a power of
    two changes no quotient while nothing under- or overflows.)"""
    rows = []
    for m in range(128):
        top = ((127 + exponent) << 7) + m                      # bits of the largest
        below = torch.arange(top - 127 * 14, top, device="cuda", dtype=torch.int32).view(14, 127)
        rows.append(torch.cat([torch.full((14, 1), top, device="cuda", dtype=torch.int32), below], 1))
    x = (torch.cat(rows) << 16).view(torch.float32).bfloat16()
    n = x.size(0)
    codes, scales = u8(n, 128), f32(n, 1)
    B.biv_add_rmsnorm_fp8(x, None, torch.ones(128, device="cuda").bfloat16(), EPS,
                          y=torch.empty_like(x), keep=codes, keep_scales=scales)
    want, ws = quantised(x.float())
    assert same(scales, ws) and same(codes, want)
    both = torch.cat([x, x.flip(0)], 1)
    keep, ks = u8(n, 256), f32(n, 2)
    B.biv_silu_mul_keep_fp8(both, None, keep, ks)
    assert same(keep[:, :128], want) and same(keep[:, 128:], want.flip(0))
    assert same(ks[:, :1], ws) and same(ks[:, 1:], ws.flip(0))


@gpu
def test_rows_with_infinities_and_nan(B):
    x = stream(6, 272, 3, spread=False).bfloat16()
    clean = x.clone()
    x[1, 5], x[3, 200] = float("inf"), float("nan")
    w = torch.ones(272, device="cuda").bfloat16()

    def run(t):
        y, c, s, k, ks = torch.empty_like(t), u8(6, 272), f32(6, 3), u8(6, 272), f32(6, 3)
        B.biv_add_rmsnorm_fp8(t, None, w, EPS, y=y, codes=c, scales=s, keep=k, keep_scales=ks)
        return y, c, s, k, ks
    a, b = run(clean), run(x)
    ok = torch.tensor([0, 2, 4, 5], device="cuda")
    assert all(same(p[ok], q[ok]) for p, q in zip(a, b))
    y, c, _, k, _ = b
    assert bool(y[1, 5].isnan()) and bool(y[3].isnan().all())
    nan = k.view(torch.float8_e4m3fn).float().isnan()
    assert bool(nan[1, 5]) and bool(nan[3, 200]) and not bool(nan[ok].any())


@gpu
def test_an_fp8_product_reads_the_codes(B):
    """Norm, FP8 product: the codes and scales go straight into the GEMM."""
    rows, d, N = 70, 512, 256
    x = stream(rows, d, 8, spread=False).bfloat16()
    w = torch.ones(d, device="cuda").bfloat16()
    codes, scales, y = u8(rows, d), f32(rows, 4), torch.empty_like(x)
    B.biv_add_rmsnorm_fp8(x, None, w, EPS, y=y, codes=codes, scales=scales)
    W = torch.randn(N, d, device="cuda").to(torch.float8_e4m3fn)
    sb = torch.rand(N // 128, d // 128, device="cuda") + 0.5
    out = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    B.biv_gemm(B.gemm_desc(codes, W.view(torch.uint8), out, sa=scales, sb=sb))
    Wd = W.to(F64) * sb.to(F64).repeat_interleave(128, 0).repeat_interleave(128, 1)
    a = values(codes, scales)
    want, size = a @ Wd.t(), a.abs() @ Wd.abs().t()
    assert bool(((out.to(F64) - want).abs() <= 2.0 ** -8 * want.abs() + d * 2.0 ** -22 * size).all())
    # and the codes stand for y to e4m3's half step (2^-4 of the value, or of the smallest normal code)
    yd = y.to(F64)
    s = scales.to(F64).repeat_interleave(128, 1)
    assert bool(((a - yd).abs() <= 2.0 ** -4 * yd.abs() * (1 + 2.0 ** -4) + s * 2.0 ** -10 + 2.0 ** -8 * yd.abs()).all())


def rounding(t):
    return 2.0 ** -8 if t is torch.bfloat16 else 2.0 ** -24


@gpu
@pytest.mark.parametrize("rows,d", SHAPES + [(2500, 64), (3000, 2048)])
@pytest.mark.parametrize("dy_t,dx_t", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("res", [True, False])
def test_rmsnorm_backward(B, rows, d, dy_t, dx_t, res):
    dy_t, dx_t = TYPES[dy_t], TYPES[dx_t]
    pad = 8 if rows % 2 else 0
    x = stream(rows, d, rows, spread=False)
    keep, ks = quantised(x.bfloat16().float())
    inv = torch.rsqrt(x.square().mean(1) + EPS)
    g = torch.Generator(device="cuda").manual_seed(d)
    w = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).bfloat16()
    dy, dx = rows_of(rows, d, pad, dy_t), rows_of(rows, d, pad, dx_t)
    dy.copy_(torch.randn(rows, d, device="cuda", generator=g))
    dres = torch.randn(rows, d, device="cuda", generator=g).to(dx_t) if res else None
    dw = f32(d)
    ws = torch.empty(B.biv_rmsnorm_backward_fp8_workspace(rows, d), dtype=torch.uint8, device="cuda").fill_(255)
    B.biv_rmsnorm_backward_fp8(keep, ks, inv, w, dy, dx, dw, ws, dres=dres)
    xv, dv, iv = values(keep, ks), dy.to(F64), inv.to(F64)[:, None]
    gw = dv * w.to(F64)
    want = iv * gw - xv * iv ** 3 * (gw * xv).mean(1, keepdim=True)
    size = iv * gw.abs() + xv.abs() * iv ** 3 * (gw * xv).abs().mean(1, keepdim=True)
    if res:
        want, size = want + dres.to(F64), size + dres.to(F64).abs()
    tol = (d + 16) * 2.0 ** -24 * size
    assert bool(((dx.to(F64) - want).abs() <= tol + rounding(dx_t) * (want.abs() + tol)).all())
    t = dv * xv * iv
    assert bool(((dw.to(F64) - t.sum(0)).abs() <= (rows + 8) * 2.0 ** -24 * t.abs().sum(0) + 1e-38).all())
    if pad:
        assert bool((dx.as_strided((rows, d + pad), (d + pad, 1))[:, d:] == 7).all())
    # again, added to dw, dx over dres
    more, over = dw.clone(), dres.clone() if res else None
    B.biv_rmsnorm_backward_fp8(keep, ks, inv, w, dy, over if res else dx, more, ws, dres=over, accumulate=True)
    assert same(over if res else dx, dx) and same(more, dw + dw)
    if dy_t is dx_t:      # dx over dy
        B.biv_rmsnorm_backward_fp8(keep, ks, inv, w, dy, dy, dw, ws, dres=dres)
        assert same(dy, dx)


@gpu
def test_rmsnorm_backward_no_rows(B):
    e = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    w, ws, dw = torch.ones(64, device="cuda").bfloat16(), e(64, t=torch.uint8), torch.ones(64, device="cuda")
    args = (e(0, 64, t=torch.uint8), e(0, 1), e(0), w, e(0, 64), e(0, 64))
    B.biv_rmsnorm_backward_fp8(*args, dw, ws, accumulate=True)
    assert bool((dw == 1).all())
    B.biv_rmsnorm_backward_fp8(*args, dw, ws)
    assert bool((dw == 0).all())


@gpu
@pytest.mark.parametrize("rows,I", [(1, 16), (3, 128), (7, 144), (13, 688), (5, 1408), (300, 256), (2, 6144), (1, 40000)])
@pytest.mark.parametrize("pad", [0, 8])
def test_silu_mul_keep_bits(B, rows, I, pad):  # noqa: E741
    gu = rows_of(rows, 2 * I, pad)
    gu.copy_(stream(rows, 2 * I, 6))
    y, ref = rows_of(rows, I, pad), rows_of(rows, I, pad)
    B.biv_silu_mul(gu, ref)
    keep, ks = u8(rows, 2 * I), f32(rows, 2 * groups(I))
    B.biv_silu_mul_keep_fp8(gu, y, keep, ks)
    assert same(y, ref)
    for half in (0, 1):
        want, s = quantised(gu[:, half * I:half * I + I].float())
        assert same(keep[:, half * I:half * I + I], want)
        assert same(ks[:, half * groups(I):(half + 1) * groups(I)], s)
    k2, ks2 = u8(rows, 2 * I), f32(rows, 2 * groups(I))
    B.biv_silu_mul_keep_fp8(gu, None, k2, ks2)
    assert same(k2, keep) and same(ks2, ks)
    if pad:
        assert bool((y.as_strided((rows, I + pad), (I + pad, 1))[:, I:] == 7).all())


@gpu
@pytest.mark.parametrize("rows,I", [(1, 16), (3, 128), (7, 144), (13, 688), (5, 1408), (300, 256), (2, 6144)])
@pytest.mark.parametrize("dy_t,dg_t", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
def test_silu_mul_backward(B, rows, I, dy_t, dg_t):  # noqa: E741
    dy_t, dg_t = TYPES[dy_t], TYPES[dg_t]
    pad = 8 if rows % 2 else 0
    x = stream(rows, 2 * I, I, spread=False)
    (kg, sg), (ku, su) = quantised(x[:, :I].bfloat16().float()), quantised(x[:, I:].bfloat16().float())
    keep, ks = torch.cat([kg, ku], 1), torch.cat([sg, su], 1)
    dy, dgu, y = rows_of(rows, I, pad, dy_t), rows_of(rows, 2 * I, pad, dg_t), rows_of(rows, I, pad)
    dy.copy_(stream(rows, I, 9, spread=False))
    B.biv_silu_mul_backward_fp8(keep, ks, dy, dgu, y=y)
    g, u, d = values(kg, sg), values(ku, su), dy.to(F64)
    s = torch.sigmoid(g)
    # 10 FP32 operations and one expf; 1 + g (1 - s) may cancel: its parts are counted.  The
    # operations include gate = code * s: a relative error of 2^-24 in the exponent, so one of
    # |g| 2^-24 in e^-g, and with it in the sigmoid and in 1 - s.  Where e^-g overflows (g < -88.7)
    # the sigmoid becomes 0, and products below 2^-126 may too
    for got, want, size, t in (
            (dgu[:, :I], d * u * s * (1 + g * (1 - s)), (d * u).abs() * (1 + g.abs()), dg_t),
            (dgu[:, I:], d * g * s, (d * g).abs(), dg_t), (y, g * s * u, (g * u).abs(), torch.bfloat16)):
        tol = ((10 + 2 * g.abs()) * 2.0 ** -24 + 2 * 2.0 ** -22) * size * s + 2.0 ** -126 * (1 + size)
        assert bool(((got.to(F64) - want).abs() <= tol + rounding(t) * (want.abs() + tol)).all())
    again = torch.empty(rows, 2 * I, dtype=dg_t, device="cuda")
    B.biv_silu_mul_backward_fp8(keep, ks, dy, again)
    assert same(again, dgu)
    if pad:
        assert bool((dgu.as_strided((rows, 2 * I + pad), (2 * I + pad, 1))[:, 2 * I:] == 7).all())


@gpu
def test_every_gate_divides_exactly(B):
    """silu(gate) of all 65536 bf16 gates, alone in their groups with zeros and among
    others, has biv_silu_mul's bits (the quotient is formed without a division)."""
    g = torch.arange(65536, device="cuda").to(torch.int32)
    g = g.to(torch.int16).view(torch.bfloat16)
    rows = [g.view(512, 128)]                                  # neighbours: groups of one exponent
    rows.append(g.view(128, 512).t().contiguous().view(512, 128))     # groups of all magnitudes
    alone = torch.zeros(65536 // 8, 128, dtype=torch.bfloat16, device="cuda")
    alone[:, ::16] = g.view(-1, 8)
    rows.append(alone)
    for gate in rows:
        for up in (1.0, -0.7265625, 3e38, 1e-30):
            gu = torch.cat([gate, torch.full_like(gate, up)], 1)
            y, ref = torch.empty_like(gate), torch.empty_like(gate)
            B.biv_silu_mul(gu, ref)
            keep, ks = u8(gate.size(0), 256), f32(gate.size(0), 2)
            B.biv_silu_mul_keep_fp8(gu, y, keep, ks)
            assert bool((y.isnan() == ref.isnan()).all())
            assert same(torch.where(ref.isnan(), 0.0, y), torch.where(ref.isnan(), 0.0, ref))


@gpu
def test_large_gates(B):
    """Gates where exp overflows or vanishes: the limits, no NaN."""
    g = torch.tensor([[-448.0, -200.0, -100.0, -88.0, 88.0, 100.0, 200.0, 448.0] * 2], device="cuda")
    keep, ks = u8(1, 32), torch.ones(1, 2, device="cuda")
    keep[:, :16] = g.to(torch.float8_e4m3fn).view(torch.uint8)
    keep[:, 16:] = torch.ones(1, 16, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    dgu, y = torch.empty(1, 32, device="cuda"), torch.empty(1, 16, dtype=torch.bfloat16, device="cuda")
    B.biv_silu_mul_backward_fp8(keep, ks, torch.ones(1, 16, device="cuda"), dgu, y=y)
    v = keep.view(torch.float8_e4m3fn).to(F64)[:, :16]
    assert bool(dgu.isfinite().all()) and bool(y.isfinite().all())
    assert torch.allclose(dgu[:, :16].to(F64), (v > 0).to(F64), atol=1e-30)
    assert torch.allclose(dgu[:, 16:].to(F64), v.clamp_min(0), atol=1e-30)


@gpu
def test_differences_through_norm_and_mlp(B):
    """Norm, then SiLU-mul of its halves: the chain of both backward passes along a
    direction, against a difference of the function of the kept values in 64 bits."""
    rows, d = 12, 512
    I = d // 2  # noqa: E741
    x = stream(rows, d, 2, spread=False).bfloat16()
    w = (1 + 0.2 * torch.randn(d, device="cuda")).bfloat16()
    y, keep, ks, inv = torch.empty_like(x), u8(rows, d), f32(rows, 4), f32(rows)
    B.biv_add_rmsnorm_fp8(x, None, w, EPS, y=y, keep=keep, keep_scales=ks, inv=inv)
    xv = values(keep, ks)
    inv = (1 / (xv.square().mean(1) + EPS).sqrt()).float()       # of the kept values, as the difference sees it
    v = xv * inv.to(F64)[:, None] * w.to(F64)
    k2, s2 = u8(rows, d), f32(rows, 4)
    B.biv_silu_mul_keep_fp8(v.bfloat16(), None, k2, s2)
    gv = torch.cat([values(k2[:, :I].contiguous(), s2[:, :2]), values(k2[:, I:].contiguous(), s2[:, 2:])], 1)
    g = torch.Generator(device="cuda").manual_seed(1)
    dy = torch.randn(rows, I, device="cuda", generator=g)
    dgu, dx, dw = torch.empty(rows, d, device="cuda"), torch.empty(rows, d, device="cuda"), f32(d)
    B.biv_silu_mul_backward_fp8(k2, s2, dy, dgu)
    ws = torch.empty(B.biv_rmsnorm_backward_fp8_workspace(rows, d), dtype=torch.uint8, device="cuda")
    B.biv_rmsnorm_backward_fp8(keep, ks, inv, w, dgu, dx, dw, ws)

    def mlp(t):
        return (torch.nn.functional.silu(t[:, :I]) * t[:, I:] * dy.to(F64)).sum()

    def norm(t, wt):
        return (t / (t.square().mean(1, keepdim=True) + EPS).sqrt() * wt * dgu.to(F64)).sum()

    a = torch.randn(rows, d, device="cuda", generator=g, dtype=F64)
    b = torch.randn(d, device="cuda", generator=g, dtype=F64)
    e = 1e-6
    diff = (mlp(gv + e * a) - mlp(gv - e * a)) / (2 * e)
    assert abs(float(diff - (dgu.to(F64) * a).sum())) <= 2.0 ** -16 * float((dgu.to(F64) * a).abs().sum())
    wt = w.to(F64)
    diff = (norm(xv + e * a, wt + e * b) - norm(xv - e * a, wt - e * b)) / (2 * e)
    got, size = (dx.to(F64) * a).sum() + (dw.to(F64) * b).sum(), (dx.to(F64) * a).abs().sum() + (dw.to(F64) * b).abs().sum()
    assert abs(float(diff - got)) <= 2.0 ** -14 * float(size)


@gpu
def test_offsets_beyond_32_bits(B):
    """More than 2^31 elements of gate_up, kept rows and gradients."""
    rows, I = 90000, 12288  # noqa: E741
    gu = torch.empty(rows, 2 * I, dtype=torch.bfloat16, device="cuda")
    tail = stream(64, 2 * I, 3, spread=False).bfloat16()
    gu.zero_()
    gu[-64:] = tail
    y, keep, ks = torch.empty(rows, I, dtype=torch.bfloat16, device="cuda"), u8(rows, 2 * I), f32(rows, 2 * groups(I))
    B.biv_silu_mul_keep_fp8(gu, y, keep, ks)
    y2, k2, s2 = torch.empty(64, I, dtype=torch.bfloat16, device="cuda"), u8(64, 2 * I), f32(64, 2 * groups(I))
    B.biv_silu_mul_keep_fp8(tail, y2, k2, s2)
    assert same(y[-64:], y2) and same(keep[-64:], k2) and same(ks[-64:], s2) and bool((ks[:-64] == 1).all())
    dgu, small = torch.empty_like(gu), torch.empty_like(tail)
    B.biv_silu_mul_backward_fp8(keep, ks, y, dgu)
    B.biv_silu_mul_backward_fp8(k2, s2, y2, small)
    assert same(dgu[-64:], small) and bool((dgu[:-64] == 0).all())


@gpu
def test_a_graph_and_other_streams_repeat_the_bits(B):
    rows, d = 500, 2048
    x, r = stream(rows, d, 1).bfloat16(), stream(rows, d, 2).bfloat16()
    w = torch.ones(d, device="cuda").bfloat16()
    dy = stream(rows, d, 3, spread=False).bfloat16()
    gdy = stream(rows, d // 2, 4, spread=False).bfloat16()

    def outputs():
        return dict(out=torch.empty_like(x), y=torch.empty_like(x), codes=u8(rows, d), scales=f32(rows, 16),
                    keep=u8(rows, d), ks=f32(rows, 16), inv=f32(rows), dx=torch.empty_like(x), dw=f32(d),
                    a=torch.empty_like(gdy), k2=u8(rows, d), s2=f32(rows, 16), dgu=torch.empty_like(x),
                    ws=torch.empty(B.biv_rmsnorm_backward_fp8_workspace(rows, d), dtype=torch.uint8, device="cuda"))

    def run(o, s=None):
        B.biv_add_rmsnorm_fp8(x, r, w, EPS, residual_out=o["out"], y=o["y"], codes=o["codes"], scales=o["scales"],
                              keep=o["keep"], keep_scales=o["ks"], inv=o["inv"], stream=s)
        B.biv_silu_mul_keep_fp8(o["y"], o["a"], o["k2"], o["s2"], stream=s)
        B.biv_silu_mul_backward_fp8(o["k2"], o["s2"], gdy, o["dgu"], stream=s)
        B.biv_rmsnorm_backward_fp8(o["keep"], o["ks"], o["inv"], w, o["dgu"], o["dx"], o["dw"], o["ws"], dres=dy,
                                   stream=s)

    ref, captured = outputs(), outputs()
    run(ref)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(captured)
    for _ in range(2):
        g.replay()
    others = [(torch.cuda.Stream(), outputs()) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o in others:
            run(o, s)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    for o in [captured] + [o for _, o in others]:
        for k in ref:
            if k != "ws":
                assert same(ref[k], o[k]), k


@gpu
@pytest.mark.parametrize("exponent", [-50, -42, 42, 50, 56])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_rmsnorm_backward_of_large_and_small_rows(B, exponent, t):
    """Rows of 2^42 and more, whose inv^3 is below FP32's range, and of 2^-42 and less
    (eps 0), whose inv^3 is above it, beside ordinary ones: the projection is there."""
    rows, d, t = 9, 272, TYPES[t]
    x = stream(rows, d, 5, spread=False)
    x[::2] *= 2.0 ** exponent
    keep, ks = quantised(x.bfloat16().float())
    inv = (1 / x.to(F64).square().mean(1).sqrt()).float()
    g = torch.Generator(device="cuda").manual_seed(d)
    w = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).bfloat16()
    xh = values(keep, ks) * inv.to(F64)[:, None]
    # a gradient along the row, of the row's size: dx is of the order of 1
    dy = ((xh + torch.randn(rows, d, device="cuda", generator=g)) / inv[:, None]).to(t)
    dx, dw = torch.empty(rows, d, dtype=t, device="cuda"), f32(d)
    ws = torch.empty(B.biv_rmsnorm_backward_fp8_workspace(rows, d), dtype=torch.uint8, device="cuda")
    B.biv_rmsnorm_backward_fp8(keep, ks, inv, w, dy, dx, dw, ws)
    iv, gw = inv.to(F64)[:, None], dy.to(F64) * w.to(F64)
    want = iv * (gw - xh * (gw * xh).mean(1, keepdim=True))
    size = iv * (gw.abs() + xh.abs() * (gw * xh).abs().mean(1, keepdim=True))
    tol = (d + 16) * 2.0 ** -24 * size
    assert bool(((dx.to(F64) - want).abs() <= tol + rounding(t) * (want.abs() + tol)).all())
    terms = dy.to(F64) * xh
    assert bool(((dw.to(F64) - terms.sum(0)).abs() <= (rows + 8) * 2.0 ** -24 * terms.abs().sum(0) + 1e-38).all())

@gpu
def test_silu_mul_keeps_groups_of_nan_and_infinities(B):
    """Kept codes and scales of groups that hold NaN and infinities, alone and among
    others, are those that biv_act_quant_fp8 writes of each half."""
    rows, I = 8, 272  # noqa: E741
    gu = stream(rows, 2 * I, 3, spread=False).bfloat16()
    nan, inf = float("nan"), float("inf")
    gu[0, :128] = nan                       # a whole group, of gate
    gu[1, I + 128:I + 256] = nan            # of up
    gu[2, 256:I] = nan                      # the last, short one
    gu[3, ::3] = nan
    gu[4, 7], gu[4, I + 9] = inf, -inf
    gu[5, :128], gu[5, I:I + 128] = inf, -inf
    gu[6, 0], gu[6, 1:128] = inf, nan
    y, keep, ks = torch.empty(rows, I, dtype=torch.bfloat16, device="cuda"), u8(rows, 2 * I), f32(rows, 2 * groups(I))
    B.biv_silu_mul_keep_fp8(gu, y, keep, ks)
    ref = torch.empty_like(y)
    B.biv_silu_mul(gu, ref)
    assert bool((y.isnan() == ref.isnan()).all())
    assert same(torch.where(ref.isnan(), 0.0, y), torch.where(ref.isnan(), 0.0, ref))
    for half in (0, 1):
        want, s = u8(rows, I), f32(rows, groups(I))
        B.biv_act_quant_fp8(gu[:, half * I:half * I + I].contiguous(), want, s)
        assert same(keep[:, half * I:half * I + I], want)
        assert same(ks[:, half * groups(I):(half + 1) * groups(I)], s)

@gpu
def test_zeros_keep_their_sign(B):
    """The code of -0 is 0x80, as the rule's quotient -0 / s and biv_act_quant_fp8 give it:
    of zeros of r', of the normed rows (0 times a negative weight), of gate and of up."""
    rows, d = 6, 272
    x = stream(rows, d, 8, spread=False).bfloat16()
    x[:, ::5], x[:, 1::5] = 0.0, -0.0
    x[5, :128] = -0.0                       # a group of zeros alone
    w = torch.where(torch.arange(d, device="cuda") % 3 == 0, -1.0, 1.5).bfloat16()
    c, s, k, ks, inv = u8(rows, d), f32(rows, groups(d)), u8(rows, d), f32(rows, groups(d)), f32(rows)
    B.biv_add_rmsnorm_fp8(x, None, w, EPS, codes=c, scales=s, keep=k, keep_scales=ks, inv=inv)
    want, wants = u8(rows, d), f32(rows, groups(d))
    B.biv_act_quant_fp8(x, want, wants)
    assert bool((want[:, 1::5] == 0x80).all()) and bool((want[:5, ::5] == 0).all())
    assert same(k, want) and same(ks, wants)
    v = (x.float() * inv[:, None]) * w.float()
    want, wants = quantised(v)
    assert bool((want[:, 1::15] == 0x80).any())
    assert same(c, want) and same(s, wants)
    both = torch.cat([x, x.flip(0)], 1)
    keep, ks2 = u8(rows, 2 * d), f32(rows, 2 * groups(d))
    B.biv_silu_mul_keep_fp8(both, None, keep, ks2)
    assert same(keep[:, :d], k) and same(keep[:, d:], k.flip(0)) and same(ks2[:, :groups(d)], ks)

@gpu
def test_silu_mul_backward_in_fp32_has_the_bf16_forms_bits(B):
    """Kept values that bf16 holds (every finite gate that a code and a power of two
    make, and many ups): FP32 gradients are biv_silu_mul_backward's, bit for bit."""
    codes = torch.arange(256, device="cuda", dtype=torch.uint8)
    codes = codes[(codes & 0x7F) != 0x7F]                       # no NaN
    g = torch.Generator(device="cuda").manual_seed(3)
    rows, I = 24, 256  # noqa: E741
    pick = lambda: codes[torch.randint(0, codes.numel(), (rows, I), device="cuda", generator=g)]  # noqa: E731
    kg, ku = pick(), pick()
    kg[:, :254] = codes
    sg = (2.0 ** torch.arange(-18, 6, device="cuda", dtype=torch.float32))[:, None].expand(rows, 2).contiguous()
    su = 2.0 ** torch.randint(-9, 3, (rows, 2), device="cuda", generator=g).float()
    keep, ks = torch.cat([kg, ku], 1), torch.cat([sg, su], 1)
    gate_up = torch.cat([values(kg, sg), values(ku, su)], 1)
    assert bool((gate_up == gate_up.bfloat16().to(F64)).all())
    for t in ("f32", "bf16"):
        dy = torch.randn(rows, I, device="cuda", generator=g).to(TYPES[t])
        got, ref = torch.empty(rows, 2 * I, device="cuda"), torch.empty(rows, 2 * I, device="cuda")
        B.biv_silu_mul_backward_fp8(keep, ks, dy, got)
        B.biv_silu_mul_backward(gate_up.bfloat16(), dy.float(), ref)
        assert same(got, ref)

@gpu
@pytest.mark.parametrize("rows,d", [(5, 144), (33, 688), (16, 2048), (3, 8192)])
def test_add_rmsnorm_over_its_input(B, rows, d):
    """y over x and r' over the residual: the bits of separate outputs."""
    x, r = stream(rows, d, 1).bfloat16(), stream(rows, d, 2).bfloat16()
    w = (1 + 0.2 * torch.randn(d, device="cuda")).bfloat16()

    def run(x, r, y, out):
        c, s, k, ks, inv = u8(rows, d), f32(rows, groups(d)), u8(rows, d), f32(rows, groups(d)), f32(rows)
        B.biv_add_rmsnorm_fp8(x, r, w, EPS, residual_out=out, y=y, codes=c, scales=s, keep=k, keep_scales=ks, inv=inv)
        return [c, s, k, ks, inv, y, r if out is None else out]
    apart = run(x, r, torch.empty_like(x), torch.empty_like(r))
    assert all(same(a, b) for a, b in zip(apart, run(x, r, x, r)))


@gpu
def test_norm_offsets_beyond_32_bits(B):
    """More than 2^31 elements of rows, kept rows and gradients."""
    rows, d = 263000, 8192
    e = lambda n, t: torch.empty(n, d, dtype=t, device="cuda")  # noqa: E731
    x, y, k, dx = e(rows, torch.bfloat16), e(rows, torch.bfloat16), e(rows, torch.uint8), e(rows, torch.bfloat16)
    tail = stream(64, d, 3, spread=False).bfloat16()
    x.fill_(1.0)
    x[-64:] = tail
    w = torch.ones(d, device="cuda").bfloat16()
    ks, inv, dw = f32(rows, groups(d)), f32(rows), f32(d)
    B.biv_add_rmsnorm_fp8(x, None, w, EPS, y=y, keep=k, keep_scales=ks, inv=inv)
    y2, k2, s2, i2 = e(64, torch.bfloat16), u8(64, d), f32(64, groups(d)), f32(64)
    B.biv_add_rmsnorm_fp8(tail, None, w, EPS, y=y2, keep=k2, keep_scales=s2, inv=i2)
    assert same(y[-64:], y2) and same(k[-64:], k2) and same(ks[-64:], s2) and same(inv[-64:], i2)
    assert bool((y[:-64] == 1).all())
    ws = torch.empty(B.biv_rmsnorm_backward_fp8_workspace(rows, d), dtype=torch.uint8, device="cuda")
    B.biv_rmsnorm_backward_fp8(k, ks, inv, w, x, dx, dw, ws)
    small, dws = e(64, torch.bfloat16), f32(d)
    B.biv_rmsnorm_backward_fp8(k2, s2, i2, w, tail, small, dws, ws)
    assert same(dx[-64:], small)
    # (rows of ones along themselves have no gradient: what is left are roundings of 1)
    assert float(dx[:-64].abs().max()) <= (d + 16) * 2.0 ** -23

# ----------------------------------------------------------- on the host ----
def test_refusals_on_the_host(B):
    lib = B.load()
    INV, WS = B.BIV_ERR_INVALID, B.BIV_ERR_WORKSPACE
    n = C.c_size_t(0)
    p = 0x10000000                       # never dereferenced: nothing is launched

    def norm(**kw):
        d = B.NormFp8Desc(p, 32, p, 32, p, 32, p, p, 32, p, p, p, p, p, 4, 32, EPS)
        for k, v in kw.items():
            setattr(d, k, v)
        return lib.biv_add_rmsnorm_fp8(C.byref(d), None)

    assert lib.biv_add_rmsnorm_fp8(None, None) == INV and norm(rows=0) == B.BIV_OK
    for bad in (dict(rows=-1), dict(d=24), dict(d=8208), dict(x=None), dict(x=p + 2), dict(x_stride=31),
                dict(x_stride=36), dict(w=None), dict(residual=p + 2), dict(r_stride=16), dict(residual_out=p + 2),
                dict(ro_stride=16), dict(residual=None), dict(y=p + 2), dict(y_stride=16), dict(scales=None),
                dict(codes=None), dict(codes=p + 1), dict(keep=None), dict(keep_scales=None),
                dict(y=None, codes=None, scales=None)):
        assert norm(**bad) == INV, bad

    assert lib.biv_rmsnorm_backward_fp8_workspace(4, 32, C.byref(n)) == B.BIV_OK
    need = n.value
    for rows, d in ((-1, 32), (4, 0), (4, 8208)):
        assert lib.biv_rmsnorm_backward_fp8_workspace(rows, d, C.byref(n)) == INV

    def back(**kw):
        d = B.NormBwdFp8Desc(p, p, p, p, p, 32, 1, p, 32, p, 32, 1, p, 0, 4, 32, p, need)
        for k, v in kw.items():
            setattr(d, k, v)
        return lib.biv_rmsnorm_backward_fp8(C.byref(d), None)

    for bad in (dict(rows=-1), dict(d=24), dict(keep=None), dict(keep_scales=None), dict(inv=None), dict(w=None),
                dict(dy=None), dict(dy=p + 4), dict(dy_stride=16), dict(dy_dtype=2), dict(dx=None), dict(dx_dtype=5),
                dict(dx_stride=34), dict(dres=p + 8), dict(dres_stride=8), dict(dw=None), dict(accumulate=3),
                dict(workspace=p + 4)):
        assert back(**bad) == INV, bad
    assert back(workspace=None) == WS and back(workspace_bytes=need - 1) == WS

    def keep(gu=p, gs=64, y=p, ys=32, k=p, s=p, rows=4, I=32):  # noqa: E741
        return lib.biv_silu_mul_keep_fp8(gu, gs, y, ys, k, s, rows, I, None)

    assert keep(rows=0) == B.BIV_OK
    for bad in (dict(gu=None), dict(gu=p + 2), dict(gs=32), dict(y=p + 2), dict(ys=16), dict(k=None), dict(s=None),
                dict(k=p + 1), dict(rows=-1), dict(I=24), dict(I=0)):
        assert keep(**bad) == INV, bad

    def sback(k=p, s=p, dy=p, dys=32, yt=1, dg=p, dgs=64, gt=1, y=p, ys=32, rows=4, I=32):  # noqa: E741
        return lib.biv_silu_mul_backward_fp8(k, s, dy, dys, yt, dg, dgs, gt, y, ys, rows, I, None)

    assert sback(rows=0) == B.BIV_OK
    for bad in (dict(k=None), dict(k=p + 1), dict(s=None), dict(dy=None), dict(dys=16), dict(yt=2), dict(dg=None),
                dict(dgs=32), dict(gt=-1), dict(y=p + 2), dict(ys=8), dict(rows=-1), dict(I=40)):
        assert sback(**bad) == INV, bad


@gpu
def test_refusals_of_the_binding(B):
    x = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(32, device="cuda").bfloat16()
    y, c, s = torch.empty_like(x), u8(4, 32), f32(4, 1)
    for bad in (dict(x=x.float()), dict(x=x.cpu()), dict(w=w[:16]), dict(y=y.float()), dict(codes=c), dict(y=y[:2]),
                dict(codes=c[:2], scales=s), dict(codes=c, scales=s[:2]), dict(keep=c), dict(inv=s[:3, 0]),
                dict(residual=x.t().contiguous().t())):
        with pytest.raises(ValueError):
            B.biv_add_rmsnorm_fp8(**{**dict(x=x, residual=None, w=w, eps=EPS, y=y), **bad})
    with pytest.raises(B.BivError):
        B.biv_add_rmsnorm_fp8(x, None, w, EPS)
    dy, ws = torch.empty(4, 32, device="cuda"), u8(1 << 16)
    ok = dict(keep=c, keep_scales=s, inv=f32(4), w=w, dy=dy, dx=torch.empty_like(dy), dw=f32(32), workspace=ws)
    for bad in (dict(keep=c[:2]), dict(dy=dy.half()), dict(dx=y[:2]), dict(dres=x), dict(dw=f32(16)), dict(inv=f32(2))):
        with pytest.raises(ValueError):
            B.biv_rmsnorm_backward_fp8(**{**ok, **bad})
    with pytest.raises(ValueError):
        B.biv_silu_mul_keep_fp8(x[:, :31], None, c, s)
    with pytest.raises(ValueError):
        B.biv_silu_mul_backward_fp8(c, f32(4, 1), dy[:, :16], x.half())

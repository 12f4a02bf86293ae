"""The end of a trainer's step with its large arrays left out or kept in 8 bits: norm,
MLP, norm, LM-head loss, their gradients from what was kept, and the optimizer step,
as one run, eager and captured.

The whole chain is formed again in 64 bits from the arrays that the forward left
(kept codes, the bf16 inputs of the products, lse).  Against that, every step of the
run is FP32: sums of at most 4096 products, each off by at most 4096 2^-23 of its
magnitudes, and exp of a logit that is off by 256 2^-23 of its magnitudes (about 5
here); in the 2-norm, where such errors are far from aligned, 2^-11 of the result
bounds the chain of nine of them (each at most 4096 2^-23 / 8 = 2^-14 there).  The LM
head's p terms carry 2^-16 besides."""
import pytest
import torch

pytestmark = pytest.mark.gpu
F64 = torch.float64
T, D, WIDE, V = 300, 256, 688, 4100      # rows, hidden, MLP width, vocabulary
EPS = 1e-6


@pytest.fixture(scope="module")
def B():
    from invariant_forward_bitwise_gb300 import biv, build
    build.build()
    biv.load()
    return biv


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def values(codes, scales):
    """What kept rows stand for, in 64 bits."""
    return codes.view(torch.float8_e4m3fn).to(F64) * scales.to(F64).repeat_interleave(128, 1)[:, :codes.shape[1]]


class Tail:
    """Weights, inputs and every buffer of the run."""

    def __init__(self, B, seed=0):
        from invariant_forward_bitwise_gb300.optim import AdamW
        self.B = B
        g = torch.Generator(device="cuda").manual_seed(seed)
        bf = lambda *s, by=1.0: (torch.randn(*s, device="cuda", generator=g) * by).bfloat16()  # noqa: E731
        e = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device="cuda")                # noqa: E731
        b16, u8 = torch.bfloat16, torch.uint8
        self.attn, self.res = bf(T, D, by=0.5), bf(T, D)
        self.w1, self.w2 = 1 + bf(D, by=0.1), 1 + bf(D, by=0.1)
        self.Wgu, self.Wd, self.Wh = bf(2 * WIDE, D, by=0.08), bf(D, WIDE, by=0.05), bf(V, D, by=0.15)
        self.target = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
        self.target[:77] = -100                       # a prompt
        self.weight = 0.5 + torch.rand(T, device="cuda", generator=g)
        self.r1, self.y1, self.r2, self.y2 = (e(T, D, t=b16) for _ in range(4))
        self.k1, self.s1, self.i1 = e(T, D, t=u8), e(T, 2), e(T)
        self.k2, self.s2, self.i2 = e(T, D, t=u8), e(T, 2), e(T)
        self.gu, self.act, self.m = e(T, 2 * WIDE, t=b16), e(T, WIDE, t=b16), e(T, D, t=b16)
        self.kg, self.sg = e(T, 2 * WIDE, t=u8), e(T, 2 * ((WIDE + 127) // 128))
        self.lp, self.lse, self.dlp, self.dlse = (e(T) for _ in range(4))
        self.stats = e(4)
        self.dy2, self.dr2, self.dr1 = (e(T, D) for _ in range(3))
        self.dWh, self.dWd, self.dWgu = e(V, D), e(D, WIDE), e(2 * WIDE, D)
        self.dw1, self.dw2 = e(D), e(D)
        self.dgu, self.act2 = e(T, 2 * WIDE), e(T, WIDE, t=b16)
        self.ws = e(64 << 20, t=u8)
        self.lws = e(B.biv_lm_head_loss_workspace(T, V), t=u8)
        self.gws = e(B.biv_lm_head_backward_workspace(T, V, D, torch.float32, torch.float32), t=u8)
        self.nws = e(B.biv_rmsnorm_backward_fp8_workspace(T, D), t=u8)
        self.params = [self.Wh, self.Wd, self.Wgu, self.w1, self.w2]
        self.opt = AdamW(self.params, [self.dWh, self.dWd, self.dWgu, self.dw1, self.dw2], lr=0.01, max_norm=1.0)

    def run(self):
        B = self.B
        B.biv_add_rmsnorm_fp8(self.attn, self.res, self.w1, EPS, residual_out=self.r1, y=self.y1, keep=self.k1,
                              keep_scales=self.s1, inv=self.i1)
        B.biv_gemm(B.gemm_desc(self.y1, self.Wgu, self.gu), self.ws)
        B.biv_silu_mul_keep_fp8(self.gu, self.act, self.kg, self.sg)
        B.biv_gemm(B.gemm_desc(self.act, self.Wd, self.m), self.ws)
        B.biv_add_rmsnorm_fp8(self.m, self.r1, self.w2, EPS, residual_out=self.r2, y=self.y2, keep=self.k2,
                              keep_scales=self.s2, inv=self.i2)
        B.biv_lm_head_loss(self.y2, self.Wh, self.target, self.lp, self.lse, self.stats, self.lws, weight=self.weight,
                           dlp=self.dlp, dlse=self.dlse, z_coef=1e-2)
        # (gu, act and the norms' inputs are not needed from here on)
        B.biv_lm_head_backward(self.y2, self.Wh, self.target, self.lse, self.dlp, self.dy2, self.dWh, self.gws,
                               dlse=self.dlse)
        B.biv_rmsnorm_backward_fp8(self.k2, self.s2, self.i2, self.w2, self.dy2, self.dr2, self.dw2, self.nws)
        self.dact = self.dr2 @ self.Wd.float()
        B.biv_silu_mul_backward_fp8(self.kg, self.sg, self.dact, self.dgu, y=self.act2)
        torch.matmul(self.dr2.t(), self.act2.float(), out=self.dWd)
        torch.matmul(self.dgu.t(), self.y1.float(), out=self.dWgu)
        self.dy1 = self.dgu @ self.Wgu.float()
        B.biv_rmsnorm_backward_fp8(self.k1, self.s1, self.i1, self.w1, self.dy1, self.dr1, self.dw1, self.nws,
                                   dres=self.dr2)
        self.opt.step()

    def wanted(self, Wh, Wd, Wgu, w1, w2):
        """The gradients in 64 bits, from what the forward left."""
        on = self.target != -100
        w = self.weight.to(F64) * on
        c = w / w.sum()
        y2 = self.y2.to(F64)
        p = torch.exp(y2 @ Wh.t() - self.lse.to(F64)[:, None])
        dz = p * (c + 2e-2 * c * self.lse.to(F64))[:, None]
        rows = torch.nonzero(on)[:, 0]
        dz[rows, self.target[rows].long()] -= c[rows]
        dy2, out = dz @ Wh, {"dWh": dz.t() @ y2}

        def norm_back(k, s, inv, gain, dy):
            x, inv, g = values(k, s), inv.to(F64)[:, None], dy * gain
            return inv * g - x * (inv ** 3 * (g * x).mean(1, keepdim=True)), (dy * x * inv).sum(0)
        dr2, out["dw2"] = norm_back(self.k2, self.s2, self.i2, w2, dy2)
        n = self.sg.shape[1] // 2
        gate, up = values(self.kg[:, :WIDE].contiguous(), self.sg[:, :n]), values(self.kg[:, WIDE:].contiguous(), self.sg[:, n:])
        s, dact = torch.sigmoid(gate), dr2 @ Wd
        dgu = torch.cat([dact * up * s * (1 + gate * (1 - s)), dact * gate * s], 1)
        out["dWd"] = dr2.t() @ self.act2.to(F64)
        out["dWgu"] = dgu.t() @ self.y1.to(F64)
        dr1, out["dw1"] = norm_back(self.k1, self.s1, self.i1, w1, dgu @ Wgu)
        return {**out, "dy2": dy2, "dr2": dr2, "dgu": dgu, "dr1": dr1 + dr2}


@pytest.fixture(autouse=True)
def full_precision():
    """The products that the test itself takes from torch are FP32."""
    old = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    yield
    torch.backends.cuda.matmul.allow_tf32 = old


def test_the_run_against_64_bits(B):
    s = Tail(B)
    before = [p.clone() for p in s.params]
    s.run()
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    want = s.wanted(*[p.to(F64) for p in before])
    for name, ref in want.items():
        off = float((getattr(s, name).to(F64) - ref).norm() / ref.norm())
        assert off <= 2.0 ** -11, (name, off)
    assert bool((s.dy2[:77] == 0).all())
    # what was kept stands for what was there: at most half a step of e4m3 off, or of its smallest step
    for k, sc, x in ((s.k1, s.s1, s.r1), (s.k2, s.s2, s.r2)):
        step = sc.to(F64).repeat_interleave(128, 1)[:, :D]
        x = x.to(F64)
        assert bool(((values(k, sc) - x).abs() <= torch.maximum(x.abs() * 2.0 ** -4, step * 2.0 ** -10) * 1.0001).all())
    total = torch.stack([getattr(s, n).to(F64).square().sum() for n in ("dWh", "dWd", "dWgu", "dw1", "dw2")]).sum().sqrt()
    assert abs(float(s.opt.norm[0]) - float(total)) <= 2.0 ** -20 * float(total)
    assert all(not same(p, b) for p, b in zip(s.params, before))


def test_captured_runs_equal_eager_ones(B):
    ends = []
    for captured in (False, True):
        s = Tail(B, seed=4)
        if captured:
            keep = [p.clone() for p in s.params]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                s.run()                              # warm-up, taken back below
            torch.cuda.current_stream().wait_stream(side)
            for p, k in zip(s.params, keep):
                p.copy_(k)
            for t in s.opt.exp_avg + s.opt.exp_avg_sq:
                t.zero_()
            s.opt.steps.zero_()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                s.run()
            for _ in range(3):
                g.replay()
        else:
            for _ in range(3):
                s.run()
        torch.cuda.synchronize()
        assert B.biv_poll_error() == 0
        ends.append([t.clone() for t in s.params + [s.lp, s.stats, s.dWh, s.dy2, s.dr1, s.dw1]])
    assert all(same(a, b) for a, b in zip(*ends))


def test_workspaces_are_far_below_the_logits(B):
    t, v = 8192, 131072
    logits = 4 * t * v
    assert B.biv_lm_head_loss_workspace(t, v) < logits // 32
    assert B.biv_lm_head_backward_workspace(t, v, 2048) < logits // 6
    assert B.biv_lm_head_backward_workspace(t, v, 2048, torch.float32, torch.float32) < logits // 4

"""One group-relative step on the tiny decoder from end to end: rollout logprobs,
trainer recompute, policy loss, the LM head's and final norm's gradients through
the library's own GEMM and backward kernels, clipped AdamW in place, and the
next rollout from graphs that were captured before the update."""
import math

import numpy as np
import pytest
import torch

import synth
from oracle import trainer as tr
from oracle.codecs import bf16_to_f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from invariant_forward_bitwise_gb300 import biv, build
    build.build()
    biv.load()
    return biv


def f64(t):
    t = t.detach().cpu().contiguous()
    if t.dtype == torch.bfloat16:
        return bf16_to_f32(t.view(torch.int16).numpy().view(np.uint16)).astype(np.float64)
    return t.numpy().astype(np.float64)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


class Step:
    """A recompute of the sequences and the buffers of the step behind it."""

    def __init__(self, B, state="e4m3"):
        from invariant_forward_bitwise_gb300.model import DecodeGraphs, DenseModel, PagedKV, Runner, prefill_rows
        from invariant_forward_bitwise_gb300.optim import AdamW
        self.B, cfg = B, synth.TINY
        W = synth.dense_weights(cfg, seed=0, random_gains=True, lm_scale=10.0)
        self.cfg, self.m = cfg, DenseModel(cfg, W, max_rows=1024, max_pos=512)
        self.kv = PagedKV(cfg, pages=256, max_seqs=32, max_pages=8)
        self.seqs = synth.tiny_sequences(cfg, n=8, seed=1)
        self.graphs = DecodeGraphs(self.m, self.kv, use_graphs=True)
        # the recompute's rows, as one step
        for i, s in enumerate(self.seqs):
            self.kv.admit(i, s.length)
        self.kv.sync_table()
        lens = [s.length - s.prompt_len for s in self.seqs]
        rows = prefill_rows(self.seqs, list(range(8)), [0] * 8, [s.length - 1 for s in self.seqs],
                            [s.prompt_len - 1 for s in self.seqs])
        spec = Runner(self.m).load_rows(self.kv, *rows[:5])
        self.m.reserve(self.kv, [spec])
        self.m.step(self.kv, spec)
        torch.cuda.synchronize()
        for i in range(8):
            self.kv.release(i)
        self.n = n = sum(lens)
        assert spec.T_lm == n
        self.lp = self.m.lp[:n].clone()
        self.target = self.m.targets[:n].clone()
        N = (n + 7) // 8 * 8                         # the gradient GEMMs' K: whole 16-byte rows
        self.y = torch.zeros(N, cfg.hidden, dtype=torch.bfloat16, device="cuda")
        self.y[:n] = self.m.ylm[:n]
        self.x = self.m.r[self.m.lm_rows[:n].long()].clone()
        self.start = torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), device="cuda")
        g = synth.rng(11)
        self.adv = torch.from_numpy(g.standard_normal(8).astype(np.float32)).cuda()
        f, V, d = dict(device="cuda"), cfg.vocab, cfg.hidden
        self.logits, self.dz = torch.empty(n, V, **f), torch.zeros(N, V, dtype=torch.bfloat16, device="cuda")
        self.lp2, self.ent, self.stats = torch.empty(n, **f), torch.empty(n, **f), torch.empty(8, **f)
        self.ws = torch.empty(B.biv_policy_loss_workspace(n, 8), dtype=torch.uint8, device="cuda")
        self.dW, self.dh = torch.empty(V, d, **f), torch.empty(N, d, **f)
        self.dx, self.dnorm = torch.empty(n, d, **f), torch.empty(d, **f)
        self.gws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        self.params = [self.m.W["lm_head"], self.m.W["final_norm"]]
        self.opt = AdamW(self.params, [self.dW, self.dnorm], lr=1e-3, weight_decay=[0.1, 0.0], max_norm=0.5,
                         bits=8 if state == "e4m3" else 32, rounding="stochastic", seed=5)

    def run(self, old_lp):
        B = self.B
        W, norm = self.params
        B.biv_gemm(B.gemm_desc(self.y[:self.n], W, self.logits), self.gws)
        d = B.policy_desc(self.start, self.adv, self.stats, self.ws, T=self.n, old_lp=old_lp, ent_coef=0.01,
                          reduce=B.LOSS_SEQ_MEAN)
        B.biv_policy_loss_logits(d, self.logits, self.target, self.lp2, self.ent, self.dz[:self.n])
        B.biv_gemm(B.gemm_desc(self.dz.t().contiguous(), self.y.t().contiguous(), self.dW), self.gws)
        B.biv_gemm(B.gemm_desc(self.dz, W.t().contiguous(), self.dh), self.gws)
        B.biv_rmsnorm_backward(self.x, norm, self.dh[:self.n], self.dx, self.dnorm, self.cfg.eps, ws=self.gws)
        self.opt.step()

    def rollout(self):
        from invariant_forward_bitwise_gb300.model import rollout
        return rollout(self.m, self.kv, self.seqs, max_tokens=512, graphs=self.graphs)


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_group_relative_step(B, state):
    from invariant_forward_bitwise_gb300.model import recompute, rollout
    s = Step(B, state)
    rolled = np.concatenate(s.rollout())
    assert np.array_equal(rolled.view(np.uint32), s.lp.cpu().numpy().view(np.uint32))
    # the loss on the recomputed logprobs: the sampling policy is the same to the
    # bit, so the ratio is 1, nothing is clipped and the KL statistics are 0
    old = torch.from_numpy(rolled).cuda()
    dlp, stats = torch.empty(s.n, device="cuda"), torch.empty(8, device="cuda")
    d = B.policy_desc(s.start, s.adv, stats, s.ws, T=s.n, old_lp=old, reduce=B.LOSS_SEQ_MEAN)
    B.biv_policy_loss(d, s.lp, dlp)
    torch.cuda.synchronize()
    assert stats[4:7].tolist() == [0.0, 0.0, 0.0] and int(stats[7]) == s.n
    w, seq = tr.row_weights(s.n, s.start.tolist(), None, "seq", 1.0)
    assert np.allclose(f64(dlp), -w * f64(s.adv)[seq], rtol=2.0 ** -22)
    # the step: gradients against the oracle's, from the same logits
    before = [p.clone() for p in s.params]
    s.run(old)
    torch.cuda.synchronize()
    assert B.biv_poll_error() == 0
    zz, tgt = f64(s.logits), s.target.cpu().numpy()
    lp, H, _, _ = tr.token_logprobs(zz, tgt)
    # (the fused LM head and the logits' route agree to rounding)
    assert np.max(np.abs(lp - f64(s.lp))) < 1e-3
    _, want = tr.policy_loss(lp, w, f64(s.adv)[seq], f64(old), None, gamma=0.01, H=H)
    dz = tr.policy_dz(zz, tgt, want, w, 0.01)
    y = f64(s.y[:s.n])
    # dz is rounded to bf16 once (2^-8 of each term); the GEMM sums in FP32
    assert np.all(np.abs(f64(s.dW) - dz.T @ y) <= (2.0 ** -8 + 1e-4) * (np.abs(dz).T @ np.abs(y)) + 1e-12)
    W0 = f64(before[0])
    dh = dz @ W0
    assert np.all(np.abs(f64(s.dh[:s.n]) - dh) <= (2.0 ** -8 + 1e-4) * (np.abs(dz) @ np.abs(W0)) + 1e-12)
    total = math.sqrt(np.sum(f64(s.dW) ** 2) + np.sum(f64(s.dnorm) ** 2))
    assert abs(float(s.opt.norm[0]) - total) <= 2.0 ** -21 * total
    # the weights moved where the gradient points, and graphs captured before the
    # update now give what the new weights give eagerly
    for p, b, g in zip(s.params, before, (s.dW, s.dnorm)):
        big = g.abs() > 0.1 * g.abs().max()
        moved = (p.float() - b.float())[big]
        assert float((moved * g[big]).sum()) < 0 and not same(p, b)
    after = np.concatenate(s.rollout())
    eager = np.concatenate(rollout(s.m, s.kv, s.seqs, max_tokens=512, use_graphs=False))
    again = np.concatenate(recompute(s.m, s.kv, s.seqs, max_tokens=512))
    assert np.array_equal(after.view(np.uint32), eager.view(np.uint32))
    assert np.array_equal(after.view(np.uint32), again.view(np.uint32)) and not np.array_equal(after, rolled)


def test_captured_step_equals_eager(B):
    """The whole step in one graph, replayed twice: the bits of two eager steps."""
    ends = []
    for captured in (False, True):
        s = Step(B)
        old = s.lp.clone()
        if captured:
            keep = [p.clone() for p in s.params]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                s.run(old)                           # warm-up, taken back below
            torch.cuda.current_stream().wait_stream(side)
            for p, k in zip(s.params, keep):
                p.copy_(k)
            for t in s.opt.exp_avg + s.opt.exp_avg_sq + s.opt.exp_avg_scale + s.opt.exp_avg_sq_scale:
                t.zero_()
            s.opt.steps.zero_()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                s.run(old)
            for _ in range(2):
                g.replay()
        else:
            for _ in range(2):
                s.run(old)
        torch.cuda.synchronize()
        ends.append([t.clone() for t in s.params + s.opt.exp_avg + s.opt.exp_avg_sq + [s.opt.steps, s.stats]])
    assert all(same(a, b) for a, b in zip(*ends)) and ends[0][-2].tolist() == [2, 0]


def weights_and_step(bits, M, seed=3):
    """An optimizer over 50 M weights whose last two tensors a GEMM and an LM head read."""
    from invariant_forward_bitwise_gb300.optim import AdamW
    gen = torch.Generator(device="cuda").manual_seed(seed)
    N, K = 4096, 2048
    shapes = [(N, K)] * 6
    p = [(torch.randn(s, device="cuda", generator=gen) * 0.02).bfloat16() for s in shapes]
    g = [torch.randn(s, device="cuda", generator=gen).bfloat16() for s in shapes]
    opt = AdamW(p, g, lr=0.01, bits=bits, rounding="stochastic", seed=1)
    h = torch.randn(M, K, device="cuda", generator=gen).bfloat16()
    target = torch.randint(0, N, (M,), device="cuda", generator=gen, dtype=torch.int32)
    return opt, p, h, target


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("M", [16, 300])
@pytest.mark.parametrize("between", ["nothing", "gemm", "row op"])
def test_the_call_after_a_step_reads_the_new_weights(B, bits, M, between):
    """A GEMM, or the fused LM head, right behind the step in its stream or graph
    gives the bits of the same calls with a synchronisation after each; with a GEMM
    of other weights between too, and with b_early behind a row op."""
    outs = []
    for how in ("waiting", "eager", "graph"):
        opt, p, h, target = weights_and_step(bits, M)
        N = p[0].shape[0]
        c = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        c0, lp, act = torch.empty_like(c), torch.empty(M, device="cuda"), torch.empty_like(h[:, :1024])
        ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        lws = torch.empty(B.biv_lm_head_logprob_workspace(M, N), dtype=torch.uint8, device="cuda")

        def calls(sync):
            for second in (lambda: B.biv_gemm(B.gemm_desc(h, p[5], c, b_early=between == "row op"), ws),
                           lambda: B.biv_lm_head_logprob(h, p[5], target, lp, lws)):
                opt.step()
                sync()
                if between == "gemm":
                    B.biv_gemm(B.gemm_desc(h, p[4], c0), ws)
                if between == "row op":
                    B.biv_silu_mul(h, act)
                sync()
                second()
                sync()
        seen = []
        graph = None
        if how == "graph":
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                calls(lambda: None)
        for _ in range(4):
            if graph:
                graph.replay()
            else:
                calls(torch.cuda.synchronize if how == "waiting" else lambda: None)
            seen += [c.clone(), lp.clone()]
        torch.cuda.synchronize()
        assert B.biv_poll_error() == 0 and opt.steps.tolist() == [8, 0]
        outs.append(seen + [x.clone() for x in p])
    for other in outs[1:]:
        assert all(same(a, b) for a, b in zip(outs[0], other))
    assert not same(outs[0][0], outs[0][2]) and not same(outs[0][1], outs[0][3])


@pytest.mark.parametrize("M", [16, 300])
def test_a_gemm_may_read_the_output_of_the_call_before_as_b(B, M):
    """B straight from a GEMM (folded in the CTA, or from partials) or a row op."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    rnd = lambda *s: (torch.randn(*s, device="cuda", generator=gen) * 0.1).bfloat16()  # noqa: E731
    h, ws = rnd(M, 1024), torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    outs = []
    ins = [(rnd(2048, 2048), rnd(1024, 2048), rnd(2048, 2048)) for _ in range(6)]
    for sync in (torch.cuda.synchronize, lambda: None):
        w, w2 = torch.zeros(2048, 1024, dtype=torch.bfloat16, device="cuda"), rnd(2048, 1024)
        for a, b, gu in ins:
            c = torch.empty(M, 2048, dtype=torch.bfloat16, device="cuda")
            c2 = torch.empty_like(c)
            B.biv_gemm(B.gemm_desc(a, b, w), ws)
            sync()
            B.biv_gemm(B.gemm_desc(h, w, c), ws)
            sync()
            B.biv_silu_mul(gu, w2)
            sync()
            B.biv_gemm(B.gemm_desc(h, w2, c2), ws)
            sync()
            outs += [c, c2]
    torch.cuda.synchronize()
    n = len(outs) // 2
    assert all(same(x, y) for x, y in zip(outs[:n], outs[n:]))

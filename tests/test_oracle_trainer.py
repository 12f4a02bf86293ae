"""Pins for the oracle's trainer end, and the library's argument checks (CPU
only; nothing is launched): the policy loss's gradient against central finite
differences and torch autograd, AdamW against torch's own optimizer in float64,
the roundings against their definition."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from oracle import codecs
from oracle import trainer as tr

F64 = np.float64


def _case(seed, T=12, V=17):
    g = np.random.default_rng(seed)
    z = g.standard_normal((T, V)) * 2
    target = g.integers(0, V, T)
    start = [0, 4, 4, 9, 11]                       # an empty sequence; one row behind the last
    mask = (g.random(T) < 0.8).astype(np.uint8)
    mask[4:9] = 0                                  # a sequence of which nothing counts
    lp = tr.token_logprobs(z, target)[0]
    old = lp - g.choice([-0.5, -0.1, 0.0, 0.1, 0.5], T)
    ref = lp + g.standard_normal(T) * 0.3
    return z, target, start, mask, old, ref, g.standard_normal(T)


@pytest.mark.parametrize("reduce", ["token", "seq", "sum"])
@pytest.mark.parametrize("dual,beta,gamma,it", [(0.0, 0.0, 0.0, 1.0), (1.5, 0.1, 0.05, 0.7)])
def test_policy_loss_gradient(reduce, dual, beta, gamma, it):
    z, target, start, mask, old, ref, adv = _case(1)
    w, seq = tr.row_weights(len(z), start, mask, reduce, 5.0)
    assert w[4:9].max() == 0 and w[11] == 0
    assert reduce == "sum" or math.isclose(w.sum(), 1.0)

    def loss(zz):
        lp, H, _, _ = tr.token_logprobs(zz, target, it)
        return tr.policy_loss(lp, w, adv, old, ref, 0.2, 0.3, dual, beta, gamma, H)[0][0]
    lp, H, _, _ = tr.token_logprobs(z, target, it)
    stats, dlp = tr.policy_loss(lp, w, adv, old, ref, 0.2, 0.3, dual, beta, gamma, H)
    dz = tr.policy_dz(z, target, dlp, w, gamma, it)
    eps, fd = 1e-6, np.zeros_like(z)
    for i in np.ndindex(z.shape):
        a, b = z.copy(), z.copy()
        a[i] += eps
        b[i] -= eps
        fd[i] = (loss(a) - loss(b)) / (2 * eps)
    assert np.max(np.abs(fd - dz)) < 1e-8          # eps^2 f''' + rounding 1e-16 / eps
    # autograd of the same loss written with library operations
    zt = torch.tensor(z, requires_grad=True)
    logp = torch.log_softmax(zt * it, 1)
    lpt = logp[torch.arange(len(z)), torch.tensor(target)]
    r = torch.exp(lpt - torch.tensor(old))
    A, wt = torch.tensor(adv), torch.tensor(w)
    pg = -torch.minimum(r * A, r.clamp(0.8, 1.3) * A)
    if dual:
        pg = torch.where(A < 0, torch.minimum(pg, -A * dual), pg)
    e = torch.tensor(ref) - lpt
    total = (wt * (pg + beta * (torch.exp(e) - e - 1) + gamma * (logp.exp() * logp).sum(1))).sum()
    total.backward()
    assert abs(total.item() - stats[0]) < 1e-12
    assert np.max(np.abs(zt.grad.numpy() - dz)) < 1e-12


def test_policy_loss_of_nothing_is_zero():
    w, _ = tr.row_weights(3, [0, 3], [0, 0, 0], "token", 1.0)
    stats, dlp = tr.policy_loss([np.nan] * 3, w, [np.nan] * 3)
    assert not stats.any() and not dlp.any()


def test_adamw_against_torch():
    g = np.random.default_rng(2)
    w0 = g.standard_normal(50)
    p = torch.nn.Parameter(torch.tensor(w0))
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    w, m, v = w0, np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        gr = g.standard_normal(50)
        p.grad = torch.tensor(gr)
        opt.step()
        w, m, v = tr.adamw(w, gr, m, v, t, 1e-2, 0.1, 0.9, 0.99, 1e-8)
    assert np.allclose(w, p.detach().numpy(), atol=1e-13)


def test_stochastic_rounding_by_its_definition():
    y = np.array([0.0, 1.0, 1.03, -1.03, 447.9, 0.001, 2.0 ** -9])
    lo = tr.stochastic(y, np.zeros(7, np.uint64), 4, -6)
    hi = tr.stochastic(y, np.full(7, 65535, np.uint64), 4, -6)
    assert lo.tolist() == [0.0, 1.0, 1.0, -1.0, 416.0, 0.0, 2.0 ** -9]
    assert hi.tolist() == [0.0, 1.0, 1.125, -1.125, 448.0, 2.0 ** -9, 2.0 ** -9]
    # every result is an e4m3 value, and the mean over all 65536 draws is y
    bits = np.arange(65536, dtype=np.uint64)
    q = tr.stochastic(np.full(65536, 1.03), bits, 4, -6)
    assert abs(q.mean() - 1.03) <= 0.125 / 65536
    assert np.array_equal(tr.e4m3_nearest(q), q)
    for x in tr.random_bits(0, 1 << 16, 7, 3):
        assert abs(x.mean() / 65535 - 0.5) < 5 / math.sqrt(12 * len(x))


def test_codecs_agree_on_the_grid():
    """grid_step and the codec describe the same e4m3 grid."""
    vals = codecs.e4m3_to_f32(np.arange(0x7F, dtype=np.uint8)).astype(F64)
    assert np.allclose(np.diff(vals), tr.grid_step(vals[:-1], 4, -6))


# ------------------------------------------------------------- refusals ----
@pytest.fixture(scope="module")
def B():
    from invariant_forward_bitwise_gb300 import biv, build
    build.build()
    biv.load()
    return biv


def _policy(B, **kw):
    d = B.PolicyDesc()
    d.T, d.nseq = 8, 2
    for f in ("seq_start", "adv", "stats", "workspace", "old_lp", "ref_lp"):
        setattr(d, f, 0x10000)                    # never dereferenced: no launch here
    d.clip_lo, d.clip_hi, d.norm = 0.2, 0.2, 1.0
    d.workspace_bytes = B.biv_policy_loss_workspace(8, 2)
    for k, x in kw.items():
        setattr(d, k, x)
    return d


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), b"sizes"), (dict(nseq=-1), b"sizes"), (dict(seq_start=None), b"null"),
    (dict(adv=None), b"null"), (dict(stats=None), b"null"), (dict(clip_lo=1.5), b"clip"),
    (dict(clip_hi=-0.1), b"clip"), (dict(clip_lo=float("nan")), b"clip"), (dict(dual_clip=0.5), b"dual"),
    (dict(kl_coef=0.1, ref_lp=None), b"ref_lp"), (dict(kl_coef=float("nan")), b"kl_coef"),
    (dict(ent_coef=2000.0), b"ent_coef"),
    (dict(reduce=3), b"reduce"), (dict(reduce=2, norm=0.0), b"norm"),
    (dict(reduce=2, norm=float("inf")), b"norm"), (dict(workspace=0x10008), b"aligned")])
def test_policy_loss_refuses(B, kw, word):
    lib = B.load()
    st = lib.biv_policy_loss(C.byref(_policy(B, **kw)), C.c_void_p(0x20000), C.c_void_p(0x30000), None)
    assert st == B.BIV_ERR_INVALID and word in lib.biv_last_error()


def test_policy_loss_refuses_small_workspace_and_entropy(B):
    lib = B.load()
    d = _policy(B)
    d.workspace_bytes -= 1
    lp = C.c_void_p(0x20000)
    assert lib.biv_policy_loss(C.byref(d), lp, None, None) == B.BIV_ERR_WORKSPACE
    assert lib.biv_policy_loss(C.byref(_policy(B, workspace=None)), lp, None, None) == B.BIV_ERR_WORKSPACE
    assert lib.biv_policy_loss(C.byref(_policy(B, ent_coef=0.1)), lp, None, None) == B.BIV_ERR_INVALID
    assert lib.biv_policy_loss(C.byref(_policy(B)), None, None, None) == B.BIV_ERR_INVALID
    assert lib.biv_policy_loss(None, None, None, None) == B.BIV_ERR_INVALID
    assert lib.biv_policy_loss(C.byref(_policy(B, T=0, stats=None)), None, None, None) == B.BIV_ERR_INVALID


@pytest.mark.parametrize("kw", [
    dict(z=None), dict(target=None), dict(lp=None), dict(ent=None), dict(V=0), dict(V=262145, ld=262145, ldz=262145),
    dict(ld=99), dict(ldz=99), dict(zt=2), dict(dzt=2), dict(it=0.0), dict(it=-1.0), dict(it=float("nan")),
    dict(it=float("inf")), dict(z=0x100001), dict(dz=0x900002), dict(dz=0x100010), dict(dz=0x100000, dzt=0, ldz=104),
    dict(dz=0x100000 - 16)])
def test_policy_loss_logits_refuses(B, kw):
    lib = B.load()
    a = dict(z=0x100000, ld=100, zt=1, target=0x20000, V=100, it=1.0, lp=0x30000, ent=0x40000, dz=0x900000,
             ldz=100, dzt=1) | kw
    st = lib.biv_policy_loss_logits(C.byref(_policy(B)), a["z"], a["ld"], a["zt"], a["target"], a["V"], a["it"],
                                    a["lp"], a["ent"], a["dz"], a["ldz"], a["dzt"], None)
    assert st == B.BIV_ERR_INVALID, lib.biv_last_error()


def _tensors(B, n, **kw):
    arr = (B.OptTensor * n)()
    for i, a in enumerate(arr):
        base = (i + 1) << 24
        a.param, a.grad, a.m, a.v = base, base + (1 << 20), base + (2 << 20), base + (3 << 20)
        a.numel, a.lr_scale = 1000, 1.0
        a.param_dtype, a.grad_dtype, a.state_dtype = B.F32, B.F32, B.F32
        for k, x in kw.items():
            setattr(a, k, x)
    return arr


def _plan(B, arr):
    n, k = C.c_int64(-1), C.c_int(-1)
    return B.load().biv_opt_plan(arr, len(arr), C.byref(n), C.byref(k)), n.value


def test_opt_plan_lays_out_chunks(B):
    arr = _tensors(B, 4)
    arr[1].numel, arr[2].numel, arr[3].numel = 0, 5000, 2048
    arr[3].grad += 4
    st, chunks = _plan(B, arr)
    assert st == B.BIV_OK and chunks == 1 + 0 + 3 + 1
    assert [a.first_chunk for a in arr] == [0, 1, 1, 4]
    assert [a.rng_base for a in arr] == [0, 1024, 1024, 1024 + 5120]
    assert [a.vec for a in arr] == [3, 0, 3, 0]
    arr[0].grad += 16
    assert _plan(B, arr)[0] == B.BIV_OK and arr[0].vec == 1
    assert _plan(B, (B.OptTensor * 0)()) == (B.BIV_OK, 0)


@pytest.mark.parametrize("kw", [
    dict(numel=-1), dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(param_dtype=2),
    dict(grad_dtype=2), dict(state_dtype=5), dict(state_dtype=0), dict(state_dtype=2), dict(param=0x1000002),
    dict(grad=0x1100001), dict(master=0x2000000), dict(param_dtype=0, master=0x2000002)])
def test_opt_plan_refuses(B, kw):
    assert _plan(B, _tensors(B, 1, **kw))[0] == B.BIV_ERR_INVALID


def test_opt_plan_refuses_shared_memory(B):
    for f in ("param", "m", "v"):
        arr = _tensors(B, 3)
        setattr(arr[2], f, getattr(arr[0], f) + 3996)            # the last element of tensor 0's array
        assert _plan(B, arr)[0] == B.BIV_ERR_INVALID and b"same memory" in B.load().biv_last_error()
    arr = _tensors(B, 3)
    arr[1].grad = arr[2].m + 400
    assert _plan(B, arr)[0] == B.BIV_ERR_INVALID and b"gradient" in B.load().biv_last_error()
    arr = _tensors(B, 3)
    arr[1].grad = arr[2].grad                                   # one gradient for two tensors: only read
    assert _plan(B, arr)[0] == B.BIV_OK
    arr[1].param = arr[0].param + 4000                          # side by side
    assert _plan(B, arr)[0] == B.BIV_OK


@pytest.mark.parametrize("kw", [dict(beta1=1.0), dict(beta2=-0.1), dict(beta1=float("nan")), dict(eps=0.0), dict(eps=1e-40),
                                dict(rounding=2), dict(lr=None), dict(step=None), dict(tensors=None),
                                dict(n=-1), dict(chunks=-1), dict(n=0), dict(kinds=0), dict(kinds=1 << 12)])
def test_adamw_refuses(B, kw):
    d = B.AdamWDesc()
    d.tensors, d.n, d.chunks, d.kinds, d.lr, d.step = 0x1000, 1, 1, 1, 0x2000, 0x3000
    d.beta1, d.beta2, d.eps = 0.9, 0.999, 1e-8
    for k, x in kw.items():
        setattr(d, k, x)
    assert B.load().biv_adamw(C.byref(d), None) == B.BIV_ERR_INVALID


def test_grad_norm_refuses(B):
    lib = B.load()
    ws, need = C.c_void_p(0x10000), B.biv_grad_norm_workspace(9)
    t, out = C.c_void_p(0x1000), C.c_void_p(0x2000)
    for args, st in (((t, 1, 9, -1.0, out, ws, need), B.BIV_ERR_INVALID),
                     ((t, 1, 9, float("nan"), out, ws, need), B.BIV_ERR_INVALID),
                     ((t, 1, 9, 1.0, None, ws, need), B.BIV_ERR_INVALID),
                     ((None, 1, 9, 1.0, out, ws, need), B.BIV_ERR_INVALID),
                     ((t, 1, 9, 1.0, out, ws, need - 1), B.BIV_ERR_WORKSPACE),
                     ((t, 1, 9, 1.0, out, None, need), B.BIV_ERR_WORKSPACE)):
        assert lib.biv_grad_norm(*args, None) == st

"""The multi-tensor AdamW step and the gradient norm against the float64
oracle: every type combination, odd sizes, unaligned tensors, 8-bit states,
both roundings, the clip, steps that are skipped, captured steps, and the same
bits for a tensor whatever is updated beside it.

Tolerances.  The FP32 update rounds each of its operations once (2^-24): m
takes 4, v 6, the moved distance about 16 with the bias corrections; a clip
coefficient adds the norm's error (2^-22) and two roundings: 2^-18 is ample.  A nearest rounding is off by half a step (bf16 2^-8,
e4m3 2^-4, or 2^-10 below 2^-6), a stochastic one by less than a step."""
import numpy as np
import pytest
import torch

import synth
from oracle import trainer as tr
from oracle.codecs import bf16_to_f32, e4m3_to_f32

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def O():
    from invariant_forward_bitwise_gb300 import build, optim
    build.build()
    return optim


@pytest.fixture(scope="module")
def B(O):
    from invariant_forward_bitwise_gb300 import biv
    biv.load()
    return biv


def f64(t):
    t = t.detach().cpu().reshape(-1)
    if t.dtype == torch.bfloat16:
        return bf16_to_f32(t.view(torch.int16).numpy().view(np.uint16)).astype(np.float64)
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return e4m3_to_f32(t.view(torch.uint8).numpy()).astype(np.float64)
    return t.numpy().astype(np.float64)


def bits(t):
    return t.detach().contiguous().view(-1).view(torch.uint8).cpu().numpy()


def same(a, b):
    return np.array_equal(bits(a), bits(b))


def f32(x):
    return float(np.float32(x))


def tensors(g, sizes, param, grad, state, shift=0):
    """Lists of params, grads, masters, states and scales; `shift` elements off
    the start of their storage."""
    typ = {"f32": torch.float32, "bf16": torch.bfloat16, "master": torch.bfloat16}
    e8 = state == "e4m3"
    out = dict(params=[], grads=[], master=[] if param == "master" else None, exp_avg=[], exp_avg_sq=[],
               exp_avg_scale=[] if e8 else None, exp_avg_sq_scale=[] if e8 else None)

    def put(x, dt):
        t = torch.zeros(len(x) + shift, dtype=dt, device="cuda")
        t[shift:] = torch.from_numpy(x.astype(np.uint8 if dt == torch.uint8 else np.float32)).to(dt).cuda()
        return t[shift:]
    for n in sizes:
        w = g.standard_normal(n) * 0.05
        size = np.exp(g.standard_normal(n) * 2)
        out["params"].append(put(w, typ[param]))
        if param == "master":
            out["master"].append(put(w, torch.float32))
        out["grads"].append(put(g.standard_normal(n) * 1e-2 * size, typ[grad]))
        if not e8:
            out["exp_avg"].append(put(g.standard_normal(n) * 1e-2 * size, torch.float32))
            out["exp_avg_sq"].append(put((g.standard_normal(n) * 1e-2 * size) ** 2, torch.float32))
        else:
            nb = (n + 127) // 128
            out["exp_avg"].append(put(g.integers(0, 0x7F, n) | (g.integers(0, 2, n) << 7), torch.uint8))
            out["exp_avg_sq"].append(put(g.integers(1, 0x7F, n), torch.uint8))
            out["exp_avg_scale"].append(put(np.abs(g.standard_normal(nb)) * 1e-5, torch.float32))
            out["exp_avg_sq_scale"].append(put(np.abs(g.standard_normal(nb)) * 1e-5 + 1e-7, torch.float32))
    return out


def lists(ts, f):
    return {k: None if v is None else f(v) for k, v in ts.items()}


def snapshot(ts):
    return lists(ts, lambda v: [t.clone() for t in v])


def rng_bases(sizes):
    base, out = 0, []
    for n in sizes:
        out.append(base)
        base += (n + 127) // 128 * 128
    return out


def check(was, now, sizes, t, lr, wd, param, state, rounding="nearest", seed=0, coef=1.0, slack=0.0):
    """One step from `was` to `now`; slack: relative error of coef."""
    sr, b2 = rounding == "stochastic", 0.999
    for i, (n, base) in enumerate(zip(sizes, rng_bases(sizes))):
        if n == 0:
            continue
        w = f64(was["master"][i] if param == "master" else was["params"][i])
        g, m, v = f64(was["grads"][i]), f64(was["exp_avg"][i]), f64(was["exp_avg_sq"][i])
        if state == "e4m3":
            m = m * np.repeat(f64(was["exp_avg_scale"][i]), 128)[:n]
            v = (v * np.repeat(f64(was["exp_avg_sq_scale"][i]), 128)[:n]) ** 2
        w2, m2, v2 = tr.adamw(w, g, m, v, t, lr, wd[i], b2=b2, coef=coef)
        mb = 0.9 * np.abs(m) + 0.1 * np.abs(g * coef)
        me, ve = (4 * U + slack) * mb, (6 * U + 2 * slack) * v2
        moved = lr * (mb / (1 - 0.9 ** t)) / (np.sqrt(v2 / (1 - b2 ** t)) + 1e-8)
        we = (16 * U + 3 * slack) * moved + 3 * U * (np.abs(w) + moved)
        hm, hv, hw = tr.random_bits(base, n, seed, t)
        gw = f64(now["params"][i])
        if param == "f32":
            assert np.all(np.abs(gw - w2) <= we)
        elif param == "master":
            assert np.all(np.abs(f64(now["master"][i]) - w2) <= we)
            assert same(now["params"][i], now["master"][i].bfloat16())
        elif sr:
            assert np.all(np.abs(gw - w2) <= tr.grid_step(w2, 8, -126) + we)
            assert np.mean(gw != tr.stochastic(w2, hw, 8, -126)) <= 2e-3 + 1.0 / n
        else:
            assert np.all(np.abs(gw - w2) <= 2.0 ** -8 * np.abs(w2) + we)
        if state == "f32":
            assert np.all(np.abs(f64(now["exp_avg"][i]) - m2) <= me)
            assert np.all(np.abs(f64(now["exp_avg_sq"][i]) - v2) <= ve)
            continue
        r2 = np.sqrt(v2)
        for k, x, err, h in (("exp_avg", m2, me, hm), ("exp_avg_sq", r2, (4 * U + slack) * r2, hv)):
            s = tr.block_scale(x)
            blk_err = np.repeat([np.max(err[j:j + 128]) for j in range(0, n, 128)], 128)[:n] / 448
            got_s = np.repeat(f64(now[k + "_scale"][i]), 128)[:n]
            assert np.all(np.abs(got_s - s) <= 2 * U * s + blk_err)
            y, got = x / s, f64(now[k][i])
            step = tr.grid_step(y, 4, -6)
            tol = 6 * U * np.abs(y) + (err + np.abs(y) * blk_err) / s
            if sr:
                assert np.all(np.abs(got - y) <= step + tol)
                q = tr.stochastic(y, h, 4, -6)
            else:
                # a positive root below half the smallest code takes that code
                floor = (k == "exp_avg_sq") & (x > 0) & (y < 2.0 ** -10)
                assert np.all(np.abs(got - y) <= np.where(floor, 2.0 ** -9, step / 2) + tol)
                q = tr.e4m3_nearest(y)
            if k == "exp_avg_sq":
                q = np.where((x > 0) & (q == 0), 2.0 ** -9, q)
                assert np.all((got > 0) == (x > 0))
            # values next to a border may go either way; all others are the oracle's
            assert np.mean(got != q) <= 2e-3 + 1.0 / n
            assert np.all(np.abs(got) <= 448)


SIZES = [1, 127, 128, 129, 2047, 2048, 2049, 0, 5000, 7]


@pytest.mark.parametrize("param", ["f32", "master", "bf16"])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("state", ["f32", "e4m3"])
@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
def test_adamw_types(O, param, grad, state, rounding):
    g = synth.rng(len(param) * 8 + len(grad) * 4 + len(state))
    ts = tensors(g, SIZES, param, grad, state)
    wd = [f32(0.1 * (i % 2)) for i in range(len(SIZES))]
    steps = torch.tensor([6, 0], dtype=torch.int32, device="cuda")
    seed = (5 << 32) + 77
    opt = O.AdamW(**ts, lr=3e-3, weight_decay=wd, rounding=rounding, seed=seed, step=steps)
    for t in (7, 8):
        was = snapshot(ts)
        opt.step()
        torch.cuda.synchronize()
        assert steps.tolist() == [t, 0]
        check(was, ts, SIZES, t, f32(3e-3), wd, param, state, rounding, seed)
        assert all(same(a, b) for a, b in zip(was["grads"], ts["grads"]))


@pytest.mark.parametrize("state", ["f32", "e4m3"])
@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
def test_states_are_the_bits_of_the_stated_operations(O, state, rounding):
    """m, v, their scales and codes in numpy float32 (IEEE, one rounding per
    operation), over three steps that feed on one another."""
    F = np.float32
    n = 5000
    ts = tensors(synth.rng(31), [n], "f32", "f32", state)
    b1, c1, b2, c2 = F(0.9), F(1 - 0.9), F(0.999), F(1 - 0.999)
    f = lambda t: f64(t).astype(F)  # noqa: E731
    g, m, v = f(ts["grads"][0]), f(ts["exp_avg"][0]), f(ts["exp_avg_sq"][0])
    if state == "e4m3":
        ms, vs = f(ts["exp_avg_scale"][0]), f(ts["exp_avg_sq_scale"][0])
    opt = O.AdamW(**ts, lr=1e-3, rounding=rounding, seed=77, weight_decay=0.1)
    w, lr = f(ts["params"][0]), F(1e-3)
    for t in (1, 2, 3):
        opt.step()
        torch.cuda.synchronize()
        if state == "e4m3":
            m, v = m * np.repeat(ms, 128)[:n], v * np.repeat(vs, 128)[:n]
            v = v * v
        m, v = b1 * m + c1 * g, b2 * v + (c2 * g) * g
        rate, rbc2 = lr / F(1 - 0.9 ** t), F(1 / np.sqrt(1 - 0.999 ** t))
        w = w * (F(1) - lr * F(0.1)) - (rate * m) / (np.sqrt(v) * rbc2 + F(1e-8))
        # (root and quotient may miss their rounding where the value all but ties)
        assert np.mean(f(ts["params"][0]) != w) <= 1e-3
        w = f(ts["params"][0])
        if state == "f32":
            assert np.array_equal(f(ts["exp_avg"][0]), m) and np.array_equal(f(ts["exp_avg_sq"][0]), v)
            continue
        hm, hv, _ = tr.random_bits(0, n, 77, t)
        held = []
        for x, h in ((m, hm), (np.sqrt(v), hv)):
            a = np.array([np.max(np.abs(x[j:j + 128])) for j in range(0, n, 128)], F)
            y = x * np.repeat(F(448) * (F(1) / a), 128)[:n]
            if rounding == "stochastic":     # the sum y 512 + bits / 65536 below 2^-6 is rounded once
                small = np.floor(np.abs(y) * F(512) + h.astype(F) / F(65536)) / F(512)
                big = (np.abs(y).view(np.uint32) + (h.astype(np.uint32) << 4) & 0xFFF00000).view(F)
                y = np.copysign(np.minimum(np.where(np.abs(y) < F(2.0 ** -6), small, big), F(448)), y)
            held += [tr.e4m3_nearest(y).astype(F), a * (F(1) / F(448))]
        m, ms, v, vs = held
        v = np.where((np.sqrt(f64(ts["exp_avg_sq"][0])) > 0) & (v == 0), F(2.0 ** -9), v)
        assert np.array_equal(f(ts["exp_avg"][0]), m) and np.array_equal(f(ts["exp_avg_scale"][0]), ms)
        assert np.array_equal(f(ts["exp_avg_sq"][0]), v) and np.array_equal(f(ts["exp_avg_sq_scale"][0]), vs)


@pytest.mark.parametrize("param,grad,state", [("f32", "f32", "f32"), ("master", "bf16", "e4m3"),
                                              ("bf16", "f32", "e4m3"), ("bf16", "bf16", "f32")])
def test_unaligned_tensors_and_neighbours(O, param, grad, state):
    """Tensors one element, or 16 bytes, off their storage's start give the bits of
    aligned ones, what lies before them is left alone, and tensors beside them
    change nothing."""
    a, b, c, d, alone = (tensors(synth.rng(3), [5000, 300], param, grad, state, shift) for shift in (0, 1, 4, 8, 0))
    # codes aligned, their scales not
    if state == "e4m3":
        for k in ("exp_avg_scale", "exp_avg_sq_scale"):
            d[k] = tensors(synth.rng(3), [5000, 300], param, grad, state, 1)[k]
    for ts in (a, b, c, d, lists(alone, lambda v: v[:1])):
        O.AdamW(**ts, lr=1e-3, weight_decay=0.1).step()
    torch.cuda.synchronize()
    for k, v in a.items():
        for i, t in enumerate(v or []):
            for off, n in ((b, 1), (c, 4), (d, 1 if "scale" in k else 8)):
                assert same(t, off[k][i]), (k, i, n)
                assert not bool(off[k][i].as_strided((n,), (1,), 0).float().any())
        assert v is None or same(v[0], alone[k][0])


def test_first_step_from_zero_states(O):
    """New states are zeros; the first step moves each weight by lr, less the
    part of eps, whatever the gradient's size; a zero gradient moves nothing."""
    p = torch.zeros(300, device="cuda")
    gr = torch.full((300,), 1e-3, device="cuda")
    gr[::3] = 0
    gr[1::3] = -20
    for nbits in (32, 8):
        p.zero_()
        opt = O.AdamW([p], [gr], lr=0.5, bits=nbits)
        opt.step()
        torch.cuda.synchronize()
        want = -0.5 * np.sign(f64(gr)) * (np.abs(f64(gr)) / (np.abs(f64(gr)) + 1e-8))
        assert np.all(np.abs(f64(p) - want) <= 16 * U)
        assert opt.steps.tolist() == [1, 0]


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", [[1], [0, 5, 0], SIZES, [70001, 3, 300000], [70000000]])
def test_grad_norm(O, B, grad, sizes):
    ts = tensors(synth.rng(sum(sizes)), sizes, "f32", grad, "f32")
    opt = O.AdamW(**ts, max_norm=0.25)
    out = torch.zeros(4, device="cuda")
    B.biv_grad_norm(opt.table, opt.n, opt.chunks, 0.25, out, opt.ws)
    torch.cuda.synchronize()
    ref = float(np.sqrt(sum(np.sum(f64(x) ** 2) for x in ts["grads"])))
    norm, coef = f64(out)[:2]
    # each square takes at most 4 roundings on the way into its thread's sums, whose
    # own sums keep what they lose; the root halves that, and is rounded once
    assert abs(norm - ref) <= 4 * U * ref
    assert abs(coef - min(1.0, 0.25 / (ref + 1e-6))) <= 64 * U
    first = out.clone()
    B.biv_grad_norm(opt.table, opt.n, opt.chunks, 0.0, out, opt.ws)
    torch.cuda.synchronize()
    assert out[0] == first[0] and out[1] == 1.0 and int(out[2:].view(torch.int32).abs().sum()) == 0


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_clipped_steps(O, state):
    ts = tensors(synth.rng(21), SIZES, "master", "f32", state)
    for x in ts["grads"]:
        x.mul_(100)
    was = snapshot(ts)
    O.AdamW(**ts, lr=1e-3, max_norm=0.5).step()
    torch.cuda.synchronize()
    ref = float(np.sqrt(sum(np.sum(f64(x) ** 2) for x in ts["grads"])))
    assert ref > 0.5
    check(was, ts, SIZES, 1, f32(1e-3), [0.0] * len(SIZES), "master", state, coef=0.5 / (ref + 1e-6),
          slack=2.0 ** -18)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e30])
def test_a_step_without_a_finite_norm_changes_nothing(O, bad):
    ts = tensors(synth.rng(4), SIZES, "bf16", "f32", "e4m3")
    ts["grads"][4][1000] = bad
    was = snapshot(ts)
    opt = O.AdamW(**ts, lr=1e-3, max_norm=1.0, weight_decay=0.1)
    opt.step()
    torch.cuda.synchronize()
    assert opt.steps.tolist() == [0, 0] and not np.isfinite(f64(opt.norm)[0])
    for k, v in ts.items():
        assert v is None or all(same(a, b) for a, b in zip(v, was[k])), k
    ts["grads"][4][1000] = 0.0                     # the next one goes through
    opt.step()
    torch.cuda.synchronize()
    assert opt.steps.tolist() == [1, 0] and not same(ts["params"][4], was["params"][4])


def test_stochastic_rounding_keeps_the_mean(O):
    """Steps far below half a bf16 spacing: nearest rounding leaves the weight,
    stochastic rounding moves it by the right distance on average; a rerun
    repeats its bits."""
    n, lr, steps = 1 << 16, 1e-4, 20
    ends = {}
    for rounding in ("nearest", "stochastic", "stochastic"):
        p = torch.ones(n, dtype=torch.bfloat16, device="cuda")
        opt = O.AdamW([p], [torch.ones(n, device="cuda")], lr=lr, rounding=rounding, seed=3)
        for _ in range(steps):
            opt.step()
        torch.cuda.synchronize()
        assert rounding not in ends or same(p, ends[rounding])
        ends[rounding] = p
    assert bool((ends["nearest"] == 1).all())
    # below 1 the spacing is 2^-8; a step's rounding varies by at most half of it
    sigma = 2.0 ** -9 * np.sqrt(steps) / np.sqrt(n)
    assert abs(f64(ends["stochastic"]).mean() - (1 - lr * steps)) < 5 * sigma + 1e-6


def test_second_moments_decay_under_stochastic_rounding(O):
    """A decay of 0.1% a step is far below an 8-bit spacing (6% and more); it
    shows in the mean of the held roots, and rounding to nearest holds still."""
    n, steps = 1 << 16, 20
    r0 = np.full(n, 0x58, np.uint8)                 # 16, between 15 and 18 on the grid
    r0[::128] = 0x7E                                # the block's largest, 448
    for rounding in ("stochastic", "nearest"):
        opt = O.AdamW([torch.ones(n, device="cuda")], [torch.zeros(n, device="cuda")],
                      exp_avg=[torch.zeros(n, dtype=torch.uint8, device="cuda")],
                      exp_avg_sq=[torch.from_numpy(r0.copy()).cuda()],
                      exp_avg_sq_scale=[torch.ones(n // 128, device="cuda")], lr=0.0, rounding=rounding, seed=9)
        for _ in range(steps):
            opt.step()
        torch.cuda.synchronize()
        r = f64(opt.exp_avg_sq[0]) * np.repeat(f64(opt.exp_avg_sq_scale[0]), 128)
        largest = 448 * 0.999 ** (steps / 2)
        assert np.all(np.abs(r[::128] - largest) <= 1e-4 * largest)   # its own scale follows it
        low, want = r[r0 == 0x58], 16 * 0.999 ** (steps / 2)
        if rounding == "nearest":
            # the code stays, its scale shrinks with the block's largest
            assert np.all(np.abs(low - want) <= 1e-4 * want)
        else:
            # spacing 1 below 16 and 2 above: a step's rounding varies by at most 1
            assert abs(low.mean() - want) < 5 * np.sqrt(steps) / np.sqrt(len(low)) + 1e-4 * want


def test_captured_steps(O):
    """Replays count on, read a new learning rate and new gradients, and give
    the bits of eager steps, while another captured optimizer runs beside."""
    made = [tensors(synth.rng(6), SIZES, "bf16", "f32", "e4m3") for _ in range(2)]
    eager, graph = (O.AdamW(**ts, lr=1e-3, max_norm=1.0, rounding="stochastic", seed=4) for ts in made)
    other_ts = tensors(synth.rng(7), [50000], "master", "bf16", "f32")
    other = O.AdamW(**other_ts, lr=1e-3, max_norm=1.0)
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graph.step()
    with torch.cuda.graph(g2):
        other.step()
    side = torch.cuda.Stream()
    for i in range(3):
        for ts in made:
            for x in ts["grads"]:
                x.mul_(1.5)
        for o in (eager, graph):
            o.set_lr(1e-3 / (i + 1))
        eager.step()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            g2.replay()
        g.replay()
        torch.cuda.synchronize()
    assert eager.steps.tolist() == graph.steps.tolist() == other.steps.tolist() == [3, 0]
    for k, v in made[0].items():
        assert v is None or all(same(a, b) for a, b in zip(v, made[1][k])), k
    again = tensors(synth.rng(7), [50000], "master", "bf16", "f32")
    o = O.AdamW(**again, lr=1e-3, max_norm=1.0)
    for _ in range(3):
        o.step()
    torch.cuda.synchronize()
    assert same(other_ts["params"][0], again["params"][0]) and same(other_ts["exp_avg"][0], again["exp_avg"][0])


def test_mixed_kinds_in_one_call(O):
    """Large matrices with 8-bit states, gains in FP32 beside them, in any order:
    each as in a call of its own, and one step is counted."""
    kinds = [("bf16", "bf16", "e4m3"), ("f32", "f32", "f32"), ("master", "f32", "e4m3"), ("bf16", "f32", "f32")]
    names = ["params", "grads", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"]

    def build():
        g = synth.rng(17)
        parts = [tensors(g, [9000, 31], *k) for k in kinds]
        flat = {k: sum(([p[k][0] if p[k] else None] for p in parts), []) +
                sum(([p[k][1] if p[k] else None] for p in parts), []) for k in names}
        return parts, flat
    parts, flat = build()
    opt = O.AdamW(**flat, lr=1e-3, max_norm=0.1)
    opt.step()
    torch.cuda.synchronize()
    assert opt.steps.tolist() == [1, 0]
    alone, _ = build()
    for p in alone:
        o = O.AdamW(**p, lr=1e-3, max_norm=0.1)
        o.norm.copy_(opt.norm)
        o.max_norm = 0.0                             # the whole call's norm stands in for its own
        o.step()
    torch.cuda.synchronize()
    for p, q in zip(parts, alone):
        for k in names:
            assert p[k] is None or all(same(a, b) for a, b in zip(p[k], q[k])), k


def test_offsets_beyond_32_bits(O):
    """A tensor of 2^31 + 5000 weights with 8-bit states: its end as a tensor of
    its own."""
    n, tail = (1 << 31) + 5000, 5000
    ts = tensors(synth.rng(8), [tail], "bf16", "bf16", "e4m3")
    big = {"params": torch.zeros(n, dtype=torch.bfloat16, device="cuda"),
           "grads": torch.zeros(n, dtype=torch.bfloat16, device="cuda"),
           "exp_avg": torch.zeros(n, dtype=torch.uint8, device="cuda"),
           "exp_avg_sq": torch.zeros(n, dtype=torch.uint8, device="cuda"),
           "exp_avg_scale": torch.zeros((n + 127) // 128, device="cuda"),
           "exp_avg_sq_scale": torch.zeros((n + 127) // 128, device="cuda")}
    for k, t in big.items():
        m = ts[k][0].numel()
        t[t.numel() - m:] = ts[k][0]
    O.AdamW(**{k: [v] for k, v in big.items()}, lr=1e-3, max_norm=0.1).step()
    O.AdamW(**ts, lr=1e-3, max_norm=0.1).step()
    torch.cuda.synchronize()
    for k, t in big.items():
        m = ts[k][0].numel()
        assert same(t[t.numel() - m:], ts[k][0]), k
    assert not bool(big["params"][:1 << 20].any()) and not bool(big["exp_avg"][1 << 30:(1 << 30) + 4096].any())


def test_many_small_tensors_and_lr_scales(O):
    g = synth.rng(12)
    sizes = [int(x) for x in g.integers(0, 700, 500)]
    ts = tensors(g, sizes, "f32", "f32", "f32")
    was = snapshot(ts)
    ls = [f32(x) for x in g.random(500)]
    O.AdamW(**ts, lr=1e-2, lr_scale=ls).step()
    torch.cuda.synchronize()
    for i, n in enumerate(sizes):
        if n:
            check(lists(was, lambda v: v[i:i + 1]), lists(ts, lambda v: v[i:i + 1]), [n], 1, f32(1e-2) * ls[i],
                  [0.0], "f32", "f32")


def test_extreme_gradients(O):
    """Tiny, denormal and huge gradients, and a block of zeros: 8-bit states
    stay finite, nothing is divided by zero, no weight is thrown off.  |m| is at
    most sqrt(v) times the root of the sum of 0.1^2 0.81^j / (0.001 0.999^j) <
    7.3, so a step is at most 7.3 lr sqrt(1 - b2^t) / (1 - b1^t) < 2.1 lr here,
    doubled for a root or mean rounded by half a step."""
    gr = torch.zeros(1024, device="cuda")
    gr[128:256] = 1e-40
    gr[256:384] = 1e-30
    gr[384:512] = 1e15
    gr[512:640:2] = 1e-12
    gr[513:640:2] = 1.0
    p = torch.ones(1024, device="cuda")
    opt = O.AdamW([p], [gr], lr=1e-3, bits=8)
    for _ in range(3):
        opt.step()
    torch.cuda.synchronize()
    assert np.all(np.isfinite(f64(p))) and np.all(f64(p)[:128] == 1.0)
    assert np.all(np.isfinite(f64(opt.exp_avg[0]))) and np.all(np.isfinite(f64(opt.exp_avg_sq[0])))
    assert np.all(np.abs(f64(p) - 1) <= 3 * 4.2e-3)


@pytest.mark.parametrize("param", ["f32", "master", "bf16"])
def test_infinite_second_moments(O, param):
    """A gradient whose square is beyond FP32 makes v infinite and leaves its weight
    where it is, by the stated operations; its neighbours step as ever."""
    n = 4100
    ts = tensors(synth.rng(5), [n], param, "f32", "f32")
    ts["exp_avg"][0].zero_()
    ts["exp_avg_sq"][0].zero_()
    g = ts["grads"][0]
    g.fill_(0.01)
    for i, x in ((3, 1e21), (2047, -1e25), (2048, 1e22), (4099, -1e23)):
        g[i] = x
    was = ts["params"][0].clone()
    opt = O.AdamW(lr=1e-2, **ts)
    for _ in range(2):
        opt.step()
    torch.cuda.synchronize()
    big = g.abs() > 1.0
    v, w = opt.exp_avg_sq[0], ts["params"][0]
    assert torch.all(torch.isinf(v[big])) and torch.all(torch.isfinite(v[~big]))
    assert same(w[big], was[big]) and torch.all(w[~big] != was[~big]) and torch.all(torch.isfinite(w))


def test_optimizer_refuses(O, B):
    p, g = torch.zeros(8, device="cuda"), torch.zeros(8, device="cuda")
    O.AdamW([p], [g])
    for kw in (dict(params=[]), dict(grads=[g, g]), dict(grads=[g[:7]]), dict(grads=[g.half()]), dict(grads=[g.cpu()]),
               dict(params=[p.double()]), dict(params=[torch.zeros(16, device="cuda")[::2]]),
               dict(bits=4), dict(rounding="up"), dict(max_norm=-1.0), dict(max_norm=float("nan")),
               dict(weight_decay=[0.1, 0.1]), dict(lr=torch.zeros(2, device="cuda")), dict(lr=torch.zeros(1)),
               dict(step=torch.zeros(1, dtype=torch.int32, device="cuda")), dict(exp_avg=[torch.zeros(7, device="cuda")]),
               dict(exp_avg=[torch.zeros(8, dtype=torch.uint8, device="cuda")],
                    exp_avg_sq=[torch.zeros(8, device="cuda")]), dict(params=[p.cpu()])):
        with pytest.raises(ValueError):
            O.AdamW(**(dict(params=[p], grads=[g]) | kw))
    with pytest.raises(B.BivError):
        O.AdamW([p], [g], master=[torch.zeros(8, device="cuda")])     # an f32 weight has no master
    with pytest.raises(B.BivError):
        O.AdamW([p, p], [g, g])                                       # the same weight twice
    with pytest.raises(B.BivError):
        O.AdamW([p], [p])                                             # the gradient is the weight
    for kw in (dict(betas=(1.0, 0.9)), dict(eps=0.0)):
        with pytest.raises(B.BivError):
            O.AdamW([p], [g], **kw).step()


@pytest.mark.parametrize("param", ["f32", "master", "bf16"])
@pytest.mark.parametrize("state", ["f32", "e4m3"])
@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), "weight"])
def test_nan_and_infinity_stay_visible(O, param, state, rounding, bad):
    """Without a clip a NaN or infinite gradient, or a NaN weight, leaves NaN in its
    weight (no draw of random bits may carry it into a zero) and a moment that is
    not finite; all else has the bits of a run in which that gradient is 0."""
    at = [(4, 1000), (5, 2047), (8, 77), (8, 4999), (9, 0)]      # whole chunks, the last of them, a short tensor
    runs = []
    for spoil in (False, True):
        ts = tensors(synth.rng(41), SIZES, param, "f32", state)
        for i, j in at:
            for k in ("grads", "exp_avg", "exp_avg_sq"):
                ts[k][i][j] = 0
            if spoil and bad == "weight":
                ts["params"][i][j] = float("nan")
                if param == "master":
                    ts["master"][i][j] = float("nan")
            elif spoil:
                ts["grads"][i][j] = bad
        opt = O.AdamW(**ts, lr=1e-3, weight_decay=0.1, rounding=rounding, seed=8)
        seen = []
        for _ in range(2):
            opt.step()
            torch.cuda.synchronize()
            seen.append(snapshot(ts))
        runs.append(seen)
    e8, inf = state == "e4m3", isinstance(bad, float) and np.isinf(bad)
    for step, (clean, got) in enumerate(zip(*runs)):
        for i, n in enumerate(SIZES):
            hit = np.zeros(n, bool)
            hit[[j for t, j in at if t == i]] = True
            # the block of an infinite moment: its scale is infinite, so all that it
            # holds is lost at the next step
            lost = hit.copy()
            if e8 and inf:
                for j in np.nonzero(hit)[0]:
                    lost[j // 128 * 128:j // 128 * 128 + 128] = True
            weights = ["params"] + (["master"] if param == "master" else [])
            for k in weights:
                w, ref = f64(got[k][i]), f64(clean[k][i])
                spoiled = lost if step else hit
                assert np.all(np.isnan(w[spoiled])), (k, i, step)
                assert np.array_equal(w[~spoiled], ref[~spoiled])
            if bad == "weight":
                assert same(got["exp_avg"][i], clean["exp_avg"][i])
                assert same(got["exp_avg_sq"][i], clean["exp_avg_sq"][i])
                continue
            m, v = f64(got["exp_avg"][i]), f64(got["exp_avg_sq"][i])
            if e8:
                with np.errstate(invalid="ignore"):          # 0 times an infinite scale
                    m = m * np.repeat(f64(got["exp_avg_scale"][i]), 128)[:n]
                    v = v * np.repeat(f64(got["exp_avg_sq_scale"][i]), 128)[:n]
                assert np.all(np.isnan(f64(got["exp_avg"][i])[hit]))
            assert not np.any(np.isfinite(m[hit])) and not np.any(np.isfinite(v[hit]))
            for k in ("exp_avg", "exp_avg_sq"):
                x, ref = f64(got[k][i]), f64(clean[k][i])
                assert np.array_equal(x[~lost], ref[~lost]), (k, i, step)


@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
def test_an_infinite_second_moment_in_an_8_bit_block(O, rounding):
    """A gradient of 1e22 (its square is beyond FP32): at the next step the positive
    second moments of its block are infinite and their weights only decay, zero ones
    are NaN; other blocks are not touched."""
    n = 5000
    ts, ref = (tensors(synth.rng(43), [n], "f32", "f32", "e4m3") for _ in range(2))
    for x in (ts, ref):
        for k in ("grads", "exp_avg", "exp_avg_sq"):
            x[k][0][[130, 140]] = 0
    ts["grads"][0][130] = 1e22
    opts = [O.AdamW(**x, lr=1e-3, weight_decay=0.1, rounding=rounding, seed=8) for x in (ts, ref)]
    w = []
    for _ in range(2):
        for o in opts:
            o.step()
        torch.cuda.synchronize()
        w.append(f64(ts["params"][0]))
    keep = np.float32(1) - np.float32(1e-3) * np.float32(0.1)
    blk = np.arange(128, 256)
    blk = blk[blk != 140]
    assert np.array_equal(w[1][blk], (w[0][blk].astype(np.float32) * keep).astype(np.float64))
    assert np.isnan(w[1][140]) and np.all(np.isinf(f64(ts["exp_avg_sq_scale"][0])[1:2]))
    out = np.r_[0:128, 256:n]
    assert np.array_equal(w[1][out], f64(ref["params"][0])[out])

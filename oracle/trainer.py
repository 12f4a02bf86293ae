"""The trainer's end of a step, in float64: the clipped policy loss with its
gradient and the AdamW update.  TEST INFRASTRUCTURE ONLY.

The pages name the recipe (GRPO without importance correction, "Finish RL
Training Faster", section "两组结果，要连同分母一起读") and the measure (k3 KL,
section "零差异需要一个精确的比较对象") but print no formulas; these are the
plainest readings.

  r = exp(clamp(lp - old)), pg = max(-A r, -A clip(r)), dual bound -A dual for A < 0
  kl = exp(e) - e - 1, e = clamp(ref - lp);  loss = sum w (pg + beta kl - gamma H)
  AdamW: m, v moving means of g and g^2 with bias correction, decay on w itself
"""
from __future__ import annotations

import numpy as np

from oracle import codecs

F64 = np.float64
FAR = 20.0
BLOCK = 128
TINY = 2.0 ** -100


def row_weights(T, seq_start, mask, reduce, norm):
    """(weight per row, sequence per row or -1); reduce: token, seq or sum."""
    seq = np.full(T, -1)
    for s in range(len(seq_start) - 1):
        seq[seq_start[s]:seq_start[s + 1]] = s
    use = seq >= 0
    if mask is not None:
        use &= np.asarray(mask[:T]) != 0
    w = np.zeros(T, F64)
    n = np.bincount(seq[use], minlength=max(1, len(seq_start) - 1))
    live = int(np.sum(n > 0))
    for t in np.nonzero(use)[0]:
        w[t] = {"token": 1.0 / use.sum(), "seq": 1.0 / (live * n[seq[t]]), "sum": 1.0 / norm}[reduce]
    return w, seq


def policy_loss(lp, w, adv, old=None, ref=None, lo=0.2, hi=0.2, dual=0.0, beta=0.0, gamma=0.0, H=None):
    """Per-row advantage adv; rows of weight 0 are left out.  Returns (stats
    [8], dlp [T])."""
    T = len(lp)
    on = np.asarray(w) > 0
    stats, dlp = np.zeros(8, F64), np.zeros(T, F64)
    for t in np.nonzero(on)[0]:
        x, A, wt = F64(lp[t]), F64(adv[t]), w[t]
        gap = x - F64(old[t]) if old is not None else F64(0)
        d = min(max(gap, -FAR), FAR)
        r = np.exp(d)
        u, c = -A * r, -A * min(max(r, 1 - lo), 1 + hi)
        taken = u >= c
        pg = max(u, c)
        if dual > 0 and A < 0 and pg > -A * dual:
            pg, taken = -A * dual, False
        g = u if taken and abs(gap) < FAR else 0.0
        kl = 0.0
        if ref is not None:
            far = F64(ref[t]) - x
            e = min(max(far, -FAR), FAR)
            kl = np.expm1(e) - e
            if abs(far) < FAR:
                g -= beta * np.expm1(e)
        h = F64(H[t]) if H is not None else 0.0
        dlp[t] = wt * g
        stats[:4] += wt * (pg + beta * kl - gamma * h), wt * pg, wt * kl, wt * h
        stats[4] += not taken
        stats[5] += np.expm1(d) - d
        stats[6] = max(stats[6], abs(gap))
    n = int(on.sum())
    stats[4:6] /= max(n, 1)
    stats[7] = n
    return stats, dlp


def token_logprobs(z, target, it=1.0):
    """z [T, V] -> (lp [T], entropy [T], p [T, V], log p [T, V])."""
    x = np.asarray(z, F64) * it
    x = x - np.max(x, axis=1, keepdims=True)
    logp = x - np.log(np.sum(np.exp(x), axis=1, keepdims=True))
    p = np.exp(logp)
    H = -np.sum(np.where(p > 0, p * np.where(p > 0, logp, 0), 0), axis=1)
    return logp[np.arange(len(x)), target], H, p, logp


def policy_dz(z, target, dlp, w, gamma, it=1.0):
    """The loss's gradient by the logits, from its gradient by lp."""
    _, H, p, logp = token_logprobs(z, target, it)
    dz = -p * dlp[:, None] + gamma * w[:, None] * p * (np.where(p > 0, logp, 0) + H[:, None])
    dz[np.arange(len(dlp)), target] += dlp
    return it * np.where((w > 0)[:, None], dz, 0.0)


# ------------------------------------------------------------------ AdamW --
def adamw(w, g, m, v, t, lr, wd, b1=0.9, b2=0.999, eps=1e-8, coef=1.0):
    """(w, m, v) after step t (1 is the first), v the mean of squares."""
    w, g, m, v = (np.asarray(a, F64) for a in (w, g, m, v))
    g = g * coef
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    w = w - lr * wd * w - lr * (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps)
    return w, m, v


def block_scale(x):
    """Scale of each block of 128 (the last one shorter) as an array like x."""
    s = np.empty(len(x), F64)
    for i in range(0, len(x), BLOCK):
        s[i:i + BLOCK] = max(np.max(np.abs(x[i:i + BLOCK])), TINY) / 448.0
    return s


def mix32(x):
    x = np.asarray(x, np.uint64)
    m = np.uint64(0xFFFFFFFF)
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0x7FEB352D)) & m
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0x846CA68B)) & m
    return x ^ (x >> np.uint64(16))


def random_bits(first, n, seed, t):
    """The hash of elements first .. first + n - 1 at step t: (16 bits for m,
    16 for the root of v, 16 for the weight)."""
    m = np.uint64(0xFFFFFFFF)
    i = np.arange(first, first + n, dtype=np.uint64)
    key = mix32((seed + t * 0x9E3779B9) & 0xFFFFFFFF) ^ np.uint64(((seed >> 32) * 0x9E3779B1) & 0xFFFFFFFF)
    h = mix32((((i & m) ^ key) + (i >> np.uint64(32)) * np.uint64(0x85EBCA6B)) & m)
    return h & np.uint64(0xFFFF), h >> np.uint64(16), mix32(h ^ np.uint64(0x9E3779B9)) & np.uint64(0xFFFF)


def grid_step(y, digits, low):
    """Spacing at y of the grid of `digits` significant bits, exponents >= low."""
    e = np.where(np.asarray(y) == 0, low, np.frexp(np.abs(y))[1] - 1)
    return np.ldexp(1.0, np.maximum(e, low) - (digits - 1))


def stochastic(y, bits, digits, low):
    """|y| up with a chance of the part cut off (16 random bits), sign kept."""
    s = grid_step(y, digits, low)
    return np.copysign(np.floor(np.abs(y) / s + bits.astype(F64) / 65536.0) * s, y)


def e4m3_nearest(y):
    return codecs.e4m3_to_f32(codecs.f32_to_e4m3(np.asarray(y, np.float32))).astype(F64)

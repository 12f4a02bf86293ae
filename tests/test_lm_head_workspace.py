"""The workspace of the LM head's gradient over its sizes, on the host: the bound that
include/biv.h states, and its place beside the logits that it replaces."""
import random

import pytest
import torch

MIB = 1 << 20


@pytest.fixture(scope="module")
def B():
    from invariant_forward_bitwise_gb300 import biv, build
    build.build()
    biv.load()
    return biv


def up(n, to=256):
    return (n + to - 1) // to * to


def bound(T, V, K, f32):
    t, k = up(T), up(K)
    # all chunks, of at most 8192 columns: up to a chunk more than V
    dz = min(max(192 * MIB, t * 48 * 1024), t * (up(V) + 8192) * 2) * (2 if f32 else 1)
    return dz + max(192 * MIB, 4 * t * k) + t * (3 * k + 64) + MIB


def sizes():
    r = random.Random(5)
    log = lambda lo, hi: int(round(2 ** r.uniform(lo, hi)))  # noqa: E731
    some = [(T, V, K) for T in (1, 13, 200, 257, 1000, 2000, 8192) for V in (1, 4096, 32003, 151936)
            for K in (8, 256, 2048)]
    return some + [(log(0, 20), log(0, 23.9), 8 * log(0, 13)) for _ in range(4000)]


def test_the_stated_bound(B):
    f, b = torch.float32, torch.bfloat16
    for T, V, K in sizes():
        for dh, dw in ((b, b), (f, b), (f, f)):
            n = B.biv_lm_head_backward_workspace(T, V, K, dh, dw)
            assert 0 < n <= bound(T, V, K, dh is f), (T, V, K, dh, n)


def test_few_rows_of_a_large_vocabulary(B):
    """However large the vocabulary, of dz no more than 192 MiB a part is held (three
    chunks of up to 4096 rows)."""
    for T in (1, 13, 200, 256, 600, 1000, 1500, 4096):
        for V in (131072, 151936, 1 << 23):
            for K in (8, 256, 2048):
                rest = max(192 * MIB, 4 * up(T) * up(K)) + up(T) * (3 * up(K) + 64) + MIB
                assert B.biv_lm_head_backward_workspace(T, V, K) <= 192 * MIB + rest
                assert B.biv_lm_head_backward_workspace(T, V, K, torch.float32) <= 384 * MIB + rest


@pytest.mark.parametrize("K", [256, 2048])
def test_a_micro_batch_is_far_below_its_logits(B, K):
    for T in (2048, 4096, 8192):
        logits = 4 * T * 151936
        assert B.biv_lm_head_backward_workspace(T, 151936, K) < logits // 4
        assert B.biv_lm_head_backward_workspace(T, 151936, K, torch.float32, torch.float32) < logits // 1.9


def test_refusals(B):
    for bad in (dict(dh_dtype=torch.float16), dict(dw_dtype=torch.float64), dict(T=-1), dict(V=0), dict(K=12)):
        with pytest.raises(B.BivError):
            B.biv_lm_head_backward_workspace(**{**dict(T=4, V=8, K=8), **bad})

"""GPU tests of decode over pages of very different V scales: what a page brings to the answer keeps its accuracy
whatever its probability and its scale are for themselves."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import rope_block as rb
from tests.block_harness import Cache, bound, check_rows, f64, randn, run_decode, run_prefill

pytestmark = pytest.mark.gpu

LAYOUTS = [(32, 8, 128), (64, 8, 64), (8, 1, 256), (16, 1, 128), (16, 1, 64), (2, 2, 128)]


def _check_decode(got, c, b, q, sm, window=0):
    """got [Hq, d] within the roundings of a kernel that weighs keys in f16 relative to the largest p * vscale, with
    2^15 of room above it: bound() with what is lost of weights below 2^-29 of it (2^-40 of it on every key)."""
    k, v, vs = c.sequence(b)
    L = c.lens[b]
    ref, size, _, tiny_w, score = rb.attention(q[None], k, v, vs, [L - 1], sm, window)
    lost = 2.0 ** -15 * tiny_w[0]
    lim = bound(ref[0], size[0], lost, score[0], c.d, L)
    assert np.isfinite(got).all()
    worst = float((np.abs(got - ref[0]) / lim).max())
    assert worst <= 1.0, (b, worst)


@pytest.mark.parametrize("k", [14, 20, 26, 40, 80])
@pytest.mark.parametrize("hq,hkv,d", LAYOUTS)
def test_large_valued_pages_of_small_probability(hq, hkv, d, k):
    """Every third page has 2^-k of the others' probability and 2^k of their V scale: half of the answer."""
    g = np.random.default_rng(k)
    c = Cache(hkv, d, [400, 37, 6000, 16], seed=k, spread=0.0)
    c.k[:] = 0                                             # scores from dimension 0 alone, in log2 units under sm = ln 2
    for b, L in enumerate(c.lens):
        for p in range(-(-L // 16)):
            blk, rows = c.tables[b, p], min(16, L - 16 * p)
            large = p % 3 == 1
            x = -g.uniform(1, 1.2, (hkv, rows)) * k if large else -g.uniform(0, 1, (hkv, rows))
            c.k[blk, :, :rows, 0] = oracle.e4m3_encode(x.astype(np.float32))
            c.ks[blk], c.vs[blk] = 1.0, 2.0 ** (k / 2 if large else -k / 2)
    c.cuda()
    q = torch.ones((4, hq, d), dtype=torch.bfloat16)
    out = f64(run_decode(c, q.cuda(), math.log(2)))
    pre = f64(run_prefill(c, q.cuda(), torch.arange(5, dtype=torch.int32).cuda(), 1, math.log(2)))
    for b, L in enumerate(c.lens):
        _check_decode(out[b], c, b, f64(q[b]), math.log(2))
        check_rows(pre[b:b + 1], c, b, f64(q[b:b + 1]), [L - 1], math.log(2), 0, True, b)


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("hq,hkv,d", LAYOUTS)
def test_pages_2_to_the_40_apart(hq, hkv, d, window):
    """V scales from 2^-20 to 2^20 and K scales over 2^20, at random."""
    g = np.random.default_rng(d)
    c = Cache(hkv, d, [400, 37, 3000], seed=5, spread=0.0, scale=2.0 ** -7)
    c.vs = (c.vs * 2.0 ** g.uniform(-20, 20, c.vs.shape)).astype(np.float32)
    c.ks = (c.ks * 2.0 ** g.uniform(-20, 0, c.ks.shape)).astype(np.float32)
    c.cuda()
    q = randn((3, hq, d), 3)
    out = f64(run_decode(c, q.cuda(), d ** -0.5, window))
    for b in range(3):
        _check_decode(out[b], c, b, f64(q[b]), d ** -0.5, window)


@pytest.mark.parametrize("hq,hkv,d", LAYOUTS)
def test_scores_of_2_to_the_30(hq, hkv, d):
    """Scores at which fp32 steps by 64: the key far above the others is the answer."""
    c = Cache(hkv, d, [100], seed=1)
    for p in range(7):
        blk = c.tables[0, p]
        c.k[blk], c.ks[blk] = 0x40, 2.0 ** (8 + p)         # codes of 2
        c.k[blk, :, 3] = 0x7E                              # ... and of 448
    c.cuda()
    q = torch.full((1, hq, d), 64.0, dtype=torch.bfloat16)
    out = f64(run_decode(c, q.cuda(), 1.0))
    want = np.repeat(rb.values(c.v, c.vs, c.tables[0], 100)[99 // 16 * 16 + 3], hq // hkv, 0)
    assert (np.abs(out[0] - want) <= 2.0 ** -8 * (1 + 2.0 ** -10) * np.abs(want)).all()

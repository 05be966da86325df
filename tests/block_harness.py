"""Shared plumbing of the rotary-append and block-scale tests: seeded
block-scaled caches, and error bounds counted from the roundings."""
import numpy as np
import torch

import oracle
from oracle import rope_block as rb
from fp8_kv_cache_fp8kv_gb300 import binding as fk

# A rotation in fp32: the fraction of a turn is rounded to 2^-26 of a turn
# (9.4e-8 rad), sincospi to at most 2 ulp of 1 (1.2e-7), one product and one
# fma round by 2^-24 each: below 3.4e-7 (|x| + |y|) < 2^-21 (|x| + |y|).
ROPE_REL = 2.0 ** -21
BF16 = 2.0 ** -8       # half a step, relative to the value


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


class Cache:
    """A block-scaled cache of `lens` tokens a sequence, pages in random order
    among `extra` unused ones, codes and scales random; everything that no
    sequence owns is NaN: the codes of unused pages and of rows behind a
    sequence's end, the scales of unused pages."""

    def __init__(self, hkv, d, lens, seed=0, extra=3, capacity=None, spread=2.0, scale=0.01):
        g = np.random.default_rng(seed)
        cap = [max(n, c) for n, c in zip(lens, capacity or lens)]
        pages = [-(-n // 16) for n in cap]
        self.nb = sum(pages) + extra
        self.lens = list(lens)
        perm = g.permutation(self.nb)
        self.mb = max([1] + pages)
        self.tables = np.zeros((len(lens), self.mb), np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.tables[b, :n] = perm[at:at + n]
            self.tables[b, n:] = 2 ** 30          # never read
            at += n
        shape = (self.nb, hkv, 16, d)
        self.hkv, self.d = hkv, d
        self.k = np.full(shape, 0x7F, np.uint8)
        self.v = np.full(shape, 0xFF, np.uint8)
        self.ks = np.full((self.nb, hkv), np.nan, np.float32)
        self.vs = np.full((self.nb, hkv), np.nan, np.float32)
        for b, n in enumerate(lens):
            for p in range(-(-n // 16)):
                blk, rows = self.tables[b, p], min(16, n - 16 * p)
                for c, s in ((self.k, self.ks), (self.v, self.vs)):
                    x = (g.standard_normal((hkv, rows, d)) * 100).astype(np.float32)
                    c[blk, :, :rows] = oracle.e4m3_encode(x)
                    s[blk] = (scale * 2.0 ** g.uniform(-spread, spread, hkv)).astype(np.float32)

    def cuda(self):
        self.gk, self.gv = torch.from_numpy(self.k.copy()).cuda(), torch.from_numpy(self.v.copy()).cuda()
        self.gks, self.gvs = torch.from_numpy(self.ks.copy()).cuda(), torch.from_numpy(self.vs.copy()).cuda()
        self.gt = torch.from_numpy(self.tables).cuda()
        self.gl = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        return self

    def pull(self):
        """The device's codes and scales."""
        self.k, self.v = self.gk.cpu().numpy(), self.gv.cpu().numpy()
        self.ks, self.vs = self.gks.cpu().numpy(), self.gvs.cpu().numpy()
        return self

    def sequence(self, b):
        """k, v values and V scales [L, H, d] / [L, H] of sequence b."""
        L = self.lens[b]
        ids = self.tables[b, : -(-L // 16)]
        return (rb.values(self.k, self.ks, self.tables[b], L), rb.values(self.v, self.vs, self.tables[b], L),
                np.repeat(self.vs[ids].astype(np.float64), 16, 0)[:L])


def bound(ref, size, tiny, score, d, keys):
    """Per element, from the roundings of the kernels:
      2^-8 |ref|             the output's bf16
      2^-11 size             the probabilities' f16 (an average over the keys)
      tiny                   f16 probabilities below 2^-14 (2^-25 each)
      2 delta size           a score's error delta moves p and the sum: d fp32
                             products summed (2^-23 an addition, tensor cores
                             may cut) on sums of at most `score`, the scaling,
                             exp2's argument and exp2 itself (2^-20)
      (keys / 16 + 64) 2^-23 size   the sums over keys, per 16-key MMA and merge"""
    delta = score * (d + 16) * 2.0 ** -23 + 2.0 ** -20
    return BF16 * np.abs(ref) + size * (2.0 ** -11 + 2 * delta + (keys / 16 + 64) * 2.0 ** -23) + tiny + 1e-30


def check_rows(got, c, b, q, positions, sm, window, prefill, what=""):
    """got [R, Hq, d] against sequence b of cache c for queries q (fp64) at `positions`."""
    k, v, vs = c.sequence(b)
    ref, size, tiny, tiny_w, score = rb.attention(q, k, v, vs, positions, sm, window)
    lim = bound(ref, size, tiny_w if prefill else tiny, score, c.d, len(k))
    assert np.isfinite(got).all(), what
    worst = float((np.abs(got - ref) / lim).max()) if got.size else 0.0
    assert worst <= 1.0, (what, worst)


def run_decode(c, q, sm, window=0, max_len=None, ws=None, out=None, stream=None):
    B, hq, d = q.shape
    mx = max(c.lens + [1]) if max_len is None else max_len
    mx = min(mx, c.mb * 16)
    own = ws is None
    ws = fk.alloc_workspace(B, hq, c.hkv, d, mx, 16, window) if own else ws
    out = torch.full_like(q, float("nan")) if out is None else out
    fk.fp8kv_paged_decode_block(q, c.gk, c.gv, c.gks, c.gvs, c.gt, c.gl, mx, sm, window, out, ws, stream)
    if own:
        torch.cuda.synchronize()
        assert fk.fp8kv_read_error(ws) == 0
    return out


def run_prefill(c, q, starts, max_q, sm, window=0, max_len=None, ws=None, out=None):
    T, hq, d = q.shape
    mx = min(max(c.lens + [1]) if max_len is None else max_len, c.mb * 16)
    own = ws is None
    ws = fk.alloc_prefill_workspace(len(c.lens), max_q, mx, hq, c.hkv, d, 16, window) if own else ws
    out = torch.full_like(q, float("nan")) if out is None else out
    fk.fp8kv_paged_prefill_block(q, c.gk, c.gv, c.gks, c.gvs, c.gt, c.gl, starts, max_q, mx, sm, window, out, ws)
    if own:
        torch.cuda.synchronize()
        assert fk.fp8kv_read_error(ws) == 0
    return out


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def randn(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)

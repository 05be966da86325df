"""fp8kv_paged_decode_weights: its output bit for bit that of the decode call of the same cache, its weights against
the definition in 64 bits.

Tolerance of a weight: the FP32 sum old * decay + sum_h p_h rounds at most g + 2 times, each within 2^-24 of the result
or a part of it (18 * 2^-24 < 2^-19); a probability is off by twice its scores' error, which is that of FP32 sums of d
products, at most 256 * 2^-24 * sum |q k| sm <= 2^-16 * 10 = 2^-12.7, and of exp2 (2^-21): 2^-11.5 of sum_h p_h in all."""
import math

import pytest
import torch

from fp8_kv_cache_fp8kv_gb300 import binding as fk
from tests.spec_harness import PAGE, Cache, attend, queries

pytestmark = pytest.mark.gpu


def plain_decode(c, q, window, sm, scales=None):
    B, hq, d = q.shape
    ws = fk.alloc_workspace(B, hq, c.hkv, d, c.max_len, 16, window)
    out = torch.empty_like(q)
    if scales is not None:
        fk.fp8kv_paged_decode_per_head(q, c.k, c.v, c.tables, c.seq_lens, c.max_len, *scales, sm, window, out, ws)
    elif c.fmt == "bf16":
        fk.fp8kv_paged_decode_bf16(q, c.k, c.v, c.tables, c.seq_lens, c.max_len, sm, window, out, ws)
    else:
        call = fk.fp8kv_paged_decode if c.fmt == "e4m3" else fk.fp8kv_paged_decode_e5m2
        call(q, c.k, c.v, c.tables, c.seq_lens, c.max_len, *c.scale, sm, window, out, ws)
    return out


def run(c, q, w, decay, window=0, sm=None, scales=None, workspace=None, stream=None, out=None):
    B, hq, d = q.shape
    sm = 1 / math.sqrt(d) if sm is None else sm
    ws = fk.alloc_weights_workspace(B, hq, c.hkv, d, c.max_len, window=window) if workspace is None else workspace
    out = torch.empty_like(q) if out is None else out
    kind = c.kind_args()
    if scales is not None:
        kind.update(k_scales=scales[0], v_scales=scales[1])
    fk.fp8kv_paged_decode_weights(q, c.k, c.v, c.tables, c.seq_lens, c.max_len, sm, window, out, w, decay, ws, stream=stream, **kind)
    return out, ws


def reference(c, q, w, decay, window, sm, scales=None):
    """(weights in 64 bits, what is added to each)"""
    want, added = w.double().clone(), torch.zeros_like(w, dtype=torch.float64)
    g = q.shape[1] // c.hkv
    decay = float(torch.tensor(decay, dtype=torch.float32))
    for b, n in enumerate(c.lens):
        if n == 0:
            continue
        lo = max(0, n - window) if window > 0 else 0
        t = torch.arange(lo, n, device=w.device)
        page = c.tables[b].long()[t // PAGE]
        seen = (torch.arange(n) >= lo)[None]
        for h in range(c.hkv):
            k, v = c.rows("k", b, h, scales=scales), c.rows("v", b, h, scales=scales)
            p = attend(q[b:b + 1, h * g:(h + 1) * g], k, v, seen, sm)[2].sum(0)[0, lo:]
            old = want[page, h, t % PAGE] * decay
            old[-1] = 0
            want[page, h, t % PAGE] = old + p
            added[page, h, t % PAGE] = p
    return want, added


def check(lens, hq, hkv, d, fmt="e4m3", window=0, decay=0.9, seed=0, per_head=False):
    c = Cache(lens, hkv, d, fmt, seed)
    q = queries(len(lens), hq, d, seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    w = torch.rand((c.blocks, hkv, PAGE), generator=g).cuda()
    # what no call may read: the newest token's place, and places that hold no token
    untouched = torch.ones_like(w, dtype=torch.bool)
    for b, n in enumerate(lens):
        t = torch.arange(max(0, n - window) if window > 0 else 0, n, device="cuda")
        untouched[c.tables[b].long()[t // PAGE], :, t % PAGE] = False
        if n:
            w[c.tables[b, (n - 1) // PAGE].long(), :, (n - 1) % PAGE] = math.nan
    clean = torch.nan_to_num(w)
    w[untouched] = math.nan
    before = w.clone()
    scales = None
    if per_head:
        scales = tuple(torch.rand(hkv, generator=g).cuda() * s + s for s in c.scale)
    sm = 1 / math.sqrt(d)
    out, ws = run(c, q, w, decay, window, scales=scales)
    torch.cuda.synchronize()
    assert fk.fp8kv_read_error(ws) == 0
    if scales is not None and fmt == "e5m2":       # the one form no other decode call has
        for b, n in enumerate(lens):
            for h in range(hkv):
                heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
                ref, mass, _ = attend(q[b:b + 1, heads], c.rows("k", b, h, scales=scales), c.rows("v", b, h, scales=scales),
                                      torch.ones((1, n), dtype=torch.bool), sm)
                assert ((out[b, heads].double() - ref[0]).abs() <= 2.0 ** -8 * ref[0].abs() + 2.0 ** -9 * mass[0] + 1e-6).all()
    else:
        assert torch.equal(out.view(torch.int16), plain_decode(c, q, window, sm, scales).view(torch.int16))
    want, added = reference(c, q, clean, decay, window, sm, scales)
    assert torch.equal(w[untouched].view(torch.int32), before[untouched].view(torch.int32))
    err = (w.double() - want).abs()[~untouched]
    bound = (2.0 ** -11.5 * added + 2.0 ** -19 * want)[~untouched] + 1e-30
    assert torch.isfinite(w[~untouched]).all()
    assert (err <= bound).all(), (err / bound).max().item()
    # the same call on the same input gives the same bits
    again = before.clone()
    run(c, q, again, decay, window, scales=scales, workspace=ws)
    assert torch.equal(again.view(torch.int32), w.view(torch.int32))


LAYOUTS = [(32, 8, 128), (64, 8, 64), (8, 1, 256), (8, 8, 128), (16, 1, 128), (16, 1, 64), (32, 2, 256), (4, 2, 64)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", LAYOUTS)
def test_layouts(hq, hkv, d, fmt):
    check([700, 33, 0, 1, 16], hq, hkv, d, fmt)


@pytest.mark.parametrize("window", [1, 15, 16, 17, 128, 600, 10 ** 6])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_windows(window, d):
    check([700, 33, 129, 1, 16, 128], 8, 2, d, window=window, seed=window)


@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0, 3.0])
def test_decays(decay):
    check([257, 40], 8, 2, 128, decay=decay)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_per_head_scales(fmt):
    check([300, 90], 16, 4, 128, fmt, per_head=True)


@pytest.mark.parametrize("lens,hq,hkv", [([40000], 8, 1), ([9000, 20000], 16, 2), ([9000], 4, 4)])
def test_units_split_over_many_ctas(lens, hq, hkv):
    """Both merges: in the decode grid, and by its own kernel."""
    check(lens, hq, hkv, 128, seed=3)


def test_more_scores_than_one_launch_holds():
    """A bound that makes a sequence's scores exceed their share of a launch: the batch runs in several."""
    check([20, 300, 0, 1000, 77], 32, 2, 64, seed=4)
    c = Cache([20, 300, 0, 1000, 77], 2, 64, "e4m3", 4)
    wide = torch.full((5, 400000 // 16), -7, dtype=torch.int32, device="cuda")
    wide[:, : c.tables.shape[1]] = c.tables
    q = queries(5, 32, 64, 5)
    w = torch.rand((c.blocks, 2, PAGE)).cuda()
    a = w.clone()
    one, _ = run(c, q, a, 0.9)
    c.tables, c.max_len = wide, 400000
    many, ws = run(c, q, w, 0.9)
    assert fk.fp8kv_read_error(ws) == 0
    # (another split of the sums: the outputs may differ in their last place)
    assert ((one.double() - many.double()).abs() <= 2.0 ** -7 * one.double().abs() + 1e-4).all()
    assert ((a.double() - w.double()).abs() <= 2.0 ** -11 * a.double()).all()


def test_many_sequences():
    check([1 + (i * 7) % 60 for i in range(520)], 4, 2, 64, seed=6)


def test_bad_block_ids_and_lengths():
    c = Cache([64, 64], 1, 64, "e4m3", 5)
    good = c.tables.clone()
    c.tables[0, 1] = 10 ** 6
    w = torch.zeros((c.blocks, 1, PAGE), device="cuda")
    q = queries(2, 4, 64, 1)
    out, ws = run(c, q, w, 1.0)
    assert fk.fp8kv_read_error(ws) == 1
    assert (w[good[0, 1].long()] == 0).all() and (w[good[1].long()] != 0).all()
    c.tables, c.max_len = good, 50
    out, ws = run(c, q, w, 1.0)
    assert fk.fp8kv_read_error(ws) == 1                     # longer than the bound: clamped

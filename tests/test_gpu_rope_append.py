"""GPU tests of the rotary append: into the per-tensor caches through a slot
mapping, into the block-scaled cache by sequence, and a whole serving run
(chunked prompts, then decode steps) over the latter."""
import numpy as np
import pytest
import torch

import oracle
from fp8_kv_cache_fp8kv_gb300 import binding as fk
from oracle import rope_block as rb
from tests.block_harness import BF16, ROPE_REL, Cache, bits, check_rows, f64, randn, run_decode, run_prefill

pytestmark = pytest.mark.gpu


def _freq(R, base=10000.0):
    return torch.tensor([base ** (-i / (R // 2)) for i in range(R // 2)], dtype=torch.float32)


def _fused(T, hq, hkv, d, seed, pad=0):
    """q, k, v as slices of one projection's rows, with `pad` elements between tokens."""
    x = randn((T, (hq + 2 * hkv) * d + pad), seed).cuda()
    return (x[:, :hq * d].unflatten(1, (hq, d)), x[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
            x[:, (hq + hkv) * d:(hq + 2 * hkv) * d].unflatten(1, (hkv, d)))


def _check_q(got, want, mag):
    lim = BF16 * np.abs(want) + 2 * ROPE_REL * mag
    assert (np.abs(f64(got) - want) <= lim).all()


def _check_codes(got, want, mag, scale, encode, decode):
    """Each code is the conversion of some value within the fp32 rotation's error of `want` (conversions are monotonic)."""
    lo, hi = want - ROPE_REL * mag, want + ROPE_REL * mag
    s = np.float32(scale)
    with np.errstate(over="ignore"):
        a = decode(encode((lo.astype(np.float32) / s).astype(np.float32)))
        z = decode(encode((hi.astype(np.float32) / s).astype(np.float32)))
    v = decode(got)
    assert ((a <= v) & (v <= z)).all(), int(((a > v) | (v > z)).sum())


def _slots(T, nb, bs, seed):
    return torch.from_numpy(np.random.default_rng(seed).permutation(nb * bs)[:T].astype(np.int64))


def _at(cache, slots, bs):
    return cache[slots // bs, :, slots % bs]


CASES = [  # hq, hkv, d, R, pairs, axes, T
    (32, 8, 128, 128, False, 1, 37), (8, 2, 64, 64, True, 1, 16), (8, 1, 256, 256, False, 3, 33),
    (4, 4, 128, 64, False, 2, 1), (6, 3, 64, 16, True, 4, 17), (2, 1, 256, 48, True, 3, 5), (64, 8, 64, 32, False, 1, 100),
    (1, 1, 128, 112, False, 1, 15),
]


@pytest.mark.parametrize("fmt", [fk.CACHE_E4M3, fk.CACHE_E5M2, fk.CACHE_BF16])
@pytest.mark.parametrize("hq,hkv,d,R,pairs,axes,T", CASES)
def test_slots(hq, hkv, d, R, pairs, axes, T, fmt):
    bs, nb = 16, T // 16 + 4
    q, k, v = _fused(T, hq, hkv, d, 7 * T + d, pad=8 * (T % 3))
    rng = np.random.default_rng(T)
    pos = rng.integers(0, 200000, (axes, T)).astype(np.int32)
    axis = (np.arange(R // 2) % axes).astype(np.uint8)
    freq, slots = _freq(R), _slots(T, nb, bs, T)
    wide = fmt == fk.CACHE_BF16
    kc = torch.full((nb, hkv, bs, d), 1, dtype=torch.bfloat16 if wide else torch.uint8, device="cuda")
    vc = kc.clone()
    ksc, vsc = (1.0, 1.0) if wide else (0.011, 0.007)
    qo = torch.full((T, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    fk.fp8kv_rope_append(q, k, v, torch.from_numpy(pos).cuda(), freq.cuda(), slots.cuda(), qo, kc, vc, ksc, vsc,
                         freq_axis=torch.from_numpy(axis).cuda(), style=int(pairs), cache_format=fmt)
    torch.cuda.synchronize()
    wq, mq = rb.rope(f64(q), pos, freq.numpy(), axis, pairs)
    wk, mk = rb.rope(f64(k), pos, freq.numpy(), axis, pairs)
    _check_q(qo, wq, mq)
    if wide:
        _check_q(_at(kc, slots.cuda(), bs), wk, mk)
        assert torch.equal(_at(vc, slots.cuda(), bs), v)
    else:
        gk, gv = _at(kc.cpu(), slots, bs).numpy(), _at(vc.cpu(), slots, bs).numpy()
        e5 = fmt == fk.CACHE_E5M2
        enc, dec = (oracle.e5m2_encode, oracle.e5m2_decode) if e5 else (oracle.e4m3_encode, oracle.e4m3_decode)
        _check_codes(gk, wk, mk, ksc, enc, dec)
        assert np.array_equal(gv, (oracle.quantize_bf16_e5m2 if e5 else oracle.quantize_bf16)(bits(v), vsc))
    rest = torch.ones(nb * bs, dtype=torch.bool)
    rest[slots] = False
    left = torch.nonzero(rest)[:, 0].cuda()
    assert (_at(kc, left, bs) == 1).all() and (_at(vc, left, bs) == 1).all()


def test_slots_without_rotation_are_quant_append():
    T, hkv, d, bs, nb = 50, 3, 128, 16, 6
    _, k, v = _fused(T, 1, hkv, d, 1)
    k[3, 1, 5], k[4, 0, 0], v[9, 2, 1] = float("inf"), float("nan"), float("-inf")
    slots = _slots(T, nb, bs, 2)
    slots[7], slots[8], slots[9] = -1, nb * bs, 2 ** 40      # skipped
    slots = slots.cuda()
    hs = torch.tensor([0.5, 0.013, 3.0], device="cuda")
    for bsz, blocks in ((16, 6), (1, 96), (5, 20)):
        for per_head in (False, True):
            for e5 in (False, True):
                if e5 and per_head:
                    continue
                a, b, c, e = (torch.full((blocks, hkv, bsz, d), 9, dtype=torch.uint8, device="cuda") for _ in range(4))
                fk.fp8kv_rope_append(None, k, v, None, None, slots, None, a, b, 0.01, 0.02,
                                     k_scales=hs if per_head else None, v_scales=hs if per_head else None,
                                     cache_format=fk.CACHE_E5M2 if e5 else fk.CACHE_E4M3)
                kk, vv = k.contiguous(), v.contiguous()
                if per_head:
                    fk.fp8kv_quant_append_per_head(kk, vv, slots, c, e, hs, hs)
                elif e5:
                    fk.fp8kv_quant_append_e5m2(kk, vv, slots, c, e, 0.01, 0.02)
                else:
                    fk.fp8kv_quant_append(kk, vv, slots, c, e, 0.01, 0.02)
                assert torch.equal(a, c) and torch.equal(b, e)


def test_skipped_tokens_have_their_queries_rotated():
    T, hq, d = 20, 2, 64
    q, k, v = _fused(T, hq, 1, d, 4)
    kc = torch.zeros((1, 1, 16, d), dtype=torch.uint8, device="cuda")
    vc, qo = kc.clone(), torch.zeros((T, hq, d), dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(T, dtype=torch.int32).cuda()
    fk.fp8kv_rope_append(q, k, v, pos, _freq(64).cuda(), torch.full((T,), -1).cuda(), qo, kc, vc)
    _check_q(qo, *rb.rope(f64(q), pos.cpu().numpy(), _freq(64).numpy()))
    assert not kc.any() and not vc.any()


def test_positions_of_any_size():
    """2^20 and far beyond, negative ones too: the angle is reduced exactly.  (At 2^31 - 1 the frequency's quotient by
    2 pi, held to 2^-48, leaves 2^-17 of a turn: 5e-5 rad.)"""
    pos = np.asarray([0, 1, -1, 4095, 4096, -4096, 2 ** 20, 2 ** 20 + 1, -(2 ** 20) - 7, 2 ** 24 + 1, 2 ** 31 - 1,
                      -2 ** 31], dtype=np.int64)
    T, d = len(pos), 128
    q, k, v = _fused(T, 2, 1, d, 3)
    kc = torch.zeros((1, 1, 16, d), dtype=torch.bfloat16, device="cuda")
    vc, qo = kc.clone(), torch.empty((T, 2, d), dtype=torch.bfloat16, device="cuda")
    freq = _freq(128)
    freq[0] = 3.0
    fk.fp8kv_rope_append(q, k, v, torch.from_numpy(pos.astype(np.int32)).cuda(), freq.cuda(), torch.arange(T).cuda(), qo,
                         kc, vc, cache_format=fk.CACHE_BF16)
    want, mag = rb.rope(f64(q), pos, freq.numpy())
    angle = 2 * np.pi * np.abs(pos) * 3.0 / (2 * np.pi) * 2.0 ** -47        # what 2^-48 of the angle, twice, comes to
    lim = BF16 * np.abs(want) + (2 * ROPE_REL + angle[:, None, None]) * mag
    assert (np.abs(f64(qo) - want) <= lim).all()


def test_queries_in_place_and_axes_out_of_range():
    T, hq, d = 33, 4, 128
    q, k, v = (x.contiguous() for x in _fused(T, hq, 2, d, 5))
    pos = torch.randint(0, 1000, (2, T), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    axis = torch.tensor([0, 1] * 32, dtype=torch.uint8)
    bad = axis.clone()
    bad[axis == 0] = 200                           # read as axis 0
    kc = torch.zeros((4, 2, 16, d), dtype=torch.uint8, device="cuda")
    vc, slots, freq = kc.clone(), torch.arange(T).cuda(), _freq(128).cuda()
    a, b = torch.empty_like(q), q.clone()
    fk.fp8kv_rope_append(q, k, v, pos, freq, slots, a, kc, vc, freq_axis=axis.cuda())
    fk.fp8kv_rope_append(b, k, v, pos, freq, slots, b, kc, vc, freq_axis=bad.cuda())
    assert torch.equal(a, b)


def test_the_binding_refuses_rows_it_cannot_read():
    q, k, v = _fused(4, 2, 2, 64, 1)
    kc = torch.zeros((1, 2, 16, 64), dtype=torch.uint8, device="cuda")
    vc, slots, qo = kc.clone(), torch.arange(4).cuda(), torch.empty((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    args = dict(positions=torch.arange(4, dtype=torch.int32).cuda(), inv_freq=_freq(64).cuda(), slot_mapping=slots,
                q_out=qo, k_cache=kc, v_cache=vc)
    for bad in (dict(k_new=k.transpose(1, 2).contiguous().transpose(1, 2)), dict(k_new=k.float()),
                dict(v_new=v.cpu()), dict(q=q[:, :, ::2].repeat(1, 1, 2)[:, :, ::1].transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises((ValueError, TypeError)):
            fk.fp8kv_rope_append(**{**dict(q=q, k_new=k, v_new=v), **args, **bad})
    x = torch.zeros(4 * 256 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fk.Fp8kvError):             # rows not on 16 bytes
        fk.fp8kv_rope_append(q=None, k_new=x[1:513].view(4, 2, 64), v_new=v, **{**args, "q_out": None})
    with pytest.raises(fk.Fp8kvError):             # one row for all tokens
        fk.fp8kv_rope_append(q=None, k_new=k[:1].expand(4, 2, 64), v_new=v, **{**args, "q_out": None})


# ------------------------------------------------------------------ block scales

def _block_append(c, q, k, v, pos, freq, starts, ws, qo=None, axis=None, pairs=False, max_len=None):
    mx = c.mb * 16 if max_len is None else max_len
    fk.fp8kv_rope_append_block(q, k, v, pos, freq, qo, c.gk, c.gv, c.gks, c.gvs, c.gt, c.gl,
                               None if starts is None else torch.tensor(starts, dtype=torch.int32).cuda(), mx, ws,
                               freq_axis=axis, style=int(pairs))


def _check_block(c, before, k, v, starts, wk, mk):
    """The device's cache after an append of wk (+- ROPE_REL mk) and v to the cache `before`."""
    c.pull()
    lens = c.lens
    want_v, want_vs = rb.append(before.v, before.vs, f64(v), before.tables, lens, starts)
    assert np.array_equal(c.vs, want_vs, equal_nan=True)
    assert np.array_equal(c.v, want_v)
    want_k, want_ks = rb.append(before.k, before.ks, wk, before.tables, lens, starts)
    assert np.array_equal(c.ks, want_ks, equal_nan=True)       # (no largest value of these seeds is next to a border)
    new = np.zeros(c.k.shape[:1] + c.k.shape[2:3], bool)
    for b, L in enumerate(lens):
        n = starts[b + 1] - starts[b]
        for p in range(L - n, L):
            blk, r, t = before.tables[b, p // 16], p % 16, starts[b] + p - (L - n)
            new[blk, r] = True
            for h in range(c.hkv):
                _check_codes(c.k[blk, h, r], wk[t, h], mk[t, h], want_ks[blk, h], oracle.e4m3_encode, oracle.e4m3_decode)
    keep = ~np.broadcast_to(new[:, None], c.k.shape[:3])
    assert np.array_equal(c.k[keep], want_k[keep])


def _copy(c):
    z = Cache.__new__(Cache)
    z.__dict__.update(c.__dict__)
    z.k, z.v, z.ks, z.vs = c.k.copy(), c.v.copy(), c.ks.copy(), c.vs.copy()
    return z


def _history(hkv, d, hist, counts, seed, scale=0.01):
    """A cache that holds `hist` tokens a sequence and has room for `counts` more."""
    c = Cache(hkv, d, hist, seed=seed, capacity=[a + b for a, b in zip(hist, counts)], scale=scale)
    c.lens = [a + b for a, b in zip(hist, counts)]
    return c


BLOCK_CASES = [  # hq, hkv, d, R, pairs, axes, history, new tokens
    (32, 8, 128, 128, False, 1, [0, 5, 16, 31, 0], [1, 1, 1, 1, 40]),
    (8, 2, 64, 64, True, 3, [3, 0, 12, 100], [14, 16, 70, 0]),
    (8, 1, 256, 256, False, 2, [15, 17, 0], [1, 31, 33]),
    (4, 3, 128, 32, True, 1, [0, 9], [200, 7]),
    (6, 6, 64, 16, False, 1, [1], [15]),
    (2, 5, 256, 240, False, 4, [7, 8, 9, 10], [9, 8, 7, 6]),
]


@pytest.mark.parametrize("scale", [0.002, 0.05])     # pages that grow, pages that keep their scale
@pytest.mark.parametrize("hq,hkv,d,R,pairs,axes,hist,counts", BLOCK_CASES)
def test_block_append(hq, hkv, d, R, pairs, axes, hist, counts, scale):
    c = _history(hkv, d, hist, counts, seed=hq + d, scale=scale)
    before = _copy(c)
    c.cuda()
    starts = [0] + np.cumsum(counts).tolist()
    T = starts[-1]
    q, k, v = _fused(T, hq, hkv, d, 11 * T, pad=16)
    rng = np.random.default_rng(T)
    pos = rng.integers(0, 100000, (axes, T)).astype(np.int32)
    axis = (np.arange(R // 2) % axes).astype(np.uint8)
    qo = torch.full((T, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = fk.alloc_append_workspace()
    _block_append(c, q, k, v, torch.from_numpy(pos).cuda(), _freq(R).cuda(), starts, ws, qo,
                  torch.from_numpy(axis).cuda(), pairs)
    assert fk.fp8kv_read_error(ws) == 0
    _check_q(qo, *rb.rope(f64(q), pos, _freq(R).numpy(), axis, pairs))
    _check_block(c, before, k, v, starts, *rb.rope(f64(k), pos, _freq(R).numpy(), axis, pairs))
    # once more on the same cache: nothing moves
    a = [x.clone() for x in (c.gk, c.gv, c.gks, c.gvs)]
    _block_append(c, q, k, v, torch.from_numpy(pos).cuda(), _freq(R).cuda(), starts, ws, qo,
                  torch.from_numpy(axis).cuda(), pairs)
    for x, y in zip(a, (c.gk, c.gv, c.gks, c.gvs)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_block_append_without_rotation_infinities_and_zeros():
    hkv, d = 3, 128
    c = _history(hkv, d, [4, 0, 20], [10, 18, 3], seed=1, scale=0.0005)
    before = _copy(c)
    c.cuda()
    starts = [0, 10, 28, 31]
    _, k, v = _fused(31, 1, hkv, d, 2)
    k[2, 0, 7], k[3, 0, 7], v[11, 2, 0], v[12, 2, 1] = float("inf"), float("nan"), float("-inf"), float("nan")
    k[10:26, 1], v[10:26, 1] = 0.0, float("inf")        # a page of zeros, a page without a finite value
    k[0, 2, 0], v[28, 0, 3] = 3e38, 1e-39               # beyond the largest scale; subnormal
    ws = fk.alloc_append_workspace()
    _block_append(c, None, k, v, None, None, starts, ws)
    assert fk.fp8kv_read_error(ws) == 0
    c.pull()
    for got, gots, x, old, olds in ((c.k, c.ks, k, before.k, before.ks), (c.v, c.vs, v, before.v, before.vs)):
        want, scales = rb.append(old, olds, f64(x), before.tables, c.lens, starts)
        assert np.array_equal(gots, scales, equal_nan=True)
        nan = (want & 0x7F) == 0x7F                     # a NaN's sign is the hardware's
        assert np.array_equal(got[~nan], want[~nan]) and ((got[nan] & 0x7F) == 0x7F).all()
    assert 2.0 ** -40 in c.ks and 2.0 ** 40 in c.ks and 2.0 ** -40 in c.vs


def test_block_append_default_positions_and_decode_rows():
    """No positions: each token's place in its sequence; no q_starts: one row per sequence, empty ones left alone."""
    hq, hkv, d = 4, 2, 64
    c = _history(hkv, d, [15, 0, 16, 3], [1, 0, 1, 1], seed=4)
    before = _copy(c)
    c.cuda()
    q, k, v = _fused(4, hq, hkv, d, 6)
    qo = torch.full((4, hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = fk.alloc_append_workspace()
    _block_append(c, q, k, v, None, _freq(64).cuda(), None, ws, qo)
    assert fk.fp8kv_read_error(ws) == 0
    rows = [0, 2, 3]
    pos = [15, 16, 3]
    wq, mq = rb.rope(f64(q[rows]), pos, _freq(64).numpy())
    _check_q(qo[rows], wq, mq)
    assert (qo[1] == 5.0).all()
    wk, mk = rb.rope(f64(k[rows]), pos, _freq(64).numpy())
    _check_block(c, before, k, v[rows], [0, 1, 1, 2, 3], wk, mk)


def test_block_append_leaves_padding_rows_and_skips_what_does_not_fit():
    hq, hkv, d = 4, 1, 128
    T = 60
    q, k, v = _fused(T, hq, hkv, d, 3)
    for starts, lens, bad in (
            ([0, 20, 40], [20, 20], None),            # rows 40.. are padding
            ([5, 20, 40], [20, 20], None),            # and rows before the first
            ([0, 20, 40], [10, 20], 0),               # more new tokens than tokens
            ([0, 20, 61], [20, 41], 1),               # past the packed rows
            ([-3, 20, 40], [23, 20], 0), ([0, 20, 10], [20, 20], 1), ([0, 20, 40], [20, 81], 1),
            ([0, 20, 40], [-5, 20], 0), ([0, 2 ** 31 - 1, -2 ** 31], [20, 20], None)):
        c = Cache(hkv, d, [80, 80], seed=1)
        before = _copy(c)
        c.lens = lens
        c.cuda()
        qo = torch.full((T, hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
        ws = fk.alloc_append_workspace()
        _block_append(c, q, k, v, None, _freq(128).cuda(), starts, ws, qo, max_len=80)
        err = fk.fp8kv_read_error(ws)
        wild = starts[1] > T
        assert err == (1 if bad is not None or wild else 0), (starts, lens)
        done = torch.zeros(T, dtype=torch.bool)
        for b in range(2):
            if b != bad and not wild:
                done[starts[b]:starts[b + 1]] = True
        assert (qo[~done.cuda()] == 5.0).all() and (qo[done.cuda()] != 5.0).any(-1).all()
        c.pull()
        for b in range(2):
            if b == bad or wild:
                assert np.array_equal(c.k[c.tables[b]], before.k[c.tables[b]])


def test_block_append_reports_bad_blocks_and_writes_nothing_there():
    hq, hkv, d = 2, 2, 64
    c = Cache(hkv, d, [48, 48], seed=2)
    before = _copy(c)
    c.cuda()
    c.gt[0, 1], c.gt[1, 2] = c.nb, -1
    q, k, v = _fused(96, hq, hkv, d, 3)
    qo = torch.zeros((96, hq, d), dtype=torch.bfloat16, device="cuda")
    ws = fk.alloc_append_workspace()
    _block_append(c, q, k, v, None, _freq(64).cuda(), [0, 48, 96], ws, qo)
    assert fk.fp8kv_read_error(ws) == 1
    pos = list(range(48)) * 2
    _check_q(qo, *rb.rope(f64(q), pos, _freq(64).numpy()))
    c.pull()
    written = {int(c.tables[b, p]) for b, p in ((0, 0), (0, 2), (1, 0), (1, 1))}
    for blk in range(c.nb):
        same = np.array_equal(c.k[blk], before.k[blk]) and np.array_equal(c.v[blk], before.v[blk])
        assert same == (blk not in written)


def test_block_append_offsets_past_32_bits():
    hkv, d = 8, 128
    small = _history(hkv, d, [10, 0], [20, 40], seed=3)
    before = _copy(small)
    nb = (1 << 32) // (hkv * 16 * d) + 64
    shift = nb - small.nb
    small.cuda()
    gk = torch.empty((nb, hkv, 16, d), dtype=torch.uint8, device="cuda")
    gv = torch.empty_like(gk)
    gks, gvs = torch.empty((nb, hkv), device="cuda"), torch.empty((nb, hkv), device="cuda")
    gk[shift:], gv[shift:], gks[shift:], gvs[shift:] = small.gk, small.gv, small.gks, small.gvs
    small.gk, small.gv, small.gks, small.gvs = gk, gv, gks, gvs
    small.gt = torch.from_numpy(np.where(small.tables < small.nb, small.tables + shift, 0).astype(np.int32)).cuda()
    _, k, v = _fused(60, 1, hkv, d, 3)
    ws = fk.alloc_append_workspace()
    _block_append(small, None, k, v, None, None, [0, 20, 60], ws)
    assert fk.fp8kv_read_error(ws) == 0
    small.gk, small.gv, small.gks, small.gvs = gk[shift:], gv[shift:], gks[shift:], gvs[shift:]
    _check_block(small, before, k, v, [0, 20, 60], f64(k), np.zeros(k.shape))


def test_many_sequences_find_their_pages():
    """More sequences than one level of the search covers, empty ones among them."""
    hkv, d, B = 1, 64, 1100
    counts = [(7 * i) % 5 if i % 3 else 0 for i in range(B)]
    hist = [(5 * i) % 19 for i in range(B)]
    c = _history(hkv, d, hist, counts, seed=5)
    before = _copy(c)
    c.cuda()
    starts = [0] + np.cumsum(counts).tolist()
    _, k, v = _fused(starts[-1], 1, hkv, d, 8)
    ws = fk.alloc_append_workspace()
    _block_append(c, None, k, v, None, None, starts, ws)
    assert fk.fp8kv_read_error(ws) == 0
    _check_block(c, before, k, v, starts, f64(k), np.zeros(k.shape))


@pytest.mark.parametrize("hq,hkv,d,window", [(32, 8, 128, 0), (16, 2, 64, 40), (8, 1, 256, 0)])
def test_a_serving_run(hq, hkv, d, window):
    """Two prompt chunks, then decode steps, of three sequences over one block-scaled cache, the calls back to back on a
    side stream with one workspace: every attention output against the oracle on the cache as it stands, and the cache
    against the rotated keys within E4M3's half step."""
    B, chunks, steps = 3, ([30, 17, 64], [11, 40, 1]), 6
    total = [sum(x) + steps for x in zip(*chunks)]
    c = _history(hkv, d, [0] * B, total, seed=1).cuda()
    sm, freq = d ** -0.5, _freq(d, 1e6)
    mx = c.mb * 16
    have = [0] * B
    ws = fk.alloc_prefill_workspace(B, 64, mx, hq, hkv, d, 16, window)
    wsd = fk.alloc_workspace(B, hq, hkv, d, mx, 16, window)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    want_k = [np.zeros((n, hkv, d)) for n in total]
    want_v = [np.zeros((n, hkv, d)) for n in total]
    for step in range(len(chunks) + steps):
        decode = step >= len(chunks)
        counts = [1] * B if decode else chunks[step]
        starts = [0] + np.cumsum(counts).tolist()
        q, k, v = _fused(starts[-1], hq, hkv, d, 100 + step)
        have = [a + b for a, b in zip(have, counts)]
        c.lens = list(have)
        c.gl.copy_(torch.tensor(have, dtype=torch.int32))
        gst = torch.tensor(starts, dtype=torch.int32).cuda()
        qo = torch.empty((starts[-1], hq, d), dtype=torch.bfloat16, device="cuda")
        out = torch.full_like(qo, float("nan"))
        fq = freq.cuda()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            fk.fp8kv_rope_append_block(q, k, v, None, fq, qo, c.gk, c.gv, c.gks, c.gvs, c.gt, c.gl,
                                       None if decode else gst, mx, wsd if decode else ws)
            if decode:
                run_decode(c, qo, sm, window, mx, wsd, out)
            else:
                run_prefill(c, qo, gst, max(counts), sm, window, mx, ws, out)
        st.synchronize()
        assert fk.fp8kv_read_error(wsd if decode else ws) == 0
        c.pull()
        for b, n in enumerate(counts):
            pos = list(range(have[b] - n, have[b]))
            rows = slice(starts[b], starts[b + 1])
            want_k[b][pos] = rb.rope(f64(k[rows]), pos, freq.numpy())[0]
            want_v[b][pos] = f64(v[rows])
            _check_q(qo[rows], *rb.rope(f64(q[rows]), pos, freq.numpy()))
            check_rows(f64(out[rows]), c, b, f64(qo[rows]), pos, sm, window, not decode, (step, b))
    for b in range(B):
        k, v, _ = c.sequence(b)
        ids = c.tables[b, : -(-have[b] // 16)]
        for got, want, s in ((k, want_k[b], c.ks), (v, want_v[b], c.vs)):
            # a code is rounded once when it is written and, where its page grew, once more as a subnormal: half a
            # step each (2^-4 of a normal value, 2^-10 scales of a subnormal one)
            step = np.repeat(s[ids].astype(np.float64), 16, 0)[:have[b], :, None]
            assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) * (1 + 2.0 ** -15) + 2 * 2.0 ** -10 * step).all()


def test_captured_append_and_decode_advance_with_their_lengths():
    """A decode step captured once (append, then attention) and replayed while the lengths and inputs change in place."""
    hq, hkv, d, steps = 8, 2, 128, 20
    c = _history(hkv, d, [13, 30], [steps, steps], seed=6).cuda()
    c.gl.copy_(torch.tensor([14, 31], dtype=torch.int32))
    freq = _freq(128).cuda()
    x = torch.zeros((2, (hq + 2 * hkv) * d), dtype=torch.bfloat16, device="cuda")
    q, k, v = (x[:, :hq * d].unflatten(1, (hq, d)), x[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
               x[:, (hq + hkv) * d:].unflatten(1, (hkv, d)))
    qo = torch.empty((2, hq, d), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(qo)
    mx = c.mb * 16
    ws = fk.alloc_workspace(2, hq, hkv, d, mx)

    def call():
        fk.fp8kv_rope_append_block(q, k, v, None, freq, qo, c.gk, c.gv, c.gks, c.gvs, c.gt, c.gl, None, mx, ws)
        run_decode(c, qo, 0.1, 0, mx, ws, out)
    c.gl.zero_()                                    # warm up on empty sequences: nothing is written
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(steps):
        x.copy_(randn(tuple(x.shape), 50 + i, 1.0 + 0.5 * i))
        c.lens = [14 + i, 31 + i]
        c.gl.copy_(torch.tensor(c.lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.pull()
        for b in range(2):
            check_rows(f64(out[b:b + 1]), c, b, f64(qo[b:b + 1]), [c.lens[b] - 1], 0.1, 0, False, (i, b))
    assert fk.fp8kv_read_error(ws) == 0


@pytest.mark.parametrize("at", [1, 2, 31, 32, 33, 64, 68])
def test_starts_that_fall_are_reported_and_nothing_out_of_range_is_written(at):
    """Whichever sequence the starts fall at, also where the search for a CTA's sequence would pass it by."""
    hkv, d, B, n = 1, 64, 70, 20
    for start in (0, 3, n * at - 1, n * at - 40):
        if start < 0:
            continue
        c = Cache(hkv, d, [48] * B, seed=at).cuda()
        starts = [n * i for i in range(B + 1)]
        starts[at + 1] = start
        ws = fk.alloc_append_workspace()
        _, k, v = _fused(n * B, 1, hkv, d, 4)
        _block_append(c, None, k, v, None, None, starts, ws)
        assert fk.fp8kv_read_error(ws) == 1
        owned = {int(x) for row in c.tables for x in row}
        before = _copy(c)
        c.pull()
        for blk in set(range(c.nb)) - owned:
            assert np.array_equal(c.k[blk], before.k[blk]) and np.array_equal(c.v[blk], before.v[blk])


def test_appends_and_attention_on_two_streams_at_once():
    """Two sets of sequences of one cache, each with a stream and workspaces of its own, their calls in flight
    together: the outcome of each is what it is alone."""
    hq, hkv, d, steps = 16, 4, 128, 30
    freq = _freq(d).cuda()
    kw = dict(hkv=hkv, d=d, hist=[600, 37, 255, 1200], counts=[40] * 4, seed=8)

    def run(order):
        c = _history(**kw).cuda()
        outs, streams = [], []
        for half in order:
            rows = slice(2 * half, 2 * half + 2)
            q, k, v = _fused(80, hq, hkv, d, 20 + half)
            gt, gl = c.gt[rows].contiguous(), c.gl[rows].contiguous()
            gs = torch.tensor([0, 40, 80], dtype=torch.int32).cuda()
            ws = fk.alloc_prefill_workspace(2, 40, c.mb * 16, hq, hkv, d)
            wsd = fk.alloc_workspace(2, hq, hkv, d, c.mb * 16)
            qo = torch.empty((80, hq, d), dtype=torch.bfloat16, device="cuda")
            out, dec = torch.full_like(qo, float("nan")), torch.full_like(qo[:2], float("nan"))
            outs.append((half, qo, out, dec, ws, wsd, gt, gl, gs, q, k, v))
            streams.append(torch.cuda.Stream())
        torch.cuda.synchronize()
        for (half, qo, out, dec, ws, wsd, gt, gl, gs, q, k, v), st in zip(outs, streams):
            with torch.cuda.stream(st):
                fk.fp8kv_rope_append_block(q, k, v, None, freq, qo, c.gk, c.gv, c.gks, c.gvs, gt, gl, gs, c.mb * 16, ws)
                for _ in range(steps):
                    fk.fp8kv_paged_prefill_block(qo, c.gk, c.gv, c.gks, c.gvs, gt, gl, gs, 40, c.mb * 16, 0.1, 0, out, ws)
                    fk.fp8kv_paged_decode_block(qo[:2], c.gk, c.gv, c.gks, c.gvs, gt, gl, c.mb * 16, 0.1, 0, dec, wsd)
            if len(order) == 1:
                st.synchronize()
        torch.cuda.synchronize()
        for o in outs:
            assert fk.fp8kv_read_error(o[4]) == 0 and fk.fp8kv_read_error(o[5]) == 0
        c.pull()
        pages = {o[0]: [int(x) for r in (2 * o[0], 2 * o[0] + 1) for x in c.tables[r, : -(-c.lens[r] // 16)]] for o in outs}
        return {o[0]: (bits(o[1]), bits(o[2]), bits(o[3]), c.k[pages[o[0]]], c.v[pages[o[0]]], c.ks[pages[o[0]]])
                for o in outs}

    alone = {**run([0]), **run([1])}
    both = run([0, 1])
    for half in (0, 1):
        for x, y in zip(alone[half], both[half]):
            assert np.array_equal(x, y)

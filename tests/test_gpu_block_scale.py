"""GPU tests of attention over the block-scaled cache: decode and prefill
against the fp64 oracle, element by element within the roundings' bound."""
import numpy as np
import pytest
import torch

from fp8_kv_cache_fp8kv_gb300 import binding as fk
from oracle import rope_block as rb
from tests.block_harness import Cache, check_rows, f64, randn, run_decode, run_prefill

pytestmark = pytest.mark.gpu

LAYOUTS = [(32, 8, 128), (64, 8, 64), (8, 1, 256), (4, 4, 128), (3, 3, 64), (4, 2, 256), (16, 1, 64), (16, 1, 128),
           (16, 1, 256)]


def _decode_case(c, hq, sm, window, seed, **kw):
    q = randn((len(c.lens), hq, c.d), seed + 1)
    out = f64(run_decode(c, q.cuda(), sm, window, **kw))
    for b, L in enumerate(c.lens):
        if L == 0:
            assert not out[b].any()
        else:
            check_rows(out[b:b + 1], c, b, f64(q[b:b + 1]), [L - 1], sm, window, False, "sequence %d of %d" % (b, L))


@pytest.mark.parametrize("hq,hkv,d", LAYOUTS)
def test_decode_layouts_and_lengths(hq, hkv, d):
    c = Cache(hkv, d, [1, 0, 15, 16, 17, 33, 500, 2049, 0], seed=hq + d).cuda()
    _decode_case(c, hq, d ** -0.5, 0, hq)


@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 4000])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (16, 2, 64), (8, 1, 256)])
def test_decode_windows(hq, hkv, d, window):
    c = Cache(hkv, d, [1, 16, 17, 100, 101, 0, 1500], seed=window).cuda()
    _decode_case(c, hq, d ** -0.5, window, window)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (16, 2, 64), (8, 1, 256), (16, 1, 128)])
@pytest.mark.parametrize("exponent", [0, 30, -30])
def test_scales_that_differ_by_2_to_the_40(hq, hkv, d, exponent):
    """Neighbouring pages 2^40 apart: the small ones count as exactly where the large ones weigh little."""
    c = Cache(hkv, d, [400, 37], seed=5, spread=0.0, scale=2.0 ** -7)
    sign = np.where(np.arange(c.nb) % 2, 1.0, -1.0)[:, None]
    c.vs = (c.vs * 2.0 ** (min(max(exponent, -12), 12) + 20 * sign)).astype(np.float32)
    c.ks = (c.ks * 2.0 ** np.random.default_rng(1).uniform(-20, 0, c.ks.shape)).astype(np.float32)
    c.cuda()
    _decode_case(c, hq, d ** -0.5, 0, 3)
    _prefill_case(c, hq, [9, 37], d ** -0.5, 0, 4)


def test_small_value_pages_survive_beside_large_ones():
    """All the probability on a page whose V scale is 2^-20 of its neighbour's: the answer is that page's values, to
    the accuracy of its own scale, and not lost in the neighbour's."""
    hq, hkv, d = 4, 1, 128
    c = Cache(hkv, d, [32], seed=8, spread=0.0)
    a, z = c.tables[0, :2]
    c.k[:] = 0
    c.k[a, 0, 3] = 0x70                    # the one key that every query meets: codes of 128
    c.vs[a], c.vs[z] = 2.0 ** -18, 2.0 ** 2
    c.cuda()
    q = torch.ones((1, hq, d), dtype=torch.bfloat16)
    out = f64(run_decode(c, q.cuda(), 1.0))
    want = rb.values(c.v, c.vs, c.tables[0], 32)[3, 0]
    assert np.abs(out[0] - want).max() <= 2.0 ** -8 * np.abs(want).max()
    out = f64(run_prefill(c, q.cuda(), torch.tensor([0, 1], dtype=torch.int32).cuda(), 1, 1.0))
    assert np.abs(out[0] - want).max() <= 2.0 ** -8 * np.abs(want).max()


def test_zero_value_sink_keeps_its_weight():
    """A first page of zero values with the least scale still takes its share of the softmax."""
    for hq, hkv, d in ((4, 1, 128), (8, 1, 64), (4, 1, 256)):
        c = Cache(hkv, d, [300], seed=2)
        a = c.tables[0, 0]
        c.v[a], c.vs[a] = 0, 2.0 ** -40
        c.ks[a] *= 3
        c.cuda()
        _decode_case(c, hq, d ** -0.5, 0, 1)
        _prefill_case(c, hq, [200], d ** -0.5, 0, 1)


@pytest.mark.parametrize("sm", [0.0, -0.1, 30.0])
def test_score_scales(sm):
    for hq, hkv, d in ((8, 2, 128), (8, 1, 64), (8, 1, 256)):
        c = Cache(hkv, d, [70, 200], seed=4, scale=0.003).cuda()
        q = randn((2, hq, d), 9, 0.1)
        out = f64(run_decode(c, q.cuda(), sm))
        for b in range(2):
            check_rows(out[b:b + 1], c, b, f64(q[b:b + 1]), [c.lens[b] - 1], sm, 0, False)
        _prefill_case(c, hq, [70, 45], sm, 0, 9, qscale=0.1)


def test_decode_more_sequences_than_one_launch():
    c = Cache(1, 64, [(37 * i) % 60 for i in range(520)], seed=6).cuda()
    _decode_case(c, 4, 0.125, 0, 2)


def test_decode_long_context_split_over_the_grid():
    for hq, hkv, d, L in ((32, 4, 128, 40000), (8, 1, 256, 20000), (64, 4, 64, 20000)):
        c = Cache(hkv, d, [L], seed=7).cuda()
        _decode_case(c, hq, d ** -0.5, 0, 3)


def _prefill_case(c, hq, counts, sm, window, seed, qscale=1.0):
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    q = randn((int(starts[-1]), hq, c.d), seed + 1, qscale)
    out = f64(run_prefill(c, q.cuda(), torch.from_numpy(starts).cuda(), max(counts), sm, window))
    for b, n in enumerate(counts):
        L = c.lens[b]
        check_rows(out[starts[b]:starts[b + 1]], c, b, f64(q[starts[b]:starts[b + 1]]), list(range(L - n, L)), sm,
                   window, True, "sequence %d: %d of %d" % (b, n, L))


@pytest.mark.parametrize("hq,hkv,d", LAYOUTS)
def test_prefill_layouts(hq, hkv, d):
    c = Cache(hkv, d, [1, 0, 17, 40, 200, 333], seed=hq + d).cuda()
    _prefill_case(c, hq, [1, 0, 17, 3, 70, 33], d ** -0.5, 0, 1)
    _prefill_case(c, hq, [1, 0, 1, 1, 1, 1], d ** -0.5, 0, 2)     # one query tile a sequence


@pytest.mark.parametrize("window", [1, 16, 40, 5000])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (16, 2, 64), (4, 1, 256)])
def test_prefill_windows(hq, hkv, d, window):
    c = Cache(hkv, d, [17, 300, 200], seed=window).cuda()
    _prefill_case(c, hq, [17, 90, 5], d ** -0.5, window, 1)
    _prefill_case(c, hq, [2, 1, 3], d ** -0.5, window, 2)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (16, 2, 64), (4, 1, 256)])
def test_prefill_splits_a_long_context(hq, hkv, d):
    c = Cache(hkv, d, [5000, 777], seed=1).cuda()
    _prefill_case(c, hq, [5, 2], d ** -0.5, 0, 1)
    _prefill_case(c, hq, [40, 20], d ** -0.5, 0, 2)


def test_prefill_rows_are_the_decode_of_their_prefix():
    """The last row of a chunk and the decode of the same sequence agree within both bounds."""
    c = Cache(8, 128, [1000], seed=3).cuda()
    q = randn((1, 32, 128), 5).cuda()
    a = f64(run_decode(c, q, 128 ** -0.5))
    b = f64(run_prefill(c, q, torch.tensor([0, 1], dtype=torch.int32).cuda(), 1, 128 ** -0.5))
    assert np.abs(a - b).max() <= 2 * 2.0 ** -8 * np.abs(a).max()


def test_bad_block_ids_are_reported_and_read_as_block_0():
    for d, hq in ((128, 8), (64, 8), (256, 8)):
        c = Cache(2, d, [100, 60], seed=2).cuda()
        c.gt[0, 2] = c.nb
        c.gt[1, 1] = -7
        c.gks[0], c.gvs[0] = 0.01, 0.01            # block 0 may be one that no sequence owns
        c.gk[0], c.gv[0] = 0x30, 0x30
        ws = fk.alloc_workspace(2, hq, 2, d, 100)
        out = run_decode(c, randn((2, hq, d), 1).cuda(), 0.1, ws=ws)
        torch.cuda.synchronize()
        assert fk.fp8kv_read_error(ws) == 1 and torch.isfinite(out).all()
        for counts in ([3, 2], [90, 60]):
            ws = fk.alloc_prefill_workspace(2, max(counts), 100, hq, 2, d)
            starts = torch.tensor([0, counts[0], sum(counts)], dtype=torch.int32).cuda()
            out = run_prefill(c, randn((sum(counts), hq, d), 1).cuda(), starts, max(counts), 0.1, ws=ws)
            torch.cuda.synchronize()
            assert fk.fp8kv_read_error(ws) == 1 and torch.isfinite(out).all()


def test_captured_and_replayed_on_another_stream():
    c = Cache(8, 128, [300, 77, 0], seed=9).cuda()
    q = randn((3, 32, 128), 1).cuda()
    starts = torch.tensor([0, 40, 45, 45], dtype=torch.int32).cuda()
    qp = randn((45, 32, 128), 2).cuda()
    ws = fk.alloc_workspace(3, 32, 8, 128, 300)
    wsp = fk.alloc_prefill_workspace(3, 40, 300, 32, 8, 128)
    out, outp = torch.zeros_like(q), torch.zeros_like(qp)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        run_decode(c, q, 0.1, ws=ws, out=out)
        run_prefill(c, qp, starts, 40, 0.1, ws=wsp, out=outp)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        run_decode(c, q, 0.1, ws=ws, out=out)
        run_prefill(c, qp, starts, 40, 0.1, ws=wsp, out=outp)
    q.copy_(randn((3, 32, 128), 3))
    qp.copy_(randn((45, 32, 128), 4))
    c.gvs *= 2                                    # the scales are read at replay
    c.pull()
    for _ in range(3):
        out.zero_(), outp.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check_rows(f64(out[:1]), c, 0, f64(q[:1]), [299], 0.1, 0, False)
        check_rows(f64(out[1:2]), c, 1, f64(q[1:2]), [76], 0.1, 0, False)
        assert not out[2].any()
        check_rows(f64(outp[:40]), c, 0, f64(qp[:40]), list(range(260, 300)), 0.1, 0, True)
        check_rows(f64(outp[40:]), c, 1, f64(qp[40:]), list(range(72, 77)), 0.1, 0, True)
    assert fk.fp8kv_read_error(ws) == 0 and fk.fp8kv_read_error(wsp) == 0


def test_cache_offsets_past_32_bits():
    """Pages behind the first 4 GiB of each cache."""
    hq, hkv, d = 32, 8, 128
    small = Cache(hkv, d, [100, 40], seed=3)
    nb = (1 << 32) // (hkv * 16 * d) + 64
    shift = nb - small.nb
    big_k = torch.empty((nb, hkv, 16, d), dtype=torch.uint8, device="cuda")
    big_v = torch.empty_like(big_k)
    ks, vs = (torch.full((nb, hkv), float("nan"), device="cuda") for _ in range(2))
    small.cuda()
    big_k[shift:], big_v[shift:], ks[shift:], vs[shift:] = small.gk, small.gv, small.gks, small.gvs
    q = randn((2, hq, d), 1)
    qp, starts = randn((30, hq, d), 2), torch.tensor([0, 20, 30], dtype=torch.int32).cuda()
    small.gk, small.gv, small.gks, small.gvs = big_k, big_v, ks, vs
    small.gt = torch.from_numpy(np.where(small.tables < small.nb, small.tables + shift, 0).astype(np.int32)).cuda()
    out = f64(run_decode(small, q.cuda(), 0.1))
    outp = f64(run_prefill(small, qp.cuda(), starts, 20, 0.1))
    for b, L in enumerate(small.lens):
        check_rows(out[b:b + 1], small, b, f64(q[b:b + 1]), [L - 1], 0.1, 0, False)
    check_rows(outp[:20], small, 0, f64(qp[:20]), list(range(80, 100)), 0.1, 0, True)
    check_rows(outp[20:], small, 1, f64(qp[20:]), list(range(30, 40)), 0.1, 0, True)


@pytest.mark.parametrize("L,stage", [(1500, 0), (20000, 1)])   # CTA 0's part of 1500 keys is one stage
@pytest.mark.parametrize("hq,hkv,d,n", [(8, 2, 128, 5), (8, 2, 128, 30), (8, 2, 64, 8), (8, 1, 256, 60),
                                        (16, 2, 128, 100)])
def test_a_wait_that_runs_out_is_reported_and_ends_the_call(hq, hkv, d, n, L, stage):
    """One stage's scores never arrive: every role gives up, and after fp8kv_workspace_init the call is right again."""
    c = Cache(hkv, d, [L], seed=4).cuda()
    q = randn((n, hq, d), 1).cuda()
    starts = torch.tensor([0, n], dtype=torch.int32).cuda()
    ws = fk.alloc_prefill_workspace(1, n, L, hq, hkv, d)
    out = torch.full_like(q, 7.0)
    assert fk.debug_paged_prefill_block_stall(q, c.gk, c.gv, c.gks, c.gvs, c.gt, c.gl, starts, n, L, 0.1, 0, out, ws,
                                              stage, 2_000_000) == 0
    torch.cuda.synchronize()
    assert fk.fp8kv_read_error(ws) == 5
    fk.fp8kv_workspace_init(ws)
    run_prefill(c, q, starts, n, 0.1, ws=ws, out=out)
    torch.cuda.synchronize()
    assert fk.fp8kv_read_error(ws) == 0
    check_rows(f64(out), c, 0, f64(q), list(range(L - n, L)), 0.1, 0, True)


@pytest.mark.parametrize("hq,hkv,d,n", [(4, 1, 128, 8), (4, 1, 128, 16), (4, 1, 128, 17), (4, 1, 128, 32), (4, 1, 128, 33),
                                        (8, 1, 64, 4), (8, 1, 64, 8), (8, 1, 64, 16), (8, 1, 64, 17), (8, 1, 256, 8),
                                        (8, 1, 256, 9), (8, 1, 256, 16), (16, 1, 256, 40), (2, 2, 64, 1)])
def test_short_chunks_at_the_borders_of_their_copies(hq, hkv, d, n):
    """Chunks of exactly and just over a quarter, a half and the whole of a query tile, over ranges that end inside a
    stage, a granule and a page."""
    for L, window in ((n, 0), (n + 1, 0), (190, 0), (257, 20), (1027, 0), (2100, 1000)):
        if L < n:
            continue
        c = Cache(hkv, d, [L, n + 3], seed=L + n).cuda()
        _prefill_case(c, hq, [n, max(1, n - 1)], d ** -0.5, window, 7)


def test_rescaled_rows_of_a_short_chunk():
    """Scores that grow along the sequence, so that every stage moves the running maximum by far more than the lazy
    threshold; and scores that fall, so that none does."""
    for hq, hkv, d, n in ((4, 1, 128, 5), (4, 1, 128, 20), (8, 1, 64, 3), (8, 1, 256, 6), (8, 1, 256, 60)):
        for up in (True, False):
            c = Cache(hkv, d, [900], seed=3, spread=0.0)
            for p in range(-(-900 // 16)):
                c.ks[c.tables[0, p]] *= 0.5 * (p + 1) if up else 0.5 * (57 - p)
            c.k = (c.k & 0x7F).astype(np.uint8)            # all keys positive: a score's size follows its page's scale
            c.cuda()
            starts = torch.tensor([0, n], dtype=torch.int32).cuda()
            q = randn((n, hq, d), 5).abs()
            out = f64(run_prefill(c, q.cuda(), starts, n, d ** -0.5))
            check_rows(out, c, 0, f64(q), list(range(900 - n, 900)), d ** -0.5, 0, True, (d, n, up))


@pytest.mark.parametrize("hq,hkv,d,n", [(4, 1, 128, 7), (4, 1, 128, 25), (4, 2, 128, 200), (8, 1, 64, 40), (4, 1, 256, 70)])
@pytest.mark.parametrize("window", [0, 60])
def test_nan_keys_stay_out_of_the_rows_that_do_not_attend_them(hq, hkv, d, n, window):
    """A key of NaN codes inside a chunk: the rows before it, and those whose window has passed it, come out as they
    do without it; the rows that attend it are NaN."""
    L, t = 400, 400 - n // 2
    c = Cache(hkv, d, [L], seed=d + n).cuda()
    q = randn((n, hq, d), 4)
    starts = torch.tensor([0, n], dtype=torch.int32).cuda()
    c.gk[int(c.tables[0, t // 16]), :, t % 16] = 0x7F
    out = f64(run_prefill(c, q.cuda(), starts, n, 0.1, window))
    dec = f64(run_decode(c, q[-1:].cuda(), 0.1, window))
    attends = [t <= p and (window == 0 or p - t < window) for p in range(L - n, L)]
    for i, (p, hit) in enumerate(zip(range(L - n, L), attends)):
        if hit:
            assert np.isnan(out[i]).all()
        else:
            check_rows(out[i:i + 1], c, 0, f64(q[i:i + 1]), [p], 0.1, window, True, p)
    assert np.isnan(dec).all() == attends[-1]


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (16, 2, 64), (4, 1, 256)])
@pytest.mark.parametrize("counts", [[3, 1], [90, 40]])
def test_prefill_leaves_rows_that_no_sequence_has(hq, hkv, d, counts):
    """Rows of q before the first sequence and behind the last: out keeps what it held."""
    c = Cache(hkv, d, [300, 40], seed=d).cuda()
    first, T = 5, 5 + sum(counts) + 9
    q = randn((T, hq, d), 3)
    starts = torch.tensor([first, first + counts[0], first + sum(counts)], dtype=torch.int32).cuda()
    out = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    out = f64(run_prefill(c, q.cuda(), starts, max(counts), 0.1, out=out))
    assert (out[:first] == 7).all() and (out[first + sum(counts):] == 7).all()
    at = first
    for b, n in enumerate(counts):
        check_rows(out[at:at + n], c, b, f64(q[at:at + n]), list(range(c.lens[b] - n, c.lens[b])), 0.1, 0, True, b)
        at += n


@pytest.mark.parametrize("hq,hkv,d,n", [(4, 1, 128, 70), (8, 1, 64, 40), (1, 1, 128, 300), (16, 1, 64, 17)])
@pytest.mark.parametrize("window", [0, 100])
def test_rescaled_rows_of_a_long_chunk(hq, hkv, d, n, window):
    """The same for chunks of several query tiles: scores that grow from page to page move the maximum in both halves
    of every stage, behind value products that are on their way."""
    for grow in (lambda p: 0.5 * (p + 1), lambda p: 0.5 * (57 - p), lambda p: 8.0 if p % 8 == 5 else 0.25 + 0.1 * p):
        c = Cache(hkv, d, [900], seed=3, spread=0.0)
        for p in range(-(-900 // 16)):
            c.ks[c.tables[0, p]] *= grow(p)
        c.k = (c.k & 0x7F).astype(np.uint8)
        c.cuda()
        starts = torch.tensor([0, n], dtype=torch.int32).cuda()
        q = randn((n, hq, d), 5).abs()
        out = f64(run_prefill(c, q.cuda(), starts, n, d ** -0.5, window))
        check_rows(out, c, 0, f64(q), list(range(900 - n, 900)), d ** -0.5, window, True, (d, n))


@pytest.mark.parametrize("hq,hkv,d,lens,counts,window", [
    (32, 8, 128, [900, 300, 257, 1500, 700], [300, 0, 257, 64, 460], 200),      # pairs of tiles: 20 of 8 heads
    (16, 8, 128, [300 + 7 * i for i in range(40)], [i % 9 for i in range(40)], 0),   # short chunks, some of no row
    (2, 1, 128, [300] * 153, [1] * 153, 0),
])
def test_prefill_of_more_units_than_a_wave(hq, hkv, d, lens, counts, window):
    c = Cache(hkv, d, lens, seed=len(lens)).cuda()
    _prefill_case(c, hq, counts, d ** -0.5, window, 3)


def test_lengths_out_of_bounds_are_reported_and_leave_the_others():
    hq, hkv, d = 32, 8, 128
    c = Cache(hkv, d, [300, 250, 200], seed=1).cuda()
    counts = (200, 150, 100)
    q = randn((450, hq, d), 2)
    starts = torch.tensor([0, 200, 350, 450], dtype=torch.int32).cuda()
    for bad, length in ((0, 301), (1, 149), (2, -1)):       # past the bound, fewer keys than new tokens, negative
        ws = fk.alloc_prefill_workspace(3, 200, 300, hq, hkv, d)
        lens = [300, 250, 200]
        lens[bad] = length
        c.gl.copy_(torch.tensor(lens, dtype=torch.int32))
        out = f64(run_prefill(c, q.cuda(), starts, 200, 0.1, max_len=300, ws=ws))
        assert fk.fp8kv_read_error(ws) == 1
        for b, n in enumerate(counts):
            if b != bad:
                L = c.lens[b]
                rows = slice(int(starts[b]), int(starts[b + 1]))
                check_rows(out[rows], c, b, f64(q[rows]), list(range(L - n, L)), 0.1, 0, True, (bad, b))


def test_one_workspace_shared_by_captured_calls_of_different_shapes():
    """Calls of different shapes that share one workspace, captured into one graph and replayed."""
    hq, hkv, d = 32, 8, 128
    c = Cache(hkv, d, [700, 600], seed=5).cuda()
    qa, qb = randn((1100, hq, d), 1), randn((700, hq, d), 2)
    sa, sb = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, 600, 1100], [0, 300, 700]))
    ws = fk.alloc_prefill_workspace(2, 600, 700, hq, hkv, d)
    outs = [torch.zeros_like(x).cuda() for x in (qa, qb)]
    ga, gb = qa.cuda(), qb.cuda()

    def call():
        run_prefill(c, ga, sa, 600, 0.1, ws=ws, out=outs[0])
        run_prefill(c, gb, sb, 400, 0.1, ws=ws, out=outs[1])
    call()
    torch.cuda.synchronize()
    want = [x.clone() for x in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for x in outs:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))
    out = f64(outs[1])
    check_rows(out[:300], c, 0, f64(qb[:300]), list(range(400, 700)), 0.1, 0, True)
    check_rows(out[300:], c, 1, f64(qb[300:]), list(range(200, 600)), 0.1, 0, True)
    assert fk.fp8kv_read_error(ws) == 0

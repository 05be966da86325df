"""GPU tests of calls that follow one another on a stream with nothing between: each may be resident while the one
before still writes what it reads (queries, page scales, pages)."""
import pytest
import torch

from fp8_kv_cache_fp8kv_gb300 import binding as fk
from tests.block_harness import Cache, randn, run_decode, run_prefill

pytestmark = pytest.mark.gpu

STEPS = 24


def _same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def _run(step, state, sync, graph):
    """The steps from a fresh `state`, one after the other or with a synchronisation behind every call."""
    def pause():
        if sync:
            torch.cuda.synchronize()
    for s in range(2):                     # (the first time sets the kernels up)
        st = state()
        torch.cuda.synchronize()
        if graph and s:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                for i in range(STEPS):
                    step(st, i, pause)
            g.replay()
        else:
            for i in range(STEPS):
                step(st, i, pause)
        torch.cuda.synchronize()
    return st


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 1, 64), (8, 2, 256)])
def test_attend_append_attend_over_page_scales(hq, hkv, d, graph):
    """Decode, prefill, append, and again: every append makes its page's scales grow and rewrites the queries, so that
    attention with what was there before would differ."""
    B, L = 3, 70
    data = [randn((B, hq + 2 * hkv, d), 10 + i, 1.5 ** i).cuda() for i in range(STEPS)]
    freq = torch.tensor([10000.0 ** (-i / (d // 2)) for i in range(d // 2)]).cuda()
    lens = [torch.tensor([L + i + 1 + b for b in range(B)], dtype=torch.int32).cuda() for i in range(STEPS)]
    starts = torch.arange(B + 1, dtype=torch.int32).cuda()
    mx = L + STEPS + B

    def state():
        c = Cache(hkv, d, [L + b for b in range(B)], seed=d, capacity=[mx] * B, scale=0.001).cuda()
        c.lens = [mx] * B
        c.out = torch.zeros((STEPS, 4, B, hq, d), dtype=torch.bfloat16, device="cuda")
        c.qo = torch.zeros((B, hq, d), dtype=torch.bfloat16, device="cuda")
        c.ws = [fk.alloc_workspace(B, hq, hkv, d, mx), fk.alloc_prefill_workspace(B, 1, mx, hq, hkv, d)]
        return c

    def step(c, i, pause):
        q, k, v = data[i].split((hq, hkv, hkv), 1)
        c.gl = lens[i - 1] if i else lens[0] - 1
        for j in range(2):
            run_decode(c, c.qo, 0.1, 0, mx, c.ws[0], c.out[i, 2 * j])
            pause()
            run_prefill(c, c.qo, starts, 1, 0.1, 0, mx, c.ws[1], c.out[i, 2 * j + 1])
            pause()
            if j == 0:
                c.gl = lens[i]
                fk.fp8kv_rope_append_block(q, k, v, None, freq, c.qo, c.gk, c.gv, c.gks, c.gvs, c.gt, c.gl, None, mx,
                                           c.ws[0])
                pause()

    want, got = _run(step, state, True, False), _run(step, state, False, graph)
    assert not torch.equal(want.out[:, 0], want.out[:, 2]) and torch.isfinite(want.out).all()
    for a, b in ((want.out, got.out), (want.gk, got.gk), (want.gv, got.gv), (want.gks, got.gks), (want.gvs, got.gvs)):
        assert _same(a, b)
    assert all(fk.fp8kv_read_error(w) == 0 for w in got.ws)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 1, 64), (8, 2, 256)])
def test_attend_append_attend_over_one_scale(hq, hkv, d, graph):
    """The same over a cache with one scale per tensor: rope append, decode, prefill of one and of several tiles."""
    n, L = 129, 300
    data = [randn((n, hq + 2 * hkv, d), 10 + i).cuda() for i in range(STEPS)]
    freq = torch.tensor([10000.0 ** (-i / (d // 2)) for i in range(d // 2)]).cuda()
    pos = torch.arange(L - n, L, dtype=torch.int32).cuda()
    slots = torch.arange(L - n, L).cuda()
    nb = -(-L // 16)
    tables = torch.arange(nb, dtype=torch.int32)[None].cuda()
    one, lens = torch.tensor([0, 1], dtype=torch.int32).cuda(), torch.tensor([L], dtype=torch.int32).cuda()
    many = torch.tensor([0, n], dtype=torch.int32).cuda()

    class State:
        def __init__(self):
            self.k, self.v = (torch.zeros((nb, hkv, 16, d), dtype=torch.uint8, device="cuda") for _ in range(2))
            self.qo = torch.zeros((n, hq, d), dtype=torch.bfloat16, device="cuda")
            self.dec = torch.zeros((STEPS, 2, 1, hq, d), dtype=torch.bfloat16, device="cuda")
            self.pre = torch.zeros((STEPS, n, hq, d), dtype=torch.bfloat16, device="cuda")
            self.ws = [fk.alloc_workspace(1, hq, hkv, d, L), fk.alloc_prefill_workspace(1, n, L, hq, hkv, d)]

    def step(s, i, pause):
        q, k, v = data[i].split((hq, hkv, hkv), 1)
        fk.fp8kv_rope_append(q, k, v, pos, freq, slots, s.qo, s.k, s.v, 0.01, 0.01)
        pause()
        fk.fp8kv_paged_decode(s.qo[-1:], s.k, s.v, tables, lens, L, 0.01, 0.01, 0.1, 0, s.dec[i, 0], s.ws[0])
        pause()
        fk.fp8kv_paged_prefill(s.qo, s.k, s.v, tables, lens, many, n, L, 0.01, 0.01, 0.1, 0, s.pre[i], s.ws[1])
        pause()
        fk.fp8kv_rope_append(q, k, v, pos, freq, slots, s.qo, s.k, s.v, 0.01, 0.01)
        pause()
        fk.fp8kv_paged_prefill(s.qo[-1:], s.k, s.v, tables, lens, one, 1, L, 0.01, 0.01, 0.1, 0, s.dec[i, 1], s.ws[1])
        pause()

    want, got = _run(step, State, True, False), _run(step, State, False, graph)
    assert torch.isfinite(want.pre).all() and not torch.equal(want.pre[0], want.pre[1])
    for a, b in ((want.dec, got.dec), (want.pre, got.pre), (want.k, got.k), (want.v, got.v)):
        assert _same(a, b)
    assert all(fk.fp8kv_read_error(w) == 0 for w in got.ws)

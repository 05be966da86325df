"""Drafted trees, commits, attention weights and eviction as a serving loop uses them, next to the calls that were
there: appended, attended, committed, decoded and cut back, step after step, eagerly and as a replayed graph."""
import math

import pytest
import torch

from fp8_kv_cache_fp8kv_gb300 import binding as fk
from tests.spec_harness import PAGE, Cache, attend, attended, depths, queries, random_tree, rng, run_tree

pytestmark = pytest.mark.gpu
E = 2.0 ** -9                                  # of sum_t p_t |v_t|; see test_gpu_tree.py


def rope(x, pos, inv):
    """The rotation by halves, in 64 bits."""
    a = pos.double()[:, None] * inv.double()
    c, s = a.cos()[:, None], a.sin()[:, None]
    h = x.shape[-1] // 2
    x = x.double()
    return torch.cat((x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s), -1)


def test_serving_loop():
    """Three rounds of draft, check and commit on two sequences, a decode step that adds up weights, an eviction, and
    a decode over what it left: each step against 64-bit attention over the rows that should be there."""
    hq, hkv, d, r = 8, 2, 128, rng(1)
    lens = [200, 77]
    c = Cache(lens, hkv, d, "e4m3", 3, room=120)
    inv = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    mirror = {(w, b, h): c.rows(w, b, h) for w in "kv" for b in range(2) for h in range(hkv)}
    commit_ws = fk.alloc_append_workspace()
    new_lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    for step in range(3):
        trees = [random_tree(12, r), random_tree(9, r)]
        dep = [depths(t) for t in trees]
        q, k, v = queries(21, hq, d, 10 + step), queries(21, hkv, d, 20 + step), queries(21, hkv, d, 30 + step)
        pos = torch.tensor([lens[b] + x for b in range(2) for x in dep[b]], dtype=torch.int32, device="cuda")
        place = [(b, lens[b] + i) for b in range(2) for i in range(len(trees[b]))]
        slots = torch.tensor([int(c.tables[b, p // PAGE]) * PAGE + p % PAGE for b, p in place], device="cuda")
        qr = torch.empty_like(q)
        fk.fp8kv_rope_append(q, k, v, pos, inv, slots, qr, c.k, c.v, *c.scale)
        c.seq_lens = torch.tensor([lens[0] + 12, lens[1] + 9], dtype=torch.int32, device="cuda")
        c.max_len = int(c.seq_lens.max())
        out, err = run_tree(c, qr, trees)
        assert err == 0
        start = [0, 12]
        for b, tree in enumerate(trees):
            n = len(tree)
            for h in range(hkv):
                rows = slice(start[b], start[b] + n)
                ks = torch.cat((mirror["k", b, h], c.rows("k", b, h, lens[b] + n)[lens[b]:]))
                vs = torch.cat((mirror["v", b, h], c.rows("v", b, h, lens[b] + n)[lens[b]:]))
                # what was appended is the rotated key, within its rounding to E4M3 (2^-4, or the least step)
                exact = rope(k[rows, h:h + 1].float(), pos[rows], inv)[:, 0]
                assert ((ks[lens[b]:] - exact).abs() <= 2.0 ** -4 * exact.abs() + c.scale[0] * 2.0 ** -9).all()
                heads = slice(4 * h, 4 * h + 4)
                ref, mass, _ = attend(qr[rows, heads], ks, vs, attended(tree, lens[b], 0), 1 / math.sqrt(d))
                assert ((out[rows, heads].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + E * mass + 1e-6).all()
        # a path from the root to the deepest node
        paths = []
        for b, tree in enumerate(trees):
            i, path = dep[b].index(max(dep[b])), []
            while i >= 0:
                path.append(i)
                i = tree[i]
            paths.append(path[::-1])
        for b, path in enumerate(paths):
            for h in range(hkv):
                for w in "kv":
                    rows = c.rows(w, b, h, lens[b] + len(trees[b]))[lens[b]:]
                    mirror[w, b, h] = torch.cat((mirror[w, b, h], rows[path]))
        acc = torch.full((2, 12), -1, dtype=torch.int32)
        for b, path in enumerate(paths):
            acc[b, : len(path)] = torch.tensor(path)
        fk.fp8kv_tree_commit(c.k, c.v, c.tables, c.seq_lens, torch.tensor([0, 12, 21], dtype=torch.int32, device="cuda"),
                             acc.cuda(), c.max_len, new_lens, commit_ws)
        lens = [lens[b] + len(paths[b]) for b in range(2)]
        assert new_lens.tolist() == lens
        for key, rows in mirror.items():
            assert torch.equal(c.rows(*key, n=lens[key[1]]), rows)
    # decode steps that keep account, then an eviction by it
    c.seq_lens, c.max_len, c.lens = new_lens.clone(), max(lens), lens
    w = torch.zeros((c.blocks, hkv, PAGE), device="cuda")
    ws = fk.alloc_weights_workspace(2, hq, hkv, d, c.max_len)
    total = {(b, h): torch.zeros(lens[b], dtype=torch.float64, device="cuda") for b in range(2) for h in range(hkv)}
    for step in range(4):
        q = queries(2, hq, d, 50 + step)
        out = torch.empty_like(q)
        fk.fp8kv_paged_decode_weights(q, c.k, c.v, c.tables, c.seq_lens, c.max_len, 1 / math.sqrt(d), 0, out, w, 1.0, ws,
                                      **c.kind_args())
        for b in range(2):
            for h in range(hkv):
                seen = torch.ones((1, lens[b]), dtype=torch.bool)
                heads = slice(4 * h, 4 * h + 4)
                ref, mass, p = attend(q[b:b + 1, heads], mirror["k", b, h], mirror["v", b, h], seen, 1 / math.sqrt(d))
                assert ((out[b, heads].double() - ref[0]).abs() <= 2.0 ** -8 * ref[0].abs() + E * mass[0] + 1e-6).all()
                total[b, h][-1] = 0
                total[b, h] += p.sum(0)[0]
    budget, sinks, recent = 60, 4, 16
    kept = torch.zeros((2, hkv, budget), dtype=torch.int32, device="cuda")
    fk.fp8kv_evict(c.k, c.v, w, c.tables, c.seq_lens, c.max_len, budget, sinks, recent, new_lens, commit_ws, kept=kept)
    assert new_lens.tolist() == [budget, budget] and fk.fp8kv_read_error(commit_ws) == 0
    for (b, h), t in total.items():
        at = kept[b, h].long()
        assert (at.diff() > 0).all() and at[:sinks].tolist() == list(range(sinks))
        assert at[-recent:].tolist() == list(range(lens[b] - recent, lens[b]))
        out_of = torch.ones(lens[b], dtype=torch.bool, device="cuda")
        out_of[at] = False
        # the 64-bit weights agree with the choice up to what the kept account may be off by (2^-11)
        assert t[at[sinks:-recent]].min() >= t[out_of].max() * (1 - 2.0 ** -10)
        for x in "kv":
            assert torch.equal(c.rows(x, b, h, n=budget), mirror[x, b, h][at])
    c.lens, c.seq_lens, c.max_len = [budget, budget], new_lens.clone(), budget
    q = queries(2, hq, d, 70)
    out, err = run_tree(c, q, [[-1], [-1]])                 # one node: a decode step
    assert err == 0
    for (b, h) in total:
        heads = slice(4 * h, 4 * h + 4)
        at = kept[b, h].long()
        ref, mass, _ = attend(q[b:b + 1, heads], mirror["k", b, h][at], mirror["v", b, h][at],
                              torch.ones((1, budget), dtype=torch.bool), 1 / math.sqrt(d))
        assert ((out[b, heads].double() - ref[0]).abs() <= 2.0 ** -8 * ref[0].abs() + E * mass[0] + 1e-6).all()


def _setup(seed):
    hq, hkv, d = 16, 4, 128
    c = Cache([900, 333, 20], hkv, d, "e4m3", seed)
    trees = [random_tree(30, rng(seed)), random_tree(7, rng(seed + 1)), random_tree(20, rng(seed + 2))]
    q, q1 = queries(57, hq, d, seed), queries(3, hq, d, seed + 1)
    starts = torch.tensor([0, 30, 37, 57], dtype=torch.int32, device="cuda")
    flat = torch.tensor(sum(trees, []), dtype=torch.int32, device="cuda")
    acc = torch.tensor([[0, 3, 9, 21], [0, 6, -1, -1], [0, 1, 2, 19]], dtype=torch.int32, device="cuda")
    s = dict(c=c, q=q, q1=q1, starts=starts, flat=flat, acc=acc, out=torch.empty_like(q), out1=torch.empty_like(q1),
             w=torch.rand((c.blocks, hkv, PAGE), generator=torch.Generator().manual_seed(seed)).cuda(),
             lens=torch.zeros(3, dtype=torch.int32, device="cuda"), lens2=torch.zeros(3, dtype=torch.int32, device="cuda"),
             kept=torch.zeros((3, hkv, 100), dtype=torch.int32, device="cuda"),
             tree_ws=fk.alloc_tree_workspace(3, 30, 900, hq, hkv, d), dec_ws=fk.alloc_weights_workspace(3, hq, hkv, d, 900),
             ws=fk.alloc_append_workspace())
    torch.cuda.synchronize()
    return s


def _step(s, stream=None):
    """Check a tree, commit its path, decode over the committed lengths with account, cut back: one chain on a stream."""
    c = s["c"]
    fk.fp8kv_paged_tree_attention(s["q"], c.k, c.v, c.tables, c.seq_lens, s["starts"], s["flat"], 30, 900, 0.09, 0, s["out"],
                                  s["tree_ws"], stream=stream, **c.kind_args())
    fk.fp8kv_tree_commit(c.k, c.v, c.tables, c.seq_lens, s["starts"], s["acc"], 900, s["lens"], s["ws"], stream=stream)
    fk.fp8kv_paged_decode_weights(s["q1"], c.k, c.v, c.tables, s["lens"], 900, 0.09, 0, s["out1"], s["w"], 0.9, s["dec_ws"],
                                  stream=stream, **c.kind_args())
    fk.fp8kv_evict(c.k, c.v, s["w"], c.tables, s["lens"], 900, 100, 4, 10, s["lens2"], s["ws"], kept=s["kept"], stream=stream)


def _state(s):
    return [s[n].clone() for n in ("out", "out1", "w", "lens", "lens2", "kept")] + [s["c"].k.clone(), s["c"].v.clone()]


def same(a, b):
    for x, y in zip(a, b):
        v = torch.int16 if x.dtype == torch.bfloat16 else torch.int32 if x.dtype == torch.float32 else x.dtype
        assert torch.equal(x.view(v), y.view(v))


def test_graph_replays_what_the_calls_do():
    eager = _setup(5)
    _step(eager)
    _step(eager)
    torch.cuda.synchronize()
    s = _setup(5)
    side = torch.cuda.Stream()
    _setup_other = _setup(6)
    with torch.cuda.stream(side):
        _step(_setup_other, side)               # attributes set before any capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(s)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    same(_state(s), _state(eager))
    assert all(fk.fp8kv_read_error(s[n]) == 0 for n in ("tree_ws", "dec_ws", "ws"))


def test_two_streams_at_once():
    alone = [_setup(7), _setup(8)]
    for s in alone:
        for _ in range(5):
            _step(s)
    torch.cuda.synchronize()
    both = [_setup(7), _setup(8)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, st in zip(both, streams):
            _step(s, st)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        same(_state(a), _state(b))


def test_back_to_back_without_a_pause():
    """Calls that may be resident before the one in front has finished see what it wrote."""
    s = _setup(9)
    for _ in range(20):
        _step(s)
    torch.cuda.synchronize()
    t = _setup(9)
    for _ in range(20):
        _step(t)
        torch.cuda.synchronize()
    same(_state(s), _state(t))

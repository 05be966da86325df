"""fp8kv_tree_commit and fp8kv_evict against their definitions, bit for bit: they move rows and choose by comparing."""
import math

import pytest
import torch

from fp8_kv_cache_fp8kv_gb300 import binding as fk
from tests.spec_harness import PAGE, Cache, rng

pytestmark = pytest.mark.gpu


def bits(x):
    return x.view(torch.int16) if x.dtype == torch.bfloat16 else x.view(torch.int32) if x.dtype == torch.float32 else x


def moved(x, table, h, source, target):
    """x [blocks, Hkv, 16, ...] with head h's rows at places `source` of a sequence copied to `target`, all at once."""
    t = table.long()
    source, target = torch.tensor(source, dtype=torch.int64), torch.tensor(target, dtype=torch.int64)
    x[t[target // PAGE], h, target % PAGE] = x[t[source // PAGE], h, source % PAGE].clone()


def commit(c, counts, accepted, max_len=None):
    dev = "cuda"
    starts = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).to(dev)
    acc = torch.tensor(accepted, dtype=torch.int32, device=dev)
    new = torch.full((len(counts),), -5, dtype=torch.int32, device=dev)
    ws = fk.alloc_append_workspace()
    fk.fp8kv_tree_commit(c.k, c.v, c.tables, c.seq_lens, starts, acc, c.max_len if max_len is None else max_len, new, ws)
    torch.cuda.synchronize()
    return new, fk.fp8kv_read_error(ws)


def check_commit(lens, nodes, hkv, d, fmt, paths, seed=0):
    c = Cache([n + m for n, m in zip(lens, nodes)], hkv, d, fmt, seed)
    k, v = c.k.cpu().clone(), c.v.cpu().clone()
    table = c.tables.cpu()
    width = max(1, max(len(p) for p in paths))
    new, err = commit(c, nodes, [p + [-1] * (width - len(p)) for p in paths])
    assert err == 0
    assert new.tolist() == [n + len(p) for n, p in zip(lens, paths)]
    for b, p in enumerate(paths):
        for h in range(hkv):
            for x in (k, v):
                moved(x, table[b], h, [lens[b] + i for i in p], [lens[b] + i for i in range(len(p))])
    assert torch.equal(bits(c.k.cpu()), bits(k)) and torch.equal(bits(c.v.cpu()), bits(v))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("context", [0, 13, 300])
def test_commit(d, fmt, context):
    r = rng(d + context)
    nodes = [1, 7, 64, 256, 5, 0]
    paths = [sorted(r.sample(range(n), r.randint(0, n))) for n in nodes]
    paths[4] = [0, 1, 2, 3, 4]                # the path that moves nothing
    check_commit([context, context + 1, context + 9, context, 3, 4], nodes, 3, d, fmt, paths, seed=d)


def test_commit_whole_and_last_rows():
    check_commit([5, 5, 5], [256, 256, 33], 1, 128, "e4m3", [list(range(256)), list(range(1, 256)), [32]])
    check_commit([5], [40], 2, 64, "e4m3", [[]])


def test_commit_ends_a_bad_path_and_reports():
    for path, good in (([0, 3, 3, 4], 2), ([2, 1, 5, 6], 1), ([4, 6, 8, 9], 2), ([9, -1, 3, 4], 0), ([8, 1, 2, 3], 0)):
        c = Cache([20 + 8], 1, 64)
        k = c.k.cpu().clone()
        new, err = commit(c, [8], [path])
        assert new.tolist() == [20 + good] and err == 1, path
        moved(k, c.tables.cpu()[0], 0, [20 + i for i in path[:good]], [20 + i for i in range(good)])
        assert torch.equal(c.k.cpu(), k)
    c = Cache([20 + 8], 1, 64)
    new, err = commit(c, [8], [[1, 5, -9, 7]])          # any negative entry ends a path
    assert new.tolist() == [22] and err == 0


def test_commit_bad_blocks_and_lengths():
    c = Cache([40, 40], 2, 128)
    good = c.tables.clone()
    c.tables[0, 2] = 10 ** 6                              # tokens 32..39: sources and targets of sequence 0
    k = c.k.cpu().clone()
    new, err = commit(c, [4, 4], [[1, 2, 3], [1, 2, 3]])
    assert err == 1 and new.tolist() == [39, 39]
    for h in range(2):
        moved(k, good.cpu()[1], h, [37, 38, 39], [36, 37, 38])
    assert torch.equal(c.k.cpu(), k)
    c = Cache([40, 40], 2, 128)
    k = c.k.cpu().clone()
    new, err = commit(c, [4, 4], [[0, 1], [0, 1]], max_len=30)   # longer than the bound: clamped, and reported
    assert err == 1 and new.tolist() == [28, 28] and torch.equal(c.k.cpu(), k)


# ------------------------------------------------------------------ eviction

def choose(w, n, budget, sinks, recent):
    """The kept places of one head's weights [n], by sorting."""
    if n <= budget:
        return list(range(n))
    free = list(range(sinks, n - recent))
    value = [(-math.inf, 0) if math.isnan(w[t]) else (w[t], 1) for t in free]
    order = sorted(range(len(free)), key=lambda i: (-value[i][0] if value[i][1] else math.inf, -value[i][1], free[i]))
    take = [free[i] for i in order[: budget - sinks - recent]]
    return sorted(list(range(sinks)) + take + list(range(n - recent, n)))


def check_evict(lens, hkv, d, fmt, budget, sinks, recent, make=None, seed=0, with_kept=True, max_len=None):
    c = Cache(lens, hkv, d, fmt, seed)
    g = torch.Generator().manual_seed(seed + 7)
    w = torch.randn((c.blocks, hkv, PAGE), generator=g).exp() if make is None else make((c.blocks, hkv, PAGE), g)
    k, v, table = c.k.cpu().clone(), c.v.cpu().clone(), c.tables.cpu()
    gpu_w = w.cuda()
    w = w.clone()
    new = torch.full((len(lens),), -5, dtype=torch.int32, device="cuda")
    kept = torch.full((len(lens), hkv, budget), -9, dtype=torch.int32, device="cuda") if with_kept else None
    ws = fk.alloc_append_workspace()
    fk.fp8kv_evict(c.k, c.v, gpu_w, c.tables, c.seq_lens, c.max_len if max_len is None else max_len, budget, sinks, recent, new,
                   ws, kept=kept)
    torch.cuda.synchronize()
    assert fk.fp8kv_read_error(ws) == 0
    assert new.tolist() == [min(n, budget) for n in lens]
    for b, n in enumerate(lens):
        t = torch.arange(n)
        for h in range(hkv):
            held = w[table[b].long()[t // PAGE], h, t % PAGE].tolist()
            want = choose(held, n, budget, sinks, recent)
            if with_kept:
                got = kept[b, h].tolist()
                assert got == want + [-1] * (budget - len(want)), (b, h)
            for x in (k, v, w):
                moved(x, table[b], h, want, list(range(len(want))))
    assert torch.equal(bits(c.k.cpu()), bits(k)) and torch.equal(bits(c.v.cpu()), bits(v))
    assert torch.equal(bits(gpu_w.cpu()), bits(w))


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_evict(d, fmt):
    check_evict([500, 99, 100, 101, 0, 1, 16, 777], 2, d, fmt, 100, 4, 20, seed=d)


@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (17, 0, 0), (50, 25, 25), (50, 50, 0), (50, 0, 50),
                                                  (333, 1, 1), (399, 0, 0)])
def test_budgets(budget, sinks, recent):
    check_evict([400, 401, 33], 3, 64, "e4m3", budget, sinks, recent, seed=budget)


def ties(shape, g):
    return torch.randint(0, 3, shape, generator=g).float()


def zeros(shape, g):
    return torch.zeros(shape) * torch.where(torch.rand(shape, generator=g) < 0.5, -1.0, 1.0)    # of both signs


def odd(shape, g):
    w = torch.randn(shape, generator=g)
    r = torch.rand(shape, generator=g)
    w[r < 0.1] = math.inf
    w[(r > 0.1) & (r < 0.2)] = -math.inf
    w[(r > 0.2) & (r < 0.3)] = math.nan
    w[(r > 0.3) & (r < 0.4)] *= 1e-42                 # subnormal
    w[(r > 0.4) & (r < 0.5)] *= 1e30
    return w


def near(shape, g):
    return (1.0 + torch.randint(0, 2000, shape, generator=g) * 2.0 ** -23).float()    # the last bits decide


@pytest.mark.parametrize("make", [ties, zeros, odd, near])
@pytest.mark.parametrize("budget", [40, 300, 900])
def test_weights_that_are_hard_to_order(make, budget):
    check_evict([1000, 950, 5000], 2, 64, "e4m3", budget, 3, 17, make=make, seed=budget)


@pytest.mark.parametrize("lens,hkv,budget", [([30000], 1, 5000), ([9000, 20000], 1, 8999), ([4096] * 20, 8, 1000), ([700] * 40, 8, 65)])
def test_clusters_of_every_size(lens, hkv, budget):
    check_evict(lens, hkv, 64, "e4m3", budget, 4, 30, seed=1, with_kept=budget != 1000)


def test_largest_bound_and_short_sequences():
    """A bound of the longest supported length, over sequences that are far shorter."""
    c = Cache([600, 40], 1, 64, "e4m3", 3)
    wide = torch.full((2, 393216 // 16), -7, dtype=torch.int32, device="cuda")
    wide[:, : c.tables.shape[1]] = c.tables
    k, table = c.k.cpu().clone(), c.tables.cpu()
    w = torch.rand((c.blocks, 1, PAGE))
    new, ws = torch.zeros(2, dtype=torch.int32, device="cuda"), fk.alloc_append_workspace()
    fk.fp8kv_evict(c.k, c.v, w.cuda(), wide, c.seq_lens, 393216, 64, 0, 1, new, ws)
    torch.cuda.synchronize()
    assert fk.fp8kv_read_error(ws) == 0 and new.tolist() == [64, 40]
    t = torch.arange(600)
    want = choose(w[table[0].long()[t // PAGE], 0, t % PAGE].tolist(), 600, 64, 0, 1)
    moved(k, table[0], 0, want, list(range(64)))
    assert torch.equal(c.k.cpu(), k)
    with pytest.raises(fk.Fp8kvError):
        more = torch.cat((wide, wide[:, :1]), 1)
        fk.fp8kv_evict(c.k, c.v, w.cuda(), more, c.seq_lens, 393217, 64, 0, 1, new, ws)


def test_evict_bad_blocks_and_lengths():
    c = Cache([64, 64], 1, 64, "e4m3", 5)
    good = c.tables.cpu().clone()
    c.tables[0, 1] = -3                                   # tokens 16..31: their weights count as 0
    w = torch.rand((c.blocks, 1, PAGE)) + 1
    k, gw = c.k.cpu().clone(), w.cuda()
    new, ws = torch.zeros(2, dtype=torch.int32, device="cuda"), fk.alloc_append_workspace()
    kept = torch.zeros((2, 1, 40), dtype=torch.int32, device="cuda")
    fk.fp8kv_evict(c.k, c.v, gw, c.tables, c.seq_lens, 64, 40, 0, 0, new, ws, kept=kept)
    torch.cuda.synchronize()
    assert fk.fp8kv_read_error(ws) == 1 and new.tolist() == [40, 40]
    for b in range(2):
        t = torch.arange(64)
        held = w[good[b].long()[t // PAGE], 0, t % PAGE]
        if b == 0:
            held[16:32] = 0
        want = choose(held.tolist(), 64, 40, 0, 0)
        assert kept[b, 0].tolist() == want
        pairs = [(s, i) for i, s in enumerate(want) if b == 1 or (s // 16 != 1 and i // 16 != 1)]
        moved(k, good[b], 0, [s for s, _ in pairs], [i for _, i in pairs])
    assert torch.equal(c.k.cpu(), k)
    c = Cache([64], 1, 64, "e4m3", 5)
    fk.fp8kv_evict(c.k, c.v, torch.rand((c.blocks, 1, PAGE)).cuda(), c.tables, c.seq_lens, 60, 40, 0, 0, new[:1], ws)
    assert fk.fp8kv_read_error(ws) == 1 and new[0].item() == 40

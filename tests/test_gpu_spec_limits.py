"""What the tree attention, the path commit, the weighted decode and the eviction do at the edges of what they are given:
entries out of range (reported and replaced as documented: the call then gives what it gives with the replaced value),
rows of no sequence, caches past 2^31 and 2^32 bytes, a wait that runs out, a call on another stream."""
import math
import time

import pytest
import torch

from fp8_kv_cache_fp8kv_gb300 import binding as fk
from tests.spec_harness import PAGE, Cache, queries, random_tree, rng, run_tree

pytestmark = pytest.mark.gpu
LAYOUTS = [(32, 8, 128, "e4m3"), (8, 1, 256, "bf16"), (64, 8, 64, "e5m2")]


def trees_of(nodes, seed=0):
    r = rng(seed)
    return [random_tree(n, r, min(n, 2)) for n in nodes]


@pytest.mark.parametrize("hq,hkv,d,fmt", LAYOUTS)
def test_parents_out_of_range_are_roots(hq, hkv, d, fmt):
    c = Cache([300, 45], hkv, d, fmt)
    trees = trees_of([40, 9])
    bad, good = [list(t) for t in trees], [list(t) for t in trees]
    for b, i, p in ((0, 5, 5), (0, 17, 39), (0, 30, -2), (0, 0, 255), (1, 8, 2 ** 31 - 1), (1, 3, -2 ** 31)):
        bad[b][i], good[b][i] = p, -1
    q = queries(49, hq, d, 3)
    a, err = run_tree(c, q, bad, window=20)
    assert err == 1
    b, err = run_tree(c, q, good, window=20)
    assert err == 0 and torch.equal(a, b)


@pytest.mark.parametrize("hq,hkv,d,fmt", LAYOUTS)
def test_block_ids_out_of_range_read_block_0(hq, hkv, d, fmt):
    c = Cache([700, 100], hkv, d, fmt)
    k, v = c.k.clone(), c.v.clone()
    c.k[0], c.v[0] = k[int(c.tables[0, 0])], v[int(c.tables[0, 0])]     # numbers in every row of block 0
    trees = trees_of([20, 7])
    q = queries(27, hq, d, 3)
    good = c.tables.clone()
    c.tables[0, 3] = c.blocks
    c.tables[0, 30] = -1
    c.tables[1, 6] = 2 ** 31 - 1       # (of the newest tokens)
    good[0, 3] = good[0, 30] = good[1, 6] = 0
    a, err = run_tree(c, q, trees)
    assert err == 1
    c.tables = good
    b, err = run_tree(c, q, trees)
    assert err == 0 and torch.equal(a, b)


def test_lengths_and_starts_out_of_range_are_clamped():
    c = Cache([200, 90, 64, 300], 8, 128)
    trees = trees_of([16, 12, 8, 10])
    q = queries(46, 32, 128, 3)
    starts = torch.tensor([0, 16, 28, 36, 46], dtype=torch.int32, device="cuda")

    def both(given, clamped, max_nodes=16, max_len=300):
        outs = []
        for lens, st, code in ((given[0], given[1], 1), (clamped[0], clamped[1], 0)):
            c.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
            out, err = run_tree(c, q, trees, max_nodes=max_nodes, max_len=max_len,
                                starts=torch.tensor(st, dtype=torch.int32, device="cuda"))
            assert err == code
            outs.append(out)
        assert torch.equal(*outs)
        return outs[0]

    s = starts.tolist()
    both(([200, 90, 64, 301], s), ([200, 90, 64, 300], s))              # longer than the bound
    # more nodes than max_nodes: the first 8 of 16 and 8 of 12 are taken, as the newest tokens
    out, err = run_tree(c, q, trees, max_nodes=8, starts=starts)
    assert err == 1 and torch.all(out[8:16] == 123) and torch.all(out[24:28] == 123) and torch.all(out[44:] == 123)
    assert torch.isfinite(out).all() and not torch.any(torch.all(out[:8] == 123, -1))
    # a negative length, a negative count: no rows of theirs
    c.seq_lens = torch.tensor([200, -90, 64, 300], dtype=torch.int32, device="cuda")
    out, err = run_tree(c, q, trees, starts=starts)
    assert err == 1 and torch.all(out[16:28] == 123) and not torch.any(torch.all(out[28:] == 123, -1))
    c.seq_lens = torch.tensor([200, 90, 64, 300], dtype=torch.int32, device="cuda")
    out, err = run_tree(c, q, trees, starts=torch.tensor([0, 16, 10, 18, 28], dtype=torch.int32, device="cuda"))
    assert err == 1 and torch.all(out[28:] == 123)
    # rows that do not exist are not touched: behind the last, before the first
    for st in ([0, 16, 28, 36, 47], [-1, 16, 28, 36, 46], [0, 16, 28, 2 ** 31 - 5, 2 ** 31 - 1]):
        out, err = run_tree(c, q, trees, starts=torch.tensor(st, dtype=torch.int32, device="cuda"))
        skipped = [b for b in range(4) if st[b] < 0 or st[b] + min(16, max(0, st[b + 1] - st[b])) > 46]
        assert err == 1 and skipped
        for b in skipped:
            assert torch.all(out[s[b]:s[b + 1]] == 123) or st[b] > 46


@pytest.mark.parametrize("nodes,hq,hkv,d", [(3, 32, 8, 128), (20, 32, 8, 128), (60, 32, 8, 128), (9, 8, 1, 256), (9, 64, 8, 64)])
def test_rows_of_no_sequence_stay(nodes, hq, hkv, d):
    """Rows behind the last sequence, and sequences without nodes between others."""
    c = Cache([500, 40, 130, 0, 900], hkv, d)
    trees = trees_of([nodes, 0, nodes // 2, 0, nodes - 1])
    used = sum(len(t) for t in trees)
    q = queries(used + 5, hq, d, 3)
    out, err = run_tree(c, q, trees, max_nodes=nodes + 3)
    assert err == 0 and torch.all(out[used:] == 123) and not torch.any(torch.all(out[:used] == 123, -1))
    alone, err = run_tree(c, q[:used].contiguous(), trees, max_nodes=nodes + 3)
    assert err == 0 and torch.equal(out[:used], alone)


def far(c, weights=None):
    """The cache's pages at the end of one of more than 2^32 bytes a side, its weights along."""
    page = c.hkv * PAGE * c.d * c.k.element_size()
    first = (2 ** 32 + 2 ** 20) // page
    for name in ("k", "v"):
        x = getattr(c, name)
        big = torch.empty((first + c.blocks, *x.shape[1:]), dtype=x.dtype, device="cuda")
        big[first:] = x
        setattr(c, name, big)
    c.tables = torch.where(c.tables >= 0, c.tables + first, c.tables)
    if weights is not None:
        w = torch.empty((first + c.blocks, *weights.shape[1:]), device="cuda")
        w[first:] = weights
        weights = w
    return first, weights


@pytest.mark.parametrize("hq,hkv,d,fmt", LAYOUTS)
def test_pages_past_32_bits_tree(hq, hkv, d, fmt):
    c = Cache([900, 33], hkv, d, fmt)
    trees, q = trees_of([30, 9]), queries(39, hq, d, 3)
    near, err = run_tree(c, q, trees)
    assert err == 0
    far(c)
    out, err = run_tree(c, q, trees)
    assert err == 0 and torch.equal(near, out)


@pytest.mark.parametrize("hkv,d,fmt", [(8, 128, "e4m3"), (2, 256, "bf16")])
def test_pages_past_32_bits_moved_and_weighed(hkv, d, fmt):
    results = []
    for at_the_end in (False, True):
        c = Cache([900, 33, 400], hkv, d, fmt)
        g = torch.Generator().manual_seed(1)
        w = torch.rand((c.blocks, hkv, PAGE), generator=g).cuda()
        first = 0
        if at_the_end:
            first, w = far(c, w)
        q = queries(3, 4 * hkv, d, 3)
        ws = fk.alloc_weights_workspace(3, 4 * hkv, hkv, d, 900)
        out = torch.empty_like(q)
        fk.fp8kv_paged_decode_weights(q, c.k, c.v, c.tables, c.seq_lens, 900, 1 / math.sqrt(d), 0, out, w, 0.9, ws, **c.kind_args())
        new = torch.empty(3, dtype=torch.int32, device="cuda")
        starts = torch.tensor([0, 20, 25, 40], dtype=torch.int32, device="cuda")
        paths = torch.tensor([[3, 9, 19], [2, -1, -1], [1, 14, -1]], dtype=torch.int32, device="cuda")
        fk.fp8kv_tree_commit(c.k, c.v, c.tables, c.seq_lens, starts, paths, 900, new, ws)
        cut, kept = torch.empty_like(new), torch.empty((3, hkv, 200), dtype=torch.int32, device="cuda")
        fk.fp8kv_evict(c.k, c.v, w, c.tables, new, 900, 200, 4, 30, cut, ws, kept=kept)
        torch.cuda.synchronize()
        assert fk.fp8kv_read_error(ws) == 0
        results.append([out, new, cut, kept, c.k[first:].view(torch.uint8), c.v[first:].view(torch.uint8), w[first:]])
        del c, w
    for a, b in zip(*results):
        assert torch.equal(a, b)


LIMIT_NS = 20_000_000


@pytest.mark.parametrize("stage", [0, 1, 3])
@pytest.mark.parametrize("nodes,hq,hkv,d,fmt", [(8, 32, 8, 128, "e4m3"), (30, 32, 8, 128, "e4m3"), (64, 32, 8, 128, "e5m2"),
                                                (8, 64, 8, 256, "e4m3"), (8, 64, 8, 256, "bf16"), (30, 64, 8, 64, "bf16")])
def test_a_wait_that_runs_out(nodes, hq, hkv, d, fmt, stage):
    c = Cache([6000] * 3, hkv, d, fmt)
    trees = trees_of([nodes] * 3)
    q = queries(3 * nodes, hq, d, 3)
    good, err = run_tree(c, q, trees)
    assert err == 0
    ws = fk.alloc_tree_workspace(3, nodes, c.max_len, hq, hkv, d)
    starts = torch.tensor([0, nodes, 2 * nodes, 3 * nodes], dtype=torch.int32, device="cuda")
    flat = torch.tensor(sum(trees, []), dtype=torch.int32, device="cuda")
    args = (q, c.k, c.v, c.tables, c.seq_lens, starts, flat, nodes, c.max_len, 1 / math.sqrt(d), 0)
    out = torch.full_like(q, 123)
    t0 = time.perf_counter()
    assert fk.debug_paged_tree_stall(*args, out, ws, stage, LIMIT_NS, **c.kind_args()) == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5
    again = torch.full_like(q, 123)
    fk.fp8kv_paged_tree_attention(*args, again, ws, **c.kind_args())
    torch.cuda.synchronize()
    assert torch.all(again == 123) and fk.fp8kv_read_error(ws) == 5      # skipped
    fk.fp8kv_workspace_init(ws)
    fk.fp8kv_paged_tree_attention(*args, again, ws, **c.kind_args())
    torch.cuda.synchronize()
    assert torch.equal(again, good) and fk.fp8kv_read_error(ws) == 0


def test_the_stall_hook_without_a_stall_is_the_plain_call():
    c = Cache([600], 8, 128)
    trees = trees_of([8])
    q = queries(8, 32, 128, 3)
    good, _ = run_tree(c, q, trees)
    ws = fk.alloc_tree_workspace(1, 8, 600, 32, 8, 128)
    out = torch.full_like(q, 123)
    starts = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    flat = torch.tensor(trees[0], dtype=torch.int32, device="cuda")
    args = (q, c.k, c.v, c.tables, c.seq_lens, starts, flat, 8, 600, 128 ** -0.5, 0, out, ws)
    assert fk.debug_paged_tree_stall(*args, 1000, LIMIT_NS, **c.kind_args()) == 0
    torch.cuda.synchronize()
    assert fk.fp8kv_read_error(ws) == 0 and torch.equal(out, good)


def test_no_weights_are_added_after_a_timeout():
    """The decode skips its work on a workspace whose error word says so, and the weights stay as they were."""
    c = Cache([700, 80], 8, 128)
    q = queries(2, 32, 128, 3)
    ws = fk.alloc_weights_workspace(2, 32, 8, 128, 700)
    w = torch.rand((c.blocks, 8, PAGE), generator=torch.Generator().manual_seed(1)).cuda()
    before, out = w.clone(), torch.full_like(q, 123)
    args = (q, c.k, c.v, c.tables, c.seq_lens, 700, 128 ** -0.5, 0, out, w, 0.9, ws)
    ws[:4].view(torch.int32).fill_(5)
    ws[256:].fill_(0x55)
    fk.fp8kv_paged_decode_weights(*args, **c.kind_args())
    torch.cuda.synchronize()
    assert torch.all(out == 123) and torch.equal(w, before) and fk.fp8kv_read_error(ws) == 5
    fk.fp8kv_workspace_init(ws)
    fk.fp8kv_paged_decode_weights(*args, **c.kind_args())
    torch.cuda.synchronize()
    assert fk.fp8kv_read_error(ws) == 0 and not torch.equal(w, before)


def test_another_stream():
    c = Cache([700, 80], 8, 128)
    trees, q = trees_of([20, 7]), queries(27, 32, 128, 3)
    good, _ = run_tree(c, q, trees)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, err = run_tree(c, q, trees, stream=side)
    assert err == 0 and torch.equal(out, good)

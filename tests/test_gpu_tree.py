"""fp8kv_paged_tree_attention against its definition in 64 bits.

Tolerance, element by element: the output's own rounding, 2^-8 |ref|, and what relative errors of the weights move,
at most e sum_t p_t |v_t|.  e counts: a weight's rounding to f16, 2^-11 (bf16 cache: two bf16, 2^-16); an error x of a
score (natural units) changes a weight by x and the sum it is divided by by as much.  x: Q's E4M3 split, at most 2^-18 of
the row's largest element each, sm sum_i |k_i| 2^-18 max|q| <= 128^-0.5 * 128 * 0.8 * 2^-18 * 4.5 = 2^-13 (d = 256:
2^-12.5); FP32 sums of d products, within d 2^-24 sum |q k| sm <= 256 * 2^-24 * 10 = 2^-12.7; exp2 and its argument,
2^-21 of a score of up to 20.  2 (2^-12.5 + 2^-12.7) + 2^-11 < 2^-9.6: e = 2^-9 with room for the tensor cores' summation order.
"""
import math

import pytest
import torch

from tests.spec_harness import (Cache, attended, chain, depths, queries, random_tree, rng, run_tree, tree_reference)

pytestmark = pytest.mark.gpu
E = 2.0 ** -9


def check(out, ref, mass, rows=None):
    got = out.double()
    assert torch.isfinite(got).all()
    bound = 2.0 ** -8 * ref.abs() + E * mass + 1e-6
    worst = ((got - ref).abs() / bound)
    worst = worst if rows is None else worst[rows]
    assert worst.max().item() <= 1.0, "max err/bound %.3f at %s" % (worst.max().item(), torch.nonzero(worst == worst.max())[0].tolist())


def case(lens, nodes, hq, hkv, d, fmt="e4m3", window=0, seed=0, sm=None, roots=1, trees=None):
    c = Cache([n + m for n, m in zip(lens, nodes)], hkv, d, fmt, seed)
    r = rng(seed)
    trees = [random_tree(m, r, min(m, roots)) for m in nodes] if trees is None else trees
    starts = [sum(nodes[:b]) for b in range(len(nodes))]
    q = queries(max(1, sum(nodes)), hq, d, seed + 1)
    out, err = run_tree(c, q, trees, window, sm)
    assert err == 0
    ref, mass = tree_reference(c, q, trees, starts, window, 1 / math.sqrt(d) if sm is None else sm)
    check(out, ref, mass)


LAYOUTS = [(32, 8, 128), (64, 8, 64), (8, 1, 256), (8, 8, 128), (16, 1, 128), (16, 1, 256), (4, 2, 64)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", LAYOUTS)
def test_layouts(hq, hkv, d, fmt):
    case([700, 33, 0, 1], [9, 5, 7, 1], hq, hkv, d, fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("nodes", [1, 2, 31, 32, 33, 64, 65, 100, 256])
def test_tree_sizes(nodes, fmt):
    case([500, 17], [nodes, max(1, nodes // 2)], 8, 2, 128, fmt, seed=nodes)


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("nodes", [40, 129])
def test_tree_sizes_other_heads(nodes, d):
    case([500, 17], [nodes, max(1, nodes // 2)], 16, 2, d, seed=nodes)


@pytest.mark.parametrize("context", [0, 1, 15, 16, 17, 111, 112, 127, 128, 129, 255, 1000, 2049])
def test_contexts(context):
    case([context, context + 5], [10, 20], 8, 2, 128, seed=context)


@pytest.mark.parametrize("fmt,d", [("e4m3", 128), ("e4m3", 256), ("bf16", 64)])
@pytest.mark.parametrize("window", [1, 2, 5, 16, 40, 128, 1000, 100000])
def test_windows(window, fmt, d):
    case([300, 7, 1100, 0], [40, 12, 33, 9], 8, 2, d, fmt, window=window, seed=window)


def test_chain_is_a_causal_chunk():
    """The tree that is a chain is what fp8kv_paged_prefill computes, within both roundings."""
    from fp8_kv_cache_fp8kv_gb300 import binding as fk
    nodes, lens = [33, 7, 128], [500, 7, 900]
    c = Cache(lens, 2, 128, "e4m3", 5)
    q = queries(sum(nodes), 8, 128, 6)
    out, err = run_tree(c, q, [chain(n) for n in nodes], window=100)
    assert err == 0
    starts = torch.tensor([0, 33, 40, 168], dtype=torch.int32, device="cuda")
    ws = fk.alloc_prefill_workspace(3, 128, 900, 8, 2, 128, window=100)
    want = torch.empty_like(q)
    fk.fp8kv_paged_prefill(q, c.k, c.v, c.tables, c.seq_lens, starts, 128, 900, *c.scale, 1 / math.sqrt(128), 100, want, ws)
    ref, mass = tree_reference(c, q, [chain(n) for n in nodes], [0, 33, 40], 100, 1 / math.sqrt(128))
    check(out, ref, mass)
    assert ((out.double() - want.double()).abs() <= 2.0 ** -7 * ref.abs() + 2 * E * mass + 1e-6).all()


def test_star_and_forest():
    """Every node a child of the root; every node a root."""
    star = [[-1] + [0] * 40, [-1] * 23]
    case([200, 90], [41, 23], 8, 2, 128, trees=star)


def test_many_short_sequences():
    lens = [rng(3).randrange(0, 90) for _ in range(70)]
    nodes = [rng(i).randrange(0, 12) for i in range(70)]
    case(lens, nodes, 16, 8, 64, seed=4)


def test_more_sequences_than_one_launch():
    case([20 + i % 7 for i in range(300)], [1 + i % 3 for i in range(300)], 4, 2, 64, seed=8)


def test_long_context_with_mean():
    """A sum of 40,000 values with a mean of their own: an accumulator of few bits would swamp."""
    c = Cache([40000 + 20], 1, 128, "e4m3", 1)
    c.v = (c.v.view(c.dtype).float().abs()).to(c.dtype).view(torch.uint8)
    q = queries(20, 4, 128, 2) * 0.05
    tree = [random_tree(20, rng(1))]
    out, err = run_tree(c, q, tree)
    assert err == 0
    check(out, *tree_reference(c, q, tree, [0], 0, 1 / math.sqrt(128)))


@pytest.mark.parametrize("order", ["rising", "falling"])
@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
def test_references_move(fmt, order):
    """Scores that grow (or fall) by hundreds of octaves along the context: references move, sums are rescaled."""
    c = Cache([900 + 40], 2, 128, fmt, 3)
    t = torch.arange(940, device="cuda")
    ramp = t.float() / 940 if order == "rising" else 1 - t.float() / 940
    page = c.tables[0].long()[t // 16]
    big = torch.ones(128, device="cuda") * (4.0 if fmt == "bf16" else 400.0)
    rows = (ramp[:, None] * big).to(c.dtype)
    c.k[page, :, t % 16] = (rows if fmt == "bf16" else rows.view(torch.uint8))[:, None]
    q = queries(40, 8, 128, 2).abs() * 0.5
    tree = [random_tree(40, rng(2))]
    out, err = run_tree(c, q, tree)
    assert err == 0
    # scores here reach 128 * 0.4 * 4 / 11 = 18 (e4m3) or as much in bf16; E's count of the FP32 sums scales with them
    check(out, *tree_reference(c, q, tree, [0], 0, 1 / math.sqrt(128)))


def test_one_key_and_a_large_crowd():
    """One key of weight 1 and 65,536 of 2^-17 each, a third of the answer: small weights must not round away."""
    n = 65536
    c = Cache([n + 1], 1, 128, "e4m3", 2)
    k = torch.zeros((n + 1, 128), device="cuda")
    k[0] = 1.0
    t = torch.arange(n + 1, device="cuda")
    page = c.tables[0].long()[t // 16]
    c.k[page, 0, t % 16] = k.to(c.dtype).view(torch.uint8)
    c.scale = (1.0, c.scale[1])
    q = torch.ones((1, 1, 128), dtype=torch.bfloat16, device="cuda")
    sm = 17 * math.log(2) / 128
    out, err = run_tree(c, q, [[-1]], sm=sm)
    assert err == 0
    check(out, *tree_reference(c, q, [[-1]], [0], 0, sm))


@pytest.mark.parametrize("sm", [0.0, -0.09, 1.5])
def test_score_scales(sm):
    # (scores of up to 1.5 * 11 * 4.5 = 75: their FP32 error scales alike, so q is cut to keep E's count)
    c = Cache([333], 2, 128, "e4m3", 7)
    q = queries(13, 8, 128, 3) * (0.05 if sm > 1 else 1.0)
    tree = [random_tree(13, rng(3))]
    out, err = run_tree(c, q, tree, sm=sm)
    assert err == 0
    check(out, *tree_reference(c, q, tree, [0], 0, sm))


def test_query_ranges():
    """Rows of tiny and of huge queries, one with a large outlier, one of zeros, beside each other."""
    c = Cache([222], 1, 128, "e4m3", 9)
    q = queries(8, 4, 128, 4).float()
    q[0] *= 2.0 ** -120
    q[1] = 0
    q[2, :, 5] = 30.0
    q[3] *= 2.0 ** -10
    q = q.to(torch.bfloat16)
    tree = [random_tree(8, rng(5))]
    out, err = run_tree(c, q, tree)
    assert err == 0
    # row 2: Q's split is off by up to 2^-18 * 30 an element, four times what E counts of it
    ref, mass = tree_reference(c, q, tree, [0], 0, 1 / math.sqrt(128))
    mass[2] *= 2
    check(out, ref, mass)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_per_head_scales(fmt):
    c = Cache([400, 90], 4, 128, fmt, 11)
    q = queries(30, 16, 128, 5)
    trees = [random_tree(20, rng(6)), random_tree(10, rng(7))]
    ks = torch.tensor([0.5, 1.0, 1.7, 0.1], device="cuda") * c.scale[0]
    vs = torch.tensor([1.5, 0.3, 1.0, 2.1], device="cuda") * c.scale[1]
    out, err = run_tree(c, q, trees, scales=(ks, vs))
    assert err == 0
    check(out, *tree_reference(c, q, trees, [0, 20], 0, 1 / math.sqrt(128), scales=(ks, vs)))
    same = torch.full((4,), c.scale[0], device="cuda"), torch.full((4,), c.scale[1], device="cuda")
    a, _ = run_tree(c, q, trees, scales=same)
    b, _ = run_tree(c, q, trees)
    assert torch.equal(a, b)

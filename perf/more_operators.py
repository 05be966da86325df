"""Measured cases of speculative decoding and of eviction over the paged cache.

Four operators, one layer's worth of a serving step:

* ``tree``: attention of a tree of drafted tokens per sequence over its cache (E4M3, E5M2 or bf16 pages): every node
  attends the sequence's context, its ancestors in the tree and itself;
* ``commit``: the accepted path's rows moved behind the context, where the next step finds them;
* ``weights``: one query token per sequence, whose attention weights are added up for every cached token;
* ``evict``: per kv head, the tokens of the largest accumulated weight kept (with the first and the newest ones) and
  moved to the front of the sequence's pages, in their order.

``own`` selects the library's calls; otherwise ``run`` computes the same in elementary torch operations.
"""
import math
import random

import torch

own = False

PAGE = 16
TOP = {"e4m3": 448.0, "e5m2": 57344.0, "bf16": None}
FLOAT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    llama = dict(hq=32, hkv=8, d=128)
    return [
        # a single chat that checks a short draft: latency counts
        dict(name="tree 1x4096 8 nodes", op="tree", batch=1, context=4096, nodes=8, window=0, fmt="e4m3", **llama),
        # the serving batch, drafts of two or three branches
        dict(name="tree 8x20K 16 nodes", op="tree", batch=8, context=20000, nodes=16, window=0, fmt="e4m3", **llama),
        # the serving batch, wide drafts
        dict(name="tree 8x20K 64 nodes", op="tree", batch=8, context=20000, nodes=64, window=0, fmt="e4m3", **llama),
        # an uncalibrated bf16 cache, eight query heads to a kv head, an odd batch
        dict(name="tree 5x9K bf16 d64", op="tree", batch=5, context=9001, nodes=33, window=0, fmt="bf16", hq=64, hkv=8,
             d=64),
        # a sliding-window layer of wide heads in the E5M2 cache
        dict(name="tree 16x8K d256 window 512", op="tree", batch=16, context=8192, nodes=25, window=512, fmt="e5m2",
             hq=8, hkv=1, d=256),
        # after a check: three or four drafted tokens of each sequence stay
        dict(name="commit 8 of 16 nodes", op="commit", batch=8, context=300, nodes=16, accept=4, fmt="e4m3", **llama),
        # a large batch with long accepted paths in the bf16 cache
        dict(name="commit 64 of 64 nodes", op="commit", batch=64, context=777, nodes=64, accept=21, fmt="bf16", hq=64,
             hkv=8, d=64),
        # a decode step that keeps account of attention: one chat
        dict(name="weights 1x4096", op="weights", batch=1, context=4096, window=0, fmt="e4m3", **llama),
        # the same of the serving batch
        dict(name="weights 8x20K", op="weights", batch=8, context=20000, window=0, fmt="e4m3", **llama),
        # steady state: a cache that has grown past its budget by a few pages is cut back
        dict(name="evict 16x1100 to 1024", op="evict", batch=16, context=1100, budget=1024, sinks=4, recent=256,
             fmt="e4m3", **llama),
        # long prompts cut to a fifth
        dict(name="evict 8x20K to 4096", op="evict", batch=8, context=20000, budget=4096, sinks=4, recent=512,
             fmt="e4m3", **llama),
        # one very long context cut to a sixteenth
        dict(name="evict 1x128K to 8191", op="evict", batch=1, context=131072, budget=8191, sinks=16, recent=1000,
             fmt="e4m3", hq=64, hkv=8, d=128),
    ]


LAYOUTS = [(32, 8, 128), (64, 8, 64), (8, 1, 256), (64, 8, 128), (16, 16, 64), (16, 8, 128), (32, 2, 128)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "commit", "weights", "evict"])
    hq, hkv, d = rng.choice(LAYOUTS)
    case = dict(op=op, hq=hq, hkv=hkv, d=d, fmt=rng.choice(["e4m3", "e4m3", "e5m2", "bf16"]))
    wide = 2 if case["fmt"] == "bf16" else 1
    if op == "commit":
        nodes = _log(rng, 2, 64)
        case.update(batch=_log(rng, 1, 64), context=_log(rng, 10, 800), nodes=nodes, accept=_log(rng, 1, nodes))
        return case
    batch = _log(rng, 1, 16)
    most = min(131072 if op == "evict" else 60000, 330_000_000 // (2 * hkv * d * wide) // batch)
    context = _log(rng, 30, most)
    case.update(batch=batch, context=context)
    if op == "tree":
        most = max(2, min(128, 150_000_000_000 // (4 * hq * d * batch * context)))
        case.update(nodes=_log(rng, 1, most), window=rng.choice([0, 0, 128, 1000]))
    elif op == "weights":
        case.update(window=rng.choice([0, 0, 0, 512]))
    else:
        budget = _log(rng, 20, max(21, min(context, 16384)))
        case.update(budget=budget, sinks=rng.choice([0, 4, budget // 10]), recent=rng.choice([1, budget // 4, budget // 2]))
    return case


def _spread(mean, n, part):
    """n whole numbers evenly spaced in mean * (1 +- part): ragged, with a sum that the case alone fixes."""
    if n == 1:
        return [mean]
    return [max(1, int(round(mean * (1 - part + 2 * part * i / (n - 1))))) for i in range(n)]


def _nodes(case):
    return _spread(case["nodes"], case["batch"], 0.25)


def _lens(case):
    """Tokens of each sequence in the cache, its drafted ones included."""
    context = _spread(case["context"], case["batch"], 0.1)
    return [c + n for c, n in zip(context, _nodes(case))] if case["op"] in ("tree", "commit") else context


def _trees(case):
    """The parent of every node of each sequence's tree: a root (the last accepted token), drafts that prefer young
    parents, so that a few long branches and many short ones come out."""
    rng = random.Random(case["nodes"] * 1000003 + case["batch"])
    return [[-1] + [max(rng.randrange(i), rng.randrange(i)) for i in range(1, n)] for n in _nodes(case)]


def _depths(tree):
    depth = []
    for p in tree:
        depth.append(0 if p < 0 else depth[p] + 1)
    return depth


def _accepted(case):
    return [min(n, max(1, c)) for n, c in zip(_nodes(case), _spread(case["accept"], case["batch"], 0.3))]


# ------------------------------------------------------------------ inputs

def _stored(shape, fmt, g, dev):
    """Unit-normal data as the cache holds it: codes that fill their format (under a calibrated scale), or bf16."""
    x = torch.randn(shape, generator=g, device=dev)
    if fmt == "bf16":
        return x.to(torch.bfloat16)
    return x.mul_(TOP[fmt] / 4.5).clamp_(-TOP[fmt], TOP[fmt]).to(FLOAT[fmt]).view(torch.uint8)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    order = torch.Generator().manual_seed(seed)
    op, hkv, d, batch = case["op"], case["hkv"], case["d"], case["batch"]
    mix = torch.randperm(batch, generator=order).tolist()
    lens = [_lens(case)[i] for i in mix]
    pages = [-(-n // PAGE) for n in lens]
    blocks = sum(pages) + 3
    perm = torch.randperm(blocks, generator=order)
    s = dict(case=case, sm=1.0 / math.sqrt(d), max_len=max(lens))
    s["tables"] = torch.nn.utils.rnn.pad_sequence(perm[: sum(pages)].split(pages), batch_first=True).to(
        torch.int32).to(dev)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    shape = (blocks, hkv, PAGE, d)
    s["k_cache"], s["v_cache"] = (_stored(shape, case["fmt"], g, dev) for _ in range(2))
    s["k_scale"], s["v_scale"] = (4.5 / TOP[case["fmt"]], 4.0 / TOP[case["fmt"]]) if TOP[case["fmt"]] else (1.0, 1.0)
    if op in ("tree", "commit"):
        trees = [_trees(case)[i] for i in mix]
        counts = [len(t) for t in trees]
        s["max_nodes"] = max(counts)
        s["starts"] = torch.tensor([0] + counts, dtype=torch.int32, device=dev).cumsum(0, dtype=torch.int32)
    if op == "tree":
        s["parents"] = torch.tensor(sum(trees, []), dtype=torch.int32, device=dev)
        s["q"] = torch.randn((sum(counts), case["hq"], d), generator=g, device=dev).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
    elif op == "commit":
        # the accepted path of each tree, a -1 behind the shorter ones
        took = [_accepted(case)[i] for i in mix]
        path = [torch.randperm(n - 1, generator=order)[: c - 1].sort()[0] + 1 for n, c in zip(counts, took)]
        s["accepted"] = torch.nn.utils.rnn.pad_sequence([torch.cat((torch.zeros(1, dtype=torch.int64), p)) for p in path],
                                                        batch_first=True, padding_value=-1).to(torch.int32).to(dev)
    else:
        # what earlier steps have added up: a few tokens hold most of it, some nothing
        w = torch.randn((blocks, hkv, PAGE), generator=g, device=dev).mul_(2.0).exp_()
        s["weights"] = torch.where(w < 0.1, 0.0, w)
    if op == "weights":
        s["q"] = torch.randn((batch, case["hq"], d), generator=g, device=dev).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["decay"] = 0.98
    if op in ("commit", "evict"):
        s["new_lens"] = torch.zeros(batch, dtype=torch.int32, device=dev)
    if op == "evict":
        s["kept"] = torch.empty((batch, hkv, case["budget"]), dtype=torch.int32, device=dev)
    return s


# ------------------------------------------------------------------ plain forms

def _values(cache, fmt):
    return cache if fmt == "bf16" else cache.view(FLOAT[fmt])


def _gathered(s, rows):
    """K and V in 32 bits, [B, Hkv, tokens, d], of the pages that the last `rows` tokens of each sequence may attend,
    and the place of each token in its sequence, [B, tokens]."""
    case, tables = s["case"], s["tables"].long()
    first, count = torch.zeros_like(s["lens"]), tables.shape[1]
    if case["window"]:
        first = (s["lens"] - rows - case["window"]).clamp_min(0) // PAGE
        count = min(count, (case["window"] + rows) // PAGE + 2)
    page = first[:, None] + torch.arange(count, device="cuda")
    ids = tables.gather(1, page.clamp_max(tables.shape[1] - 1))
    k, v = ((_values(s[c + "_cache"][ids], case["fmt"]).float() * s[c + "_scale"]).transpose(1, 2).flatten(2, 3)
            for c in "kv")
    return k, v, (page[..., None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(1).long()


def _softmax(scores, mask):
    """softmax over the last axis where the mask is true, zeros elsewhere and where it leaves nothing."""
    scores.masked_fill_(~mask, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = scores.sub_(top).exp_()
    return p.div_(p.sum(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).tiny))


def _plain_tree(s):
    case, n = s["case"], s["max_nodes"]
    starts, lens = s["starts"].long(), s["lens"].long()
    counts = starts.diff()
    context = lens - counts
    i = torch.arange(n, device="cuda")
    token = (starts[:-1, None] + i).clamp_max(s["q"].shape[0] - 1)                    # [B, n]
    real = i < counts[:, None]
    # who descends from whom: the parent relation, squared until it stands
    parent = torch.where(real, s["parents"].long()[token], -1)
    reach = ((parent[..., None] == i) | torch.eye(n, dtype=torch.bool, device="cuda")).float()
    for _ in range(max(1, (n - 1).bit_length())):
        reach = (reach @ reach).clamp_max_(1.0)
    depth = reach.sum(-1).long() - 1                                                  # [B, n]
    k, v, place = _gathered(s, n)
    q = s["q"][token].float().unflatten(2, (case["hkv"], -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    # [B, n, tokens]: the context, and the node's own branch
    node = place - context[:, None]
    drafted = (node >= 0) & (node < counts[:, None])
    at = node.clamp(0, n - 1)
    mask = reach.gather(2, at[:, None].expand(-1, n, -1)) > 0.5
    mask = (mask & drafted[:, None]) | (node < 0)[:, None]
    if case["window"]:
        position = torch.where(node < 0, place, context[:, None] + depth.gather(1, at))
        mask &= position[:, None] > (context[:, None] + depth)[..., None] - case["window"]
    mask = mask[:, None].expand(-1, case["hq"] // case["hkv"], -1, -1).flatten(1, 2)[:, None]
    o = _softmax((q @ k.transpose(-1, -2)).mul_(s["sm"]), mask) @ v
    o = o.unflatten(2, (-1, n)).permute(0, 3, 1, 2, 4).flatten(2, 3)                  # [B, n, Hq, d]
    s["out"][token[real]] = o[real].to(torch.bfloat16)
    return s["out"]


def _slots(s, place):
    """Block and row of places [B, ...] in their sequences."""
    b = torch.arange(place.shape[0], device="cuda").view(-1, *[1] * (place.dim() - 1))
    return s["tables"].long()[b, place // PAGE], place % PAGE


def _plain_commit(s):
    starts, lens = s["starts"].long(), s["lens"].long()
    context = lens - starts.diff()
    path = s["accepted"].long()
    took = (path >= 0).cumprod(1)
    rank = torch.arange(path.shape[1], device="cuda")
    b, i = took.nonzero(as_tuple=True)
    block, row = _slots(s, context[:, None] + path.clamp_min(0))
    to_block, to_row = _slots(s, context[:, None] + torch.minimum(rank.expand_as(path), lens[:, None] - context[:, None] - 1))
    for name in ("k_cache", "v_cache"):
        s[name][to_block[b, i], :, to_row[b, i]] = s[name][block[b, i], :, row[b, i]]
    s["new_lens"].copy_(context + took.sum(1))
    return _answer_commit(s)


def _answer_commit(s):
    fmt = s["case"]["fmt"]
    return {"k": _values(s["k_cache"], fmt), "v": _values(s["v_cache"], fmt), "lens": s["new_lens"]}


def _plain_weights(s):
    case, lens = s["case"], s["lens"].long()
    k, v, place = _gathered(s, 1)
    q = s["q"].float().unflatten(1, (case["hkv"], -1))
    mask = place < lens[:, None]
    if case["window"]:
        mask &= place >= lens[:, None] - case["window"]
    p = _softmax((q @ k.transpose(-1, -2)).mul_(s["sm"]), mask[:, None, None])        # [B, Hkv, g, tokens]
    s["out"].copy_((p @ v).flatten(1, 2))
    added = p.sum(2).transpose(1, 2)[mask]                                            # [pairs, Hkv]
    newest = (place == lens[:, None] - 1)[mask]
    block, row = _slots(s, place.clamp_max(s["tables"].shape[1] * PAGE - 1))
    at = (block[mask], slice(None), row[mask])
    s["weights"][at] = torch.where(newest[:, None], 0.0, s["weights"][at] * s["decay"]) + added
    return {"out": s["out"], "weights": s["weights"]}


def _plain_evict(s):
    case, lens = s["case"], s["lens"].long()
    place = torch.arange(s["max_len"], device="cuda").expand(case["batch"], -1)
    block, row = _slots(s, place)
    w = s["weights"][block, :, row].transpose(1, 2)                                   # [B, Hkv, tokens]
    n = lens[:, None, None]
    place = place[:, None]
    w = torch.where((place < case["sinks"]) | (place >= n - case["recent"]), math.inf, w)
    w = torch.where(place < n, w, -math.inf)
    count = lens.clamp_max(case["budget"])
    rank = torch.arange(case["budget"], device="cuda")
    # the largest first, of equal ones the first: as many as there is room for, back in their order
    first = w.sort(dim=-1, descending=True, stable=True)[1][..., : case["budget"]]
    none = rank >= count[:, None, None]
    kept = torch.where(none[..., : first.shape[-1]], s["max_len"], first).sort(dim=-1)[0]
    s["kept"].fill_(-1)
    s["kept"][..., : kept.shape[-1]] = torch.where(none[..., : kept.shape[-1]], -1, kept)
    b, h, i = (s["kept"] >= 0).nonzero(as_tuple=True)
    at = s["kept"][b, h, i].long()
    tables = s["tables"].long()
    for name in ("k_cache", "v_cache", "weights"):
        s[name][tables[b, i // PAGE], h, i % PAGE] = s[name][tables[b, at // PAGE], h, at % PAGE]
    s["new_lens"].copy_(count)
    return _answer_evict(s)


def _answer_evict(s):
    return {**_answer_commit(s), "weights": s["weights"], "kept": s["kept"]}


# ------------------------------------------------------------------ the library's calls

def _cache_kind(fk, s):
    """The arguments that say what the cache holds."""
    return dict(k_scale=s["k_scale"], v_scale=s["v_scale"],
                cache_format={"e4m3": fk.CACHE_E4M3, "e5m2": fk.CACHE_E5M2, "bf16": fk.CACHE_BF16}[s["case"]["fmt"]])


def _own_workspace(s, make):
    """The caller-owned workspace, allocated once for a state, as a serving loop does."""
    if "workspace" not in s:
        s["workspace"] = make()
    return s["workspace"]


def _own_tree(s):
    from fp8_kv_cache_fp8kv_gb300 import binding as fk
    case = s["case"]
    ws = _own_workspace(s, lambda: fk.alloc_tree_workspace(case["batch"], s["max_nodes"], s["max_len"], case["hq"],
                                                           case["hkv"], case["d"], window=case["window"]))
    fk.fp8kv_paged_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["starts"], s["parents"],
                                  s["max_nodes"], s["max_len"], s["sm"], case["window"], s["out"], ws,
                                  **_cache_kind(fk, s))
    return s["out"]


def _own_commit(s):
    from fp8_kv_cache_fp8kv_gb300 import binding as fk
    ws = _own_workspace(s, fk.alloc_append_workspace)
    fk.fp8kv_tree_commit(s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["starts"], s["accepted"], s["max_len"],
                         s["new_lens"], ws)
    return _answer_commit(s)


def _own_weights(s):
    from fp8_kv_cache_fp8kv_gb300 import binding as fk
    case = s["case"]
    ws = _own_workspace(s, lambda: fk.alloc_weights_workspace(case["batch"], case["hq"], case["hkv"], case["d"],
                                                              s["max_len"], window=case["window"]))
    fk.fp8kv_paged_decode_weights(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["max_len"], s["sm"],
                                  case["window"], s["out"], s["weights"], s["decay"], ws, **_cache_kind(fk, s))
    return {"out": s["out"], "weights": s["weights"]}


def _own_evict(s):
    from fp8_kv_cache_fp8kv_gb300 import binding as fk
    case = s["case"]
    ws = _own_workspace(s, fk.alloc_append_workspace)
    fk.fp8kv_evict(s["k_cache"], s["v_cache"], s["weights"], s["tables"], s["lens"], s["max_len"], case["budget"],
                   case["sinks"], case["recent"], s["new_lens"], ws, kept=s["kept"])
    return _answer_evict(s)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tree": _own_tree, "commit": _own_commit, "weights": _own_weights, "evict": _own_evict}[op](state)
    return {"tree": _plain_tree, "commit": _plain_commit, "weights": _plain_weights, "evict": _plain_evict}[op](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    hq, hkv, d, op, batch = case["hq"], case["hkv"], case["d"], case["op"], case["batch"]
    row = 2 * hkv * d * (2 if case["fmt"] == "bf16" else 1)     # K and V of a token
    if op == "commit":
        rows = sum(_accepted(case))
        return {"bytes": rows * (2 * row + 4) + batch * 12, "flops": 0}
    if op == "evict":
        moved = bytes_ = 0
        for n in _lens(case):
            if n > case["budget"]:
                moved += case["budget"] - case["sinks"]
                bytes_ += n * hkv * 4 + (n - 1) // PAGE * 4 + 4
            bytes_ += min(n, case["budget"]) * hkv * 4 + 8
        return {"bytes": bytes_ + moved * (2 * row + hkv * 4), "flops": 0}
    window = case["window"]
    tokens = pages = pairs = rows = 0
    trees = _trees(case) if op == "tree" else [[-1]] * batch
    for n, tree in zip(_lens(case), trees):
        depth = _depths(tree)
        context = n - len(tree)
        lo = max(0, context + 1 - window) if window else 0
        tokens += n - lo
        pages += (n - 1) // PAGE - lo // PAGE + 1
        for at in depth:
            pairs += min(context + at + 1, window) if window else context + at + 1
        rows += len(tree)
    moved = tokens * row + pages * 4 + rows * hq * d * 4 + batch * 4
    if op == "weights":
        return {"bytes": moved + tokens * hkv * 8, "flops": pairs * hq * (4 * d + 1)}
    return {"bytes": moved + rows * 4 + batch * 4, "flops": 4 * hq * d * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits

def _pages_of(s, name, b, h, n):
    """The first n rows of sequence b and kv head h in 64 bits, [n, d]."""
    ids = s["tables"][b, : -(-n // PAGE)].long()
    scale = float(torch.tensor(s[name[0] + "_scale"], dtype=torch.float32))
    return _values(s[name][ids, h], s["case"]["fmt"]).double().flatten(0, 1)[:n] * scale


def _branch(tree, i):
    while i >= 0:
        yield i
        i = tree[i]


def _exact_tree(s):
    case = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    starts, lens, parents = s["starts"].tolist(), s["lens"].tolist(), s["parents"].tolist()
    group = case["hq"] // case["hkv"]
    for b, n in enumerate(lens):
        tree = parents[starts[b]:starts[b + 1]]
        context, depth = n - len(tree), _depths(tree)
        seen = torch.zeros((len(tree), n), dtype=torch.bool)
        for i in range(len(tree)):
            last = context + depth[i]
            oldest = max(0, last - case["window"] + 1) if case["window"] else 0
            seen[i, oldest:context] = True
            for j in _branch(tree, i):
                seen[i, context + j] = context + depth[j] >= oldest
        seen = seen.to("cuda")
        for h in range(case["hkv"]):
            k, v = _pages_of(s, "k_cache", b, h, n), _pages_of(s, "v_cache", b, h, n)
            heads = slice(h * group, (h + 1) * group)
            z = torch.einsum("rgd,td->grt", s["q"][starts[b]:starts[b + 1], heads].double(), k).mul_(s["sm"])
            z.masked_fill_(~seen, -math.inf)
            out[starts[b]:starts[b + 1], heads] = torch.einsum("grt,td->rgd", torch.softmax(z, -1), v)
    return out


def _exact_weights(s):
    case = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    weights = s["weights"].double()
    group, decay = case["hq"] // case["hkv"], float(torch.tensor(s["decay"], dtype=torch.float32))
    for b, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - case["window"]) if case["window"] else 0
        at = torch.arange(lo, n, device="cuda")
        block, row = s["tables"][b].long()[at // PAGE], at % PAGE
        for h in range(case["hkv"]):
            k, v = _pages_of(s, "k_cache", b, h, n)[lo:], _pages_of(s, "v_cache", b, h, n)[lo:]
            heads = slice(h * group, (h + 1) * group)
            p = torch.softmax(s["q"][b, heads].double() @ k.T * s["sm"], -1)
            out[b, heads] = p @ v
            old = weights[block, h, row] * decay
            old[-1] = 0.0
            weights[block, h, row] = old + p.sum(0)
    return {"out": out, "weights": weights}


def _exact_moved(s, lists):
    """The caches (and weights) after the rows of each (sequence, kv head)'s list moved to the places given."""
    fmt, tables = s["case"]["fmt"], s["tables"].long().cpu()
    names = [n for n in ("k_cache", "v_cache", "weights") if n in s]
    out = {n[0] if n != "weights" else n: (_values(s[n], fmt) if n != "weights" else s[n]).double() for n in names}
    for b, per_head in enumerate(lists):
        for h, (source, target) in enumerate(per_head):
            for x in out.values():
                x[tables[b][target // PAGE].cuda(), h, (target % PAGE).cuda()] = x[
                    tables[b][source // PAGE].cuda(), h, (source % PAGE).cuda()]
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "tree":
        return _exact_tree(s)
    if op == "weights":
        return _exact_weights(s)
    lists, count = [], []
    if op == "commit":
        starts, lens = s["starts"].tolist(), s["lens"].tolist()
        for b, path in enumerate(s["accepted"].tolist()):
            context = lens[b] - (starts[b + 1] - starts[b])
            path = torch.tensor([p for p in path if p >= 0])
            lists.append([(context + path, context + torch.arange(len(path)))] * case["hkv"])
            count.append(context + len(path))
        return {**_exact_moved(s, lists), "lens": torch.tensor(count, dtype=torch.int32, device="cuda")}
    kept = torch.full(s["kept"].shape, -1, dtype=torch.int32)
    tables, weights = s["tables"].long().cpu(), s["weights"].cpu()
    for b, n in enumerate(s["lens"].tolist()):
        per_head, size = [], min(n, case["budget"])
        at = torch.arange(n)
        held = weights[tables[b][at // PAGE], :, at % PAGE]
        for h in range(case["hkv"]):
            chosen = set(range(min(case["sinks"], n))) | set(range(max(0, n - case["recent"]), n))
            if n <= case["budget"]:
                chosen = set(at.tolist())
            value = held[:, h].tolist()
            for t in sorted((t for t in range(n) if t not in chosen), key=lambda t: (-value[t], t)):
                if len(chosen) >= size:
                    break
                chosen.add(t)
            source = torch.tensor(sorted(chosen))
            kept[b, h, :size] = source
            per_head.append((source, torch.arange(size)))
        lists.append(per_head)
        count.append(size)
    return {**_exact_moved(s, lists), "lens": torch.tensor(count, dtype=torch.int32, device="cuda"), "kept": kept.cuda()}

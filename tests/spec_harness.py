"""Shared plumbing of the tests of drafted trees, attention weights and eviction: seeded paged caches of every format,
and the operators' definitions in 64 bits, row by row."""
import math
import random

import torch

from fp8_kv_cache_fp8kv_gb300 import binding as fk

PAGE = 16
FORMATS = {"e4m3": (fk.CACHE_E4M3, torch.float8_e4m3fn, 448.0), "e5m2": (fk.CACHE_E5M2, torch.float8_e5m2, 57344.0),
           "bf16": (fk.CACHE_BF16, torch.bfloat16, None)}
NAN_BYTE = 0x7F     # a NaN code of E4M3 and E5M2; 0x7F7F is a huge bf16


class Cache:
    """A paged cache of sequences of the given lengths, pages in random order.  Every place that holds no token is
    filled with NaN codes (bf16: NaN), every page that no sequence owns as well."""

    def __init__(self, lens, hkv, d, fmt="e4m3", seed=0, device="cuda", spare=3, room=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hkv, self.d, self.fmt = list(lens), hkv, d, fmt
        self.kind, self.dtype, top = FORMATS[fmt]
        pages = [-(-(n + room) // PAGE) for n in lens]
        self.blocks = sum(pages) + spare
        ids = torch.randperm(self.blocks, generator=g)[: sum(pages)].split(pages)
        self.tables = torch.nn.utils.rnn.pad_sequence(ids, batch_first=True, padding_value=-7).to(torch.int32)
        if self.tables.shape[1] == 0:
            self.tables = torch.full((len(lens), 1), -7, dtype=torch.int32)
        shape = (self.blocks, hkv, PAGE, d)
        x = torch.randn((2, *shape), generator=g)
        raw = x.to(torch.bfloat16) if top is None else (x * (top / 4.5)).clamp(-top, top).to(self.dtype)
        self.scale = (1.0, 1.0) if top is None else (4.5 / top, 4.1 / top)
        live = torch.zeros((self.blocks, PAGE), dtype=torch.bool)
        for b, n in enumerate(lens):
            t = torch.arange(n)
            live[self.tables[b].long()[t // PAGE], t % PAGE] = True
        dead = ~live[:, None, :, None].expand(shape)
        k, v = raw[0].clone(), raw[1].clone()
        if top is None:
            k[dead], v[dead] = math.nan, math.nan
        else:
            k, v = k.view(torch.uint8), v.view(torch.uint8)
            k[dead], v[dead] = NAN_BYTE, NAN_BYTE
        self.k, self.v = k.to(device), v.to(device)
        self.tables = self.tables.to(device)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device=device)
        self.max_len = max(list(lens) + [1])

    def values(self, which):
        x = self.k if which == "k" else self.v
        return x.double() if self.fmt == "bf16" else x.view(self.dtype).double()

    def rows(self, which, b, h, n=None, scales=None):
        """The first n rows of sequence b and kv head h as the values they stand for, float64 [n, d]."""
        n = self.lens[b] if n is None else n
        t = torch.arange(n, device=self.k.device)
        page = self.tables[b].long()[t // PAGE]
        x = self.k if which == "k" else self.v
        x = x[page, h, t % PAGE]
        x = x.double() if self.fmt == "bf16" else x.view(self.dtype).double()
        s = self.scale["kv".index(which)] if scales is None else scales["kv".index(which)][h].item()
        return x * float(torch.tensor(s, dtype=torch.float32))

    def kind_args(self):
        return dict(k_scale=self.scale[0], v_scale=self.scale[1], cache_format=self.kind)


def random_tree(n, rng, roots=1):
    return [-1 if i < roots else max(rng.randrange(i), rng.randrange(i)) for i in range(n)]


def chain(n):
    return list(range(-1, n - 1))


def depths(tree):
    out = []
    for p in tree:
        out.append(0 if p < 0 else out[p] + 1)
    return out


def attended(tree, context, window):
    """bool [n, context + n]: what each node attends, from the definition."""
    n, dep = len(tree), depths(tree)
    seen = torch.zeros((n, context + n), dtype=torch.bool)
    for i in range(n):
        at = context + dep[i]
        for t in range(context):
            seen[i, t] = window <= 0 or t > at - window
        j = i
        while j >= 0:
            seen[i, context + j] = window <= 0 or dep[j] > dep[i] - window
            j = tree[j]
    return seen


def attend(q, k, v, seen, sm):
    """float64 attention of rows q [r, g, d] over k, v [t, d] where seen [r, t]; also sum_t p_t |v_t|, which bounds
    what relative errors of the weights can do."""
    z = torch.einsum("rgd,td->grt", q.double(), k) * sm
    z = z.masked_fill(~seen.to(z.device), -math.inf)
    p = torch.softmax(z, -1)
    return torch.einsum("grt,td->rgd", p, v), torch.einsum("grt,td->rgd", p, v.abs()), p


def tree_reference(c, q, trees, starts, window, sm, scales=None):
    out, mass = torch.zeros(q.shape, dtype=torch.float64, device=q.device), torch.zeros(q.shape, dtype=torch.float64,
                                                                                       device=q.device)
    g = q.shape[1] // c.hkv
    for b, tree in enumerate(trees):
        if not tree:
            continue
        seen = attended(tree, c.lens[b] - len(tree), window)
        rows = slice(starts[b], starts[b] + len(tree))
        for h in range(c.hkv):
            heads = slice(h * g, (h + 1) * g)
            out[rows, heads], mass[rows, heads], _ = attend(q[rows, heads], c.rows("k", b, h, scales=scales),
                                                            c.rows("v", b, h, scales=scales), seen, sm)
    return out, mass


def run_tree(c, q, trees, window=0, sm=None, scales=None, max_nodes=None, out=None, workspace=None, max_len=None,
             starts=None, stream=None):
    """fp8kv_paged_tree_attention over the whole batch: (out, error word)."""
    dev = c.k.device
    T, hq, d = q.shape
    sm = 1.0 / math.sqrt(d) if sm is None else sm
    max_nodes = max(len(t) for t in trees) if max_nodes is None else max_nodes
    max_len = c.max_len if max_len is None else max_len
    if starts is None:
        starts = torch.tensor([0] + [len(t) for t in trees]).cumsum(0).to(torch.int32).to(dev)
    flat = torch.tensor(sum(trees, []) + [-1] * (T - sum(len(t) for t in trees)), dtype=torch.int32, device=dev)
    ws = fk.alloc_tree_workspace(len(trees), max_nodes, max_len, hq, c.hkv, d, window=window) if workspace is None else workspace
    out = torch.full_like(q, 123.0) if out is None else out
    kind = c.kind_args()
    if scales is not None:
        kind.update(k_scales=scales[0], v_scales=scales[1])
    fk.fp8kv_paged_tree_attention(q, c.k, c.v, c.tables, c.seq_lens, starts, flat, max_nodes, max_len, sm, window, out,
                                  ws, stream=stream, **kind)
    torch.cuda.synchronize()
    return out, fk.fp8kv_read_error(ws)


def queries(rows, hq, d, seed, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((rows, hq, d), generator=g).to(torch.bfloat16).to(device)


def rng(seed):
    return random.Random(seed)

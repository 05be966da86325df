"""Measured cases of the rotary append and of attention over a block-scaled fp8 cache.

Four operators, one layer's worth of a serving step:

* ``rope_append``: rotate q and k by their positions (one axis, or several for images and video), write k and v at a
  slot mapping into an E4M3, E5M2 or bf16 paged cache;
* ``rope_append_block``: the same for each sequence's newest tokens into an E4M3 cache with one scale per page and
  kv head, requantising a page that outgrows its scale;
* ``decode_block``: one query token per sequence over such a cache;
* ``prefill_block``: a causal chunk per sequence over such a cache.

``own`` selects the library's calls; otherwise ``run`` computes the same in elementary torch operations.
"""
import math

import torch

own = False

PAGE = 16
E4M3_MAX, E5M2_MAX = 448.0, 57344.0
EXP_LO, EXP_HI = -40, 40        # the powers of two a page's scale may take


# ------------------------------------------------------------------ cases

def listed():
    llama = dict(hq=32, hkv=8, d=128)
    return [
        # one decode step's new tokens of the 8-sequence serving batch into the per-tensor E4M3 cache
        dict(name="append 8 new tokens", op="rope_append", tokens=8, axes=1, style="halves", rotary=128, fmt="e4m3",
             **llama),
        # a prompt with images: three position axes, interleaved over the frequencies, an odd token count
        dict(name="append 1999, 3 axes", op="rope_append", tokens=1999, axes=3, style="halves", rotary=128, fmt="e4m3",
             **llama),
        # a long prompt into the bf16 cache, half of each head rotated in adjacent pairs
        dict(name="append 16000 bf16", op="rope_append", tokens=16000, axes=1, style="pairs", rotary=32, fmt="bf16",
             hq=64, hkv=8, d=64),
        # one decode step's new tokens into the block-scaled cache
        dict(name="block append 8 tokens", op="rope_append_block", batch=8, chunk=1, axes=1, style="halves",
             rotary=128, **llama),
        # ragged prompt chunks of 8 sequences, positions on three axes
        dict(name="block append 8x2000", op="rope_append_block", batch=8, chunk=2000, axes=3, style="halves",
             rotary=128, **llama),
        # a single chat at a short context: latency counts
        dict(name="decode 1x4096", op="decode_block", batch=1, context=4096, window=0, padded=False, **llama),
        # the serving batch at ~20K tokens a sequence
        dict(name="decode 8x20K", op="decode_block", batch=8, context=20000, window=0, padded=False, **llama),
        # one very long context
        dict(name="decode 1x128K", op="decode_block", batch=1, context=131072, window=0, padded=False, hq=64, hkv=8,
             d=128),
        # a sliding-window layer in a batch padded with an empty slot
        dict(name="decode 9x16K window 128", op="decode_block", batch=9, context=16001, window=128, padded=True, hq=64,
             hkv=8, d=64),
        # a few drafted tokens of each sequence checked at once: one query tile, the keys split over many CTAs
        dict(name="prefill 8x20K chunk 9", op="prefill_block", batch=8, context=20000, chunk=9, window=0, **llama),
        # chunked prefill of the serving batch
        dict(name="prefill 8x20K chunk 512", op="prefill_block", batch=8, context=20000, chunk=512, window=0, **llama),
        # a wide-head sliding-window layer, ragged chunks of an odd size
        dict(name="prefill 4x9K d256", op="prefill_block", batch=4, context=9001, chunk=777, window=512, hq=8, hkv=1,
             d=256),
    ]


LAYOUTS = [(32, 8, 128), (64, 8, 64), (8, 1, 256), (64, 8, 128), (16, 16, 64), (16, 8, 128), (32, 2, 128)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_append", "rope_append_block", "decode_block", "prefill_block"])
    hq, hkv, d = rng.choice(LAYOUTS)
    case = dict(op=op, hq=hq, hkv=hkv, d=d)
    if op in ("rope_append", "rope_append_block"):
        case.update(axes=rng.choice([1, 1, 2, 3]), style=rng.choice(["halves", "pairs"]),
                    rotary=rng.choice([d, d, d // 2, d // 4]))
        most = min(16000, 65536000 // (hq * d + 2 * hkv * d))
        if op == "rope_append":
            case.update(tokens=_log(rng, 1, most), fmt=rng.choice(["e4m3", "e5m2", "bf16"]))
        elif rng.random() < 0.4:
            case.update(batch=_log(rng, 1, 256), chunk=1)
        else:
            batch = rng.randint(1, 16)
            case.update(batch=batch, chunk=_log(rng, 2, most // batch))
    elif op == "decode_block":
        batch = _log(rng, 1, 64)
        most = min(131072, 330_000_000 // (2 * hkv * d) // batch)
        case.update(batch=batch, context=_log(rng, 40, max(41, most)), window=rng.choice([0, 0, 128, 512]),
                    padded=rng.random() < 0.3 and batch > 1)
    else:
        batch = rng.randint(1, 8)
        context = _log(rng, 300, 20000)
        most = min(1024, context // 2, 2_600_000_000 // (batch * context * hq * d // 128))
        case.update(batch=batch, context=context, chunk=_log(rng, 2, max(3, most)), window=rng.choice([0, 0, 128, 1000]))
    return case


def _spread(mean, n, part):
    """n whole numbers evenly spaced in mean * (1 +- part): ragged, with a sum that the case alone fixes."""
    if n == 1:
        return [mean]
    return [max(1, int(round(mean * (1 - part + 2 * part * i / (n - 1))))) for i in range(n)]


def _contexts(case):
    if case["op"] == "rope_append_block":
        # a short history in front of each chunk: the append touches the newest pages only
        return [n + 5 + 7 * i for i, n in enumerate(_chunks(case))]
    lens = _spread(case["context"], case["batch"], 0.1)
    if case.get("padded"):
        lens[-1] = 0
    return lens


def _chunks(case):
    return _spread(case["chunk"], case["batch"], 0.5)


# ------------------------------------------------------------------ inputs

def _sections(case):
    """Axis of each frequency: the axes interleaved over the frequencies."""
    return torch.arange(case["rotary"] // 2) % case["axes"]


def _rope_inputs(case, g, dev, first, counts):
    """inv_freq, axis of each frequency and positions [axes, T] of the new tokens: a text position, and for more axes
    the row and column of an image patch."""
    half = case["rotary"] // 2
    inv_freq = (500000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(dev)
    pos = torch.cat([torch.arange(n) + f for f, n in zip(first, counts)]).to(torch.int32)
    pos = torch.stack([pos] + [pos // 37 + 1, pos % 37][: case["axes"] - 1]).to(dev)
    return inv_freq, _sections(case).to(torch.uint8).to(dev), pos.contiguous()


def _projected(case, T, g, dev):
    """q, k and v of T tokens as the slices of one fused projection's output, with a few large channels in k."""
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    x = torch.randn((T, (hq + 2 * hkv) * d), generator=g, device=dev)
    big = torch.randint(0, d, (hkv, 2), generator=g, device=dev) + torch.arange(hkv, device=dev)[:, None] * d + hq * d
    x[:, big.reshape(-1)] *= 6.0
    x = x.to(torch.bfloat16)
    return (x[:, : hq * d].unflatten(1, (hq, d)), x[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
            x[:, (hq + hkv) * d:].unflatten(1, (hkv, d)))


def _codes(shape, g, dev):
    """E4M3 codes of unit-normal data that fills the format."""
    x = torch.randn(shape, generator=g, device=dev).mul_(100.0).clamp_(-E4M3_MAX, E4M3_MAX)
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _block_cache(case, lens, g, dev):
    """A block-scaled cache holding the sequences, pages in random order: pages differ in scale as their tokens do."""
    hkv, d = case["hkv"], case["d"]
    pages = [-(-n // PAGE) for n in lens]
    nb = sum(pages) + 3
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(int(torch.randint(0, 2**31, (1,), generator=g,
                                                                                        device=dev))))
    tables = torch.nn.utils.rnn.pad_sequence(perm[: sum(pages)].split(pages), batch_first=True).to(torch.int32)
    shape = (nb, hkv, PAGE, d)
    k, v = _codes(shape, g, dev), _codes(shape, g, dev)
    ks, vs = (0.01 * 2.0 ** (2 * torch.rand((nb, hkv), generator=g, device=dev) - 1) for _ in range(2))
    return k, v, ks, vs, tables.to(dev)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    order = torch.Generator().manual_seed(seed)
    op, d = case["op"], case["d"]
    s = dict(case=case, sm=1.0 / math.sqrt(d))
    if op == "rope_append":
        T, hkv = case["tokens"], case["hkv"]
        nb = -(-T // PAGE) + 5
        s["q"], s["k"], s["v"] = _projected(case, T, g, dev)
        s["inv_freq"], s["axis"], s["pos"] = _rope_inputs(case, g, dev, [20000], [T])
        s["slots"] = torch.randperm(nb * PAGE, generator=order)[:T].to(dev)
        shape = (nb, hkv, PAGE, d)
        for name in ("k_cache", "v_cache"):
            s[name] = (torch.randn(shape, generator=g, device=dev).to(torch.bfloat16) if case["fmt"] == "bf16"
                       else _codes(shape, g, dev))
        # calibrated per-tensor scales: the tensor's largest value at the format's maximum
        top = {"e4m3": E4M3_MAX, "e5m2": E5M2_MAX, "bf16": None}[case["fmt"]]
        s["k_scale"], s["v_scale"] = (30.0 / top, 5.0 / top) if top else (1.0, 1.0)
        s["q_out"] = torch.empty((T, case["hq"], d), dtype=torch.bfloat16, device=dev)
        return s
    mix = torch.randperm(case["batch"], generator=order).tolist()
    lens = [_contexts(case)[i] for i in mix]
    s["max_len"] = max(lens)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["tables"] = _block_cache(case, lens, g, dev)
    if op == "decode_block":
        s["q"] = torch.randn((case["batch"], case["hq"], d), generator=g, device=dev).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        return s
    counts = [_chunks(case)[i] for i in mix]
    T = sum(counts)
    s["max_q"] = max(counts)
    s["starts"] = torch.tensor([0] + counts, dtype=torch.int32, device=dev).cumsum(0, dtype=torch.int32)
    if op == "prefill_block":
        s["q"] = torch.randn((T, case["hq"], d), generator=g, device=dev).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        return s
    s["q"], s["k"], s["v"] = _projected(case, T, g, dev)
    s["inv_freq"], s["axis"], s["pos"] = _rope_inputs(case, g, dev, [n - c for n, c in zip(lens, counts)], counts)
    s["q_out"] = torch.empty((T, case["hq"], d), dtype=torch.bfloat16, device=dev)
    return s


# ------------------------------------------------------------------ plain forms

def _rotated(x, s):
    """x [T, H, d] in 32 bits, rotated; angles in 64 bits (a position of 20,000 times a frequency of 1 loses its
    fraction in 32)."""
    R, x = s["case"]["rotary"], x.float()
    angle = s["pos"].double()[s["axis"].long()].T * s["inv_freq"].double()
    c, n = angle.cos().float()[:, None], angle.sin().float()[:, None]
    y = x.clone()
    first, second = ((slice(0, R, 2), slice(1, R, 2)) if s["case"]["style"] == "pairs"
                     else (slice(0, R // 2), slice(R // 2, R)))
    y[..., first] = x[..., first] * c - x[..., second] * n
    y[..., second] = x[..., second] * c + x[..., first] * n
    return y


def _to_format(x, fmt):
    """The cache's rounding of values that are already divided by their scale, as the bytes (or bf16) it holds."""
    if fmt == "bf16":
        return x.to(torch.bfloat16)
    top, kind = (E4M3_MAX, torch.float8_e4m3fn) if fmt == "e4m3" else (E5M2_MAX, torch.float8_e5m2)
    return x.clamp(-top, top).to(kind).view(torch.uint8)


def _as_values(cache, fmt):
    return cache if fmt == "bf16" else cache.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2)


def _plain_rope_append(s):
    fmt = s["case"]["fmt"]
    s["q_out"].copy_(_rotated(s["q"], s))
    at = (s["slots"] // PAGE, slice(None), s["slots"] % PAGE)
    s["k_cache"][at] = _to_format(_rotated(s["k"], s) / s["k_scale"], fmt)
    s["v_cache"][at] = _to_format(s["v"].float() / s["v_scale"], fmt)
    return _answer_rope_append(s)


def _answer_rope_append(s):
    fmt = s["case"]["fmt"]
    return {"q": s["q_out"], "k": _as_values(s["k_cache"], fmt), "v": _as_values(s["v_cache"], fmt)}


def _least_power(amax):
    """The least power of two 2^e, e in [EXP_LO, EXP_HI], with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, x = torch.frexp(amax)
    e = torch.where(amax > 0, x - 9 + (m > 0.875), torch.full_like(x, EXP_LO)).clamp(EXP_LO, EXP_HI)
    return torch.ldexp(torch.ones_like(amax), e)


def _rows(s):
    """Sequence and place in it of every new token."""
    t = torch.arange(s["q"].shape[0], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["starts"], t, right=True) - 1
    n = s["starts"].diff()
    return b, (s["lens"] - n)[b] + t - s["starts"][b], n


def _plain_append_one(s, x, cache, scales):
    """x [T, H, d] in 32 bits into the block-scaled cache."""
    b, p, n = _rows(s)
    page = s["tables"][b, p // PAGE].long()
    amax = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    new = torch.full_like(scales, -1.0).scatter_reduce_(0, page[:, None].expand_as(amax), amax, "amax")
    # each sequence's first touched page may hold older rows, which keep their scale if the new rows fit
    first = s["lens"] - n
    held = s["tables"][torch.arange(len(first), device="cuda"), first // PAGE].long()
    old = torch.zeros_like(scales)
    old[held] = torch.where((first % PAGE > 0)[:, None], scales[held], 0.0)
    grown = torch.where((old > 0) & (new <= E4M3_MAX * old), old, torch.maximum(old, _least_power(new)))
    scale = torch.where(new >= 0, grown, scales)
    rows = cache[held]
    again = _to_format(rows.view(torch.float8_e4m3fn).float() * (scales[held] / scale[held])[..., None, None], "e4m3")
    keep = (torch.arange(PAGE, device="cuda") >= (first % PAGE)[:, None])[:, None, :, None]
    cache[held] = torch.where(keep, rows, again)
    cache[page, :, (p % PAGE).long()] = _to_format(x / scale[page][..., None], "e4m3")
    scales.copy_(scale)


def _plain_rope_append_block(s):
    s["q_out"].copy_(_rotated(s["q"], s))
    _plain_append_one(s, _rotated(s["k"], s), s["k_cache"], s["k_scales"])
    _plain_append_one(s, s["v"].float(), s["v_cache"], s["v_scales"])
    return _answer_rope_append_block(s)


def _answer_rope_append_block(s):
    return {"q": s["q_out"], "k": _as_values(s["k_cache"], "e4m3"), "v": _as_values(s["v_cache"], "e4m3"),
            "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _gathered(s, rows):
    """K and V in 32 bits, [B, Hkv, tokens, d], of the pages that the last `rows` tokens of each sequence may attend,
    and the position of each token, [B, tokens]."""
    case, tables = s["case"], s["tables"].long()
    first, count = torch.zeros_like(s["lens"]), tables.shape[1]
    if case["window"]:
        first = (s["lens"] - rows + 1 - case["window"]).clamp_min(0) // PAGE
        count = min(count, (case["window"] + rows) // PAGE + 2)
    page = first[:, None] + torch.arange(count, device="cuda")
    ids = tables.gather(1, page.clamp_max(tables.shape[1] - 1))
    k, v = (((s[c + "_cache"][ids].view(torch.float8_e4m3fn).float() * s[c + "_scales"][ids][..., None, None])
             .transpose(1, 2).flatten(2, 3)) for c in "kv")
    return k, v, (page[..., None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(1)


def _weighted(scores, mask, v):
    """softmax over the last axis where the mask is true (zeros where it leaves nothing), times v."""
    scores.masked_fill_(~mask, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return (p @ v).div_(total.clamp_min(torch.finfo(torch.float32).tiny))


def _plain_decode_block(s):
    case, lens = s["case"], s["lens"].long()
    k, v, t = _gathered(s, 1)
    q = s["q"].float().unflatten(1, (case["hkv"], -1))
    mask = t < lens[:, None]
    if case["window"]:
        mask &= t >= lens[:, None] - case["window"]
    o = _weighted((q @ k.transpose(-1, -2)).mul_(s["sm"]), mask[:, None, None], v)
    return s["out"].copy_(o.flatten(1, 2))


def _plain_prefill_block(s):
    case = s["case"]
    k, v, t = _gathered(s, s["max_q"])
    starts, lens = s["starts"].long(), s["lens"].long()
    n = starts.diff()
    i = torch.arange(s["max_q"], device="cuda")
    q = s["q"][(starts[:-1, None] + i).clamp_max(s["q"].shape[0] - 1)].float()       # [B, rows, Hq, d]
    q = q.unflatten(2, (case["hkv"], -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)        # [B, Hkv, g * rows, d]
    p = ((lens - n)[:, None] + i)[..., None]
    t = t[:, None]
    mask = t <= p
    if case["window"]:
        mask &= t > p - case["window"]
    mask = mask[:, None].expand(-1, case["hq"] // case["hkv"], -1, -1).flatten(1, 2)[:, None]
    o = _weighted((q @ k.transpose(-1, -2)).mul_(s["sm"]), mask, v)
    o = o.unflatten(2, (-1, s["max_q"])).permute(0, 3, 1, 2, 4).flatten(2, 3)         # [B, rows, Hq, d]
    b, place, _ = _rows(s)
    return s["out"].copy_(o[b, place - (lens - n)[b]])


# ------------------------------------------------------------------ the library's calls

def _own_workspace(s, make):
    """The caller-owned workspace, allocated once for a state, as a serving loop does."""
    if "workspace" not in s:
        s["workspace"] = make()
    return s["workspace"]


def _own_rope_append(s):
    from fp8_kv_cache_fp8kv_gb300 import binding as fk
    case = s["case"]
    fmt = {"e4m3": fk.CACHE_E4M3, "e5m2": fk.CACHE_E5M2, "bf16": fk.CACHE_BF16}[case["fmt"]]
    fk.fp8kv_rope_append(s["q"], s["k"], s["v"], s["pos"], s["inv_freq"], s["slots"], s["q_out"], s["k_cache"],
                         s["v_cache"], s["k_scale"], s["v_scale"], freq_axis=s["axis"],
                         style=fk.ROPE_PAIRS if case["style"] == "pairs" else fk.ROPE_HALVES, cache_format=fmt)
    return _answer_rope_append(s)


def _own_rope_append_block(s):
    from fp8_kv_cache_fp8kv_gb300 import binding as fk
    case = s["case"]
    ws = _own_workspace(s, fk.alloc_append_workspace)
    fk.fp8kv_rope_append_block(s["q"], s["k"], s["v"], s["pos"], s["inv_freq"], s["q_out"], s["k_cache"], s["v_cache"],
                               s["k_scales"], s["v_scales"], s["tables"], s["lens"], s["starts"], s["max_len"], ws,
                               freq_axis=s["axis"],
                               style=fk.ROPE_PAIRS if case["style"] == "pairs" else fk.ROPE_HALVES)
    return _answer_rope_append_block(s)


def _own_decode_block(s):
    from fp8_kv_cache_fp8kv_gb300 import binding as fk
    case = s["case"]
    ws = _own_workspace(s, lambda: fk.alloc_workspace(case["batch"], case["hq"], case["hkv"], case["d"], s["max_len"],
                                                      PAGE, case["window"]))
    fk.fp8kv_paged_decode_block(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["tables"], s["lens"],
                                s["max_len"], s["sm"], case["window"], s["out"], ws)
    return s["out"]


def _own_prefill_block(s):
    from fp8_kv_cache_fp8kv_gb300 import binding as fk
    case = s["case"]
    ws = _own_workspace(s, lambda: fk.alloc_prefill_workspace(case["batch"], s["max_q"], s["max_len"], case["hq"],
                                                              case["hkv"], case["d"], PAGE, case["window"]))
    fk.fp8kv_paged_prefill_block(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["tables"],
                                 s["lens"], s["starts"], s["max_q"], s["max_len"], s["sm"], case["window"], s["out"], ws)
    return s["out"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope_append": _own_rope_append, "rope_append_block": _own_rope_append_block,
                "decode_block": _own_decode_block, "prefill_block": _own_prefill_block}[op](state)
    return {"rope_append": _plain_rope_append, "rope_append_block": _plain_rope_append_block,
            "decode_block": _plain_decode_block, "prefill_block": _plain_prefill_block}[op](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    hq, hkv, d, op = case["hq"], case["hkv"], case["d"], case["op"]
    if op in ("rope_append", "rope_append_block"):
        block = op == "rope_append_block"
        T = sum(_chunks(case)) if block else case["tokens"]
        each = 2 if case.get("fmt") == "bf16" else 1
        moved = T * (2 * hq * d * 2 + 2 * hkv * d * (2 + each) + 4 * case["axes"])
        if block:
            pages = sum((n - 1) // PAGE - (n - c) // PAGE + 1 for n, c in zip(_contexts(case), _chunks(case)))
            moved += pages * (hkv * 8 + 4)
        else:
            moved += T * 8
        return {"bytes": moved, "flops": T * (hq + hkv) * case["rotary"] * 3}
    window = case["window"]
    if op == "decode_block":
        tokens = pages = 0
        for n in _contexts(case):
            lo = max(0, n - window) if window else 0
            tokens += n - lo
            pages += (n - 1) // PAGE - lo // PAGE + 1 if n else 0
        rows = case["batch"]
        pairs = tokens
    else:
        tokens = pages = pairs = 0
        for n, c in zip(_contexts(case), _chunks(case)):
            lo = max(0, n - c + 1 - window) if window else 0
            tokens += n - lo
            pages += (n - 1) // PAGE - lo // PAGE + 1
            pairs += sum(min(p + 1, window) if window else p + 1 for p in range(n - c, n))
        rows = sum(_chunks(case))
    return {"bytes": tokens * 2 * hkv * d + pages * (hkv * 8 + 4) + rows * hq * d * 4, "flops": 4 * hq * d * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits

def _nearest(x, digits, least, top):
    """x rounded to `digits` binary digits after the leading one, half to even, no finer than 2^(least - digits),
    at most top in magnitude."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp_min(least) - digits)
    return torch.round(x / step).mul_(step).clamp_(-top, top)


_E4M3, _E5M2 = (3, -6, E4M3_MAX), (2, -14, E5M2_MAX)


def _turned(x, s):
    """The rotation as a product of complex numbers."""
    R, x = s["case"]["rotary"], x.double()
    angle = torch.stack([s["pos"][a].double() for a in _sections(s["case"]).tolist()], 1) * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    head = x[..., :R]
    if s["case"]["style"] == "pairs":
        z = torch.complex(head[..., 0::2].contiguous(), head[..., 1::2].contiguous()) * turn
        head = torch.stack((z.real, z.imag), -1).flatten(-2)
    else:
        z = torch.complex(head[..., :R // 2].contiguous(), head[..., R // 2:].contiguous()) * turn
        head = torch.cat((z.real, z.imag), -1)
    return torch.cat((head, x[..., R:]), -1)


def _exact_page(cache, scales, page, r0, rows):
    """rows [Hkv, count, d] in 64 bits appended behind r0 older rows of a page, in place."""
    power = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((1, 2)) / E4M3_MAX)).clamp(EXP_LO, EXP_HI))
    scale = power
    if r0:
        old = scales[page]
        scale = torch.where(rows.abs().amax((1, 2)) <= E4M3_MAX * old, old, torch.maximum(old, power))
        cache[page, :, :r0] = _nearest(cache[page, :, :r0] * (old / scale)[:, None, None], *_E4M3)
    cache[page, :, r0:r0 + rows.shape[1]] = _nearest(rows / scale[:, None, None], *_E4M3)
    scales[page] = scale


def _exact_head(s, b, h, q, first):
    """Query rows q [R, g, d] of sequence b and kv head h, the first at position `first`."""
    n, window = int(s["lens"][b]), s["case"]["window"]
    ids = s["tables"][b, : -(-n // PAGE)].long()
    at = first + torch.arange(q.shape[0], device=q.device)[:, None]
    t = torch.arange(n, device=q.device)
    seen = (t <= at) & (t > at - window) if window else t <= at
    k, v = ((s[c + "_cache"][ids, h].view(torch.float8_e4m3fn).double() * s[c + "_scales"][ids, h].double()[:, None, None])
            .flatten(0, 1)[:n] for c in "kv")
    z = torch.einsum("rgd,td->grt", q.double(), k).mul_(s["sm"]).masked_fill_(~seen, -math.inf)
    return torch.einsum("grt,td->rgd", torch.softmax(z, -1), v)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("rope_append", "rope_append_block"):
        out = {"q": _turned(s["q"], s)}
    if op == "rope_append":
        kind = {"e4m3": _E4M3, "e5m2": _E5M2, "bf16": None}[case["fmt"]]
        for name, x in (("k", _turned(s["k"], s)), ("v", s["v"].double())):
            cache = _as_values(s[name + "_cache"], case["fmt"]).double()
            flat = cache.transpose(1, 2).flatten(0, 1)                       # [slots, Hkv, d]
            scale = float(torch.tensor(s[name + "_scale"], dtype=torch.float32))
            flat[s["slots"]] = x if kind is None else _nearest(x / scale, *kind)
            out[name] = flat.unflatten(0, (-1, PAGE)).transpose(1, 2).contiguous()
        return out
    lens, starts = s["lens"].tolist(), s["starts"].tolist() if "starts" in s else list(range(case["batch"] + 1))
    counts = [b - a for a, b in zip(starts, starts[1:])]
    if op == "rope_append_block":
        tables = s["tables"].tolist()
        for name, x in (("k", _turned(s["k"], s)), ("v", s["v"].double())):
            cache, scales = _as_values(s[name + "_cache"], "e4m3").double(), s[name + "_scales"].double()
            for b, (n, c) in enumerate(zip(lens, counts)):
                p = n - c
                while p < n:
                    count = min(PAGE - p % PAGE, n - p)
                    at = starts[b] + p - (n - c)
                    _exact_page(cache, scales, tables[b][p // PAGE], p % PAGE, x[at:at + count].transpose(0, 1))
                    p += count
            out[name], out[name + "_scales"] = cache, scales
        return out
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["hq"] // case["hkv"]
    for b, (n, c) in enumerate(zip(lens, counts)):
        for h in range(case["hkv"] if n else 0):
            heads = slice(h * group, (h + 1) * group)
            out[starts[b]:starts[b + 1], heads] = _exact_head(s, b, h, s["q"][starts[b]:starts[b + 1], heads], n - c)
    return out

"""The rotary append and the block-scaled calls without a GPU: the C ABI
refuses bad arguments before it touches the device, and the binding refuses
shapes that do not fit and tensors that are not on one."""
import ctypes

import pytest
import torch

from fp8_kv_cache_fp8kv_gb300 import binding as fk
from fp8_kv_cache_fp8kv_gb300 import build as fbuild

FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: every call below fails validation first
OFF1, OFF2, OFF4, OFF16 = (ctypes.c_void_p(0x10000 + n) for n in (1, 2, 4, 16))


@pytest.fixture(scope="module", autouse=True)
def lib():
    fbuild.build()
    return fk.load()


def _append(lib, **kw):
    a = dict(q=FAKE, qs=4096, qo=FAKE, k=FAKE, ks=1024, v=FAKE, vs=1024, pos=FAKE, ax=1, f=FAKE, fa=None, R=128,
             style=0, slots=FAKE, T=4, kc=FAKE, vc=FAKE, nb=10, bs=16, hq=32, hkv=8, d=128, fmt=0, sk=0.5, sv=0.5,
             hk=None, hv=None)
    a.update(kw)
    return lib.fp8kv_rope_append(a["q"], a["qs"], a["qo"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["ax"],
                                 a["f"], a["fa"], a["R"], a["style"], a["slots"], a["T"], a["kc"], a["vc"], a["nb"],
                                 a["bs"], a["hq"], a["hkv"], a["d"], a["fmt"], a["sk"], a["sv"], a["hk"], a["hv"],
                                 None)


BAD_ROWS = [
    (dict(q=None), 1), (dict(qo=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(q=OFF2), 1), (dict(qo=OFF2), 1),
    (dict(k=OFF2), 1), (dict(v=OFF2), 1), (dict(qs=4095), 1), (dict(qs=4088), 1), (dict(ks=1016), 1),
    (dict(vs=1025), 1), (dict(vs=0), 1), (dict(ks=-1024), 1), (dict(ks=1 << 62), 1), (dict(qs=4104), 1),
    (dict(d=96), 2), (dict(d=512), 2), (dict(R=24), 2), (dict(R=144), 1), (dict(R=-16), 1), (dict(style=2), 1),
    (dict(style=-1), 1), (dict(ax=0), 1), (dict(ax=5), 1), (dict(f=None), 1), (dict(f=OFF2), 1), (dict(pos=OFF2), 1),
    (dict(T=-1), 1), (dict(nb=0), 1), (dict(hkv=0), 1), (dict(hq=-1), 1), (dict(hq=0), 1), (dict(hkv=70000), 1),
]


@pytest.mark.parametrize("kw,code", BAD_ROWS + [
    (dict(T=1 << 31), 2), (dict(pos=None), 1), (dict(bs=0), 1), (dict(fmt=3), 1), (dict(fmt=-1), 1), (dict(sk=0.0), 1),
    (dict(sv=float("nan")), 1), (dict(hk=FAKE), 1), (dict(hv=FAKE), 1), (dict(hk=OFF2, hv=FAKE), 1),
    (dict(fmt=2), 1), (dict(fmt=2, sk=1.0, sv=1.0, hk=FAKE, hv=FAKE), 1), (dict(kc=None), 1), (dict(vc=OFF4), 1),
    (dict(slots=None), 1), (dict(slots=OFF4), 1), (dict(nb=1 << 58), 1),
    (dict(T=0, q=None, k=None, v=None, slots=None, kc=None), 0),
])
def test_rope_append_validates(lib, kw, code):
    # q == q_out needs contiguous queries: the one listed stride above a row is refused for that
    assert _append(lib, **kw) == code


def _block(lib, **kw):
    a = dict(q=FAKE, qs=4096, qo=FAKE, k=FAKE, ks=1024, v=FAKE, vs=1024, T=4, pos=FAKE, ax=1, f=FAKE, fa=None, R=128,
             style=0, kc=FAKE, vc=FAKE, sk=FAKE, sv=FAKE, nb=10, bt=FAKE, mb=8, sl=FAKE, st=FAKE, msl=128, B=2, hq=32,
             hkv=8, d=128, bs=16, ws=FAKE, wsb=256)
    a.update(kw)
    return lib.fp8kv_rope_append_block(a["q"], a["qs"], a["qo"], a["k"], a["ks"], a["v"], a["vs"], a["T"], a["pos"],
                                       a["ax"], a["f"], a["fa"], a["R"], a["style"], a["kc"], a["vc"], a["sk"],
                                       a["sv"], a["nb"], a["bt"], a["mb"], a["sl"], a["st"], a["msl"], a["B"],
                                       a["hq"], a["hkv"], a["d"], a["bs"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", BAD_ROWS + [
    (dict(bs=32), 2), (dict(nb=1 << 31), 2), (dict(nb=1 << 29), 2), (dict(T=1 << 31), 2), (dict(B=-1), 1),
    (dict(B=65536), 1), (dict(msl=-1), 1), (dict(msl=129), 1), (dict(mb=-1), 1), (dict(st=None), 1),
    (dict(pos=None, ax=2), 1), (dict(kc=None), 1), (dict(vc=OFF4), 1), (dict(sk=None), 1), (dict(sv=OFF2), 1),
    (dict(bt=None), 1), (dict(bt=OFF2), 1), (dict(sl=None), 1), (dict(st=OFF2), 1), (dict(ws=None), 3),
    (dict(ws=OFF16), 3), (dict(wsb=255), 3), (dict(B=0, T=0, st=None), 0), (dict(T=0, k=None), 0),
    (dict(msl=0, mb=0, k=None), 0),
])
def test_rope_append_block_validates(lib, kw, code):
    assert _block(lib, **kw) == code


def _decode(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, nb=100, bt=FAKE, mb=8, sl=FAKE, msl=128, B=2, hq=32, hkv=8,
             d=128, bs=16, sm=0.088, win=0, out=FAKE, ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return lib.fp8kv_paged_decode_block(a["q"], a["k"], a["v"], a["ks"], a["vs"], a["nb"], a["bt"], a["mb"], a["sl"],
                                        a["msl"], a["B"], a["hq"], a["hkv"], a["d"], a["bs"], a["sm"], a["win"],
                                        a["out"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(ks=None), 1), (dict(vs=None), 1), (dict(ks=OFF2), 1), (dict(vs=OFF1), 1), (dict(d=96), 2), (dict(bs=32), 2),
    (dict(hq=30), 1), (dict(hq=256), 2), (dict(sm=float("inf")), 1), (dict(q=None), 1), (dict(q=OFF2), 1),
    (dict(k=OFF4), 1), (dict(out=None), 1), (dict(bt=None), 1), (dict(sl=OFF2), 1), (dict(mb=4), 1), (dict(nb=0), 1),
    (dict(nb=1 << 31), 2), (dict(B=-1), 1), (dict(B=70000), 1), (dict(B=0, q=None, ks=None, out=None), 0),
])
def test_decode_block_validates(lib, kw, code):
    assert _decode(lib, **kw) == code


def _prefill(lib, **kw):
    a = dict(q=FAKE, T=64, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, nb=100, bt=FAKE, mb=8, sl=FAKE, qs=FAKE, mq=64, msl=128,
             B=2, hq=32, hkv=8, d=128, bs=16, sm=0.088, win=0, out=FAKE, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return lib.fp8kv_paged_prefill_block(a["q"], a["T"], a["k"], a["v"], a["ks"], a["vs"], a["nb"], a["bt"], a["mb"],
                                         a["sl"], a["qs"], a["mq"], a["msl"], a["B"], a["hq"], a["hkv"], a["d"],
                                         a["bs"], a["sm"], a["win"], a["out"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(ks=None), 1), (dict(vs=None), 1), (dict(ks=OFF2), 1), (dict(d=96), 2), (dict(bs=32), 2), (dict(hq=30), 1),
    (dict(hq=256), 2), (dict(sm=float("nan")), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(qs=None), 1),
    (dict(mb=4), 1), (dict(mq=200), 1), (dict(mq=-1), 1), (dict(T=-1), 1), (dict(nb=1 << 31), 2),
    (dict(B=0, q=None, ks=None), 0), (dict(mq=0, ks=None), 0), (dict(T=0, ks=None), 0),
])
def test_prefill_block_validates(lib, kw, code):
    assert _prefill(lib, **kw) == code


def test_stall_hook_validates(lib):
    f = lib.fp8kv_debug_paged_prefill_block_stall
    a = [FAKE, 64, FAKE, FAKE, FAKE, FAKE, 100, FAKE, 8, FAKE, FAKE, 64, 128, 2, 32, 8, 128, 16, 0.088, 0, FAKE, FAKE,
         1 << 30, None]
    assert f(*a, -1, 1000) == 1 and f(*a, 0, 0) == 1 and f(*a, 0, 500_000_001) == 1
    a[16] = 96
    assert f(*a, 0, 1000) == 2


# ------------------------------------------------------------------ the binding

def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _append_args(**kw):
    a = dict(q=_bf(6, 4, 64), k_new=_bf(6, 2, 64), v_new=_bf(6, 2, 64), positions=_i32(6),
             inv_freq=torch.zeros(32), slot_mapping=torch.zeros(6, dtype=torch.int64), q_out=_bf(6, 4, 64),
             k_cache=torch.zeros((3, 2, 16, 64), dtype=torch.uint8),
             v_cache=torch.zeros((3, 2, 16, 64), dtype=torch.uint8))
    a.update(kw)
    return a


def _block_args(**kw):
    a = _append_args(k_scales=torch.zeros((3, 2)), v_scales=torch.zeros((3, 2)), block_tables=_i32(2, 4),
                     seq_lens=_i32(2), q_starts=_i32(3), max_seq_len=64, workspace=torch.zeros(256, dtype=torch.uint8))
    del a["slot_mapping"]
    a.update(kw)
    return a


@pytest.mark.parametrize("kw", [
    dict(k_new=_bf(6, 3, 64)), dict(v_new=_bf(5, 2, 64)), dict(q=_bf(5, 4, 64)), dict(q=_bf(6, 4, 32)),
    dict(q_out=_bf(6, 3, 64)), dict(q_out=None), dict(q=None),
    dict(v_cache=torch.zeros((4, 2, 16, 64), dtype=torch.uint8)),
])
@pytest.mark.parametrize("block", [False, True])
def test_appends_refuse_mismatched_shapes(kw, block):
    # (rows that fit reach the device check first: either refusal is one)
    with pytest.raises((ValueError, TypeError)):
        (fk.fp8kv_rope_append_block if block else fk.fp8kv_rope_append)(**(_block_args if block else _append_args)(**kw))


def test_rope_arguments_are_checked():
    f = fk._rope_args
    assert f(None, None, None, 64, 6, 0)[4] == 0
    for bad in (dict(positions=_i32(5)), dict(positions=_i32(2, 5)), dict(positions=_i32(1, 2, 6)),
                dict(inv_freq=torch.zeros(33)), dict(freq_axis=torch.zeros(31, dtype=torch.uint8))):
        a = dict(positions=None, inv_freq=torch.zeros(32), freq_axis=None)
        a.update(bad)
        with pytest.raises(ValueError):
            f(a["positions"], a["inv_freq"], a["freq_axis"], 64, 6, 0)


def test_host_tensors_are_refused():
    with pytest.raises(TypeError):
        fk.fp8kv_rope_append(**_append_args())
    with pytest.raises(TypeError):
        fk.fp8kv_rope_append_block(**_block_args())
    q, kc = _bf(2, 4, 64), torch.zeros((3, 2, 16, 64), dtype=torch.uint8)
    sc, ws = torch.zeros((3, 2)), torch.zeros(1024, dtype=torch.uint8)
    with pytest.raises(TypeError):
        fk.fp8kv_paged_decode_block(q, kc, kc, sc, sc, _i32(2, 4), _i32(2), 64, 0.1, 0, _bf(2, 4, 64), ws)
    with pytest.raises(TypeError):
        fk.fp8kv_paged_prefill_block(q, kc, kc, sc, sc, _i32(2, 4), _i32(2), _i32(3), 1, 64, 0.1, 0, _bf(2, 4, 64), ws)
    for bad in (torch.zeros((3, 3)), torch.zeros(3), torch.zeros((4, 2))):
        with pytest.raises(ValueError):
            fk.fp8kv_paged_decode_block(q, kc, kc, bad, sc, _i32(2, 4), _i32(2), 64, 0.1, 0, _bf(2, 4, 64), ws)
        with pytest.raises(ValueError):
            fk.fp8kv_paged_prefill_block(q, kc, kc, sc, bad, _i32(2, 4), _i32(2), _i32(3), 1, 64, 0.1, 0,
                                         _bf(2, 4, 64), ws)


def test_work_units_of_the_block_append_never_meet():
    """Sequence b owns the CTA indices [q_starts[b] / 16 + 2b, q_starts[b + 1] / 16 + 2(b + 1)): at least as many as
    the pages its tokens touch, and the last index is inside the grid of num_tokens / 16 + 2 batch."""
    g = torch.Generator().manual_seed(0)
    for _ in range(300):
        B = int(torch.randint(1, 9, (1,), generator=g))
        n = torch.randint(0, 50, (B,), generator=g).tolist()
        hist = torch.randint(0, 40, (B,), generator=g).tolist()
        starts = [int(torch.randint(0, 20, (1,), generator=g))]
        for x in n:
            starts.append(starts[-1] + x)
        T = starts[-1] + int(torch.randint(0, 20, (1,), generator=g))
        for b in range(B):
            pages = (hist[b] + n[b] - 1) // 16 - hist[b] // 16 + 1 if n[b] else 0
            first, after = starts[b] // 16 + 2 * b, starts[b + 1] // 16 + 2 * (b + 1)
            assert first + pages <= after <= T // 16 + 2 * B

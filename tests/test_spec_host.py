"""Drafted trees, attention weights and eviction without a GPU: the C ABI refuses bad arguments before it touches the device, the binding refuses
shapes that do not fit and tensors that are not on one, and the cut of a tree's work over CTAs is whole."""
import ctypes
import os
import subprocess

import pytest
import torch

from fp8_kv_cache_fp8kv_gb300 import binding as fk
from fp8_kv_cache_fp8kv_gb300 import build as fbuild

FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: every call below fails validation first
OFF2, OFF4 = ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10004)


@pytest.fixture(scope="module", autouse=True)
def lib():
    fbuild.build()
    return fk.load()


def _tree(lib, **kw):
    a = dict(q=FAKE, T=20, k=FAKE, v=FAKE, nb=100, bt=FAKE, mb=8, sl=FAKE, st=FAKE, par=FAKE, n=16, msl=128, B=2, hq=32,
             hkv=8, d=128, bs=16, fmt=0, ks=0.5, vs=0.5, hk=None, hv=None, sm=0.1, win=0, out=FAKE, ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return lib.fp8kv_paged_tree_attention(
        a["q"], a["T"], a["k"], a["v"], a["nb"], a["bt"], a["mb"], a["sl"], a["st"], a["par"], a["n"], a["msl"], a["B"],
        a["hq"], a["hkv"], a["d"], a["bs"], a["fmt"], a["ks"], a["vs"], a["hk"], a["hv"], a["sm"], a["win"], a["out"],
        a["ws"], a["wsb"], None)


SHAPES = [(dict(d=96), 2), (dict(d=512), 2), (dict(bs=32), 2), (dict(B=-1), 1), (dict(B=65536), 1), (dict(nb=0), 1),
          (dict(nb=1 << 31), 2), (dict(nb=1 << 29), 2), (dict(mb=-1), 1), (dict(msl=-1), 1), (dict(msl=129), 1),
          (dict(hkv=0), 1), (dict(hkv=70000), 1), (dict(fmt=3), 1), (dict(fmt=-1), 1), (dict(k=None), 1), (dict(v=None), 1),
          (dict(k=OFF4), 1), (dict(v=OFF4), 1), (dict(bt=None), 1), (dict(bt=OFF2), 1), (dict(sl=None), 1), (dict(sl=OFF2), 1)]
SCALED = [(dict(ks=0.0), 1), (dict(vs=float("nan")), 1), (dict(sm=float("inf")), 1), (dict(hk=FAKE), 1), (dict(hv=FAKE), 1),
          (dict(hk=OFF2, hv=FAKE), 1), (dict(fmt=2), 1), (dict(fmt=2, ks=1.0, vs=1.0, hk=FAKE, hv=FAKE), 1),
          (dict(hq=30), 1), (dict(hq=256), 2), (dict(q=None), 1), (dict(q=OFF4), 1), (dict(out=None), 1), (dict(out=OFF4), 1)]


@pytest.mark.parametrize("kw,code", SHAPES + SCALED + [
    (dict(st=None), 1), (dict(st=OFF2), 1), (dict(par=None), 1), (dict(par=OFF2), 1), (dict(n=257, msl=4096, mb=256), 2),
    (dict(n=-1), 1), (dict(n=129), 1), (dict(T=-1), 1),
    (dict(B=0, q=None, out=None), 0), (dict(T=0, q=None, out=None), 0), (dict(n=0, q=None, out=None), 0),
])
def test_tree_attention_validates(lib, kw, code):
    assert _tree(lib, **kw) == code


@pytest.mark.parametrize("args", [(2, 16, 128, 32, 8, 96, 16, 0), (2, 300, 4096, 32, 8, 128, 16, 0), (2, 16, 8, 32, 8, 128, 16, 0),
                                  (2, 16, 128, 30, 8, 128, 16, 0), (-1, 16, 128, 32, 8, 128, 16, 0)])
def test_tree_workspace_size_of_bad_shapes(lib, args):
    assert lib.fp8kv_paged_tree_workspace_size(*args) == 0


def test_stall_hook_validates(lib):
    base = [FAKE, 20, FAKE, FAKE, 100, FAKE, 8, FAKE, FAKE, FAKE, 16, 128, 2, 32, 8, 128, 16, 0, 0.5, 0.5, None, None, 0.1,
            0, FAKE, FAKE, 1 << 20, None]
    for stage, limit in ((-1, 1000), (0, 0), (0, 500000001)):
        assert lib.fp8kv_debug_paged_tree_stall(*base, stage, limit) == 1


def test_binding_refuses_host_tensors_and_wrong_shapes():
    q = torch.zeros((4, 8, 64), dtype=torch.bfloat16)
    cache = torch.zeros((3, 2, 16, 64), dtype=torch.uint8)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(256, dtype=torch.uint8)
    ok = dict(q=q, k_cache=cache, v_cache=cache, block_tables=i32(2, 3), seq_lens=i32(2), q_starts=i32(3), parents=i32(4),
              max_nodes=4, max_seq_len=40, sm_scale=0.1, window=0, out=q, workspace=ws)
    with pytest.raises(TypeError):
        fk.fp8kv_paged_tree_attention(**ok)                       # not on a GPU
    for bad in (dict(q_starts=i32(2)), dict(parents=i32(5)), dict(out=q[:2])):
        with pytest.raises(ValueError):
            fk.fp8kv_paged_tree_attention(**{**ok, **bad})


CUTS = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "tree_walk.h"
using namespace fp8kv;
using namespace fp8kv::tree;
static unsigned rnd = 12345;
static int next(int n) { rnd = rnd * 1664525u + 1013904223u; return static_cast<int>((rnd >> 8) % n); }
int main() {
    for (int trial = 0; trial < 400; ++trial) {
        const int B = 1 + next(9), H = 1 + next(5), most = 1 + next(40), minp = 1 + next(20), window = next(3) ? 0 : 1 + next(100);
        std::vector<int> L(B), n(B), blocks(B);
        std::vector<int64_t> pre(B + 1, 0);
        for (int b = 0; b < B; ++b) {
            n[b] = next(4) ? next(30) : 0;
            L[b] = n[b] + (next(5) ? next(400) : 0);
            blocks[b] = n[b] ? 1 + next(3) : 0;
            const int np = unit_pages(L[b], n[b], window);
            // the pages are those of the first attended key up to the last token
            if (n[b]) {
                int lo = window > 0 ? L[b] - n[b] + 1 - window : 0;
                if (lo < 0) lo = 0;
                if (first_key(L[b], n[b], window) != lo || np != (L[b] - 1) / 16 - lo / 16 + 1) return 1;
            } else if (np != 0) return 2;
            pre[b + 1] = pre[b] + static_cast<int64_t>(np + kLeadPages) * H * blocks[b];
        }
        const int64_t P = pre[B];
        if (P == 0) continue;
        const int C = cta_count(P, most, minp);
        if (C < 1 || C > most || C > P) return 3;
        const Partition part = make_partition(P, C);
        std::vector<int> got(P, 0);
        std::vector<int> slots(2 * C, 0);
        for (int c = 0; c < C; ++c) {
            const int64_t r0 = range_start(part, c), e = range_start(part, c + 1);
            for (int64_t pos = r0; pos < e;) {
                const Segment s = segment_at(pos, e, pre.data(), B, [&](int b) { return blocks[b]; },
                                             [&](int b) { return unit_pages(L[b], n[b], window); });
                const int np = unit_pages(L[s.b], n[s.b], window);
                if (s.np != np || s.hk < 0 || s.hk >= H || s.rb < 0 || s.rb >= blocks[s.b]) return 4;
                if (s.base != pre[s.b] + (static_cast<int64_t>(s.hk) * blocks[s.b] + s.rb) * (np + kLeadPages)) return 5;
                if (s.lp0 < 0 || s.lp1 < s.lp0 || s.lp1 > np) return 6;
                pos = unit_end(s);
                if (s.lp0 == s.lp1) {
                    if (pos < e) return 10;      // only where the range ends in a lead
                    continue;
                }
                for (int p = s.lp0; p < s.lp1; ++p) ++got[s.base + kLeadPages + p];
                const int c0 = cta_of(part, s.base + kLeadPages), c1 = cta_of(part, s.base + kLeadPages + np - 1);
                if ((c0 == c1) != (s.lp0 == 0 && s.lp1 == np) || c < c0 || c > c1) return 7;
                if (c0 != c1) {
                    const int64_t slot = partial_slot(part, c, s.base);
                    if (slot != 2 * c + (c == c0) || slots[slot]++) return 8;
                }
            }
        }
        for (int b = 0; b < B; ++b)
            for (int u = 0; u < H * blocks[b]; ++u) {
                const int np = unit_pages(L[b], n[b], window);
                const int64_t base = pre[b] + static_cast<int64_t>(u) * (np + kLeadPages);
                for (int64_t p = 0; p < kLeadPages + np; ++p)
                    if (got[base + p] != (p >= kLeadPages)) return 9;
            }
    }
    return 0;
}
"""


def test_every_page_of_every_unit_is_walked_once(tmp_path):
    src = tmp_path / "cuts.cpp"
    src.write_text(CUTS)
    exe = tmp_path / "cuts"
    csrc = os.path.join(os.path.dirname(fbuild.__file__), "csrc")
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def _commit(lib, **kw):
    a = dict(k=FAKE, v=FAKE, nb=100, bt=FAKE, mb=8, sl=FAKE, st=FAKE, acc=FAKE, n=16, msl=128, B=2, hkv=8, d=128, bs=16,
             fmt=0, new=FAKE, ws=FAKE, wsb=256)
    a.update(kw)
    return lib.fp8kv_tree_commit(a["k"], a["v"], a["nb"], a["bt"], a["mb"], a["sl"], a["st"], a["acc"], a["n"], a["msl"],
                                 a["B"], a["hkv"], a["d"], a["bs"], a["fmt"], a["new"], a["ws"], a["wsb"], None)


def _evict(lib, **kw):
    a = dict(k=FAKE, v=FAKE, w=FAKE, nb=100, bt=FAKE, mb=8, sl=FAKE, msl=128, budget=64, sinks=4, recent=16, B=2, hkv=8,
             d=128, bs=16, fmt=0, new=FAKE, kept=None, ws=FAKE, wsb=256)
    a.update(kw)
    return lib.fp8kv_evict(a["k"], a["v"], a["w"], a["nb"], a["bt"], a["mb"], a["sl"], a["msl"], a["budget"], a["sinks"],
                           a["recent"], a["B"], a["hkv"], a["d"], a["bs"], a["fmt"], a["new"], a["kept"], a["ws"], a["wsb"],
                           None)


MOVES = [(dict(new=None), 1), (dict(new=OFF2), 1), (dict(ws=None), 3), (dict(ws=OFF4), 3), (dict(wsb=255), 3)]


@pytest.mark.parametrize("kw,code", SHAPES + MOVES + [
    (dict(st=None), 1), (dict(st=OFF2), 1), (dict(acc=None), 1), (dict(acc=OFF2), 1), (dict(n=-1), 1), (dict(n=257), 2),
    (dict(B=0, k=None, ws=None), 0), (dict(n=0, k=None, ws=None), 0), (dict(n=0, B=-1), 1),
])
def test_tree_commit_validates(lib, kw, code):
    assert _commit(lib, **kw) == code


@pytest.mark.parametrize("kw,code", SHAPES + MOVES + [
    (dict(w=None), 1), (dict(w=OFF4), 1), (dict(kept=OFF2), 1), (dict(budget=0), 1), (dict(sinks=-1), 1),
    (dict(recent=-1), 1), (dict(sinks=40, recent=25), 1), (dict(sinks=2**31 - 1, recent=2**31 - 1), 1),
    (dict(msl=393217, mb=30000), 2), (dict(B=0, k=None, w=None, ws=None), 0),
])
def test_evict_validates(lib, kw, code):
    assert _evict(lib, **kw) == code


def test_binding_refuses_what_commit_and_evict_cannot_take():
    cache, ws = torch.zeros((3, 2, 16, 64), dtype=torch.uint8), torch.zeros(256, dtype=torch.uint8)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    ok = dict(k_cache=cache, v_cache=cache, block_tables=i32(2, 3), seq_lens=i32(2), q_starts=i32(3), accepted=i32(2, 4),
              max_seq_len=40, new_lens=i32(2), workspace=ws)
    with pytest.raises(TypeError):
        fk.fp8kv_tree_commit(**ok)
    for bad in (dict(q_starts=i32(2)), dict(accepted=i32(3, 4)), dict(accepted=i32(2))):
        with pytest.raises(ValueError):
            fk.fp8kv_tree_commit(**{**ok, **bad})
    ok = dict(k_cache=cache, v_cache=cache, weights=torch.zeros((3, 2, 16)), block_tables=i32(2, 3), seq_lens=i32(2),
              max_seq_len=40, budget=8, sinks=1, recent=1, new_lens=i32(2), workspace=ws)
    with pytest.raises(TypeError):
        fk.fp8kv_evict(**ok)
    with pytest.raises(ValueError):
        fk.fp8kv_evict(**{**ok, "kept": i32(2, 2, 9)})


def _weights(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, nb=100, bt=FAKE, mb=8, sl=FAKE, msl=128, B=2, hq=32, hkv=8, d=128, bs=16, fmt=0, ks=0.5,
             vs=0.5, hk=None, hv=None, sm=0.1, win=0, out=FAKE, w=FAKE, decay=0.9, ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return lib.fp8kv_paged_decode_weights(
        a["q"], a["k"], a["v"], a["nb"], a["bt"], a["mb"], a["sl"], a["msl"], a["B"], a["hq"], a["hkv"], a["d"], a["bs"],
        a["fmt"], a["ks"], a["vs"], a["hk"], a["hv"], a["sm"], a["win"], a["out"], a["w"], a["decay"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", SHAPES + SCALED + [
    (dict(w=None), 1), (dict(w=OFF4), 1), (dict(decay=-0.1), 1), (dict(decay=float("nan")), 1),
    (dict(decay=float("inf")), 1), (dict(B=0, q=None, out=None, w=None), 0),
])
def test_decode_weights_validates(lib, kw, code):
    assert _weights(lib, **kw) == code


def test_binding_refuses_what_the_weights_cannot_take():
    q = torch.zeros((2, 8, 64), dtype=torch.bfloat16)
    cache, ws = torch.zeros((3, 2, 16, 64), dtype=torch.uint8), torch.zeros(256, dtype=torch.uint8)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    ok = dict(q=q, k_cache=cache, v_cache=cache, block_tables=i32(2, 3), seq_lens=i32(2), max_seq_len=40, sm_scale=0.1,
              window=0, out=q, weights=torch.zeros((3, 2, 16)), decay=1.0, workspace=ws)
    with pytest.raises(TypeError):
        fk.fp8kv_paged_decode_weights(**ok)
    for bad in (dict(out=q[:1]), dict(seq_lens=i32(3))):
        with pytest.raises(ValueError):
            fk.fp8kv_paged_decode_weights(**{**ok, **bad})

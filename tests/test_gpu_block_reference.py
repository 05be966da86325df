"""GPU tests of the block-scaled prefill's reference maxima: windows that start in different stages of a key range
inside one warp, so that some rows meet their first keys while others outgrow the reference they hold."""
import numpy as np
import pytest
import torch

from tests.block_harness import Cache, check_rows, f64, randn, run_prefill

pytestmark = pytest.mark.gpu

L, FIRST = 900, 173      # keys; the first key that the first row attends, 13 rows into its page


def _check(hq, hkv, d, n, by):
    """n new tokens at the end of L keys behind a window that lets the first attend FIRST and later keys.  Scores, or V
    scales, grow by more than the 2^16 that f16 holds from the first stage of the range to the second (from one stage
    to the next for scores).  The sequence is there often enough that no key range is split, which would end a CTA's
    range before the second stage."""
    window = L - n + 1 - FIRST
    c = Cache(hkv, d, [L], seed=3, spread=0.0)
    stage = 4 if d == 256 else 8                       # pages
    for p in range(-(-L // 16)):
        blk = c.tables[0, p]
        if by == "scores":
            c.ks[blk] *= 0.5 * (p + 1)
        else:
            c.vs[blk] = 2.0 ** (-18 if p < FIRST // 16 + stage else 12)
    c.k = (c.k & 0x7F).astype(np.uint8)                # all keys positive: a score's size follows its page's scale
    c.cuda()
    tiles = -(-n * (hq // hkv) // 128)
    units = hkv * (tiles if d == 256 or tiles == 1 else -(-tiles // 2))
    copies = torch.cuda.get_device_properties(0).multi_processor_count // units + 1
    c.lens *= copies
    c.gt, c.gl = c.gt.repeat(copies, 1), c.gl.repeat(copies)
    q = randn((n, hq, d), 5).abs()
    starts = torch.arange(copies + 1, dtype=torch.int32, device="cuda") * n
    out = run_prefill(c, q.repeat(copies, 1, 1).cuda(), starts, n, d ** -0.5, window).view(copies, n, hq, d)
    check_rows(f64(out[0]), c, 0, f64(q), list(range(L - n, L)), d ** -0.5, window, True, (d, n, by))
    assert torch.equal(out, out[:1].expand_as(out))


@pytest.mark.parametrize("by", ["scores", "value scales"])
@pytest.mark.parametrize("hq,hkv,d,n", [
    (1, 1, 256, 300), (2, 1, 256, 150), (2, 2, 256, 60), (2, 1, 256, 30),     # 64-key stages; two copies of the rows
    (1, 1, 128, 128), (2, 2, 128, 60), (1, 1, 128, 30), (2, 1, 128, 16),      # one tile, copies of 60 rows and of 32
    (2, 2, 64, 128), (1, 1, 64, 60), (1, 1, 64, 30), (2, 1, 64, 16),
])
def test_windows_that_start_in_two_stages_of_a_short_chunk(hq, hkv, d, n, by):
    _check(hq, hkv, d, n, by)


@pytest.mark.parametrize("by", ["scores", "value scales"])
@pytest.mark.parametrize("hq,hkv,d,n", [(1, 1, 128, 512), (2, 1, 128, 200), (2, 2, 128, 129), (1, 1, 64, 512),
                                        (2, 1, 64, 200), (4, 2, 64, 90)])
def test_windows_that_start_in_two_stages_of_a_long_chunk(hq, hkv, d, n, by):
    _check(hq, hkv, d, n, by)

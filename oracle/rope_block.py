"""fp8kv oracle -- TEST INFRASTRUCTURE ONLY.

Rotary positions, the block-scaled append and attention over values, in numpy
fp64 (fp32 where the definition says fp32).  It shares no code with the CUDA
library.  Pinned by ``tests/test_oracle_rope_block.py``.
"""
import math

import numpy as np

import oracle

E4M3_MAX = 448.0
EXP_LO, EXP_HI = -40, 40
PAGE = 16


def bf16(bits):
    """fp64 values of bf16 bit patterns (uint16)."""
    b = np.ascontiguousarray(bits, dtype=np.uint16).astype(np.uint32) << 16
    return b.view(np.float32).astype(np.float64)


def rope(x, positions, inv_freq, freq_axis=None, pairs=False):
    """x fp64 [T, H, d] turned by positions int [axes, T] * inv_freq fp32 [R/2];
    returns the turned values and, for each element, |x| + |y| of its pair (the
    size an fp32 rotation's error is relative to; 0 where nothing turns)."""
    x = np.asarray(x, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float32).astype(np.float64)
    half = f.size
    axis = np.zeros(half, dtype=int) if freq_axis is None else np.asarray(freq_axis, dtype=int)
    pos = np.atleast_2d(np.asarray(positions, dtype=np.int64))
    # the angle in turns, reduced by whole turns in integers of 2^-80 of a turn:
    # pos * f / (2 pi) with 1 / (2 pi) to 120 bits
    ipi = _inv_two_pi_scaled(120)
    ang = np.empty((x.shape[0], half))
    for i in range(half):
        m, e = math.frexp(float(f[i]))
        mi = int(m * 2 ** 53)                       # f = mi * 2^(e - 53)
        shift = 120 + 53 - e
        for t in range(x.shape[0]):
            n = int(pos[axis[i], t]) * mi * ipi     # turns = n * 2^-shift
            frac = n % (1 << shift) if shift > 0 else 0
            ang[t, i] = 2 * math.pi * (frac / (1 << shift))
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    y, mag = x.copy(), np.zeros_like(x)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if pairs else (slice(0, half), slice(half, 2 * half))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, mag


def _inv_two_pi_scaled(bits):
    """floor(2^bits / (2 pi)) by Machin's formula in integers."""
    p = bits + 64

    def arctan_inv(n):
        term = total = (1 << p) // n
        k, sign = 1, -1
        while term:
            term //= n * n
            k += 2
            total += sign * (term // k)
            sign = -sign
        return total
    pi = 4 * (4 * arctan_inv(5) - arctan_inv(239))
    return (1 << (bits + p)) // (2 * pi)


def least_power(amax):
    """The least 2^e, e in [-40, 40], with amax <= 448 * 2^e."""
    e = EXP_LO
    while e < EXP_HI and amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return np.float32(2.0 ** e)


def encode_scaled(x, scale):
    """E4M3(x / s): fp32 values, one fp32 division."""
    with np.errstate(all="ignore"):
        return oracle.e4m3_encode((np.asarray(x, np.float32) / np.float32(scale)).astype(np.float32))


def append_page(codes, scale, r0, rows):
    """rows fp64 [n, d] behind r0 older rows of one (page, head): (codes [16, d], scale) afterwards."""
    codes = codes.copy()
    finite = np.abs(rows[np.isfinite(rows)])
    amax = np.float32(finite.max()) if finite.size else np.float32(0)
    old = np.float32(scale)
    if r0 and amax <= np.float32(E4M3_MAX) * old:
        new = old
    else:
        new = max(least_power(amax), old) if r0 else least_power(amax)
        if r0:
            v = oracle.e4m3_decode(codes[:r0]).astype(np.float32) * np.float32(old / new)
            codes[:r0] = oracle.e4m3_encode(v)
    codes[r0:r0 + rows.shape[0]] = encode_scaled(rows, new)
    return codes, np.float32(new)


def append(cache, scales, rows, tables, lens, starts):
    """append_page over every page that the sequences' newest rows [T, H, d] touch."""
    cache, scales = cache.copy(), scales.copy()
    for b, L in enumerate(lens):
        n = starts[b + 1] - starts[b]
        p = L - n
        while p < L:
            cnt = min(PAGE - p % PAGE, L - p)
            t = starts[b] + p - (L - n)
            for h in range(cache.shape[1]):
                blk = tables[b][p // PAGE]
                cache[blk, h], scales[blk, h] = append_page(cache[blk, h], scales[blk, h], p % PAGE, rows[t:t + cnt, h])
            p += cnt
    return cache, scales


def values(cache, scales, table, L):
    """fp64 [L, H, d] of a sequence's tokens."""
    n = -(-L // PAGE)
    ids = np.asarray(table[:n], dtype=int)
    v = oracle.e4m3_decode(cache[ids]) * scales[ids].astype(np.float64)[..., None, None]
    return np.swapaxes(v, 1, 2).reshape(n * PAGE, cache.shape[1], cache.shape[3])[:L]


def attention(q, k, v, vscale, positions, sm, window=0):
    """Rows q fp64 [R, Hq, d] at `positions` over k, v fp64 [L, H, d].

    Returns the outputs [R, Hq, d] and what an error bound is made of:
    ``size`` sum p |v| / sum p; ``tiny`` and ``tiny_w``, what 2^-25 of the
    largest probability (of the largest p * vscale, vscale [L, H]) on every key
    amounts to; ``score`` the largest |sm| * sum |q k| of a row."""
    R, hq, d = q.shape
    g = hq // k.shape[1]
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    tiny, tiny_w, score = np.zeros(q.shape), np.zeros(q.shape), np.zeros((R, hq, 1))
    for r in range(R):
        hi = positions[r] + 1
        lo = max(0, hi - window) if window > 0 else 0
        if hi <= lo:
            continue
        for h in range(hq):
            kk, vv, vs = k[lo:hi, h // g], v[lo:hi, h // g], vscale[lo:hi, h // g]
            s = sm * (kk @ q[r, h])
            p = np.exp(s - s.max())
            l = p.sum()
            out[r, h] = p @ vv / l
            size[r, h] = p @ np.abs(vv) / l
            tiny[r, h] = 2.0 ** -25 * np.abs(vv).sum(0) / l
            tiny_w[r, h] = 2.0 ** -25 * (p * vs).max() * (np.abs(vv) / vs[:, None]).sum(0) / l
            score[r, h] = abs(sm) * (np.abs(kk) @ np.abs(q[r, h])).max()
    return out, size, tiny, tiny_w, score

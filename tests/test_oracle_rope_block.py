"""Pins of the rotary and block-scale oracle: facts the mathematics fixes."""
import math

import numpy as np
import pytest

import oracle
from oracle import rope_block as rb


def test_inverse_two_pi():
    from fractions import Fraction
    got = Fraction(rb._inv_two_pi_scaled(120), 1 << 120)
    assert abs(float(got) - 1 / (2 * math.pi)) < 2 ** -54
    # 2 pi to 32 digits
    assert abs(got * Fraction("6.28318530717958647692528676655900577") - 1) < Fraction(1, 10 ** 30)


@pytest.mark.parametrize("pairs", [False, True])
def test_rope_matches_plain_angles_and_keeps_lengths(pairs):
    g = np.random.default_rng(0)
    x = g.standard_normal((6, 2, 32))
    pos = g.integers(0, 1000, (2, 6))
    f = (10000.0 ** (-np.arange(8) / 8)).astype(np.float32)
    axis = np.arange(8) % 2
    y, mag = rb.rope(x, pos, f, axis, pairs)
    for t in range(6):
        for i in range(8):
            a = int(pos[axis[i], t]) * float(f[i])
            p, q = (2 * i, 2 * i + 1) if pairs else (i, i + 8)
            z = complex(x[t, 1, p], x[t, 1, q]) * complex(math.cos(a), math.sin(a))
            assert abs(z.real - y[t, 1, p]) < 1e-11 and abs(z.imag - y[t, 1, q]) < 1e-11
            assert mag[t, 1, p] == abs(x[t, 1, p]) + abs(x[t, 1, q])
    assert np.array_equal(y[..., 16:], x[..., 16:]) and not mag[..., 16:].any()
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))


def test_rope_turns_add_up_at_large_positions():
    """Turning by p and then by q is turning by p + q, also at 2^30."""
    x = np.random.default_rng(1).standard_normal((1, 1, 8))
    f = np.asarray([1.0, 0.37, 1e-3, 1e-6], dtype=np.float32)
    a, b = 2 ** 30 + 12345, -98765
    y1, _ = rb.rope(rb.rope(x, [[a]], f)[0], [[b]], f)
    y2, _ = rb.rope(x, [[a + b]], f)
    assert np.abs(y1 - y2).max() < 1e-12


def test_least_power_brackets():
    for amax in [0.0, 1e-30, 448 * 2.0 ** -40, 448 * 2.0 ** -39, 1.0, 447.9, 448.0, 448.1, 1e6, 448 * 2.0 ** 40, 1e30]:
        s = float(rb.least_power(np.float32(amax)))
        e = math.log2(s)
        assert e == int(e) and -40 <= e <= 40
        assert np.float32(amax) <= 448 * s or e == 40
        assert e == -40 or np.float32(amax) > 448 * s / 2


def test_append_page_keeps_or_grows():
    g = np.random.default_rng(2)
    rows = g.standard_normal((4, 8))
    codes, s = rb.append_page(np.full((16, 8), 0x7F, np.uint8), np.float32(np.nan), 0, rows)
    assert np.abs(rows).max() <= 448 * s and np.abs(rows).max() > 224 * s
    small, s2 = rb.append_page(codes, s, 4, rows[:1] * 0.5)
    assert s2 == s and np.array_equal(small[:4], codes[:4])
    big, s3 = rb.append_page(codes, s, 4, rows[:1] * 100)
    assert s3 > s
    # a power of two: the older rows stand for the same values but where they became subnormal
    a, b = oracle.e4m3_decode(codes[:4]) * s, oracle.e4m3_decode(big[:4]) * s3
    normal = np.abs(b) >= 2.0 ** -6 * s3
    assert normal.any() and np.array_equal(a[normal], b[normal]) and np.abs(a - b).max() <= 2.0 ** -10 * s3


def test_attention_matches_the_scalar_oracle():
    g = np.random.default_rng(3)
    B, hq, hkv, d, L = 1, 4, 2, 16, 50
    kc = g.integers(0, 120, (L, hkv, d)).astype(np.uint8)
    vc = g.integers(0, 120, (L, hkv, d)).astype(np.uint8)
    q = (g.integers(0x3F00, 0x4000, (B, hq, d))).astype(np.uint16)
    ref = oracle.decode_attention(q, kc, vc, np.asarray([L]), 0.01, 0.02, 0.25, 20)
    k, v = oracle.e4m3_decode(kc) * np.float32(0.01), oracle.e4m3_decode(vc) * np.float32(0.02)
    out = rb.attention(rb.bf16(q), k, v, np.full((L, hkv), 0.02), [L - 1], 0.25, 20)[0]
    assert np.abs(out - ref).max() < 1e-9


def test_a_negative_score_scale_has_the_bound_of_its_size():
    """Queries and the score scale negated together: the same answer, and the same sizes to bound errors by."""
    g = np.random.default_rng(4)
    q, k, v = g.standard_normal((2, 4, 16)), g.standard_normal((20, 2, 16)), g.standard_normal((20, 2, 16))
    for a, b in zip(rb.attention(q, k, v, np.ones((20, 2)), [15, 19], 0.3),
                    rb.attention(-q, k, v, np.ones((20, 2)), [15, 19], -0.3)):
        assert np.array_equal(a, b)

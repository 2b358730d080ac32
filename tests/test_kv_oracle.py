"""Pins of the key-value cache oracle (CPU): hand examples and independent
restatements, so that a mistake in it does not pass for the kernels' result."""

from fractions import Fraction

import numpy as np
import pytest

import oracle.kv_oracle as K
from tests import kv_cases as C


def test_hand_vector():
    # range [-1, 2]: s = 3 / 15 rounded to 16 bits; z = rint(1 / s) = 5
    x = np.array([-1.0, 0.0, 2.0, 0.31, 0.29, -0.11] + [0.0] * 10)
    codes, word = K.quantize(x, 4)
    s = Fraction(0.2).limit_denominator(10**9)
    step = Fraction(2) ** -18  # 16 significant bits from 2^-3 down
    s16 = round(s / step) * step
    assert int(word) & 0xFF == 5
    assert np.uint32(int(word) & 0xFFFFFF00).view(np.float32) == np.float32(float(s16))
    assert codes.tolist()[:6] == [0, 5, 15, 7, 6, 4]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_codes_are_the_nearest_grid_points(bits, dtype):
    """Against exact rationals: every code is a nearest point of the grid
    (an even distance to its neighbour only at a tie), clamped, and the step
    is the range over the levels within the roundings that the format has."""
    rng = np.random.default_rng(bits)
    x = rng.standard_normal((40, 32)) * np.exp(rng.standard_normal((40, 1)))
    x[3] = np.abs(x[3])
    x[4] = -np.abs(x[4])
    x[5] = rng.integers(-20, 21, 32) / 2.0
    x, _ = C.cast(x, dtype)
    codes, words = K.quantize(x, bits)
    top = 2**bits - 1
    for row, c, w in zip(x, codes, words):
        s = Fraction(float((w & np.uint32(0xFFFFFF00)).view(np.float32)))
        z = int(w & np.uint32(0xFF))
        lo, hi = min(Fraction(0), *(Fraction(float(v)) for v in row)), max(Fraction(0), *(Fraction(float(v)) for v in row))
        assert abs(s * top / (hi - lo) - 1) <= Fraction(1, 2**16) + Fraction(1, 2**22)
        assert abs(-lo / s - z) <= Fraction(1, 2) and 0 <= z <= top
        for v, k in zip(row, c):
            q = Fraction(float(v)) / s
            n = k - z
            if 0 < k < top:
                assert abs(q - n) <= Fraction(1, 2)
                assert abs(q - n) < Fraction(1, 2) or n % 2 == 0
            else:
                assert (k == 0 and q - n <= Fraction(1, 2)) or (k == top and q - n >= -Fraction(1, 2))


def test_zero_and_tiny_vectors_read_as_zero_and_bad_ones_as_nan():
    x = np.zeros((6, 16))
    x[1] = 1e-41
    x[2, 3] = np.inf
    x[3, 0] = np.nan
    x[4, :2] = [3e38, -3e38]
    x[5] = -2.5
    codes, words = K.quantize(x, 8)
    v = K.values(K.pack(codes, 8), words, 8)
    assert not v[0].any() and not v[1].any()
    assert np.isnan(v[2:5]).all()
    assert np.allclose(v[5], -2.5, rtol=2.0**-16)


def test_pack_is_the_frameworks_bitstream():
    import oracle.gptq_oracle as O

    rng = np.random.default_rng(0)
    for bits in (4, 8):
        codes = rng.integers(0, 2**bits, (7, 48))
        assert np.array_equal(K.pack(codes, bits), O.pack(codes, bits))
        assert np.array_equal(K.unpack(K.pack(codes, bits), bits), codes)


def test_attention_is_softmax_row_by_row():
    """Against plain loops over keys, in another order of operations."""
    rng = np.random.default_rng(2)
    table, lens, starts, n_pages = C.batch(rng, [21, 0, 9], [3, 0, 2], 16)
    cache = C.cache(rng, n_pages, 2, 16, 16, 8)
    q = rng.standard_normal((5, 4, 16))
    slopes = np.array([0.5, 0.25, 0.1, 0.0])
    out, mag, written, bad = K.attention(q, cache, table, lens, starts, 0.3, slopes)
    assert written.all() and not bad
    for b, (n, m) in enumerate(((3, 21), (0, 0), (2, 9))):
        for i in range(n):
            for h in range(4):
                num, den = np.zeros(16), 0.0
                for j in range(m - n + i + 1):
                    page, off = table[b, j // 16], j % 16
                    k, v = (K.values(cache[x + "_codes"][page, h // 2, off], cache[x + "_grid"][page, h // 2, off], 8)
                            for x in "kv")
                    e = np.exp(0.3 * float(q[starts[b] + i, h] @ k) + slopes[h] * (j - (m - n + i)))
                    num, den = num + e * v, den + e
                assert np.allclose(out[starts[b] + i, h], num / den, rtol=1e-12, atol=1e-14)


def test_the_bound_rejects_planted_mistakes():
    """Half a grid step of one key, a key too many, a slope with the wrong
    sign and weights rounded to bf16 all leave the attention bound."""
    rng = np.random.default_rng(3)
    table, lens, _, n_pages = C.batch(rng, [40], [1], 16)
    cache = C.cache(rng, n_pages, 1, 16, 64, 8)
    q = 1.5 * rng.standard_normal((1, 1, 64))
    slopes = np.array([0.3])
    ref, mag, _, _ = K.attention(q, cache, table, lens, None, 0.125, slopes)
    bound = C.attention_bound(ref, mag, q, cache, 0.125, slopes, "f16", "f16", 40)

    def off(cache=cache, lens=lens, slopes=slopes):
        return np.abs(K.attention(q, cache, table, lens, None, 0.125, slopes)[0] - ref)

    assert np.all(off() <= bound)
    assert np.any(off(lens=np.array([41])) > bound)
    assert np.any(off(slopes=-slopes) > bound)
    moved = dict(cache, v_grid=cache["v_grid"].copy())
    moved["v_grid"][table[0, 2], 0, 7] += 1  # one zero point
    assert np.any(off(cache=moved) > bound)

"""The MXFP4 oracle: nearest search over all codes and exponents, the byte order, the attention."""
import math

import numpy as np
import pytest

from oracle import mxfp4 as o4


def _nearest(x):
    """The code nearest to x among all sixteen; of two as near, the one with an even mantissa bit."""
    best = min(range(8), key=lambda c: (abs(abs(x) - o4.VALUES[c]), c % 2))
    return best + (8 if math.copysign(1.0, x) < 0 else 0)


def test_encode_is_the_nearest_value():
    v = o4.VALUES
    xs = list(v) + list((v[1:] + v[:-1]) / 2) + [7.0, 100.0, 1e-30, 0.26, 0.74, 5.0001, 4.9999]
    xs += list(np.random.default_rng(1).uniform(0, 7, 500))
    for x in xs:
        for s in (x, -x):
            assert o4.encode(s) == _nearest(s), s
    assert o4.encode(-0.0) == 8 and o4.encode(0.0) == 0
    assert np.array_equal(o4.encode(o4.decode(np.arange(16)))[1:8], np.arange(16)[1:8])


@pytest.mark.parametrize("mode", ["rceil", "floor"])
def test_scale_exponent_by_search(mode):
    g = np.random.default_rng(2)
    amax = np.concatenate([np.ldexp(g.uniform(1, 2, 200), g.integers(-126, 126, 200)),
                           np.ldexp(1.5, np.arange(-120, 120, 7)), np.ldexp(1.0, np.arange(-120, 120, 7)), [0.0]])
    e = o4.scale_exponent(amax, mode)
    for a, got in zip(amax, e):
        if a == 0:
            want = -127
        elif mode == "rceil":
            want = next((k for k in range(-127, 128) if a <= 6 * 2.0 ** k), 127)
        else:
            want = max(-127, min(127, math.floor(math.log2(a)) - 2))
        assert got == want, a


def test_byte_order_is_its_definition():
    codes = np.random.default_rng(4).integers(0, 16, size=(3, 128)).astype(np.uint8)
    packed = o4.pack_rows(codes)
    for row in range(3):
        for b in range(4):
            for g in range(8):
                for j in range(2):
                    byte = packed[row, 8 * g + 2 * b + j]
                    assert byte & 15 == codes[row, 32 * b + 4 * g + 2 * j]
                    assert byte >> 4 == codes[row, 32 * b + 4 * g + 2 * j + 1]
    assert np.array_equal(o4.unpack_rows(packed), codes)


def test_attend_is_the_softmax():
    g = np.random.default_rng(6)
    q, k, v = g.standard_normal(128), g.standard_normal((5, 128)), g.standard_normal((5, 128))
    o, lse, _, _ = o4.attend(q, k, v)
    s = [sum(float(a) * float(b) for a, b in zip(q, row)) / math.sqrt(128) for row in k]
    z = sum(math.exp(x) for x in s)
    np.testing.assert_allclose(o, sum(math.exp(x) / z * row for x, row in zip(s, v)), atol=1e-13)
    assert abs(lse - math.log(z)) < 1e-13
    assert np.array_equal(o4.attend(q, k[:1], v[:1])[0], v[0])
    o, lse, _, _ = o4.attend(q, k[:0], v[:0])
    assert not o.any() and lse == -math.inf

"""The norm-and-rotation oracle against a pure-Python loop, invariants and central differences."""
import math

import numpy as np
import pytest

from oracle import norm_rope as onr


def _loop(x, w, pos, freq, axis, pairing, eps, norm):
    T, H, _ = x.shape
    y = np.zeros_like(x)
    for t in range(T):
        for h in range(H):
            row = [float(v) for v in x[t, h]]
            r = 1.0 / math.sqrt(sum(v * v for v in row) / 128 + eps) if norm else 1.0
            u = [v * r * (1.0 if w is None else float(w[h][i] if np.ndim(w) == 2 else w[i])) for i, v in enumerate(row)]
            for p in range(64):
                a, b = (2 * p, 2 * p + 1) if pairing == "interleaved" else (p, p + 64)
                ang = float(pos[t][axis[p]]) * float(freq[p])
                y[t, h, a] = u[a] * math.cos(ang) - u[b] * math.sin(ang)
                y[t, h, b] = u[a] * math.sin(ang) + u[b] * math.cos(ang)
    return y


@pytest.mark.parametrize("pairing", ["interleaved", "half"])
@pytest.mark.parametrize("dims,wkind,norm", [((128,), "one", True), ((44, 42, 42), "heads", True), ((32, 16), None, False)])
def test_forward_is_the_loop(pairing, dims, wkind, norm):
    g = np.random.default_rng(3)
    x = g.standard_normal((3, 2, 128))
    w = {None: None, "one": g.standard_normal(128), "heads": g.standard_normal((2, 128))}[wkind]
    pos = g.integers(0, 50, size=(3, len(dims)))
    freq, axis = onr.axes_frequencies(dims)
    got = onr.norm_rope(x, w, onr.angles(pos, freq, axis), pairing, 1e-5, norm)
    np.testing.assert_allclose(got, _loop(x, w, pos, freq, axis, pairing, 1e-5, norm), rtol=0, atol=1e-13)
    # beyond the axes' dims nothing turns
    u = onr.norm_rope(x, w, None, pairing, 1e-5, norm)
    a, b = onr.pair_indices(pairing)
    still = freq == 0
    assert np.array_equal(got[..., a[still]], u[..., a[still]]) and np.array_equal(got[..., b[still]], u[..., b[still]])


def test_rotation_keeps_lengths_and_relative_positions():
    g = np.random.default_rng(5)
    q, k = g.standard_normal((2, 1, 1, 128))
    freq, axis = onr.axes_frequencies((128,))
    dots = []
    for shift in (0, 7, 1000):
        yq = onr.norm_rope(q, None, onr.angles(np.array([11 + shift]), freq, axis), "half", norm=False)
        yk = onr.norm_rope(k, None, onr.angles(np.array([4 + shift]), freq, axis), "half", norm=False)
        np.testing.assert_allclose(np.linalg.norm(yq), np.linalg.norm(q), rtol=1e-13)
        dots.append(float((yq * yk).sum()))
    np.testing.assert_allclose(dots, dots[0], rtol=0, atol=1e-9)


@pytest.mark.parametrize("pairing", ["interleaved", "half"])
@pytest.mark.parametrize("wkind,norm", [("one", True), ("heads", True), ("one", False), (None, True)])
def test_gradients_are_the_differences(pairing, wkind, norm):
    g = np.random.default_rng(9)
    x = g.standard_normal((2, 3, 128))
    w = {None: None, "one": 1 + 0.3 * g.standard_normal(128), "heads": 1 + 0.3 * g.standard_normal((3, 128))}[wkind]
    dy = g.standard_normal(x.shape)
    freq, axis = onr.axes_frequencies((64, 64))
    ang = onr.angles(g.integers(0, 30, size=(2, 2)), freq, axis)
    f = lambda xx, ww: float((onr.norm_rope(xx, ww, ang, pairing, 1e-3, norm) * dy).sum())  # noqa: E731
    dx, dw, dabs = onr.norm_rope_bwd(dy, x, w, ang, pairing, 1e-3, norm)
    eps = 1e-6
    for idx in [(0, 0, 0), (1, 2, 127), (0, 1, 64), (1, 0, 33)]:
        xp, xm = x.copy(), x.copy()
        xp[idx] += eps
        xm[idx] -= eps
        assert abs((f(xp, w) - f(xm, w)) / (2 * eps) - dx[idx]) < 1e-7
    if w is not None:
        for idx in ([(0, 5), (2, 100)] if w.ndim == 2 else [(5,), (100,)]):
            wp, wm = w.copy(), w.copy()
            wp[idx] += eps
            wm[idx] -= eps
            assert abs((f(x, wp) - f(x, wm)) / (2 * eps) - dw[idx]) < 1e-7
        assert (dabs >= np.abs(dw) - 1e-12).all()

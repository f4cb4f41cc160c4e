"""Per-head RMS norm and multi-axis rotary positions of Q and K, and their gradients (float64).

For a row x of 128 (token t, head h), weight w and the pair (a, b) of elements on axis s with
frequency f:
    r = 1 / sqrt(mean(x^2) + eps)   (1 without the norm),   u = x r w,   angle = position[t, s] f,
    y_a = u_a cos - u_b sin,   y_b = u_a sin + u_b cos.
The pairs are (2i, 2i + 1) ("interleaved") or (i, i + 64) ("half").

Parity: pinned in the CPU tests by a pure-Python loop over pairs, by the rotation's invariants and
by central differences of the forward.
"""
from __future__ import annotations

import numpy as np

HEAD_DIM = 128


def pair_indices(pairing: str):
    i = np.arange(HEAD_DIM // 2)
    return (2 * i, 2 * i + 1) if pairing == "interleaved" else (i, i + HEAD_DIM // 2)


def axes_frequencies(dims, theta=10000.0):
    """(inv_freq, axis) of the 64 pairs for head_dim split among the axes; 0 beyond them."""
    freq, axis = np.zeros(64), np.zeros(64, dtype=int)
    at = 0
    for a, d in enumerate(dims):
        for j in range(d // 2):
            freq[at], axis[at] = float(theta) ** (-2.0 * j / d), a
            at += 1
    return freq, axis


def angles(positions, inv_freq, axis):
    """(T, 64) angles of every token and pair."""
    p = np.asarray(positions, dtype=np.float64)
    p = p[:, None] if p.ndim == 1 else p
    return p[:, np.asarray(axis)] * np.asarray(inv_freq, dtype=np.float64)


def _inv_rms(x, eps, norm):
    return 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) if norm else np.ones(x.shape[:-1] + (1,))


def norm_rope(x, w, angle, pairing="interleaved", eps=1e-6, norm=True):
    """x (T, H, 128), w None, (128,) or (H, 128), angle (T, 64) or None."""
    x = np.asarray(x, dtype=np.float64)
    u = x * _inv_rms(x, eps, norm) * (1.0 if w is None else np.asarray(w, dtype=np.float64))
    if angle is None:
        return u
    c, s = np.cos(angle)[:, None, :], np.sin(angle)[:, None, :]
    a, b = pair_indices(pairing)
    y = np.empty_like(u)
    y[..., a] = u[..., a] * c - u[..., b] * s
    y[..., b] = u[..., a] * s + u[..., b] * c
    return y


def norm_rope_bwd(dy, x, w, angle, pairing="interleaved", eps=1e-6, norm=True):
    """(dx, dw, |dw|): the gradients, and the sums of the magnitudes of dw's terms (for error bounds)."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    g = dy.copy()
    if angle is not None:
        c, s = np.cos(angle)[:, None, :], np.sin(angle)[:, None, :]
        a, b = pair_indices(pairing)
        g[..., a] = dy[..., a] * c + dy[..., b] * s
        g[..., b] = dy[..., b] * c - dy[..., a] * s
    r = _inv_rms(x, eps, norm)
    h = g if w is None else g * np.asarray(w, dtype=np.float64)
    dx = r * h
    if norm:
        dx = dx - x * r ** 3 * np.mean(h * x, axis=-1, keepdims=True)
    if w is None:
        return dx, None, None
    term = g * x * r
    over = (0,) if np.ndim(w) == 2 else (0, 1)
    return dx, term.sum(axis=over), np.abs(term).sum(axis=over)

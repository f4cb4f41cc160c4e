"""Norm and rotation of Q and K: weights of another type than the data, positions in other orders than (tokens,
axes), backward outputs inside wider tensors, and calls from two host threads. Tolerances as in the other
tests of these operators: 2^-20 of |u_a| + |u_b| forward, 2^-19 of the magnitudes a gradient is made of, half a
step of a BF16 output (2^-8 of the value), and 2^-15 of the terms' magnitudes for a weight's gradient."""
import threading

import numpy as np
import pytest
import torch

from oracle import norm_rope as onr

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import precision_attention_forward_b200 as lp
    from tests.test_norm_rope_gpu import TORCH, _case, _dev, _mag, _round

OTHER = {"bf16": "fp32", "fp32": "bf16"}


def _mixed(seed, T, hq, hk, dt, kind, axes=(44, 42, 42)):
    """A case whose weights are of the type that the data is not."""
    q, k, w, pos, ang = _case(seed, T, hq, hk, dt, axes, kind)
    g = np.random.default_rng(seed + 1)
    w = [_round(1 + 0.3 * g.standard_normal(x.shape), OTHER[dt]) for x in w]
    return q, k, w, pos, ang, [_dev(x, OTHER[dt]) for x in w]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["one", "heads"])
@pytest.mark.parametrize("hq,hk", [(8, 4), (3, 1)])
def test_weights_of_the_other_type(dt, kind, hq, hk):
    T, pairing = 203, "half" if hq == 3 else "interleaved"
    q, k, w, pos, ang, tw = _mixed(hq, T, hq, hk, dt, kind)
    tq, tk, p = _dev(q, dt), _dev(k, dt), torch.from_numpy(pos).cuda()
    rope = lp.RotaryAxes((44, 42, 42), pairing=pairing)
    for out in ("bf16", "fp32"):
        ys = lp.lpfa_qk_norm_rope(tq, tk, p, rope, *tw, out_dtype=TORCH[out])
        for y, x, wt in zip(ys, (q, k), w):
            ref = onr.norm_rope(x, wt, ang, pairing)
            tol = _mag(x, wt, ang, pairing) * 2.0 ** -20 + (np.abs(ref) * 2.0 ** -8 if out == "bf16" else 0)
            assert (np.abs(y.double().cpu().numpy() - ref) <= tol).all()
    meta = lp.lpfa_varlen_meta_from_lengths([100, 103])
    got = lp.lpfa_qk_norm_rope_mxfp8(tq, tk, p, rope, meta, *tw)
    for i in range(2):  # ys is FP32 here
        payload, scales = lp.lpfa_quantize_mxfp8_varlen(ys[i], meta)
        assert torch.equal(got[2 * i], payload) and torch.equal(got[2 * i + 1], scales)
    g = np.random.default_rng(5)
    dy = [_round(g.standard_normal(x.shape), dt) for x in (q, k)]
    res = lp.lpfa_qk_norm_rope_bwd(*(_dev(d, dt) for d in dy), tq, tk, p, rope, *tw)
    _check_gradients(res, dy, (q, k), w, ang, pairing, dt)
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)


def _check_gradients(res, dy, xs, w, ang, pairing, dt):
    a, b = onr.pair_indices(pairing)
    for i, (d, x, wt) in enumerate(zip(dy, xs, w)):
        rx, rw, _ = onr.norm_rope_bwd(d, x, wt, ang, pairing)
        h = np.empty(d.shape)
        h[..., a] = h[..., b] = np.abs(d[..., a].astype(np.float64)) + np.abs(d[..., b])
        ax = np.abs(x.astype(np.float64))
        r = 1.0 / np.sqrt((ax * ax).mean(-1, keepdims=True) + 1e-6)
        hw = h * np.abs(wt)
        made = r * hw + ax * r ** 3 * (hw * ax).mean(-1, keepdims=True)
        tol = made * 2.0 ** -19 + (np.abs(rx) * 2.0 ** -8 if dt == "bf16" else 0)
        assert (np.abs(res[i].double().cpu().numpy() - rx) <= tol).all()
        terms = (h * ax * r).sum(axis=(0,) if wt.ndim == 2 else (0, 1))
        assert res[2 + i].dtype == torch.float32 and res[2 + i].shape == wt.shape
        assert (np.abs(res[2 + i].double().cpu().numpy() - rw) <= terms * 2.0 ** -15).all()


@pytest.mark.parametrize("pos64", [False, True])
def test_positions_in_any_order(pos64):
    """Equal positions give equal bits, however they lie: (axes, tokens) transposed, every third row of a wider
    tensor, one column of it, one row for all tokens."""
    T = 75
    q, k, _, pos, _ = _case(3, T, 4, 2, "bf16", (44, 42, 42), pos64=pos64)
    tq, tk, p = _dev(q, "bf16"), _dev(k, "bf16"), torch.from_numpy(pos).cuda()
    rope = lp.RotaryAxes((44, 42, 42))
    want = lp.lpfa_qk_norm_rope(tq, tk, p, rope)
    wide = torch.full((3 * T, 7), 10 ** 6, dtype=p.dtype, device="cuda")
    wide[1::3, 2:5] = p
    spread = torch.full((T, 6), 10 ** 6, dtype=p.dtype, device="cuda")
    spread[:, 1::2] = p
    meta = lp.lpfa_varlen_meta_from_lengths([T])
    mx = lp.lpfa_qk_norm_rope_mxfp8(tq, tk, p, rope, meta)
    bwd = lp.lpfa_qk_norm_rope_bwd(tq, tk, tq, tk, p, rope)
    for view in (p.t().contiguous().t(), wide[1::3, 2:5], spread[:, 1::2]):
        assert not view.is_contiguous()
        for a, b in ((want, lp.lpfa_qk_norm_rope(tq, tk, view, rope)), (mx, lp.lpfa_qk_norm_rope_mxfp8(tq, tk, view, rope, meta)),
                     (bwd[:2], lp.lpfa_qk_norm_rope_bwd(tq, tk, tq, tk, view, rope)[:2])):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    one = lp.RotaryAxes((128,))
    assert all(torch.equal(x, y) for x, y in zip(lp.lpfa_qk_norm_rope(tq, tk, p[:, 1], one),
                                                 lp.lpfa_qk_norm_rope(tq, tk, p[:, 1:2].contiguous(), one)))
    same = p[:1].expand(T, 3)
    assert all(torch.equal(x, y) for x, y in zip(lp.lpfa_qk_norm_rope(tq, tk, same, rope),
                                                 lp.lpfa_qk_norm_rope(tq, tk, same.contiguous(), rope)))


def test_any_frequency_and_axis_for_each_pair():
    T, hq, hk = 40, 4, 1
    q, k, w, _, _ = _case(9, T, hq, hk, "fp32", (128,))
    g = np.random.default_rng(4)
    freq, axis = g.standard_normal(64) * 0.1, g.integers(0, 8, 64)
    pos = g.integers(-3000, 3000, size=(T, 8)).astype(np.int32)
    for pairing in ("interleaved", "half"):
        rope = lp.RotaryAxes.from_frequencies(freq, axis, pairing)
        ys = lp.lpfa_qk_norm_rope(_dev(q, "fp32"), _dev(k, "fp32"), torch.from_numpy(pos).cuda(), rope, *(_dev(x, "fp32") for x in w))
        for y, x, wt in zip(ys, (q, k), w):
            ang = onr.angles(pos, freq, axis)
            tol = _mag(x, wt, ang, pairing) * 2.0 ** -20
            assert (np.abs(y.double().cpu().numpy() - onr.norm_rope(x, wt, ang, pairing)) <= tol).all()


@pytest.mark.parametrize("dt,kind", [("bf16", "one"), ("fp32", "heads")])
@pytest.mark.parametrize("hq,hk", [(8, 4), (5, 2)])
def test_backward_into_parts_of_wider_tensors(dt, kind, hq, hk):
    T = 333
    q, k, w, pos, _ = _case(31, T, hq, hk, dt, (128,), kind)
    tq, tk, p = _dev(q, dt), _dev(k, dt), torch.from_numpy(pos).cuda()
    rope, tw = lp.RotaryAxes((128,), pairing="half"), [_dev(x, dt) for x in w]
    g = torch.Generator(device="cuda").manual_seed(1)
    dq, dk = (torch.randn(t.shape, generator=g, device="cuda").to(t.dtype) for t in (tq, tk))
    want = lp.lpfa_qk_norm_rope_bwd(dq, dk, tq, tk, p, rope, *tw)
    wide = torch.full((T, hq + hk + 3, 256), 7.0, dtype=tq.dtype, device="cuda")
    swapped = torch.full((hq, T, 128), 7.0, dtype=tq.dtype, device="cuda")
    for views in ((wide[:, 1:1 + hq, 64:192], wide[:, 2 + hq:2 + hq + hk, 64:192]),
                  (swapped.transpose(0, 1), wide[:, 2 + hq:2 + hq + hk, 64:192])):
        wide.fill_(7.0)
        got = lp.lpfa_qk_norm_rope_bwd(dq, dk, tq, tk, p, rope, *tw, dq=views[0], dk=views[1])
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        mask = torch.ones_like(wide, dtype=torch.bool)
        mask[:, 2 + hq:2 + hq + hk, 64:192] = False
        if views[0].data_ptr() != swapped.data_ptr():
            mask[:, 1:1 + hq, 64:192] = False
        assert (wide[mask] == 7.0).all()


def test_two_host_threads():
    """Each on a stream of its own, each with the results that it has alone."""
    sets = []
    for seed, T, hq, hk, dt, kind in ((1, 500, 8, 4, "bf16", "one"), (2, 77, 3, 1, "fp32", "heads")):
        q, k, w, pos, _ = _case(seed, T, hq, hk, dt, (128,), kind)
        sets.append((_dev(q, dt), _dev(k, dt), torch.from_numpy(pos).cuda(), lp.RotaryAxes((128,)), *(_dev(x, dt) for x in w)))
    once = lambda s: [*lp.lpfa_qk_norm_rope(*s), *lp.lpfa_qk_norm_rope_bwd(s[0], s[1], *s)]  # noqa: E731
    want = [once(s) for s in sets]
    torch.cuda.synchronize()
    got, errors, gate = [None, None], [], threading.Barrier(2)

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                gate.wait()
                for _ in range(200):
                    got[i] = once(sets[i])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)

"""Norm and rotation of Q and K on the GPU: forward, MXFP8 and gradients against the float64 oracle.

Tolerances. FP32: r comes from 128 squares summed in chains of 8 and trees (relative error up to
12 * 2^-24, half of it in r), 1.5 * 2^-24 of its own, and a value takes five more roundings and cos
and sin within 2^-23 each; 2^-20 of |u_a| + |u_b| covers them. An output in BF16 adds half a step,
2^-8 of the value (and 2^-9 * 2^-126 for nothing: no value here is subnormal). A gradient in the same
way, with three sums in it: 2^-19 of the magnitudes it is made of. A weight's gradient: 2^-19 a term,
and at most 300 additions in a row, 300 * 2^-24 < 2^-15 of the sum of the terms' magnitudes.
"""
import numpy as np
import pytest
import torch

import workloads as wl
from oracle import mxfp8 as omx
from oracle import norm_rope as onr

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import precision_attention_forward_b200 as lp

TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _round(x, dtype):
    return wl.round_to_bf16(x.astype(np.float32)) if dtype == "bf16" else x.astype(np.float32)


def _dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(TORCH[dtype]).cuda()


def _case(seed, T, hq, hk, dtype="bf16", axes=(128,), weights="one", pos_top=5000, pos64=False):
    """Inputs as float32 arrays (exact in dtype), positions, and the oracle's angles."""
    g = np.random.default_rng(seed)
    gain = np.exp(0.5 * g.standard_normal((hq + hk, 128)))
    x = _round(g.standard_normal((T, hq + hk, 128)) * gain, dtype)
    shape = {None: lambda h: None, "one": lambda h: (128,), "heads": lambda h: (h, 128)}[weights]
    w = [None if h == 0 or shape(h) is None else _round(1 + 0.3 * g.standard_normal(shape(h)), dtype) for h in (hq, hk)]
    pos = g.integers(0, pos_top, size=(T, len(axes))).astype(np.int64 if pos64 else np.int32)
    freq, axis = onr.axes_frequencies(axes)
    return x[:, :hq], x[:, hq:], w, pos, onr.angles(pos, freq, axis)


def _mag(x, w, ang, pairing, eps=1e-6, norm=True):
    """|u_a| + |u_b| at both elements of every pair."""
    u = np.abs(onr.norm_rope(x, w, None, pairing, eps, norm))
    a, b = onr.pair_indices(pairing)
    s = np.empty_like(u)
    s[..., a] = s[..., b] = u[..., a] + u[..., b]
    return s


CASES = [
    # T, Hq, Hk, dtype, out, pairing, axes, weights, norm
    (1, 16, 16, "bf16", "bf16", "half", (128,), "one", True),
    (7, 4, 4, "bf16", "bf16", "interleaved", (44, 42, 42), "one", True),
    (33, 3, 1, "bf16", "fp32", "interleaved", (44, 42, 42), "heads", True),
    (130, 1, 1, "fp32", "fp32", "half", (128,), "one", True),
    (257, 5, 0, "fp32", "bf16", "half", (32, 48, 16), "one", True),
    (65, 32, 8, "fp32", "fp32", "interleaved", (128,), "heads", True),
    (40, 12, 4, "bf16", "bf16", "half", (128,), None, True),
    (19, 6, 2, "bf16", "fp32", "interleaved", (64,), "one", False),
    (3001, 8, 4, "bf16", "bf16", "half", (64, 64), "one", True),
    (700, 24, 24, "bf16", "bf16", "interleaved", (44, 42, 42), "heads", True),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward_matches_the_oracle(case):
    T, hq, hk, dt, out, pairing, axes, wk, norm = CASES[case]
    q, k, w, pos, ang = _case(100 + case, T, hq, hk, dt, axes, wk, pos64=case % 2 == 1)
    qk = _dev(np.concatenate([q, k], axis=1), dt)  # strided views of a joint tensor
    tq, tk = qk[:, :hq], (qk[:, hq:] if hk else None)
    tw = [None if x is None else _dev(x, dt) for x in w]
    rope = lp.RotaryAxes(axes, pairing=pairing)
    p = torch.from_numpy(pos).cuda()
    yq, yk = lp.lpfa_qk_norm_rope(tq, tk, p if len(axes) > 1 else p[:, 0], rope, tw[0], tw[1], norm=norm,
                                  out_dtype=TORCH[out])
    torch.cuda.synchronize()
    for name, y, x, wt in (("q", yq, q, w[0]), ("k", yk, k, w[1])):
        if y is None:
            continue
        ref = onr.norm_rope(x, wt, ang, pairing, norm=norm)
        tol = _mag(x, wt, ang, pairing, norm=norm) * 2.0 ** -20 + (np.abs(ref) * 2.0 ** -8 if out == "bf16" else 0)
        d = np.abs(y.double().cpu().numpy() - ref)
        assert (d <= tol).all(), (name, float((d / np.maximum(tol, 1e-300)).max()))
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)


def test_far_positions_and_negative_ones():
    """Angles of a million turns: the product is exact up to the frequency's rounding, 2^-53 of it."""
    T = 64
    q, _, w, _, _ = _case(7, T, 4, 0, "fp32")
    g = np.random.default_rng(8)
    pos = np.concatenate([g.integers(10 ** 6, 2 ** 31 - 1, T // 2), -g.integers(1, 10 ** 6, T // 2)]).astype(np.int64)
    freq, axis = onr.axes_frequencies((128,))
    for dt in (torch.int64, torch.int32):
        y, _ = lp.lpfa_qk_norm_rope(_dev(q, "fp32"), None, torch.from_numpy(pos).to(dt).cuda(), lp.RotaryAxes((128,)))
        ref = onr.norm_rope(q, None, onr.angles(pos, freq, axis))
        # the oracle's own angle (FP64 product and cosine) is good to |angle| 2^-52
        tol = _mag(q, None, None, "interleaved") * (2.0 ** -20 + 2.0 ** 31 * 2.0 ** -51)
        assert (np.abs(y.double().cpu().numpy() - ref) <= tol).all()


def test_no_rotation_and_partial_rotation_leave_elements_exact():
    q, k, _, pos, _ = _case(11, 50, 4, 4, "bf16")
    tq, tk, p = _dev(q, "bf16"), _dev(k, "bf16"), torch.from_numpy(pos).cuda()
    y, _ = lp.lpfa_qk_norm_rope(tq, tk, None, None, norm=False)
    assert torch.equal(y, tq)
    for pairing in ("interleaved", "half"):
        rope = lp.RotaryAxes((48,), pairing=pairing)
        y, yk = lp.lpfa_qk_norm_rope(tq, tk, p, rope, norm=False)
        a, b = onr.pair_indices(pairing)
        still = np.sort(np.concatenate([a[24:], b[24:]]))
        assert torch.equal(y[..., still], tq[..., still]) and torch.equal(yk[..., still], tk[..., still])
    f = [0.0] * 60 + [0.25] * 4
    y, _ = lp.lpfa_qk_norm_rope(tq, None, p, lp.RotaryAxes.from_frequencies(f), norm=False)
    assert torch.equal(y[..., :120], tq[..., :120]) and not torch.equal(y[..., 120:], tq[..., 120:])


def test_zero_rows_and_large_rows():
    """A zero row stays zero (eps holds it up); huge and tiny rows are normalised like any other."""
    x = np.zeros((4, 4, 128), dtype=np.float32)
    x[1], x[2], x[3] = 1e15, 1e-12, np.random.default_rng(1).standard_normal((4, 128)).astype(np.float32)
    for eps in (1e-6, 0.0):
        rows = x if eps else x[1:]
        y, _ = lp.lpfa_qk_norm_rope(_dev(rows, "fp32"), None, None, None, eps=eps)
        ref = onr.norm_rope(rows, None, None, eps=eps)
        assert (np.abs(y.double().cpu().numpy() - ref) <= np.abs(ref) * 2.0 ** -20).all()


def test_in_place_and_into_strided_outputs():
    q, k, w, pos, _ = _case(21, 77, 8, 8, "bf16")
    tw = [_dev(x, "bf16") for x in w]
    rope, p = lp.RotaryAxes((128,), pairing="half"), torch.from_numpy(pos).cuda()
    joint = _dev(np.concatenate([q, k], axis=1), "bf16")
    want = lp.lpfa_qk_norm_rope(joint[:, :8], joint[:, 8:], p, rope, *tw)
    wide = torch.full((77, 20, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    got = lp.lpfa_qk_norm_rope(joint[:, :8], joint[:, 8:], p, rope, *tw, q_out=wide[:, 2:10, 64:192], k_out=wide[:, 10:18, 64:192])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    mask = torch.ones_like(wide, dtype=torch.bool)
    mask[:, 2:18, 64:192] = False
    assert (wide[mask] == 7.0).all()
    lp.lpfa_qk_norm_rope(joint[:, :8], joint[:, 8:], p, rope, *tw, q_out=joint[:, :8], k_out=joint[:, 8:])
    assert torch.equal(joint[:, :8], want[0]) and torch.equal(joint[:, 8:], want[1])


MX_CASES = [
    ([1], 4, 4, "bf16", "half", None), ([5, 128, 129], 8, 2, "bf16", "interleaved", "one"),
    ([300, 1, 77, 256], 3, 1, "fp32", "half", "heads"), ([2048, 100], 16, 16, "bf16", "interleaved", "one"),
    ([64] * 40, 2, 0, "fp32", "interleaved", "one"),
]


@pytest.mark.parametrize("mode", ["rceil", "floor"])
@pytest.mark.parametrize("case", range(len(MX_CASES)))
def test_mxfp8_is_the_quantizer_after_the_fp32_result(case, mode):
    lens, hq, hk, dt, pairing, wk = MX_CASES[case]
    T = sum(lens)
    q, k, w, pos, ang = _case(200 + case, T, hq, hk, dt, (44, 42, 42), wk)
    q = q.copy()
    q[0, 0] = 0  # a zero block: byte 0
    meta = lp.lpfa_varlen_meta_from_lengths(lens)
    tq, tk = _dev(q, dt), (_dev(k, dt) if hk else None)
    tw = [None if x is None else _dev(x, dt) for x in w]
    rope, p = lp.RotaryAxes((44, 42, 42), pairing=pairing), torch.from_numpy(pos).cuda()
    got = lp.lpfa_qk_norm_rope_mxfp8(tq, tk, p, rope, meta, *tw, scaling_mode=mode)
    y = lp.lpfa_qk_norm_rope(tq, tk, p, rope, *tw, out_dtype=torch.float32)
    for i, (x, yx) in enumerate(((q, y[0]), (k, y[1]))):
        if yx is None:
            assert got[2] is None and got[3] is None
            continue
        payload, scales = lp.lpfa_quantize_mxfp8_varlen(yx, meta, scaling_mode=mode)
        assert torch.equal(got[2 * i], payload) and torch.equal(got[2 * i + 1], scales)
        if mode == "rceil":  # and the oracle's values, to half an E4M3 step (2^-4, or of 2^-9 below 2^-6) of a block
            ref = onr.norm_rope(x, w[i], ang, pairing)
            val = omx.dequantize_mxfp8(payload.cpu().numpy(), scales.cpu().numpy(), lens, x.shape[1])
            top = np.abs(ref).reshape(T, -1, 4, 32).max(-1).repeat(32, -1).reshape(ref.shape)
            assert (np.abs(val - ref) <= np.abs(ref) * 2.0 ** -4 * 1.001 + top * 2.0 ** -16).all()
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)


BWD_CASES = [
    # T, Hq, Hk, dtype, pairing, weights, norm
    (1, 4, 4, "fp32", "half", "one", True), (9, 3, 1, "fp32", "interleaved", "heads", True),
    (333, 8, 4, "fp32", "half", "heads", True), (1025, 4, 4, "bf16", "interleaved", "one", True),
    (70, 5, 0, "bf16", "half", "one", True), (31, 8, 8, "fp32", "interleaved", None, True),
    (45, 4, 1, "fp32", "half", "one", False), (600, 32, 8, "bf16", "half", "heads", True),
    (20000, 1, 1, "fp32", "interleaved", "one", True), (40, 1, 1, "bf16", "half", "heads", True),
]


@pytest.mark.parametrize("case", range(len(BWD_CASES)))
def test_gradients_match_the_oracle(case):
    T, hq, hk, dt, pairing, wk, norm = BWD_CASES[case]
    axes = (44, 42, 42) if case % 2 else (128,)
    q, k, w, pos, ang = _case(300 + case, T, hq, hk, dt, axes, wk)
    g = np.random.default_rng(900 + case)
    dq, dk = (_round(g.standard_normal(x.shape), dt) for x in (q, k))
    tw = [None if x is None else _dev(x, dt) for x in w]
    args = (_dev(q, dt), _dev(k, dt) if hk else None, torch.from_numpy(pos).cuda(), lp.RotaryAxes(axes, pairing=pairing))
    got = lp.lpfa_qk_norm_rope_bwd(_dev(dq, dt), _dev(dk, dt) if hk else None, *args, *tw, norm=norm)
    again = lp.lpfa_qk_norm_rope_bwd(_dev(dq, dt), _dev(dk, dt) if hk else None, *args, *tw, norm=norm)
    torch.cuda.synchronize()
    for i, (x, dy, wt) in enumerate(((q, dq, w[0]), (k, dk, w[1]))):
        dx, dw = got[i], got[2 + i]
        if dx is None:
            assert dw is None
            continue
        assert torch.equal(dx, again[i])
        rx, rw, rabs = onr.norm_rope_bwd(dy, x, wt, ang, pairing, norm=norm)
        # what dx is made of: r |h| and |x| r^3 mean |h x|, with |h| <= (|dy_a| + |dy_b|) |w|
        a, b = onr.pair_indices(pairing)
        h = np.empty(dy.shape)
        h[..., a] = h[..., b] = np.abs(dy[..., a].astype(np.float64)) + np.abs(dy[..., b])
        h = h * (1.0 if wt is None else np.abs(wt))
        ax = np.abs(x.astype(np.float64))
        r = 1.0 / np.sqrt((ax * ax).mean(-1, keepdims=True) + 1e-6) if norm else 1.0
        made = r * h + (ax * r ** 3 * (h * ax).mean(-1, keepdims=True) if norm else 0)
        tol = made * 2.0 ** -19 + (np.abs(rx) * 2.0 ** -8 if dt == "bf16" else 0)
        d = np.abs(dx.double().cpu().numpy() - rx)
        assert (d <= tol).all(), float((d / tol).max())
        if wt is None:
            assert dw is None
            continue
        assert dw.dtype == torch.float32 and dw.shape == wt.shape and torch.equal(dw, again[2 + i])
        dwt = np.abs(dw.double().cpu().numpy() - rw)
        # |g x r| is bounded by (|dy_a| + |dy_b|) |x| r, of which rabs is a part: scale by both
        over = (0,) if np.ndim(wt) == 2 else (0, 1)
        terms = (np.where(np.ones_like(h, bool), h / (1.0 if wt is None else np.maximum(np.abs(wt), 1e-30)), 0) * ax * r).sum(axis=over)
        assert (dwt <= np.maximum(terms, rabs) * 2.0 ** -15).all(), float((dwt / terms).max())
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)


@pytest.mark.parametrize("case", [
    # Rows of weights per head: parts of the tokens (some of them empty) and second rounds of 64 tokens a block;
    # the last two have a row per head on one side and one row on the other.
    (20011, 3, 1, "fp32", "half", "heads", "heads"), (19200, 8, 4, "bf16", "interleaved", "heads", "heads"),
    (500, 7, 2, "bf16", "half", "heads", "heads"), (1, 2, 1, "fp32", "half", "heads", "heads"),
    (700, 12, 8, "fp32", "interleaved", "heads", "heads"), (301, 8, 2, "bf16", "half", "heads", "one"),
    (1200, 4, 8, "fp32", "half", "one", "heads"),
])
def test_weight_gradients_per_head(case):
    T, hq, hk, dt, pairing, *kinds = case
    seed = T + hq
    q, k, w, pos, ang = _case(seed, T, hq, hk, dt, (128,), "heads")
    w = [x if kind == "heads" else np.ascontiguousarray(x[0]) for x, kind in zip(w, kinds)]
    g = np.random.default_rng(seed)
    dq, dk = (_round(g.standard_normal(x.shape), dt) for x in (q, k))
    rest = (torch.from_numpy(pos).cuda(), lp.RotaryAxes((128,), pairing=pairing), *(_dev(x, dt) for x in w))
    got = lp.lpfa_qk_norm_rope_bwd(*(_dev(x, dt) for x in (dq, dk, q, k)), *rest)
    torch.cuda.synchronize()
    a, b = onr.pair_indices(pairing)
    for i, (x, dy) in enumerate(((q, dq), (k, dk))):
        rx, rw, _ = onr.norm_rope_bwd(dy, x, w[i], ang, pairing)
        h = np.empty(dy.shape)
        h[..., a] = h[..., b] = np.abs(dy[..., a].astype(np.float64)) + np.abs(dy[..., b])
        ax = np.abs(x.astype(np.float64))
        r = 1.0 / np.sqrt((ax * ax).mean(-1, keepdims=True) + 1e-6)
        hw = h * np.abs(w[i])
        made = r * hw + ax * r ** 3 * (hw * ax).mean(-1, keepdims=True)  # the bounds of the cases above
        tol = made * 2.0 ** -19 + (np.abs(rx) * 2.0 ** -8 if dt == "bf16" else 0)
        assert (np.abs(got[i].double().cpu().numpy() - rx) <= tol).all()
        terms = (h * ax * r).sum(axis=(0,) if kinds[i] == "heads" else (0, 1))
        assert got[2 + i].shape == w[i].shape
        assert (np.abs(got[2 + i].double().cpu().numpy() - rw) <= terms * 2.0 ** -15).all()
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)


def test_gradients_are_the_differences_of_the_forward():
    """Central differences of the FP32 forward: truncation (step 2^-6)^2 / 6 of the third derivative and
    2^-20 * 16 / step of rounding; 2e-3 of the gradient's size covers both."""
    T, H = 3, 4
    q, _, w, pos, _ = _case(55, T, H, 0, "fp32", (128,))
    g = torch.Generator(device="cuda").manual_seed(3)
    x, wt, p = _dev(q, "fp32"), _dev(w[0], "fp32"), torch.from_numpy(pos).cuda()
    dy = torch.randn(T, H, 128, generator=g, device="cuda")
    rope = lp.RotaryAxes((128,), pairing="half")
    f = lambda a, b: float((lp.lpfa_qk_norm_rope(a, None, p, rope, b)[0].double() * dy.double()).sum())  # noqa: E731
    dx, _, dw, _ = lp.lpfa_qk_norm_rope_bwd(dy, None, x, None, p, rope, wt)
    step = 2.0 ** -6
    for _ in range(4):
        v = torch.randn(x.shape, generator=g, device="cuda")
        num = (f(x + step * v, wt) - f(x - step * v, wt)) / (2 * step)
        assert abs(num - float((dx.double() * v).sum())) <= 2e-3 * float((dx.double() * v).abs().sum())
        u = torch.randn(wt.shape, generator=g, device="cuda")
        num = (f(x, wt + step * u) - f(x, wt - step * u)) / (2 * step)
        assert abs(num - float((dw.double() * u).sum())) <= 2e-3 * float((dw.double() * u).abs().sum())


def test_gradient_in_place_strided_and_captured():
    q, k, w, pos, _ = _case(61, 201, 8, 4, "bf16")
    joint = _dev(np.concatenate([q, k], axis=1), "bf16")
    tw = [_dev(x, "bf16") for x in w]
    rope, p = lp.RotaryAxes((128,)), torch.from_numpy(pos).cuda()
    d = torch.randn(201, 12, 128, device="cuda").bfloat16()
    call = lambda **kw: lp.lpfa_qk_norm_rope_bwd(d[:, :8], d[:, 8:], joint[:, :8], joint[:, 8:], p, rope, *tw, **kw)  # noqa: E731
    want = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = call(stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, side, held):
        assert torch.equal(a, b) and torch.equal(a, c)
    call(dq=d[:, :8], dk=d[:, 8:])
    assert torch.equal(d[:, :8], want[0]) and torch.equal(d[:, 8:], want[1])


def test_forward_captured_on_streams_and_inside_guards():
    q, k, w, pos, _ = _case(63, 130, 4, 4, "bf16")
    tq, tk, p = _dev(q, "bf16"), _dev(k, "bf16"), torch.from_numpy(pos).cuda()
    rope, meta = lp.RotaryAxes((128,)), lp.lpfa_varlen_meta_from_lengths([100, 30])
    want = lp.lpfa_qk_norm_rope(tq, tk, p, rope)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = lp.lpfa_qk_norm_rope(tq, tk, p, rope, stream=s)
    raw = lp.lpfa_qk_norm_rope(tq, tk, p, rope, stream=s.cuda_stream)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = lp.lpfa_qk_norm_rope(tq, tk, p, rope)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(want[0], x[0]) and torch.equal(want[1], x[1]) for x in (side, raw, held))
    mx = lp.lpfa_qk_norm_rope_mxfp8(tq, tk, p, rope, meta)
    outs, bufs = [], []
    for t in mx:
        buf = torch.full((t.numel() + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        bufs.append(buf)
        outs.append(buf[256:256 + t.numel()].view(t.shape))
    lp.lpfa_qk_norm_rope_mxfp8(tq, tk, p, rope, meta, q_payload=outs[0], q_scales=outs[1], k_payload=outs[2], k_scales=outs[3])
    torch.cuda.synchronize()
    for t, o, b in zip(mx, outs, bufs):
        assert torch.equal(t, o) and (b[:256] == 0xA5).all() and (b[256 + t.numel():] == 0xA5).all()


def test_refusals():
    q, k = torch.zeros(4, 2, 128, device="cuda").bfloat16(), torch.zeros(4, 2, 128, device="cuda").bfloat16()
    p, rope = torch.zeros(4, 1, dtype=torch.int32, device="cuda"), lp.RotaryAxes((128,))
    w = torch.ones(128, device="cuda").bfloat16()
    f = lp.lpfa_qk_norm_rope
    wide = torch.zeros(4, 4, 128, device="cuda").bfloat16()
    bad = [
        lambda: f(q[..., :64], None, p, rope), lambda: f(q.half(), None, p, rope), lambda: f(q.cpu(), None, p, rope),
        lambda: f(q, k.float(), p, rope), lambda: f(q, k[:3], p, rope), lambda: f(q[:0], None, p[:0], rope),
        lambda: f(q, k, p[:3], rope), lambda: f(q, k, p.float(), rope), lambda: f(q, k, p.cpu(), rope),
        lambda: f(q, k, None, rope), lambda: f(q, k, p, "half"), lambda: f(q, k, p, lp.RotaryAxes((64, 64))),
        lambda: f(q, k, p, rope, w[:64]), lambda: f(q, k, p, rope, w, w.float()), lambda: f(q, None, p, rope, w, w),
        lambda: f(q, k, p, rope, torch.ones(3, 128, device="cuda").bfloat16()), lambda: f(q, k, p, rope, eps=-1.0),
        lambda: f(q, k, p, rope, eps=float("nan")), lambda: f(q, k, p, rope, out_dtype=torch.float16),
        lambda: f(q, None, p, rope, k_out=k), lambda: f(q, k, p, rope, q_out=q[:, :1].expand(4, 2, 128)),
        lambda: f(q, k, p, rope, q_out=torch.zeros(4, 2, 128, device="cuda")),
        lambda: f(q.transpose(1, 2).contiguous().transpose(1, 2), None, p, rope),
        lambda: lp.lpfa_qk_norm_rope_mxfp8(q, k, p, rope, lp.lpfa_varlen_meta_from_lengths([5])),
        lambda: lp.lpfa_qk_norm_rope_mxfp8(q, k, p, rope, lp.lpfa_varlen_meta_from_lengths([4]), scaling_mode="up"),
        lambda: lp.lpfa_qk_norm_rope_mxfp8(q, k, p, rope, lp.lpfa_varlen_meta_fill_host([4])),
        lambda: lp.lpfa_qk_norm_rope_bwd(q, None, q, k, p, rope), lambda: lp.lpfa_qk_norm_rope_bwd(q.float(), k, q, k, p, rope),
        lambda: lp.lpfa_qk_norm_rope_bwd(q, k, q, k, p, rope, dq_weight=torch.zeros(128, device="cuda")),
        lambda: lp.lpfa_qk_norm_rope_bwd(q, k, q, k, p, rope, w, dq_weight=torch.zeros(2, 128, device="cuda")),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError("case %d was not refused" % i)
    # what only the library can tell: alignment, an output laid over its input differently
    odd = torch.zeros(4 * 2 * 128 + 8, device="cuda").bfloat16()[1:1 + 4 * 2 * 128].view(4, 2, 128)
    for call in (lambda: f(odd, None, p, rope), lambda: f(wide[:, :2], None, p, rope, q_out=wide[:, ::2])):
        with pytest.raises(lp.LpfaError) as e:
            call()
        assert e.value.status == lp.LPFA_ERR_INVALID_ARG
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)


def test_training_chain_through_the_attention():
    """norm + rotation -> MXFP8 -> attention -> its backward -> the norm's backward, all finite, with the
    last step's gradients those of the oracle for the dQ and dK that came in."""
    lens, H = [200, 57], 4
    T = sum(lens)
    q, k, w, pos, ang = _case(77, T, H, H, "bf16", (44, 42, 42))
    meta = lp.lpfa_varlen_meta_from_lengths(lens)
    tq, tk = _dev(q, "bf16"), _dev(k, "bf16")
    tw = [_dev(x, "bf16") for x in w]
    rope, p = lp.RotaryAxes((44, 42, 42)), torch.from_numpy(pos).cuda()
    v = torch.randn(T, H, 128, device="cuda").bfloat16()
    qp, qs, kp, ks = lp.lpfa_qk_norm_rope_mxfp8(tq, tk, p, rope, meta, *tw)
    vp, vs = lp.lpfa_quantize_mxfp8_varlen(v, meta)
    o, lse = lp.lpfa_attn_fwd_varlen(qp, qs, kp, ks, vp, vs, meta, meta)
    do = torch.randn_like(o)
    dqr, dkr, _ = lp.lpfa_attn_bwd_varlen(qp, qs, kp, ks, vp, vs, o, do, lse, meta, meta)
    dq, dk, dwq, dwk = lp.lpfa_qk_norm_rope_bwd(dqr, dkr, tq, tk, p, rope, *tw)
    torch.cuda.synchronize()
    for d, dr, x, wt, dw in ((dq, dqr, q, w[0], dwq), (dk, dkr, k, w[1], dwk)):
        rx, rw, _ = onr.norm_rope_bwd(dr.float().cpu().numpy(), x, wt, ang)
        assert np.linalg.norm(d.double().cpu().numpy() - rx) <= 2.0 ** -8 * np.linalg.norm(rx)
        assert np.linalg.norm(dw.double().cpu().numpy() - rw) <= 1e-4 * np.linalg.norm(rw)
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)

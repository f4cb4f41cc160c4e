"""The MXFP4 cache on the GPU: written bytes and values read back exactly those of the oracle, and the
attention over the cache within its rounding.

Tolerance of the attention against float64 on the cached values. P is rounded to FP16 (11 bits):
2^-11 of the mean |v|. K's codes and BF16 Q are exact in the product; S sums 128 products in FP32 in
chunks that the matrix unit may truncate, 2^-20 of the largest sum |q k| / sqrt(128) =: D, and a weight
moves by as much twice over (numerator and sum); ex2 and lg2 are good to 2^-21. V's scale is held
relative to the largest one and vanishes 2^-22 below it: 2^-21 of the largest |v|. O in BF16 adds half
a step, 2^-8 of the value.
"""
import math

import numpy as np
import pytest
import torch

import workloads as wl
from oracle import meta as ometa
from oracle import mxfp4 as o4
from oracle import mxfp8 as omx
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import precision_attention_forward_b200 as lp


def _table(g, seqs, width, extra=3):
    """A random assignment of pages, with some pages unused and garbage in a wider table's tail."""
    pages = seqs * width + extra
    t = g.permutation(pages)[: seqs * width].reshape(seqs, width).astype(np.int32)
    return t, pages


def _random_cache(g, pages, heads, page, lo=120, hi=130):
    """Random codes and scale bytes in every row."""
    mk = lambda n, a, b: g.integers(a, b, size=(pages, heads, page, n), dtype=np.uint8)  # noqa: E731
    return [mk(64, 0, 256), mk(4, lo, hi), mk(64, 0, 256), mk(4, lo, hi)]


def _handle(arrays):
    return lp.Kv4Cache.from_tensors(*[torch.from_numpy(a).cuda() for a in arrays])


WRITE = [
    # lengths, starts, heads, page, dtype, mode
    ([1], [0], 1, 16, "bf16", "rceil"), ([1] * 9, [0, 15, 16, 17, 100, 31, 32, 63, 64], 4, 16, "bf16", "rceil"),
    ([5, 70, 33], [3, 0, 130], 3, 64, "fp32", "rceil"), ([300, 1, 17], None, 8, 128, "bf16", "floor"),
    ([257], [1000], 2, 256, "fp32", "floor"), ([40] * 20, [7] * 20, 5, 32, "bf16", "rceil"),
]


@pytest.mark.parametrize("case", range(len(WRITE)))
def test_write_and_read_are_exact(case):
    lens, starts, H, page, dt, mode = WRITE[case]
    g = np.random.default_rng(400 + case)
    T, S = sum(lens), len(lens)
    st = starts or [0] * S
    width = max(-(-(a + n) // page) for a, n in zip(st, lens)) + 1
    table, pages = _table(g, S, width)
    cache = _random_cache(g, pages, H, page)
    h = _handle(cache)
    x = []
    for _ in range(2):
        v = (g.standard_normal((T, H, 128)) * np.exp(3 * g.standard_normal((T, H, 1)))).astype(np.float32)
        v[0, 0, :32] = 0                        # a zero block
        v[0, 0, 32:40] = [6, 7, 5, 2.5, -0.25, 0.75, -1.25, 3.5]  # ties and a maximum between the codes
        v[T - 1, H - 1, 64:96] = 1e-38          # near the smallest scale
        x.append(wl.round_to_bf16(v) if dt == "bf16" else v)
    joint = torch.from_numpy(np.concatenate(x, axis=1)).to(torch.bfloat16 if dt == "bf16" else torch.float32).cuda()
    meta = lp.lpfa_varlen_meta_from_lengths(lens)
    tt = torch.from_numpy(table).cuda()
    tstart = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    lp.lpfa_kv4_write(joint[:, :H], joint[:, H:], h, tt, meta, start=tstart, scaling_mode=mode)
    got = lp.lpfa_kv4_read(h, tt, meta, start=tstart)
    torch.cuda.synchronize()
    want = [a.copy() for a in cache]
    cu = np.concatenate([[0], np.cumsum(lens)])
    codes, exps = [], []
    for i, v in enumerate(x):
        c, e = o4.quantize_rows(v, mode)
        codes.append(c)
        exps.append(e)
        for s in range(S):
            for j in range(lens[s]):
                at = st[s] + j
                pg, row = table[s, at // page], at % page
                want[2 * i][pg, :, row] = o4.pack_rows(c[cu[s] + j])
                want[2 * i + 1][pg, :, row] = (e[cu[s] + j] + 127).astype(np.uint8)
    for a, t in zip(want, (h.k, h.k_scales, h.v, h.v_scales)):
        assert np.array_equal(a, t.cpu().numpy())  # written exactly, and nothing else touched
    for i in range(2):
        payload, scales = got[2 * i].cpu().numpy(), got[2 * i + 1].cpu().numpy()
        ref = o4.decode(codes[i]) * np.ldexp(1.0, exps[i]).repeat(32, -1)
        assert np.array_equal(omx.dequantize_mxfp8(payload, scales, lens, H), ref)
        pad = np.full(scales.shape, 0x7F, dtype=np.uint8)  # rows past an end
        m = ometa.from_lengths(lens)
        for s in range(S):
            for b in range(m.scale_off[s + 1] - m.scale_off[s]):
                for r in range(min(128, lens[s] - 128 * b)):
                    base = (np.arange(H) + (m.scale_off[s] + b) * H) * 512 + (r % 32) * 16 + (r // 32) * 4
                    for kb in range(4):
                        pad[base + kb] = exps[i][cu[s] + 128 * b + r][:, kb] + 127
        assert np.array_equal(scales, pad)
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)


def test_bad_pages_are_skipped_and_reported():
    g = np.random.default_rng(5)
    H, page = 2, 16
    table = np.array([[0, 9], [-1, 1], [2, 3]], dtype=np.int32)  # pool of 4: 9 and -1 are not in it
    cache = _random_cache(g, 4, H, page)
    h = _handle(cache)
    x = torch.randn(30 + 20 + 40, H, 128, device="cuda").bfloat16()
    meta = lp.lpfa_varlen_meta_from_lengths([30, 20, 40])  # the last has 40 tokens, its table room for 32
    tt = torch.from_numpy(table).cuda()
    lp.lpfa_kv4_write(x, x, h, tt, meta)
    st, site = lp.lpfa_device_status()
    assert (st, site) == (lp.LPFA_ERR_INVALID_ARG, 300)
    c, e = o4.quantize_rows(x.float().cpu().numpy())
    for pg, rows, first in ((0, 16, 0), (1, 4, 30 + 16), (2, 16, 50), (3, 16, 66)):
        assert np.array_equal(h.k[pg, :, :rows].cpu().numpy(), o4.pack_rows(c[first:first + rows]).swapaxes(0, 1))
        assert np.array_equal(h.k[pg, :, rows:].cpu().numpy(), cache[0][pg, :, rows:])
    k, ks, v, vs = lp.lpfa_kv4_read(h, tt, meta)
    assert lp.lpfa_device_status() == (lp.LPFA_ERR_INVALID_ARG, 301)
    val = omx.dequantize_mxfp8(k.cpu().numpy(), ks.cpu().numpy(), [30, 20, 40], H)
    ref = o4.decode(c) * np.ldexp(1.0, e).repeat(32, -1)
    ref[16:30] = ref[30:46] = ref[82:90] = 0
    assert np.array_equal(val, ref)
    start = torch.tensor([0, 0, -5], dtype=torch.int32, device="cuda")
    before = h.k.clone()
    lp.lpfa_kv4_write(x[:3], x[:3], h, torch.tensor([[0], [1], [2]], dtype=torch.int32, device="cuda"),
                      lp.lpfa_varlen_meta_from_lengths([1, 1, 1]), start=start)
    assert lp.lpfa_device_status() == (lp.LPFA_ERR_INVALID_ARG, 300)
    assert torch.equal(h.k[2:], before[2:])
    # lengths and pages of the attention
    q = torch.randn(3, 4, 128, device="cuda").bfloat16()
    m1 = lp.lpfa_varlen_meta_from_lengths([1, 1, 1])
    lens = torch.tensor([30, -7, 1000], dtype=torch.int32, device="cuda")
    good = np.array([[0, 1], [-1, 1], [2, 3]], dtype=np.int32)
    o, lse = lp.lpfa_attn_fwd_kv4(q, h, torch.from_numpy(good).cuda(), lens, m1)
    assert lp.lpfa_device_status() == (lp.LPFA_ERR_INVALID_ARG, 302)
    _check(o, lse, q, h, good, [30, 0, 32], [1, 1, 1], False)
    o, lse = lp.lpfa_attn_fwd_kv4(q, h, tt, torch.tensor([30, 20, 9], dtype=torch.int32, device="cuda"), m1)
    assert lp.lpfa_device_status() == (lp.LPFA_ERR_INVALID_ARG, 303)
    _check(o, lse, q, h, table, [30, 20, 9], [1, 1, 1], False, skip=lambda s, at: not 0 <= table[s, at // page] < 4)


def _check(o, lse, q, h, table, kv_lens, q_lens, causal, skip=None, only=None):
    page, Hk = h.page_size, h.heads
    arr = [t.cpu().numpy() for t in (h.k, h.k_scales, h.v, h.v_scales)]
    qn, on, ln = q.double().cpu().numpy(), o.double().cpu().numpy(), lse.double().cpu().numpy()
    group = qn.shape[1] // Hk
    t0 = 0
    for s, (n, L) in enumerate(zip(kv_lens, q_lens)):
        for kh in range(Hk):
            if only is not None and (s, kh) not in only:
                continue
            seen = np.arange(n)
            if skip is not None:
                seen = seen[~np.array([skip(s, a) for a in seen], dtype=bool)]
            tb = np.where((table[s] >= 0) & (table[s] < h.num_pages), table[s], 0)
            k, v = (o4.cached_rows(arr[i], arr[i + 1], tb, n, kh, page) if n else np.zeros((0, 128)) for i in (0, 2))
            vmax = np.abs(v).max() if n else 0.0
            for j in range(L):
                lim = max(0, n - L + j + 1) if causal else n
                rows = seen[seen < lim]
                for gq in range(group):
                    hq, t = kh * group + gq, t0 + j
                    ro, rl, mean, D = o4.attend(qn[t, hq], k[rows], v[rows])
                    if not len(rows):
                        assert not on[t, hq].any() and ln[hq, t] == -math.inf
                        continue
                    dl = D * 2.0 ** -20 + 2.0 ** -20
                    assert abs(ln[hq, t] - rl) <= dl + abs(rl) * 2.0 ** -22, (s, kh, j, gq)
                    tol = np.abs(ro) * 2.0 ** -8 + mean * (2.0 ** -11 + 2 * dl) * 1.01 + vmax * 2.0 ** -21
                    d = np.abs(on[t, hq] - ro)
                    assert (d <= tol).all(), (s, kh, j, gq, float((d / tol).max()))
        t0 += L


ATTN = [
    # kv lengths, query lengths, Hq, Hk, page, causal
    ([1], [1], 1, 1, 16, False),
    ([0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65], [1] * 12, 4, 2, 16, False),
    ([127, 128, 129, 255, 256, 257, 513, 1000], [1] * 8, 2, 2, 128, False),
    ([5000, 3, 777], [1] * 3, 8, 1, 64, True),
    ([40, 3, 0, 1, 200], [5, 5, 2, 3, 7], 8, 4, 32, True),       # rows that see no key
    ([40, 3, 0, 1, 200], [5, 5, 2, 3, 7], 8, 4, 32, False),
    ([300, 90], [20, 1], 12, 4, 256, True),                      # many rows, ragged query lengths
    ([2050], [33], 24, 3, 64, True),
    ([700] * 6, [3] * 6, 6, 6, 16, True),
]


@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention_matches_the_oracle(case):
    kv, ql, Hq, Hk, page, causal = ATTN[case]
    g = np.random.default_rng(700 + case)
    S, width = len(kv), max(1, -(-max(kv) // page))
    table, pages = _table(g, S, width)
    cache = _random_cache(g, pages, Hk, page)
    # Rows that no length reaches, and unused pages, hold the worst there is: scale bytes of 255.
    owned = np.zeros((pages, page), dtype=bool)
    for s, n in enumerate(kv):
        for at in range(n):
            owned[table[s, at // page], at % page] = True
    for a in cache:
        a[np.broadcast_to(~owned[:, None], a.shape[:3])] = 255
    wide = np.full((S, width + 2), 2 ** 31 - 1, dtype=np.int32)  # entries that no token needs
    wide[:, :width] = table
    for s, n in enumerate(kv):
        wide[s, -(-n // page):] = -5
    h = _handle(cache)
    T = sum(ql)
    qj = torch.from_numpy(2 * g.standard_normal((T, Hq + 3, 128)).astype(np.float32)).bfloat16().cuda()
    q = qj[:, 2:2 + Hq]  # strided
    meta = lp.lpfa_varlen_meta_from_lengths(ql)
    tt, lens = torch.from_numpy(wide).cuda(), torch.tensor(kv, dtype=torch.int32, device="cuda")
    o, lse = lp.lpfa_attn_fwd_kv4(q, h, tt, lens, meta, causal=causal)
    o2, lse2 = lp.lpfa_attn_fwd_kv4(q, h, tt, lens, meta, causal=causal)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _check(o, lse, q, h, table, kv, ql, causal)
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)


def test_attention_over_wide_ranges_of_scales():
    """Scales over 30 binades in K (softmax all on one key) and 20 in V, which grow along the sequence, so
    that the reference moves; and queries from 2^-30 to 2^30."""
    g = np.random.default_rng(31)
    n, page = 900, 64
    table, pages = _table(g, 3, -(-n // page))
    cache = _random_cache(g, pages, 2, page, 110, 140)
    rise = np.zeros((pages, page), dtype=np.int64)
    for s in range(3):
        for at in range(n):
            rise[table[s, at // page], at % page] = 117 + (at * 20) // n
    cache[3][...] = rise[:, None, :, None]
    cache[1][..., :] = 127
    h = _handle(cache)
    q = torch.from_numpy((g.standard_normal((3, 4, 128)) * np.ldexp(1.0, [[[-30]], [[0]], [[5]]])).astype(np.float32)).bfloat16().cuda()
    lens = torch.tensor([n, n - 1, n - 13], dtype=torch.int32, device="cuda")
    o, lse = lp.lpfa_attn_fwd_kv4(q, h, torch.from_numpy(table).cuda(), lens, lp.lpfa_varlen_meta_from_lengths([1, 1, 1]))
    _check(o, lse, q, h, table, [n, n - 1, n - 13], [1, 1, 1], False)
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)


def test_one_key_constant_values_and_closed_forms():
    H, page = 2, 16
    g = np.random.default_rng(8)
    cache = _random_cache(g, 8, H, page)
    cache[2][...] = 0x33  # 1.5 everywhere
    cache[3][...] = 128   # times 2
    h = _handle(cache)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
    q = torch.randn(1, H, 128, device="cuda").bfloat16()
    meta = lp.lpfa_varlen_meta_from_lengths([1])
    for n in (1, 40, 128):
        o, lse = lp.lpfa_attn_fwd_kv4(q, h, table, torch.tensor([n], dtype=torch.int32, device="cuda"), meta)
        # constant V gives V: numerator and sum differ by P's rounding, 2^-11, below BF16's half step of 3
        assert (o == 3.0).all()
    z = torch.zeros_like(q)
    o, lse = lp.lpfa_attn_fwd_kv4(z, h, table, torch.tensor([100], dtype=torch.int32, device="cuda"), meta)
    assert torch.allclose(lse, torch.full_like(lse, math.log(100.0)), rtol=0, atol=2e-6)


def test_many_sequences_large_batches_and_long_splits():
    g = np.random.default_rng(12)
    for S, kvmax, Hq, Hk, page in ((600, 90, 4, 4, 16), (300, 400, 8, 8, 32), (2, 9000, 2, 1, 128), (1, 40000, 4, 2, 256)):
        kv = [int(x) for x in g.integers(0, kvmax + 1, S)]
        kv[-1] = kvmax
        table, pages = _table(g, S, -(-kvmax // page))
        h = _handle(_random_cache(g, pages, Hk, page))
        q = torch.from_numpy(2 * g.standard_normal((S, Hq, 128)).astype(np.float32)).bfloat16().cuda()
        o, lse = lp.lpfa_attn_fwd_kv4(q, h, torch.from_numpy(table).cuda(), torch.tensor(kv, dtype=torch.int32, device="cuda"),
                                      lp.lpfa_varlen_meta_from_lengths([1] * S))
        pick = {(int(s), int(g.integers(Hk))) for s in list(g.integers(0, S, 25)) + [S - 1]}
        _check(o, lse, q, h, table, kv, [1] * S, False, only=pick)
        # nothing is left out where no oracle row was taken
        empty = torch.tensor([n == 0 for n in kv], device="cuda")
        assert torch.isfinite(o).all() and torch.equal(torch.isinf(lse).all(0), empty)
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)


def test_decoding_steps_in_a_graph_with_growing_lengths():
    """Append one token and attend, captured once and replayed as the lengths grow in place; each replay
    agrees with the oracle. Streams: the same step on a stream of its own gives the same bits."""
    g = np.random.default_rng(20)
    S, Hq, Hk, page = 3, 4, 2, 16
    table, pages = _table(g, S, 4)
    h = _handle(_random_cache(g, pages, Hk, page))
    tt = torch.from_numpy(table).cuda()
    meta = lp.lpfa_varlen_meta_from_lengths([1] * S)
    start = torch.tensor([14, 30, 0], dtype=torch.int32, device="cuda")
    lens = start + 1
    q = torch.zeros(S, Hq, 128, device="cuda").bfloat16()
    k, v = torch.zeros(S, Hk, 128, device="cuda").bfloat16(), torch.zeros(S, Hk, 128, device="cuda").bfloat16()
    out, lse = torch.empty_like(q), torch.empty(Hq, S, device="cuda")

    def step(stream=None, o=out, l=lse):
        lp.lpfa_kv4_write(k, v, h, tt, meta, start=start, stream=stream)
        lp.lpfa_attn_fwd_kv4(q, h, tt, lens, meta, out=o, lse=l, stream=stream)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(6):
        for x in (q, k, v):
            x.copy_(torch.from_numpy(g.standard_normal(x.shape).astype(np.float32)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        _check(out, lse, q, h, table, lens.tolist(), [1] * S, False)
        side = torch.cuda.Stream()
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        step(side, o2, l2)
        side.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        start += 1
        lens += 1
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)


def test_outputs_stay_inside_their_buffers():
    g = np.random.default_rng(25)
    kv, ql, Hq, Hk, page = [100, 7], [3, 2], 6, 2, 32
    table, pages = _table(g, 2, 4)
    h = _handle(_random_cache(g, pages, Hk, page))
    T = sum(ql)
    q = torch.randn(T, Hq, 128, device="cuda").bfloat16()
    meta, lens = lp.lpfa_varlen_meta_from_lengths(ql), torch.tensor(kv, dtype=torch.int32, device="cuda")
    ob = torch.full((T * Hq * 128 + 256,), 9.0, dtype=torch.bfloat16, device="cuda")
    lb = torch.full((T * Hq + 64,), 9.0, device="cuda")
    o, l = ob[128:-128].view(T, Hq, 128), lb[32:-32].view(Hq, T)
    lp.lpfa_attn_fwd_kv4(q, h, torch.from_numpy(table).cuda(), lens, meta, causal=True, out=o, lse=l)
    torch.cuda.synchronize()
    assert (ob[:128] == 9).all() and (ob[-128:] == 9).all() and (lb[:32] == 9).all() and (lb[-32:] == 9).all()
    _check(o, l, q, h, table, kv, ql, True)


def test_serving_chain_agrees_with_the_forward_over_the_read_cache():
    """norm + rotation -> cache -> attention, against the cache read back as MXFP8 and the block-scaled
    forward in bf16 PV mode, with queries that MXFP8 holds exactly. Both are within their own bounds of
    the oracle: P to 2^-11 here and 2^-9 there, and two BF16 outputs."""
    g = np.random.default_rng(40)
    lens, H, page = [190, 65, 300], 4, 64
    T, S = sum(lens), len(lens)
    x = torch.from_numpy(g.standard_normal((T, 2 * H, 128)).astype(np.float32)).bfloat16().cuda()
    v = torch.from_numpy(g.standard_normal((T, H, 128)).astype(np.float32)).bfloat16().cuda()
    meta = lp.lpfa_varlen_meta_from_lengths(lens)
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
    rope = lp.RotaryAxes((128,), pairing="half")
    qp, qs, _, _ = lp.lpfa_qk_norm_rope_mxfp8(x[:, :H], None, pos, rope, meta)
    _, k = lp.lpfa_qk_norm_rope(x[:, :H], x[:, H:], pos, rope)
    table, pages = _table(g, S, -(-max(lens) // page))
    cache, tt = lp.Kv4Cache(pages, H, page), torch.from_numpy(table).cuda()
    lp.lpfa_kv4_write(k, v, cache, tt, meta)
    q = lp.lpfa_dequantize_mxfp8_varlen(qp, qs, meta)
    o, lse = lp.lpfa_attn_fwd_kv4(q, cache, tt, torch.tensor(lens, dtype=torch.int32, device="cuda"), meta)
    kp, ks, vp, vs = lp.lpfa_kv4_read(cache, tt, meta)
    o8, lse8 = lp.lpfa_attn_fwd_varlen(qp, qs, kp, ks, vp, vs, meta, meta)
    torch.cuda.synchronize()
    assert float((lse - lse8).abs().max()) <= gu.LSE_MAX_ABS
    d = (o.double() - o8.double())
    assert float(d.norm() / o8.double().norm()) <= gu.O_REL_L2 and float(d.abs().max()) <= gu.O_MAX_ABS
    _check(o, lse, q, cache, table, lens, lens, False, only={(1, 2)})
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)


def test_refusals():
    h = lp.Kv4Cache(4, 2, 16)
    x = torch.zeros(3, 2, 128, device="cuda").bfloat16()
    q = torch.zeros(3, 4, 128, device="cuda").bfloat16()
    m = lp.lpfa_varlen_meta_from_lengths([1, 1, 1])
    t = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    n = torch.zeros(3, dtype=torch.int32, device="cuda")
    W, R, A = lp.lpfa_kv4_write, lp.lpfa_kv4_read, lp.lpfa_attn_fwd_kv4
    bad = [
        lambda: lp.Kv4Cache(0, 2, 16), lambda: lp.Kv4Cache(4, 2, 48), lambda: lp.Kv4Cache(4, 0, 16),
        lambda: lp.Kv4Cache(4, 2, 16, device="cpu"),
        lambda: lp.Kv4Cache.from_tensors(h.k, h.k_scales, h.v, h.v_scales[:3]),
        lambda: lp.Kv4Cache.from_tensors(h.k[:, :, ::2], h.k_scales, h.v, h.v_scales),
        lambda: W(x, x[:2], h, t, m), lambda: W(x.half(), x.half(), h, t, m), lambda: W(x, x.float(), h, t, m),
        lambda: W(q, q, h, t, m), lambda: W(x[:2], x[:2], h, t, m), lambda: W(x.cpu(), x.cpu(), h, t, m),
        lambda: W(x, x, h, t.long(), m), lambda: W(x, x, h, t[:2], m), lambda: W(x, x, h, t.cpu(), m),
        lambda: W(x, x, h, t, m, start=n.long()), lambda: W(x, x, h, t, m, start=n[:2]),
        lambda: W(x, x, h, t, m, scaling_mode="up"), lambda: W(x, x, h, t, lp.lpfa_varlen_meta_fill_host([1, 1, 1])),
        lambda: R(h, t, m, k_payload=x), lambda: R(h, t[:, :0], m),
        lambda: A(q.float(), h, t, n, m), lambda: A(q[:, :3], h, t, n, m), lambda: A(q[:2], h, t, n, m),
        lambda: A(q, h, t, None, m), lambda: A(q, h, t, n.long(), m), lambda: A(q, h, t, n[:2], m),
        lambda: A(q, h, t, n, m, out=q[:2]), lambda: A(q, h, t, n, m, lse=torch.zeros(3, 4, device="cuda")),
        lambda: A(q, h, torch.zeros(2, 3, dtype=torch.int32, device="cuda").t(), n, m),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError("case %d was not refused" % i)
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)

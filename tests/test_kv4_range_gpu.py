"""The attention over the MXFP4 cache where the scales of K and V lie far apart: between the four channel
blocks of a head, between the keys, and between what a row sees or weighs and what it does not.

Tolerance, for each channel apart, against float64 on the cached values. With p_j the softmax weights:
* a weight is rounded to FP16 (half a step, 2^-12 of it) after its product with V's scale, or before it and
  once more after: 2^-11 of sum p_j |v_j|;
* a weight times its scale below FP16's normal range is off by at most 2^-20 of the largest p_j 2^e_j of its
  channel block (e_j: the block's scale), times a code of at most 6, for each key;
* S moves by 2^-20 of its largest sum of magnitudes, and with it every weight, twice over; ex2, lg2: 2^-20;
* O in BF16: 2^-8 of the value. (No value here is below 2^-100 of the largest in its channel block.)
"""
import math

import numpy as np
import pytest
import torch

from oracle import mxfp4 as o4

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import precision_attention_forward_b200 as lp


def _run(seed, lens, q_lens, Hq, Hk, page, sf_of, q_of, causal=False, k_codes=None):
    """sf_of(g, which, seq, n) -> scale bytes (n, Hk, 4) of K (which 0) or V (1); q_of(g, shape) -> queries;
    k_codes: one byte for all of K's codes (random ones)."""
    g = np.random.default_rng(seed)
    S, width = len(lens), -(-max(lens) // page)
    pages = S * width + 1
    table = g.permutation(pages)[: S * width].reshape(S, width).astype(np.int32)
    mk = lambda n: g.integers(0, 256, size=(pages, Hk, page, n), dtype=np.uint8)  # noqa: E731
    cache = [mk(64), mk(4), mk(64), mk(4)]
    if k_codes is not None:
        cache[0][...] = k_codes
    for s, n in enumerate(lens):
        at = np.arange(n)
        for which in range(2):
            cache[2 * which + 1][table[s, at // page], :, at % page] = sf_of(g, which, s, n)
    h = lp.Kv4Cache.from_tensors(*[torch.from_numpy(a).cuda() for a in cache])
    q = torch.from_numpy(q_of(g, (sum(q_lens), Hq, 128)).astype(np.float32)).bfloat16().cuda()
    args = (q, h, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
            lp.lpfa_varlen_meta_from_lengths(q_lens))
    o, lse = lp.lpfa_attn_fwd_kv4(*args, causal=causal)
    o2, lse2 = lp.lpfa_attn_fwd_kv4(*args, causal=causal)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)
    qn, on, ln = q.double().cpu().numpy(), o.double().cpu().numpy(), lse.double().cpu().numpy()
    group, t0 = Hq // Hk, 0
    for s, (n, L) in enumerate(zip(lens, q_lens)):
        at = np.arange(n)
        for kh in range(Hk):
            k, v = (o4.cached_rows(cache[i], cache[i + 1], table[s], n, kh, page) for i in (0, 2))
            unit = np.ldexp(1.0, cache[3][table[s, at // page], kh, at % page].astype(np.int64) - 127).repeat(32, -1)
            for j in range(L):
                lim = max(0, n - L + j + 1) if causal else n
                for hq in range(kh * group, (kh + 1) * group):
                    x = qn[t0 + j, hq]
                    ro, rl, mean, D = o4.attend(x, k[:lim], v[:lim])
                    sc = k[:lim] @ x / math.sqrt(128.0)
                    p = np.exp(sc - rl)
                    dl = D * 2.0 ** -20 + 2.0 ** -20
                    assert abs(ln[hq, t0 + j] - rl) <= dl + abs(rl) * 2.0 ** -22, (s, kh, j, hq)
                    floor = lim * 6 * 2.0 ** -20 * (p[:, None] * unit[:lim]).max(axis=0)
                    tol = np.abs(ro) * 2.0 ** -8 + mean * (2.0 ** -11 + 2 * dl) * 1.01 + floor
                    d = np.abs(on[t0 + j, hq] - ro)
                    assert (d <= tol).all(), (s, kh, j, hq, int((d / tol).argmax()), float((d / tol).max()))
        t0 += L


def _unit(g, shape):
    return g.standard_normal(shape)


def _near(g, n, Hk, at=127):
    return g.integers(at - 2, at + 2, size=(n, Hk, 4))


@pytest.mark.parametrize("apart", [10, 21, 22, 30, 60, 110])
@pytest.mark.parametrize("shape", [([1], [1], 1, 1, 16), ([40, 333], [1, 1], 4, 2, 16), ([900], [3], 8, 2, 64)])
def test_channel_blocks_of_v_far_apart(apart, shape):
    """One channel block of V `apart` binades above the others: theirs are what they would be without it."""
    def sf(g, which, s, n):
        b = _near(g, n, shape[3])
        if which:
            b[..., 1] += apart
        return b
    _run(apart, *shape, sf, _unit)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("apart", [12, 25, 45, 90])
def test_a_large_v_that_hardly_weighs_or_is_not_seen(apart, causal):
    """Keys whose V is 2^apart above the rest: the last ones (causal rows before them do not see them), and some
    to which K gives next to no weight."""
    lens, q_lens, Hq, Hk = [50, 700, 1500], [5, 5, 4], 4, 2

    def sf(g, which, s, n):
        b = _near(g, n, Hk)
        if which:
            b[-2:] += apart
            b[:: 37] += apart
        else:
            b[::37] = 134  # scores of hundreds: weights of 1 or of 0
        return b
    _run(100 + apart, lens, q_lens, Hq, Hk, 32, sf, _unit, causal)


@pytest.mark.parametrize("step", [1, -1])
def test_v_rises_or_falls_along_the_sequence_while_weights_do_the_reverse(step):
    """V's scale over 60 binades along the keys, K's over 6, in either direction."""
    lens, Hk = [1300, 200], 2

    def sf(g, which, s, n):
        ramp = (np.arange(n) * (60 if which else 6) // n)[:: step if which else -step]
        return _near(g, n, Hk, 100 if which else 122) + ramp[:, None, None]
    _run(7 + step, lens, [1, 2], 4, Hk, 64, sf, _unit)


def test_many_small_weights_on_large_values_keep_their_part():
    """One key with nearly all the weight, and a thousand whose weights of 2^-30 stand on values 2^20 larger:
    together they are half of the result."""
    def sf(g, which, s, n):
        b = np.full((n, 1, 4), 147 if which else 120)
        b[500] = 127
        return b
    # K is all ones times its scale: the score is 128 * 1.838 / sqrt(128) = 20.8 = 30 log 2 at key 500, else 0.2.
    _run(50, [1024], [1], 1, 1, 16, sf, lambda g, shape: np.full(shape, 1.838), k_codes=0x22)


def test_scales_of_k_over_thirty_binades_and_of_queries_over_sixty():
    """K's scales far apart between the blocks of a row and between rows, queries from 2^-30 to 2^30 (with K's
    scales the other way, so that the scores stay finite and of all sizes)."""
    lens, Hq, Hk = [400, 31, 90], 2, 2
    shift = [-30, 0, 30]

    def sf(g, which, s, n):
        return _near(g, n, Hk) if which else g.integers(97, 124, size=(n, Hk, 4)) - shift[s]
    _run(60, lens, [1, 1, 1], Hq, Hk, 16, sf, lambda g, shape: g.standard_normal(shape) * np.ldexp(1.0, shift)[:, None, None])


@pytest.mark.parametrize("Hq,q_len", [(4, 1), (16, 1), (16, 6)])
def test_every_scale_there_is(Hq, q_len):
    """Scale bytes of V drawn from a hundred binades for every key and block, zero blocks (byte 0) among
    them, with 8 and with 16 query rows a block."""
    lens, Hk = [260] * 24, 1

    def sf(g, which, s, n):
        if not which:
            return _near(g, n, Hk, 125)
        b = g.integers(77, 177, size=(n, Hk, 4))
        if s % 2:
            b[g.random(b.shape) < 0.1] = 0
        return b
    _run(70 + Hq + q_len, lens, [q_len] * 24, Hq, Hk, 64, sf, _unit)

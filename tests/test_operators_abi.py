"""C-ABI argument checks of the norm-and-rotation and cache entry points that need no GPU: every call
here is refused before the library touches CUDA."""
import ctypes

import pytest

import precision_attention_forward_b200 as lp

FAKE = 0x10000  # an aligned, never-dereferenced "device" address


def _meta(n=2, tokens=300):
    m = lp._Meta()
    m.num_seqs, m.total_tokens, m.total_scale_blocks, m.max_seqlen, m.dev = n, tokens, (tokens + 127) // 128 + n, tokens, FAKE
    return m


def _rows(heads=4, ptr=FAKE, ts=512, hs=128):
    return lp._Rows(ptr, ts, hs, heads)


def _op(**over):
    rope = over.pop("rope", lp.RotaryAxes((128,)))
    o = lp._NormRope(rope._ptr if rope is not None else None, FAKE, 1, 0, 0, 1, 1e-6, FAKE, 0, FAKE, 0, 0)
    for k, v in over.items():
        setattr(o, k, v)
    return o


def _refused(st, word=""):
    assert st == lp.LPFA_ERR_INVALID_ARG
    assert word in lp._lib.lpfa_last_error_message().decode()


def _forward(**over):
    a = dict(q=_rows(), k=_rows(), dt=0, tokens=300, hd=128, op=_op(), qo=_rows(ptr=2 * FAKE), ko=_rows(ptr=3 * FAKE), odt=0)
    a.update(over)
    return lp._lib.lpfa_qk_norm_rope(a["q"], a["k"], a["dt"], a["tokens"], a["hd"], a["op"], a["qo"], a["ko"], a["odt"], None)


def _rope(**over):
    r = lp.RotaryAxes((64, 64))
    for k, v in over.items():
        if isinstance(v, tuple):
            getattr(r._c, k)[v[0]] = v[1]
        else:
            setattr(r._c, k, v)
    return r


@pytest.mark.parametrize("over,word", [
    (dict(q=None), "q"), (dict(q=_rows(ptr=None)), "q"), (dict(q=_rows(heads=0)), "heads"), (dict(q=_rows(ptr=FAKE + 2)), "aligned"),
    (dict(q=_rows(ts=4)), "stride"), (dict(q=_rows(heads=1000), k=_rows(heads=30)), "heads"), (dict(dt=2), "dtype"),
    (dict(odt=7), "dtype"), (dict(tokens=0), "tokens"), (dict(tokens=2 ** 31), "tokens"), (dict(hd=64), "head_dim"),
    (dict(op=None), "op"), (dict(op=_op(norm=2)), "norm"), (dict(op=_op(eps=float("inf"))), "eps"), (dict(op=_op(eps=-1.0)), "eps"),
    (dict(op=_op(q_weight=FAKE + 8)), "weights"), (dict(op=_op(k_weight_head_stride=4)), "weights"), (dict(op=_op(weight_dtype=3)), "weight"),
    (dict(op=_op(positions=None)), "positions"), (dict(op=_op(positions=FAKE + 4, pos_int64=1)), "positions"),
    (dict(op=_op(rope=_rope(axes=0))), "axes"), (dict(op=_op(rope=_rope(axes=9))), "axes"), (dict(op=_op(rope=_rope(pairing=2))), "pairing"),
    (dict(op=_op(rope=_rope(axis=(3, 2)))), "axis"), (dict(op=_op(rope=_rope(inv_freq=(0, float("nan"))))), "finite"),
    (dict(qo=_rows(heads=3)), "heads"), (dict(ko=None), "k_out"), (dict(qo=_rows(ts=1024)), "place"), (dict(qo=_rows(), odt=1), "place"),
])
def test_norm_rope_is_checked(over, word):
    _refused(_forward(**over), word)


def test_mxfp8_and_backward_are_checked():
    f, q, k, op = lp._lib.lpfa_qk_norm_rope_mxfp8, _rows(), _rows(), _op()
    _refused(f(q, k, 0, 128, None, op, 0, FAKE, FAKE, FAKE, FAKE, None), "meta")
    _refused(f(q, k, 0, 128, _meta(), op, 5, FAKE, FAKE, FAKE, FAKE, None), "mode")
    _refused(f(q, k, 0, 128, _meta(), op, 0, FAKE, None, FAKE, FAKE, None), "NULL")
    _refused(f(q, k, 0, 128, _meta(), op, 0, FAKE, FAKE, FAKE + 4, FAKE, None), "aligned")
    b, g = lp._lib.lpfa_qk_norm_rope_bwd, _rows()
    need = lp._lib.lpfa_qk_norm_rope_bwd_workspace_bytes(4, 4, op)
    assert need > 0 and lp._lib.lpfa_qk_norm_rope_bwd_workspace_bytes(4, 4, _op(q_weight=None, k_weight=None)) == 0
    per_head = _op(q_weight_head_stride=128, k_weight_head_stride=128)
    assert lp._lib.lpfa_qk_norm_rope_bwd_workspace_bytes(4, 4, per_head) == 4 * need
    _refused(b(None, g, q, k, 0, 300, 128, op, g, g, FAKE, FAKE, FAKE, need, None), "dq_out")
    _refused(b(g, g, q, k, 0, 300, 128, op, g, None, FAKE, FAKE, FAKE, need, None), "dk")
    _refused(b(g, g, q, k, 0, 300, 128, op, g, g, None, FAKE, FAKE, need, None), "dq_weight")
    _refused(b(g, g, q, k, 0, 300, 128, op, g, g, FAKE, FAKE, None, need, None), "workspace")
    _refused(b(g, g, q, k, 0, 300, 128, op, g, g, FAKE, FAKE, FAKE, need - 1, None), "too small")
    _refused(b(g, g, q, k, 0, 300, 128, op, _rows(ts=1024), g, FAKE, FAKE, FAKE, need, None), "place")


def _cache(**over):
    c = lp._Kv4Cache(FAKE, FAKE, FAKE, FAKE, 8, 4, 64)
    for k, v in over.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("cache,table,word", [
    (_cache(k=None), None, "cache"), (_cache(v_sf=FAKE + 4), None, "aligned"), (_cache(num_pages=0), None, "pages"),
    (_cache(page_size=48), None, "page_size"), (_cache(page_size=8), None, "page_size"), (_cache(page_size=512), None, "page_size"),
    (_cache(heads=0), None, "heads"), (_cache(), lp._PageTable(None, 4, 4), "table"), (_cache(), lp._PageTable(FAKE, 4, 0), "table"),
    (_cache(), lp._PageTable(FAKE, 4, 2 ** 25), "table"), (_cache(), lp._PageTable(FAKE + 2, 4, 4), "misaligned"),
])
def test_cache_and_table_are_checked(cache, table, word):
    t = table or lp._PageTable(FAKE, 4, 4)
    _refused(lp._lib.lpfa_kv4_write(_rows(), _rows(), 0, 128, cache, t, None, _meta(), 0, None), word)
    _refused(lp._lib.lpfa_kv4_read(cache, t, None, _meta(), 128, FAKE, FAKE, FAKE, FAKE, None), word)
    _refused(lp._lib.lpfa_attn_fwd_kv4(_rows(), 128, cache, t, FAKE, _meta(), 0, FAKE, FAKE, None), word)


def test_cache_calls_are_checked():
    t, c, m = lp._PageTable(FAKE, 4, 4), _cache(), _meta()
    w, r, a = lp._lib.lpfa_kv4_write, lp._lib.lpfa_kv4_read, lp._lib.lpfa_attn_fwd_kv4
    _refused(w(_rows(3), _rows(), 0, 128, c, t, None, m, 0, None), "heads")
    _refused(w(_rows(), None, 0, 128, c, t, None, m, 0, None), "v")
    _refused(w(_rows(), _rows(), 9, 128, c, t, None, m, 0, None), "dtype")
    _refused(w(_rows(), _rows(), 0, 128, c, t, None, m, 9, None), "mode")
    _refused(w(_rows(), _rows(), 0, 64, c, t, None, m, 0, None), "head_dim")
    _refused(w(_rows(), _rows(), 0, 128, c, t, FAKE + 2, m, 0, None), "start")
    _refused(w(_rows(), _rows(), 0, 128, c, t, None, None, 0, None), "meta")
    _refused(r(c, t, None, m, 128, None, FAKE, FAKE, FAKE, None), "NULL")
    _refused(r(c, t, None, m, 128, FAKE + 8, FAKE, FAKE, FAKE, None), "aligned")
    _refused(a(_rows(6), 128, c, t, FAKE, m, 0, FAKE, FAKE, None), "multiple")
    _refused(a(_rows(), 128, c, t, None, m, 0, FAKE, FAKE, None), "NULL")
    _refused(a(_rows(), 128, c, t, FAKE, m, 2, FAKE, FAKE, None), "causal")
    _refused(a(_rows(), 128, c, t, FAKE, m, 0, FAKE + 4, FAKE, None), "aligned")
    _refused(a(_rows(ts=4), 128, c, t, FAKE, m, 0, FAKE, FAKE, None), "stride")


def test_plans_are_checked():
    for bad in (dict(dims=(63,)), dict(dims=(100, 40)), dict(dims=()), dict(theta=0.0), dict(theta=(1e4, 1e4)),
                dict(pairing="both"), dict(dims=(2,) * 9)):
        with pytest.raises(ValueError):
            lp.RotaryAxes(**bad)
    for f, ax in (([1.0] * 63, None), ([1.0] * 64, [0] * 63), ([1.0] * 64, [-1] + [0] * 63), ([float("inf")] * 64, None),
                  ([1.0] * 64, [8] + [0] * 63)):
        with pytest.raises(ValueError):
            lp.RotaryAxes.from_frequencies(f, ax)
    r = lp.RotaryAxes((44, 42, 42), theta=(1e4, 1e4, 256.0))
    assert r.axes == 3 and r.axis.count(0) == 22 and r.inv_freq[0] == 1.0 and r.inv_freq[43] == 1.0
    assert abs(r.inv_freq[44] - 256.0 ** (-2 / 42)) < 1e-15
    assert ctypes.sizeof(lp._Rotary) == 8 + 64 * 8 + 64

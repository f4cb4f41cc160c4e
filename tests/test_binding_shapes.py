"""The attention calls of the binding compare the tensors' shapes with each other and with the metadata: a cache
of fewer heads than the queries, say, is refused, and not read past its end. Every call here is refused before
the library is called, so the tensors may as well lie on the CPU."""
import pytest
import torch

import precision_attention_forward_b200 as lp

LENS_Q, LENS_K, H = [5, 130], [128, 3], 4
MQ, MK = lp.lpfa_varlen_meta_fill_host(LENS_Q), lp.lpfa_varlen_meta_fill_host(LENS_K)
U8, BF16, F32 = torch.uint8, torch.bfloat16, torch.float32


def _rows(n, heads=H, dtype=U8):
    return torch.zeros(n, heads, 128, dtype=dtype)


def _args(**over):
    a = dict(q=_rows(135), q_sf=torch.zeros(MQ.scale_bytes(H), dtype=U8), k=_rows(131),
             k_sf=torch.zeros(MK.scale_bytes(H), dtype=U8), v=_rows(131), v_sf=torch.zeros(MK.scale_bytes(H), dtype=U8))
    a.update(over)
    return a


BAD = [
    (dict(k=_rows(131, 1), v=_rows(131, 1), k_sf=torch.zeros(MK.scale_bytes(1), dtype=U8),
          v_sf=torch.zeros(MK.scale_bytes(1), dtype=U8)), "k must"),      # a grouped cache read back
    (dict(v=_rows(131, 1)), "v must"), (dict(k=_rows(130)), "k must"), (dict(v=_rows(7)), "v must"), (dict(k=_rows(131, 8)), "k must"),
    (dict(q=_rows(134)), "q must"), (dict(q=torch.zeros(135, H, 64, dtype=U8)), "q must"),
    (dict(q_sf=torch.zeros(MQ.scale_bytes(H) - 512, dtype=U8)), "q_sf must"),
    (dict(k_sf=torch.zeros(MK.scale_bytes(1), dtype=U8)), "k_sf must"),
    (dict(v_sf=torch.zeros(MK.scale_bytes(H) - 1, dtype=U8)), "v_sf must"),
    (dict(k_sf=torch.zeros(2 * MK.scale_bytes(H), dtype=U8)[::2]), "k_sf must"),
]


@pytest.mark.parametrize("case", range(len(BAD)))
def test_forward_backward_and_shared_queries_compare_shapes(case):
    over, word = BAD[case]
    a = _args(**over)
    t = [a[n] for n in ("q", "q_sf", "k", "k_sf", "v", "v_sf")]
    with pytest.raises(ValueError, match=word):
        lp.lpfa_attn_fwd_varlen(*t, MQ, MK)
    o = torch.zeros(a["q"].shape, dtype=BF16)
    lse = torch.zeros(H, a["q"].shape[0])
    with pytest.raises(ValueError, match=word):
        lp.lpfa_attn_bwd_varlen(*t, o, o, lse, MQ, MK)
    if word != "q must" and word != "q_sf must":  # a shared query set is one sequence
        one = lp.lpfa_varlen_meta_fill_host([7])
        t[0], t[1] = _rows(7), torch.zeros(one.scale_bytes(H), dtype=U8)
        with pytest.raises(ValueError, match=word):
            lp.lpfa_attn_fwd_shared_q(*t, one, MK)


@pytest.mark.parametrize("mode", ["fp8", "bf16v", "mxfp8"])
def test_other_modes_compare_shapes(mode):
    dt = BF16 if mode == "bf16v" else U8
    a = _args(v=_rows(131, 2, dt), v_sf=None if mode != "mxfp8" else _args()["v_sf"])
    with pytest.raises(ValueError, match="v must"):
        lp.lpfa_attn_fwd_varlen(a["q"], a["q_sf"], a["k"], a["k_sf"], a["v"], a["v_sf"], MQ, MK, pv_mode=mode)


@pytest.mark.parametrize("over,word", [
    (dict(out=_rows(134, dtype=BF16)), "out must"), (dict(out=_rows(135, dtype=F32)), "out must"),
    (dict(out=_rows(135, 8, BF16)[:, ::2]), "out must"), (dict(lse=torch.zeros(H, 134)), "lse must"),
    (dict(lse=torch.zeros(135, H).t()), "lse must"), (dict(lse=torch.zeros(H, 135).bfloat16()), "lse must"),
])
def test_given_outputs_are_compared(over, word):
    a = _args()
    with pytest.raises(ValueError, match=word):
        lp.lpfa_attn_fwd_varlen(a["q"], a["q_sf"], a["k"], a["k_sf"], a["v"], a["v_sf"], MQ, MK, **over)

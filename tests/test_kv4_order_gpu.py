"""The attention over the cache takes the sequences longest first where there are a few rounds of blocks: every
sequence is taken once, whatever the lengths. Rows are compared with the oracle for some sequences (within the
tolerance of the other attention tests); a sequence that nobody took would leave its rows as they were filled."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import precision_attention_forward_b200 as lp
    from tests.test_kv4_gpu import _check, _handle, _random_cache, _table

LENGTHS = {
    "equal": lambda g, n: np.full(n, 1100),
    "one long": lambda g, n: np.where(np.arange(n) == n - 1, 1500, g.integers(0, 3, n)),
    "ragged": lambda g, n: np.append(g.integers(0, 1400, n - 1), 1400),
    "falling": lambda g, n: np.linspace(1300, 0, n).astype(int),
    "rising, in pairs": lambda g, n: np.linspace(0, 1300, n).astype(int) // 2 * 2,
    "around the least that is sorted": lambda g, n: g.integers(1020, 1025, n),
    "just below it": lambda g, n: np.append(g.integers(0, 1023, n - 1), 1023),
    "empty": lambda g, n: np.zeros(n, dtype=int),
}


@pytest.mark.parametrize("seqs,heads", [(300, 1), (75, 4), (1100, 1), (2, 150), (297, 4)])
@pytest.mark.parametrize("lengths", list(LENGTHS))
def test_every_sequence_is_taken_once(lengths, seqs, heads):
    g = np.random.default_rng(seqs + heads)
    page, shared = 64, 40  # the sequences take their pages from a few dozen
    kv = [int(x) for x in LENGTHS[lengths](g, seqs)]
    width = 24
    h = _handle(_random_cache(g, shared, heads, page))
    table = g.integers(0, shared, size=(seqs, width)).astype(np.int32)
    q = torch.from_numpy(2 * g.standard_normal((seqs, heads, 128)).astype(np.float32)).bfloat16().cuda()
    o = torch.full((seqs, heads, 128), float("nan"), device="cuda").bfloat16()
    lse = torch.full((heads, seqs), float("nan"), device="cuda")
    lp.lpfa_attn_fwd_kv4(q, h, torch.from_numpy(table).cuda(), torch.tensor(kv, dtype=torch.int32, device="cuda"),
                         lp.lpfa_varlen_meta_from_lengths([1] * seqs), out=o, lse=lse)
    assert not torch.isnan(o).any() and not torch.isnan(lse).any()
    pick = {(int(s), int(g.integers(heads))) for s in [0, seqs - 1, int(np.argmax(kv)), *g.integers(0, seqs, 6)]}
    _check(o, lse, q, h, table, kv, [1] * seqs, False, only=pick)
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)


def test_lengths_out_of_range_are_still_reported_and_the_rest_is_right():
    g = np.random.default_rng(3)
    seqs, page = 300, 64
    h = _handle(_random_cache(g, 40, 1, page))
    table = g.integers(0, 40, size=(seqs, 20)).astype(np.int32)  # room for 1280
    kv = [int(x) for x in g.integers(0, 1281, seqs)]
    told = list(kv)
    told[7], told[200], told[299] = -5, 2 ** 31 - 1, 1281
    kv[7], kv[200], kv[299] = 0, 1280, 1280
    q = torch.from_numpy(2 * g.standard_normal((seqs, 1, 128)).astype(np.float32)).bfloat16().cuda()
    o, lse = lp.lpfa_attn_fwd_kv4(q, h, torch.from_numpy(table).cuda(), torch.tensor(told, dtype=torch.int32, device="cuda"),
                                  lp.lpfa_varlen_meta_from_lengths([1] * seqs))
    assert lp.lpfa_device_status() == (lp.LPFA_ERR_INVALID_ARG, 302)
    _check(o, lse, q, h, table, kv, [1] * seqs, False, only={(s, 0) for s in (0, 7, 100, 200, 298, 299)})

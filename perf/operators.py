"""The operators around the attention, as cases that can be timed and compared.

Four operators: the per-head norm and multi-axis rotation of Q and K (forward and backward), the
same straight into MXFP8, the paged MXFP4 key/value cache (write, then read back as MXFP8), and
the attention over that cache. ``run`` computes them in plain torch operations where ``own`` is
false and through the library's public calls where it is true; both start from the same state.
"""
from __future__ import annotations

import math
import random

import torch

own = False

D = 128
BLOCK = 32
EPS = 1e-6
THETA = 10000.0
AXES = {1: (128,), 3: (44, 42, 42)}  # head_dim elements of each rotary axis
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------- the cases

def listed():
    return [
        # One decoding step of eight sequences: the smallest call, where the launch counts.
        dict(name="norm_rope_step", op="norm_rope", seqs=8, max_len=1, ragged=False, heads_q=16, heads_k=16,
             dtype="bf16", axes=1, pairing="half", per_head=False, lens_seed=1),
        # The self-attention input of one long video sequence: time, height and width axes.
        dict(name="norm_rope_video", op="norm_rope", seqs=1, max_len=32768, ragged=False, heads_q=24, heads_k=24,
             dtype="bf16", axes=3, pairing="interleaved", per_head=False, lens_seed=2),
        # The training step of the dense workload: gradients of Q, K and both weights.
        dict(name="norm_rope_bwd_dense", op="norm_rope_bwd", seqs=4, max_len=2048, ragged=False, heads_q=16,
             heads_k=16, dtype="bf16", axes=3, pairing="interleaved", per_head=False, lens_seed=3),
        # fp32 training with fewer key heads, one weight row per head and an odd token count.
        dict(name="norm_rope_bwd_fp32", op="norm_rope_bwd", seqs=3, max_len=2333, ragged=True, heads_q=32,
             heads_k=8, dtype="fp32", axes=1, pairing="half", per_head=True, lens_seed=4),
        # Inference on the dense workload: Q and K go straight into the attention's format.
        dict(name="norm_rope_mxfp8_dense", op="norm_rope_mxfp8", seqs=4, max_len=2048, ragged=False, heads_q=16,
             heads_k=16, dtype="bf16", axes=3, pairing="interleaved", per_head=False, lens_seed=5),
        # Packed ragged fp32 sequences, tails inside a 128-token block.
        dict(name="norm_rope_mxfp8_ragged", op="norm_rope_mxfp8", seqs=16, max_len=8192, ragged=True, heads_q=16,
             heads_k=16, dtype="fp32", axes=1, pairing="half", per_head=False, lens_seed=6),
        # One new token for each of 64 cached sequences.
        dict(name="kv4_append_step", op="kv4_cache", seqs=64, max_len=1, ragged=False, heads_k=8, dtype="bf16",
             page=64, start_max=4000, lens_seed=7),
        # Prompts of 16 ragged sequences written to the cache and read back for a long chunk.
        dict(name="kv4_prompt", op="kv4_cache", seqs=16, max_len=8192, ragged=True, heads_k=16, dtype="bf16",
             page=128, start_max=0, lens_seed=8),
        # One token of one short sequence: latency.
        dict(name="attn_kv4_short", op="attn_kv4", seqs=1, q_len=1, kv_max=513, ragged=False, heads_q=16, heads_k=16,
             page=16, causal=False, lens_seed=9),
        # A serving batch: ragged lengths (one of them empty), four query heads to a key head.
        dict(name="attn_kv4_batch", op="attn_kv4", seqs=64, q_len=1, kv_max=8192, ragged=True, heads_q=32, heads_k=8,
             page=64, causal=False, lens_seed=10),
        # Two very long sequences: the split over the keys has to fill the card.
        dict(name="attn_kv4_long", op="attn_kv4", seqs=2, q_len=1, kv_max=131072, ragged=False, heads_q=16,
             heads_k=16, page=128, causal=False, lens_seed=11),
        # Five drafted tokens for each sequence, each seeing the keys up to its own.
        dict(name="attn_kv4_draft", op="attn_kv4", seqs=8, q_len=5, kv_max=4096, ragged=True, heads_q=16, heads_k=4,
             page=32, causal=True, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "norm_rope_mxfp8", "kv4_cache", "attn_kv4"])
    seed = rng.randrange(1 << 20)
    if op == "attn_kv4":
        heads_k = rng.choice([1, 2, 4, 8, 16])
        group = rng.choice([1, 1, 2, 4, 8])
        seqs = _log_int(rng, 1, 48)
        kv_max = _log_int(rng, 64, max(128, min(65536, 2 ** 22 // (seqs * heads_k))))
        return dict(op=op, seqs=seqs, q_len=rng.choice([1, 1, 1, 2, 3, 4, 7]), kv_max=kv_max, ragged=True,
                    heads_q=heads_k * group, heads_k=heads_k, page=rng.choice([16, 32, 64, 128]),
                    causal=rng.random() < 0.5, lens_seed=seed)
    seqs = _log_int(rng, 1, 24)
    if op == "kv4_cache":
        heads_k = rng.choice([1, 2, 4, 8, 16])
        max_len = _log_int(rng, 1, max(2, 2 ** 20 // (seqs * heads_k)))
        return dict(op=op, seqs=seqs, max_len=max_len, ragged=True, heads_k=heads_k,
                    dtype=rng.choice(["bf16", "fp32"]), page=rng.choice([16, 32, 64, 128]),
                    start_max=rng.choice([0, 100, 1000]), lens_seed=seed)
    heads_k = rng.choice([1, 2, 3, 8, 16, 32])
    heads_q = heads_k * rng.choice([1, 1, 2, 4])
    top = 2 ** 19 if op == "norm_rope" else 2 ** 18
    max_len = _log_int(rng, 1, max(2, min(16384, top // (seqs * (heads_q + heads_k)))))
    return dict(op=op, seqs=seqs, max_len=max_len, ragged=True, heads_q=heads_q, heads_k=heads_k,
                dtype=rng.choice(["bf16", "fp32"]), axes=rng.choice([1, 3]),
                pairing=rng.choice(["interleaved", "half"]), per_head=rng.random() < 0.3, lens_seed=seed)


def _lengths(case):
    """Tokens of each sequence: the new ones, or the cached ones for the attention."""
    rng = random.Random(case["lens_seed"])
    top = case["kv_max"] if case["op"] == "attn_kv4" else case["max_len"]
    if not case["ragged"]:
        return [top] * case["seqs"]
    low = max(1, top // 64)
    lens = [rng.randint(low, top) for _ in range(case["seqs"])]
    if case["op"] == "attn_kv4" and case["seqs"] >= 8:
        lens[3] = 0  # a sequence whose cache is empty
    return lens


def _starts(case):
    rng = random.Random(case["lens_seed"] + 1)
    return [rng.randint(0, case["start_max"]) for _ in range(case["seqs"])]


def work(case):
    lens = _lengths(case)
    T = sum(lens)
    es = 4 if case.get("dtype") == "fp32" else 2
    if case["op"] == "attn_kv4":
        hq, hk, L = case["heads_q"], case["heads_k"], case["q_len"]
        rows = case["seqs"] * L * hq
        return {"bytes": T * hk * 2 * (D // 2 + D // BLOCK) + rows * (D * 4 + 4), "flops": 4.0 * T * L * hq * D}
    if case["op"] == "kv4_cache":
        e = 2 * T * case["heads_k"] * D  # K and V
        return {"bytes": e * (es + 2 * 17 / 32 + 33 / 32), "flops": 4.0 * e}
    e = T * (case["heads_q"] + case["heads_k"]) * D
    pos = T * case["axes"] * 4
    if case["op"] == "norm_rope":
        return {"bytes": e * 2 * es + pos, "flops": 8.0 * e}
    if case["op"] == "norm_rope_bwd":
        return {"bytes": e * 3 * es + pos, "flops": 16.0 * e}
    return {"bytes": e * (es + 33 / 32) + pos, "flops": 12.0 * e}


# ---------------------------------------------------------------------------------- the states

def _positions(lens, axes):
    """int32 (T, axes): running positions of one axis, or (time, height, width) of a patch grid."""
    rows = []
    for n in lens:
        i = torch.arange(n, dtype=torch.int64)
        if axes == 1:
            rows.append(i[:, None])
        else:
            side = max(1, int(round(n ** (1 / 3))))
            rows.append(torch.stack([i // (side * side), (i // side) % side, i % side], dim=1))
    return torch.cat(rows).to(torch.int32).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens = _lengths(case)
    T = sum(lens)
    st = {"case": dict(case), "lens": lens, "T": T}

    def randn(*shape, dtype=torch.bfloat16, gain=None):
        x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
        return (x if gain is None else x * gain).to(dtype)

    if case["op"] in ("norm_rope", "norm_rope_bwd", "norm_rope_mxfp8"):
        dt = DTYPES[case["dtype"]]
        hq, hk = case["heads_q"], case["heads_k"]
        # A projection's output: channels of different size.
        gain = torch.exp(0.5 * torch.randn(hq + hk, D, generator=gen, device="cuda"))
        qk = randn(T, hq + hk, D, dtype=dt, gain=gain)
        st["q"], st["k"] = qk[:, :hq], qk[:, hq:]  # the views that a joint projection gives
        wshape = (lambda h: (h, D)) if case["per_head"] else (lambda h: (D,))
        st["qw"] = (1 + 0.2 * torch.randn(wshape(hq), generator=gen, device="cuda")).to(dt)
        st["kw"] = (1 + 0.2 * torch.randn(wshape(hk), generator=gen, device="cuda")).to(dt)
        st["pos"] = _positions(lens, case["axes"])
        if case["op"] == "norm_rope_bwd":
            st["dq"], st["dk"] = randn(T, hq, D, dtype=dt), randn(T, hk, D, dtype=dt)
    else:
        hk, page = case["heads_k"], case["page"]
        if case["op"] == "kv4_cache":
            starts = _starts(case)
            dt = DTYPES[case["dtype"]]
            gain = torch.exp(0.5 * torch.randn(hk, D, generator=gen, device="cuda"))
            st["k"], st["v"] = randn(T, hk, D, dtype=dt, gain=gain), randn(T, hk, D, dtype=dt)
            st["start"] = torch.tensor(starts, dtype=torch.int32).cuda()
            ends = [a + n for a, n in zip(starts, lens)]
            # (sequence, position) of every new token
            seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).cuda()
            first = torch.cumsum(torch.tensor([0] + lens[:-1]), 0).cuda()
            st["token_seq"], st["token_at"] = seq, torch.arange(T, device="cuda") - first[seq] + st["start"][seq]
        else:
            ends = lens
        width = max(1, max(-(-n // page) for n in ends))
        pages = case["seqs"] * width
        st["table"] = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).view(case["seqs"], width)
        st["pages"] = pages
        k, ks = _random_pages(pages, hk, page, gen)
        v, vs = _random_pages(pages, hk, page, gen)
        st["cache"] = [k, ks, v, vs]
        if case["op"] == "attn_kv4":
            st["kv_lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
            # Queries of twice unit size: a softmax that has found what it looks for.
            st["q"] = randn(case["seqs"] * case["q_len"], case["heads_q"], D, gain=2.0)
    if case["op"] in ("norm_rope_mxfp8", "kv4_cache"):
        st["atoms"] = _atom_index(lens)
    # What a program keeps between calls: sequence metadata, the rotary plan, the cache's handle.
    if own:
        import precision_attention_forward_b200 as lp

        if case["op"] == "attn_kv4":
            st["meta"] = lp.lpfa_varlen_meta_from_lengths([case["q_len"]] * case["seqs"])
        else:
            st["meta"] = lp.lpfa_varlen_meta_from_lengths(lens)
        if "pos" in st:
            st["rope"] = lp.RotaryAxes(AXES[case["axes"]], theta=THETA, pairing=case["pairing"])
        else:
            st["handle"] = lp.Kv4Cache.from_tensors(*st["cache"])
    return st


def _random_pages(pages, heads, page, gen):
    """Pages of unit normal values in the cache's format, a thousand pages at a time."""
    codes = torch.empty((pages, heads, page, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, heads, page, D // BLOCK), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (heads * page * D))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        x = torch.randn(n, heads, page, D, generator=gen, device="cuda")
        codes[a:a + n], scales[a:a + n] = _to_mxfp4(x)
    return codes, scales


def _atom_index(lens):
    """Where the scales of (token, block) stand in the padded scale storage of one head: (block of
    128 tokens, byte) for each token and 32-element block, and the number of 128-token blocks."""
    blocks, rows = [], []
    off = 0
    for n in lens:
        r = torch.arange(n)
        blocks.append(off + r // 128)
        rows.append(r % 128)
        off += -(-n // 128)
    block, row = torch.cat(blocks), torch.cat(rows)
    byte = ((row % 32) * 16 + (row // 32) * 4)[:, None] + torch.arange(4)[None, :]
    return block.cuda(), byte.cuda(), off


# ---------------------------------------------------------------------------------- plain forms

def _frequencies(axes, device):
    """(axis, inverse frequency) of each of the 64 pairs, in 64 bits."""
    ax, fr = [], []
    for a, d in enumerate(AXES[axes]):
        for j in range(d // 2):
            ax.append(a)
            fr.append(THETA ** (-2.0 * j / d))
    return torch.tensor(ax, device=device), torch.tensor(fr, dtype=torch.float64, device=device)


def _cos_sin(st):
    """cos and sin of every (token, pair): angles in 64 bits, the factors in 32."""
    ax, fr = _frequencies(st["case"]["axes"], st["pos"].device)
    angle = st["pos"].double()[:, ax] * fr
    return torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]


def _pairs(x, pairing):
    return (x[..., 0::2], x[..., 1::2]) if pairing == "interleaved" else (x[..., :64], x[..., 64:])


def _unpairs(a, b, pairing):
    return torch.stack([a, b], dim=-1).flatten(-2) if pairing == "interleaved" else torch.cat([a, b], dim=-1)


def _norm_rope(x, w, cos, sin, pairing):
    x = x.float()
    u = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    a, b = _pairs(u, pairing)
    return _unpairs(a * cos - b * sin, a * sin + b * cos, pairing)


def _norm_rope_bwd(dy, x, w, cos, sin, pairing):
    a, b = _pairs(dy.float(), pairing)
    g = _unpairs(a * cos + b * sin, b * cos - a * sin, pairing)
    xf = x.float()
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS)
    xn = xf * r
    gx = g * xn
    dw = gx.sum(dim=0) if w.dim() == 2 else gx.sum(dim=(0, 1))
    h = g * w.float()
    dx = r * (h - xn * (h * xn).mean(-1, keepdim=True))
    return dx.to(x.dtype), dw


def _exponent(amax, top_mantissa, top_exponent):
    """The smallest e with amax <= top_mantissa * 2^top_exponent * 2^e; -127 where amax is 0."""
    m, x = torch.frexp(amax)
    e = x - 1 - top_exponent + (2 * m > top_mantissa).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)


def _to_mxfp8(x):
    """(E4M3 values, scale bytes) of (..., 128) values, one scale for 32."""
    xb = x.unflatten(-1, (4, BLOCK))
    e = _exponent(xb.abs().amax(-1), 1.75, 8)
    y = torch.ldexp(xb, -e[..., None]).flatten(-2)
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _to_e2m1(x):
    """(E2M1 magnitudes with sign, scale bytes)."""
    xb = x.unflatten(-1, (4, BLOCK))
    e = _exponent(xb.abs().amax(-1), 1.5, 2)
    y = torch.ldexp(xb, -e[..., None]).flatten(-2)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6), y), (e + 127).to(torch.uint8)


def _to_mxfp4(x):
    """The cache's bytes of (..., 128) values: element 32 b + 4 g + 2 j + n is the low (n = 0) or
    high nibble of byte 8 g + 2 b + j."""
    y, sf = _to_e2m1(x)
    a = y.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code + 8 * torch.signbit(y).to(torch.uint8)
    c = code.unflatten(-1, (4, 8, 2, 2)).transpose(-4, -3)
    return (c[..., 0] + 16 * c[..., 1]).flatten(-3), sf


def _from_mxfp4(codes):
    """The E2M1 values of the cache's bytes, in 32 bits, in the order of head_dim."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).unflatten(-2, (8, 4, 2)).transpose(-4, -3).flatten(-4)
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    return table[c.int()]


def _scales(sf):
    return torch.ldexp(torch.ones((), device=sf.device), sf.int() - 127)


def _atoms(sf, atoms):
    """(T, H, 4) scale bytes into the padded storage; rows without a token hold 2^0."""
    block, byte, blocks = atoms
    H = sf.shape[1]
    out = torch.full((blocks, H, 512), 127, dtype=torch.uint8, device=sf.device)
    out[block[:, None, None], torch.arange(H, device=sf.device)[None, :, None], byte[:, None, :]] = sf
    return out.view(-1).view(torch.float8_e8m0fnu)


def _token_slots(st):
    """(page, row) of every new token."""
    page, at = st["case"]["page"], st["token_at"]
    return st["table"][st["token_seq"], at // page].long(), at % page


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "norm_rope":
        cos, sin = _cos_sin(st)
        return [_norm_rope(st[x], st[x + "w"], cos, sin, case["pairing"]).to(st[x].dtype) for x in "qk"]
    if op == "norm_rope_bwd":
        cos, sin = _cos_sin(st)
        (dq, dqw), (dk, dkw) = [_norm_rope_bwd(st["d" + x], st[x], st[x + "w"], cos, sin, case["pairing"])
                                for x in "qk"]
        return [dq, dk, dqw, dkw]
    if op == "norm_rope_mxfp8":
        cos, sin = _cos_sin(st)
        (q, qs), (k, ks) = [_to_mxfp8(_norm_rope(st[x], st[x + "w"], cos, sin, case["pairing"])) for x in "qk"]
        return [q, _atoms(qs, st["atoms"]), k, _atoms(ks, st["atoms"])]
    if op == "kv4_cache":
        page, row = _token_slots(st)
        out = []
        for x, (codes, scales) in zip("kv", (st["cache"][:2], st["cache"][2:])):
            c, sf = _to_mxfp4(st[x].float())
            codes[page, :, row] = c
            scales[page, :, row] = sf
            out += [_from_mxfp4(codes[page, :, row]).to(torch.float8_e4m3fn), _atoms(scales[page, :, row], st["atoms"])]
        return out
    # attention: every sequence padded to the table's width
    S, L, hq, hk = case["seqs"], case["q_len"], case["heads_q"], case["heads_k"]
    kv = []
    for codes, scales in (st["cache"][:2], st["cache"][2:]):
        x = _from_mxfp4(codes[st["table"]].transpose(1, 2).flatten(2, 3))  # (S, hk, N, 128)
        sf = _scales(scales[st["table"]].transpose(1, 2).flatten(2, 3))
        kv.append((x.unflatten(-1, (4, BLOCK)) * sf[..., None]).flatten(-2))
    k, v = kv
    N = k.shape[2]
    q = st["q"].float().view(S, L, hk, hq // hk, D).permute(0, 2, 3, 1, 4).reshape(S, hk, (hq // hk) * L, D)
    s = (q @ k.transpose(-1, -2)) / math.sqrt(D)
    limit = st["kv_lens"][:, None].expand(S, L)
    if case["causal"]:
        limit = limit - (L - 1) + torch.arange(L, device=q.device)
    seen = torch.arange(N, device=q.device)[None, None, :] < limit[:, :, None]  # (S, L, N)
    seen = seen[:, None, None].expand(S, hk, hq // hk, L, N).reshape(S, hk, -1, N)
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(s - top)
    l = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(l > 0, l, torch.ones_like(l))
    lse = torch.log(l) + top
    o = o.view(S, hk, hq // hk, L, D).permute(0, 3, 1, 2, 4).reshape(S * L, hq, D)
    lse = lse.view(S, hk, hq // hk, L).permute(1, 2, 0, 3).reshape(hq, S * L)
    return [o.to(torch.bfloat16), lse]


# ---------------------------------------------------------------------------------- the library's calls

def _own(st):
    import precision_attention_forward_b200 as lp

    case = st["case"]
    op = case["op"]
    e4m3, e8m0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    if op == "norm_rope":
        return lp.lpfa_qk_norm_rope(st["q"], st["k"], st["pos"], st["rope"], st["qw"], st["kw"], eps=EPS)
    if op == "norm_rope_bwd":
        return lp.lpfa_qk_norm_rope_bwd(st["dq"], st["dk"], st["q"], st["k"], st["pos"], st["rope"], st["qw"],
                                        st["kw"], eps=EPS)
    if op == "norm_rope_mxfp8":
        q, qs, k, ks = lp.lpfa_qk_norm_rope_mxfp8(st["q"], st["k"], st["pos"], st["rope"], st["meta"], st["qw"],
                                                  st["kw"], eps=EPS)
        return [q.view(e4m3), qs.view(e8m0), k.view(e4m3), ks.view(e8m0)]
    if op == "kv4_cache":
        lp.lpfa_kv4_write(st["k"], st["v"], st["handle"], st["table"], st["meta"], start=st["start"])
        k, ks, v, vs = lp.lpfa_kv4_read(st["handle"], st["table"], st["meta"], start=st["start"])
        return [k.view(e4m3), ks.view(e8m0), v.view(e4m3), vs.view(e8m0)]
    return lp.lpfa_attn_fwd_kv4(st["q"], st["handle"], st["table"], st["kv_lens"], st["meta"],
                                causal=case["causal"])


def run(state):
    return list(_own(state) if own else _plain(state))


# ---------------------------------------------------------------------------------- 64 bits

def _exact_rotation(case, pos):
    """The 2 x 2 rotations of every token as complex numbers, (T, 64)."""
    turns = []
    for a, d in enumerate(AXES[case["axes"]]):
        f = torch.pow(torch.tensor(THETA, dtype=torch.float64, device=pos.device),
                      -torch.arange(0, d, 2, dtype=torch.float64, device=pos.device) / d)
        turns.append(pos[:, a].double().outer(f))
    t = torch.cat(turns, dim=1)
    return torch.complex(torch.cos(t), torch.sin(t))


def _exact_complex(x, pairing):
    if pairing == "interleaved":
        return torch.view_as_complex(x.reshape(*x.shape[:-1], 64, 2).contiguous())
    return torch.complex(x[..., :64].contiguous(), x[..., 64:].contiguous())


def _exact_real(z, pairing):
    if pairing == "interleaved":
        return torch.view_as_real(z).reshape(*z.shape[:-1], 128)
    return torch.cat([z.real, z.imag], dim=-1)


def _exact_grid(x, step_of, top):
    """x rounded to the nearest value of a small float format, ties to even, saturating."""
    step = step_of(x.abs())
    return (torch.round(x / step) * step).clamp(-top, top)


def _exact_block_scale(x, top):
    """log2 of the least power of two 2^e with max |x| <= top * 2^e, by trial of two."""
    amax = x.reshape(*x.shape[:-1], 4, 32).abs().amax(-1)
    e = torch.floor(torch.log2(torch.where(amax > 0, amax / top, torch.ones_like(amax))))
    e = torch.where(amax <= top * torch.exp2(e), e, e + 1)
    return torch.where(amax > 0, e, torch.full_like(e, -127.0))


def _exact_atoms(e, lens):
    """Scale values 2^e of (T, H, 4) exponents in the padded storage, sequence by sequence."""
    parts, at = [], 0
    for n in lens:
        blocks = -(-n // 128)
        pad = torch.zeros((blocks * 128, e.shape[1], 4), dtype=torch.float64, device=e.device)
        pad[:n] = e[at:at + n]
        at += n
        # (block, row quarter, row in quarter, head, kb) -> (block, head, row in quarter, quarter, kb)
        parts.append(pad.view(blocks, 4, 32, e.shape[1], 4).permute(0, 3, 2, 1, 4).reshape(-1))
    return torch.exp2(torch.cat(parts))


def exact(case, seed):
    st = prepare(case, seed)
    lens = st["lens"]
    op = case["op"]
    if op.startswith("norm_rope"):
        turn = _exact_rotation(case, st["pos"])[:, None, :]
        ys, es, dxs, dws = [], [], [], []
        for x, w in ((st["q"].double(), st["qw"].double()), (st["k"].double(), st["kw"].double())):
            rms = torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS)
            if op != "norm_rope_bwd":
                ys.append(_exact_real(_exact_complex(x / rms * w, case["pairing"]) * turn, case["pairing"]))
                continue
            dy = st["dq" if not dxs else "dk"].double()
            g = _exact_real(_exact_complex(dy, case["pairing"]) * turn.conj(), case["pairing"])
            n = x / rms
            dws.append((g * n).sum(0) if w.dim() == 2 else (g * n).sum(0).sum(0))
            # the norm's Jacobian: (I - n n^T / 128) / rms
            gw = g * w
            dxs.append((gw - n * ((n * gw).sum(-1, keepdim=True) / D)) / rms)
        if op == "norm_rope":
            return ys
        if op == "norm_rope_bwd":
            return dxs + dws
        out = []
        for y in ys:
            e = _exact_block_scale(y, 448.0)
            z = y / torch.exp2(e).repeat_interleave(32, dim=-1)
            z = _exact_grid(z, lambda a: torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3), 448.0)
            out += [z, _exact_atoms(e, lens)]
        return out
    grid = lambda a: torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()  # noqa: E731
    if op == "kv4_cache":
        out = []
        for x in (st["k"].double(), st["v"].double()):
            e = _exact_block_scale(x, 6.0)
            out += [_exact_grid(x / torch.exp2(e).repeat_interleave(32, dim=-1), grid, 6.0), _exact_atoms(e, lens)]
        return out
    L, hq, hk = case["q_len"], case["heads_q"], case["heads_k"]
    values = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    i = torch.arange(D, device="cuda")
    where = 8 * (i % 32 // 4) + 2 * (i // 32) + (i % 4) // 2
    o = torch.zeros((case["seqs"] * L, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((hq, case["seqs"] * L), -math.inf, dtype=torch.float64, device="cuda")
    for s, n in enumerate(lens):
        if not n:
            continue
        pages = st["table"][s, : -(-n // case["page"])].long()
        for h in range(hk):
            kv = []
            for codes, scales in (st["cache"][:2], st["cache"][2:]):
                c = codes[pages, h].reshape(-1, 64)[:n][:, where].int() >> (4 * (i % 2)).int()
                x = values[(c & 7).long()] * (1 - 2 * ((c >> 3) & 1)).double()
                kv.append(x * torch.exp2(scales[pages, h].reshape(-1, 4)[:n].double() - 127).repeat_interleave(32, 1))
            heads = slice(h * (hq // hk), (h + 1) * (hq // hk))
            for j in range(L):
                m = n - (L - 1 - j) if case["causal"] else n
                if m <= 0:
                    continue
                t = s * L + j
                z = st["q"][t, heads].double() @ kv[0][:m].T / math.sqrt(D)
                lse[heads, t] = torch.logsumexp(z, -1)
                o[t, heads] = torch.softmax(z, -1) @ kv[1][:m]
    return [o, lse]

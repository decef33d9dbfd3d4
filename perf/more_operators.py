"""Measured cases of long contexts over the 8-bit KV page cache: appending
keys whose positions are rotated on the way, outlines of pages, the selection
of pages by what their outlines promise (with attention over them), and
attention of sequences that share a prefix.

The cache holds one head's tokens in pages of `page_tokens` tokens, e4m3 codes
with one power-of-two scale per page for the keys and one for the values.  A
page is a run of 16-token tiles; byte b of a key tile of head_dim D is

    [D/64][4][16][16]            token t, dim 64 j + 16 g + b, at [j][g][t][b]

and of a value tile

    [D/64][4][16][4][4]          token 4 g + r, dim 64 h + 16 c + i, at [h][g][i][c][r]

A rotation takes the pair (x, y) to (x c - y s, y c + x s) with c and s of the
token's position, in 32 bits, each product and sum rounded.

A page's outline is, for each dim, the largest and the smallest number of its
keys' codes, rounded outwards to whole numbers of a power-of-two unit u of the
page's keys, the smallest with which none exceeds 127.

A page's score is the largest over the row's queries of

    sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d

with the query rounded to whole numbers of a power of two, the smallest with
which none exceeds 127 * 128; sums are whole numbers, rounded once to 32 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3_MAX = 448.0
E_MIN, E_MAX = -126, 119  # exponents of a page's scale
Q_MAX = 127.0 * 128.0


def listed():
    return [
        # one user's next token, its queries rotated with it: latency is all there is
        _append("append_one_user", seqs=1, kv_heads=8, group=4, new=1, length=777, ragged=0.0, head_dim=128, rotary=128, interleaved=False,
                moved=0, page_tokens=16, dtype="bf16", outlines=True),
        # whole prompts of the KV workload's length and heads
        _append("append_prompts", seqs=4, kv_heads=32, group=1, new=4096, length=4096, ragged=0.0, head_dim=128, rotary=128, interleaved=False,
                moved=0, page_tokens=16, dtype="bf16", outlines=True),
        # chunks of ragged prompts that begin inside a page and whose earlier pages were partly given up; half of a head rotated, in neighbouring pairs
        _append("append_ragged_chunk", seqs=7, kv_heads=4, group=3, new=515, length=5003, ragged=0.6, head_dim=64, rotary=32, interleaved=True,
                moved=1024, page_tokens=32, dtype="fp16", outlines=False),
        # the pages that one user's turn filled
        _outline("outline_one_user", seqs=1, kv_heads=8, new=291, length=777, ragged=0.0, head_dim=128, page_tokens=16),
        # all pages of long contexts, once, before they are selected from
        _outline("outline_long", seqs=2, kv_heads=8, new=131072, length=131072, ragged=0.5, head_dim=128, page_tokens=16),
        # one user's next token over a middling context: a quarter of the pages, and attention over them
        _select("sparse_one_user", seqs=1, kv_heads=8, group=4, new=1, length=4011, ragged=0.0, head_dim=128, page_tokens=16, keep=64, sink=1,
                recent=4, dtype="bf16", attend=True),
        # a decoding step of the KV workload's 512 heads
        _select("select_kv_step", seqs=16, kv_heads=32, group=1, new=1, length=4096, ragged=0.3, head_dim=128, page_tokens=16, keep=64, sink=1,
                recent=4, dtype="bf16", attend=False),
        # two long contexts: a thirty-second of the pages, and attention over them
        _select("sparse_long", seqs=2, kv_heads=8, group=8, new=1, length=131072, ragged=0.5, head_dim=128, page_tokens=16, keep=256, sink=1,
                recent=16, dtype="bf16", attend=True),
        # a draft of five tokens over large pages, odd group
        _select("select_draft", seqs=9, kv_heads=8, group=5, new=5, length=32003, ragged=0.9, head_dim=64, page_tokens=64, keep=33, sink=0,
                recent=2, dtype="fp16", attend=False),
        # four short conversations behind one instruction
        _shared("shared_few", seqs=4, kv_heads=8, group=4, new=1, prefix=1001, length=67, ragged=0.5, head_dim=128, page_tokens=16, dtype="bf16"),
        # a decoding step of the KV workload behind a prefix of its length
        _shared("shared_kv_step", seqs=16, kv_heads=32, group=1, new=1, prefix=4096, length=512, ragged=0.5, head_dim=128, page_tokens=16, dtype="bf16"),
        # many conversations over one long document
        _shared("shared_many", seqs=96, kv_heads=8, group=8, new=1, prefix=32768, length=700, ragged=0.9, head_dim=128, page_tokens=16, dtype="bf16"),
    ]


def _append(name, **c):
    return {"name": name, "op": "append", **c}


def _outline(name, **c):
    return {"name": name, "op": "outline", **c}


def _select(name, **c):
    return {"name": name, "op": "select", **c}


def _shared(name, **c):
    return {"name": name, "op": "shared", **c}


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "outline", "select", "select", "shared", "shared", "shared"])
    heads = rng.choice([1, 2, 3, 4, 8, 12, 32])
    seqs = _log_int(rng, 1, 24)
    dim = rng.choice([64, 128, 128, 192, 256])
    c = {"op": op, "seqs": seqs, "kv_heads": heads, "ragged": rng.choice([0.0, 0.3, 0.6, 0.9]), "head_dim": dim,
         "page_tokens": rng.choice([16, 16, 32, 64])}
    dtype = rng.choice(["bf16", "fp16"])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    if op == "append":
        group = rng.choice([0, 1, 2, 5, 8])
        most = (4 * 32 * 4096 * 128 * 5) // (seqs * heads * dim * (3 + 2 * group))  # as much to move as append_prompts
        new = max(1, min(rng.choice([1, 1, _log_int(rng, 2, 4096)]), most))
        length = max(new, min(most, new + rng.choice([0, _log_int(rng, 1, 4096)])))
        rotary = max(16, dim // rng.choice([1, 1, 2, 4]) // 16 * 16)
        return {**c, "group": group, "new": new, "length": length, "rotary": rotary, "interleaved": rng.random() < 0.5,
                "moved": rng.choice([0, 0, 100, 5000]), "dtype": dtype, "outlines": rng.random() < 0.5}
    most = (16 * 131072 * 128) // (seqs * heads * dim)
    if op == "outline":
        length = max(1, min(most, _log_int(rng, 1, 131072)))
        return {**c, "new": rng.choice([1, length, rng.randint(1, length)]), "length": length}
    if op == "select":
        new = rng.choice([1, 1, 1, 2, 5])
        length = max(new, min(most, _log_int(rng, 64, 131072)))
        pages = -(-length // c["page_tokens"])
        sink, recent = rng.randint(0, 2), rng.randint(2, 5)
        return {**c, "group": group, "new": new, "length": length, "keep": sink + recent + rng.randint(0, max(pages // 2, 1)),
                "sink": sink, "recent": recent, "dtype": dtype, "attend": rng.random() < 0.5 and length <= 40000}
    seqs = _log_int(rng, 1, 96)
    new = rng.choice([1, 1, 1, 2, 5])
    rows = seqs * new * group
    prefix = max(1, min(_log_int(rng, 1, 32768), (8 * 768 * 32768 * 128) // (heads * rows * dim)))
    length = max(new, min(_log_int(rng, 1, 1500), (96 * 8 * 700 * 128) // (seqs * heads * dim)))
    return {**c, "seqs": seqs, "group": group, "new": new, "prefix": prefix, "length": length, "dtype": dtype}


def _spread(n, most, ragged, phase, least):
    """n whole numbers from `most` down to about most * (1 - ragged), the first of them `most`."""
    return [max(least, int(round(most * (1.0 - ragged * ((i * phase) % 1.0))))) for i in range(n)]


def _lengths(case):
    """Tokens held by each sequence, the new ones among them."""
    least = 1 if case["op"] == "outline" else case["new"]
    return _spread(case["seqs"], case["length"], case["ragged"], 0.6180339887, least)


def _counts(case):
    """New tokens of each sequence of an append."""
    return _spread(case["seqs"], case["new"], case["ragged"], 0.7548776662, 1)


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + salt) & 0x7FFFFFFF)
    return g


def _values(gen, shape):
    """N(0, 1) with four wide channels, as keys and values have them."""
    x = torch.randn(shape, generator=gen, device="cuda")
    wide = torch.randperm(shape[-1], generator=gen, device="cuda")[:4]
    x[..., wide] *= 20.0
    return x


def _power(e):
    """2^e in 32 bits, from the bits; 0 below the normal numbers."""
    return (e.clamp(-127, 127).to(torch.int32) + 127 << 23).view(torch.float32)


def _exponent(amax):
    """Smallest e with amax <= 448 * 2^e, within the range of a page's scale."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, e - 9 + (m > 0.875), E_MIN).clamp(E_MIN, E_MAX)


def _quantise(x, e):
    """e4m3 codes (uint8) of x / 2^e; what is not finite becomes NaN's code."""
    y = (x * _power(-e)).clamp(-E4M3_MAX, E4M3_MAX)
    code = torch.nan_to_num(y).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.where(torch.isfinite(x), code, 0x7F)


def _pack_k(c):
    """Codes [..., tokens, D] as key pages [..., tokens * D]."""
    *lead, t, d = c.shape
    c = c.reshape(*lead, t // 16, 16, d // 64, 4, 16)
    n = len(lead)
    return c.permute(*range(n), n, n + 2, n + 3, n + 1, n + 4).reshape(*lead, t * d)


def _unpack_k(c, t, d):
    lead = c.shape[:-1]
    n = len(lead)
    c = c.reshape(*lead, t // 16, d // 64, 4, 16, 16)
    return c.permute(*range(n), n, n + 3, n + 1, n + 2, n + 4).reshape(*lead, t, d)


def _pack_v(c):
    """Codes [..., tokens, D] as value pages [..., tokens * D]."""
    *lead, t, d = c.shape
    c = c.reshape(*lead, t // 16, 4, 4, d // 64, 4, 16)  # tile, g, r, h, c, i
    n = len(lead)
    return c.permute(*range(n), n, n + 3, n + 1, n + 5, n + 4, n + 2).reshape(*lead, t * d)


def _unpack_v(c, t, d):
    lead = c.shape[:-1]
    n = len(lead)
    c = c.reshape(*lead, t // 16, d // 64, 4, 16, 4, 4)  # tile, h, g, i, c, r
    return c.permute(*range(n), n, n + 2, n + 5, n + 1, n + 4, n + 3).reshape(*lead, t, d)


def _decoded(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _full_pages(gen, n_pages, pt, d, pack):
    """n_pages pages of values as an earlier append left them: codes and scales."""
    codes = torch.empty((n_pages, pt * d), dtype=torch.uint8, device="cuda")
    scales = torch.empty(n_pages, device="cuda")
    step = max(1, (1 << 26) // (pt * d))
    for at in range(0, n_pages, step):
        x = _values(gen, (min(step, n_pages - at), pt, d))
        e = _exponent(x.abs().amax((1, 2)))
        codes[at:at + step] = pack(_quantise(x, e[:, None, None]))
        scales[at:at + step] = _power(e)
    return codes, scales


def _table(gen, rows, per_row, first=0):
    """Page ids in no order, as a pool that has been in use gives them."""
    ids = first + torch.randperm(rows * per_row, generator=gen, device="cuda")
    return ids.to(torch.int32).reshape(rows, per_row)


def prepare(case, seed):
    seqs, heads, pt, d = case["seqs"], case["kv_heads"], case["page_tokens"], case["head_dim"]
    op = case["op"]
    s = {"case": case, "page_tokens": pt, "head_dim": d}
    g = _gen(seed, 1)
    lens = _lengths(case)
    per_row = -(-max(lens) // pt) + 2  # two spare pages a row
    n_pages = seqs * heads * per_row
    s["pages"] = _table(g, seqs * heads, per_row).reshape(seqs, heads, per_row)
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")[:, None].expand(seqs, heads).contiguous()
    if op == "shared":
        prefix_pages = -(-case["prefix"] // pt)
        s["prefix_pages"] = _table(g, heads, prefix_pages, n_pages)
        s["prefix_lengths"] = torch.full((heads,), case["prefix"], dtype=torch.int32, device="cuda")
        n_pages += heads * prefix_pages
    s["k_codes"], s["k_scales"] = _full_pages(g, n_pages, pt, d, _pack_k)
    if op == "select":  # the outlines of full pages, and of last ones that were full before
        s["outline_codes"], s["outline_scales"] = _outlines_of(s["k_codes"], s["k_scales"], pt, d)
    if op == "outline" or op == "append" and case["outlines"]:
        s["outline_codes"] = torch.zeros((n_pages, 2, d), dtype=torch.int8, device="cuda")
        s["outline_scales"] = torch.ones(n_pages, device="cuda")
    if op == "outline" or op == "select" and not case["attend"]:
        s["v_codes"], s["v_scales"] = torch.zeros_like(s["k_codes"]), torch.ones_like(s["k_scales"])
    else:
        s["v_codes"], s["v_scales"] = _full_pages(g, n_pages, pt, d, _pack_v)
    if op == "outline":
        s["counts"] = torch.tensor([min(n, case["new"]) for n in lens], dtype=torch.int32, device="cuda")
        return s
    dtype, group = DTYPES[case["dtype"]], case["group"]
    if op == "append":
        s["counts"] = torch.tensor(_counts(case), dtype=torch.int32, device="cuda")
        s["k"] = _values(g, (seqs, case["new"], heads, d)).to(dtype)
        s["v"] = _values(g, (seqs, case["new"], heads, d)).to(dtype)
        s["q"] = torch.randn((seqs, case["new"], heads * group, d), generator=g, device="cuda").to(dtype) if group else None
        # where evictions moved tokens to lower places their positions are given
        s["positions"] = None
        if case["moved"]:
            at = s["lengths"][:, 0] - s["counts"] + case["moved"]
            s["positions"] = (at[:, None] + torch.arange(case["new"], device="cuda", dtype=torch.int32)).contiguous()
        half = case["rotary"] // 2
        n = case["length"] + case["new"] + case["moved"]
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        angle = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        return s
    s["q"] = torch.randn((seqs, case["new"], heads * group, d), generator=g, device="cuda").to(dtype)
    return s


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        from lossless_bit_level_amd import ibp_kv

        cache = ibp_kv.ibp_kv_cache(state["k_codes"], state["k_scales"], state["v_codes"], state["v_scales"],
                                    state["page_tokens"], state["head_dim"])
        outlines = (state["outline_codes"], state["outline_scales"]) if "outline_codes" in state else None
        pages, lengths = state["pages"], state["lengths"]
        if op == "append":
            q = ibp_kv.ibp_kv_append_rotated(cache, pages, lengths, state["k"], state["v"], state["cos"], state["sin"],
                                             positions=state["positions"], q=state["q"], counts=state["counts"],
                                             interleaved=c["interleaved"], outlines=outlines)
            return _append_out(state, q)
        if op == "outline":
            ibp_kv.ibp_kv_outline(cache, outlines, pages, lengths, n_new=c["new"], counts=state["counts"])
            return {"outlines": state["outline_codes"], "scales": state["outline_scales"]}
        if op == "select":
            pages, lengths, places = ibp_kv.ibp_kv_select(cache, outlines, pages, lengths, state["q"], keep_pages=c["keep"],
                                                          sink_pages=c["sink"], recent_pages=c["recent"])
            out = ibp_kv.ibp_kv_attention(cache, pages, lengths, state["q"])[0] if c["attend"] else None
            return {"pages": pages, "lengths": lengths, "places": places, "out": out}
        return {"out": ibp_kv.ibp_kv_attention_shared(cache, state["prefix_pages"], state["prefix_lengths"], pages, lengths, state["q"])}
    if op == "append":
        return _plain_append(state)
    if op == "outline":
        return _plain_outline(state)
    if op == "select":
        got = _plain_select(state)
        got["out"] = _plain_attention(state, got["pages"], got["lengths"]) if c["attend"] else None
        return got
    return _plain_shared(state)


def _append_out(state, q):
    """The rotated queries and the whole cache: the e4m3 numbers its bytes stand for, the scales, the outlines."""
    out = {"k": state["k_codes"].view(torch.float8_e4m3fn), "v": state["v_codes"].view(torch.float8_e4m3fn),
           "k_scales": state["k_scales"], "v_scales": state["v_scales"]}
    if state["q"] is not None:
        out["q"] = q
    if "outline_codes" in state:
        out["outlines"], out["outline_scales"] = state["outline_codes"], state["outline_scales"]
    return out


def _rotated(x, cos, sin, interleaved):
    """x [..., D] in 32 bits with its first 2 * cos.shape[-1] dims rotated."""
    half = cos.shape[-1]
    x = x.float()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, x[..., 2 * half:]], -1)


def _positions(state):
    """[seqs, new] positions of the new tokens (all heads of a sequence have the same length here)."""
    if state["positions"] is not None:
        return state["positions"].long()
    start = state["lengths"][:, 0].long() - state["counts"].long()
    return start[:, None] + torch.arange(state["case"]["new"], device=start.device)


def _outlines_of(codes, scales, pt, d, tokens=None):
    """Outlines of key pages: int8 [n, 2, d] (largest, smallest) and scales; `tokens`: how many of a page's tokens there are (default: all)."""
    got, got_scales = [], []
    step = max(1, (1 << 26) // (pt * d))
    for at in range(0, codes.shape[0], step):
        x = _decoded(_unpack_k(codes[at:at + step], pt, d))
        here = torch.ones(x.shape[:2], dtype=torch.bool, device=x.device) if tokens is None else \
            torch.arange(pt, device=x.device) < tokens[at:at + step, None]
        odd = (here & torch.isnan(x).any(-1)).any(-1)
        hi = torch.where(here[..., None], x, -math.inf).nan_to_num(nan=0.0, neginf=-math.inf).amax(1)
        lo = torch.where(here[..., None], x, math.inf).nan_to_num(nan=0.0, posinf=math.inf).amin(1)
        m, e = torch.frexp(torch.maximum(hi.abs(), lo.abs()).amax(1))
        e = torch.where(m > 0, e - 7 + (m > 127 / 128), -15).clamp(min=-15)
        up = _power(-e)[:, None]
        got.append(torch.stack([torch.ceil(hi * up), torch.floor(lo * up)], 1).to(torch.int8))
        s = scales[at:at + step] * _power(e)
        got_scales.append(torch.where(odd, math.nan, s))
    return torch.cat(got), torch.cat(got_scales)


def _touched(state, new):
    """Ids [rows, touched] of the pages that a row's last tokens are in, how many of each page's tokens there are, and which of them are such pages."""
    pt, lengths, table = state["page_tokens"], state["lengths"], state["pages"]
    b, heads = lengths.shape
    rows = b * heads
    end = lengths.reshape(rows).long()
    start = end - state["counts"].long().repeat_interleave(heads, output_size=rows)
    touched = (new + pt - 1) // pt + 1
    at = (start // pt)[:, None] + torch.arange(touched, device=end.device)
    used = at * pt < end[:, None]
    ids = table.reshape(rows, -1).gather(1, at.clamp(max=table.shape[-1] - 1)).long()
    return ids, (end[:, None] - at * pt).clamp(max=pt), used


def _plain_outline(state):
    _outline_into(state, state["case"]["new"])
    return {"outlines": state["outline_codes"], "scales": state["outline_scales"]}


def _outline_into(state, new):
    pt, d = state["page_tokens"], state["head_dim"]
    ids, tokens, used = _touched(state, new)
    ids, tokens = ids[used], tokens[used]
    codes, scales = _outlines_of(state["k_codes"][ids], state["k_scales"][ids], pt, d, tokens)
    state["outline_codes"][ids] = codes
    state["outline_scales"][ids] = scales


def _plain_append(state):
    pt, d = state["page_tokens"], state["head_dim"]
    k, lengths, table = state["k"], state["lengths"], state["pages"]
    b, new, heads, _ = k.shape
    rows = b * heads
    at = _positions(state).clamp(max=state["cos"].shape[0] - 1)
    cos, sin = state["cos"][at][:, :, None], state["sin"][at][:, :, None]
    turned = _rotated(k, cos, sin, state["case"]["interleaved"])
    q = None
    if state["q"] is not None:  # rows past a sequence's count get zeros
        there = torch.arange(new, device=k.device) < state["counts"][:, None]
        q = torch.where(there[..., None, None], _rotated(state["q"], cos, sin, state["case"]["interleaved"]), 0.0).to(k.dtype)
    end = lengths.reshape(rows).long()
    start = end - state["counts"].long().repeat_interleave(heads, output_size=rows)
    touched = (new + pt - 1) // pt + 1
    j = (start // pt)[:, None] + torch.arange(touched, device=k.device)
    j = j.clamp(max=table.shape[-1] - 1)
    ids = table.reshape(rows, -1).gather(1, j).long()
    pos = j[..., None] * pt + torch.arange(pt, device=k.device)
    fresh = (pos >= start[:, None, None]) & (pos < end[:, None, None])
    old = pos < start[:, None, None]
    used = fresh.any(-1)
    token = (pos - start[:, None, None]).clamp(0, new - 1).reshape(rows, -1, 1).expand(-1, -1, d)
    # a table has spare pages, so that a row's pages past its last token are its own: they are written back as they are
    for x, codes, scales, pack, unpack in ((turned, state["k_codes"], state["k_scales"], _pack_k, _unpack_k),
                                           (state["v"], state["v_codes"], state["v_scales"], _pack_v, _unpack_v)):
        x = x.permute(0, 2, 1, 3).reshape(rows, new, d).gather(1, token).float().reshape(rows, touched, pt, d)
        finite = torch.where(torch.isfinite(x) & fresh[..., None], x.abs(), 0.0)
        e = _exponent(finite.amax((2, 3)))
        before = torch.frexp(scales[ids])[1] - 1
        e = torch.where(old.any(-1), torch.maximum(e, before), e)
        held = codes[ids]
        was = unpack(held, pt, d)
        keep = _decoded(was) * _power(before - e)[..., None, None]
        c = torch.where(fresh[..., None], _quantise(x, e[..., None, None]), 0)
        c = torch.where(old[..., None], _quantise(keep, torch.zeros_like(e)[..., None, None]), c)
        codes[ids] = torch.where(used[..., None], pack(c), held)
        scales[ids] = torch.where(used, _power(e), scales[ids])
    if "outline_codes" in state:
        _outline_into(state, new)
    return _append_out(state, q)


def _order(score):
    """Whole numbers in the order of the scores: -0 is 0, NaN is above all numbers."""
    bits = (score + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    return torch.where(torch.isnan(score), 1 << 31, key)


def _plain_scores(state):
    """[rows, pages] scores in 32 bits."""
    q, table = state["q"], state["pages"]
    b, new, q_heads, d = q.shape
    heads, m = table.shape[1:]
    rows, group = b * heads, q_heads // heads
    x = q.reshape(b, new, heads, group, d).permute(0, 2, 1, 3, 4).reshape(rows, new * group, d).float()
    frac, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(frac > 0, e - 14 + (frac > Q_MAX / 16384), 0).clamp(min=-126)
    whole = torch.round(x * _power(-e)[..., None])
    # two limbs of at most 127 each: sums of products with the outlines stay exact in 32 bits
    high = torch.floor((whole + 64) / 128)
    limbs = (high, whole - 128 * high)
    ids = table.reshape(rows, m).long()
    outline = state["outline_codes"][ids].float().transpose(2, 3).reshape(rows, m, 2 * d)  # hi, lo of each dim
    up, down = whole > 0, whole < 0
    sums = [torch.matmul(torch.stack([torch.where(up, y, 0), torch.where(down, y, 0)], -1).reshape(rows, new * group, 2 * d),
                         outline.transpose(1, 2)) for y in limbs]
    total = (128 * sums[0].double() + sums[1].double()).float() * _power(e)[..., None]
    return total.amax(1) * state["outline_scales"][ids]


def _plain_select(state):
    c, pt = state["case"], state["page_tokens"]
    pages, lengths = state["pages"], state["lengths"]
    b, heads, n = pages.shape
    held = ((lengths + pt - 1) // pt).clamp(0, n)[..., None]
    at = torch.arange(n, device=pages.device)
    key = _order(_plain_scores(state).reshape(b, heads, n))
    key = torch.where((at < c["sink"]) | (at >= held - c["recent"]), 1 << 32, key)
    key = torch.where(at < held, key, -(1 << 32))
    order = torch.sort(key, dim=-1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(-1, order, at.expand_as(order).contiguous())
    kept = (rank < c["keep"]) & (at < held)
    place = torch.where(kept, torch.cumsum(kept, -1) - 1, c["keep"])
    out = [torch.full((b, heads, c["keep"] + 1), -1, dtype=torch.int32, device=pages.device).scatter_(-1, place, x)[..., :-1].contiguous()
           for x in (pages, at.to(torch.int32).expand_as(pages))]
    left = held.clamp(max=c["keep"])
    return {"pages": out[0], "lengths": (lengths - (held - left)[..., 0] * pt).to(torch.int32), "places": out[1]}


def _gathered(state, ids):
    """Keys and values [..., pages * page_tokens, D] of the pages `ids` in 32 bits."""
    pt, d = state["page_tokens"], state["head_dim"]
    ids = ids.long().clamp(min=0)
    shape = (*ids.shape[:-1], ids.shape[-1] * pt, d)
    k = (_decoded(_unpack_k(state["k_codes"][ids], pt, d)) * state["k_scales"][ids][..., None, None]).reshape(shape)
    v = (_decoded(_unpack_v(state["v_codes"][ids], pt, d)) * state["v_scales"][ids][..., None, None]).reshape(shape)
    return k, v


def _own_scores(state, pages, lengths):
    """Scores [rows, new * group, tokens] of the rows' own tokens, minus infinity where a query does not see one, and their values."""
    pt, q = state["page_tokens"], state["q"]
    b, new, q_heads, d = q.shape
    heads, per_row = pages.shape[1:]
    rows, group = b * heads, q_heads // heads
    x = q.reshape(b, new, heads, group, d).permute(0, 2, 1, 3, 4).reshape(rows, new * group, d).float()
    k, v = _gathered(state, pages.reshape(rows, per_row))
    s = torch.matmul(x, k.transpose(1, 2)) * (1.0 / math.sqrt(d))
    end = lengths.reshape(rows, 1, 1)
    at = end - new + torch.arange(new, device=q.device).repeat_interleave(group, output_size=new * group)[None, :, None]
    pos = torch.arange(per_row * pt, device=q.device)
    return torch.where(pos <= at, s, -math.inf), torch.where(pos[:, None] < end, v, 0.0)


def _heads_last(x, b, new, heads, group, dtype):
    return x.reshape(b, heads, new, group, -1).permute(0, 2, 1, 3, 4).reshape(b, new, heads * group, -1).to(dtype)


def _plain_attention(state, pages, lengths):
    q = state["q"]
    b, new, q_heads, _ = q.shape
    heads = pages.shape[1]
    s, v = _own_scores(state, pages, lengths)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return _heads_last(torch.matmul(p, v) / p.sum(-1, keepdim=True), b, new, heads, q_heads // heads, q.dtype)


def _plain_shared(state):
    q, pages = state["q"], state["pages"]
    b, new, q_heads, d = q.shape
    heads = pages.shape[1]
    group = q_heads // heads
    own_s, own_v = _own_scores(state, pages, state["lengths"])
    k, v = _gathered(state, state["prefix_pages"])                       # [heads, tokens, d]
    x = q.reshape(b, new, heads, group, d).permute(2, 0, 1, 3, 4).reshape(heads, b * new * group, d).float()
    s = torch.matmul(x, k.transpose(1, 2)) * (1.0 / math.sqrt(d))
    s = torch.where(torch.arange(k.shape[1], device=q.device) < state["prefix_lengths"][:, None, None], s, -math.inf)
    del k
    top = own_s.amax(-1).reshape(b, heads, new, group)
    top = torch.maximum(top, s.amax(-1).reshape(heads, b, new, group).transpose(0, 1))
    p = torch.exp(s - top.transpose(0, 1).reshape(heads, -1, 1))
    del s
    out = torch.matmul(p, v).reshape(heads, b, new, group, d).transpose(0, 1)
    total = p.sum(-1).reshape(heads, b, new, group).transpose(0, 1)
    p = torch.exp(own_s - top.reshape(b * heads, new * group, 1))
    out = out + torch.matmul(p, own_v).reshape(b, heads, new, group, d)
    total = total + p.sum(-1).reshape(b, heads, new, group)
    return {"out": _heads_last(out / total[..., None], b, new, heads, group, q.dtype)}


def work(case):
    heads, pt, d, lens = case["kv_heads"], case["page_tokens"], case["head_dim"], _lengths(case)
    if case["op"] == "append":
        # 16-bit keys and values in, codes out, a scale for each page written; queries in and out; a row of the tables for each position; outlines
        counts = _counts(case)
        touched = heads * sum(-(-n // pt) - (n - c) // pt for n, c in zip(lens, counts))
        values = 2.0 * heads * d * sum(counts)
        moved = (3.0 + 2.0 * case["group"]) * values + touched * (2 * 4 + 4) + 4.0 * case["rotary"] * max(counts)
        if case["outlines"]:
            moved += touched * (2 * d + 4)
        return {"bytes": moved, "flops": 1.5 * values * (1 + case["group"]) * case["rotary"] / d + 2 * values}
    if case["op"] == "outline":
        counts = [min(n, case["new"]) for n in lens]
        pages = [(-(-n // pt) - (n - c) // pt, n - (n - c) // pt * pt) for n, c in zip(lens, counts)]
        return {"bytes": float(heads * sum(t * d + p * (2 * d + 3 * 4) for p, t in pages)), "flops": 2.0 * heads * d * sum(t for _, t in pages)}
    rows, seqs = case["new"] * case["group"], case["seqs"]
    queries = 2.0 * seqs * heads * rows * d
    if case["op"] == "select":
        held = [-(-n // pt) for n in lens]
        free = [max(h - case["sink"] - case["recent"], 0) if h > case["keep"] else 0 for h in held]
        kept = sum(min(h, case["keep"]) for h in held)
        moved = queries + heads * (sum(free) * (2.0 * d + 2 * 4) + kept * 3 * 4) + 8.0 * seqs * heads
        flops = 4.0 * d * rows * heads * sum(free)
        if case["attend"]:
            tokens = heads * sum(n if h <= case["keep"] else n - (h - case["keep"]) * pt for n, h in zip(lens, held))
            moved += 2.0 * tokens * d + heads * kept * 2 * 4 + 2.0 * queries
            flops += 4.0 * d * rows * tokens
        return {"bytes": moved, "flops": flops}
    tokens = heads * (case["prefix"] + sum(lens))
    pages = heads * (-(-case["prefix"] // pt) + sum(-(-n // pt) for n in lens))
    return {"bytes": 2.0 * tokens * d + pages * 3 * 4 + 2.0 * queries, "flops": 4.0 * d * rows * heads * (seqs * case["prefix"] + sum(lens))}


# --- the same from the definitions, in 64 bits -----------------------------


def _number(code):
    """The number an e4m3 code stands for."""
    sign = -1.0 if code & 0x80 else 1.0
    e, m = (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return math.nan
    return sign * (m * 2.0 ** -9 if e == 0 else (1.0 + m / 8.0) * 2.0 ** (e - 7))


def _numbers():
    return torch.tensor([_number(c) for c in range(256)], dtype=torch.float64, device="cuda")


def _k_place(pt, d):
    """Byte of (token, dim) in a key page."""
    t, x = torch.meshgrid(torch.arange(pt), torch.arange(d), indexing="ij")
    return ((t // 16) * 16 * d + (x // 64) * 1024 + (x % 64 // 16) * 256 + (t % 16) * 16 + x % 16).cuda()


def _v_place(pt, d):
    """Byte of (token, dim) in a value page."""
    t, x = torch.meshgrid(torch.arange(pt), torch.arange(d), indexing="ij")
    return ((t // 16) * 16 * d + (x // 64) * 1024 + (t % 16 // 4) * 256 + (x % 16) * 16 + (x % 64 // 16) * 4 + t % 4).cuda()


def _nearest(x):
    """The e4m3 number nearest to x, ties to the even one, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "outline": _exact_outline, "select": _exact_select, "shared": _exact_shared}[case["op"]](s)


def _exact_turn(x, s, b, first):
    """x [tokens, heads, d] of sequence b, whose first token has the place `first`, with its pairs turned as complex numbers."""
    n, half = x.shape[0], s["cos"].shape[1]
    at = torch.arange(first, first + n, device=x.device) if s["positions"] is None else s["positions"][b, :n].long()
    unit = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]
    low = torch.arange(half, device=x.device)
    a, c = (2 * low, 2 * low + 1) if s["case"]["interleaved"] else (low, low + half)
    y = torch.complex(x[..., a], x[..., c]) * unit
    x = x.clone()
    x[..., a], x[..., c] = y.real, y.imag
    return x


def _exact_append(s):
    pt, d = s["page_tokens"], s["head_dim"]
    table, lens, counts = s["pages"].cpu().numpy(), s["lengths"].cpu().numpy(), s["counts"].cpu().numpy()
    got, tokens_of = {}, {}
    for name, place in (("k", _k_place(pt, d)), ("v", _v_place(pt, d))):
        codes, scales = _numbers()[s[name + "_codes"].long()], s[name + "_scales"].double()
        for b in range(table.shape[0]):
            end, first = int(lens[b, 0]), int(lens[b, 0]) - int(counts[b])
            x = s[name][b, :end - first].double()
            if name == "k":
                x = _exact_turn(x, s, b, first)
            for p in range(first // pt, -(-end // pt)):
                # every head of a sequence has the same length here
                lo, hi = max(first, p * pt), min(end, (p + 1) * pt)
                ids = torch.from_numpy(table[b, :, p].astype(np.int64)).cuda()
                page = torch.zeros((len(ids), pt, d), dtype=torch.float64, device="cuda")
                page[:, lo - p * pt:hi - p * pt] = x[lo - first:hi - first].permute(1, 0, 2)
                most = page.abs().amax((1, 2))
                before = max(0, lo - p * pt)
                scale = torch.exp2(torch.ceil(torch.log2(most / E4M3_MAX)).clamp(E_MIN, E_MAX))
                if before:
                    scale = torch.maximum(scale, scales[ids])
                    page[:, :before] = codes[ids][:, place[:before].reshape(-1)].reshape(-1, before, d) * scales[ids][:, None, None]
                numbers = _nearest(page / scale[:, None, None])
                flat = torch.empty((len(ids), pt * d), dtype=torch.float64, device="cuda")
                flat[:, place.reshape(-1)] = numbers.reshape(len(ids), -1)
                codes[ids], scales[ids] = flat, scale
                tokens_of[(b, p)] = hi - p * pt
        got[name], got[name + "_scales"] = codes, scales
    if s["q"] is not None:
        got["q"] = torch.zeros_like(s["q"], dtype=torch.float64)
        for b, c in enumerate(counts):
            got["q"][b, :int(c)] = _exact_turn(s["q"][b, :int(c)].double(), s, b, int(lens[b, 0]) - int(c))
    if "outline_codes" in s:
        scales, place = s["outline_scales"].double(), _k_place(pt, d)
        for (b, p), n in tokens_of.items():
            ids = torch.from_numpy(table[b, :, p].astype(np.int64)).cuda()
            scales[ids] = got["k_scales"][ids] * _exact_unit(got["k"][ids][:, place[:n].reshape(-1)])
        got["outlines"], got["outline_scales"] = None, scales
    return got


def _exact_unit(numbers):
    """Smallest power of two of which 127 are at least the largest of each row's numbers."""
    return torch.exp2(torch.ceil(torch.log2(numbers.abs().amax(-1) / 127.0)).clamp(min=-15.0))


def _exact_outline(s):
    pt, d = s["page_tokens"], s["head_dim"]
    table, lens, counts = s["pages"].cpu().numpy(), s["lengths"].cpu().numpy(), s["counts"].cpu().numpy()
    numbers, place = _numbers(), _k_place(pt, d)
    codes, scales = s["outline_codes"].double(), s["outline_scales"].double()
    for b in range(table.shape[0]):
        end = int(lens[b, 0])
        first, last = (end - int(counts[b])) // pt, -(-end // pt)
        for at, to, n in ((first, last - 1, pt), (last - 1, last, end - (last - 1) * pt)):  # the last page may be partly filled
            ids = torch.from_numpy(table[b, :, at:to].reshape(-1).astype(np.int64)).cuda()
            for part in ids.split(1 << 13):
                x = numbers[s["k_codes"][part][:, place[:n].reshape(-1)].long()]
                unit = _exact_unit(x)
                x = x.reshape(len(part), n, d) / unit[:, None, None]
                codes[part] = torch.stack([torch.ceil(x.amax(1)), torch.floor(x.amin(1))], 1)
                scales[part] = unit * s["k_scales"][part].double()
    return {"outlines": codes.to(torch.int8), "scales": scales}


def _exact_tokens(s, ids, n):
    """The first n tokens of the pages `ids`: keys and values [n, d] in 64 bits."""
    pt, d = s["page_tokens"], s["head_dim"]
    numbers, ids = _numbers(), ids[:-(-n // pt)].long()
    key = numbers[s["k_codes"][ids][:, _k_place(pt, d)].long()] * s["k_scales"][ids].double()[:, None, None]
    value = numbers[s["v_codes"][ids][:, _v_place(pt, d)].long()] * s["v_scales"][ids].double()[:, None, None]
    return key.reshape(-1, d)[:n], value.reshape(-1, d)[:n]


def _exact_select(s):
    c, pt, q = s["case"], s["page_tokens"], s["q"].double()
    b, new, q_heads, d = q.shape
    pages, lens = s["pages"].cpu().numpy(), s["lengths"].cpu().numpy()
    heads, group = pages.shape[1], q_heads // pages.shape[1]
    got = [np.full((b, heads, c["keep"]), -1, np.int32) for _ in range(2)]
    out = torch.zeros_like(q) if c["attend"] else None
    left = lens.copy()
    unit = torch.exp2(torch.ceil(torch.log2(q.abs().amax(-1, keepdim=True) / Q_MAX)))
    whole = torch.round(q / unit)
    for i in range(b):
        for h in range(heads):
            n = int(lens[i, h])
            held = -(-n // pt)
            ids = s["pages"][i, h, :held].long()
            stays = np.arange(held)
            mine = slice(h * group, (h + 1) * group)
            if held > c["keep"]:
                hi, lo = s["outline_codes"][ids].double().unbind(1)
                x = whole[i, :, mine].reshape(-1, d)
                score = (x.clamp(min=0) @ hi.T + x.clamp(max=0) @ lo.T).float() * unit[i, :, mine].reshape(-1, 1).float()
                score = (score.amax(0) * s["outline_scales"][ids]).cpu().numpy()
                middle = np.arange(c["sink"], held - c["recent"])
                best = middle[np.lexsort((middle, -score[middle]))][:c["keep"] - c["sink"] - c["recent"]]
                stays = np.concatenate([np.arange(c["sink"]), np.sort(best), np.arange(held - c["recent"], held)])
                left[i, h] = n - (held - len(stays)) * pt
            got[0][i, h, :len(stays)], got[1][i, h, :len(stays)] = pages[i, h, stays], stays
            if c["attend"]:
                m = int(left[i, h])
                key, value = _exact_tokens(s, ids[torch.from_numpy(stays).cuda()], m)
                for t in range(new):
                    seen = m - new + t + 1
                    p = torch.softmax(q[i, t, mine] @ key[:seen].T / math.sqrt(d), -1)
                    out[i, t, mine] = p @ value[:seen]
    return {"pages": torch.from_numpy(got[0]), "lengths": torch.from_numpy(left), "places": torch.from_numpy(got[1]), "out": out}


def _exact_shared(s):
    q = s["q"].double()
    b, new, q_heads, d = q.shape
    heads = s["pages"].shape[1]
    group, lens = q_heads // heads, s["lengths"].cpu().numpy()
    out = torch.zeros_like(q)
    for h in range(heads):
        mine = slice(h * group, (h + 1) * group)
        key, value = _exact_tokens(s, s["prefix_pages"][h], s["case"]["prefix"])
        first = (q[:, :, mine].reshape(-1, d) @ key.T / math.sqrt(d)).reshape(b, new, group, -1)
        for i in range(b):
            n = int(lens[i, h])
            own_key, own_value = _exact_tokens(s, s["pages"][i, h], n)
            for t in range(new):
                seen = n - new + t + 1
                rest = q[i, t, mine] @ own_key[:seen].T / math.sqrt(d)
                p = torch.softmax(torch.cat([first[i, t], rest], -1), -1)
                out[i, t, mine] = p[:, :first.shape[-1]] @ value + p[:, first.shape[-1]:] @ own_value[:seen]
    return {"out": out}

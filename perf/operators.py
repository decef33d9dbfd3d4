"""Measured cases of the 8-bit KV page cache: appending keys and values,
attention over the pages, and eviction of pages by accumulated weight.

The cache holds one head's tokens in pages of `page_tokens` tokens, e4m3 codes
with one power-of-two scale per page for the keys and one for the values.  A
page is a run of 16-token tiles; byte b of a key tile of head_dim D is

    [D/64][4][16][16]            token t, dim 64 j + 16 g + b, at [j][g][t][b]

and of a value tile

    [D/64][4][16][4][4]          token 4 g + r, dim 64 h + 16 c + i, at [h][g][i][c][r]

Sequences have a table of page ids per key/value head, lengths that count the
tokens once the new ones are in, and one accumulated attention weight per
page.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3_MAX = 448.0
E_MIN, E_MAX = -126, 119  # exponents of a page's scale


def listed():
    return [
        # one user's next token: a handful of pages are touched, so latency is all there is
        _append("append_one_user", seqs=1, kv_heads=8, new=1, length=777, ragged=0.0, head_dim=128, page_tokens=16, dtype="bf16"),
        # a decoding step of the KV workload's 16 sequences of 32 heads
        _append("append_step", seqs=16, kv_heads=32, new=1, length=4096, ragged=0.3, head_dim=128, page_tokens=16, dtype="bf16"),
        # whole prompts of the KV workload's length
        _append("append_prompts", seqs=4, kv_heads=32, new=4096, length=4096, ragged=0.0, head_dim=128, page_tokens=16, dtype="bf16"),
        # chunks of ragged prompts that begin inside a page, fp16, larger pages
        _append("append_ragged_chunk", seqs=7, kv_heads=4, new=515, length=5003, ragged=0.6, head_dim=64, page_tokens=32, dtype="fp16"),
        # one user's next token over a short context
        _attention("attend_one_user", seqs=1, kv_heads=8, group=4, new=1, length=291, ragged=0.0, head_dim=128, page_tokens=16, dtype="bf16", weights=True),
        # a decoding step of the KV workload: 16 sequences, 32 heads of their own, 4096 tokens
        _attention("attend_kv_step", seqs=16, kv_heads=32, group=1, new=1, length=4096, ragged=0.0, head_dim=128, page_tokens=16, dtype="bf16", weights=True),
        # two users with long contexts, eight query heads to a key head
        _attention("attend_long", seqs=2, kv_heads=8, group=8, new=1, length=131072, ragged=0.5, head_dim=128, page_tokens=16, dtype="bf16", weights=True),
        # a draft of five tokens checked at once, odd group, ragged lengths, large pages, no eviction
        _attention("attend_draft", seqs=9, kv_heads=8, group=5, new=5, length=8011, ragged=0.9, head_dim=64, page_tokens=64, dtype="fp16", weights=False),
        # wide heads
        _attention("attend_wide", seqs=5, kv_heads=4, group=3, new=2, length=16001, ragged=0.7, head_dim=256, page_tokens=32, dtype="bf16", weights=True),
        # one user's heads are trimmed to a budget
        _evict("evict_one_user", seqs=1, kv_heads=8, pages=65, ragged=0.0, page_tokens=16, keep=48, sink=1, recent=4),
        # the KV workload's 512 heads are halved
        _evict("evict_kv", seqs=16, kv_heads=32, pages=256, ragged=0.2, page_tokens=16, keep=128, sink=1, recent=8),
        # long contexts are cut to a quarter
        _evict("evict_long", seqs=24, kv_heads=32, pages=16384, ragged=0.5, page_tokens=16, keep=4096, sink=2, recent=64),
    ]


def _append(name, **c):
    return {"name": name, "op": "append", **c}


def _attention(name, **c):
    return {"name": name, "op": "attention", **c}


def _evict(name, **c):
    return {"name": name, "op": "evict", **c}


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "evict"])
    heads = rng.choice([1, 2, 3, 4, 8, 12, 32])
    seqs = _log_int(rng, 1, 24)
    ragged = rng.choice([0.0, 0.3, 0.6, 0.9])
    page_tokens = rng.choice([16, 16, 32, 64])
    if op == "evict":
        pages = _log_int(rng, 9, 16384)
        pages = max(9, min(pages, (24 * 32 * 16384) // (seqs * heads)))
        sink = rng.randint(0, 2)
        recent = rng.randint(1, 6)
        return {"op": op, "seqs": seqs, "kv_heads": heads, "pages": pages, "ragged": ragged,
                "page_tokens": page_tokens, "keep": rng.randint(sink + recent, pages - 1), "sink": sink, "recent": recent}
    dim = rng.choice([64, 128, 128, 192, 256])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "append":
        new = rng.choice([1, 1, _log_int(rng, 2, 4096)])
        # the new values cost at most what append_prompts does
        new = max(1, min(new, (4 * 32 * 4096 * 128) // (seqs * heads * dim)))
        most = (4 * 32 * 4096 * 128) // (seqs * heads * dim)
        length = max(new, min(most, new + rng.choice([0, _log_int(rng, 1, 4096)])))
        return {"op": op, "seqs": seqs, "kv_heads": heads, "new": new, "length": length, "ragged": ragged,
                "head_dim": dim, "page_tokens": page_tokens, "dtype": dtype}
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    new = rng.choice([1, 1, 1, 2, 3, 8])
    length = _log_int(rng, 1, 131072)
    # as much to read as attend_kv_step at most, and as much to compute as attend_long
    most = (16 * 32 * 4096 * 128) // (seqs * heads * dim)
    length = max(new, min(length, most, 8 * most // (group * new)))
    return {"op": op, "seqs": seqs, "kv_heads": heads, "group": group, "new": new, "length": length, "ragged": ragged,
            "head_dim": dim, "page_tokens": page_tokens, "dtype": dtype, "weights": rng.random() < 0.75}


def _spread(n, most, ragged, phase, least):
    """n whole numbers from `most` down to about most * (1 - ragged), the first of them `most`."""
    return [max(least, int(round(most * (1.0 - ragged * ((i * phase) % 1.0))))) for i in range(n)]


def _lengths(case):
    """Tokens held by each sequence, the new ones among them."""
    return _spread(case["seqs"], case["length"], case["ragged"], 0.6180339887, case["new"])


def _counts(case):
    """New tokens of each sequence of an append."""
    return _spread(case["seqs"], case["new"], case["ragged"], 0.7548776662, 1)


def _page_counts(case):
    return _spread(case["seqs"], case["pages"], case["ragged"], 0.6180339887, 1)


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
    x = _values(gen, (n_pages, pt, d))
    e = _exponent(x.abs().amax((1, 2)))
    codes = pack(_quantise(x, e[:, None, None])).contiguous()
    return codes, _power(e)


def _table(gen, rows, per_row):
    """Page ids in no order, as a pool that has been in use gives them."""
    ids = torch.randperm(rows * per_row, generator=gen, device="cuda")
    return ids.to(torch.int32).reshape(rows, per_row)


def prepare(case, seed):
    seqs, heads, pt = case["seqs"], case["kv_heads"], case["page_tokens"]
    s = {"case": case, "page_tokens": pt}
    g = _gen(seed, 1)
    if case["op"] == "evict":
        n = case["pages"]
        s["pages"] = _table(g, seqs * heads, n).reshape(seqs, heads, n)
        counts = torch.tensor(_page_counts(case), dtype=torch.int32, device="cuda")
        tail = torch.randint(1, pt + 1, (seqs, heads), generator=g, device="cuda", dtype=torch.int32)
        s["lengths"] = ((counts[:, None] - 1) * pt + tail).contiguous()
        # heavy-tailed weights on a coarse grid: equal ones, and many zeros
        w = torch.exp(2.0 * torch.randn((seqs, heads, n), generator=g, device="cuda"))
        s["weights"] = torch.round(w * 64.0) / 64.0
        return s
    d, dtype = case["head_dim"], DTYPES[case["dtype"]]
    lens = _lengths(case)
    per_row = -(-max(lens) // pt) + 2  # two spare pages a row
    s["pages"] = _table(g, seqs * heads, per_row).reshape(seqs, heads, per_row)
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")[:, None].expand(seqs, heads).contiguous()
    s["k_codes"], s["k_scales"] = _full_pages(g, seqs * heads * per_row, pt, d, _pack_k)
    s["v_codes"], s["v_scales"] = _full_pages(g, seqs * heads * per_row, pt, d, _pack_v)
    s["head_dim"] = d
    if case["op"] == "append":
        s["counts"] = torch.tensor(_counts(case), dtype=torch.int32, device="cuda")
        s["k"] = _values(g, (seqs, case["new"], heads, d)).to(dtype)
        s["v"] = _values(g, (seqs, case["new"], heads, d)).to(dtype)
    else:
        s["q"] = torch.randn((seqs, case["new"], heads * case["group"], d), generator=g, device="cuda").to(dtype)
        s["weights"] = torch.rand((seqs, heads, per_row), generator=g, device="cuda") if case["weights"] else None
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        from lossless_bit_level_amd import ibp_kv

        c = state["case"]
        if op == "evict":
            pages, weights, lengths = ibp_kv.ibp_kv_evict(state["pages"], state["weights"], state["lengths"], state["page_tokens"],
                                                          keep_pages=c["keep"], sink_pages=c["sink"], recent_pages=c["recent"])
            return {"pages": pages, "weights": weights, "lengths": lengths}
        cache = ibp_kv.ibp_kv_cache(state["k_codes"], state["k_scales"], state["v_codes"], state["v_scales"],
                                    state["page_tokens"], state["head_dim"])
        if op == "append":
            ibp_kv.ibp_kv_append(cache, state["pages"], state["lengths"], state["k"], state["v"], counts=state["counts"])
            return _cache_out(state)
        out, weights = ibp_kv.ibp_kv_attention(cache, state["pages"], state["lengths"], state["q"], weights=state["weights"])
        return {"out": out, "weights": weights}
    if op == "evict":
        return _plain_evict(state)
    return _plain_append(state) if op == "append" else _plain_attention(state)


def _cache_out(state):
    """The whole cache: the e4m3 numbers its bytes stand for, and the scales."""
    return {"k": state["k_codes"].view(torch.float8_e4m3fn), "v": state["v_codes"].view(torch.float8_e4m3fn),
            "k_scales": state["k_scales"], "v_scales": state["v_scales"]}


def _plain_append(state):
    pt, d = state["page_tokens"], state["head_dim"]
    k, lengths, table = state["k"], state["lengths"], state["pages"]
    b, new, heads, _ = k.shape
    rows = b * heads
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
    for x, codes, scales, pack, unpack in ((k, state["k_codes"], state["k_scales"], _pack_k, _unpack_k),
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
        scale = _power(e)
        codes[ids] = torch.where(used[..., None], pack(c), held)
        scales[ids] = torch.where(used, scale, scales[ids])
    return _cache_out(state)


def _plain_attention(state):
    pt, d = state["page_tokens"], state["head_dim"]
    q, table = state["q"], state["pages"]
    b, new, q_heads, _ = q.shape
    heads, per_row = table.shape[1], table.shape[2]
    rows, group = b * heads, q_heads // heads
    ids = table.reshape(rows, per_row).long()
    k = (_decoded(_unpack_k(state["k_codes"][ids], pt, d)) * state["k_scales"][ids][..., None, None]).reshape(rows, per_row * pt, d)
    x = q.reshape(b, new, heads, group, d).permute(0, 2, 1, 3, 4).reshape(rows, new * group, d).float()
    s = torch.matmul(x, k.transpose(1, 2)) * (1.0 / math.sqrt(d))
    del k
    end = state["lengths"].reshape(rows, 1, 1)
    at = end - new + torch.arange(new, device=q.device).repeat_interleave(group, output_size=new * group)[None, :, None]
    pos = torch.arange(per_row * pt, device=q.device)
    s = torch.where(pos <= at, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0.0, 1.0, total)
    del s
    v = (_decoded(_unpack_v(state["v_codes"][ids], pt, d)) * state["v_scales"][ids][..., None, None]).reshape(rows, per_row * pt, d)
    v = torch.where(pos[:, None] < end, v, 0.0)
    out = torch.matmul(p, v).reshape(b, heads, new, group, d).permute(0, 2, 1, 3, 4).reshape(b, new, q_heads, d).to(q.dtype)
    weights = state["weights"]
    if weights is not None:
        weights = weights + p.sum(1).reshape(rows, per_row, pt).sum(-1).reshape(b, heads, per_row)
    return {"out": out, "weights": weights}


def _plain_evict(state):
    c, pt = state["case"], state["page_tokens"]
    pages, weights, lengths = state["pages"], state["weights"], state["lengths"]
    n = pages.shape[-1]
    held = ((lengths + pt - 1) // pt).clamp(0, n)[..., None]
    at = torch.arange(n, device=pages.device)
    # whole numbers in the order of the weights: -0 is 0, NaN is above all; then the protected pages, and below all what holds nothing
    bits = (weights + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    key = torch.where(torch.isnan(weights), 1 << 31, key)
    key = torch.where((at < c["sink"]) | (at >= held - c["recent"]), 1 << 32, key)
    key = torch.where(at < held, key, -(1 << 32))
    order = torch.sort(key, dim=-1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(-1, order, at.expand_as(order).contiguous())
    kept = (rank < c["keep"]) & (at < held)
    left = held.clamp(max=c["keep"])
    place = torch.where(kept, torch.cumsum(kept, -1) - 1, left + torch.cumsum(~kept, -1) - 1)
    out_pages = torch.empty_like(pages).scatter_(-1, place, pages)
    out_weights = torch.empty_like(weights).scatter_(-1, place, torch.where(kept | (at >= held), weights, 0.0))
    return {"pages": out_pages, "weights": out_weights, "lengths": (lengths - (held - left)[..., 0] * pt).to(torch.int32)}


def work(case):
    heads, pt = case["kv_heads"], case["page_tokens"]
    if case["op"] == "evict":
        # ids and weights of every held page are read once and written once
        return {"bytes": 16.0 * heads * sum(_page_counts(case)) + 8.0 * heads * case["seqs"], "flops": 0}
    d, lens = case["head_dim"], _lengths(case)
    if case["op"] == "append":
        # 16-bit keys and values in, codes out, a scale for each page written
        touched = sum(-(-n // pt) - (n - c) // pt for n, c in zip(lens, _counts(case)))
        values = 2.0 * heads * d * sum(_counts(case))
        return {"bytes": 3.0 * values + heads * touched * (2 * 4 + 4), "flops": 4.0 * values}
    rows = case["new"] * case["group"]
    tokens = float(heads * sum(lens))
    held = heads * sum(-(-n // pt) for n in lens)
    moved = 2.0 * tokens * d + held * (2 * 4 + 4 + (8 if case["weights"] else 0))
    moved += 4.0 * case["seqs"] * heads * rows * d
    return {"bytes": moved, "flops": 4.0 * tokens * rows * d}


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
    return {"append": _exact_append, "attention": _exact_attention, "evict": _exact_evict}[case["op"]](s)


def _exact_append(s):
    pt, d = s["page_tokens"], s["head_dim"]
    table, lens, counts = s["pages"].cpu().numpy(), s["lengths"].cpu().numpy(), s["counts"].cpu().numpy()
    got = {}
    for name, place in (("k", _k_place(pt, d)), ("v", _v_place(pt, d))):
        codes, scales = _numbers()[s[name + "_codes"].long()], s[name + "_scales"].double()
        for b in range(table.shape[0]):
            x = s[name][b].double()
            for p in range((int(lens[b, 0]) - int(counts[b])) // pt, -(-int(lens[b, 0]) // pt)):
                # every head of a sequence has the same length here
                end, first = int(lens[b, 0]), int(lens[b, 0]) - int(counts[b])
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
                flat = torch.empty((len(ids), pt * d), dtype=torch.float64, device="cuda")
                flat[:, place.reshape(-1)] = _nearest(page / scale[:, None, None]).reshape(len(ids), -1)
                codes[ids], scales[ids] = flat, scale
        got[name], got[name + "_scales"] = codes, scales
    return got


def _exact_attention(s):
    pt, d, q = s["page_tokens"], s["head_dim"], s["q"].double()
    b, new, q_heads, _ = q.shape
    heads, group = s["pages"].shape[1], q_heads // s["pages"].shape[1]
    numbers, k_place, v_place = _numbers(), _k_place(pt, d), _v_place(pt, d)
    lens = s["lengths"].cpu().numpy()
    out = torch.zeros_like(q)
    weights = None if s["weights"] is None else s["weights"].double()
    for i in range(b):
        for h in range(heads):
            n = int(lens[i, h])
            held = -(-n // pt)
            ids = s["pages"][i, h, :held].long()
            key = numbers[s["k_codes"][ids][:, k_place].long()] * s["k_scales"][ids].double()[:, None, None]
            value = numbers[s["v_codes"][ids][:, v_place].long()] * s["v_scales"][ids].double()[:, None, None]
            key, value = key.reshape(-1, d)[:n], value.reshape(-1, d)[:n]
            mass = torch.zeros(held * pt, dtype=torch.float64, device="cuda")
            for t in range(new):
                seen = n - new + t + 1
                if seen <= 0:
                    continue
                rows = slice(h * group, (h + 1) * group)
                p = torch.softmax(q[i, t, rows] @ key[:seen].T / math.sqrt(d), -1)
                out[i, t, rows] = p @ value[:seen]
                mass[:seen] += p.sum(0)
            if weights is not None:
                weights[i, h, :held] += mass.reshape(held, pt).sum(1)
    return {"out": out, "weights": weights}


def _exact_evict(s):
    c, pt = s["case"], s["page_tokens"]
    pages, weights, lengths = (s[x].cpu().numpy().copy() for x in ("pages", "weights", "lengths"))
    for i in np.ndindex(lengths.shape):
        held = -(-int(lengths[i]) // pt)
        if held <= c["keep"]:
            continue
        middle = np.arange(c["sink"], held - c["recent"])
        best = middle[np.lexsort((middle, -weights[i][middle]))][:c["keep"] - c["sink"] - c["recent"]]
        stays = np.concatenate([np.arange(c["sink"]), np.sort(best), np.arange(held - c["recent"], held)])
        goes = np.setdiff1d(np.arange(held), stays)
        pages[i][:held] = pages[i][np.concatenate([stays, goes])]
        weights[i][:held] = np.concatenate([weights[i][stays], np.zeros(len(goes), np.float32)])
        lengths[i] -= len(goes) * pt
    return {"pages": torch.from_numpy(pages), "weights": torch.from_numpy(weights).double(), "lengths": torch.from_numpy(lengths)}

"""Plain oracle of long and shared contexts over the 8-bit KV pages
(include/ibp_kv_long.h): numpy, token by token, no code shared with the
library.  The rotation is defined in 32 bits, the rest in whole numbers or 64
bits."""
import numpy as np

from oracle import kv_oracle as kv


def rotate(x, cos, sin, position, interleaved):
    """x [d] (float64 of 16-bit numbers) at a position: float32 [d]."""
    x = np.asarray(x).astype(np.float32).copy()
    half = cos.shape[1]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    if 0 <= position < len(cos):
        c, s = cos[position].astype(np.float32), sin[position].astype(np.float32)
    else:
        c = s = np.full(half, np.nan, np.float32)
    with np.errstate(all="ignore"):
        first, second = x[a] * c - x[b] * s, x[b] * c + x[a] * s
    x[a], x[b] = first, second
    return x


def rotated(x, cos, sin, lengths, max_pages, page_tokens, positions=None, counts=None, interleaved=False):
    """x [n_seqs, n_new, heads, d] rotated, zeros for tokens that do not exist;
    lengths are those of the kv heads (heads a multiple of them)."""
    n_seqs, n_new, heads, _ = x.shape
    kv_heads = lengths.shape[1]
    out = np.zeros(x.shape, np.float32)
    for s in range(n_seqs):
        for h in range(heads):
            n = kv.row_length(lengths[s, h // (heads // kv_heads)], max_pages, page_tokens)
            origin, count = kv.new_tokens(n, counts, s, n_new)
            for i in range(max(0, -origin), count):
                at = origin + i if positions is None else int(positions[s, i])
                out[s, i, h] = rotate(x[s, i, h], cos, sin, at, interleaved)
    return out


def outline(k_codes, k_scales, place, page_tokens, pages, lengths, codes, scales, n_new, counts=None):
    """Brings codes int8 [n_pages, 2, d] and scales up to date, in place."""
    n_seqs, heads, max_pages = pages.shape
    for s in range(n_seqs):
        for h in range(heads):
            n = kv.row_length(lengths[s, h], max_pages, page_tokens)
            origin, count = kv.new_tokens(n, counts, s, n_new)
            if count == 0 or n == 0:
                continue
            for p in range(max(origin, 0) // page_tokens, -(-n // page_tokens)):
                page = int(pages[s, h, p])
                if not 0 <= page < len(k_scales):
                    continue
                x = kv.NUMBERS[k_codes[page][place[:min(page_tokens, n - p * page_tokens)]]]
                if np.isnan(x).any() or not np.isfinite(k_scales[page]):
                    codes[page], scales[page] = 0, np.nan
                    continue
                e = -15
                while np.abs(x).max() > 127 * 2.0 ** e:
                    e += 1
                codes[page, 0] = np.ceil(x.max(0) / 2.0 ** e)
                codes[page, 1] = np.floor(x.min(0) / 2.0 ** e)
                with np.errstate(over="ignore"):
                    scales[page] = np.float32(k_scales[page] * np.float32(2.0 ** e))


def whole_query(q):
    """(whole numbers, power of two) of a query, None if it takes no part."""
    if not np.isfinite(q).all():
        return None
    top, e = np.abs(q).max(), -126
    if top == 0:
        return np.zeros(len(q), np.int64), 1.0
    while top > 127 * 128 * 2.0 ** e:
        e += 1
    return np.rint(q / 2.0 ** e).astype(np.int64), 2.0 ** e


def score(queries, codes, scale):
    """Score (float32) of a page for whole_query's pairs."""
    with np.errstate(over="ignore", invalid="ignore"):
        best = np.float32(-np.inf)
        for whole, t in queries:
            total = int((np.where(whole > 0, whole * codes[0], whole * codes[1])).sum())
            best = max(best, np.float32(np.float32(total) * np.float32(t)))
        return np.float32(best * np.float32(scale))


def select(codes, scales, pages, lengths, page_tokens, q, keep, sink, recent, counts=None):
    """(pages, lengths, places) of the selection; q [n_seqs, n_new, q_heads, d]."""
    n_seqs, heads, max_pages = pages.shape
    group = q.shape[2] // heads
    out = np.full((n_seqs, heads, keep), -1, np.int32)
    places, left = out.copy(), np.zeros((n_seqs, heads), np.int32)
    codes = codes.astype(np.int64)
    for s in range(n_seqs):
        for h in range(heads):
            n = kv.row_length(lengths[s, h], max_pages, page_tokens)
            origin, count = kv.new_tokens(n, counts, s, q.shape[1])
            held = -(-n // page_tokens)
            stay = list(range(held))
            if held > keep:
                queries = [whole_query(q[s, i, h * group + g]) for i in range(max(0, -origin), count) for g in range(group)]
                queries = [x for x in queries if x is not None]

                def rank(p):  # NaN first, then the larger, then the lower position
                    page = int(pages[s, h, p])
                    x = score(queries, codes[page], scales[page]) if 0 <= page < len(scales) else np.float32(-np.inf)
                    return (0, 0.0, p) if np.isnan(x) else (1, -float(x), p)
                middle = sorted(range(sink, held - recent), key=rank)[:keep - sink - recent]
                stay = sorted(list(range(sink)) + middle + list(range(held - recent, held)))
            out[s, h, :len(stay)] = pages[s, h][stay]
            places[s, h, :len(stay)] = stay
            left[s, h] = n - (held - len(stay)) * page_tokens
    return out, left, places


def scales_of(scales, page_tokens, pages_row, n):
    """The magnitude of the scale of each of a row's first n tokens, 0 in holes."""
    at = np.arange(n) // page_tokens
    ids = pages_row[at] if n else np.zeros(0, np.int64)
    inside = (ids >= 0) & (ids < len(scales))
    return np.where(inside, np.abs(scales.astype(np.float64)[np.where(inside, ids, 0)]), 0.0)


def attention_shared(k_pool, v_pool, page_tokens, prefix_pages, prefix_lengths, pages, lengths, q, scale, counts=None,
                     rounding=0.0, tiny=0.0, weight=2.0 ** -16, own_weight=None, floor=2.0 ** -32, least=0.0):
    """(out, error): float64 results and how far a computation in 32 bits may
    be off, derived as in kv_oracle.attention: a score is a sum of d products,
    each rounding at most 2^-23 of the sum of magnitudes; weights enter the
    second product rounded by `weight` at most, half a step of their type
    (2^-11 for 16-bit numbers of 11 bits); sums over n tokens add n roundings.
    Numbers of 11 bits have their smallest step, 2^-24, where the row's largest
    product of weight and scale of values is at least 2^7: each product of a
    weight and a code of values may be off by half of that (`floor`; 0 where
    no such numbers are used).
    own_weight: `weight` of the rows' own tokens, where it is another than the
    prefix's.  least: one of those may be off by that much of
    the row's largest.
    Exponentials below 2^-126, the smallest normal number of 32 bits, may come
    out as 0.  They are taken relative to a statistic that no score of the row
    exceeds by more than 2^8 once the sums are divided by their total, so that
    each costs at most 2^-118 of its value."""
    n_seqs, n_new, q_heads, d = q.shape
    heads, max_pages = pages.shape[1:]
    group = q_heads // heads
    kp, vp = kv.k_place(page_tokens, d), kv.v_place(page_tokens, d)
    out, err = np.zeros(q.shape), np.full(q.shape, float(tiny))
    u = 2.0 ** -23
    for h in range(heads):
        m = kv.row_length(prefix_lengths[h], prefix_pages.shape[1], page_tokens)
        first_k, first_on = kv.read_rows(*k_pool, kp, page_tokens, prefix_pages[h], m)
        first_v, _ = kv.read_rows(*v_pool, vp, page_tokens, prefix_pages[h], m)
        first_s = scales_of(v_pool[1], page_tokens, prefix_pages[h], m)
        first_w = np.full(m, weight)
        for s in range(n_seqs):
            n = kv.row_length(lengths[s, h], max_pages, page_tokens)
            origin, count = kv.new_tokens(n, counts, s, n_new)
            own_k, own_on = kv.read_rows(*k_pool, kp, page_tokens, pages[s, h], n)
            own_v, _ = kv.read_rows(*v_pool, vp, page_tokens, pages[s, h], n)
            own_s = scales_of(v_pool[1], page_tokens, pages[s, h], n)
            own_w = np.full(n, weight if own_weight is None else own_weight)
            for i in range(max(0, -origin), count):
                see = np.concatenate([first_on, own_on & (np.arange(n) <= origin + i)])
                if not see.any():
                    continue
                kk, vv = np.concatenate([first_k, own_k])[see], np.concatenate([first_v, own_v])[see]
                unit, half_step = np.concatenate([first_s, own_s])[see], np.concatenate([first_w, own_w])[see]
                for g in range(group):
                    x = q[s, i, h * group + g]
                    with np.errstate(invalid="ignore", over="ignore"):
                        sc = scale * (kk @ x)
                        top = np.max(sc)
                        if top == -np.inf:
                            continue
                        p = np.exp(sc - top)
                        p /= p.sum()
                        o = p @ vv
                        e = abs(scale) * (np.abs(kk) @ np.abs(x)) * (d + 4) * u + (np.abs(sc) + abs(top)) * 4 * u
                        common = float(np.sum(p * e)) + len(kk) * u + half_step
                        out[s, i, h * group + g] = o
                        err[s, i, h * group + g] += 2.0 ** -118 * np.abs(vv).sum(0)
                        err[s, i, h * group + g] += least * p.max() * np.abs(vv[:int(first_on.sum())]).sum(0)
                        with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
                            codes = np.where(unit[:, None] != 0, np.abs(vv) / unit[:, None], 0.0)
                            err[s, i, h * group + g] += floor * np.max(p * unit) * codes.sum(0)
                        err[s, i, h * group + g] += rounding * np.abs(o) + (1 + rounding) * ((p * (e + common)) @ np.abs(vv))
    return out, err

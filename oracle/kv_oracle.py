"""Plain 64-bit oracle of the 8-bit KV page cache (include/ibp_kv.h): numpy,
token by token, no code shared with the library."""
import numpy as np

E_MIN, E_MAX = -126, 119
E4M3_MAX = 448.0


def number_table():
    """The 256 numbers that e4m3 codes stand for."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if e == 15 and m == 7 else (-x if c & 0x80 else x)
    return out


NUMBERS = number_table()
_POSITIVE = NUMBERS[:127]  # 0 .. 448, ascending


def nearest_code(x):
    """Codes of the numbers nearest to x, ties to the even code, at most 448
    in magnitude; 0x7F for what is not finite."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.where(np.isfinite(x), np.abs(x), 0.0), E4M3_MAX)
    hi = np.minimum(np.searchsorted(_POSITIVE, a, side="left"), 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = _POSITIVE[hi] - a, a - _POSITIVE[lo]
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def k_place(page_tokens, d):
    """Byte of (token, dim) in a key page."""
    t, x = np.meshgrid(np.arange(page_tokens), np.arange(d), indexing="ij")
    return (t // 16) * 16 * d + (x // 64) * 1024 + (x % 64 // 16) * 256 + (t % 16) * 16 + x % 16


def v_place(page_tokens, d):
    """Byte of (token, dim) in a value page."""
    t, x = np.meshgrid(np.arange(page_tokens), np.arange(d), indexing="ij")
    return (t // 16) * 16 * d + (x // 64) * 1024 + (t % 16 // 4) * 256 + (x % 16) * 16 + \
        (x % 64 // 16) * 4 + t % 4


def exponent(amax):
    """Smallest e in [-126, 119] with amax <= 448 * 2^e."""
    e = E_MIN
    while e < E_MAX and amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return e


def row_length(length, max_pages, page_tokens):
    return min(max(int(length), 0), max_pages * page_tokens)


def new_tokens(length, counts, s, n_new):
    """(position of token 0, count) of sequence s's new tokens."""
    c = n_new if counts is None else min(max(int(counts[s]), 0), n_new)
    return length - c, c


def append(codes, scales, place, page_tokens, pages, lengths, x, counts=None):
    """Append x [n_seqs, n_new, heads, d] (float64) in place to the pool
    (codes uint8 [n_pages, bytes], scales float32)."""
    n_seqs, heads, max_pages = pages.shape
    n_new = x.shape[1]
    for s in range(n_seqs):
        for h in range(heads):
            n = row_length(lengths[s, h], max_pages, page_tokens)
            origin, count = new_tokens(n, counts, s, n_new)
            first = max(origin, 0)
            if count == 0 or n == 0:
                continue
            for p in range(first // page_tokens, -(-n // page_tokens)):
                page = int(pages[s, h, p])
                if not 0 <= page < len(scales):
                    continue
                lo, hi = max(first, p * page_tokens), min(n, (p + 1) * page_tokens)
                new = x[s, lo - origin:hi - origin, h]
                e = exponent(np.max(np.abs(new[np.isfinite(new)]), initial=0.0))
                old = max(0, first - p * page_tokens)
                was = codes[page][place[:old]]
                if old:
                    was_scale = float(scales[page])
                    while e < E_MAX and was_scale > 2.0 ** e:
                        e += 1
                    if was_scale != 2.0 ** e:
                        was = nearest_code(NUMBERS[was] * was_scale / 2.0 ** e)
                full = np.zeros((page_tokens, x.shape[3]), np.uint8)
                full[:old] = was
                full[lo - p * page_tokens:hi - p * page_tokens] = \
                    np.where(np.isfinite(new), nearest_code(new / 2.0 ** e), 0x7F)
                codes[page, place.reshape(-1)] = full.reshape(-1)
                scales[page] = 2.0 ** e


def read_rows(codes, scales, place, page_tokens, pages_row, n):
    """The first n tokens of a row (float64 [n, d]) and which are no holes."""
    d = place.shape[1]
    out, there = np.zeros((n, d)), np.zeros(n, bool)
    for p in range(-(-n // page_tokens)):
        page, hi = int(pages_row[p]), min(n, (p + 1) * page_tokens)
        if 0 <= page < len(scales):
            out[p * page_tokens:hi] = NUMBERS[codes[page][place[:hi - p * page_tokens]]] * float(scales[page])
            there[p * page_tokens:hi] = True
    return out, there


def attention(k_pool, v_pool, page_tokens, pages, lengths, q, scale, weights=None, counts=None,
              rounding=0.0, tiny=0.0):
    """(out, weights_out, out_error, weights_error): float64 results, and how
    far a computation in 32 bits may be off.

    The errors: a score is a sum of d products in 32 bits, each rounding (of
    either kind) at most 2^-23 of the sum of magnitudes; taken to an
    exponent that is a relative error of the weight.  The weights enter the
    second product with 16 bits, and sums over n tokens add n more roundings.
    `rounding` is half a step of the output's type, `tiny` half its smallest.
    """
    n_seqs, n_new, q_heads, d = q.shape
    heads, max_pages = pages.shape[1:]
    group = q_heads // heads
    kp, vp = k_place(page_tokens, d), v_place(page_tokens, d)
    out, out_err = np.zeros(q.shape), np.full(q.shape, tiny)
    w_out = None if weights is None else weights.astype(np.float64).copy()
    w_err = None if weights is None else np.abs(w_out) * 2.0 ** -22
    u = 2.0 ** -23
    for s in range(n_seqs):
        for h in range(heads):
            n = row_length(lengths[s, h], max_pages, page_tokens)
            origin, count = new_tokens(n, counts, s, n_new)
            key, there = read_rows(*k_pool, kp, page_tokens, pages[s, h], n)
            value, _ = read_rows(*v_pool, vp, page_tokens, pages[s, h], n)
            for i in range(count):
                seen = origin + i + 1
                if seen <= 0 or not there[:seen].any():
                    continue
                on = np.flatnonzero(there[:seen])
                kk, vv = key[on], value[on]
                for g in range(group):
                    x = q[s, i, h * group + g]
                    with np.errstate(invalid="ignore", over="ignore"):
                        sc = scale * (kk @ x)
                        top = np.max(sc)
                        if top == -np.inf:
                            continue
                        p = np.exp(sc - top)
                        p /= p.sum()
                        out[s, i, h * group + g] = o = p @ vv
                        # relative errors of the weights
                        e = abs(scale) * (np.abs(kk) @ np.abs(x)) * (d + 4) * u + (np.abs(sc) + abs(top)) * 4 * u
                        common = float(np.sum(p * e)) + len(on) * u + 2.0 ** -16
                        out_err[s, i, h * group + g] += rounding * np.abs(o) + (1 + rounding) * ((p * (e + common)) @ np.abs(vv))
                        if w_out is not None:
                            # a page's share is kept as the logarithm of its sum
                            lse = abs(top) * 1.4427 + np.log2(len(on)) + 1
                            for pg in np.unique(on // page_tokens):
                                at = on // page_tokens == pg
                                m = float(p[at].sum())
                                lg = lse + abs(np.log2(m)) if m > 0 else 0.0
                                w_out[s, h, pg] += m
                                w_err[s, h, pg] += float((p[at] * (e[at] + common)).sum()) + m * lg * 4 * u
    if w_out is not None:
        w_err += np.abs(w_out) * u * (n_new * group + 4) + 1e-30
    return out, w_out, out_err, w_err


def evict(pages, weights, lengths, page_tokens, keep, sink, recent):
    pages, weights, lengths = pages.copy(), weights.copy(), lengths.copy()
    n_seqs, heads, max_pages = pages.shape
    for s in range(n_seqs):
        for h in range(heads):
            n = row_length(lengths[s, h], max_pages, page_tokens)
            lengths[s, h] = n
            held = -(-n // page_tokens)
            if held <= keep:
                continue
            w = weights[s, h]

            def rank(i):  # heavier first, then the lower position
                return (0, 0.0, i) if np.isnan(w[i]) else (1, -float(w[i]), i)
            middle = sorted(range(sink, held - recent), key=rank)[:keep - sink - recent]
            stay = sorted(list(range(sink)) + middle + list(range(held - recent, held)))
            go = sorted(set(range(held)) - set(stay))
            pages[s, h, :held] = pages[s, h][stay + go]
            weights[s, h, :held] = np.concatenate([w[stay], np.zeros(len(go), np.float32)])
            lengths[s, h] = n - len(go) * page_tokens
    return pages, weights, lengths

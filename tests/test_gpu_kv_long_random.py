"""Seeded random calls of long and shared contexts over the KV pages against the
oracle: sizes, types, lengths, counts, holes, positions and scales of every kind
together, a few steps over one cache as a server makes them."""
import numpy as np
import pytest

from test_gpu_kv import DTYPES, Pages, grid, kv, np_of, values  # noqa: F401
from test_gpu_kv_long import Outlines, append_rotated, check_select, check_shared, gpu, shared_pool, tables
from test_gpu_kv_paths import noise, queries

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def sizes(rng):
    return (int(rng.integers(1, 6)), int(rng.integers(1, 4)), int(rng.choice([1, 2, 3, 5, 8])), int(rng.choice([16, 32, 64])),
            int(rng.choice([64, 128, 192, 256])), ("bf16", "fp16")[int(rng.integers(2))])


def table_values(rng, shape, low, high):
    """Whole numbers, a few of them outside what a table may hold."""
    x = rng.integers(low, high + 1, shape)
    return np.where(rng.random(shape) < 0.1, rng.choice([-3, 0, high + 5, 10 ** 6], shape), x).astype(np.int32)


@pytest.mark.parametrize("seed", range(24))
def test_steps_over_one_cache(kv, seed):
    """Prompts, chunks and tokens appended with rotations and outlines; after each a
    selection from what is there."""
    rng = np.random.default_rng(seed)
    seqs, heads, group, pt, d, dtype = sizes(rng)
    m = int(rng.integers(2, 8))
    p = Pages(kv, seqs, heads, m, pt, d, seed=seed)
    p.pages[rng.random(p.pages.shape) < 0.08] = rng.choice([-1, p.n_pages, 2 ** 31 - 1])
    p.upload()
    o = Outlines(p, seed)
    rotary = int(rng.choice(np.arange(16, d + 1, 16)))
    interleaved = bool(rng.integers(2))
    cos, sin = tables(m * pt + 50, rotary // 2)
    lens = np.zeros(seqs, np.int64)
    for step in range(4):
        new = int(rng.choice([1, 1, 2, int(rng.integers(1, m * pt + 4))]))
        counts = None if rng.random() < 0.4 else rng.integers(-1, new + 2, seqs)
        lens = np.minimum(lens + (new if counts is None else np.clip(counts, 0, new)), m * pt + 3)
        lengths = grid(seqs, heads, lens)
        if rng.random() < 0.3:
            lengths = table_values(rng, lengths.shape, 0, m * pt)
        positions = None if rng.random() < 0.5 else table_values(rng, (seqs, new), 0, m * pt + 49)
        amp = float(2.0 ** rng.integers(-12, 12))
        x, y, q = (values(100 * seed + 10 * step + i, (seqs, new, h, d), DTYPES[dtype], amp) for i, h in ((1, heads), (2, heads), (3, heads * group)))
        append_rotated(kv, p, lengths, x, y, cos, sin, positions=positions, q=q if rng.random() < 0.8 else None, counts=counts,
                       interleaved=interleaved, outlines=o if rng.random() < 0.7 else None)
        p.check()
        some = None if rng.random() < 0.5 else int(rng.integers(0, m * pt + 2))
        if some != 0:
            o.expect(p, lengths, m * pt if some is None else some)
            kv.ibp_kv_outline(p.cache, o.t, p.gpu_pages, gpu(lengths), n_new=some)
        o.check()
        recent = (new + pt - 2) // pt + 1 + int(rng.integers(0, 2))
        keep = recent + int(rng.integers(0, m))
        if np.isfinite(q.double().numpy()).all():
            check_select(kv, p, o, lengths, q, keep, int(rng.integers(0, keep - recent + 1)), recent, counts=counts)


@pytest.mark.parametrize("seed", range(24))
def test_selections(kv, seed):
    """Rows of up to some thousand pages, with many equal scores."""
    rng = np.random.default_rng(100 + seed)
    seqs, heads, group, pt, d, dtype = sizes(rng)
    m = int(np.exp(rng.uniform(0, np.log(3000))))
    new = int(rng.choice([1, 1, 2, 7]))
    p = noise(kv, seqs, heads, m, pt, d, seed=seed, n_pages=int(rng.choice([7, 400])))
    p.pages[rng.random(p.pages.shape) < 0.05] = -1
    p.upload()
    o = Outlines(p, seed)
    o.codes[:] = np.sort(o.codes, 1)[:, ::-1]
    o.scales[:] = rng.choice(np.array([1, 1, 0.5, 2.0 ** -20, 0, np.nan], np.float32), p.n_pages, p=[.4, .2, .2, .1, .05, .05])
    o.t = (gpu(o.codes), gpu(o.scales))
    recent = (new + pt - 2) // pt + 1 + int(rng.integers(0, 3))
    keep = recent + int(rng.integers(0, m + 2))
    q = queries(seed, seqs, new, heads * group, d, dtype)
    check_select(kv, p, o, table_values(rng, (seqs, heads), 0, m * pt), q, keep, int(rng.integers(0, keep - recent + 1)), recent,
                 counts=None if rng.random() < 0.5 else rng.integers(0, new + 1, seqs))


@pytest.mark.parametrize("seed", range(40))
def test_shared_prefixes(kv, seed):
    """1 to some hundred query rows to a head; prefixes and own rows of any length."""
    rng = np.random.default_rng(200 + seed)
    seqs, heads, group, pt, d, dtype = sizes(rng)
    if rng.random() < 0.4:
        seqs, heads = int(rng.integers(6, 40)), int(rng.integers(1, 3))
    new = int(rng.choice([1, 1, 2, 7]))
    prefix, own = int(np.exp(rng.uniform(0, np.log(120)))), int(rng.integers(1, 12))
    p = shared_pool(kv, seqs, heads, prefix, own, pt, d, seed=seed)
    for table in (p.prefix, p.pages):
        table[rng.random(table.shape) < 0.08] = rng.choice([-1, p.n_pages])
    kind = rng.integers(3)
    if kind:
        p.v[1] *= rng.choice(np.array([1, 2.0 ** -10, 0.7, 0, -1] if kind == 1 else [1, 2.0 ** -5], np.float32), p.n_pages)
    p.upload()
    check_shared(kv, p, table_values(rng, heads, 0, prefix * pt), table_values(rng, (seqs, heads), 0, own * pt),
                 queries(seed, seqs, new, heads * group, d, dtype), scale=float(rng.choice([0.02, -0.03, 0.1])),
                 counts=None if rng.random() < 0.6 else rng.integers(-1, new + 2, seqs))

"""The 8-bit KV page cache on the GPU, path by path: rows cut into parts and
joined, by workgroups and by waves, at every head size and number of query
rows; rows that keep their shares of the softmax in LDS and in the workspace;
each eviction kernel about the row lengths it begins and ends at; appends of
every 16-bit value.  Which path a case takes is read off the workspace it asks
for, so that a changed rule fails here instead of leaving a path out.
Tolerances are those of oracle/kv_oracle.py."""
import numpy as np
import pytest

from oracle import kv_oracle as orc
from test_gpu_kv import DTYPES, Pages, close, expect, grid, kv, np_of, run_attention, run_evict, same_eviction  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def noise(kv, seqs, heads, max_pages, pt, d, seed, n_pages=4096):
    """Pages of random finite codes with scales of their own; rows share them,
    since attention only reads."""
    p = Pages(kv, 1, 1, 1, pt, d, seed, n_pages=min(n_pages, seqs * heads * max_pages))
    rng = np.random.default_rng(seed)
    for codes, scales in (p.k, p.v):
        codes[:] = rng.integers(0, 0x50, codes.shape, dtype=np.uint8) | (rng.integers(0, 2, codes.shape, dtype=np.uint8) << 7)
        scales[:] = 2.0 ** rng.integers(-3, 2, scales.shape)
    p.pages = rng.integers(0, p.n_pages, (seqs, heads, max_pages)).astype(np.int32)
    p.upload()
    return p


def queries(seed, seqs, new, q_heads, d, dtype):
    return torch.randn(seqs, new, q_heads, d, generator=torch.Generator().manual_seed(seed)).to(DTYPES[dtype])


def parts_of(kv, p, group, new):
    """(units, parts) of a call without weights; no parts where no row is cut."""
    seqs, heads, _ = p.pages.shape
    m = group * new
    rows = min(m, 16 if m <= 16 else 32)
    units = seqs * heads * -(-m // (16 if m <= 16 else 32))
    lengths = torch.zeros(seqs, heads, dtype=torch.int32, device="cuda")
    n = kv.ibp_kv_attention_workspace_bytes(p.cache, p.gpu_pages, lengths, heads * group, new, False)
    return units, (n - 8 * units) // (rows * (4 * p.d + 8)) if n else 0


def step_tokens(d, m):
    """Tokens that a wave of the attention kernel takes at a time."""
    return 64 if d == 64 and m <= 16 else 32


# --------------------------------------------------- rows cut into parts ----


@pytest.mark.parametrize("join", ["waves", "workgroups"])
@pytest.mark.parametrize("group,new", [(1, 1), (16, 1), (17, 1), (5, 5), (8, 4), (11, 3), (16, 5)])
@pytest.mark.parametrize("d", [64, 128, 192, 256])
def test_cut_rows(kv, d, group, new, join):
    """Ragged rows, none and one token among them, in parts that a wave joins
    per query row (few parts) or a workgroup (many); 1 to 80 query rows, so one
    unit to a head or several."""
    pt, dtype = {64: 64, 128: 16, 192: 32, 256: 16}[d], "bf16" if new % 2 else "fp16"
    cap = step_tokens(d, group * new) * (20 if join == "waves" else 90)
    seqs, heads, m = 5, 2, cap // pt
    p = noise(kv, seqs, heads, m, pt, d, seed=d + group)
    units, parts = parts_of(kv, p, group, new)
    assert parts > units and (parts <= 8 * units) == (join == "waves")
    lens = [0, 1, new + 3, cap * 11 // 20 + 7, cap]
    lengths = grid(seqs, heads, lens)
    lengths[3, 1] = cap - 1
    q = queries(group, seqs, new, heads * group, d, dtype)
    w = np.random.default_rng(3).random((seqs, heads, m), dtype=np.float32)
    out, wo = run_attention(kv, p, lengths, q, w, scale=0.02)
    close(out, wo, expect(p, lengths, q, w, scale=0.02))
    alone, none = run_attention(kv, p, lengths, q, scale=0.02)
    assert none is None and torch.equal(alone, out)
    again, wo2 = run_attention(kv, p, lengths, q, w, scale=0.02)
    assert torch.equal(again, out) and np.array_equal(wo2, wo)


@pytest.mark.parametrize("d,group,new", [(64, 9, 3), (256, 5, 5), (192, 1, 1)])
def test_cut_one_row_into_many_parts(kv, d, group, new):
    """A row alone: more parts than a wave has lanes."""
    pt, n = 64, 30011
    p = noise(kv, 1, 1, 480, pt, d, seed=d)
    units, parts = parts_of(kv, p, group, new)
    assert units == 1 and parts > 64
    q = queries(1, 1, new, group, d, "fp16")
    w = np.zeros((1, 1, 480), np.float32)
    for length in (n, 20 * 64):
        out, wo = run_attention(kv, p, [[length]], q, w, scale=0.02)
        close(out, wo, expect(p, [[length]], q, w, scale=0.02))


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("group,new", [(3, 9), (16, 5), (2, 6)])
def test_cut_rows_holes_counts_and_nan(kv, d, group, new):
    """Holes at the front, inside and in whole rows; counts below n_new, none,
    more; lengths outside the table; NaN values that some of the queries see."""
    pt = 16
    cap = step_tokens(d, group * new) * 24
    seqs, heads, m = 7, 2, cap // pt
    p = noise(kv, seqs, heads, m, pt, d, seed=group, n_pages=1 << 20)
    p.pages = np.random.default_rng(5).permutation(seqs * heads * m).reshape(seqs, heads, m).astype(np.int32)
    lens = [cap, cap - 5, 3, cap // 2, 40, cap - 100, cap // 2 + 9]
    for pos, dim in ((lens[5] - 1, 3), (lens[5] - 3, 50), (lens[5] - 3, 16), (7, 33)):
        p.v[0][p.pages[5, 0, pos // pt], orc.v_place(pt, d)[pos % pt, dim]] = 0x7F
    # past the row's end, where nothing sees it
    p.v[0][p.pages[6, :, -(-lens[6] // pt):]] = 0xFF
    p.k[0][p.pages[6, :, -(-lens[6] // pt):]] = 0xFF
    p.pages[0, 0, :5], p.pages[0, 1, 7:60], p.pages[1], p.pages[3, 0, m // 4] = -1, p.n_pages, -1, 2 ** 31 - 1
    p.upload()
    units, parts = parts_of(kv, p, group, new)
    assert parts > units
    lengths = grid(seqs, heads, [*lens[:3], lens[3], -4, *lens[5:]])
    lengths[0, 1] = cap + 5000
    q = queries(2, seqs, new, heads * group, d, "bf16")
    w = np.random.default_rng(1).random((seqs, heads, m), dtype=np.float32)
    for counts in (None, [new, new, new, 2, new, new, 0], [1, 99, new - 1, 0, -1, 2, new]):
        out, wo = run_attention(kv, p, lengths, q, w, scale=0.02, counts=counts)
        close(out, wo, expect(p, lengths, q, w, scale=0.02, counts=counts))
        assert not out[1].any() and np.array_equal(wo[1], w[1]) and np.array_equal(wo[4], w[4])
        assert np.isnan(out[5].float().numpy()).any()


@pytest.mark.parametrize("table", [512, 1600])
def test_chunk_of_a_prompt(kv, table):
    """1200 query rows a head, 38 units: uncut, and cut."""
    seqs, heads, group, new, d, pt = 2, 1, 4, 300, 64, 16
    p = noise(kv, seqs, heads, table // pt, pt, d, seed=4)
    units, parts = parts_of(kv, p, group, new)
    assert units == 76 and (parts == 0 if table == 512 else parts > units)
    lengths = np.array([[table - 9], [new + 17]], np.int32)
    q = queries(3, seqs, new, heads * group, d, "bf16")
    w = np.zeros(p.pages.shape, np.float32)
    out, wo = run_attention(kv, p, lengths, q, w, scale=0.05)
    close(out, wo, expect(p, lengths, q, w, scale=0.05))


@pytest.mark.parametrize("group,new,d,m,where", [(16, 1, 64, 70, "workspace"), (16, 1, 64, 60, "lds"), (8, 4, 128, 40, "workspace"),
                                                 (8, 4, 128, 30, "lds"), (1, 1, 256, 1100, "workspace")])
def test_uncut_rows_with_shares(kv, group, new, d, m, where):
    """More rows than the chip holds workgroups, one workgroup each, over tables
    whose shares fit LDS, or not."""
    seqs, heads, pt = 50, 8, 64
    p = noise(kv, seqs, heads, m, pt, d, seed=d)
    assert parts_of(kv, p, group, new)[1] == 0
    gl = torch.zeros(seqs, heads, dtype=torch.int32, device="cuda")
    n = kv.ibp_kv_attention_workspace_bytes(p.cache, p.gpu_pages, gl, heads * group, new, True)
    assert n == (0 if where == "lds" else seqs * heads * group * new * m * pt // 16 * 4)
    lens = [(17 * i) % 101 for i in range(seqs)]
    lens[3] = min(m * pt, 4100)
    q = queries(5, seqs, new, heads * group, d, "bf16")
    w = np.random.default_rng(2).random((seqs, heads, m), dtype=np.float32)
    lengths = grid(seqs, heads, lens)
    out, wo = run_attention(kv, p, lengths, q, w, scale=0.02)
    close(out, wo, expect(p, lengths, q, w, scale=0.02))


# ------------------------------------------------------------ eviction ----


@pytest.mark.parametrize("m", [1024, 1025, 4096, 4097, 5000, 16383, 16384, 16385])
def test_evict_at_the_kernels_edges(kv, m):
    """Rows about the lengths at which one kernel takes over from another:
    distinct weights, equal ones, many ties, neighbours by one step of the type
    (which takes the most rounds to tell apart); every budget from the least."""
    rng = np.random.default_rng(m)
    seqs, heads, pt = 5, 2, 32
    pages = rng.permutation(seqs * heads * m).reshape(seqs, heads, m).astype(np.int32)
    weights = np.empty(pages.shape, np.float32)
    weights[0] = np.exp(3 * rng.standard_normal((heads, m)))
    weights[1] = 0.75
    weights[2] = rng.integers(0, 3, (heads, m))
    near = np.float32(1.0).view(np.int32) + rng.permutation(m).astype(np.int32)
    weights[3, 0] = near.view(np.float32)
    weights[3, 1] = -(near // 3 * 3).view(np.float32)
    weights[3, :, 5], weights[3, :, 9] = 3e38, -3e38
    weights[4] = rng.choice(np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, 2.0], np.float32), (heads, m))
    full = np.full((seqs, heads), m * pt, np.int32)
    ragged = rng.integers(0, m * pt + 1, (seqs, heads)).astype(np.int32)
    ragged[0], ragged[1, 0], ragged[1, 1], ragged[2, 0] = [m * pt - 3, m * pt + 900], 0, -8, 1
    for keep, sink, recent in ((4, 1, 3), (m // 3, 2, 5), (m // 2, 0, 1), (m - 1, 3, 1), (m, 1, 1)):
        for lengths in (full, ragged):
            same_eviction(run_evict(kv, pages, weights, lengths, pt, keep, sink, recent),
                          orc.evict(pages, weights, lengths, pt, keep, sink, recent))


# -------------------------------------------------------------- append ----


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_every_16_bit_value(kv, dtype):
    """All 65,536 values: as they follow each other, so that a page's are alike;
    spread, so that a page has every size; and cut to the range of scales from
    the lowest to the highest."""
    d, pt, n = 64, 16, 1024
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(DTYPES[dtype])
    assert int(x.view(torch.int16).int().bitwise_and(0xFFFF).unique().numel()) == 1 << 16
    rows = [x, x.reshape(64, 1024).T.reshape(-1)]
    top = float(torch.finfo(x.dtype).max)
    for e in (-126, -125, -124, -110, -40, -30, -24, -20, -17, -16, -8, 0, 3, 7, 8, 60, 118, 119):
        if 448 * 2.0 ** e <= top:
            y = x.double().clamp(-448 * 2.0 ** e, 448 * 2.0 ** e)
            rows += [y.to(x.dtype), (y * 0.9).to(x.dtype).reshape(64, 1024).T.reshape(-1)]
    x = torch.stack(rows).reshape(len(rows), n, 1, d).contiguous()
    p = Pages(kv, len(rows), 1, n // pt, pt, d)
    p.append(grid(len(rows), 1, [n] * len(rows)), x, x.flip(1))
    p.check()


@pytest.mark.parametrize("pt", [16, 32])
def test_append_brings_every_code_to_a_larger_scale(kv, pt):
    """A page's old codes, all 256, under scales 2^0 .. 2^23 times theirs, and
    from scales that are no powers of two."""
    d, seqs = 64, 26
    p = Pages(kv, seqs, 1, 1, pt, d)
    for pool in (p.k, p.v):
        pool[0][:] = np.arange(pt * d) % 256
        pool[1][:] = 2.0 ** -4
    p.k[1][p.pages[24:, 0, 0]], p.v[1][p.pages[24:, 0, 0]] = [0.75, 3.0], [1.25, 1e-30]
    p.upload()
    x = torch.zeros(seqs, 1, 1, d)
    x[:, 0, 0, 3] = 448.0 * 2.0 ** (torch.arange(seqs).clamp(max=23) - 4)
    p.append(grid(seqs, 1, [pt] * seqs), x.bfloat16(), -x.bfloat16())
    p.check()

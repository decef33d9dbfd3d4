"""Long and shared contexts over the 8-bit KV pages on the GPU: appends with
rotated positions, outlines and selections exactly as the oracle has them,
attention over a shared prefix within bounds derived from 32-bit arithmetic
(oracle/kv_long_oracle.py)."""
import numpy as np
import pytest

from oracle import kv_long_oracle as lorc
from oracle import kv_oracle as orc
from test_gpu_kv import DTYPES, Pages, close, expect, filled, grid, kv, np_of, run_attention, values  # noqa: F401
from test_gpu_kv_paths import noise, queries

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def tables(n, half, seed=0):
    """cos and sin of n positions, as float32 arrays."""
    angle = np.arange(n)[:, None] * 10000.0 ** (-np.arange(half) / max(half, 1))
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


def gpu(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Outlines:
    """Outlines of a Pages' pool, noise at first, on the GPU and as the oracle has them."""

    def __init__(self, p, seed=0):
        rng = np.random.default_rng(seed)
        self.codes = rng.integers(-128, 128, (p.n_pages, 2, p.d)).astype(np.int8)
        self.scales = rng.random(p.n_pages, dtype=np.float32)
        self.t = (gpu(self.codes), gpu(self.scales))

    def expect(self, p, lengths, n_new, counts=None):
        lorc.outline(*p.k, orc.k_place(p.pt, p.d), p.pt, p.pages, np.asarray(lengths), self.codes, self.scales, n_new, counts)

    def check(self):
        torch.cuda.synchronize()
        for name, got, want in zip(("codes", "scales"), self.t, (self.codes, self.scales)):
            got = np_of(got)
            same = (got == want) | (np.isnan(want) & np.isnan(got) if name == "scales" else False)
            bad = np.argwhere(~same)
            assert len(bad) == 0, (name, len(bad), bad[:4], got[tuple(bad[0])], want[tuple(bad[0])])


def append_rotated(kv, p, lengths, k, v, cos, sin, positions=None, q=None, counts=None, interleaved=False, outlines=None,
                   gpu_k=None, gpu_v=None, gpu_q=None, q_out=None):
    """On the GPU and in the oracle; queries are compared at once, pages by p.check()."""
    lengths = np.asarray(lengths, np.int32)
    c = None if counts is None else np.asarray(counts, np.int32)
    m = p.pages.shape[2]
    turned = lorc.rotated(k.double().numpy(), cos, sin, lengths, m, p.pt, positions, c, interleaved)
    for (codes, scales), x, place in ((p.k, turned, orc.k_place), (p.v, v.double().numpy(), orc.v_place)):
        orc.append(codes, scales, place(p.pt, p.d), p.pt, p.pages, lengths, x.astype(np.float64), c)
    if outlines is not None:
        outlines.expect(p, lengths, k.shape[1], c)
    q_gpu = None if q is None else q.cuda() if gpu_q is None else gpu_q
    out = kv.ibp_kv_append_rotated(p.cache, p.gpu_pages, gpu(lengths), k.cuda() if gpu_k is None else gpu_k,
                                   v.cuda() if gpu_v is None else gpu_v, gpu(cos), gpu(sin), positions=gpu(positions), q=q_gpu,
                                   q_out=q_out, counts=gpu(c), interleaved=interleaved,
                                   outlines=None if outlines is None else outlines.t)
    torch.cuda.synchronize()
    if q is None:
        assert out is None
    else:
        want = torch.from_numpy(lorc.rotated(q.double().numpy(), cos, sin, lengths, m, p.pt, positions, c, interleaved)).to(q.dtype)
        got = out.cpu()
        nan = want.isnan()
        assert torch.equal(got.isnan(), nan)
        assert torch.equal(got.masked_fill(nan, 0), want.masked_fill(nan, 0))
    return out


# ------------------------------------------------------ rotated appends ----


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rotary", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 96), (192, 192), (192, 64),
                                      (192, 128), (256, 256), (256, 128), (256, 32)])
@pytest.mark.parametrize("pt", [16, 32, 64])
def test_append_rotated(kv, pt, d, rotary, interleaved):
    """Ragged prompts, then chunks and tokens, queries with them: every head
    size, whole and part rotations, both orders of pairs; codes, scales and
    outlines byte for byte."""
    seqs, heads, group = 3, 2, 3
    dtype = DTYPES["bf16" if (d + rotary + pt) // 16 % 2 else "fp16"]
    p = Pages(kv, seqs, heads, 4, pt, d, seed=pt + d)
    o = Outlines(p)
    cos, sin = tables(4 * pt, rotary // 2)
    lens = np.array([1, pt - 1, 2 * pt + 3])
    n = int(lens.max())
    append_rotated(kv, p, grid(seqs, heads, lens), values(1, (seqs, n, heads, d), dtype), values(2, (seqs, n, heads, d), dtype),
                   cos, sin, q=values(3, (seqs, n, heads * group, d), dtype), counts=lens, interleaved=interleaved, outlines=o)
    p.check()
    o.check()
    for i, (new, amp) in enumerate([(1, 1.0), (5, 4.0), (1, 100.0), (pt // 2, 0.5)]):
        lens = lens + new
        append_rotated(kv, p, grid(seqs, heads, lens), values(10 + i, (seqs, new, heads, d), dtype, amp),
                       values(30 + i, (seqs, new, heads, d), dtype, amp), cos, sin,
                       q=values(50 + i, (seqs, new, heads * group, d), dtype), interleaved=interleaved, outlines=o if i % 2 else None)
        p.check()
        if i % 2:
            o.check()
        else:   # the outlines are brought up to date apart
            o.expect(p, grid(seqs, heads, lens), new)
            kv.ibp_kv_outline(p.cache, o.t, p.gpu_pages, gpu(grid(seqs, heads, lens)), n_new=new)
            o.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_rotated_positions_holes_and_lengths_outside(kv, dtype):
    """Positions given, outside the tables and below 0 among them; holes, counts
    and lengths outside; heads of a sequence that differ; no queries' rows but
    those of tokens that exist."""
    seqs, heads, d, pt, m, new = 7, 2, 128, 16, 3, 40
    p = Pages(kv, seqs, heads, m, pt, d)
    p.pages[0, 0, 1], p.pages[0, 1, 0], p.pages[1, 1, 2] = -1, p.n_pages, 2 ** 31 - 1
    p.upload()
    o = Outlines(p)
    cos, sin = tables(60, 64)
    x, y, q = (values(i, (seqs, new, h, d), DTYPES[dtype]) for i, h in ((1, heads), (2, heads), (3, 3 * heads)))
    lens = grid(seqs, heads, [48, 45, 0, -7, 100, 30, 41])
    lens[5, 1] = 3
    rng = np.random.default_rng(1)
    positions = rng.integers(0, 60, (seqs, new)).astype(np.int32)
    positions[0, 3], positions[0, 30], positions[4, 39], positions[6, 0] = -1, 60, 2 ** 31 - 1, -2 ** 31
    for at in (None, positions):
        for counts in ([40, 99, 5, 5, 21, 40, 40], [0, -3, 0, 0, 0, 0, 1], None):
            append_rotated(kv, p, lens, x, y, cos, sin, positions=at, q=q, counts=counts, outlines=o)
            p.check()
            o.check()
    append_rotated(kv, p, lens, x[:, :0], y[:, :0], cos, sin, q=q[:, :0], outlines=o)
    append_rotated(kv, p, lens, x, y, cos[:0], sin[:0], q=q, outlines=o)      # tables without positions
    p.check()
    o.check()


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_rotated_values_not_finite(kv, interleaved):
    """Infinities and NaN become NaN with their pairs and do not count for the
    scale; extremes of the type; zeros; tables that are no rotation."""
    d, pt, n = 64, 16, 48
    for dtype in (torch.bfloat16, torch.float16):
        x = values(1, (2, n, 1, d), dtype)
        x[0, 5, 0, 3], x[0, 20, 0, 40], x[0, 21, 0, 63] = float("inf"), float("nan"), float("-inf")
        x[1, :16] = 0.0
        x[1, 16:32] = torch.finfo(dtype).max
        x[1, 32:] = torch.finfo(dtype).smallest_normal / 4
        p, (cos, sin) = Pages(kv, 2, 1, 3, pt, d), tables(n, 16)
        o = Outlines(p)
        append_rotated(kv, p, grid(2, 1, [n, n]), x, x, cos, sin, q=x, interleaved=interleaved, outlines=o)
        p.check()
        o.check()
        rng = np.random.default_rng(0)
        cos, sin = (rng.choice(np.array([0.0, -0.0, 1.0, 1e-30, 3e38, np.inf, np.nan, -2.5], np.float32), cos.shape) for _ in range(2))
        append_rotated(kv, p, grid(2, 1, [n, n]), x, x, cos, sin, q=x, interleaved=interleaved, outlines=o)
        p.check()
        o.check()


@pytest.mark.parametrize("how", ["transposed", "offset", "broadcast", "in place", "given"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_rotated_strides(kv, how, interleaved):
    seqs, new, heads, group, d, pt = 2, 19, 3, 2, 128, 16
    x, y = values(1, (seqs, new, heads, d), torch.bfloat16), values(2, (seqs, new, heads, d), torch.bfloat16)
    q = values(3, (seqs, new, heads * group, d), torch.bfloat16)
    p, (cos, sin) = Pages(kv, seqs, heads, 3, pt, d), tables(60, 24)
    gx, gy, gq, out = x.cuda(), y.cuda(), q.cuda(), None
    if how == "transposed":
        gx, gy, gq = (t.transpose(1, 2).contiguous().cuda().transpose(1, 2) for t in (x, y, q))
    elif how == "offset":
        gx, gy, gq = (torch.empty(*t.shape[:3], d + 3, dtype=t.dtype, device="cuda")[..., 1:d + 1].copy_(t) for t in (x, y, q))
    elif how == "broadcast":
        x, y, q = x[:, :, :1].expand(-1, -1, heads, -1), y[:, :1].expand(-1, new, -1, -1), q[:, :, :1].expand(-1, -1, heads * group, -1)
        gx, gy = x[:, :, :1].contiguous().cuda().expand(-1, -1, heads, -1), y[:, :1].contiguous().cuda().expand(-1, new, -1, -1)
        gq = q[:, :, :1].contiguous().cuda().expand(-1, -1, heads * group, -1)
        assert gq.stride(2) == 0
    elif how == "in place":
        out = gq
    else:
        out = torch.full((seqs, heads * group, new, d + 5), 7.0, dtype=torch.bfloat16, device="cuda")[..., 3:3 + d].transpose(1, 2)
    got = append_rotated(kv, p, grid(seqs, heads, [new + 7, new]), x.contiguous(), y.contiguous(), cos, sin, q=q.contiguous(),
                         interleaved=interleaved, gpu_k=gx, gpu_v=gy, gpu_q=gq, q_out=out)
    p.check()
    assert out is None or got is out
    if how == "given":
        assert (out._base[..., :3] == 7).all() and (out._base[..., 3 + d:] == 7).all()


def test_append_rotated_like_append_of_rotated_numbers(kv):
    """With the identity as rotation the bytes are those of a plain append."""
    seqs, heads, d, pt = 2, 2, 128, 16
    x, y = values(1, (seqs, 50, heads, d), torch.float16), values(2, (seqs, 50, heads, d), torch.float16)
    a, b = Pages(kv, seqs, heads, 4, pt, d), Pages(kv, seqs, heads, 4, pt, d)
    a.append(grid(seqs, heads, [50, 50]), x, y)
    append_rotated(kv, b, grid(seqs, heads, [50, 50]), x, y, np.ones((64, 64), np.float32), np.zeros((64, 64), np.float32))
    torch.cuda.synchronize()
    for s, t in zip(a.t, b.t):
        assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))


# ------------------------------------------------------------- outlines ----


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("pt", [16, 32, 64])
def test_outline(kv, pt, d):
    """Pages of noise codes, NaN among them; every number of tokens in a page;
    holes; scales that are not powers of two, not finite, extreme."""
    seqs, heads, m = 5, 3, 7
    p = Pages(kv, seqs, heads, m, pt, d, seed=pt)
    rng = np.random.default_rng(d)
    p.k[0] = np.where(rng.random((p.n_pages, 1)) < 0.5, p.k[0] & 0xF7, p.k[0]).astype(np.uint8)   # half of the pages without NaN
    p.k[0][::7] &= 0x80                                        # zeros of both signs
    p.k[0][1::7] &= 0x83                                       # subnormal codes
    p.k[0][2::7] = 0x7E                                        # 448
    p.k[0][3::7] = 0x60 | rng.integers(0, 8, p.k[0][3::7].shape)    # one sign
    p.k[1] = rng.choice(np.array([1, 0.75, 2.0 ** -126, 2.0 ** 119, np.inf, np.nan, 2.0 ** -9], np.float32), p.n_pages)
    p.pages[0, 0, 2], p.pages[1, 1, 0] = -1, p.n_pages
    p.upload()
    o = Outlines(p)
    for lens, counts, new in (([m * pt, m * pt - 1, 1, 0, pt + 1], None, m * pt), ([2 * pt + 2, 2 * pt + 5, -3, 10 ** 6, pt], [3, 0, 9, 2 * pt, -1], 3 * pt),
                              ([pt - 1, 3, 2, 2 * pt - 3, 3 * pt + 7], None, 1)):
        lengths = grid(seqs, heads, lens)
        o.expect(p, lengths, new, counts)
        kv.ibp_kv_outline(p.cache, o.t, p.gpu_pages, gpu(lengths), n_new=new, counts=gpu(None if counts is None else np.array(counts, np.int32)))
        o.check()
    o.expect(p, grid(seqs, heads, [m * pt] * seqs), m * pt)
    kv.ibp_kv_outline(p.cache, o.t, p.gpu_pages, gpu(grid(seqs, heads, [m * pt] * seqs)))     # all that hold tokens
    o.check()


def test_outline_of_every_largest_code(kv):
    """Pages whose largest magnitude is each of the codes in turn: the unit's edge."""
    d, pt = 64, 16
    p = Pages(kv, 1, 1, 127, pt, d)
    rng = np.random.default_rng(0)
    for c in range(127):
        page = p.pages[0, 0, c]
        p.k[0][page] = rng.integers(0, c + 1, pt * d) | (rng.integers(0, 2, pt * d) << 7)
        p.k[0][page, rng.integers(0, pt * d)] = c | (128 if c % 2 else 0)
    p.upload()
    o = Outlines(p)
    o.expect(p, [[127 * pt]], 127 * pt)
    kv.ibp_kv_outline(p.cache, o.t, p.gpu_pages, gpu(np.array([[127 * pt]], np.int32)))
    o.check()


@pytest.mark.parametrize("pt,d,m,new", [(16, 64, 5000, None), (16, 128, 4097, 60001), (32, 128, 3001, None), (32, 192, 2500, 70000),
                                        (64, 256, 1501, None), (16, 64, 70000, None)])
def test_outline_many_pages_to_a_wave(kv, pt, d, m, new):
    """Rows of so many pages that a wave takes several, up to 64, which end at any
    place of a run; rows of different lengths; holes; pages that rows share."""
    p = noise(kv, 2, 2, m, pt, d, seed=m, n_pages=300)
    p.k[0][5, 3 * d + 1] = 0x7F
    p.k[1][9] = np.inf
    p.upload()
    p.pages %= 290
    p.pages[:, :, ::97] = -1
    lengths = np.array([[m * pt - 3, m * pt // 3 + 1], [(m - 1) * pt + 1, 5 * pt - 2]], np.int32)
    for row, last in enumerate(((lengths - 1) // pt).reshape(-1)):
        p.pages.reshape(4, m)[row, last] = 290 + row              # the one page of a row that is not full
    o = Outlines(p)
    n = m * pt if new is None else new
    for s in range(2):
        for h in range(2):
            first = max(int(lengths[s, h]) - n, 0) // pt
            last = (int(lengths[s, h]) - 1) // pt
            ids = np.unique(p.pages[s, h, first:last])            # each of them once is enough
            ids = np.concatenate((ids[ids >= 0], p.pages[s, h, last:last + 1])).astype(np.int32)[None, None]
            tokens = (ids.size - 1) * pt + int(lengths[s, h]) - last * pt
            lorc.outline(*p.k, orc.k_place(pt, d), pt, ids, np.array([[tokens]]), o.codes, o.scales, tokens)
    kv.ibp_kv_outline(p.cache, o.t, gpu(p.pages), gpu(lengths), n_new=new)
    o.check()


# ------------------------------------------------------------ selection ----


def outlined(p, seed=0):
    """Outlines of all pages of the pool, whatever the tables say."""
    o = Outlines(p, seed)
    rows = np.arange(p.n_pages, dtype=np.int32)[None, None]
    lorc.outline(*p.k, orc.k_place(p.pt, p.d), p.pt, rows, np.array([[p.n_pages * p.pt]]), o.codes, o.scales, p.n_pages * p.pt)
    o.t = (gpu(o.codes), gpu(o.scales))
    return o


def check_select(kv, p, o, lengths, q, keep, sink=1, recent=1, counts=None, gpu_q=None, **more):
    lengths = np.asarray(lengths, np.int32)
    c = None if counts is None else np.asarray(counts, np.int32)
    got = kv.ibp_kv_select(p.cache, o.t, p.gpu_pages, gpu(lengths), q.cuda() if gpu_q is None else gpu_q, keep, sink_pages=sink,
                           recent_pages=recent, counts=gpu(c), **more)
    torch.cuda.synchronize()
    want = lorc.select(o.codes, o.scales, p.pages, lengths, p.pt, q.double().numpy(), keep, sink, recent, c)
    for name, x, y in zip(("pages", "lengths", "places"), got, want):
        x = np_of(x)
        assert np.array_equal(x, y), (name, np.argwhere(x != y)[:4])
    return got


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("pt", [16, 64])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group,new", [(1, 1), (3, 1), (16, 1), (5, 5), (8, 4), (35, 2)])
def test_select(kv, d, pt, dtype, group, new):
    """Rows from none to more than a workgroup scores; one query to several
    groups of 16."""
    seqs, heads, m = 5, 2, 140
    p = noise(kv, seqs, heads, m, pt, d, seed=d + group)
    o = outlined(p)
    q = queries(group, seqs, new, heads * group, d, dtype)
    lengths = grid(seqs, heads, [0, 1, 15 + new, 64 * pt + 3, m * pt])
    lengths[3, 1] = m * pt - pt - 1
    for keep, sink, recent in ((3, 0, 2), (9, 1, 2), (40, 2, 5), (139, 1, 2), (150, 0, 2)):
        check_select(kv, p, o, lengths, q, keep, sink, recent)


@pytest.mark.parametrize("m", [300, 1100])
@pytest.mark.parametrize("d", [64, 256])
def test_select_many_queries(kv, d, m):
    """More queries than LDS holds at a time, over several runs of pages; some
    of a row's queries do not exist."""
    seqs, heads, group, new = 2, 1, 13, 8
    p = noise(kv, seqs, heads, m, 16, d, seed=m, n_pages=50)
    o = outlined(p)
    q = queries(1, seqs, new, heads * group, d, "fp16")
    q[0, 1:7] *= 0.1
    for counts in (None, [8, 3]):
        check_select(kv, p, o, grid(seqs, heads, [m * 16, m * 16 - 100]), q, 20, 1, 2, counts=counts)


@pytest.mark.parametrize("d", [64, 192])
@pytest.mark.parametrize("m", [255, 256, 257, 1023, 1024, 1025, 4096, 4097, 16384, 16385])
def test_select_rows_at_the_kernels_edges(kv, m, d):
    """Row lengths at which one kernel takes over from another; few distinct
    pages, so that many scores are equal."""
    p = noise(kv, 2, 2, m, 16, d, seed=m, n_pages=97)
    o = outlined(p)
    q = queries(1, 2, 1, 4 if d == 64 or m > 1025 else 38, d, "bf16")     # one group of 16 queries, or two
    lengths = grid(2, 2, [m * 16, m * 16 - 40])
    for keep, sink, recent in ((2, 1, 1), (m // 3, 0, 1), (m - 1, 3, 2)):
        check_select(kv, p, o, lengths, q, keep, sink, recent)


def test_select_scores_of_every_kind(kv):
    """Holes; outlines with NaN, infinite, zero, negative and extreme scales;
    equal scores; queries that are not finite, zero, extreme or do not exist."""
    seqs, heads, group, d, pt, m, new = 6, 2, 3, 128, 16, 70, 4
    p = noise(kv, seqs, heads, m, pt, d, seed=3)
    rng = np.random.default_rng(2)
    o = outlined(p)
    o.scales[:] = rng.choice(np.array([1, 1, 1, 0.5, 3, np.nan, np.inf, -np.inf, 0, -0.0, -1, 2.0 ** -149, 3e38], np.float32), p.n_pages)
    o.codes[::3] = o.codes[0]
    o.codes[1::9] = 0
    o.codes[4::50] = -128
    o.t = (gpu(o.codes), gpu(o.scales))
    p.pages[0, 0, [0, 3, 9]], p.pages[0, 1, 4:60], p.pages[1], p.pages[2, 0, 5] = -1, p.n_pages + 5, -1, 2 ** 31 - 1
    p.upload()
    for dtype in ("bf16", "fp16"):
        q = queries(7, seqs, new, heads * group, d, dtype)
        q[2, 1, 0, 5], q[2, 2, 4, 100], q[2, 3, 1] = float("inf"), float("nan"), 0.0
        q[3] = 0.0
        q[4, :, 0] = torch.finfo(q.dtype).max
        q[4, :, 4, ::2] = -torch.finfo(q.dtype).max
        q[4, :, 5] = torch.finfo(q.dtype).smallest_normal / 8
        q[5, :2] = float("nan")
        for counts in (None, [4, 2, 3, 1, 0, 2]):
            for keep, sink, recent in ((12, 1, 2), (33, 0, 3), (60, 2, 2)):
                check_select(kv, p, o, grid(seqs, heads, [m * pt, 900, m * pt - 5, 1000, 10 ** 6, 800]), q, keep, sink, recent, counts=counts)
    # lengths below the count: tokens before position 0
    check_select(kv, p, o, grid(seqs, heads, [3, 1, 0, -4, 17, 33]), q, 2, 0, 2)


@pytest.mark.parametrize("m", [60, 1100])
def test_select_strides_buffers_and_stream(kv, m):
    seqs, heads, group, d, pt, new, keep = 3, 2, 4, 128, 16, 2, 10
    p = noise(kv, seqs, heads, m, pt, d, seed=1)
    o = outlined(p)
    lengths = grid(seqs, heads, [900, 600, m * pt - 1])
    q = queries(2, seqs, new, heads * group, d, "bf16")
    odd = torch.empty(seqs, heads * group, new, d + 1, dtype=torch.bfloat16, device="cuda")[..., 1:].transpose(1, 2).copy_(q)
    n = kv.ibp_kv_select_workspace_bytes(p.cache, p.gpu_pages, gpu(lengths))
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    outs = [torch.full(s, 99, dtype=torch.int32, device="cuda") for s in ((seqs, heads, keep), (seqs, heads), (seqs, heads, keep))]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = check_select(kv, p, o, lengths, q, keep, 1, 2, gpu_q=odd, workspace=ws[:n], pages_out=outs[0], lengths_out=outs[1],
                       places_out=outs[2], stream=s)
    assert all(x is y for x, y in zip(got, outs)) and (ws[n:] == 0xFF).all()
    wide = torch.randn(seqs, new, 1, d, device="cuda").bfloat16().expand(-1, -1, heads * group, -1)     # one query for all heads
    check_select(kv, p, o, lengths, wide.cpu().contiguous(), keep, 1, 2, gpu_q=wide)
    if n:
        with pytest.raises(kv.IBPKVError, match="invalid argument"):
            kv.ibp_kv_select(p.cache, o.t, p.gpu_pages, gpu(lengths), q.cuda(), keep, recent_pages=2, workspace=ws[:n - 64])


@pytest.mark.parametrize("d", [64, 128])
def test_attention_over_a_selection(kv, d):
    """The selected table through ibp_kv_attention: what attention over those
    pages gives, weights by their places; with all pages kept, that of the row."""
    seqs, heads, group, pt, m, new = 3, 2, 4, 16, 80, 3
    p = filled(kv, seqs, heads, m, pt, d, [1200, 40, 777], seed=2)
    o = outlined(p)
    lengths = grid(seqs, heads, [1200, 40, 777])
    q = queries(4, seqs, new, heads * group, d, "bf16")
    for keep in (12, m):
        pages, left, places = check_select(kv, p, o, lengths, q, keep, 1, 2)
        w = torch.zeros(seqs, heads, keep, device="cuda")
        out, wo = kv.ibp_kv_attention(p.cache, pages, left, q.cuda(), weights=w)
        held, p.pages = p.pages, np_of(pages)
        want = expect(p, np_of(left), q, np.zeros((seqs, heads, keep), np.float32))
        p.pages = held
        close(out.cpu(), np_of(wo), want)
        if keep == m:
            close(out.cpu(), None, expect(p, lengths, q))
        # the weights of the table's pages
        total = torch.zeros(seqs, heads, m + 1, device="cuda")
        total.scatter_add_(2, torch.where(places < 0, m, places).long(), wo)
        assert abs(float(total.sum()) - seqs * new * heads * group) < 1e-2


def test_no_page_left_out_has_a_larger_score(kv):
    """What a selection is for: no token of a page that it leaves out scores
    higher than the bound of any page that it chose (queries that point at one
    token each; up to the rounding of the query, half a unit for each number)."""
    heads, d, pt, m = 4, 128, 16, 200
    p = filled(kv, 1, heads, m, pt, d, [m * pt], seed=5)
    o = outlined(p)
    key, place = np.zeros((heads, d), np.float32), orc.k_place(pt, d)
    for h, t in enumerate([77, 1001, 2500, 3100]):
        page = p.pages[0, h, t // pt]
        key[h] = orc.NUMBERS[p.k[0][page][place[t % pt]]] * p.k[1][page]
    q = torch.from_numpy(key)[None, None].bfloat16()
    _, _, places = check_select(kv, p, o, [[m * pt] * heads], q, 12, 1, 2)
    for h in range(heads):
        x = q[0, 0, h].double().numpy()
        query = lorc.whole_query(x)
        chosen = np_of(places)[0, h, 1:-2]
        left_out = np.setdiff1d(np.arange(1, m - 2), chosen)
        ids = p.pages[0, h]
        least = min(float(lorc.score([query], o.codes[i].astype(np.int64), o.scales[i])) for i in ids[chosen])
        for i in ids[left_out]:
            k = orc.NUMBERS[p.k[0][i][place]] * p.k[1][i]
            assert (k @ x <= least * (1 + 2.0 ** -22) + query[1] / 2 * np.abs(k).sum(1)).all()


# ------------------------------------------------------ shared prefixes ----


# Half a step of the weights in the second product: 11 bits for outputs of 8, else 16
# (a relative error of 2^-11 at most, an eighth of the output's own).
WEIGHT = {torch.bfloat16: 2.0 ** -11, torch.float16: 2.0 ** -16}


def shared_pool(kv, seqs, heads, prefix_pages, own_pages, pt, d, seed=0, n_pages=4096):
    """Pages of random codes; tables of a prefix and of own pages over them."""
    p = noise(kv, seqs, heads, own_pages, pt, d, seed, n_pages)
    rng = np.random.default_rng(seed + 1)
    p.prefix = rng.integers(0, p.n_pages, (heads, prefix_pages)).astype(np.int32)
    return p


def check_shared(kv, p, prefix_lengths, lengths, q, scale=None, counts=None, gpu_q=None, **more):
    prefix_lengths, lengths = np.asarray(prefix_lengths, np.int32), np.asarray(lengths, np.int32)
    c = None if counts is None else np.asarray(counts, np.int32)
    out = kv.ibp_kv_attention_shared(p.cache, gpu(p.prefix), gpu(prefix_lengths), p.gpu_pages, gpu(lengths),
                                     q.cuda() if gpu_q is None else gpu_q, scale=scale, counts=gpu(c), **more)
    torch.cuda.synchronize()
    fi = torch.finfo(q.dtype)
    o, err = lorc.attention_shared(p.k, p.v, p.pt, p.prefix, prefix_lengths, p.pages, lengths, q.double().numpy(),
                                   p.d ** -0.5 if scale is None else scale, c, rounding=fi.eps / 2, tiny=fi.tiny * fi.eps / 2,
                                   weight=WEIGHT[q.dtype])
    got = out.cpu()
    # past the type's largest number an infinity, which a number within its error of that
    # may be as well
    far, near = np.abs(o) - err > fi.max, np.abs(o) + err > fi.max
    infinite = near & np.isinf(got.double().numpy()) & (np.signbit(got.double().numpy()) == np.signbit(o))
    assert infinite[far].all()
    got[torch.from_numpy(infinite)] = 0
    o[infinite] = 0
    close(got, None, (o, None, err, None))
    return out


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("pt", [16, 32, 64])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group,new", [(1, 1), (3, 1), (8, 1), (5, 7)])
def test_attention_shared(kv, d, pt, dtype, group, new):
    """Ragged own rows behind one prefix: 5 to 175 query rows a head."""
    seqs, heads = 5, 2
    p = shared_pool(kv, seqs, heads, -(-400 // pt), -(-200 // pt), pt, d, seed=d + pt)
    q = queries(new, seqs, new, heads * group, d, dtype)
    check_shared(kv, p, [333, 333], grid(seqs, heads, [new, 1, 15 + new, 64 + pt, 130]), q, scale=0.02)


@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 511, 1000])
def test_attention_shared_prefix_lengths(kv, n):
    p = shared_pool(kv, 3, 1, 64, 4, 16, 128, seed=n)
    q = queries(n, 3, 1, 4, 128, "bf16")
    check_shared(kv, p, [n], grid(3, 1, [1, 40, 0]), q, scale=0.05)


@pytest.mark.parametrize("seqs,group,new", [(2, 1, 1), (16, 1, 1), (17, 1, 1), (8, 4, 1), (11, 3, 1), (16, 4, 1), (13, 5, 1), (6, 7, 4), (32, 8, 1)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_shared_rows(kv, d, seqs, group, new):
    """Query rows about the edges of a unit of the prefix, 2 to 256 of them;
    prefixes of heads that differ, in many parts."""
    heads, pt = 2, 32
    p = shared_pool(kv, seqs, heads, 90, 6, pt, d, seed=seqs)
    q = queries(group, seqs, new, heads * group, d, "fp16")
    check_shared(kv, p, [2800, 1711], grid(seqs, heads, [(i * 37) % 190 + new for i in range(seqs)]), q, scale=0.02)


def test_attention_shared_long_own_rows(kv):
    """Own rows that are cut into parts themselves."""
    seqs, heads, group, new, d, pt = 3, 2, 4, 9, 64, 64
    p = shared_pool(kv, seqs, heads, 20, 160, pt, d, seed=3)
    q = queries(1, seqs, new, heads * group, d, "bf16")
    lengths = grid(seqs, heads, [10000, 300, 5])
    lengths[0, 1] = 77
    check_shared(kv, p, [1200, 640], lengths, q, scale=0.02)
    check_shared(kv, p, [1200, 640], lengths, q, scale=0.02, counts=[9, 2, 4])


def test_attention_shared_holes_counts_and_lengths(kv):
    """Holes in the prefix and in rows, whole ones; counts below n_new; lengths
    below the count and outside; a prefix of nothing but holes; rows that see
    nothing."""
    seqs, heads, group, new, pt, d = 6, 2, 3, 5, 16, 64
    p = shared_pool(kv, seqs, heads, 20, 12, pt, d, seed=2)
    p.pages[0, 0, [0, 3, 9]], p.pages[0, 1, 4:8], p.pages[1] = -1, p.n_pages + 5, -1
    p.prefix[0, [0, 7, 19]] = -1, p.n_pages, 2 ** 31 - 1
    p.upload()
    q = queries(1, seqs, new, heads * group, d, "bf16")
    lengths = grid(seqs, heads, [150, 90, 3, 5000, -4, 77])
    for counts in (None, [5, 5, 5, 2, 5, 0], [1, 9, 4, 0, -1, 3]):
        out = check_shared(kv, p, [300, 10 ** 6], lengths, q, scale=0.03, counts=counts)
        assert not out[4].any()
    p.prefix[:] = -1
    out = check_shared(kv, p, [300, -5], lengths, q, scale=0.03)
    assert not out[1].any()


def test_attention_shared_nan(kv):
    """NaN values of the prefix reach every query, those of a row the queries
    that see them; what lies past the prefix's end reaches none."""
    seqs, heads, group, new, pt, d = 3, 1, 2, 6, 16, 128
    p = shared_pool(kv, seqs, heads, 8, 16, pt, d, seed=6, n_pages=1 << 20)
    ids = np.random.default_rng(5).permutation(p.n_pages)         # every page of its own,
    p.prefix[0], p.pages = ids[:8], ids[8:8 + seqs * 8].reshape(seqs, 1, 8).astype(np.int32)
    p.pages[1, 0] = p.prefix[0][::-1]                             # but for a row of the prefix's pages
    p.upload()
    q = queries(1, seqs, new, heads * group, d, "fp16")
    place = orc.v_place(pt, d)
    p.v[0][p.prefix[0, 6], place[4:].reshape(-1)] = 0x7F          # the prefix ends inside page 6
    p.v[1][p.prefix[0, 7]] = np.nan
    p.k[0][p.prefix[0, 7]] = 0x7F
    p.upload()
    out = check_shared(kv, p, [100], [[60], [15], [20]], q, scale=0.03)
    assert not out[[0, 2]].isnan().any()
    p.v[0][p.prefix[0, 2], place[3, 77]] = 0xFF
    p.v[0][p.pages[0, 0, 3], place[57 - 48, 5]] = 0xFF
    p.upload()
    out = check_shared(kv, p, [100], [[60], [15], [20]], q, scale=0.03)
    nan = np_of(out.isnan())
    assert nan[..., 77].all() and nan[0, 3:, :, 5].all() and not nan[0, :3, :, 5].any()
    p.v[1][p.prefix[0, 1]] = np.inf
    p.upload()
    assert kv.ibp_kv_attention_shared(p.cache, gpu(p.prefix), gpu(np.array([100], np.int32)), p.gpu_pages,
                                      gpu(np.array([[60], [15], [20]], np.int32)), q.cuda()).isnan().all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("seqs", [3, 40])
@pytest.mark.parametrize("scale", [0.02, -0.05])
def test_attention_shared_scales_of_every_kind(kv, dtype, seqs, scale):
    """Scales that are no powers of two, negative, zero, far apart; few and many
    query rows."""
    heads, group, pt, d = 2, 3, 16, 128
    p = shared_pool(kv, seqs, heads, 40, 6, pt, d, seed=9)
    rng = np.random.default_rng(4)
    p.v[1] = rng.choice(np.array([1, 1, 1, 0.75, 3, 2.0 ** -30, 2.0 ** -70, 2.0 ** -126, 0, -0.0, -0.5, -3, 2.0 ** 20], np.float32), p.n_pages)
    p.k[1] = rng.choice(np.array([1, 1, 0.5, -1, -0.3, 0, 1.7], np.float32), p.n_pages)
    p.upload()
    q = queries(2, seqs, 1, heads * group, d, dtype)
    check_shared(kv, p, [640, 333], grid(seqs, heads, [(i * 7) % 90 + 1 for i in range(seqs)]), q, scale=scale)


@pytest.mark.parametrize("seqs", [2, 40])
def test_attention_shared_queries_not_finite(kv, seqs):
    """They are NaN whole, and no other query is."""
    p = shared_pool(kv, seqs, 1, 30, 4, 16, 64, seed=1)
    q = queries(1, seqs, 1, 4, 64, "bf16")
    q[0, 0, 1, 5], q[1, 0, 2, 0], q[1, 0, 3] = float("inf"), float("nan"), torch.finfo(q.dtype).max
    out = kv.ibp_kv_attention_shared(p.cache, gpu(p.prefix), gpu(np.array([470], np.int32)), p.gpu_pages, gpu(grid(seqs, 1, [30] * seqs)),
                                     q.cuda())
    nan = np_of(out.isnan())
    assert nan[0, 0, 1].all() and nan[1, 0, 2].all()
    rest = np.ones(nan.shape[:3], bool)
    rest[0, 0, 1] = rest[1, 0, 2] = rest[1, 0, 3] = False
    assert not nan[rest].any()


def test_attention_shared_tables_without_pages(kv):
    """A prefix, rows, or both, of no pages at all."""
    p = shared_pool(kv, 3, 2, 8, 4, 16, 64, seed=2)
    q = queries(1, 3, 1, 4, 64, "fp16")
    whole, own, prefix = p.pages, p.gpu_pages, p.prefix
    p.prefix = prefix[:, :0]
    check_shared(kv, p, [100, 0], grid(3, 2, [30, 1, 64]), q)
    p.prefix, p.pages, p.gpu_pages = prefix, whole[:, :, :0], own[:, :, :0].contiguous()
    assert not check_shared(kv, p, [100, 9], grid(3, 2, [30, 1, 64]), q).any()     # no place: the tokens do not exist
    o = outlined(p)
    got = kv.ibp_kv_select(p.cache, o.t, p.gpu_pages, gpu(grid(3, 2, [30, 1, 64])), q.cuda(), 4)
    assert (got[0] == -1).all() and not got[1].any() and (got[2] == -1).all()
    kv.ibp_kv_outline(p.cache, o.t, p.gpu_pages, gpu(grid(3, 2, [30, 1, 64])))
    cos, sin = tables(70, 32)
    k = queries(2, 3, 1, 2, 64, "fp16").cuda()
    turned = kv.ibp_kv_append_rotated(p.cache, p.gpu_pages, gpu(grid(3, 2, [30, 1, 64])), k, k, gpu(cos), gpu(sin), q=q.cuda(), outlines=o.t)
    torch.cuda.synchronize()
    assert not turned.any()
    o.check()


def test_attention_shared_equals_attention_of_whole_rows(kv):
    """A prefix of whole pages in front of each row's table gives the same."""
    seqs, heads, group, new, pt, d = 4, 2, 2, 2, 16, 128
    p = filled(kv, 1, heads, 60, pt, d, [960], seed=4)
    p.prefix = p.pages[0, :, :40].copy()
    own = p.pages[0][None, :, 40:50].repeat(seqs, 0)
    lengths = grid(seqs, heads, [2, 33, 100, 160])
    q = queries(1, seqs, new, heads * group, d, "bf16")
    p.pages = own
    p.upload()
    check_shared(kv, p, [640, 640], lengths, q)
    p.pages = np.concatenate([p.prefix[None].repeat(seqs, 0), own], 2)
    p.upload()
    out, _ = run_attention(kv, p, lengths + 640, q)
    close(out, None, expect(p, lengths + 640, q))


def test_attention_shared_large_scores(kv):
    """Scores of some hundreds, of either sign: the statistics must be those of
    the prefix and the row together."""
    p = shared_pool(kv, 3, 2, 30, 10, 16, 128, seed=8)
    q = queries(2, 3, 1, 8, 128, "bf16") * 8
    for scale in (1.0, 0.0, -0.7):
        check_shared(kv, p, [470, 33], grid(3, 2, [150, 1, 60]), q, scale=scale)


def test_attention_shared_strides_buffers_and_stream(kv):
    seqs, new, heads, group, d, pt = 3, 2, 2, 4, 128, 32
    p = shared_pool(kv, seqs, heads, 40, 20, pt, d, seed=3)
    lengths, pl = grid(seqs, heads, [70, 200, 513]), np.array([1200, 1100], np.int32)
    q = queries(1, seqs, new, heads * group, d, "bf16")
    plain = check_shared(kv, p, pl, lengths, q)
    n = kv.ibp_kv_attention_shared_workspace_bytes(p.cache, gpu(p.prefix), gpu(pl), p.gpu_pages, gpu(lengths), heads * group, new)
    assert n > 0
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    odd_q = torch.empty(seqs, new, heads * group, d + 1, dtype=torch.bfloat16, device="cuda")[..., 1:].copy_(q)
    odd_out = torch.zeros(seqs, heads * group, new, d + 5, dtype=torch.bfloat16, device="cuda")[..., 3:3 + d].transpose(1, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = check_shared(kv, p, pl, lengths, q, gpu_q=odd_q, out=odd_out, workspace=ws[:n], stream=s)
    assert got is odd_out and torch.equal(got, plain) and (ws[n:] == 0xFF).all()
    assert not odd_out._base[..., :3].any() and not odd_out._base[..., 3 + d:].any()
    for _ in range(3):
        assert torch.equal(check_shared(kv, p, pl, lengths, q, workspace=ws[:n]), plain)
    with pytest.raises(kv.IBPKVError, match="invalid argument"):
        kv.ibp_kv_attention_shared(p.cache, gpu(p.prefix), gpu(pl), p.gpu_pages, gpu(lengths), q.cuda(), workspace=ws[:n - 64])


# ------------------------------------------------------------- together ----


def test_pool_without_pages(kv):
    """Every id is a hole."""
    none = [torch.empty(0, dtype=torch.uint8, device="cuda"), torch.empty(0, device="cuda")]
    cache = kv.ibp_kv_cache(*none, *none, 16, 64)
    pages = torch.zeros(2, 3, 200, dtype=torch.int32, device="cuda")
    lengths = torch.full((2, 3), 3000, dtype=torch.int32, device="cuda")
    x, q = (torch.ones(2, 1, h, 64, dtype=torch.float16, device="cuda") for h in (3, 6))
    cos, sin = (gpu(t) for t in tables(4000, 32))
    outlines = (torch.empty(0, 2, 64, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"))
    out = kv.ibp_kv_append_rotated(cache, pages, lengths, x, x, cos, sin, q=q, outlines=outlines)
    want = lorc.rotated(q.cpu().double().numpy(), np_of(cos), np_of(sin), np_of(lengths), 200, 16)
    assert torch.equal(out.cpu(), torch.from_numpy(want).half())
    kv.ibp_kv_outline(cache, outlines, pages, lengths)
    got = kv.ibp_kv_select(cache, outlines, pages, lengths, q, 9, sink_pages=2, recent_pages=1)
    assert got[2][0, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 187] and (got[1] == 9 * 16 - 8).all()
    out = kv.ibp_kv_attention_shared(cache, pages[0].contiguous(), lengths[0].contiguous(), pages, lengths, q)
    torch.cuda.synchronize()
    assert not out.any()


def test_calls_without_sequences_or_tokens(kv):
    p = noise(kv, 2, 2, 8, 16, 64, seed=1)
    o = outlined(p)
    lengths = gpu(grid(2, 2, [100, 128]))
    none = torch.zeros(2, 0, 4, 64, dtype=torch.bfloat16, device="cuda")
    pages, left, places = kv.ibp_kv_select(p.cache, o.t, p.gpu_pages, lengths, none, 4, sink_pages=1)
    torch.cuda.synchronize()
    assert np_of(places)[0, 0].tolist() == [0, 1, 2, 6] and np_of(left)[1].tolist() == [64, 64]
    prefix, pl = p.gpu_pages[0].contiguous(), lengths[0].contiguous()
    assert kv.ibp_kv_attention_shared(p.cache, prefix, pl, p.gpu_pages, lengths, none).shape == none.shape
    empty, q = p.gpu_pages[:0], torch.zeros(0, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert kv.ibp_kv_attention_shared(p.cache, prefix, pl, empty, lengths[:0], q).numel() == 0
    assert kv.ibp_kv_select(p.cache, o.t, empty, lengths[:0], q, 4)[0].shape == (0, 2, 4)
    kv.ibp_kv_outline(p.cache, o.t, empty, lengths[:0])
    cos, sin = (gpu(t) for t in tables(10, 32))
    k = torch.zeros(0, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert kv.ibp_kv_append_rotated(p.cache, empty, lengths[:0], k, k, cos, sin, q=q, outlines=o.t).numel() == 0


def test_graph_of_a_long_decoding_step(kv):
    """A step captured once and replayed: the new token is rotated and
    appended with its outlines, pages are selected and attended over, and the
    shared prefix with the row's own pages.  Every replay is checked against
    eager calls on a copy; a second graph uses the same workspaces."""
    seqs, heads, group, d, pt, m, keep = 2, 2, 3, 64, 16, 20, 6
    p = filled(kv, seqs, heads, m, pt, d, [200, 161], seed=3)
    o = outlined(p)
    dev = torch.device("cuda")
    k, v, q = (torch.zeros(seqs, 1, h, d, dtype=torch.bfloat16, device=dev) for h in (heads, heads, heads * group))
    cos, sin = (gpu(t) for t in tables(400, 32))
    prefix, pl = p.gpu_pages[0, :, :9].contiguous(), torch.full((heads,), 140, dtype=torch.int32, device=dev)

    def fresh():
        t = [x.clone() for x in p.t]
        return {"t": t, "cache": kv.ibp_kv_cache(*t, pt, d), "o": tuple(x.clone() for x in o.t),
                "lengths": gpu(grid(seqs, heads, [200, 161]))}
    some = fresh()
    ws = [torch.empty(max(n, 16), dtype=torch.uint8, device=dev) for n in (
        kv.ibp_kv_select_workspace_bytes(p.cache, p.gpu_pages, some["lengths"]),
        kv.ibp_kv_attention_shared_workspace_bytes(p.cache, prefix, pl, p.gpu_pages, some["lengths"], heads * group, 1))]

    def step(s):
        s["lengths"].add_(1)
        turned = kv.ibp_kv_append_rotated(s["cache"], p.gpu_pages, s["lengths"], k, v, cos, sin, q=q, outlines=s["o"])
        s["pages"], s["left"], s["places"] = kv.ibp_kv_select(s["cache"], s["o"], p.gpu_pages, s["lengths"], turned, keep, workspace=ws[0])
        s["sparse"], _ = kv.ibp_kv_attention(s["cache"], s["pages"], s["left"], turned)
        s["out"] = kv.ibp_kv_attention_shared(s["cache"], prefix, pl, p.gpu_pages, s["lengths"], turned, workspace=ws[1])
        many = turned.repeat(20, 1, 1, 1)
        s["many"] = kv.ibp_kv_attention_shared(s["cache"], prefix, pl, p.gpu_pages.repeat(20, 1, 1), s["lengths"].repeat(20, 1), many)

    step(some)
    torch.cuda.synchronize()
    states, graphs = [fresh(), fresh()], []
    for s in states:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step(s)
    eager = fresh()
    for i in range(20):
        for x, seed in ((k, 1), (v, 2), (q, 3)):
            x.copy_(values(100 * i + seed, tuple(x.shape), torch.bfloat16, 1.0 + i % 5))
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        step(eager)
        torch.cuda.synchronize()
        for s in states:
            for name in ("pages", "left", "places", "sparse", "out", "many", "lengths"):
                assert torch.equal(s[name], eager[name]), (i, name)
            for x, y in zip((*s["t"], *s["o"]), (*eager["t"], *eager["o"])):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), i


def test_two_calls_at_once(kv):
    """Calls on two streams over one cache, with workspaces of their own: each
    gives what it gives alone."""
    seqs, heads, group, d, pt, m = 9, 2, 5, 128, 16, 1100
    p = shared_pool(kv, seqs, heads, 300, m, pt, d, seed=11)
    o = outlined(p)
    prefix, pl = gpu(p.prefix), torch.full((heads,), 300 * pt - 7, dtype=torch.int32, device="cuda")
    lengths = [gpu(grid(seqs, heads, [m * pt - 40 * i - j for i in range(seqs)])) for j in range(2)]
    q = [queries(j, seqs, 1, heads * group, d, "bf16").cuda() for j in range(2)]
    angles = [gpu(t) for t in tables(m * pt, 64)]
    own = gpu(np.arange(seqs * heads, dtype=np.int32).reshape(seqs, heads, 1))

    def calls(j, cache, outlines, stream=None):
        k = q[j][:, :, :heads]
        turned = kv.ibp_kv_append_rotated(cache, own, gpu(grid(seqs, heads, [5 + j] * seqs)), k, k, *angles, q=q[j],
                                          outlines=outlines, stream=stream)
        chosen = kv.ibp_kv_select(p.cache, o.t, p.gpu_pages, lengths[j], q[j], 50, 1, 1, stream=stream)
        return (turned, *chosen, kv.ibp_kv_attention_shared(p.cache, prefix, pl, p.gpu_pages, lengths[j], q[j], stream=stream))

    def spare():  # what the appends write, each call's own
        t = [x.clone() for x in p.t]
        return kv.ibp_kv_cache(*t, pt, d), tuple(x.clone() for x in o.t)
    alone = []
    for j in range(2):
        alone.append(calls(j, *spare()))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        room = [spare() for _ in range(2)]
        torch.cuda.synchronize()
        got = [calls(j, *room[j], stream=streams[j]) for j in range(2)]
        torch.cuda.synchronize()
        for x, y in zip(got, alone):
            assert all(torch.equal(a, b) for a, b in zip(x, y))


def test_long_calls_have_no_gradient(kv):
    p = filled(kv, 1, 2, 10, 16, 64, [100], seed=1)
    o = outlined(p)
    lengths = torch.full((1, 2), 100, dtype=torch.int32, device="cuda")
    k, q = torch.randn(1, 1, 2, 64, device="cuda").half(), torch.randn(1, 1, 4, 64, device="cuda").half().requires_grad_()
    cos, sin = (gpu(t) for t in tables(128, 32))
    turned = kv.ibp_kv_append_rotated(p.cache, p.gpu_pages, lengths, k, k, cos, sin, q=q * 1)
    with pytest.raises(RuntimeError, match="ibp_kv_append_rotated is not implemented"):
        turned.float().sum().backward()
    prefix, pl = p.gpu_pages[0].contiguous(), lengths[0].contiguous()
    out = kv.ibp_kv_attention_shared(p.cache, prefix, pl, p.gpu_pages, lengths, q * 1)
    with pytest.raises(RuntimeError, match="ibp_kv_attention_shared is not implemented"):
        out.float().sum().backward()
    assert q.grad is None
    assert not any(x.requires_grad for x in kv.ibp_kv_select(p.cache, o.t, p.gpu_pages, lengths, q, 3))
    with pytest.raises(ValueError, match="requires a gradient"):
        kv.ibp_kv_attention_shared(p.cache, prefix, pl, p.gpu_pages, lengths, q, out=torch.empty_like(q))
    with pytest.raises(ValueError, match="requires a gradient"):
        kv.ibp_kv_append_rotated(p.cache, p.gpu_pages, lengths, k, k, cos, sin, q=q, q_out=torch.empty_like(q))
    with torch.no_grad():
        given = torch.empty_like(q)
        was = given._version
        assert kv.ibp_kv_append_rotated(p.cache, p.gpu_pages, lengths, k, k, cos, sin, q=q, q_out=given, outlines=o.t) is given
        assert given._version > was and o.t[0]._version and o.t[1]._version and p.t[0]._version


def test_pool_past_32_bits(kv):
    """Pages whose bytes, and outlines whose bytes, lie past 4 GiB."""
    pt, d = 16, 256
    n_pages = (1 << 32) // (2 * d) + 40
    codes = [torch.zeros(n_pages, pt * d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones(n_pages, device="cuda") for _ in range(2)]
    outlines = (torch.zeros(n_pages, 2, d, dtype=torch.int8, device="cuda"), torch.zeros(n_pages, device="cuda"))
    cache = kv.ibp_kv_cache(codes[0], scales[0], codes[1], scales[1], pt, d)
    ids = np.array([[[n_pages - 1, 3, n_pages - 30, 7, n_pages - 2]]], np.int32)
    n = 70
    k, v, q = values(1, (1, n, 1, d), torch.bfloat16), values(2, (1, n, 1, d), torch.bfloat16), values(3, (1, 1, 2, d), torch.bfloat16)
    cos, sin = tables(n, d // 2)
    lengths = gpu(np.array([[n]], np.int32))
    kv.ibp_kv_append_rotated(cache, gpu(ids), lengths, k.cuda(), v.cuda(), gpu(cos), gpu(sin), outlines=outlines)
    small = Pages(kv, 1, 1, 5, pt, d, n_pages=5)
    o = Outlines(small)
    append_rotated(kv, small, [[n]], k, v, cos, sin, outlines=o)
    small.check()
    for i, page in enumerate(torch.from_numpy(ids[0, 0]).long()):
        at = small.pages[0, 0, i]
        assert np.array_equal(np_of(codes[0][page]), small.k[0][at]) and np.array_equal(np_of(codes[1][page]), small.v[0][at])
        assert np.array_equal(np_of(outlines[0][page]), o.codes[at]) and float(outlines[1][page]) == o.scales[at]
    assert int((outlines[1] != 0).sum()) == 5
    pages, left, places = kv.ibp_kv_select(cache, outlines, gpu(ids), lengths, q.cuda(), 3)
    want = lorc.select(o.codes, o.scales, small.pages, np.array([[n]]), pt, q.double().numpy(), 3, 1, 1)
    assert np.array_equal(np_of(places), want[2]) and np.array_equal(np_of(pages)[0, 0], ids[0, 0][want[2][0, 0]])
    out = kv.ibp_kv_attention_shared(cache, gpu(ids[0]), gpu(np.array([n], np.int32)), gpu(ids[:, :, ::-1]), gpu(np.array([[33]], np.int32)), q.cuda())
    torch.cuda.synchronize()
    o_, err = lorc.attention_shared(small.k, small.v, pt, small.pages[0], np.array([n]), small.pages[:, :, ::-1], np.array([[33]]),
                                    q.double().numpy(), d ** -0.5, rounding=2.0 ** -8, tiny=0.0, weight=WEIGHT[torch.bfloat16])
    close(out.cpu(), None, (o_, None, err, None))

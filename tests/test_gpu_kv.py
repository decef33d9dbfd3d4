"""The 8-bit KV page cache on the GPU against the 64-bit oracle: appended
pages byte for byte, attention and page weights within bounds derived from
32-bit arithmetic (oracle/kv_oracle.py), evictions exactly."""
import numpy as np
import pytest

from oracle import kv_oracle as orc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def kv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from lossless_bit_level_amd import ibp_kv
    ibp_kv.lib()
    return ibp_kv


def np_of(x):
    return x.cpu().numpy()


class Pages:
    """A pool full of noise (NaN codes among it) with tables over it, on the
    GPU and as the oracle has it."""

    def __init__(self, kv, seqs, heads, max_pages, pt, d, seed=0, n_pages=None):
        rng = np.random.default_rng(seed)
        self.kv, self.pt, self.d = kv, pt, d
        self.n_pages = seqs * heads * max_pages + 3 if n_pages is None else n_pages
        ids = rng.permutation(self.n_pages)[:seqs * heads * max_pages]
        self.pages = ids.reshape(seqs, heads, max_pages).astype(np.int32)
        self.k = [rng.integers(0, 256, (self.n_pages, pt * d), dtype=np.uint8), np.ones(self.n_pages, np.float32)]
        self.v = [rng.integers(0, 256, (self.n_pages, pt * d), dtype=np.uint8), np.ones(self.n_pages, np.float32)]
        self.upload()

    def upload(self):
        self.t = [torch.from_numpy(x).cuda() for x in (*self.k, *self.v)]
        self.cache = self.kv.ibp_kv_cache(*self.t, self.pt, self.d)
        self.gpu_pages = torch.from_numpy(self.pages).cuda()

    def append(self, lengths, k, v, counts=None, gpu_k=None, gpu_v=None):
        """k, v: CPU tensors [seqs, new, heads, d] of the type."""
        lengths = np.asarray(lengths, np.int32)
        c = None if counts is None else np.asarray(counts, np.int32)
        for (codes, scales), x, place in ((self.k, k, orc.k_place), (self.v, v, orc.v_place)):
            orc.append(codes, scales, place(self.pt, self.d), self.pt, self.pages, lengths, x.double().numpy(), c)
        self.kv.ibp_kv_append(self.cache, self.gpu_pages, torch.from_numpy(lengths).cuda(),
                              k.cuda() if gpu_k is None else gpu_k, v.cuda() if gpu_v is None else gpu_v,
                              counts=None if c is None else torch.from_numpy(c).cuda())

    def check(self):
        torch.cuda.synchronize()
        for name, got, want in zip(("k codes", "k scales", "v codes", "v scales"), self.t, (*self.k, *self.v)):
            got = np_of(got)
            bad = np.argwhere(got != want)
            assert len(bad) == 0, (name, len(bad), bad[:4], got[tuple(bad[0])], want[tuple(bad[0])])


def values(seed, shape, dtype, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * amp
    x[..., :3] *= 20.0
    return x.to(dtype)


def grid(seqs, heads, lens):
    return np.broadcast_to(np.asarray(lens, np.int32)[:, None], (seqs, heads)).copy()


# -------------------------------------------------------------- append ----


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("pt", [16, 32, 64])
def test_append_prompt_then_steps(kv, pt, d, dtype):
    """Ragged prompts, then chunks and single tokens of growing size, so that
    pages are rescaled, then smaller ones."""
    seqs, heads, t = 3, 2, DTYPES[dtype]
    p = Pages(kv, seqs, heads, 5, pt, d, seed=pt + d)
    lens = np.array([1, pt - 1, 2 * pt + 3])
    n = int(lens.max())
    p.append(grid(seqs, heads, lens), values(1, (seqs, n, heads, d), t), values(2, (seqs, n, heads, d), t), counts=lens)
    p.check()
    for i, (new, amp) in enumerate([(1, 1.0), (5, 4.0), (1, 100.0), (pt, 0.5), (1, 1e-3), (1, 3000.0)]):
        lens = lens + new
        p.append(grid(seqs, heads, lens), values(10 + i, (seqs, new, heads, d), t, amp),
                 values(30 + i, (seqs, new, heads, d), t, amp))
        p.check()


@pytest.mark.parametrize("pt", [16, 64])
def test_append_values_at_the_edges(kv, pt):
    """Zeros, the type's extremes, subnormals, values next to a change of
    scale, infinities and NaN: each page of its own kind."""
    d, heads = 64, 1
    for dtype in (torch.bfloat16, torch.float16):
        top = torch.finfo(dtype).max
        kinds = [torch.zeros(pt, d), torch.full((pt, d), top), torch.full((pt, d), -top),
                 torch.full((pt, d), 2.0 ** -24), torch.full((pt, d), 448.0), torch.full((pt, d), 450.0),
                 torch.linspace(-448, 448, pt * d).reshape(pt, d), torch.full((pt, d), float("nan")),
                 torch.full((pt, d), float("inf")), -torch.zeros(pt, d)]
        mixed = torch.randn(pt, d, generator=torch.Generator().manual_seed(5))
        mixed[::3, ::5], mixed[1::3, ::7], mixed[2::3, ::4] = float("nan"), float("inf"), float("-inf")
        kinds.append(mixed)
        if dtype == torch.bfloat16:
            kinds.append(torch.full((pt, d), 2.0 ** -130))
        x = torch.stack(kinds).to(dtype)[:, :, None]      # one sequence a kind
        p = Pages(kv, len(kinds), heads, 2, pt, d, seed=9)
        p.append(grid(len(kinds), heads, [pt] * len(kinds)), x, x.flip(2) * 1)
        p.check()
        # one more token each: the pages past them stay as they are
        p.append(grid(len(kinds), heads, [pt + 1] * len(kinds)), x[:, :1], -x[:, :1])
        p.check()


def test_append_rescale_to_subnormals(kv):
    """A page's old codes fall under a much larger scale: rounded once more,
    NaN kept."""
    d, pt = 128, 32
    p = Pages(kv, 1, 1, 1, pt, d)
    x = values(3, (1, 9, 1, d), torch.bfloat16)
    x[0, 2, 0, 5] = float("nan")
    p.append([[9]], x, x * 2)
    for n, amp in ((10, 50.0), (12, 1e4), (13, 1e30)):
        y = values(n, (1, n - 9 if n == 10 else 2 if n == 12 else 1, 1, d), torch.bfloat16, amp)
        p.append([[n]], y, -y)
        p.check()


def test_append_again_changes_nothing(kv):
    d, pt = 64, 16
    p = Pages(kv, 2, 2, 4, pt, d)
    p.append(grid(2, 2, [20, 33]), values(1, (2, 33, 2, d), torch.float16), values(2, (2, 33, 2, d), torch.float16), counts=[20, 33])
    x, y = values(3, (2, 1, 2, d), torch.float16, 90.0), values(4, (2, 1, 2, d), torch.float16, 90.0)
    for _ in range(3):
        p.append(grid(2, 2, [21, 34]), x, y)
        p.check()


@pytest.mark.parametrize("how", ["transposed", "offset", "broadcast", "reversed"])
def test_append_strides(kv, how):
    seqs, new, heads, d, pt = 2, 19, 3, 128, 16
    x, y = values(1, (seqs, new, heads, d), torch.bfloat16), values(2, (seqs, new, heads, d), torch.bfloat16)
    p = Pages(kv, seqs, heads, 3, pt, d)
    if how == "transposed":      # stored [seqs, heads, new, d]
        gx, gy = (t.transpose(1, 2).contiguous().cuda().transpose(1, 2) for t in (x, y))
    elif how == "offset":        # no 16-byte alignment: rows of d + 3, the first element left out
        gx, gy = (torch.empty(seqs, new, heads, d + 3, dtype=torch.bfloat16, device="cuda")[..., 1:d + 1].copy_(t) for t in (x, y))
        assert gx.data_ptr() % 16 and gx.stride(2) % 8
    elif how == "broadcast":     # every head the same
        x, y = x[:, :, :1].expand(-1, -1, heads, -1), y[:, :1].expand(-1, new, -1, -1)
        gx, gy = x[:, :, :1].contiguous().cuda().expand(-1, -1, heads, -1), y[:, :1].contiguous().cuda().expand(-1, new, -1, -1)
        assert gx.stride(2) == 0 and gy.stride(1) == 0
    else:                        # a window of a longer buffer
        gx, gy = (torch.cat([t, t, t], 1).cuda()[:, new:2 * new] for t in (x, y))
    p.append(grid(seqs, heads, [new + 7, new]), x.contiguous(), y.contiguous(), gpu_k=gx, gpu_v=gy)
    p.check()


def test_append_holes_counts_and_lengths_outside(kv):
    """Holes take nothing, counts and lengths are clamped, tokens before
    position 0 do not exist; noise everywhere else stays."""
    seqs, heads, d, pt, m = 6, 2, 64, 16, 3
    p = Pages(kv, seqs, heads, m, pt, d)
    p.pages[0, 0, 1], p.pages[0, 1, 0], p.pages[1, 1, 2] = -1, p.n_pages, 2 ** 31 - 1
    p.upload()
    new = 40
    x, y = values(1, (seqs, new, heads, d), torch.bfloat16), values(2, (seqs, new, heads, d), torch.bfloat16)
    lens = grid(seqs, heads, [48, 45, 0, -7, 100, 30])      # capacity 48
    lens[5, 1] = 3                                          # heads of a sequence may differ
    p.append(lens, x, y, counts=[40, 99, 5, 5, 21, 40])
    p.check()
    p.append(lens, x, y, counts=[0, -3, 0, 0, 0, 0])
    p.check()
    p.append(grid(seqs, heads, [0] * seqs), x[:, :0], y[:, :0])
    p.check()


# ----------------------------------------------------------- attention ----


def filled(kv, seqs, heads, max_pages, pt, d, lens, seed=0, amp=1.0):
    """Pages with random tokens; what the rows do not reach stays noise."""
    p = Pages(kv, seqs, heads, max_pages, pt, d, seed)
    n = max_pages * pt
    p.k[1][:], p.v[1][:] = 2.0 ** 9, 2.0 ** 11
    full = grid(seqs, heads, [n] * seqs)
    x, y = values(seed + 1, (seqs, n, heads, d), torch.float32, amp), values(seed + 2, (seqs, n, heads, d), torch.float32)
    for s in range(seqs):   # only as far as the rows go
        m = int(lens[s])
        if m > 0:
            one = np.zeros((seqs, heads), np.int32)
            one[s] = m
            cnt = np.zeros(seqs, np.int32)
            cnt[s] = m
            for (codes, scales), t, place in ((p.k, x, orc.k_place), (p.v, y, orc.v_place)):
                orc.append(codes, scales, place(pt, d), pt, p.pages, one, t[:, :m].double().numpy(), cnt)
    # bytes past a row's length hold noise and NaN, as a reused page may
    rng = np.random.default_rng(seed + 7)
    for s in range(seqs):
        m = int(lens[s])
        if 0 < m < n and m % pt:
            for h in range(heads):
                page = p.pages[s, h, m // pt]
                for pool, place in ((p.k, orc.k_place(pt, d)), (p.v, orc.v_place(pt, d))):
                    rest = place[m % pt:].reshape(-1)
                    pool[0][page, rest] = np.where(rng.random(rest.size) < 0.3, 0x7F, rng.integers(0, 256, rest.size))
    p.upload()
    return p


def run_attention(kv, p, lengths, q, weights=None, scale=None, counts=None, **more):
    lengths = torch.from_numpy(np.ascontiguousarray(lengths, np.int32)).cuda()
    w = None if weights is None else torch.from_numpy(weights).cuda()
    c = None if counts is None else torch.from_numpy(np.asarray(counts, np.int32)).cuda()
    out, wo = kv.ibp_kv_attention(p.cache, p.gpu_pages, lengths, q.cuda(), scale=scale, weights=w, counts=c, **more)
    torch.cuda.synchronize()
    return out.cpu(), None if wo is None else np_of(wo)


def expect(p, lengths, q, weights=None, scale=None, counts=None):
    fi = torch.finfo(q.dtype)
    return orc.attention(p.k, p.v, p.pt, p.pages, np.asarray(lengths, np.int32), q.double().numpy(),
                         p.d ** -0.5 if scale is None else scale, weights, counts,
                         rounding=fi.eps / 2, tiny=fi.tiny * fi.eps / 2)


def close(out, w, want):
    o, wt, oe, we = want
    got = out.double().numpy()
    nan = np.isnan(o)
    assert np.array_equal(np.isnan(got), nan)
    off = np.where(nan, 0.0, np.abs(got - o) / np.where(nan, 1.0, oe))
    assert off.max(initial=0.0) <= 1.0, (off.max(), np.argwhere(off > 1)[:4])
    if w is not None:
        nan = np.isnan(wt)
        assert np.array_equal(np.isnan(w), nan)
        off = np.where(nan, 0.0, np.abs(w - wt) / np.where(nan, 1.0, we))
        assert off.max(initial=0.0) <= 1.0, (off.max(), np.argwhere(off > 1)[:4])


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("pt", [16, 32, 64])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group,new", [(1, 1), (3, 1), (8, 2), (5, 7), (16, 6)])
def test_attention(kv, d, pt, dtype, group, new):
    """Lengths about the edges of tiles, steps and splits, none and one among
    them; query rows from one to more than a unit holds."""
    seqs, heads = 5, 2
    lens = [0, 1, 15 + new, 64 + pt, 257]
    p = filled(kv, seqs, heads, -(-300 // pt), pt, d, lens, seed=d + pt)
    q = torch.randn(seqs, new, heads * group, d, generator=torch.Generator().manual_seed(new)).to(DTYPES[dtype])
    w = np.random.default_rng(3).random((seqs, heads, p.pages.shape[2]), dtype=np.float32)
    lengths = grid(seqs, heads, lens)
    out, wo = run_attention(kv, p, lengths, q, w)
    close(out, wo, expect(p, lengths, q, w))
    out2, none = run_attention(kv, p, lengths, q)
    assert none is None and torch.equal(out2, out)


@pytest.mark.parametrize("n", [1, 2, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000])
def test_attention_one_row_lengths(kv, n):
    p = filled(kv, 1, 1, 64, 16, 128, [n], seed=n)
    q = torch.randn(1, 1, 4, 128, generator=torch.Generator().manual_seed(n)).bfloat16()
    w = np.zeros((1, 1, 64), np.float32)
    out, wo = run_attention(kv, p, [[n]], q, w)
    close(out, wo, expect(p, [[n]], q, w))
    assert abs(wo.sum() - 4) < 1e-4 and not wo[0, 0, -(-n // 16):].any()


def test_attention_many_splits(kv):
    """One row of 40,000 tokens: the workgroups share it."""
    n, d, pt = 40003, 64, 64
    p = filled(kv, 1, 1, 640, pt, d, [n], seed=4)
    q = torch.randn(1, 2, 3, d, generator=torch.Generator().manual_seed(1)).half()
    w = np.zeros((1, 1, 640), np.float32)
    out, wo = run_attention(kv, p, [[n]], q, w)
    close(out, wo, expect(p, [[n]], q, w))


@pytest.mark.parametrize("group,new", [(16, 1), (16, 5)])
def test_attention_many_rows(kv, group, new):
    """More rows than the chip holds workgroups at once, so that none is cut,
    over tables with room for long rows; with 80 query rows a head, units of
    one head meet in the joining kernel."""
    seqs, heads, pt, d, m = 40, 8, 64, 64, 70
    lens = [(17 * i) % 101 for i in range(seqs)]
    lens[3] = 700
    p = Pages(kv, seqs, heads, m, pt, d, n_pages=seqs * heads * m)
    rng = np.random.default_rng(1)
    for pool in (p.k, p.v):
        pool[0][:] = rng.integers(0, 0x58, pool[0].shape, dtype=np.uint8) | (rng.integers(0, 2, pool[0].shape, dtype=np.uint8) << 7)
        pool[1][:] = 2.0 ** rng.integers(-3, 2, pool[1].shape)
    p.upload()
    q = torch.randn(seqs, new, heads * group, d, generator=torch.Generator().manual_seed(new)).bfloat16()
    w = rng.random((seqs, heads, m), dtype=np.float32)
    lengths = grid(seqs, heads, lens)
    out, wo = run_attention(kv, p, lengths, q, w)
    close(out, wo, expect(p, lengths, q, w))


def test_attention_large_scores(kv):
    """Scores of some hundreds: the statistics must be those of the whole row."""
    p = filled(kv, 2, 2, 40, 16, 128, [600, 500], seed=8, amp=30.0)
    q = torch.randn(2, 1, 4, 128, generator=torch.Generator().manual_seed(1)).bfloat16()
    w = np.zeros((2, 2, 40), np.float32)
    lengths = grid(2, 2, [600, 500])
    for scale in (None, 0.0, -0.3):
        out, wo = run_attention(kv, p, lengths, q, w, scale=scale)
        close(out, wo, expect(p, lengths, q, w, scale=scale))


def test_attention_holes_and_counts(kv):
    """Holes inside rows, rows of holes only, counts below n_new, lengths
    below the count and outside the table."""
    seqs, heads, pt, d, m, new = 6, 2, 16, 64, 12, 5
    lens = [150, 90, 3, 192, 40, 77]
    p = filled(kv, seqs, heads, m, pt, d, lens, seed=2)
    p.pages[0, 0, [0, 3, 9]], p.pages[0, 1, 4:8], p.pages[1] = -1, p.n_pages + 5, -1
    p.upload()
    lengths = grid(seqs, heads, [150, 90, 3, 5000, -4, 77])
    q = torch.randn(seqs, new, heads * 3, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    w = np.random.default_rng(1).random((seqs, heads, m), dtype=np.float32)
    for counts in (None, [5, 5, 5, 2, 5, 0], [1, 9, 4, 0, -1, 3]):
        out, wo = run_attention(kv, p, lengths, q, w, counts=counts)
        close(out, wo, expect(p, lengths, q, w, counts=counts))
        assert not out[1].any()
    assert np.array_equal(wo[1], w[1]) and np.array_equal(wo[4], w[4])


def test_attention_nan_stays_with_those_who_see_it(kv):
    """A NaN value at a position reaches the queries that see it, at its dim,
    and no earlier one; a NaN key makes its queries NaN whole."""
    pt, d, n, new = 16, 128, 100, 6
    for what in ("v", "k"):
        p = filled(kv, 1, 1, 8, pt, d, [n], seed=6)
        pool, place = (p.v, orc.v_place(pt, d)) if what == "v" else (p.k, orc.k_place(pt, d))
        for pos, dim in ((n - 1, 3), (n - 3, 77), (n - 3, 16)):
            pool[0][p.pages[0, 0, pos // pt], place[pos % pt, dim]] = 0xFF
        p.upload()
        q = torch.randn(1, new, 2, d, generator=torch.Generator().manual_seed(1)).half()
        w = np.zeros((1, 1, 8), np.float32)
        out, wo = run_attention(kv, p, [[n]], q, w if what == "v" else None)
        nan = np.isnan(out.numpy())[0]
        assert not nan[:new - 3].any()
        if what == "v":
            close(out, wo, expect(p, [[n]], q, w))
            assert nan[new - 3:, :, [16, 77]].all() and nan[new - 1:, :, 3].all() and nan.sum() == 2 * (3 * 2 + 1)
        else:
            assert nan[new - 3:].all()
            clean, _, err, _ = expect(p, [[n - 3]], q[:, :new - 3])
            assert (np.abs(out[:, :new - 3].double().numpy() - clean) <= err).all()


def test_attention_queries_not_finite(kv):
    p = filled(kv, 1, 2, 20, 16, 64, [300], seed=1)
    q = torch.randn(1, 1, 8, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    q[0, 0, 1, 5], q[0, 0, 6, 0] = float("inf"), float("nan")
    out, _ = run_attention(kv, p, grid(1, 2, [300]), q)
    nan = np.isnan(out[0, 0].float().numpy())
    assert nan[[1, 6]].all() and not nan[[0, 2, 3, 4, 5, 7]].any()


def test_attention_strides_and_buffers(kv):
    """Queries and outputs of any strides, one workspace for two calls,
    weights in place, another stream."""
    seqs, new, heads, group, d, pt = 3, 2, 2, 4, 128, 32
    lens = [70, 200, 513]
    p = filled(kv, seqs, heads, 20, pt, d, lens, seed=3)
    lengths = grid(seqs, heads, lens)
    q = torch.randn(seqs, new, heads * group, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    w = np.random.default_rng(1).random((seqs, heads, 20), dtype=np.float32)
    out, wo = run_attention(kv, p, lengths, q, w)
    close(out, wo, expect(p, lengths, q, w))
    gl = torch.from_numpy(lengths).cuda()
    n = kv.ibp_kv_attention_workspace_bytes(p.cache, p.gpu_pages, gl, heads * group, new, True)
    assert n > 0
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    odd_q = torch.empty(seqs, new, heads * group, d + 1, dtype=torch.bfloat16, device="cuda")[..., 1:].copy_(q)
    odd_out = torch.zeros(seqs, heads * group, new, d + 5, dtype=torch.bfloat16, device="cuda")[..., 3:3 + d].transpose(1, 2)
    gw = torch.from_numpy(w).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, gw_out = kv.ibp_kv_attention(p.cache, p.gpu_pages, gl, odd_q, weights=gw, weights_out=gw, out=odd_out, workspace=ws[:n])
    s.synchronize()
    assert got is odd_out and gw_out is gw
    assert torch.equal(got.cpu(), out) and np.array_equal(np_of(gw), wo)
    assert (ws[n:] == 0xFF).all()
    assert not odd_out._base[..., :3].any() and not odd_out._base[..., 3 + d:].any()
    again, _ = kv.ibp_kv_attention(p.cache, p.gpu_pages, gl, q.cuda(), workspace=ws[:n])
    assert torch.equal(again.cpu(), out)
    with pytest.raises(kv.IBPKVError, match="invalid argument"):
        kv.ibp_kv_attention(p.cache, p.gpu_pages, gl, q.cuda(), weights=gw, workspace=ws[:n - 64])
    torch.cuda.synchronize()


def test_calls_on_a_given_stream(kv):
    """stream=: appended, attended and evicted on a stream that waits behind
    other work, with everything the calls allocate on it; the current stream
    has its own memory in use meanwhile."""
    seqs, heads, d, pt, m = 2, 2, 128, 16, 40
    p = filled(kv, seqs, heads, m, pt, d, [500, 333], seed=3)
    lengths = grid(seqs, heads, [501, 334])
    k, v = values(1, (seqs, 1, heads, d), torch.bfloat16), values(2, (seqs, 1, heads, d), torch.bfloat16)
    q = torch.randn(seqs, 1, heads * 3, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    w = np.random.default_rng(1).random((seqs, heads, m), dtype=np.float32)
    gl, gk, gv, gq, gw = torch.from_numpy(lengths).cuda(), k.cuda(), v.cuda(), q.cuda(), torch.from_numpy(w).cuda()
    for (codes, scales), x, place in ((p.k, k, orc.k_place), (p.v, v, orc.v_place)):
        orc.append(codes, scales, place(pt, d), pt, p.pages, lengths, x.double().numpy())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        busy = torch.randn(4096, 4096, device="cuda")
        for _ in range(10):
            busy = busy @ busy * 1e-2
    kv.ibp_kv_append(p.cache, p.gpu_pages, gl, gk, gv, stream=s)
    out, wo = kv.ibp_kv_attention(p.cache, p.gpu_pages, gl, gq, weights=gw, stream=s)
    pages, weights, left = kv.ibp_kv_evict(p.gpu_pages, wo, gl, pt, keep_pages=9, recent_pages=2, stream=s)
    for _ in range(20):  # the current stream's own allocations
        torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda")
    s.synchronize()
    p.check()
    close(out.cpu(), np_of(wo), expect(p, lengths, q, w))
    same_eviction([np_of(pages), np_of(weights), np_of(left)],
                  orc.evict(p.pages, np_of(wo), lengths, pt, 9, 1, 2))


def test_pool_without_pages(kv):
    """Every id is a hole: zeros, and the weights as they were."""
    none = [torch.empty(0, dtype=torch.uint8, device="cuda"), torch.empty(0, device="cuda")]
    cache = kv.ibp_kv_cache(*none, *none, 16, 64)
    pages = torch.zeros(2, 3, 200, dtype=torch.int32, device="cuda")
    lengths = torch.full((2, 3), 3000, dtype=torch.int32, device="cuda")
    x = torch.ones(2, 1, 3, 64, dtype=torch.float16, device="cuda")
    kv.ibp_kv_append(cache, pages, lengths, x, x)
    w = torch.rand(2, 3, 200, device="cuda")
    out, wo = kv.ibp_kv_attention(cache, pages, lengths, x.repeat(1, 1, 2, 1), weights=w)
    assert not out.any() and torch.equal(wo, w)


def test_attention_without_queries(kv):
    """No new tokens: nothing to write but the weights."""
    p = filled(kv, 1, 2, 10, 16, 64, [100], seed=1)
    w = torch.rand(1, 2, 10, device="cuda")
    out, wo = kv.ibp_kv_attention(p.cache, p.gpu_pages, torch.full((1, 2), 100, dtype=torch.int32, device="cuda"),
                                  torch.zeros(1, 0, 4, 64, dtype=torch.bfloat16, device="cuda"), weights=w)
    assert out.shape == (1, 0, 4, 64) and torch.equal(wo, w)
    none = torch.zeros(0, 2, 10, dtype=torch.int32, device="cuda")
    out, wo = kv.ibp_kv_attention(p.cache, none, none[..., 0].contiguous(),
                                  torch.zeros(0, 1, 4, 64, dtype=torch.bfloat16, device="cuda"), weights=w[:0])
    assert out.numel() == 0 and wo.numel() == 0


def test_pages_shared_by_rows(kv):
    """A common prompt: two sequences name the same pages."""
    p = filled(kv, 2, 1, 10, 16, 64, [160, 160], seed=5)
    p.pages[1, 0, :6] = p.pages[0, 0, :6]
    p.upload()
    q = torch.randn(2, 1, 2, 64, generator=torch.Generator().manual_seed(1)).half()
    lengths = grid(2, 1, [130, 150])
    w = np.zeros((2, 1, 10), np.float32)
    out, wo = run_attention(kv, p, lengths, q, w)
    close(out, wo, expect(p, lengths, q, w))


def test_pool_past_32_bits(kv):
    """Pages whose bytes lie past 4 GiB."""
    pt, d, n_pages = 64, 256, (1 << 32) // (64 * 256) + 40
    codes = [torch.zeros(n_pages, pt * d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones(n_pages, device="cuda") for _ in range(2)]
    cache = kv.ibp_kv_cache(codes[0], scales[0], codes[1], scales[1], pt, d)
    pages = torch.tensor([[[n_pages - 1, 3, n_pages - 30]]], dtype=torch.int32, device="cuda")
    n = 170
    k, v = values(1, (1, n, 1, d), torch.bfloat16), values(2, (1, n, 1, d), torch.bfloat16)
    lengths = torch.tensor([[n]], dtype=torch.int32, device="cuda")
    kv.ibp_kv_append(cache, pages, lengths, k.cuda(), v.cuda())
    q = torch.randn(1, 1, 2, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    out, _ = kv.ibp_kv_attention(cache, pages, lengths, q.cuda())
    p = Pages(kv, 1, 1, 3, pt, d, n_pages=3)
    p.append([[n]], k, v)
    close(out.cpu(), None, expect(p, [[n]], q))
    ids = pages[0, 0].long().cpu()
    for i, page in enumerate(ids):
        assert np.array_equal(np_of(codes[0][page]), p.k[0][p.pages[0, 0, i]])
        assert np.array_equal(np_of(codes[1][page]), p.v[0][p.pages[0, 0, i]])
    assert int((codes[0] != 0).any(1).sum()) == 3


# ------------------------------------------------------------ eviction ----


def run_evict(kv, pages, weights, lengths, pt, keep, sink, recent):
    got = kv.ibp_kv_evict(*(torch.from_numpy(x).cuda() for x in (pages, weights, lengths)), pt,
                          keep_pages=keep, sink_pages=sink, recent_pages=recent)
    torch.cuda.synchronize()
    return [np_of(x) for x in got]


def same_eviction(got, want):
    for x, y, name in zip(got, want, ("pages", "weights", "lengths")):
        assert np.array_equal(x, y, equal_nan=name == "weights"), name


@pytest.mark.parametrize("m,keep,sink,recent", [(1, 1, 0, 1), (2, 1, 0, 1), (9, 5, 1, 1), (64, 64, 2, 2),
                                                (65, 3, 1, 2), (255, 17, 0, 1), (256, 128, 4, 8), (257, 256, 1, 1),
                                                (1000, 5, 0, 4), (1500, 700, 3, 40)])
def test_evict(kv, m, keep, sink, recent):
    """Rows of every length, weights with many equal ones."""
    rng = np.random.default_rng(m)
    seqs, heads, pt = 4, 3, 16
    pages = rng.permutation(seqs * heads * m).reshape(seqs, heads, m).astype(np.int32)
    weights = (rng.integers(0, 6, pages.shape) * rng.choice([0.25, 1.0, 1e-30, 1e30], pages.shape)).astype(np.float32)
    lengths = rng.integers(0, m * pt + 1, (seqs, heads)).astype(np.int32)
    lengths[0] = [m * pt, 0, 1]
    lengths[1, 0], lengths[1, 1] = m * pt + 100, -3
    lengths[2, 0] = min(m, keep) * pt
    lengths[2, 1] = min(m, keep + 1) * pt - pt + 1
    same_eviction(run_evict(kv, pages, weights, lengths, pt, keep, sink, recent),
                  orc.evict(pages, weights, lengths, pt, keep, sink, recent))


def test_evict_weights_of_every_kind(kv):
    """Infinities, NaN, both zeros, subnormals, negative weights; all equal;
    ties that end at the budget."""
    rng = np.random.default_rng(0)
    kinds = np.array([np.inf, -np.inf, np.nan, 0.0, -0.0, 1e-45, -1e-45, 1.0, -1.0, 1.0000001, 3.4e38], np.float32)
    pages = rng.permutation(8 * 300).reshape(8, 1, 300).astype(np.int32)
    weights = rng.choice(kinds, pages.shape)
    weights[1] = 1.0
    weights[2] = np.nan
    weights[3] = np.where(rng.random(300) < 0.5, 0.0, -0.0)
    weights[4, 0] = np.linspace(0, 1, 300)
    weights[5, 0] = np.linspace(1, 0, 300)
    lengths = np.full((8, 1), 300 * 32, np.int32)
    for keep in (2, 57, 150, 298, 299):
        same_eviction(run_evict(kv, pages, weights, lengths, 32, keep, 1, 1),
                      orc.evict(pages, weights, lengths, 32, keep, 1, 1))


def test_evict_long_rows(kv):
    rng = np.random.default_rng(2)
    m = 40001
    pages = rng.permutation(2 * m).reshape(2, 1, m).astype(np.int32)
    weights = np.round(np.exp(2 * rng.standard_normal(pages.shape)) * 8).astype(np.float32) / 8
    lengths = np.array([[m * 64 - 5], [(m - 7) * 64]], np.int32)
    for keep in (9, 20000, 39999):
        same_eviction(run_evict(kv, pages, weights, lengths, 64, keep, 2, 3),
                      orc.evict(pages, weights, lengths, 64, keep, 2, 3))


# ------------------------------------------------------------ together ----


def test_equal_inputs_give_equal_bytes(kv):
    p = filled(kv, 3, 2, 100, 16, 128, [1600, 900, 77], seed=3)
    lengths = grid(3, 2, [1600, 900, 77])
    q = torch.randn(3, 1, 8, 128, generator=torch.Generator().manual_seed(1)).bfloat16()
    w = np.random.default_rng(1).random((3, 2, 100), dtype=np.float32)
    first = run_attention(kv, p, lengths, q, w)
    for _ in range(3):
        out, wo = run_attention(kv, p, lengths, q, w)
        assert torch.equal(out, first[0]) and np.array_equal(wo, first[1])


def test_graph_of_a_decoding_step(kv):
    """A step captured once and replayed: lengths advance on the GPU, the new
    token is appended and attended, the rows are cut to a budget.  Every
    replay is checked against eager calls on a copy."""
    seqs, heads, group, d, pt, m = 2, 2, 3, 64, 16, 12
    p = filled(kv, seqs, heads, m, pt, d, [100, 61], seed=3)
    dev = torch.device("cuda")
    k, v, q = (torch.zeros(seqs, 1, h, d, dtype=torch.bfloat16, device=dev) for h in (heads, heads, heads * group))

    def fresh():
        t = [x.clone() for x in p.t]
        return {"t": t, "cache": kv.ibp_kv_cache(*t, pt, d), "pages": p.gpu_pages.clone(),
                "lengths": torch.from_numpy(grid(seqs, heads, [100, 61])).cuda(),
                "weights": torch.rand(seqs, heads, m, device=dev, generator=torch.Generator(dev).manual_seed(4))}

    def step(s):
        s["lengths"].add_(1)
        kv.ibp_kv_append(s["cache"], s["pages"], s["lengths"], k, v)
        s["out"], w = kv.ibp_kv_attention(s["cache"], s["pages"], s["lengths"], q, weights=s["weights"])
        pages, weights, lengths = kv.ibp_kv_evict(s["pages"], w, s["lengths"], pt, keep_pages=6, sink_pages=1, recent_pages=2)
        for name, x in (("pages", pages), ("weights", weights), ("lengths", lengths)):
            s[name].copy_(x)

    eager, other = fresh(), fresh()
    warm = fresh()
    step(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(other)
    for i in range(40):
        for x, seed in ((k, 1), (v, 2), (q, 3)):
            x.copy_(values(100 * i + seed, tuple(x.shape), torch.bfloat16, 1.0 + i % 5))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        step(eager)
        torch.cuda.synchronize()
        assert torch.equal(other["out"], eager["out"]), i
        for name in ("pages", "lengths", "weights"):
            assert torch.equal(other[name], eager[name]), (i, name)
        for x, y in zip(other["t"], eager["t"]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), i
    assert int(eager["lengths"].max()) <= 6 * pt


def test_example_runs_them_together(kv):
    """The example with small sizes: what evicted pages held comes back from
    the archive bit for bit (asserted inside), rows end within the budget."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "kv_decode.py")
    spec = importlib.util.spec_from_file_location("kv_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    out, lengths, weights = example.main(seqs=2, heads=3, group=2, prompt=320, steps=20, keep=12, quiet=True)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and int(lengths.max()) <= 12 * 16
    # weights of pages that are not held are 0
    held = -(-lengths.long() // 16)
    assert not weights[torch.arange(weights.shape[2], device="cuda") >= held[..., None]].any()


# ------------------------------------------------------------- autograd ----


def test_going_backward_through_a_result_raises(kv):
    """No call has a gradient: a result of inputs that require one says so when
    it is asked for, instead of counting as a constant."""
    p = filled(kv, 1, 2, 10, 16, 64, [100], seed=1)
    lengths = torch.full((1, 2), 100, dtype=torch.int32, device="cuda")
    q = torch.randn(1, 1, 4, 64, device="cuda").bfloat16().requires_grad_()
    w = torch.rand(1, 2, 10, device="cuda")
    plain, plain_w = kv.ibp_kv_attention(p.cache, p.gpu_pages, lengths, q.detach(), weights=w)
    assert not plain.requires_grad and not plain_w.requires_grad
    out, wo = kv.ibp_kv_attention(p.cache, p.gpu_pages, lengths, q * 1, weights=w)
    assert torch.equal(out.detach(), plain) and torch.equal(wo.detach(), plain_w)
    for x in (out, wo):
        with pytest.raises(RuntimeError, match="ibp_kv_attention is not implemented"):
            x.float().sum().backward()
    assert q.grad is None
    with torch.no_grad():
        out, wo = kv.ibp_kv_attention(p.cache, p.gpu_pages, lengths, q, weights=w, weights_out=w.clone())
    assert not out.requires_grad and torch.equal(out, plain) and torch.equal(wo, plain_w)
    pages, left, _ = kv.ibp_kv_evict(p.gpu_pages, w.clone().requires_grad_(), lengths, 16, 3)
    assert not pages.requires_grad
    with pytest.raises(RuntimeError, match="ibp_kv_evict is not implemented"):
        left.sum().backward()
    # codes are whole numbers: they have no gradient, as torch's own casts to such
    k = torch.randn(1, 1, 2, 64, device="cuda").bfloat16().requires_grad_()
    kv.ibp_kv_append(p.cache, p.gpu_pages, lengths, k, k)
    assert not any(t.requires_grad for t in p.t)


def test_given_outputs_without_a_gradient(kv):
    """As torch's functions with out=."""
    p = filled(kv, 1, 2, 10, 16, 64, [100], seed=1)
    lengths = torch.full((1, 2), 100, dtype=torch.int32, device="cuda")
    q, w = torch.randn(1, 1, 4, 64, device="cuda").bfloat16(), torch.rand(1, 2, 10, device="cuda")
    for bad in (dict(q=q.clone().requires_grad_(), out=q.clone()), dict(q=q, out=q.clone().requires_grad_()),
                dict(q=q, weights=w.clone().requires_grad_(), weights_out=w.clone()),
                dict(q=q.clone().requires_grad_(), weights=w, weights_out=w)):
        with pytest.raises(ValueError, match="requires a gradient"):
            kv.ibp_kv_attention(p.cache, p.gpu_pages, lengths, bad.pop("q"), **bad)
    with pytest.raises(ValueError, match="requires a gradient"):
        kv.ibp_kv_evict(p.gpu_pages, w.clone().requires_grad_(), lengths, 16, 3, weights_out=w.clone())


def test_written_tensors_have_a_new_version(kv):
    """What a call writes in place counts as changed, so that autograd notices
    where it had been saved."""
    p = filled(kv, 1, 2, 10, 16, 64, [100], seed=1)
    lengths = torch.full((1, 2), 100, dtype=torch.int32, device="cuda")
    q, w = torch.randn(1, 1, 4, 64, device="cuda").bfloat16(), torch.rand(1, 2, 10, device="cuda")
    k = torch.randn(1, 1, 2, 64, device="cuda").bfloat16()
    out, wo = torch.empty_like(q), w.clone()
    given = [torch.empty_like(x) for x in (p.gpu_pages, w, lengths)]

    def versions(*tensors):
        return [t._version for t in tensors]
    before = versions(*p.t, out, wo, *given)
    kv.ibp_kv_append(p.cache, p.gpu_pages, lengths, k, k)
    kv.ibp_kv_attention(p.cache, p.gpu_pages, lengths, q, weights=w, weights_out=wo, out=out)
    kv.ibp_kv_evict(p.gpu_pages, w, lengths, 16, 3, pages_out=given[0], weights_out=given[1], lengths_out=given[2])
    assert all(x > y for x, y in zip(versions(*p.t, out, wo, *given), before))
    only_read = (p.gpu_pages, lengths, q, w, k)
    assert versions(*only_read) == [0] * len(only_read)
    x = torch.rand(1, 2, 10, device="cuda", requires_grad=True)
    y = (x * wo).sum()                        # wo saved for the backward pass
    kv.ibp_kv_attention(p.cache, p.gpu_pages, lengths, q, weights=w, weights_out=wo)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():              # tensors that have no version
        a, b = kv.ibp_kv_attention(p.cache, p.gpu_pages, lengths, q, weights=w)
        kv.ibp_kv_attention(p.cache, p.gpu_pages, lengths, q, weights=b, weights_out=b, out=a)
    kv.ibp_kv_attention(p.cache, p.gpu_pages, lengths, q, weights=b, weights_out=b, out=a)


# --------------------------------------------------------- scales that are not finite ----


@pytest.mark.parametrize("d,group", [(64, 2), (128, 4), (256, 5)])
@pytest.mark.parametrize("scale", [float("nan"), float("inf")])
def test_attention_scale_not_finite_stays_with_those_who_see_it(kv, d, group, scale):
    """A page whose scale is not finite (no append writes one) reaches the
    queries that see a token of it and no earlier one; a page that no query
    sees reaches none."""
    pt, n, new = 16, 101, 7                       # the page from 96 on: seen by the last five
    p = filled(kv, 1, 1, 9, pt, d, [n], seed=6)
    for pool in (p.k, p.v):
        pool[1][p.pages[0, 0, 7:]] = scale        # past the row's end
    p.v[1][p.pages[0, 0, 6]] = scale
    p.upload()
    q = torch.randn(1, new, group, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    w = np.zeros((1, 1, 9), np.float32)
    out, wo = run_attention(kv, p, [[n]], q, w)
    assert out[:, 2:].isnan().all()
    p.v[1][p.pages[0, 0, 6]] = 1.0
    want = expect(p, [[n]], q, w)
    close(out[:, :2], None, (want[0][:, :2], None, want[2][:, :2], None))
    close(out[:, :0], wo, (want[0][:, :0], want[1], want[2][:, :0], want[3]))


# ------------------------------------------------------------- the example ----


def test_example_fetches_back_every_page_given_up(kv, monkeypatch):
    """What the example asks of its archive at the end, against a record of its
    calls: every page of the prompt that some head gave up, though the places of
    such pages were filled again, and given up again, meanwhile."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "kv_decode.py")
    spec = importlib.util.spec_from_file_location("kv_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    seqs, heads, prompt, pt = 2, 3, 320, example.PAGE
    asked, filled_from, gone, again = [], {}, set(), 0
    append, evict, restore = kv.ibp_kv_append, kv.ibp_kv_evict, example.restore

    def recorded_append(cache, pages, lengths, k, v, **more):
        ids, ends = np_of(pages), np_of(lengths)
        for s, h in np.ndindex(ends.shape):
            first = int(ends[s, h]) - k.shape[1]
            for at in range(-(-first // pt), -(-int(ends[s, h]) // pt)):   # pages that these tokens begin
                row = (s * heads + h) * (prompt // pt) + at if k.shape[1] == prompt else None
                filled_from[int(ids[s, h, at])] = row
        return append(cache, pages, lengths, k, v, **more)

    def recorded_evict(pages, weights, lengths, *args, **more):
        nonlocal again
        out = evict(pages, weights, lengths, *args, **more)
        ids, was, now = np_of(out[0]), np_of(lengths), np_of(out[2])
        for s, h in np.ndindex(was.shape):
            for page in ids[s, h, -(-int(now[s, h]) // pt):-(-int(was[s, h]) // pt)]:
                row = filled_from.pop(int(page))
                again += row is None
                gone.update([] if row is None else [row])
        return out

    def recorded_restore(arch, ids, d):
        asked.append(ids.tolist())
        return restore(arch, ids, d)
    monkeypatch.setattr(example.ibp_kv, "ibp_kv_append", recorded_append)
    monkeypatch.setattr(example.ibp_kv, "ibp_kv_evict", recorded_evict)
    monkeypatch.setattr(example, "restore", recorded_restore)
    example.main(seqs=seqs, heads=heads, group=2, prompt=prompt, steps=150, keep=7, quiet=True)
    assert again and len(gone) > seqs * heads * (prompt // pt - 7)
    assert len(asked) == 4 and asked[2] == asked[3]
    assert sorted(asked[2]) == sorted(gone)

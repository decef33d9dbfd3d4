"""Attention over a shared prefix whose pages' scales are of every kind, against
the 64-bit oracle and its bounds (oracle/kv_long_oracle.py): the paths of up to
32 query rows to a head and of more, held to what each of them promises."""
import numpy as np
import pytest

from oracle import kv_long_oracle as lorc
from oracle import kv_oracle as orc
from test_gpu_kv import close, grid, kv  # noqa: F401
from test_gpu_kv_long import check_shared, gpu, shared_pool
from test_gpu_kv_paths import queries

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("seqs", [3, 40])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_scales_that_are_no_powers_of_two(kv, d, seqs, dtype):
    """Value scales of 2^64 and more next to small ones: outputs are finite in bf16,
    and in fp16 infinite where the number is past its largest."""
    p = shared_pool(kv, seqs, 2, 40, 6, 16, d, seed=d)
    rng = np.random.default_rng(7)
    p.v[1] = rng.choice(np.array([1, 0.75, 1.5 * 2.0 ** 70, -1.25 * 2.0 ** 64, 1.9 * 2.0 ** 100, 2.0 ** 90, 2.0 ** -30], np.float32), p.n_pages)
    p.upload()
    q = queries(2, seqs, 1, 6, d, dtype)
    out = check_shared(kv, p, [640, 333], grid(seqs, 2, [(i * 7) % 90 + 1 for i in range(seqs)]), q, scale=0.02)
    assert not out.isnan().any()
    if dtype == "bf16":
        assert not out.isinf().any()


def led_pool(kv, seqs, heads, d, pt=16, seed=0):
    """Keys of small numbers with dim 0 zero, but for one token of the prefix, whose
    dim 0 is 240; the page that it is in."""
    p = shared_pool(kv, seqs, heads, 40, 16, pt, d, seed=seed)
    rng = np.random.default_rng(seed)
    p.prefix = rng.permutation(p.n_pages)[:heads * 40].reshape(heads, 40).astype(np.int32)
    p.k[0][:] = rng.integers(0x20, 0x30, p.k[0].shape) | (rng.integers(0, 2, p.k[0].shape) << 7)
    place, page = orc.k_place(pt, d), p.prefix[:, 3]
    p.k[0][:, place[:, 0]] = 0
    p.k[0][page, place[5, 0]] = 0x77
    p.k[1][:] = p.v[1][:] = 1
    return p, page


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("seqs", [3, 40])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -126])
@pytest.mark.parametrize("lead", [22, 26, 30, 60])
def test_page_of_zeros_that_leads_by_its_score(kv, lead, scale, seqs, dtype):
    """The heaviest token, by 2^lead, is in a page whose values are zeros, as those of
    an appended page of zeros are: the output is what the others give."""
    p, page = led_pool(kv, seqs, 2, 128, seed=lead)
    p.v[1][page] = scale
    p.upload()
    q = queries(2, seqs, 1, 6, 128, dtype)
    q[..., 0] = 8.0
    lengths = grid(seqs, 2, [(i * 7) % 90 + 1 for i in range(seqs)])
    check_shared(kv, p, [640, 333], lengths, q, scale=lead * np.log(2) / (8 * 240))


def check_promise(kv, p, prefix_lengths, lengths, q, scale, far=False):
    """Within what the header promises: 16 bits of each weight, or with more than 32
    query rows and outputs of bf16 11 of the prefix's, no less than 2^-24 of the
    largest.  `far`: scales that 16 bits are promised for in any case.  Rounding of
    outputs, scores and sums as in check_shared."""
    rows = q.shape[0] * q.shape[1] * q.shape[2] // p.pages.shape[1]
    less = q.dtype == torch.bfloat16 and rows > 32 and not far
    prefix_lengths = np.asarray(prefix_lengths, np.int32)
    out = kv.ibp_kv_attention_shared(p.cache, gpu(p.prefix), gpu(prefix_lengths), p.gpu_pages, gpu(lengths), q.cuda(), scale=scale)
    torch.cuda.synchronize()
    fi = torch.finfo(q.dtype)
    o, err = lorc.attention_shared(p.k, p.v, p.pt, p.prefix, prefix_lengths, p.pages, lengths, q.double().numpy(), scale,
                                   rounding=fi.eps / 2, tiny=fi.tiny * fi.eps / 2, weight=2.0 ** (-11 if less else -16),
                                   own_weight=2.0 ** -16, floor=0.0, least=2.0 ** -24 if less else 0.0)
    close(out.cpu(), None, (o, None, err, None))
    return out


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("seqs", [3, 40])
@pytest.mark.parametrize("apart", [9, 20, 40, 70])
def test_pages_far_below_the_largest_scale(kv, apart, seqs, dtype):
    """Half of the dims are zeros in the pages of the largest scale, so that the output
    there is what the pages far below it give, under scores that are about equal."""
    p = shared_pool(kv, seqs, 2, 40, 6, 16, 128, seed=apart)
    rng = np.random.default_rng(apart)
    p.k[1][:] = 2.0 ** -8
    p.v[1] = rng.choice(np.array([1.0, 2.0 ** -apart], np.float32), p.n_pages)
    low = orc.v_place(16, 128)[:, :64].reshape(-1)
    p.v[0][np.ix_(p.v[1] == 1.0, low)] = 0
    p.upload()
    q = queries(1, seqs, 1, 6, 128, dtype)
    out = check_promise(kv, p, [640, 333], grid(seqs, 2, [(i * 7) % 90 + 1 for i in range(seqs)]), q, 0.02, far=True)
    if dtype == "bf16":
        assert (out[..., :64] != 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("seqs", [3, 40])
@pytest.mark.parametrize("lead", [12, 26, 40])
def test_token_of_zeros_that_leads_by_its_score(kv, lead, seqs, dtype):
    """The heaviest token, by 2^lead, has values of 0 in a page like the others: outputs
    of fp16 keep 16 bits of the other weights, those of bf16 up to 2^-24 of the largest."""
    p, page = led_pool(kv, seqs, 2, 64, seed=lead)
    p.v[1][:] = 2.0 ** (lead // 2)
    p.v[0][np.ix_(page, orc.v_place(16, 64)[5])] = 0
    p.upload()
    q = queries(3, seqs, 1, 6, 64, dtype)
    q[..., 0] = 8.0
    check_promise(kv, p, [640, 333], grid(seqs, 2, [(i * 7) % 90 + 1 for i in range(seqs)]), q, lead * np.log(2) / (8 * 240))


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("seqs,group,new", [(1, 1, 1), (5, 3, 1), (32, 1, 1), (8, 4, 1), (33, 1, 1), (4, 5, 7), (16, 8, 1)])
@pytest.mark.parametrize("odd", [False, True])
def test_each_path_keeps_what_it_promises(kv, odd, seqs, group, new, dtype, d):
    """1 to 140 query rows to a head: 16 bits of the weights of own tokens, and of the
    prefix's up to 32 rows, for outputs of fp16, and with scales that are no powers of
    two (`odd`); holes in the prefix, which ends inside a page."""
    p = shared_pool(kv, seqs, 2, 30, 8, 32, d, seed=d + seqs)
    if odd:
        p.v[1] *= np.float32(0.75)
    p.prefix[0, [2, 11]], p.prefix[1, 5] = -1, p.n_pages
    p.upload()
    q = queries(seqs, seqs, new, 2 * group, d, dtype)
    check_promise(kv, p, [900, 417], grid(seqs, 2, [(i * 37) % 240 + new for i in range(seqs)]), q, 0.02, far=odd)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_some_parts_with_far_scales(kv, d):
    """A long prefix in many parts, of which one has scales far apart and one is all
    holes: their statistics join with those of the others; a head has other scales."""
    p = shared_pool(kv, 41, 2, 700, 10, 16, d, seed=d)
    p.prefix = np.random.default_rng(1).permutation(p.n_pages)[:700].astype(np.int32)[None].repeat(2, 0)
    p.prefix[1] = p.prefix[1][::-1]
    p.v[1][p.prefix[0, 100:110]] *= np.float32(2.0 ** -12)
    p.v[1][p.prefix[0, 104]] *= np.float32(-1.5)
    p.prefix[0, 300:420] = -1
    p.upload()
    q = queries(2, 41, 1, 2, d, "bf16")
    check_promise(kv, p, [700 * 16 - 3, 699 * 16], grid(41, 2, [i % 50 + 1 for i in range(41)]), q, 0.02)


@pytest.mark.parametrize("scale", [0.02, -0.05])
def test_far_scales_nan_and_keys_of_every_scale(kv, scale):
    """More than 32 rows and value scales that are no powers of two: NaN values reach
    every query, those past the prefix's end none; negative, zero and extreme scales
    of keys; a value scale that is not finite."""
    seqs, d, pt = 20, 64, 16
    p = shared_pool(kv, seqs, 1, 12, 8, pt, d, seed=5, n_pages=1 << 20)
    ids = np.random.default_rng(5).permutation(p.n_pages)
    p.prefix[0] = ids[:12]
    p.pages = ids[12:12 + 20].reshape(seqs, 1, 1).astype(np.int32)
    p.v[1] *= np.float32(1.25)
    p.k[1] = np.random.default_rng(4).choice(np.array([1, 0.5, -1, -0.3, 0, 1.7, 2.0 ** -140], np.float32), p.n_pages)
    place = orc.v_place(pt, d)
    p.v[0][p.prefix[0, 9], place[7:].reshape(-1)] = 0x7F          # the prefix ends inside page 9
    p.v[1][p.prefix[0, 10]] = np.nan
    p.upload()
    q, lengths = queries(3, seqs, 1, 2, d, "bf16"), grid(seqs, 1, [i % 16 + 1 for i in range(seqs)])
    out = check_promise(kv, p, [9 * 16 + 7], lengths, q, scale, far=True)
    assert not out.isnan().any()
    p.v[0][p.prefix[0, 2], place[3, 40]] = 0xFF
    p.upload()
    nan = check_promise(kv, p, [9 * 16 + 7], lengths, q, scale, far=True).isnan()
    assert nan[..., 40].all() and not nan[..., :40].any()
    p.v[1][p.prefix[0, 1]] = np.inf
    p.upload()
    assert check_promise(kv, p, [9 * 16 + 7], lengths, q, scale, far=True).isnan().all()

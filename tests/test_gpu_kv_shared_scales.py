"""Attention over a shared prefix whose pages' scales are of every kind, against
the 64-bit oracle and its bounds (oracle/kv_long_oracle.py): the paths of up to
32 query rows to a head and of more, held to what each of them promises."""
import numpy as np
import pytest

from oracle import kv_oracle as orc
from test_gpu_kv import grid, kv  # noqa: F401
from test_gpu_kv_long import check_shared, shared_pool
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

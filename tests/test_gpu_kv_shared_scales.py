"""Attention over a shared prefix whose pages' scales are of every kind, against
the 64-bit oracle and its bounds (oracle/kv_long_oracle.py): the paths of up to
32 query rows to a head and of more, held to what each of them promises."""
import numpy as np
import pytest

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

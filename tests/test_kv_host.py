"""Host-side checks of the KV page cache (no GPU needed): the oracle's own
pins, the exports of libibp_kv, and every refusal, which comes before
anything is enqueued (these calls never launch a kernel)."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import numpy as np
import pytest

from oracle import kv_oracle as orc

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "lossless_bit_level_amd", "libibp_kv.so")
HEADER = os.path.join(ROOT, "include", "ibp_kv.h")

built = pytest.mark.skipif(not os.path.exists(LIB),
                           reason="libibp_kv.so not built (run __graft_entry__.build())")


# ------------------------------------------------------------- the oracle --


def test_numbers_are_torchs_e4m3():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(orc.NUMBERS, want, equal_nan=True)
    assert orc.NUMBERS[0x7E] == 448 and orc.NUMBERS[1] == 2.0 ** -9


def test_nearest_code_rounds_like_torch_and_saturates():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * 2.0 ** rng.integers(-12, 9, 20000),
                        (orc.NUMBERS[:126] + orc.NUMBERS[1:127]) / 2,       # ties
                        orc.NUMBERS[:127], -orc.NUMBERS[:127], [448.0, -448.0, 0.0, -0.0, 2.0 ** -11]])
    x = x[np.abs(x) <= 448].astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(orc.nearest_code(x.astype(np.float64)), want)
    assert orc.nearest_code([500.0, -1e9, np.nan, np.inf, -np.inf]).tolist() == [0x7E, 0xFE, 0x7F, 0x7F, 0x7F]


@pytest.mark.parametrize("pt", [16, 32, 64])
@pytest.mark.parametrize("d", [64, 128, 192, 256])
def test_places_fill_the_page(pt, d):
    for place in (orc.k_place(pt, d), orc.v_place(pt, d)):
        assert np.array_equal(np.sort(place.reshape(-1)), np.arange(pt * d))
    assert orc.k_place(pt, d)[1, 0] == 16 and orc.k_place(pt, d)[0, 16] == 256
    assert orc.v_place(pt, d)[1, 0] == 1 and orc.v_place(pt, d)[4, 0] == 256
    assert orc.v_place(pt, d)[0, 1] == 16 and orc.v_place(pt, d)[0, 16] == 4


def test_exponent_bounds():
    for e in (-126, -20, 0, 8, 119):
        top = 448 * 2.0 ** e
        assert orc.exponent(top) == e
        assert orc.exponent(top * (1 + 2.0 ** -20)) == min(e + 1, 119)
    assert orc.exponent(0.0) == -126 and orc.exponent(3.3e38) == 119


def test_append_oracle_by_hand():
    """One head, 16-token pages: a first token of 1.0s, then one of 1000s."""
    codes, scales = np.full((2, 16 * 64), 0xAA, np.uint8), np.ones(2, np.float32)
    place, pages = orc.k_place(16, 64), np.array([[[1, 0]]], np.int32)
    orc.append(codes, scales, place, 16, pages, np.array([[1]]), np.ones((1, 1, 1, 64)))
    assert scales[1] == 2.0 ** -8                      # 448 * 2^-9 < 1 <= 448 * 2^-8
    assert (codes[1][place[0]] == orc.nearest_code(256.0)).all()
    assert (codes[1][place[1:]] == 0).all() and (codes[0] == 0xAA).all()
    orc.append(codes, scales, place, 16, pages, np.array([[2]]), np.full((1, 1, 1, 64), 1000.0))
    assert scales[1] == 4.0                            # 448 * 2 < 1000 <= 448 * 4
    assert (orc.NUMBERS[codes[1][place[0]]] == 0.25).all()
    assert (orc.NUMBERS[codes[1][place[1]]] == 256).all()  # 250 lies nearer to 256 than to 240


def test_attention_oracle_against_torch():
    rng = np.random.default_rng(1)
    d, pt, n = 64, 16, 37
    k = rng.standard_normal((1, n, 1, d))
    v = rng.standard_normal((1, n, 1, d))
    pages = np.array([[[2, 0, 1]]], np.int32)
    pools = []
    for x, place in ((k, orc.k_place(pt, d)), (v, orc.v_place(pt, d))):
        codes, scales = np.zeros((3, pt * d), np.uint8), np.ones(3, np.float32)
        orc.append(codes, scales, place, pt, pages, np.array([[n]]), x)
        pools.append((codes, scales))
    kk, _ = orc.read_rows(*pools[0], orc.k_place(pt, d), pt, pages[0, 0], n)
    vv, _ = orc.read_rows(*pools[1], orc.v_place(pt, d), pt, pages[0, 0], n)
    # a code is off by half a step: 2^-4 of the value, or of the smallest normal
    assert np.all(np.abs(kk - k[0, :, 0]) <= np.maximum(2.0 ** -4 * np.abs(k[0, :, 0]), 2.0 ** -17))
    q = rng.standard_normal((1, 4, 2, d))
    out, w, _, _ = orc.attention(pools[0], pools[1], pt, pages, np.array([[n]]), q, 0.125,
                                 weights=np.zeros((1, 1, 3), np.float32))
    tq = torch.from_numpy(q[0].transpose(1, 0, 2))
    mask = torch.ones(4, n, dtype=torch.bool).tril(n - 4)
    want = torch.nn.functional.scaled_dot_product_attention(
        tq, torch.from_numpy(kk).expand(2, n, d), torch.from_numpy(vv).expand(2, n, d), mask, scale=0.125)
    assert np.allclose(out[0].transpose(1, 0, 2), want.numpy(), rtol=1e-12, atol=1e-12)
    assert abs(w.sum() - 8) < 1e-12


def test_evict_oracle_by_hand():
    pages = np.array([[[7, 5, 3, 1, 9, 8]]], np.int32)
    w = np.array([[[0.0, 2.0, 1.0, 2.0, np.nan, 4.0]]], np.float32)
    p, ww, n = orc.evict(pages, w, np.array([[16 * 4 + 3]], np.int32), 16, 3, 1, 1)
    assert p[0, 0].tolist() == [7, 5, 9, 3, 1, 8]       # 5 before 1: equal weights, lower position
    assert n[0, 0] == 2 * 16 + 3
    assert np.array_equal(ww[0, 0], np.array([0, 2, np.nan, 0, 0, 4], np.float32), equal_nan=True)


# ------------------------------------------------------------ the library --


@built
def test_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ibp_kv_[a-z_]+)\s*\(", text)))
    assert names == ["ibp_kv_append", "ibp_kv_attention", "ibp_kv_attention_workspace_bytes",
                     "ibp_kv_evict", "ibp_kv_last_hip_error", "ibp_kv_status_string"]
    L = ctypes.CDLL(LIB)
    for n in names:
        assert hasattr(L, n), n


@built
def test_eviction_buffers_bound_every_access(tmp_path):
    """The eviction reads and writes its rows through buffers that end with the
    row.  A buffer's scalar offset takes no part in its bounds check, so that
    every access of the built kernels has it 0."""
    objdump = "/opt/rocm/llvm/bin/llvm-objdump"
    if not os.path.exists(objdump):
        pytest.skip("no llvm-objdump")
    copy = shutil.copy(LIB, tmp_path)
    subprocess.run([objdump, "--offloading", copy], cwd=tmp_path, check=True, capture_output=True, timeout=60)
    image = [f for f in os.listdir(tmp_path) if f.endswith("gfx950")]
    assert len(image) == 1
    text = subprocess.run([objdump, "-d", "--mcpu=gfx950", image[0]], cwd=tmp_path, check=True, capture_output=True,
                          text=True, timeout=60).stdout
    kernels = 0
    for kernel in re.split(r"\n(?=[0-9a-f]+ <)", text):
        if "evict_kernel" not in kernel.split("\n", 1)[0]:
            continue
        kernels += 1
        found = re.findall(r"\tbuffer_(load|store)_dword(?:x\d)? \w+(?:\[[\d:]+\])?, v\d+, s\[\d+:\d+\], (\w+) offen", kernel)
        assert {"load", "store"} <= {what for what, _ in found}
        assert len(found) == kernel.count("\tbuffer_") - kernel.count("\tbuffer_inv") - kernel.count("\tbuffer_wb")
        assert {offset for _, offset in found} == {"0"}
    assert kernels == 3


@pytest.fixture(scope="module")
def kv():
    if not os.path.exists(LIB):
        pytest.skip("libibp_kv.so not built")
    from lossless_bit_level_amd import ibp_kv
    return ibp_kv


FAKE = 0x10000  # never dereferenced


def raw(kv, cls, *values):
    """A structure filled field by field, without the tensors' checks."""
    x = cls.__new__(cls)
    ctypes.Structure.__init__(x)
    for (name, _), v in zip(cls._fields_, values):
        setattr(x, name, v)
    return x


def cache(kv, n=4, pt=16, d=128, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE):
    return raw(kv, kv.ibp_kv_cache, n, pt, d, kc, ks, vc, vs)


def table(kv, n=2, h=2, m=3, pages=FAKE, lengths=FAKE):
    return kv.ibp_kv_table(n, h, m, pages, lengths)


def tensor(kv, data=FAKE):
    return kv.ibp_kv_tensor(data, 256, 256, 128)


def test_status_strings(kv):
    for s in (0, -1, -2, -3, -5):
        assert kv.status_string(s) != "unknown status"
    assert kv.status_string(7) == "unknown status"


def test_append_refusals(kv):
    f, INV, UNS, LAY = kv.lib().ibp_kv_append, kv.IBP_ERR_INVALID_ARGUMENT, kv.IBP_ERR_UNSUPPORTED, kv.IBP_ERR_LAYOUT

    def call(c=None, t=None, dtype=0, n=1, k=None, v=None, counts=None):
        return f(cache(kv) if c is None else c, table(kv) if t is None else t, dtype, n,
                 tensor(kv) if k is None else k, tensor(kv) if v is None else v, counts, None)
    assert f(None, table(kv), 0, 1, tensor(kv), tensor(kv), None, None) == INV
    assert f(cache(kv), None, 0, 1, tensor(kv), tensor(kv), None, None) == INV
    assert f(cache(kv), table(kv), 0, 1, None, tensor(kv), None, None) == INV
    for pt in (0, 8, 24, 128):
        assert call(c=cache(kv, pt=pt)) == UNS
    for d in (0, 32, 96, 320):
        assert call(c=cache(kv, d=d)) == UNS
    assert call(dtype=2) == UNS
    for name in ("kc", "ks", "vc", "vs"):
        assert call(c=cache(kv, **{name: None})) == INV
    assert call(c=cache(kv, kc=FAKE + 8)) == LAY
    assert call(c=cache(kv, vs=FAKE + 2)) == LAY
    assert call(t=table(kv, pages=None)) == INV
    assert call(t=table(kv, lengths=None)) == INV
    assert call(t=table(kv, lengths=FAKE + 2)) == LAY
    assert call(t=table(kv, n=1 << 40)) == INV
    assert call(t=table(kv, m=1 << 28)) == INV             # capacity past 2^31
    assert call(n=1 << 31) == INV
    assert call(k=tensor(kv, None)) == INV
    assert call(v=tensor(kv, FAKE + 1)) == LAY
    assert call(counts=FAKE + 1) == LAY
    # nothing to do
    assert call(n=0) == kv.IBP_OK
    assert call(t=table(kv, n=0, pages=None, lengths=None)) == kv.IBP_OK
    assert call(t=table(kv, m=0, pages=None)) == kv.IBP_OK
    assert call(c=cache(kv, n=0, kc=None, ks=None, vc=None, vs=None)) == kv.IBP_OK


def test_attention_refusals(kv):
    f, INV, UNS, LAY = kv.lib().ibp_kv_attention, kv.IBP_ERR_INVALID_ARGUMENT, kv.IBP_ERR_UNSUPPORTED, kv.IBP_ERR_LAYOUT

    def call(c=None, t=None, dtype=0, heads=4, n=1, q=None, out=None, counts=None, scale=0.1,
             w=None, wo=None, ws=FAKE, ws_bytes=1 << 40):
        return f(cache(kv) if c is None else c, table(kv) if t is None else t, dtype, heads, n,
                 tensor(kv) if q is None else q, tensor(kv) if out is None else out, counts, scale,
                 w, wo, ws, ws_bytes, None)
    assert f(None, table(kv), 0, 4, 1, tensor(kv), tensor(kv), None, 0.1, None, None, FAKE, 1 << 40, None) == INV
    assert call(c=cache(kv, pt=48)) == UNS
    assert call(c=cache(kv, d=80)) == UNS
    assert call(dtype=7) == UNS
    assert call(t=table(kv, lengths=None)) == INV
    assert call(heads=0) == INV
    assert call(heads=5) == INV                            # no multiple of kv_heads
    assert call(q=tensor(kv, None)) == INV
    assert call(out=tensor(kv, FAKE + 1)) == LAY
    assert call(counts=FAKE + 2) == LAY
    assert call(w=FAKE) == INV and call(wo=FAKE) == INV    # one without the other
    assert call(w=FAKE, wo=FAKE + 2) == LAY
    for bad in (float("nan"), float("inf")):
        assert call(scale=bad) == INV
    assert call(n=1 << 40) == INV
    assert call(ws=FAKE + 4) == LAY
    # too little workspace, or none
    need = kv.lib().ibp_kv_attention_workspace_bytes(cache(kv), table(kv, m=4096), 4, 1, 1)
    assert need > 0
    assert call(t=table(kv, m=4096), w=FAKE, wo=FAKE, ws_bytes=need - 1) == INV
    assert call(t=table(kv, m=4096), w=FAKE, wo=FAKE, ws=None) == INV
    assert call(t=table(kv, n=0, pages=None, lengths=None)) == kv.IBP_OK


def test_workspace_bytes(kv):
    f = kv.lib().ibp_kv_attention_workspace_bytes
    assert f(cache(kv, pt=48), table(kv), 4, 1, 1) == 0
    assert f(cache(kv), table(kv), 5, 1, 1) == 0
    small, more = f(cache(kv), table(kv, m=1000), 4, 1, 0), f(cache(kv), table(kv, m=1000), 4, 1, 1)
    assert 0 < small < more
    assert more - small == 2 * 2 * 2 * 1000 * 4            # a float for a query row and tile


def test_evict_refusals(kv):
    f, INV, UNS, LAY = kv.lib().ibp_kv_evict, kv.IBP_ERR_INVALID_ARGUMENT, kv.IBP_ERR_UNSUPPORTED, kv.IBP_ERR_LAYOUT
    far = [FAKE + (i << 20) for i in range(6)]

    def call(t=None, pt=16, keep=3, sink=1, recent=1, w=far[2], po=far[3], wo=far[4], lo=far[5]):
        return f(table(kv, pages=far[0], lengths=far[1]) if t is None else t, pt, keep, sink, recent,
                 w, po, wo, lo, None)
    assert f(None, 16, 3, 1, 1, far[2], far[3], far[4], far[5], None) == INV
    assert call(pt=20) == UNS
    assert call(recent=0) == INV
    assert call(keep=1) == INV                             # below sink + recent
    assert call(sink=4) == INV
    assert call(sink=(1 << 64) - 1) == INV
    assert call(keep=(1 << 64) - 1, sink=5, recent=(1 << 64) - 1) == INV
    for name in ("w", "po", "wo", "lo"):
        assert call(**{name: None}) == INV
        assert call(**{name: far[0] + (1 << 24) + 2}) == LAY
    assert call(po=far[0]) == INV                          # in place
    assert call(wo=far[2] + 8) == INV                      # overlap
    assert call(lo=far[1]) == INV
    assert call(po=far[4]) == INV                          # two outputs
    assert call(t=table(kv, n=0, pages=None, lengths=None)) == kv.IBP_OK


def test_binding_refuses_cpu_tensors(kv):
    z = torch.zeros(2, 2048, dtype=torch.uint8)
    s = torch.zeros(2)
    with pytest.raises(ValueError, match="k_codes"):
        kv.ibp_kv_cache(z, s, z, s, 16, 128)
    t = torch.zeros(1, 1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="pages"):
        kv.ibp_kv_evict(t, torch.zeros(1, 1, 2), torch.zeros(1, 1, dtype=torch.int32), 16, 2)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        kv.ibp_kv_append(cache(kv), t, t, torch.zeros(1, 1, 1, 128), torch.zeros(1, 1, 1, 128))


def test_missing_library_raises(tmp_path):
    code = ("import lossless_bit_level_amd.ibp_kv as kv\n"
            "kv._LIB_PATH = '/nonexistent/libibp_kv.so'\n"
            "try:\n    kv.lib()\nexcept RuntimeError as e:\n    assert 'is missing' in str(e)\nelse:\n    raise SystemExit(1)\n")
    assert subprocess.run([sys.executable, "-c", code], cwd=ROOT, timeout=120).returncode == 0


def test_binding_refuses_tensors_of_two_gpus(kv):
    """The kernels run on one GPU with the addresses as they are: no tensor of
    a call may be another GPU's, nor may the stream.  (Tensors without memory;
    nothing is launched.)"""
    from torch._subclasses.fake_tensor import FakeTensorMode
    ext = kv._ext()

    class Stream:
        device = torch.device("cuda", 0)

    with FakeTensorMode(allow_non_fake_inputs=True):
        def make(i, shape, dtype):
            return torch.empty(shape, dtype=dtype, device=f"cuda:{i}")

        def both(shape, dtype=torch.float32):
            return make(0, shape, dtype), make(1, shape, dtype)
        codes, scales = both((8, 2048), torch.uint8), both((8,))
        pages, lengths = both((2, 2, 2), torch.int32), both((2, 2), torch.int32)
        weights, counts = both((2, 2, 2)), both((2,), torch.int32)
        x, q, workspace = both((2, 1, 2, 128), torch.float16), both((2, 1, 4, 128), torch.float16), both((64,), torch.uint8)

        def each(call, args):
            """Every tensor but the first from the other GPU, in turn."""
            for i, a in enumerate(args):
                if i and isinstance(a, tuple):
                    mixed = [(b[i == j] if isinstance(b, tuple) else b) for j, b in enumerate(args)]
                    with pytest.raises(ValueError, match="same GPU"):
                        call(*mixed)
        plain = cache(kv)
        each(lambda *a: ext.set_cache(plain, *a), (codes, scales, codes, scales, 16, 128))
        each(lambda *a: ext.append(plain, *a), (pages, lengths, x, x, counts, 0))
        each(lambda *a: ext.attention(plain, *a), (pages, lengths, q, None, weights, weights, counts, q, workspace, 0))
        each(ext.evict, (pages, weights, lengths, 16, 2, 1, 1, pages, weights, lengths, 0))
        # the cache's own tensors
        plain.tensors = (codes[1], scales[1], codes[1], scales[1])
        with pytest.raises(ValueError, match="same GPU"):
            ext.append(plain, pages[0], lengths[0], x[0], x[0], None, 0)
        with pytest.raises(ValueError, match="same GPU"):
            ext.attention(plain, pages[0], lengths[0], q[0], None, None, None, None, None, None, 0)
        # the stream
        for call in (lambda: kv.ibp_kv_append(plain, pages[1], lengths[1], x[1], x[1], stream=Stream),
                     lambda: kv.ibp_kv_attention(plain, pages[1], lengths[1], q[1], stream=Stream),
                     lambda: kv.ibp_kv_evict(pages[1], weights[1], lengths[1], 16, 2, stream=Stream)):
            with pytest.raises(ValueError, match="stream of another GPU"):
                call()


def test_grids_beyond_a_launch_are_refused(kv):
    """A launch has fewer than 2^32 threads: calls that need 2^24 workgroups of
    256 threads, or 2^22 of 1024, are refused before anything is enqueued."""
    L, INV = kv.lib(), kv.IBP_ERR_INVALID_ARGUMENT
    far = [FAKE + (i << 44) for i in range(6)]
    many = 1 << 24

    def evict(n, m):
        return L.ibp_kv_evict(table(kv, n=n, h=1, m=m, pages=far[0], lengths=far[1]), 16, 3, 1, 1, far[2], far[3], far[4], far[5], None)
    assert evict(many, 2) == INV and evict(many, 1024) == INV
    assert evict(many >> 2, 1025) == INV and evict(many >> 2, 4097) == INV
    assert evict(many, 16385) == INV

    def append(n, pt, new=1, m=3):
        return L.ibp_kv_append(cache(kv, pt=pt), table(kv, n=n, h=1, m=m), 0, new, tensor(kv), tensor(kv), None, None)
    for pt in (16, 32, 64):
        assert append(many * (64 // pt), pt) == INV
    assert append(1 << 12, 64, new=64 << 12, m=1 << 14) == INV

    def attention(n, heads=1, new=1, m=3, weights=None):
        return L.ibp_kv_attention(cache(kv), table(kv, n=n, h=1, m=m), 0, heads, new, tensor(kv), tensor(kv), None, 0.1,
                                  weights, weights, FAKE, (1 << 64) - 1, None)

    def workspace(n, heads=1, new=1, m=3, weights=0):
        return L.ibp_kv_attention_workspace_bytes(cache(kv), table(kv, n=n, h=1, m=m), heads, new, weights)
    assert attention(many) == INV
    assert attention(many >> 8, heads=16, new=1 << 9) == INV                       # 256 units a row
    assert attention(many >> 8, heads=16, new=4, m=1 << 14, weights=FAKE) == INV   # the joining of weights
    assert attention(many >> 6, new=0, m=1 << 14, weights=FAKE) == INV
    assert workspace(many >> 8, heads=16, new=4, m=1 << 14, weights=1) == 0
    # without a joining launch these rows are no more than the others
    assert workspace(many >> 6, m=1 << 14, weights=1) > 0


def test_binding_refuses_given_outputs_of_a_gradient(kv):
    """(Tensors without memory; nothing is launched.)"""
    from torch._subclasses.fake_tensor import FakeTensorMode
    ext, plain = kv._ext(), cache(kv)
    with FakeTensorMode():
        def make(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device="cuda:0")
        pages, lengths, w = make(2, 2, 2, dtype=torch.int32), make(2, 2, dtype=torch.int32), make(2, 2, 2)
        q, grown = make(2, 1, 4, 128, dtype=torch.float16), make(2, 1, 4, 128, dtype=torch.float16).requires_grad_()
        for args in ((grown, None, None, None, None, q), (q, None, None, None, None, grown), (grown, None, w, w, None, None),
                     (q, None, w, make(2, 2, 2).requires_grad_(), None, None)):
            with pytest.raises(ValueError, match="requires a gradient"):
                ext.attention(plain, pages, lengths, *args, None, 0)
        with pytest.raises(ValueError, match="requires a gradient"):
            ext.evict(pages, make(2, 2, 2).requires_grad_(), lengths, 16, 2, 1, 1, None, w, None, 0)


def test_attention_refuses_rows_on_each_other(kv):
    """An output whose rows share memory, a broadcast one among them, would hold
    whichever workgroup came last."""
    f, INV = kv.lib().ibp_kv_attention, kv.IBP_ERR_INVALID_ARGUMENT

    def call(out, q=None, new=2, ws=None):
        """With too little workspace at the end, so that nothing is launched."""
        return f(cache(kv), table(kv, m=4096), 0, 4, new, tensor(kv) if q is None else q, kv.ibp_kv_tensor(FAKE, *out), None, 0.1,
                 None, None, FAKE + 4 if ws is None else ws, 0, None)
    for out in ((0, 512, 128), (1024, 0, 128), (1024, 512, 0), (1024, 512, 127), (1024, -127, 128), (64, 512, 128)):
        assert call(out) == INV
    LAY = kv.IBP_ERR_LAYOUT     # the workspace's, which is looked at next
    assert call((1024, 512, 128)) == LAY and call((-1024, 512, -128)) == LAY
    assert call((1024, 0, 128), new=1) == LAY
    assert call((1024, 512, 128), q=kv.ibp_kv_tensor(FAKE, 0, 0, 0)) == LAY    # inputs may be broadcast

"""Host-side checks of long and shared contexts over the KV pages (no GPU
needed): the oracle's own pins, the exports of libibp_kv_long, and every
refusal, which comes before anything is enqueued."""
import ctypes
import os
import re
import shutil
import subprocess
import sys
import warnings

import numpy as np
import pytest

from oracle import kv_long_oracle as lorc
from oracle import kv_oracle as orc
from test_kv_host import FAKE, cache, raw, table, tensor

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "lossless_bit_level_amd", "libibp_kv_long.so")
HEADER = os.path.join(ROOT, "include", "ibp_kv_long.h")

built = pytest.mark.skipif(not os.path.exists(LIB), reason="libibp_kv_long.so not built (run __graft_entry__.build())")
OK = 0


# ------------------------------------------------------------- the oracle --


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_oracle_turns_complex_numbers(interleaved):
    """The pairs as complex numbers times e^(i angle), within three roundings."""
    rng = np.random.default_rng(0)
    d, half = 64, 24
    x = rng.standard_normal(d)
    angle = rng.uniform(-1000, 1000, (9, half))
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    y = lorc.rotate(x, cos, sin, 7, interleaved)
    a, b = (np.arange(0, 2 * half, 2), np.arange(1, 2 * half, 2)) if interleaved else (np.arange(half), np.arange(half, 2 * half))
    z = (x[a] + 1j * x[b]) * (cos[7].astype(np.float64) + 1j * sin[7])
    off = 4 * 2.0 ** -24 * (np.abs(x[a]) + np.abs(x[b]))
    assert (np.abs(y[a] - z.real) <= off).all() and (np.abs(y[b] - z.imag) <= off).all()
    assert np.array_equal(y[2 * half:], x[2 * half:].astype(np.float32))
    for outside in (-1, 9):
        y = lorc.rotate(x, cos, sin, outside, interleaved)
        assert np.isnan(y[:2 * half]).all() and np.array_equal(y[2 * half:], x[2 * half:].astype(np.float32))


def test_rotation_oracle_by_hand():
    cos, sin = np.array([[0.0] * 8, [1.0] * 8], np.float32), np.array([[1.0] * 8, [0.0] * 8], np.float32)
    x = np.arange(64.0)
    assert lorc.rotate(x, cos, sin, 0, False)[:16].tolist() == [-8.0 - i for i in range(8)] + [float(i) for i in range(8)]
    assert lorc.rotate(x, cos, sin, 0, True)[:6].tolist() == [-1, 0, -3, 2, -5, 4]
    assert np.array_equal(lorc.rotate(x, cos, sin, 1, True), x)
    # positions are places in the row where none are given; tokens before place 0 do not exist
    t = lorc.rotated(np.ones((1, 3, 1, 64)), cos, sin, np.array([[2]]), 1, 16)
    assert not t[0, 0].any() and t[0, 1, 0, 0] == -1 and t[0, 2, 0, 0] == 1
    assert np.isnan(lorc.rotated(np.ones((1, 1, 1, 64)), cos, sin, np.array([[2]]), 1, 16, positions=np.array([[5]]))[0, 0, 0, :16]).all()


def test_outline_oracle_bounds_the_keys():
    rng = np.random.default_rng(1)
    pt, d = 16, 64
    place = orc.k_place(pt, d)
    codes = rng.integers(0, 127, (6, pt * d), dtype=np.uint8) | (rng.integers(0, 2, (6, pt * d), dtype=np.uint8) << 7)
    codes[2], codes[3, 5] = 0x80, 0x7F
    codes[4] &= 0x81                                   # +-2^-9 and zeros
    scales = (2.0 ** rng.integers(-5, 5, 6)).astype(np.float32)
    scales[5] = np.inf
    out, s = np.full((6, 2, d), 99, np.int8), np.zeros(6, np.float32)
    lorc.outline(codes, scales, place, pt, np.arange(6, dtype=np.int32)[None, None], np.array([[6 * pt]]), out, s, 6 * pt)
    for p in (0, 1, 4):
        key = orc.NUMBERS[codes[p][place]] * scales[p]
        hi, lo = out[p].astype(np.float64) * s[p]
        assert (key <= hi).all() and (key >= lo).all()
        assert (hi - key.max(0) < s[p]).all() and (key.min(0) - lo < s[p]).all()
        assert np.abs(out[p]).max() > 63 or s[p] == scales[p] * 2.0 ** -15   # no smaller unit would do
    assert not out[2].any() and s[2] == scales[2] * np.float32(2.0 ** -15)
    assert np.isnan(s[[3, 5]]).all() and not out[[3, 5]].any()


def test_score_oracle_is_a_bound():
    """At least q . k for every key within the outline, up to the rounding of q,
    and reached by one of them."""
    rng = np.random.default_rng(2)
    for _ in range(50):
        d = 64
        codes = np.sort(rng.integers(-127, 128, (2, d)), 0)[::-1]
        q = rng.standard_normal(d) * 2.0 ** rng.integers(-20, 20)
        whole, t = lorc.whole_query(q)
        assert np.abs(whole).max() <= 127 * 128 and np.abs(whole).max() > 127 * 64 - 1
        assert (np.abs(whole * t - q) <= t / 2).all()
        best = lorc.score([(whole, t)], codes, 0.5)
        corner = np.where(q > 0, codes[0], codes[1]) * 0.5
        slack = t / 2 * np.abs(corner).sum() + 2.0 ** -23 * abs(float(best))
        assert abs(best - q @ corner) <= slack
        for _ in range(20):
            k = rng.uniform(codes[1], codes[0] + 1e-9) * 0.5
            assert q @ k <= best + slack
    assert lorc.whole_query(np.array([1.0, np.inf])) is None
    assert lorc.whole_query(np.zeros(3))[1] == 1.0
    assert lorc.whole_query(np.array([127.0 * 128]))[1] == 1.0 and lorc.whole_query(np.array([127.0 * 128 + 1]))[1] == 2.0


def test_select_oracle_by_hand():
    codes = np.zeros((6, 2, 64), np.int8)
    codes[:, 0, 0], codes[:, 1, 0] = [5, 9, 9, 1, 0, 7], [-1, -2, -9, 0, 0, -3]
    scales = np.array([1, 1, 1, 100, np.nan, 1], np.float32)
    pages = np.array([[[5, 0, 1, 2, 3, 4, 9, 0]]], np.int32)
    q = np.zeros((1, 1, 1, 64))
    q[..., 0] = 2.0
    def places(keep, sink, recent, n=8 * 16):
        return lorc.select(codes, scales, pages, np.array([[n]]), 16, q, keep, sink, recent)[2][0, 0].tolist()
    assert places(3, 1, 1) == [0, 5, 7]                # NaN above all numbers
    assert places(4, 1, 1) == [0, 4, 5, 7]             # then 100
    assert places(5, 1, 1) == [0, 2, 4, 5, 7]          # 9 twice: the lower place
    assert places(7, 1, 1) == [0, 1, 2, 3, 4, 5, 7]    # the hole last
    assert places(4, 0, 1, 50) == [0, 1, 2, 3]
    got = lorc.select(codes, scales, pages, np.array([[50]]), 16, q, 6, 0, 1)
    assert got[0][0, 0].tolist() == [5, 0, 1, 2, -1, -1] and got[1][0, 0] == 50
    q[..., 0] = -2.0
    assert places(4, 1, 1) == [0, 3, 5, 7]             # 18 of the page with -9


def test_shared_oracle_is_attention_of_whole_rows():
    rng = np.random.default_rng(3)
    pt, d, heads, seqs = 16, 64, 2, 3
    pools = [(rng.integers(0, 0x50, (20, pt * d), dtype=np.uint8), (2.0 ** rng.integers(-3, 2, 20)).astype(np.float32)) for _ in range(2)]
    prefix = rng.integers(0, 20, (heads, 3)).astype(np.int32)
    prefix[1, 2] = -1
    pages = rng.integers(0, 20, (seqs, heads, 4)).astype(np.int32)
    q = rng.standard_normal((seqs, 2, 4, d))
    lengths = np.array([[40, 40], [2, 2], [64, 33]], np.int32)
    out, err = lorc.attention_shared(*pools, pt, prefix, np.array([48, 48]), pages, lengths, q, 0.05, rounding=0.0)
    whole = np.concatenate([np.broadcast_to(prefix, (seqs, heads, 3)), pages], 2)
    want, _, err2, _ = orc.attention(*pools, pt, whole, lengths + 48, q, 0.05)
    assert np.allclose(out, want, rtol=1e-12, atol=1e-12)
    assert (err >= err2).all() and np.allclose(err, err2, rtol=0.05)


# ------------------------------------------------------------ the library --


@built
def test_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ibp_kv_[a-z_]+)\s*\(", text)))
    assert names == ["ibp_kv_append_rotated", "ibp_kv_attention_shared", "ibp_kv_attention_shared_workspace_bytes",
                     "ibp_kv_long_last_hip_error", "ibp_kv_outline", "ibp_kv_select", "ibp_kv_select_workspace_bytes"]
    L = ctypes.CDLL(LIB)
    for n in names:
        assert hasattr(L, n), n


@pytest.fixture(scope="module")
def kv():
    if not os.path.exists(LIB):
        pytest.skip("libibp_kv_long.so not built")
    from lossless_bit_level_amd import ibp_kv
    return ibp_kv


FAR = [FAKE + (i << 40) for i in range(12)]


def rotation(kv, n=100, rotary=64, interleaved=0, cos=FAKE, sin=FAKE, positions=None):
    return kv.ibp_kv_rotation(n, rotary, interleaved, cos, sin, positions)


def outlines(kv, codes=FAKE, scales=FAKE):
    return kv.ibp_kv_outlines(codes, scales)


def test_append_rotated_refusals(kv):
    f, INV, UNS, LAY = kv.long_lib().ibp_kv_append_rotated, kv.IBP_ERR_INVALID_ARGUMENT, kv.IBP_ERR_UNSUPPORTED, kv.IBP_ERR_LAYOUT

    def call(c=None, t=None, dtype=0, n=1, k=None, v=None, counts=None, r=None, heads=4, q=None, out=None, o=None):
        return f(cache(kv) if c is None else c, table(kv) if t is None else t, dtype, n, tensor(kv) if k is None else k,
                 tensor(kv) if v is None else v, counts, rotation(kv) if r is None else r, heads, q, out, o, None)
    assert f(None, table(kv), 0, 1, tensor(kv), tensor(kv), None, rotation(kv), 0, None, None, None, None) == INV
    assert f(cache(kv), None, 0, 1, tensor(kv), tensor(kv), None, rotation(kv), 0, None, None, None, None) == INV
    assert f(cache(kv), table(kv), 0, 1, tensor(kv), tensor(kv), None, None, 0, None, None, None, None) == INV
    assert f(cache(kv), table(kv), 0, 1, None, tensor(kv), None, rotation(kv), 0, None, None, None, None) == INV
    assert call(c=cache(kv, pt=48)) == UNS and call(c=cache(kv, d=96)) == UNS and call(dtype=2) == UNS
    for rotary in (0, 8, 24, 144, 1 << 31):
        assert call(r=rotation(kv, rotary=rotary)) == UNS
    assert call(r=rotation(kv, interleaved=2)) == UNS
    assert call(r=rotation(kv, cos=None)) == INV and call(r=rotation(kv, sin=None)) == INV
    assert call(r=rotation(kv, cos=FAKE + 8)) == LAY and call(r=rotation(kv, sin=FAKE + 4)) == LAY
    assert call(r=rotation(kv, positions=FAKE + 2)) == LAY
    assert call(k=tensor(kv, None)) == INV and call(v=tensor(kv, FAKE + 1)) == LAY and call(counts=FAKE + 1) == LAY
    assert call(t=table(kv, pages=None)) == INV and call(t=table(kv, m=1 << 28)) == INV and call(n=1 << 31) == INV
    assert call(o=outlines(kv, codes=None)) == INV and call(o=outlines(kv, scales=None)) == INV
    assert call(o=outlines(kv, codes=FAKE + 8)) == LAY and call(o=outlines(kv, scales=FAKE + 2)) == LAY
    # queries
    q = tensor(kv)
    assert call(q=q) == INV and call(out=q) == INV
    assert call(q=q, out=q, heads=0) == INV and call(q=q, out=q, heads=3) == INV
    assert call(q=tensor(kv, None), out=q) == INV and call(q=q, out=tensor(kv, FAKE + 1)) == LAY
    for strides in ((0, 512, 128), (1024, 0, 128), (1024, 512, 0), (1024, 512, -127)):
        assert call(n=2, q=q, out=kv.ibp_kv_tensor(FAKE, *strides)) == INV
    # grids beyond a launch
    assert call(t=table(kv, n=1 << 24, h=1, m=3), c=cache(kv, pt=64)) == INV
    assert call(n=1 << 20, q=q, out=q, heads=1 << 12) == INV
    assert call(t=table(kv, n=1 << 12, h=1, m=3), n=1 << 14, q=q, out=q, heads=1 << 4) == INV
    # nothing to do
    assert call(n=0) == OK and call(n=0, q=q, out=q) == OK
    assert call(t=table(kv, n=0, pages=None, lengths=None), q=q, out=q) == OK
    assert call(t=table(kv, m=0, pages=None)) == OK
    assert call(c=cache(kv, n=0, kc=None, ks=None, vc=None, vs=None), o=outlines(kv, None, None)) == OK


def test_outline_refusals(kv):
    f, INV, UNS, LAY = kv.long_lib().ibp_kv_outline, kv.IBP_ERR_INVALID_ARGUMENT, kv.IBP_ERR_UNSUPPORTED, kv.IBP_ERR_LAYOUT

    def call(c=None, o=None, t=None, n=1, counts=None):
        return f(cache(kv) if c is None else c, outlines(kv) if o is None else o, table(kv) if t is None else t, n, counts, None)
    assert f(None, outlines(kv), table(kv), 1, None, None) == INV
    assert f(cache(kv), None, table(kv), 1, None, None) == INV
    assert f(cache(kv), outlines(kv), None, 1, None, None) == INV
    assert call(c=cache(kv, pt=8)) == UNS and call(c=cache(kv, d=320)) == UNS
    assert call(o=outlines(kv, codes=None)) == INV and call(o=outlines(kv, codes=FAKE + 4)) == LAY
    assert call(t=table(kv, lengths=None)) == INV and call(t=table(kv, lengths=FAKE + 2)) == LAY
    assert call(n=1 << 31) == INV and call(counts=FAKE + 1) == LAY
    assert call(t=table(kv, n=1 << 24, h=16, m=1 << 10), n=1 << 20) == INV
    assert call(n=0) == OK and call(t=table(kv, n=0, pages=None, lengths=None)) == OK
    assert call(t=table(kv, m=0, pages=None)) == OK


def test_select_refusals(kv):
    f, INV, UNS, LAY = kv.long_lib().ibp_kv_select, kv.IBP_ERR_INVALID_ARGUMENT, kv.IBP_ERR_UNSUPPORTED, kv.IBP_ERR_LAYOUT

    def call(c=None, o=None, t=None, dtype=0, heads=4, n=1, q=None, counts=None, keep=3, sink=1, recent=1, po=FAR[3], lo=FAR[4],
             wo=FAR[5], ws=FAR[6], ws_bytes=0):
        """With no bytes of workspace, so that nothing is launched."""
        return f(cache(kv) if c is None else c, outlines(kv) if o is None else o,
                 table(kv, m=2000, pages=FAR[1], lengths=FAR[2]) if t is None else t, dtype, heads, n, tensor(kv) if q is None else q, counts,
                 keep, sink, recent, po, lo, wo, ws, ws_bytes, None)
    assert call() == INV                                      # the workspace
    assert f(None, outlines(kv), table(kv), 0, 4, 1, tensor(kv), None, 3, 1, 1, *FAR[3:7], 1 << 40, None) == INV
    assert f(cache(kv), None, table(kv), 0, 4, 1, tensor(kv), None, 3, 1, 1, *FAR[3:7], 1 << 40, None) == INV
    assert call(c=cache(kv, pt=24)) == UNS and call(dtype=2) == UNS
    assert call(o=outlines(kv, codes=FAKE + 1)) == LAY
    none = table(kv, n=0, pages=None, lengths=None)
    assert call(t=none) == OK
    for bad in (dict(recent=0), dict(keep=1), dict(sink=4), dict(keep=1 << 28), dict(sink=(1 << 64) - 1),
                dict(n=2), dict(n=18, recent=2), dict(n=1 << 31)):     # the last pages must hold the new tokens
        assert call(t=none, **bad) == INV
    assert call(t=none, n=2, recent=2) == OK and call(t=none, n=17, recent=2) == OK and call(t=none, n=0) == OK
    assert call(heads=0) == INV and call(heads=3) == INV
    assert call(q=tensor(kv, None)) == INV and call(q=tensor(kv, FAKE + 1)) == LAY
    for name in ("po", "lo", "wo"):
        assert call(**{name: None}) == INV
        assert call(**{name: FAR[9] + 2}) == LAY
    assert call(counts=FAKE + 1) == LAY and call(ws=FAR[6] + 8) == LAY

    def overlapping(**names):
        return call(ws_bytes=1 << 20, **names)
    for names in (dict(po=FAR[1]), dict(lo=FAR[2]), dict(wo=FAR[6] + 64), dict(po=FAR[5] + 8), dict(lo=FAR[3] + 4)):
        assert overlapping(**names) == INV
    assert call(heads=1 << 26, ws_bytes=1 << 40) == INV
    big = table(kv, n=1 << 22, h=1, m=2000, pages=FAR[1], lengths=FAR[2])
    assert call(t=big, heads=1, ws_bytes=1 << 40, po=FAKE + (7 << 44), lo=FAKE + (8 << 44), wo=FAKE + (9 << 44), ws=FAKE + (10 << 44)) == INV
    need = kv.long_lib().ibp_kv_select_workspace_bytes
    assert need(cache(kv), table(kv, m=1025)) == 2 * 2 * 1025 * 4
    assert need(cache(kv), table(kv, m=1024)) == 0      # rows that are chosen from as they are scored
    assert need(cache(kv, pt=24), table(kv, m=2000)) == 0


def test_attention_shared_refusals(kv):
    L = kv.long_lib()
    f, INV, UNS, LAY = L.ibp_kv_attention_shared, kv.IBP_ERR_INVALID_ARGUMENT, kv.IBP_ERR_UNSUPPORTED, kv.IBP_ERR_LAYOUT

    def call(c=None, p=None, t=None, dtype=0, heads=4, n=1, q=None, out=None, counts=None, scale=0.1, ws=FAKE, ws_bytes=0):
        """With no bytes of workspace, so that nothing is launched."""
        return f(cache(kv) if c is None else c, table(kv, n=1) if p is None else p, table(kv) if t is None else t, dtype, heads, n,
                 tensor(kv) if q is None else q, tensor(kv) if out is None else out, counts, scale, ws, ws_bytes, None)
    need = L.ibp_kv_attention_shared_workspace_bytes(cache(kv), table(kv, n=1), table(kv), 4, 1)
    assert need > 0
    assert call() == INV and call(ws_bytes=need - 1) == INV and call(ws=None, ws_bytes=need) == INV
    assert call(c=cache(kv, pt=48)) == UNS and call(c=cache(kv, d=80)) == UNS and call(dtype=7) == UNS
    none = table(kv, n=0, pages=None, lengths=None)
    assert call(t=none) == OK and call(n=0) == OK
    for bad in (table(kv, n=2), table(kv, n=1, h=3), table(kv, n=1, lengths=None), table(kv, n=1, m=1 << 28), table(kv, n=0)):
        assert call(t=none, p=bad) == INV
    assert call(t=none, p=table(kv, n=1, lengths=FAKE + 2)) == LAY
    assert f(cache(kv), None, table(kv), 0, 4, 1, tensor(kv), tensor(kv), None, 0.1, FAKE, 0, None) == INV
    assert f(cache(kv), table(kv, n=1), None, 0, 4, 1, tensor(kv), tensor(kv), None, 0.1, FAKE, 0, None) == INV
    assert call(heads=0) == INV and call(heads=5) == INV
    assert call(q=tensor(kv, None)) == INV and call(out=tensor(kv, FAKE + 1)) == LAY
    assert call(counts=FAKE + 2) == LAY and call(ws=FAKE + 4) == LAY
    for bad in (float("nan"), float("inf")):
        assert call(scale=bad) == INV
    for strides in ((0, 512, 128), (1024, 0, 128), (1024, 512, 0), (64, 512, 128)):
        assert call(n=2, out=kv.ibp_kv_tensor(FAKE, *strides)) == INV
    assert call(n=1 << 40) == INV and call(heads=4, n=1 << 24) == INV
    g = L.ibp_kv_attention_shared_workspace_bytes
    assert g(cache(kv, pt=48), table(kv, n=1), table(kv), 4, 1) == 0 and g(cache(kv), table(kv, n=1), table(kv), 5, 1) == 0
    assert g(cache(kv), table(kv, n=1), table(kv, n=1 << 22), 4, 1 << 8) == 0


def test_binding_refuses_what_does_not_fit(kv):
    """(Tensors without memory; nothing is launched.)"""
    from torch._subclasses.fake_tensor import FakeTensorMode
    ext, plain = kv._ext(), cache(kv, n=8)
    with FakeTensorMode():
        def make(*shape, dtype=torch.float32, device="cuda:0"):
            return torch.empty(shape, dtype=dtype, device=device)
        with warnings.catch_warnings():    # said once, that such a tensor was asked for its address
            warnings.simplefilter("ignore")
            make(1).data_ptr()
        i32, f16 = torch.int32, torch.float16
        pages, lengths, k, q = make(2, 2, 2, dtype=i32), make(2, 2, dtype=i32), make(2, 3, 2, 128, dtype=f16), make(2, 3, 4, 128, dtype=f16)
        cos, codes, scales = make(9, 64), make(8, 2, 128, dtype=torch.int8), make(8)
        good = dict(k=k, v=k, cos=cos, sin=cos, positions=None, q=q, q_out=None, counts=None, il=False, codes=codes, scales=scales)

        def rotated(**more):
            return ext.append_rotated(plain, pages, lengths, *{**good, **more}.values(), 0)
        for bad in (dict(cos=make(9, 32)), dict(cos=make(9, 64, dtype=torch.float64)), dict(sin=make(9, 128)[:, ::2]), dict(cos=make(64), sin=make(64)),
                    dict(positions=make(2, 2, dtype=i32)), dict(positions=make(2, 3)), dict(q=make(2, 2, 4, 128, dtype=f16)),
                    dict(q=make(2, 3, 5, 128, dtype=f16)), dict(q=make(2, 3, 4, 128, dtype=torch.bfloat16)), dict(q_out=make(2, 3, 4, 64, dtype=f16)),
                    dict(q=None, q_out=q), dict(codes=make(7, 2, 128, dtype=torch.int8)), dict(codes=make(8, 2, 128, dtype=torch.uint8)),
                    dict(scales=make(9)), dict(codes=make(8, 256, dtype=torch.int8)), dict(k=make(2, 3, 2, 64, dtype=f16)), dict(v=q),
                    dict(counts=make(3, dtype=i32)), dict(cos=make(9, 64, device="cpu")), dict(q=make(2, 3, 4, 128, dtype=f16, device="cpu"))):
            with pytest.raises(ValueError):
                rotated(**bad)
        grown = q.clone().requires_grad_()
        with pytest.raises(ValueError, match="requires a gradient"):
            rotated(q=grown, q_out=q)
        with pytest.raises(ValueError):
            ext.outline(plain, scales, codes, pages, lengths, 1, None, 0)
        sel = dict(codes=codes, scales=scales, pages=pages, lengths=lengths, q=q, keep=3, sink=1, recent=1, counts=None, po=None, lo=None, wo=None, ws=None)
        for bad in (dict(po=make(2, 2, 2, dtype=i32)), dict(lo=make(2, 3, dtype=i32)), dict(wo=make(2, 2, 3)), dict(ws=make(64)), dict(keep=1 << 40),
                    dict(q=make(2, 3, 3, 128, dtype=f16)), dict(q=make(2, 3, 4, 128)), dict(codes=make(8, 2, 64, dtype=torch.int8))):
            with pytest.raises(ValueError):
                ext.select(plain, *{**sel, **bad}.values(), 0)
        with pytest.raises((ValueError, OverflowError)):
            ext.select(plain, *{**sel, "keep": -1}.values(), 0)
        sh = dict(pp=make(2, 5, dtype=i32), pl=make(2, dtype=i32), pages=pages, lengths=lengths, q=q, scale=None, counts=None, out=None, ws=None)
        for bad in (dict(pp=make(3, 5, dtype=i32)), dict(pp=make(1, 2, 5, dtype=i32)), dict(pl=make(3, dtype=i32)), dict(pl=make(2)),
                    dict(q=make(2, 3, 3, 128, dtype=f16)), dict(out=make(2, 3, 4, 64, dtype=f16)), dict(out=make(2, 3, 4, 128)), dict(ws=make(8)),
                    dict(out=grown)):
            with pytest.raises(ValueError):
                ext.attention_shared(plain, *{**sh, **bad}.values(), 0)


def test_binding_refuses_tensors_of_two_gpus(kv):
    from torch._subclasses.fake_tensor import FakeTensorMode
    ext, plain = kv._ext(), cache(kv, n=8)

    class Stream:
        device = torch.device("cuda", 0)
    with FakeTensorMode(allow_non_fake_inputs=True):
        def both(shape, dtype=torch.float32):
            return tuple(torch.empty(shape, dtype=dtype, device=f"cuda:{i}") for i in (0, 1))
        i32, f16 = torch.int32, torch.float16
        pages, lengths, counts = both((2, 2, 2), i32), both((2, 2), i32), both((2,), i32)
        k, q, cos, positions = both((2, 1, 2, 128), f16), both((2, 1, 4, 128), f16), both((9, 64)), both((2, 1), i32)
        codes, scales, ws = both((8, 2, 128), torch.int8), both((8,)), both((64,), torch.uint8)
        kept, left, pp, pl = both((2, 2, 3), i32), both((2, 2), i32), both((2, 5), i32), both((2,), i32)

        def each(call, args):
            for i, a in enumerate(args):
                if i and isinstance(a, tuple):
                    with pytest.raises(ValueError, match="same GPU"):
                        call(plain, *[(b[i == j] if isinstance(b, tuple) else b) for j, b in enumerate(args)], 0)
        each(ext.append_rotated, (pages, lengths, k, k, cos, cos, positions, q, q, counts, False, codes, scales))
        each(ext.outline, (codes, scales, pages, lengths, 1, counts))
        each(ext.select, (codes, scales, pages, lengths, q, 3, 1, 1, counts, kept, left, kept, ws))
        each(ext.attention_shared, (pp, pl, pages, lengths, q, None, counts, q, ws))
        for call in (lambda: kv.ibp_kv_append_rotated(plain, pages[1], lengths[1], k[1], k[1], cos[1], cos[1], stream=Stream),
                     lambda: kv.ibp_kv_outline(plain, (codes[1], scales[1]), pages[1], lengths[1], stream=Stream),
                     lambda: kv.ibp_kv_select(plain, (codes[1], scales[1]), pages[1], lengths[1], q[1], 3, stream=Stream),
                     lambda: kv.ibp_kv_attention_shared(plain, pp[1], pl[1], pages[1], lengths[1], q[1], stream=Stream)):
            with pytest.raises(ValueError, match="stream of another GPU"):
                call()


def test_missing_library_raises():
    code = ("import lossless_bit_level_amd.ibp_kv as kv\n"
            "kv._LONG_LIB_PATH = '/nonexistent/libibp_kv_long.so'\n"
            "try:\n    kv.long_lib()\nexcept RuntimeError as e:\n    assert 'is missing' in str(e)\nelse:\n    raise SystemExit(1)\n")
    assert subprocess.run([sys.executable, "-c", code], cwd=ROOT, timeout=120).returncode == 0


def test_shared_oracle_bound_is_that_of_whole_rows():
    """Without the smallest step of 11-bit numbers the bound is the unshared one; half
    a step that counts for the prefix or for own tokens alone adds up to both."""
    rng = np.random.default_rng(4)
    pt, d, heads, seqs = 16, 64, 2, 3
    pools = [(rng.integers(0, 0x50, (20, pt * d), dtype=np.uint8), (2.0 ** rng.integers(-3, 2, 20)).astype(np.float32)) for _ in range(2)]
    prefix, pages = rng.integers(0, 20, (heads, 3)).astype(np.int32), rng.integers(0, 20, (seqs, heads, 4)).astype(np.int32)
    q, lengths = rng.standard_normal((seqs, 2, 4, d)), np.array([[40, 40], [2, 2], [64, 33]], np.int32)

    def bound(**more):
        return lorc.attention_shared(*pools, pt, prefix, np.array([48, 48]), pages, lengths, q, 0.05, floor=0.0, **more)[1]
    want = orc.attention(*pools, pt, np.concatenate([np.broadcast_to(prefix, (seqs, heads, 3)), pages], 2), lengths + 48, q, 0.05)[2]
    assert np.allclose(bound(), want, rtol=1e-9)
    none, first, own, both = bound(weight=0.0), bound(weight=2.0 ** -11, own_weight=0.0), bound(weight=0.0, own_weight=2.0 ** -11), bound(weight=2.0 ** -11)
    assert np.allclose(first + own, none + both, rtol=1e-9)
    for more in (first, own, bound(weight=0.0, least=2.0 ** -24)):     # the same where all values are zeros
        assert (more >= none).all() and (more > none).any((1, 3)).all()


def test_shared_workspace_is_0_for_what_the_call_refuses(kv):
    g = kv.long_lib().ibp_kv_attention_shared_workspace_bytes
    good = table(kv, n=1)
    assert g(cache(kv), good, table(kv), 4, 1) > 0
    for bad in (None, table(kv, n=2), table(kv, n=0), table(kv, n=1, h=3), table(kv, n=1, h=0), table(kv, n=1, lengths=None), table(kv, n=1, pages=None),
                table(kv, n=1, lengths=FAKE + 2), table(kv, n=1, m=1 << 28)):
        assert g(cache(kv), bad, table(kv), 4, 1) == 0
    for bad in (None, table(kv, lengths=None), table(kv, pages=FAKE + 1), table(kv, m=1 << 28), table(kv, n=1 << 30)):
        assert g(cache(kv), good, bad, 4, 1) == 0
    assert g(None, good, table(kv), 4, 1) == 0 and g(cache(kv), good, table(kv), 0, 1) == 0
    # nothing to do
    assert g(cache(kv), good, table(kv), 4, 0) == 0 and g(cache(kv), good, table(kv, n=0, pages=None, lengths=None), 4, 1) == 0


@built
def test_calls_of_the_cache_do_without_the_long_library(tmp_path):
    """Those of libibp_kv_long raise where it is missing, and no other does."""
    package = tmp_path / "lossless_bit_level_amd"
    package.mkdir()
    for name in ("__init__.py", "ibp.py", "ibp_kv.py", "libibp_kv.so", "_ibp_kv.so"):
        shutil.copy(os.path.join(ROOT, "lossless_bit_level_amd", name), package)
    code = ("import torch\n"
            "import lossless_bit_level_amd.ibp_kv as kv\n"
            "def error(call, *args):\n"
            "    try:\n        call(*args)\n"
            "    except (RuntimeError, ValueError) as e:\n        return type(e).__name__ + ' ' + str(e)\n"
            "i = torch.zeros(1, 1, 1, dtype=torch.int32)\n"
            "assert 'GPU tensor' in error(kv.ibp_kv_evict, i, i.float(), i[0], 16, 2), error(kv.ibp_kv_evict, i, i.float(), i[0], 16, 2)\n"
            "assert kv.status_string(0)\n"
            "assert 'libibp_kv_long.so is missing' in error(kv.ibp_kv_outline, None, (None, None), i, i[0])\n"
            "assert 'libibp_kv_long.so is missing' in error(kv.long_lib)\n")
    run = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, timeout=120, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr


@built
def test_selection_buffers_bound_every_access(tmp_path):
    """The selection reads ids and scores and writes what stays through buffers that
    end with the row, whatever the scores are.  A buffer's scalar offset takes no part
    in its bounds check, so that every access of the built kernels has it 0."""
    objdump = "/opt/rocm/llvm/bin/llvm-objdump"
    if not os.path.exists(objdump):
        pytest.skip("no llvm-objdump")
    copy = shutil.copy(LIB, tmp_path)
    subprocess.run([objdump, "--offloading", copy], cwd=tmp_path, check=True, capture_output=True, timeout=60)
    image = [f for f in os.listdir(tmp_path) if f.endswith("gfx950")]
    assert len(image) == 1
    text = subprocess.run([objdump, "-d", "--mcpu=gfx950", image[0]], cwd=tmp_path, check=True, capture_output=True,
                          text=True, timeout=120).stdout
    kernels = {"score_kernel": 0, "select_kernel": 0, "select_short_kernel": 0}
    for kernel in re.split(r"\n(?=[0-9a-f]+ <)", text):
        name = re.search(r"\d+(score_kernel|select_kernel|select_short_kernel)I", kernel.split("\n", 1)[0])
        if not name:
            continue
        kernels[name[1]] += 1
        found = re.findall(r"\tbuffer_(load|store)_dword(?:x\d)? \w+(?:\[[\d:]+\])?, v\d+, s\[\d+:\d+\], (\w+) offen", kernel)
        assert {what for what, _ in found} == ({"load"} if name[1] == "score_kernel" else {"load", "store"})
        assert len(found) == kernel.count("\tbuffer_") - kernel.count("\tbuffer_inv") - kernel.count("\tbuffer_wb")
        assert {offset for _, offset in found} == {"0"}
    assert kernels == {"score_kernel": 8, "select_kernel": 2, "select_short_kernel": 8}


def test_scales_whose_powers_of_two_are_infinite_are_refused(kv):
    """A factor of scores of more than 2^128 / log2(e): with a score of 0 it would be NaN."""
    INV, need = kv.IBP_ERR_INVALID_ARGUMENT, 1 << 40
    last, past = 2.358e38, 2.36e38          # 2^128 / log2(e) is 2.3586e38
    assert np.isfinite(np.float32(last) * np.float32(np.log2(np.e))) and np.isfinite(np.float32(past))
    shared, plain = kv.long_lib().ibp_kv_attention_shared, kv.lib().ibp_kv_attention
    for scale in (past, -past, 3.4e38, float("inf"), float("nan")):
        assert shared(cache(kv), table(kv, n=1), table(kv), 0, 4, 1, tensor(kv), tensor(kv), None, scale, FAKE + 4, need, None) == INV
        assert plain(cache(kv), table(kv), 0, 4, 1, tensor(kv), tensor(kv), None, scale, None, None, FAKE + 4, need, None) == INV
    for scale in (last, -last):             # refused for the workspace's alignment, not for the scale
        assert shared(cache(kv), table(kv, n=1), table(kv), 0, 4, 1, tensor(kv), tensor(kv), None, scale, FAKE + 4, need, None) == kv.IBP_ERR_LAYOUT
        assert plain(cache(kv), table(kv), 0, 4, 1, tensor(kv), tensor(kv), None, scale, None, None, FAKE + 4, need, None) == kv.IBP_ERR_LAYOUT

"""Rotary positions and the quantised cache on the CPU: tables, refusals, the oracle's parts."""
import ctypes as C
import math
import time

import numpy as np
import pytest
import torch

from calibration_free_bit_b200 import build as B
from calibration_free_bit_b200 import oq
import _cache_oracle as CO


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


FAKE = 1 << 20        # never dereferenced: validation fails first


def test_rope_frequencies_follow_their_formulas():
    i = np.arange(0, 128, 2) / 128
    f, m = oq.oq_build_rope(128, theta=500000.0).values()
    np.testing.assert_allclose(f, 500000.0 ** -i, rtol=1e-14)
    assert m == 1.0
    np.testing.assert_allclose(oq.oq_build_rope(128, scaling="linear", factor=4.0).values()[0],
                               1e4 ** -i / 4, rtol=1e-14)
    np.testing.assert_allclose(oq.oq_build_rope(128, scaling="ntk", factor=8.0).values()[0],
                               (1e4 * 8 ** (128 / 126)) ** -i, rtol=1e-14)
    f, m = oq.oq_build_rope(128, scaling="yarn", factor=16.0, original_len=4096).values()
    assert m == pytest.approx(0.1 * math.log(16.0) + 1.0, rel=1e-15)
    plain = 1e4 ** -i
    turns = 4096 * plain / (2 * math.pi)
    assert np.allclose(f[turns > 33], plain[turns > 33], rtol=1e-14)          # fast pairs stay
    assert np.allclose(f[turns < 0.8], plain[turns < 0.8] / 16, rtol=1e-14)   # slow ones scale
    assert np.all(f <= plain * (1 + 1e-14)) and np.all(f >= plain / 16 * (1 - 1e-14))
    assert np.all(np.diff(f) < 0)


@pytest.mark.parametrize("kw", [
    dict(rot_dim=8), dict(rot_dim=24), dict(rot_dim=528), dict(rot_dim=128, theta=1.0),
    dict(rot_dim=128, theta=float("inf")), dict(rot_dim=128, scaling="linear", factor=0.5),
    dict(rot_dim=128, scaling="yarn", factor=2.0, original_len=0),
    dict(rot_dim=128, layout="other"), dict(rot_dim=128, scaling="other")])
def test_rope_refusals(kw):
    with pytest.raises(oq.OQError) as e:
        oq.oq_build_rope(**kw)
    assert e.value.code == oq.OQ_EINVAL


_ROPE = []


def _rope_call(**kw):
    if not _ROPE:
        _ROPE.append(oq.oq_build_rope(128))
    a = dict(r=_ROPE[0].handle, dtype=oq.OQ_BF16, T=4, d=128, pos=FAKE, x=FAKE, y=FAKE, heads=2,
             xs=256, ys=256, k=None, ks=128, ky=FAKE, kys=128, k_heads=1)
    a.update(kw)
    return oq.lib().oq_apply_rope(a["r"], a["x"], a["xs"], a["y"], a["ys"], a["heads"], a["k"],
                                  a["ks"], a["ky"], a["kys"], a["k_heads"], a["dtype"], a["T"],
                                  a["d"], a["pos"], 0, None)


@pytest.mark.parametrize("kw", [
    dict(r=None), dict(dtype=3), dict(dtype=-1), dict(d=64), dict(d=136), dict(d=2048), dict(T=-1),
    dict(heads=0), dict(heads=1025), dict(pos=None), dict(pos=FAKE + 4), dict(x=None), dict(y=None),
    dict(x=FAKE + 2), dict(xs=-256), dict(xs=260), dict(ys=248), dict(xs=512),  # in place, 2 strides
    dict(k=FAKE, ky=None), dict(k=FAKE + 4), dict(k=FAKE, k_heads=0), dict(k=FAKE, kys=120),
    dict(k=FAKE, ks=256)])
def test_apply_rope_refusals(kw):
    assert _rope_call(**kw) == oq.OQ_EINVAL, kw


def test_no_rows_is_a_no_op():
    assert _rope_call(T=0, x=None, y=None, pos=None) == oq.OQ_OK
    assert _write(T=0, k=None, slots=None) == oq.OQ_OK
    assert _read(T=0, k=None, slots=None) == oq.OQ_OK
    assert _attend(rows=0, q=None) == oq.OQ_OK
    assert _attend(B=0, start=None) == oq.OQ_OK


def _cache(**kw):
    a = dict(kc=FAKE, vc=FAKE, kn=FAKE, vn=FAKE, pages=4, page=16, heads=2, d=128, bits=4)
    a.update(kw)
    return oq._KVCacheStruct(a["kc"], a["vc"], a["kn"], a["vn"], a["pages"], a["page"], a["heads"],
                             a["d"], a["bits"])


_R = {}


def _handles(d=128, bits=4):
    if (d, bits) not in _R:
        _R[d, bits] = (oq.oq_build_rpbh(d, 64), oq.oq_lloyd_max(d, bits))
    return _R[d, bits]


CACHE_BAD = [dict(kc=None), dict(vn=None), dict(kn=FAKE + 4), dict(pages=0), dict(page=8),
             dict(page=48), dict(page=2048), dict(heads=0), dict(heads=1025), dict(d=384),
             dict(d=256), dict(bits=3), dict(pages=1 << 31)]


def _write(cache=None, **kw):
    a = dict(k=FAKE, ks=256, v=FAKE, vs=256, dtype=oq.OQ_BF16, T=4, slots=FAKE)
    a.update(kw)
    r, c = _handles()
    s = _cache(**(cache or {}))
    return oq.lib().oq_kv_write(r.handle, c.handle, C.addressof(s), a["k"], a["ks"], a["v"],
                                a["vs"], a["dtype"], a["T"], a["slots"], None)


def _read(cache=None, **kw):
    a = dict(k=FAKE, ks=256, v=FAKE, vs=256, dtype=oq.OQ_BF16, T=4, slots=FAKE)
    a.update(kw)
    r, c = _handles()
    s = _cache(**(cache or {}))
    return oq.lib().oq_kv_read(r.handle, c.handle, C.addressof(s), a["slots"], a["T"], a["k"],
                               a["ks"], a["v"], a["vs"], a["dtype"], None)


def _attend(cache=None, **kw):
    a = dict(q=FAKE, qs=512, out=FAKE, os=512, dtype=oq.OQ_BF16, rows=4, heads=4, start=FAKE,
             prefix=FAKE, B=2, nodes=2, table=FAKE, width=4, mask=None, scale=0.1)
    a.update(kw)
    r, c = _handles()
    s = _cache(**(cache or {}))
    return oq.lib().oq_kv_attend(r.handle, c.handle, C.addressof(s), a["q"], a["qs"], a["out"],
                                 a["os"], a["dtype"], a["rows"], a["heads"], a["start"],
                                 a["prefix"], a["B"], a["nodes"], a["table"], a["width"],
                                 a["mask"], a["scale"], None)


@pytest.mark.parametrize("bad", CACHE_BAD)
def test_cache_refusals(bad):
    assert _write(cache=bad) == oq.OQ_EINVAL
    assert _read(cache=bad) == oq.OQ_EINVAL
    assert _attend(cache=bad) == oq.OQ_EINVAL


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=FAKE + 8), dict(ks=-256), dict(vs=257),
                                dict(dtype=3), dict(T=-1), dict(slots=None), dict(slots=FAKE + 4)])
def test_write_and_read_refusals(kw):
    assert _write(**kw) == oq.OQ_EINVAL
    assert _read(**kw) == oq.OQ_EINVAL
    assert _read(ks=128) == oq.OQ_EINVAL                     # tokens of the output would overlap


@pytest.mark.parametrize("kw", [
    dict(dtype=oq.OQ_F32), dict(heads=3), dict(heads=0), dict(heads=2048), dict(rows=-1),
    dict(B=-1), dict(B=65536), dict(nodes=0), dict(nodes=65), dict(width=0), dict(width=1 << 28),
    dict(scale=0.0), dict(scale=float("nan")), dict(q=None), dict(q=FAKE + 2), dict(os=504),
    dict(start=None), dict(prefix=FAKE + 2), dict(table=None), dict(mask=FAKE + 4)])
def test_attend_refusals(kw):
    assert _attend(**kw) == oq.OQ_EINVAL, kw


def test_null_handles():
    s = _cache()
    r, c = _handles()
    L = oq.lib()
    for a, b in ((None, c.handle), (r.handle, None)):
        assert L.oq_kv_write(a, b, C.addressof(s), FAKE, 256, FAKE, 256, 1, 1, FAKE,
                             None) == oq.OQ_EINVAL
    assert L.oq_kv_write(r.handle, c.handle, None, FAKE, 256, FAKE, 256, 1, 1, FAKE,
                         None) == oq.OQ_EINVAL
    assert L.oq_rope_values(None, None, None) == oq.OQ_EINVAL
    L.oq_free_rope(None)


def test_the_binding_refuses_what_it_cannot_pass_on():
    x = torch.zeros(4, 2, 128)
    rope = oq.oq_build_rope(128)
    pos = torch.zeros(4, dtype=torch.int64)
    for bad in (lambda: oq.oq_apply_rope(rope, x, pos),                         # CPU tensors
                lambda: oq.oq_apply_rope(rope, x[0], pos),
                lambda: oq.oq_apply_rope(rope, x, pos.int()),
                lambda: oq.oq_apply_rope(rope, x, pos[:3]),
                lambda: oq.oq_apply_rope(rope, x.transpose(0, 1), pos),
                lambda: oq.oq_apply_rope(rope, x, pos, k=x.double()),
                lambda: oq.KVCache.empty(2, 1, 16, 128, 4, device="cpu"),
                lambda: oq.KVCache(*[torch.zeros(2, 1, 16, 64, dtype=torch.uint8)] * 2,
                                   *[torch.zeros(2, 1, 15)] * 2, bits=4)):
        with pytest.raises(oq.OQError) as e:
            bad()
        assert e.value.code == oq.OQ_EINVAL


def test_oracle_rotation_and_packing():
    R = CO.rotation(128, 32)
    np.testing.assert_allclose(R @ R.T, np.eye(128), atol=1e-12)
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 128))
    import oracle as O
    perm, sign = O.build_rpbh(128, 0)
    np.testing.assert_allclose(x @ R.T, O.rotate(x, 32, perm, sign), atol=1e-12)
    for bits in (2, 3, 4, 6, 8):
        c = rng.integers(0, 1 << bits, (3, 128))
        assert np.array_equal(CO.unpack(CO.pack(c, bits), bits), c)
        assert np.array_equal(CO.pack(c, bits), O.pack(c.astype(np.uint8), bits))


@pytest.mark.parametrize("page,width", [(16, (1 << 27) - 15), (1024, 1 << 21), (16, 1 << 27)])
def test_attend_refuses_tables_of_too_many_tokens(page, width):
    assert _attend(cache=dict(page=page), width=width) == oq.OQ_EINVAL


def test_attend_in_place_wants_one_stride():
    """With two strides a row of out lies on another row's query."""
    assert _attend(qs=512, os=640) == oq.OQ_EINVAL
    assert "in place" in oq.lib().oq_last_error().decode()
    assert _attend(qs=640, os=512) == oq.OQ_EINVAL


def test_apply_rope_refuses_outputs_with_gradients():
    """Written outputs would lose the gradient in silence."""
    x, pos, rope = torch.zeros(4, 2, 128), torch.zeros(4, dtype=torch.int64), oq.oq_build_rope(128)
    g = torch.zeros(4, 2, 128, requires_grad=True)
    for kw in (dict(x=g, out=x), dict(x=x, k=g, out=x, k_out=x), dict(x=x, k=g, k_out=x),
               dict(x=x, out=g)):
        with pytest.raises(oq.OQError, match="gradient"):
            oq.oq_apply_rope(rope, positions=pos, **kw)
        with torch.no_grad(), pytest.raises(oq.OQError, match="CPU"):     # (and then needs a GPU)
            oq.oq_apply_rope(rope, positions=pos, **kw)


def test_a_codebook_costs_no_cache():
    """The cache's decode table (a search over 4096 factors) is made at its first use: a codebook of
    4 bits takes a seventh of the time of one of 6 bits, whose solver has four times the unknowns;
    with the search in it more than half."""
    def best(bits):
        times = []
        for _ in range(60):
            t = time.perf_counter()
            oq.oq_lloyd_max(1024, bits)
            times.append(time.perf_counter() - t)
        return min(times)
    assert best(4) <= 0.3 * best(6)


@pytest.mark.parametrize("scale", [1e300, 3.4e38, float("inf"), -1.0])
def test_attend_refuses_scales_past_fp32(scale):
    assert _attend(scale=scale) == oq.OQ_EINVAL


@pytest.mark.parametrize("T,heads", [((1 << 26) + 1, 1024), (1 << 30, 1024), ((1 << 31) - 1, 33)])
@pytest.mark.parametrize("dtype", [oq.OQ_BF16, oq.OQ_F32])
def test_cache_refuses_more_rows_than_it_counts(T, heads, dtype):
    """(One row for all tokens, stride 0, makes such calls possible.)"""
    row = heads * 128
    assert _write(cache=dict(heads=heads), T=T, dtype=dtype, ks=0, vs=0) == oq.OQ_EINVAL
    assert _read(cache=dict(heads=heads), T=T, dtype=dtype, ks=row, vs=row) == oq.OQ_EINVAL

"""Rotary positions, the quantised cache and the attention over it on the GPU, against fp64.

Tolerances.  half(t) = finfo(t).eps / 2 bounds a rounding's relative error.
  rope    fp32 products of a cosine good to 2^-22 (sincospif: 2 ulp, of turns rounded to fp32:
          2 pi 2^-25; amplitude and its product 2^-23) -> 2^-20 of the pair's length, plus the
          output's rounding.
  codes   the quantizer's parity rule: a code may differ from the oracle's by one where the unit
          value is within 1e-5 of the boundary; norms 5e-6 relative.
  read    row error <= (2^-11 + half(out) + 2^-18) |row| for 16-bit outputs (fp16 centroids: each
          is off by 2^-11 of itself at most, and R^T keeps lengths), (2^-18) |row| for fp32 ones.
  attend  queries, centroids and probabilities enter products as fp16 (2^-11 at most each, about
          2^-11 / sqrt 3 = 2.8e-4 rms).  A score of s = scale |q||k| / sqrt d typical size a is
          then off by about a sqrt(2) 2.8e-4 rms, each p by as much of itself, and a row of random
          values by sqrt(2 a^2 + 2) 2.8e-4 + half(out) / sqrt 3 of its length; the tests keep
          a <= 2 (rms 9e-4 + half/sqrt 3) and allow twice that over a whole output: 7e-3 for
          bf16, 2.5e-3 for fp16.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
import _cache_oracle as CO
from calibration_free_bit_b200 import build as B
from calibration_free_bit_b200 import oq as oq_mod

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF = {t: torch.finfo(t).eps / 2 for t in (F32, BF16, F16)}
ATTEND_TOL = {BF16: 7e-3, F16: 2.5e-3}


@pytest.fixture(scope="module")
def oq(cuda_device):
    B.build()
    return oq_mod


def gen(seed):
    return torch.Generator().manual_seed(seed)


def f64(t):
    return t.detach().cpu().double().numpy()


# ---------------------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,hq,hk,d,rot,layout,scaling,dtype", [
    (1, 1, 1, 128, 128, "half", "plain", BF16),
    (1, 32, 8, 128, 128, "interleaved", "yarn", F16),
    (7, 5, 1, 128, 32, "half", "linear", F32),
    (33, 3, 2, 256, 256, "interleaved", "ntk", F32),
    (300, 8, 2, 64, 16, "half", "plain", BF16),
    (1031, 4, 4, 128, 64, "interleaved", "plain", BF16),
    (2500, 24, 24, 128, 128, "half", "yarn", F32),
    (3, 1024, 1, 16, 16, "half", "plain", F16),
    (5, 2, 1, 1024, 512, "half", "plain", F32),
])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_matches_fp64(oq, T, hq, hk, d, rot, layout, scaling, dtype, inverse):
    g = gen(T + d)
    q, k = torch.randn(T, hq, d, generator=g).to(dtype), torch.randn(T, hk, d, generator=g).to(dtype)
    pos = torch.randint(-50, 2_000_000, (T,), generator=g)
    rope = oq.oq_build_rope(rot, layout=layout, scaling=scaling, factor=4.0, original_len=4096)
    freq, amp = rope.values()
    yq, yk = oq.oq_apply_rope(rope, q.cuda(), pos.cuda(), k=k.cuda(), inverse=inverse)
    oq.oq_check()
    for x, y in ((q, yq), (k, yk)):
        want = CO.rope(f64(x), pos.numpy(), freq, amp, rot, layout, inverse)
        size = np.abs(f64(x)).max(-1, keepdims=True) * 1.5 * amp
        bound = HALF[dtype] * np.abs(want) + 2.0 ** -20 * size
        assert np.all(np.abs(f64(y) - want) <= bound)
        assert torch.equal(y.cpu()[..., rot:], x[..., rot:])          # the rest is copied
    one = oq.oq_apply_rope(rope, q.cuda(), pos.cuda(), inverse=inverse)
    assert torch.equal(one, yq)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient_is_the_transpose_and_matches_differences(oq, layout):
    g = gen(3)
    T, H, d, rot = 9, 3, 128, 96
    x, w = torch.randn(T, H, d, generator=g).cuda(), torch.randn(T, H, d, generator=g).cuda()
    pos = torch.randint(0, 5000, (T,), generator=g).cuda()
    rope = oq.oq_build_rope(rot, layout=layout, scaling="yarn", factor=8.0, original_len=1024)
    grad = oq.oq_apply_rope(rope, w, pos, inverse=True)           # of sum(w * rope(x))
    f = lambda v: (w.double() * oq.oq_apply_rope(rope, v, pos).double()).sum().item()   # noqa: E731
    scale = w.double().norm().item() * x.double().norm().item()
    assert abs((grad.double() * x.double()).sum().item() - f(x)) <= 2.0 ** -20 * scale
    # central differences along random directions (the map is linear: only roundings remain)
    for s in range(3):
        e = torch.randn(T, H, d, generator=gen(s)).cuda()
        diff = (f(x + e) - f(x - e)) / 2
        want = (grad.double() * e.double()).sum().item()
        assert abs(diff - want) <= 2.0 ** -18 * scale


def test_rope_in_place_strided_and_padding_untouched(oq):
    g = gen(5)
    T, hq, hk, d = 13, 4, 2, 128
    qkv = torch.randn(T, hq + 2 * hk, d, generator=g).bfloat16().cuda()
    keep = qkv.clone()
    pos = torch.arange(T).cuda()
    rope = oq.oq_build_rope(64, layout="half")
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    wq, wk = oq.oq_apply_rope(rope, q.contiguous(), pos, k=k.contiguous())
    oq.oq_apply_rope(rope, q, pos, k=k, out=q, k_out=k)
    oq.oq_check()
    assert torch.equal(q, wq) and torch.equal(k, wk)
    assert torch.equal(qkv[:, hq + hk:], keep[:, hq + hk:])
    # one token's row for all positions (stride 0)
    one = keep[:1, :hq].expand(T, hq, d)
    assert torch.equal(oq.oq_apply_rope(rope, one, pos),
                       oq.oq_apply_rope(rope, one.contiguous(), pos))


# ---------------------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------------------
def make_rows(T, H, d, dtype, seed):
    g = gen(seed)
    x = torch.randn(T, H, d, generator=g) * torch.exp(torch.randn(T, H, 1, generator=g))
    x[..., 3] *= 30.0
    return x.to(dtype)


def slots_for(T, page, pages, seed):
    return torch.randperm(pages * page, generator=gen(seed))[:T]


def check_codes(got, rows, R, bits, norms):
    """The quantizer's parity rule for codes [n, d] of rows [n, d]."""
    want, norm, u = CO.quantize(rows, R, bits)
    np.testing.assert_allclose(norms, norm, rtol=5e-6)
    _, t = O.codebook(bits)
    bad = np.argwhere(got != want)
    for i, j in bad:
        assert abs(got[i, j] - want[i, j]) == 1
        assert np.min(np.abs(t - u[i, j])) <= 1e-5, (got[i, j], want[i, j], u[i, j])
    assert len(bad) <= 1 + 1e-4 * got.size


@pytest.mark.parametrize("T,H,d,h,bits,page,dtype", [
    (1, 1, 128, 128, 4, 16, BF16),
    (1, 8, 128, 64, 4, 16, F16),
    (3, 5, 128, 2, 8, 32, BF16),
    (17, 2, 128, 128, 2, 64, BF16),
    (129, 3, 128, 32, 3, 16, F16),
    (200, 1, 128, 128, 6, 128, BF16),
    (5, 40, 128, 16, 4, 1024, BF16),
    (77, 7, 256, 256, 4, 16, BF16),
    (64, 4, 256, 128, 3, 32, F16),
    (31, 2, 256, 64, 8, 64, BF16),
    (130, 1, 256, 4, 6, 16, F16),
    (9, 3, 256, 256, 2, 16, BF16),
    (33, 3, 128, 128, 4, 16, F32),
    (12, 2, 256, 32, 8, 16, F32),
    (1000, 8, 128, 128, 4, 64, BF16),
] + [(T, H, d, h, bits, 16, dtype)                    # enough rows for the tensor cores' form
     for bits in (2, 3, 4, 6, 8)
     for T, H, d, h, dtype in ((257, 1, 128, 128, BF16), (131, 3, 128, 16, F16),
                               (2600, 9, 128, 64, BF16), (256, 1, 256, 256, F16),
                               (701, 5, 256, 32, BF16))])
def test_write_and_read_match_fp64(oq, T, H, d, h, bits, page, dtype):
    pages = -(-T // page) + 2
    r, c = oq.oq_build_rpbh(d, h, 0), oq.oq_lloyd_max(d, bits)
    R = CO.rotation(d, h)
    cache = oq.KVCache.empty(pages, H, page, d, bits)
    for t in (cache.k_codes, cache.v_codes):
        t.fill_(0xA5)
    for t in (cache.k_norms, cache.v_norms):
        t.fill_(-7.0)
    k, v = make_rows(T, H, d, dtype, 1), make_rows(T, H, d, dtype, 2)
    slots = slots_for(T, page, pages, 3)
    oq.oq_kv_write(r, c, cache, k.cuda(), v.cuda(), slots.cuda())
    oq.oq_check()
    pg, at = slots.numpy() // page, slots.numpy() % page
    outs = {dt: oq.oq_kv_read(r, c, cache, slots.cuda(), out_dtype=dt) for dt in (BF16, F16, F32)}
    oq.oq_check()
    for i, (x, codes, norms) in enumerate(((k, cache.k_codes, cache.k_norms),
                                           (v, cache.v_codes, cache.v_norms))):
        packed, nn = codes.cpu().numpy(), norms.cpu().double().numpy()
        got, gn = CO.unpack(packed[pg, :, at], bits), nn[pg, :, at]
        check_codes(got.reshape(T * H, d), f64(x).reshape(T * H, d), R, bits, gn.reshape(-1))
        free = np.ones((pages, page), bool)
        free[pg, at] = False
        fp, fa = np.nonzero(free)
        assert np.all(packed[fp, :, fa] == 0xA5) and np.all(nn[fp, :, fa] == -7.0)
        want = CO.values(got, gn, R, bits)
        size = np.linalg.norm(want, axis=-1)
        for dt, out in outs.items():
            tol = 2.0 ** -18 + (0 if dt == F32 else 2.0 ** -11 + HALF[dt])
            err = np.linalg.norm(f64(out[i]) - want, axis=-1)
            assert np.all(err <= tol * size), (dt, (err / size).max())


def test_codes_are_those_of_the_activation_quantizer(oq):
    """A head's row of 128 is a row of oq_quantize_act: same rule, so the same codes up to values
    on a boundary, and the same norms up to fp32 summation."""
    T, H, d = 300, 4, 128
    r, c = oq.oq_build_rpbh(d, 64, 0), oq.oq_lloyd_max(d, 4)
    x = make_rows(T, H, d, BF16, 1).cuda()
    cache = oq.KVCache.empty(-(-T // 16), H, 16, d, 4)
    slots = torch.arange(T).cuda()
    oq.oq_kv_write(r, c, cache, x, x, slots)
    codes, s = oq.oq_quantize_act(r, c, x.view(T * H, d))
    oq.oq_check()
    got = cache.k_codes.transpose(1, 2).reshape(-1, H, d // 2)[:T].reshape(T * H, -1)
    n = cache.k_norms.transpose(1, 2).reshape(-1, H)[:T].reshape(-1)
    assert torch.equal(cache.k_codes, cache.v_codes)
    diff = (CO.unpack(got.cpu().numpy(), 4) != CO.unpack(codes.cpu().numpy(), 4)).mean()
    assert diff <= 1e-4
    torch.testing.assert_close(n, s, rtol=5e-6, atol=0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,d", [(21, 128), (300, 128), (270, 256)])
def test_padding_bad_slots_and_special_rows(oq, dtype, T, d):
    H, page = 2, 16
    pages = -(-T // page)
    r, c = oq.oq_build_rpbh(d, 128, 0), oq.oq_lloyd_max(d, 4)
    cache = oq.KVCache.empty(pages, H, page, d, 4)
    x = make_rows(T, H, d, dtype, 9)
    x[3] = 0.0                                        # an empty row: middle codes, norm 0
    slots = torch.arange(T)
    slots[5], slots[11] = -1, -1
    oq.oq_kv_write(r, c, cache, x.cuda(), x.cuda(), slots.cuda())
    oq.oq_check()
    flat = cache.k_norms.transpose(1, 2).reshape(-1, H)
    assert torch.all(flat[3] == 0) and torch.all(flat[5] == 0) and torch.all(flat[11] == 0)
    assert torch.all(cache.k_codes[0, :, 3] == 0x88) and torch.all(cache.k_codes[0, :, 5] == 0)
    k, v = oq.oq_kv_read(r, c, cache, slots.cuda(), k=torch.full((T, H, d), 3.0).to(dtype).cuda())
    assert torch.all(k[5] == 0) and torch.all(k[11] == 0) and torch.all(k[3] == 0)
    assert torch.equal(k, v)
    # the same slot read several times, and slots outside the cache
    # (in a call of the same form: few rows take another one, whose roundings differ)
    twice = slots.clone()
    twice[:4] = torch.tensor([7, 7, 0, 7])
    again, _ = oq.oq_kv_read(r, c, cache, twice.cuda(), out_dtype=dtype)
    assert torch.equal(again[0], k[7]) and torch.equal(again[3], k[7])
    before = [t.clone() for t in (cache.k_codes, cache.v_codes, cache.k_norms, cache.v_norms)]
    for bad in (pages * page, -2, 1 << 40, -(1 << 62)):
        s = torch.full((T,), -1)
        s[4] = bad
        oq.oq_kv_write(r, c, cache, x.cuda(), x.cuda(), s.cuda())
        with pytest.raises(oq.OQError) as e:
            oq.oq_check()
        assert e.value.code == oq.OQ_EDEVICE and "cache=0x1 " in str(e.value)
        out, _ = oq.oq_kv_read(r, c, cache, s.cuda(), out_dtype=dtype)
        with pytest.raises(oq.OQError):
            oq.oq_check()
        assert torch.all(out == 0)
    for a, b in zip(before, (cache.k_codes, cache.v_codes, cache.k_norms, cache.v_norms)):
        assert torch.equal(a, b)
    # infinities and NaN: their own row's norm, no other row
    y = x.clone()
    y[2, 0, 5], y[8, 1, 7] = float("inf"), float("nan")
    oq.oq_kv_write(r, c, cache, y.cuda(), y.cuda(), slots.cuda())
    oq.oq_check()
    flat2 = cache.k_norms.transpose(1, 2).reshape(-1, H)
    other = torch.ones(len(flat2), H, dtype=torch.bool, device="cuda")
    other[2, 0] = other[8, 1] = False
    assert not torch.isfinite(flat2[2, 0]) and torch.isnan(flat2[8, 1])
    assert torch.equal(flat2[other], flat[other])


@pytest.mark.parametrize("T,d", [(45, 128), (333, 128), (100, 256)])
def test_strided_rows_and_the_fused_projection(oq, T, d):
    H = 3
    r, c = oq.oq_build_rpbh(d, 64, 0), oq.oq_lloyd_max(d, 4)
    qkv = make_rows(T, 4 * H, d, BF16, 4).cuda()
    k, v = qkv[:, H:2 * H], qkv[:, 3 * H:]
    a, b = (oq.KVCache.empty(T // 16 + 2, H, 16, d, 4) for _ in range(2))
    slots = torch.randperm(T + 16, generator=gen(0))[:T].cuda()
    oq.oq_kv_write(r, c, a, k, v, slots)
    oq.oq_kv_write(r, c, b, k.contiguous(), v.contiguous(), slots)
    for x, y in ((a.k_codes, b.k_codes), (a.v_codes, b.v_codes), (a.k_norms, b.k_norms),
                 (a.v_norms, b.v_norms)):
        assert torch.equal(x, y)
    wide = torch.full((T, 3 * H, d), 5.0, dtype=F16, device="cuda")
    oq.oq_kv_read(r, c, a, slots, k=wide[:, :H], v=wide[:, H:2 * H])
    k2, v2 = oq.oq_kv_read(r, c, a, slots, out_dtype=F16)
    oq.oq_check()
    assert torch.equal(wide[:, :H], k2) and torch.equal(wide[:, H:2 * H], v2)
    assert torch.all(wide[:, 2 * H:] == 5.0)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_small_large_and_subnormal_rows(oq, dtype):
    """Rows of any size have the codes of their direction: the smallest normal and subnormal
    numbers, and rows whose squares pass fp16's range."""
    T, H, d, bits = 300, 1, 128, 4
    r, c = oq.oq_build_rpbh(d, 64, 0), oq.oq_lloyd_max(d, bits)
    cache = oq.KVCache.empty(20, H, 16, d, bits)
    x = make_rows(T, H, d, F32, 5)
    tiny = 2.0 ** -15 if dtype == F16 else 2.0 ** -30
    big = 100.0 if dtype == F16 else 2.0 ** 50
    x[::3] *= tiny
    x[1::3] *= big
    x = x.to(dtype)
    slots = torch.arange(T)
    oq.oq_kv_write(r, c, cache, x.cuda(), x.cuda(), slots.cuda())
    oq.oq_check()
    R = CO.rotation(d, 64)
    codes = CO.unpack(cache.k_codes.cpu().numpy().reshape(-1, d // 2)[:T], bits)
    norms = cache.k_norms.cpu().double().numpy().reshape(-1)[:T]
    check_codes(codes, f64(x).reshape(T, d), R, bits, norms)


def test_caches_at_16_byte_addresses(oq):
    """Code arrays that are 16- but not 32-byte aligned (a slice of a larger allocation)."""
    T, H, d, bits = 400, 1, 128, 4
    r, c = oq.oq_build_rpbh(d, 64, 0), oq.oq_lloyd_max(d, bits)
    n = 25 * H * 16 * d * bits // 8
    buf = [torch.zeros(n + 16, dtype=torch.uint8, device="cuda")[16:].view(25, H, 16, -1)
           for _ in range(2)]
    a = oq.KVCache.empty(25, H, 16, d, bits)
    b = oq.KVCache(*buf, torch.zeros_like(a.k_norms), torch.zeros_like(a.k_norms), bits=bits)
    x = make_rows(T, H, d, BF16, 6).cuda()
    slots = torch.arange(T).cuda()
    for cache in (a, b):
        oq.oq_kv_write(r, c, cache, x, x, slots)
    oq.oq_check()
    assert torch.equal(a.k_codes, b.k_codes) and torch.equal(a.v_codes, b.v_codes)
    for u, v in zip(oq.oq_kv_read(r, c, a, slots), oq.oq_kv_read(r, c, b, slots)):
        assert torch.equal(u, v)
    q = torch.randn(1, 2, d, generator=gen(1)).bfloat16().cuda()
    at = (torch.tensor([0, 1], dtype=torch.int32).cuda(),
          torch.tensor([399], dtype=torch.int32).cuda(),
          torch.arange(25, dtype=torch.int32).view(1, -1).cuda())
    assert torch.equal(oq.oq_kv_attend(r, c, a, q, *at), oq.oq_kv_attend(r, c, b, q, *at))


def test_block_rht_and_exact_marginal_handles(oq):
    """The rotation without its permutation and the f_d codebook run through the same calls."""
    T, H, d, bits = 40, 2, 128, 4
    r, c = oq.oq_build_block_rht(d, 64, 0), oq.oq_lloyd_max(d, bits, "exact")
    R = CO.rotation(d, 64, permute=False)
    cache = oq.KVCache.empty(3, H, 16, d, bits)
    x = make_rows(T, H, d, BF16, 4)
    slots = torch.arange(T)
    oq.oq_kv_write(r, c, cache, x.cuda(), x.cuda(), slots.cuda())
    k, _ = oq.oq_kv_read(r, c, cache, slots.cuda(), out_dtype=F32)
    oq.oq_check()
    codes = CO.unpack(cache.k_codes.cpu().numpy().transpose(0, 2, 1, 3).reshape(-1, H, 64)[:T], 4)
    norms = cache.k_norms.cpu().double().numpy().transpose(0, 2, 1).reshape(-1, H)[:T]
    cent = c.values()[0] * math.sqrt(d)
    z = f64(x) @ R.T
    np.testing.assert_allclose(norms, np.linalg.norm(z, axis=-1), rtol=5e-6)
    want = cent[codes] @ R * (norms / math.sqrt(d))[..., None]
    err = np.linalg.norm(f64(k) - want, axis=-1)
    assert np.all(err <= 2.0 ** -18 * np.linalg.norm(want, axis=-1))


def test_rows_past_32_bits(oq):
    """A cache of more than 2^32 bytes of codes: the last page's rows land there."""
    H, d, bits, page = 1, 256, 8, 1024
    pages = (1 << 32) // (page * 256) + 3
    r, c = oq.oq_build_rpbh(d, 64, 0), oq.oq_lloyd_max(d, bits)
    codes = torch.zeros(pages, H, page, 256, dtype=torch.uint8, device="cuda")
    norms = torch.zeros(pages, H, page, device="cuda")
    small = oq.KVCache.empty(1, H, page, d, bits)
    cache = oq.KVCache(codes, codes, norms, norms, bits=bits)     # values over keys: equal rows
    x = make_rows(5, H, d, BF16, 1).cuda()
    far = torch.tensor([pages * page - 1, 3, pages * page - 700, (1 << 24) + 5, 9]).cuda()
    near = torch.arange(5).cuda()
    oq.oq_kv_write(r, c, cache, x, x, far)
    oq.oq_kv_write(r, c, small, x, x, near)
    oq.oq_check()
    assert torch.equal(codes.view(-1, 256)[far], small.k_codes.view(-1, 256)[:5])
    assert torch.equal(norms.view(-1)[far], small.k_norms.view(-1)[:5])
    a, _ = oq.oq_kv_read(r, c, cache, far)
    b, _ = oq.oq_kv_read(r, c, small, near)
    assert torch.equal(a, b)
    # attention over the far pages
    table = torch.tensor([[pages - 1]], dtype=torch.int32).cuda()
    codes[pages - 1] = small.k_codes[0]
    norms[pages - 1] = small.k_norms[0]
    q = torch.randn(1, 2, d, generator=gen(1)).bfloat16().cuda()
    args = (torch.tensor([0, 1], dtype=torch.int32).cuda(), torch.tensor([4], dtype=torch.int32).cuda())
    got = oq.oq_kv_attend(r, c, cache, q, *args, table)
    want = oq.oq_kv_attend(r, c, small, q, *args, torch.zeros_like(table))
    oq.oq_check()
    assert torch.equal(got, want)


# ---------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------
class Serving:
    """A cache filled with random codes, ragged sequences, and the oracle's view of them."""

    def __init__(self, oq, prefixes, nodes, hq, hk, d, h, bits, page, dtype, seed, size=1.5,
                 extra_rows=0, columns=0):
        self.oq, self.hq, self.hk, self.d, self.page, self.dtype = oq, hq, hk, d, page, dtype
        rng = np.random.default_rng(seed)
        self.prefixes, self.nodes, self.bits = list(prefixes), list(nodes), bits
        total = [p + n for p, n in zip(prefixes, nodes)]
        need = [-(-t // page) for t in total]
        pages = sum(need) + 3
        order = rng.permutation(pages)
        self.table = np.full((len(total), max(need + [1]) + 1 + columns), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (pages, hk, page, d * bits // 8)
        self.codes = [rng.integers(0, 256, shape, dtype=np.uint8) for _ in range(2)]
        c, _ = O.codebook(bits)
        # norms that make the rows' own lengths |k| about sqrt d, whatever the codes drawn
        self.norms = []
        for cc in self.codes:
            rms = np.sqrt((c[CO.unpack(cc, bits)] ** 2).mean(-1))
            self.norms.append((math.sqrt(d) / rms * np.exp(0.3 * rng.standard_normal(rms.shape)))
                              .astype(np.float32))
        self.rows = sum(nodes)
        self.q = torch.from_numpy(size * rng.standard_normal((self.rows + extra_rows, hq, d))).to(dtype)
        self.start = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.mask = None
        self.rng = rng
        self.r, self.c = oq.oq_build_rpbh(d, h, 0), oq.oq_lloyd_max(d, bits)
        self.R = CO.rotation(d, h)
        self.scale = 1 / math.sqrt(d)

    def trees(self, empty=0.0):
        """Random masks: ancestors and self, or (with probability `empty`) nothing."""
        words = []
        for n in self.nodes:
            w = []
            for i in range(n):
                up = int(self.rng.integers(-1, i)) if i else -1
                m = (1 << i) | (w[up] if up >= 0 else 0)
                w.append(m)
            words += [0 if self.rng.random() < empty else m for m in w]
        self.mask = np.array(words + [0] * (len(self.q) - self.rows), dtype=np.uint64).view(np.int64)
        return self

    def visible(self, b):
        n, p = self.nodes[b], self.prefixes[b]
        see = np.ones((n, p + n), bool)
        for i in range(n):
            row = self.start[b] + i
            w = (2 << i) - 1 if self.mask is None else int(np.uint64(self.mask[row]))
            see[i, p:] = [bool((w >> j) & 1) for j in range(n)]
        return see

    def hide(self, value):
        """Put `value` in the norms of everything that no row sees (other pages, page ends)."""
        seen = np.zeros((self.norms[0].shape[0], self.page), bool)
        for b in range(len(self.nodes)):
            t = np.nonzero(self.visible(b).any(0))[0] if self.nodes[b] else np.arange(0)
            seen[self.table[b][t // self.page], t % self.page] = True
        for n in self.norms:
            n.transpose(0, 2, 1)[~seen] = value
        return self

    def gpu(self):
        cu = lambda a: torch.from_numpy(a).cuda()                         # noqa: E731
        cache = self.oq.KVCache(cu(self.codes[0]), cu(self.codes[1]), cu(self.norms[0]),
                                cu(self.norms[1]), bits=self.bits)
        return dict(r=self.r, c=self.c, cache=cache, q=self.q.cuda(), q_start=cu(self.start),
                    prefix=torch.tensor(self.prefixes, dtype=torch.int32).cuda(),
                    page_table=cu(self.table), max_nodes=max(self.nodes + [1]),
                    tree_mask=None if self.mask is None else cu(self.mask), scale=self.scale)

    def want(self, sample=None):
        """fp64 outputs [rows, hq, d] (NaN where not sampled)."""
        out = np.full((self.rows, self.hq, self.d), np.nan)
        G = self.hq // self.hk
        for b in range(len(self.nodes)):
            n, S = self.nodes[b], self.prefixes[b] + self.nodes[b]
            if n == 0:
                continue
            t = np.arange(S)
            pg, at = self.table[b][t // self.page], t % self.page
            see = self.visible(b)
            for g in (range(self.hk) if sample is None else sample):
                k, v = (CO.values(CO.unpack(c[pg, g, at], self.bits), m[pg, g, at].astype(np.float64),
                                  self.R, self.bits) for c, m in zip(self.codes, self.norms))
                for e in range(G):
                    qq = f64(self.q[self.start[b]:self.start[b] + n, g * G + e])
                    o, _ = CO.attend(qq, k, v, see, self.scale)
                    out[self.start[b]:self.start[b] + n, g * G + e] = o
        return out


def close(got, want, dtype):
    got = f64(got)[:len(want)]
    known = ~np.isnan(want).any(-1)
    assert np.all(np.isfinite(got))
    g, w = got[known], want[known]
    size = np.linalg.norm(w)
    assert np.linalg.norm(g - w) <= ATTEND_TOL[dtype] * size, np.linalg.norm(g - w) / size
    # no single row far off: 4 times the bound of the whole
    err, n = np.linalg.norm(g - w, axis=-1), np.linalg.norm(w, axis=-1)
    typical = np.sqrt((w * w).sum(-1).mean())
    assert np.all(err <= 4 * ATTEND_TOL[dtype] * np.maximum(n, typical))


ATTEND = [
    # prefixes, nodes, hq, hk, d, h, bits, page, dtype
    ([0], [1], 1, 1, 128, 128, 4, 16, BF16),                      # a first token sees itself
    ([1], [1], 4, 1, 128, 64, 4, 16, F16),
    ([15, 16, 17], [1, 1, 1], 8, 2, 128, 128, 4, 16, BF16),       # around a page's end
    ([5, 0, 333, 64], [1, 1, 1, 1], 4, 4, 128, 128, 3, 32, F16),
    ([1000], [1], 32, 8, 128, 128, 4, 16, BF16),
    ([700, 3], [1, 1], 14, 2, 128, 32, 2, 64, BF16),              # groups of 7
    ([130, 259], [1, 1], 9, 1, 128, 128, 8, 128, F16),            # a group of 9
    ([513], [1], 40, 2, 128, 128, 6, 16, BF16),                   # a group of 20
    ([300, 17], [1, 1], 4, 2, 256, 256, 4, 16, BF16),
    ([260], [1], 8, 8, 256, 64, 8, 64, F16),
    ([90, 31], [2, 5], 8, 2, 128, 128, 4, 16, BF16),              # chains
    ([0, 12, 200], [7, 1, 16], 4, 1, 128, 128, 3, 16, F16),
    ([100], [33], 8, 4, 128, 64, 4, 32, BF16),
    ([55, 1025], [64, 64], 4, 2, 128, 128, 4, 64, BF16),
    ([40], [13], 7, 1, 256, 128, 2, 16, F16),
    ([70], [64], 28, 4, 256, 128, 6, 16, BF16),
    ([500, 77], [61, 30], 16, 2, 128, 128, 8, 64, BF16),
]


# A page table that could hold this many tokens more makes a call one of much work, which is shared
# out to all SMs (few rows), instead of one for clusters.
ROOMY = 1 << 19


@pytest.mark.parametrize("case", range(len(ATTEND)))
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("roomy", [False, True])
def test_attend_matches_fp64(oq, case, tree, roomy):
    prefixes, nodes, hq, hk, d, h, bits, page, dtype = ATTEND[case]
    s = Serving(oq, prefixes, nodes, hq, hk, d, h, bits, page, dtype, seed=case,
                columns=ROOMY // page if roomy else 0)
    if tree:
        s.trees()
    s.hide(float("nan"))
    out = oq.oq_kv_attend(**s.gpu())
    oq.oq_check()
    close(out, s.want(), dtype)


@pytest.mark.parametrize("d,bits,dtype,nodes", [(128, 4, BF16, 1), (256, 3, F16, 1),
                                                (128, 8, BF16, 40)])
@pytest.mark.parametrize("hidden", [float("inf"), 3e38])
@pytest.mark.parametrize("roomy", [False, True])
def test_hidden_tokens_weigh_nothing(oq, d, bits, dtype, nodes, hidden, roomy):
    s = Serving(oq, [37, 250], [nodes, nodes], 8, 2, d, 128, bits, 16, dtype, seed=3,
                columns=ROOMY // 16 if roomy else 0).trees()
    s.hide(hidden)
    out = oq.oq_kv_attend(**s.gpu())
    oq.oq_check()
    close(out, s.want(), dtype)


@pytest.mark.parametrize("nodes", [[1, 1, 1], [2, 4, 1], [5, 9, 1], [50, 64, 3]])
@pytest.mark.parametrize("roomy", [False, True])
def test_rows_that_see_nothing_give_zeros(oq, nodes, roomy):
    s = Serving(oq, [0, 40, 0], nodes, 8, 2, 128, 128, 4, 16, BF16, seed=7,
                columns=ROOMY // 16 if roomy else 0).trees(empty=0.5)
    s.mask[:nodes[0]] = 0
    s.hide(float("nan"))
    out = oq.oq_kv_attend(**s.gpu())
    oq.oq_check()
    assert torch.all(out[:nodes[0]] == 0)
    close(out, s.want(), BF16)


@pytest.mark.parametrize("nodes,roomy", [([0, 3, 0, 2], False), ([0, 3, 0, 2], True),
                                         ([0, 40, 0, 13], False), ([0, 0, 0, 0], True)])
def test_sequences_without_rows_and_rows_behind_the_last(oq, nodes, roomy):
    s = Serving(oq, [9, 100, 33, 0], nodes, 4, 2, 128, 128, 4, 16, BF16, seed=8,
                extra_rows=6, columns=ROOMY // 16 if roomy else 0)
    a = s.gpu()
    out = torch.full_like(a["q"], 42.0)
    oq.oq_kv_attend(**a, out=out)
    oq.oq_check()
    assert torch.all(out[s.rows:] == 42.0)
    if s.rows:
        close(out[:s.rows], s.want(), BF16)


@pytest.mark.parametrize("nodes,roomy", [(1, False), (1, True), (24, False)])
def test_sequences_that_do_not_fit_are_skipped_and_reported(oq, nodes, roomy):
    s = Serving(oq, [20, 50, 60], [nodes] * 3, 4, 2, 128, 128, 4, 16, BF16, seed=9,
                columns=ROOMY // 16 if roomy else 0)
    good = oq.oq_kv_attend(**s.gpu())
    oq.oq_check()

    def run(bit, skipped=(1,), same=True, **change):
        a = s.gpu()
        a.update(change)
        out = torch.full_like(a["q"], 42.0)
        oq.oq_kv_attend(**a, out=out)
        with pytest.raises(oq.OQError) as e:
            oq.oq_check()
        assert e.value.code == oq.OQ_EDEVICE and f"attend={bit} " in str(e.value), str(e.value)
        for b in range(3):
            rows = slice(b * nodes, (b + 1) * nodes)
            if b in skipped:
                assert torch.all(out[rows] == 42.0)
            elif same:
                assert torch.equal(out[rows], good[rows])
        return out

    cu = lambda v: torch.tensor(v, dtype=torch.int32).cuda()               # noqa: E731
    run("0x2", prefix=cu([20, -1, 60]))
    run("0x2", prefix=cu([20, 1 << 30, 60]))
    run("0x2", prefix=cu([20, 2147483647, 60]))
    if nodes > 1:
        run("0x1", skipped=(0, 1, 2), max_nodes=nodes - 1)
    run("0x1", skipped=(0, 1), q_start=cu([0, -5, 2 * nodes, 3 * nodes]))
    run("0x1", skipped=(2,), q_start=cu([0, nodes, 2 * nodes, 3 * nodes + 1]))
    # a page outside the cache: its tokens are not seen, the other sequences are unharmed
    for bad in (-1, 1 << 20):
        t = s.table.copy()
        t[1, 1] = bad
        out = run("0x4", skipped=(), same=False, page_table=torch.from_numpy(t).cuda())
        assert torch.equal(out[:nodes], good[:nodes])
        assert torch.equal(out[2 * nodes:], good[2 * nodes:])
        assert torch.all(torch.isfinite(out[nodes:2 * nodes]))
        keep = s.visible
        s.visible = lambda b: keep(b) & ~((b == 1) & (np.arange(s.prefixes[b] + nodes) // 16 == 1))
        close(out, s.want(), BF16)
        s.visible = keep


@pytest.mark.parametrize("size", [1e-6, 60.0, 3e4])
def test_query_sizes(oq, size):
    """Tiny, peaked and (fp16's range apart) enormous queries: a softmax from flat to one-hot."""
    s = Serving(oq, [300], [1], 8, 2, 128, 128, 4, 16, BF16, seed=11, size=size)
    if size > 1:
        s.scale = 2.0 / size / math.sqrt(128)
    out = oq.oq_kv_attend(**s.gpu())
    oq.oq_check()
    close(out, s.want(), BF16)


def test_one_hot_softmax_and_value_sizes(oq):
    """Scores far apart (one token has all the weight), values of very different sizes."""
    s = Serving(oq, [600], [1], 4, 1, 128, 128, 4, 16, BF16, seed=12, size=40.0)
    s.norms[1] *= np.exp(3 * s.rng.standard_normal(s.norms[1].shape)).astype(np.float32)
    want = s.want()
    out = oq.oq_kv_attend(**s.gpu())
    oq.oq_check()
    # scores of size 40 are off by 40 * 4e-4 = 1.6e-2 at worst over the few tokens that matter
    err = np.linalg.norm(f64(out) - want, axis=-1)
    assert np.all(err <= 0.06 * np.linalg.norm(want, axis=-1))


@pytest.mark.parametrize("lengths,heads,nodes,bits,dtype", [
    ([3000, 17, 900, 4097, 0, 1, 2222, 128], 2, 1, 4, BF16),       # all SMs share ragged lengths
    ([2500, 1300], 2, 3, 3, F16),
    ([5000, 700], 1, 2, 8, BF16),
    ([3111, 40, 1290], 1, 33, 4, BF16),                            # many rows, many pieces
    ([2900, 128], 1, 64, 8, F16),
    ([4500], 1, 40, 2, BF16),
    ([1500, 3000], 1, 24, 6, BF16),
    ([2000, 64], 1, 17, 3, F16),
])
def test_long_and_ragged_contexts(oq, lengths, heads, nodes, bits, dtype):
    """Contexts that many workers share: every piece of every row finds its place."""
    s = Serving(oq, lengths, [nodes] * len(lengths), 2 * heads, heads, 128, 64, bits, 16, dtype,
                seed=40 + nodes, columns=ROOMY // 16).trees()
    s.hide(float("nan"))
    out = oq.oq_kv_attend(**s.gpu())
    oq.oq_check()
    close(out, s.want(), dtype)


@pytest.mark.parametrize("d,bits", [(256, 4), (256, 8)])
def test_wide_heads_over_long_contexts(oq, d, bits):
    s = Serving(oq, [1800, 33, 700], [6, 1, 4], 4, 1, d, 128, bits, 32, BF16, seed=50,
                columns=ROOMY // 32).trees()
    out = oq.oq_kv_attend(**s.gpu())
    oq.oq_check()
    close(out, s.want(), BF16)


@pytest.mark.parametrize("B,nodes,roomy", [(3, 1, False), (3, 1, True), (2, 20, False)])
def test_results_do_not_depend_on_the_run(oq, B, nodes, roomy):
    """The same call again: the same bits (no atomics decide an order)."""
    s = Serving(oq, [333, 1500, 64][:B], [nodes] * B, 8, 2, 128, 128, 4, 16, BF16, seed=13,
                columns=ROOMY // 16 if roomy else 0).trees()
    a = s.gpu()
    out = oq.oq_kv_attend(**a)
    for _ in range(5):
        assert torch.equal(oq.oq_kv_attend(**a), out)
    oq.oq_check()


def test_two_streams_and_a_captured_graph(oq):
    """Calls on two streams at once, and two graphs replayed at once."""
    cases = [Serving(oq, [900, 40], [n, n], 8, 2, 128, 128, 4, 16, BF16, seed=20 + n,
                     columns=ROOMY // 16).trees() for n in (1, 17)]
    args = [c.gpu() for c in cases]
    want = [oq.oq_kv_attend(**a) for a in args]
    torch.cuda.synchronize()
    outs = [[torch.empty_like(w) for _ in range(20)] for w in want]
    streams = [torch.cuda.Stream() for _ in args]
    for i in range(20):
        for a, o, st in zip(args, outs, streams):
            oq.oq_kv_attend(**a, out=o[i], stream=st)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        for x in o:
            assert torch.equal(x, w)
    graphs = []
    for a in args:
        o = torch.zeros_like(a["q"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            oq.oq_kv_attend(**a, out=o)
        graphs.append((g, o))
    for _ in range(5):
        for (g, o), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                o.zero_()
                g.replay()
        torch.cuda.synchronize()
        for w, (g, o) in zip(want, graphs):
            assert torch.equal(o, w)
    oq.oq_check()


def test_a_decoding_step_from_projection_to_output(oq):
    """Rotary positions, the cache's write, a drafted tree over it, the accepted tokens' read: the
    run of a serving step, against fp64 on what the cache holds; captured and replayed too."""
    Hq, Hk, d, bits, page, ctx, nodes = 8, 2, 128, 4, 16, 75, 6
    dtype = BF16
    r, c = oq.oq_build_rpbh(d, 128, 0), oq.oq_lloyd_max(d, bits)
    rope = oq.oq_build_rope(d, layout="half", scaling="yarn", factor=4.0, original_len=64)
    cache = oq.KVCache.empty(8, Hk, page, d, bits)
    pages = torch.tensor([[5, 2, 7, 0, 3, 6]], dtype=torch.int32)
    slot = lambda t: pages[0].long()[t // page] * page + t % page           # noqa: E731
    qkv = make_rows(ctx + nodes, Hq + 2 * Hk, d, dtype, 1).cuda() * 0.3
    # a tree: node 0's children 1 and 2, 3 behind 1, 4 and 5 behind 2; depth gives positions
    words = torch.tensor([0b1, 0b11, 0b101, 0b1011, 0b10101, 0b100101])
    depth = torch.tensor([0, 1, 1, 2, 2, 2])
    t = torch.arange(ctx + nodes)
    pos = torch.cat([t[:ctx], ctx + depth]).cuda()
    slots = slot(t).cuda()
    start = torch.tensor([0, nodes], dtype=torch.int32).cuda()
    prefix = torch.tensor([ctx], dtype=torch.int32).cuda()
    table, mask = pages.cuda(), words.cuda()
    out = torch.zeros(nodes, Hq, d, dtype=dtype, device="cuda")
    q, k = torch.zeros_like(qkv[:, :Hq]), torch.zeros_like(qkv[:, :Hk])

    def step():
        oq.oq_apply_rope(rope, qkv[:, :Hq], pos, k=qkv[:, Hq:Hq + Hk], out=q, k_out=k)
        oq.oq_kv_write(r, c, cache, k, qkv[:, Hq + Hk:], slots)
        oq.oq_kv_attend(r, c, cache, q[ctx:], start, prefix, table, max_nodes=nodes,
                        tree_mask=mask, out=out)
        return oq.oq_kv_read(r, c, cache, slots, out_dtype=F32)

    kh, vh = step()
    oq.oq_check()
    first = out.clone()
    freq, amp = rope.values()
    qr = CO.rope(f64(qkv[:, :Hq]), f64(pos), freq, amp, d, "half")
    assert np.linalg.norm(f64(q) - qr) <= 2 * HALF[dtype] * np.linalg.norm(qr)
    see = np.ones((nodes, ctx + nodes), bool)
    for i in range(nodes):
        see[i, ctx:] = [(int(words[i]) >> j) & 1 for j in range(nodes)]
    want = np.zeros((nodes, Hq, d))
    for h in range(Hq):
        g = h // (Hq // Hk)
        want[:, h], _ = CO.attend(f64(q[ctx:, h]), f64(kh[:, g]), f64(vh[:, g]), see, d ** -0.5)
    close(out, want, dtype)
    # the codes stand for rows close to those written (4 bits: about 10 % of a row's length)
    back = np.linalg.norm(f64(kh) - f64(k)) / np.linalg.norm(f64(k))
    assert back < 0.2
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    out.zero_()
    for x in (cache.k_codes, cache.v_codes):
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    oq.oq_check()
    assert torch.equal(out, first)


def test_timing_names_the_new_kernels(oq):
    s = Serving(oq, [50], [1], 4, 2, 128, 128, 4, 16, BF16, seed=1)
    a = s.gpu()
    x = torch.randn(4, 2, 128, dtype=BF16, device="cuda")
    slots = torch.arange(4).cuda()
    rope = oq.oq_build_rope(128)
    cache = oq.KVCache.empty(1, 2, 16, 128, 4)
    oq.oq_timing_enable(True)
    try:
        oq.oq_apply_rope(rope, x, slots)
        oq.oq_kv_write(s.r, s.c, cache, x, x, slots)
        oq.oq_kv_read(s.r, s.c, cache, slots)
        oq.oq_kv_attend(**a)
        names = [n for n, ms in oq.oq_timing_collect()]
    finally:
        oq.oq_timing_enable(False)
    assert names == ["rope", "kv_write", "kv_read", "kv_attend"]


# ---------------------------------------------------------------------------------------
# the forms of larger calls: rows on the tensor cores, row tiles of 16 side by side
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("bits", [2, 3, 4, 6, 8])
@pytest.mark.parametrize("T,H,d,h,dtype", [(1400, 3, 128, 16, F16), (4097, 1, 256, 256, F16),
                                           (1371, 3, 256, 32, BF16)])
def test_write_and_read_many_rows(oq, T, H, d, h, bits, dtype):
    test_write_and_read_match_fp64(oq, T, H, d, h, bits, 32, dtype)


@pytest.mark.parametrize("d", [128, 256])
def test_padding_and_strides_of_many_rows(oq, d):
    test_padding_bad_slots_and_special_rows(oq, BF16, 2100, d)
    test_strided_rows_and_the_fused_projection(oq, 1400, d)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_small_large_and_misaligned_rows_of_a_large_call(oq, dtype):
    """Rows of all sizes, in code arrays that are 16- but not 32-byte aligned."""
    T, d, bits = 4200, 128, 4
    r, c = oq.oq_build_rpbh(d, 64, 0), oq.oq_lloyd_max(d, bits)
    a = oq.KVCache.empty(263, 1, 16, d, bits)
    n = a.k_codes.numel()
    buf = [torch.zeros(n + 16, dtype=torch.uint8, device="cuda")[16:].view(263, 1, 16, -1)
           for _ in range(2)]
    b = oq.KVCache(*buf, torch.zeros_like(a.k_norms), torch.zeros_like(a.k_norms), bits=bits)
    x = make_rows(T, 1, d, F32, 5)
    x[::3] *= 2.0 ** -15 if dtype == F16 else 2.0 ** -30
    x[1::3] *= 100.0 if dtype == F16 else 2.0 ** 50
    x = x.to(dtype)
    slots = torch.arange(T).cuda()
    for cache in (a, b):
        oq.oq_kv_write(r, c, cache, x.cuda(), x.cuda(), slots)
    oq.oq_check()
    assert torch.equal(a.k_codes, b.k_codes) and torch.equal(a.v_codes, b.v_codes)
    for u, v in zip(oq.oq_kv_read(r, c, a, slots), oq.oq_kv_read(r, c, b, slots)):
        assert torch.equal(u.view(torch.int16), v.view(torch.int16))      # NaN of rows with infinities
    fits = torch.isfinite(x).all(-1).view(-1).numpy()                     # fp16 has no 100 times some
    assert fits.mean() > 0.9
    codes = CO.unpack(a.k_codes.cpu().numpy().reshape(-1, d // 2)[:T], bits)
    check_codes(codes[fits], f64(x).reshape(T, d)[fits], CO.rotation(d, 64), bits,
                a.k_norms.cpu().double().numpy().reshape(-1)[:T][fits])


@pytest.mark.parametrize("bits", [2, 3, 4, 6, 8])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("group,nodes", [(4, [7, 2, 8]), (1, [33, 9]), (3, [1, 11])])
@pytest.mark.parametrize("roomy", [False, True])
def test_row_tiles_side_by_side(oq, bits, dtype, group, nodes, roomy):
    """17 to 33 rows a key head: two tiles of 16, the second partly filled, or one of 128."""
    s = Serving(oq, [70, 0, 301][:len(nodes)], nodes, 2 * group, 2, 128, 64, bits, 16, dtype,
                seed=60 + bits, columns=ROOMY // 16 if roomy else 0).trees(empty=0.1)
    s.hide(float("nan"))
    out = oq.oq_kv_attend(**s.gpu())
    oq.oq_check()
    close(out, s.want(), dtype)


@pytest.mark.parametrize("bits,dtype", [(2, F16), (3, BF16), (4, F16), (6, F16), (8, BF16)])
def test_many_rows_of_many_sequences(oq, bits, dtype):
    """Enough rows that a joining warp takes several: ends of tiles, idle sequences between."""
    nodes = [64, 0, 37, 1, 64, 5, 64, 63]
    s = Serving(oq, [300, 5, 0, 77, 129, 1000, 64, 3], nodes, 18, 2, 128, 128, bits, 16, dtype,
                seed=70 + bits, extra_rows=3).trees(empty=0.05)
    s.hide(float("inf"))
    a = s.gpu()
    out = torch.full_like(a["q"], 42.0)
    oq.oq_kv_attend(**a, out=out)
    oq.oq_check()
    assert torch.all(out[s.rows:] == 42.0)
    close(out[:s.rows], s.want(), dtype)


@pytest.mark.parametrize("bits", [2, 3, 4, 6, 8])
@pytest.mark.parametrize("length,nodes,dtype", [(500, 61, BF16), (130, 40, F16)])
def test_several_pieces_of_many_rows_a_worker(oq, bits, length, nodes, dtype):
    """Short segments of many rows: a worker goes from one to the next several times.  The same
    bits every time, and (two key heads of them) the formula's values."""
    s = Serving(oq, [length + 7 * b for b in range(16)], [nodes] * 16, 32, 8, 128, 128, bits, 64,
                dtype, seed=80 + bits).trees()
    s.hide(float("nan"))
    a = s.gpu()
    out = oq.oq_kv_attend(**a)
    for _ in range(4):
        assert torch.equal(oq.oq_kv_attend(**a), out)
    oq.oq_check()
    close(out, s.want(sample=[0, 7]), dtype)


@pytest.mark.parametrize("nodes,roomy,dtype", [(1, False, BF16), (3, True, F16), (40, False, BF16)])
def test_attention_in_place(oq, nodes, roomy, dtype):
    s = Serving(oq, [300, 41], [nodes] * 2, 8, 2, 128, 128, 4, 16, dtype, seed=91,
                columns=ROOMY // 16 if roomy else 0).trees()
    a = s.gpu()
    want = oq.oq_kv_attend(**a)
    oq.oq_kv_attend(**a, out=a["q"])
    oq.oq_check()
    assert torch.equal(a["q"], want)


@pytest.mark.parametrize("hq,hk,nodes,dtype", [(1024, 1, 2, BF16), (1024, 1, 2, F16),
                                               (1024, 1024, 1, BF16), (1024, 512, 20, BF16)])
@pytest.mark.parametrize("roomy", [False, True])
def test_the_most_heads(oq, hq, hk, nodes, dtype, roomy):
    s = Serving(oq, [37], [nodes], hq, hk, 128, 128, 4, 16, dtype, seed=92,
                columns=ROOMY // 16 if roomy else 0).trees()
    out = oq.oq_kv_attend(**s.gpu())
    oq.oq_check()
    close(out, s.want(sample=sorted({0, hk // 2, hk - 1})), dtype)

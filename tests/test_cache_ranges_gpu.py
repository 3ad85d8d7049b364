"""Attention over the quantised cache where norms, scores and masks reach their ends.  Oracle and
tolerances: test_cache_gpu.py."""
import numpy as np
import pytest
import torch

import _cache_oracle as CO
import oracle as O
from test_cache_gpu import (BF16, F16, ROOMY, Serving, close, f64,  # noqa: F401  (oq: a fixture)
                            make_rows, oq)

pytestmark = pytest.mark.gpu


def first_node_only(s):
    """Every row sees its prefix and node 0; the other nodes are hidden from all."""
    s.mask = np.concatenate([np.full(n, 1) for n in s.nodes]).astype(np.int64)
    return s


@pytest.mark.parametrize("bits,nodes,dtype", [(2, 40, BF16), (3, 9, BF16), (4, 40, BF16),
                                              (4, 2, F16), (6, 33, BF16), (8, 40, BF16)])
@pytest.mark.parametrize("hidden", [1e6, 1e7, 1e30, 3e38])
def test_hidden_norms_leave_their_neighbours_alone(oq, bits, nodes, dtype, hidden):  # noqa: F811
    """Large finite norms of hidden nodes right behind the prefix, in the same tile and the same 32
    tokens as visible ones."""
    s = first_node_only(Serving(oq, [37, 250, 0], [nodes] * 3, 8, 2, 128, 128, bits, 16, dtype,
                                seed=100 + bits))
    s.hide(hidden)
    out = oq.oq_kv_attend(**s.gpu())
    oq.oq_check()
    close(out, s.want(), dtype)


@pytest.mark.parametrize("bits,nodes,dtype", [(2, 40, BF16), (4, 40, BF16), (4, 2, F16),
                                              (8, 40, BF16), (8, 1, BF16)])
@pytest.mark.parametrize("roomy", [False, True])
def test_a_loud_key_leaves_its_neighbours_alone(oq, bits, nodes, dtype, roomy):  # noqa: F811
    """One visible key 1e6 times as long as the others: rows that it points away from have the
    softmax of the others, rows that it points to have its value."""
    s = Serving(oq, [37, 250], [nodes] * 2, 8, 2, 128, 128, bits, 16, dtype, seed=110 + bits,
                columns=ROOMY // 16 if roomy else 0)
    for b in range(2):
        s.norms[0][s.table[b][0], :, 5] *= 1e6
    want = s.want()
    out = oq.oq_kv_attend(**s.gpu())
    oq.oq_check()
    close(out, want, dtype)


@pytest.mark.parametrize("bits,nodes", [(4, 40), (8, 40), (4, 3)])
def test_keys_of_all_lengths(oq, bits, nodes):  # noqa: F811
    """Key norms spread over four orders of magnitude within every 32 tokens."""
    s = Serving(oq, [300, 77], [nodes] * 2, 8, 2, 128, 128, bits, 16, BF16, seed=120 + bits, size=0.5)
    s.norms[0] *= np.exp(s.rng.uniform(-9.0, 1.0, s.norms[0].shape)).astype(np.float32)
    out = oq.oq_kv_attend(**s.gpu())
    oq.oq_check()
    close(out, s.want(), BF16)


@pytest.mark.parametrize("factor", [1e-34, 1e12])
def test_groups_of_tiny_and_large_keys(oq, factor):  # noqa: F811
    """All keys short or long, with queries that bring the scores back: the same softmax."""
    s = Serving(oq, [300, 77], [40, 40], 8, 2, 128, 128, 4, 16, BF16, seed=130)
    s.norms[0] = (s.norms[0] * factor).astype(np.float32)
    s.q = (s.q.double() / factor).to(BF16)
    out = oq.oq_kv_attend(**s.gpu())
    oq.oq_check()
    close(out, s.want(), BF16)


@pytest.mark.parametrize("d,nodes", [(128, 1), (128, 3), (256, 2), (128, 40)])
@pytest.mark.parametrize("roomy", [False, True])
def test_scores_far_below_zero(oq, d, nodes, roomy):  # noqa: F811
    """Rows that see one token have its value, however low its score (here down to -1e34)."""
    s = Serving(oq, [0] * 5, [nodes] * 5, 8, 2, d, 128, 4, 16, BF16, seed=140, size=1e16,
                columns=ROOMY // 16 if roomy else 0)
    s.norms[0] = (s.norms[0] * 1e16).astype(np.float32)
    s.mask = np.concatenate([1 << np.arange(n) for n in s.nodes]).astype(np.int64)
    out = oq.oq_kv_attend(**s.gpu())
    oq.oq_check()
    close(out, s.want(), BF16)


@pytest.mark.parametrize("T,H,d,h,bits,dtype", [
    (20000, 4, 128, 128, 2, BF16), (12000, 4, 256, 128, 2, F16), (20000, 4, 128, 32, 3, F16),
    (20000, 4, 128, 128, 4, BF16), (9000, 4, 256, 256, 4, BF16), (9000, 4, 128, 64, 6, BF16),
    (5000, 4, 256, 128, 6, F16),                                  # the tensor cores' form
    (1000, 4, 128, 128, 2, BF16), (500, 4, 256, 64, 4, F16), (1000, 4, 128, 128, 6, F16),
    (1000, 4, 128, 128, 8, BF16), (500, 4, 256, 256, 8, BF16),    # a warp a row
    (20000, 4, 128, 128, 4, torch.float32), (6000, 4, 256, 64, 8, torch.float32)])
def test_codes_are_the_nearest_centroids(oq, T, H, d, h, bits, dtype):  # noqa: F811
    """Every code is the fp64 oracle's, those beside a boundary too (of values more than 1e-13 from
    one), and so the same in calls of any size.  (At 8 bits large calls of 16-bit rows have one code
    more or less there.)"""
    rows = make_rows(T, H, d, dtype, 7)
    r, c = oq.oq_build_rpbh(d, h, 0), oq.oq_lloyd_max(d, bits)
    cache = oq.KVCache.empty(-(-T // 16), H, 16, d, bits)
    oq.oq_kv_write(r, c, cache, rows.cuda(), rows.cuda(), torch.arange(T).cuda())
    oq.oq_check()
    assert torch.equal(cache.k_codes, cache.v_codes)
    packed = cache.k_codes.transpose(1, 2).reshape(-1, H, d * bits // 8)[:T].cpu().numpy()
    R, t = CO.rotation(d, h), O.codebook(bits)[1]
    for a in range(0, T, 1000):
        want, _, u = CO.quantize(f64(rows[a:a + 1000]), R, bits)
        got = CO.unpack(packed[a:a + 1000], bits)
        for i in np.argwhere(got != want):
            assert np.abs(t - u[tuple(i)]).min() <= 1e-13, (a, i, u[tuple(i)])


@pytest.mark.parametrize("T", [50, 5000])
def test_rows_of_few_distinct_values(oq, T):  # noqa: F811
    """Rows whose rotation has exact zeros, on the middle boundary: the upper code, as the oracle's."""
    d, bits = 128, 4
    rows = torch.zeros(T, 1, d)
    rows[torch.arange(T), 0, torch.arange(T) % d] = 3.0
    rows[::3] = 1.0
    r, c = oq.oq_build_rpbh(d, 64, 0), oq.oq_lloyd_max(d, bits)
    cache = oq.KVCache.empty(-(-T // 16), 1, 16, d, bits)
    x = rows.to(BF16).cuda()
    oq.oq_kv_write(r, c, cache, x, x, torch.arange(T).cuda())
    oq.oq_check()
    got = CO.unpack(cache.k_codes.view(-1, d // 2)[:T].cpu().numpy(), bits)
    z = f64(rows[:, 0]) @ CO.rotation(d, 64).T
    z[np.abs(z) < 1e-12] = 0.0                                    # (fp64's own roundings)
    u = z / np.linalg.norm(z, axis=-1, keepdims=True) * np.sqrt(d)
    t = O.codebook(bits)[1].copy()
    t[len(t) // 2] = 0.0
    assert np.array_equal(got, np.searchsorted(t, u, side="right"))


@pytest.mark.parametrize("T,dtype", [(300, BF16), (300, torch.float32), (5000, BF16)])
def test_rows_with_one_huge_element(oq, T, dtype):  # noqa: F811
    """An element 1e7 times the others: its block has codes far from a boundary, the others' blocks lie
    within 1e-5 of the middle one and have either of its codes."""
    d, h, bits = 128, 32, 4
    rows = torch.randn(T, 1, d, generator=torch.Generator().manual_seed(8))
    rows[torch.arange(T), 0, torch.arange(T) % d] = 1e7
    rows = rows.to(dtype)
    r, c = oq.oq_build_rpbh(d, h, 0), oq.oq_lloyd_max(d, bits)
    cache = oq.KVCache.empty(-(-T // 16), 1, 16, d, bits)
    oq.oq_kv_write(r, c, cache, rows.cuda(), rows.cuda(), torch.arange(T).cuda())
    oq.oq_check()
    got = CO.unpack(cache.k_codes.view(-1, d // 2)[:T].cpu().numpy(), bits)
    want, norm, u = CO.quantize(f64(rows[:, 0]), CO.rotation(d, h), bits)
    np.testing.assert_allclose(cache.k_norms.view(-1)[:T].cpu().double().numpy(), norm, rtol=5e-6)
    near = np.abs(u) <= 1e-5
    assert near.mean() > 0.7 and np.array_equal(got[~near], want[~near])
    assert np.all((got[near] == 7) | (got[near] == 8))

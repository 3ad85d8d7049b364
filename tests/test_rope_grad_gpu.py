"""Gradients through oq_apply_rope by autograd, against the transpose in fp64 and against differences.
Tolerances as for the forward pass (test_cache_gpu.py): 2^-20 of a pair's length and a rounding."""
import numpy as np
import pytest
import torch

import _cache_oracle as CO
from test_cache_gpu import BF16, F16, F32, HALF, f64, gen, oq  # noqa: F401  (oq: a fixture)

pytestmark = pytest.mark.gpu


def within(got, x, pos, rope, layout, inverse, dtype):
    freq, amp = rope.values()
    want = CO.rope(f64(x), f64(pos).astype(np.int64), freq, amp, rope.rot_dim, layout, inverse)
    size = np.abs(f64(x)).max(-1, keepdims=True) * 1.5 * amp
    assert np.all(np.abs(f64(got) - want) <= HALF[dtype] * np.abs(want) + 2.0 ** -20 * size)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T", [1, 37])
def test_gradients_of_queries_and_keys(oq, dtype, layout, inverse, T):  # noqa: F811
    g = gen(T)
    rope = oq.oq_build_rope(64, layout=layout, scaling="yarn", factor=4.0, original_len=512)
    q, k, wq, wk = (torch.randn(T, h, 128, generator=g).to(dtype).cuda() for h in (4, 2, 4, 2))
    pos = torch.randint(-10, 70000, (T,), generator=g).cuda()
    q.requires_grad_(), k.requires_grad_()
    yq, yk = oq.oq_apply_rope(rope, q, pos, k=k, inverse=inverse)
    with torch.no_grad():
        zq, zk = oq.oq_apply_rope(rope, q, pos, k=k, inverse=inverse)
    assert torch.equal(yq, zq) and torch.equal(yk, zk) and not zq.requires_grad
    gq, gk = torch.autograd.grad((yq, yk), (q, k), (wq, wk))
    oq.oq_check()
    within(gq, wq, pos, rope, layout, not inverse, dtype)
    within(gk, wk, pos, rope, layout, not inverse, dtype)
    # one tensor alone, one output unused, one input without a gradient: the same values
    assert torch.equal(torch.autograd.grad(oq.oq_apply_rope(rope, q, pos, inverse=inverse), q, wq)[0], gq)
    yq, yk = oq.oq_apply_rope(rope, q, pos, k=k, inverse=inverse)
    a, b = torch.autograd.grad(yk, (q, k), wk, allow_unused=True)
    assert a is None and torch.equal(b, gk)
    yq, yk = oq.oq_apply_rope(rope, q, pos, k=k.detach(), inverse=inverse)
    assert yq.requires_grad and not yk.requires_grad
    assert torch.equal(torch.autograd.grad(yq, q, wq)[0], gq)


def test_gradients_match_differences(oq):  # noqa: F811
    """The map is linear: differences along a direction leave only roundings."""
    g, T = gen(1), 9
    rope = oq.oq_build_rope(96, layout="half", scaling="linear", factor=3.0)
    x, w, e = (torch.randn(T, 3, 128, generator=g).cuda() for _ in range(3))
    pos = torch.randint(0, 5000, (T,), generator=g).cuda()
    x.requires_grad_()
    (w * oq.oq_apply_rope(rope, x, pos)).sum().backward()
    f = lambda v: (w.double() * oq.oq_apply_rope(rope, v, pos).double()).sum().item()    # noqa: E731
    with torch.no_grad():
        diff = (f(x + e) - f(x - e)) / 2
    want = (x.grad.double() * e.double()).sum().item()
    assert abs(diff - want) <= 2.0 ** -18 * w.double().norm().item() * e.double().norm().item()


def test_gradients_of_any_layout_and_of_shared_inputs(oq):  # noqa: F811
    """Gradients that come expanded, strided or misaligned; a slice of a fused projection; one token's
    row for all positions; the second derivative."""
    T, H, d = 11, 2, 64
    rope = oq.oq_build_rope(d, layout="interleaved")
    pos = torch.arange(T).cuda()
    x = torch.randn(T, 3 * H, d, generator=gen(2)).cuda().requires_grad_()
    q, k = x[:, :H], x[:, H:2 * H]
    yq, yk = oq.oq_apply_rope(rope, q, pos, k=k)
    (yq.sum() + yk.transpose(0, 1).flatten()[1:].square().sum()).backward()
    with torch.no_grad():
        gk = 2 * yk
        gk[0, 0, 0] = 0
        want = oq.oq_apply_rope(rope, torch.ones_like(yq), pos, k=gk, inverse=True)
    assert torch.equal(x.grad[:, :H], want[0]) and torch.all(x.grad[:, 2 * H:] == 0)
    torch.testing.assert_close(x.grad[:, H:2 * H], want[1], rtol=0, atol=0)
    one = torch.randn(1, H, d, generator=gen(3)).cuda().requires_grad_()
    y = oq.oq_apply_rope(rope, one.expand(T, H, d), pos)
    g1, = torch.autograd.grad(y.square().sum(), one, create_graph=True)
    torch.testing.assert_close(g1, 2 * T * one, rtol=1e-5, atol=1e-5)     # turns keep lengths
    g2, = torch.autograd.grad(g1.sum(), one)
    torch.testing.assert_close(g2, torch.full_like(one, 2.0 * T), rtol=1e-5, atol=1e-5)
    empty = torch.zeros(0, H, d, device="cuda", requires_grad=True)
    oq.oq_apply_rope(rope, empty, pos[:0]).sum().backward()
    assert empty.grad.shape == empty.shape
    oq.oq_check()


def test_gradients_on_a_stream_and_in_a_captured_graph(oq):  # noqa: F811
    T, H, d = 300, 4, 128
    rope = oq.oq_build_rope(d)
    pos = torch.arange(T).cuda()
    x, w = (torch.randn(T, H, d, generator=gen(s)).bfloat16().cuda() for s in (4, 5))
    x.requires_grad_()

    def step():
        return torch.autograd.grad(oq.oq_apply_rope(rope, x, pos), x, w)[0]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    oq.oq_check()


def test_the_most_tokens(oq):  # noqa: F811
    """2^31 - 1 tokens of one head of 16, one row for all of them (86 GB of outputs and positions)."""
    T = 2 ** 31 - 1
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 * 2 ** 30:
        pytest.skip("needs 100 GB of free memory")
    rope = oq.oq_build_rope(16)
    x = torch.randn(1, 1, 16, generator=gen(0)).bfloat16().cuda()
    pos = torch.arange(T, device="cuda")
    y = oq.oq_apply_rope(rope, x.expand(T, 1, 16), pos)
    oq.oq_check()
    for at in (0, 1, 12345, 2 ** 30, T - 3000):
        n = min(3000, T - at)
        want = oq.oq_apply_rope(rope, x.expand(n, 1, 16), pos[at:at + n].clone())
        assert torch.equal(y[at:at + n], want)
    del y, pos
    torch.cuda.empty_cache()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("far", [100, 10 ** 6])
def test_positions_are_as_exact_as_fp32_products(oq, layout, far):  # noqa: F811
    """The error of fp32 rows over all pairs, rms, against fp64.  Cosine and sine within an ulp (2^-24
    rms of their size at most, 2^-24 / sqrt 2 on the whole), two products and a sum: rounded to nearest
    each adds at most 2^-24 / sqrt 3 of what it rounds: below 2^-24 (1/2 + 2/3)^(1/2) = 6.5e-8 of a
    pair's length over sqrt 2 a coordinate, 4.6e-8."""
    T, H, d = 2000, 4, 128
    x = torch.randn(T, H, d, generator=gen(6)).cuda()
    pos = torch.randint(0, far, (T,), generator=gen(7)).cuda()
    rope = oq.oq_build_rope(d, layout=layout)
    y = oq.oq_apply_rope(rope, x, pos)
    oq.oq_check()
    want = CO.rope(f64(x), f64(pos).astype(np.int64), rope.values()[0], 1.0, d, layout)
    assert np.linalg.norm(f64(y) - want) <= 5e-8 * np.linalg.norm(want)

"""Rotary positions against the fp64 definition.

Bound per element: the output's rounding u |ref|, and fp32 arithmetic -- the angle's fraction
of a turn rounded to fp32 (2^-25 turns: 2^-22 radians), cos and sin within 2 ulp, two products
and a sum -- 2^-20 of the pair's absolute sum.
"""
import numpy as np
import pytest

import synthetic
from gpu_util import to_f64, torch_dtype
from oracle import operators as ops

pytestmark = pytest.mark.gpu

F32, BF16, F16 = synthetic.F32, synthetic.BF16, synthetic.F16
U = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}


@pytest.fixture(scope="module")
def eq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import group_equivariant_linear_amd as eq
    eq.load_library()
    return eq


def check(eq, dt, T, N, H, K, d, rot, layout, inverse=False, scaling="plain", magnitude=1.0, place="apart", odd=False,
          seed=0, top=5000):
    """place: outputs apart from the inputs, in place, or slices of one wide buffer (odd: at no vector boundary)."""
    import torch
    g = torch.Generator().manual_seed(seed)
    kind = {"plain": eq.EQL_ROTARY_PLAIN, "linear": eq.EQL_ROTARY_LINEAR, "raised": eq.EQL_ROTARY_RAISED_BASE,
            "banded": eq.EQL_ROTARY_BANDED}[scaling]
    plan = eq.eqlinear_rotary_plan(N, H, K, d, rot, eq.EQL_ROTARY_INTERLEAVED if layout else eq.EQL_ROTARY_HALF,
                                   {F32: eq.EQL_F32, BF16: eq.EQL_BF16, F16: eq.EQL_F16}[dt], scaling=kind, factor=4.0,
                                   context=1024.0, magnitude=magnitude)
    tdt, W = torch_dtype(dt), (H + K) * d * N + (3 if odd else 0)
    buf = torch.randn(T, W, generator=g).to(tdt).cuda()
    at = 3 if odd else 0

    def views(b):
        return (b.as_strided((T, H, d, N), (W, d * N, N, 1), at),
                b.as_strided((T, K, d, N), (W, d * N, N, 1), at + H * d * N))

    q, k = views(buf) if place != "apart" else tuple(v.contiguous() for v in views(buf))
    pos = torch.randint(-top, top, (T,), generator=g, dtype=torch.int32).cuda()
    qn, kn, p = to_f64(q), to_f64(k), pos.cpu().numpy().astype(np.float64)
    if place == "inside":
        qo, ko = q, k
    else:
        out = torch.full((T, W), 3.0, dtype=tdt, device="cuda")
        qo, ko = views(out) if place == "wide" else tuple(torch.empty_like(v) for v in (q, k))
    eq.eqlinear_rotary(plan, q, k, pos, qo, ko, inverse=inverse)
    torch.cuda.synchronize()
    f = ops.rotary_frequencies(rot, scaling=scaling, factor=4.0, context=1024.0)
    for x, y in ((qn, to_f64(qo)), (kn, to_f64(ko))):
        ref = ops.rotary(x, p, f, rot, bool(layout), magnitude, inverse)
        size = np.abs(x).copy()
        for j in range(rot // 2):
            a, b = (2 * j, 2 * j + 1) if layout else (j, j + rot // 2)
            size[:, :, a] = size[:, :, b] = magnitude * (np.abs(x[:, :, a]) + np.abs(x[:, :, b]))
        size[:, :, rot:] = 0
        assert np.all(np.abs(y - ref) <= U[dt] * (1 + 2.0 ** -10) * np.abs(ref) + 2.0 ** -20 * size)
        assert np.array_equal(y[:, :, rot:], x[:, :, rot:])  # the rest of the head passes through
    if place == "wide" and odd:
        assert torch.all(out[:, :3] == 3.0)


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("N,d,rot", [(8, 8, 8), (8, 8, 6), (7, 16, 16), (1, 64, 64), (1, 65, 34), (2, 5, 4), (3, 2, 2),
                                     (4, 6, 2), (5, 9, 8), (16, 8, 4), (1, 3, 2), (12, 10, 10)])
def test_sizes(eq, dt, layout, N, d, rot):
    check(eq, dt, 37, N, 3, 2, d, rot, layout, seed=N)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("place", ["inside", "wide", "apart"])
@pytest.mark.parametrize("odd", [False, True])
def test_places(eq, dt, layout, place, odd):
    check(eq, dt, 29, 8, 3, 1, 8, 6, layout, place=place, odd=odd)
    check(eq, dt, 5, 7, 2, 2, 4, 4, layout, place=place, odd=odd)


@pytest.mark.parametrize("scaling", ["plain", "linear", "raised", "banded"])
@pytest.mark.parametrize("inverse", [False, True])
def test_scalings(eq, scaling, inverse):
    check(eq, F32, 64, 4, 2, 2, 32, 32, 0, inverse=inverse, scaling=scaling, magnitude=1.25)
    check(eq, F32, 64, 4, 2, 2, 32, 2, 1, inverse=inverse, scaling=scaling)


@pytest.mark.parametrize("T", [1, 2, 3, 1000])
@pytest.mark.parametrize("H,K", [(1, 1), (12, 4), (2, 7)])
def test_token_and_head_counts(eq, T, H, K):
    check(eq, BF16, T, 8, H, K, 8, 8, 0, seed=T)
    check(eq, F16, T, 3, H, K, 6, 4, 1, seed=T)


def test_far_positions(eq):
    """Positions over the whole int32 range: the angle keeps its fraction of a turn."""
    check(eq, F32, 200, 4, 1, 1, 16, 16, 0, top=2 ** 31 - 1)


def test_queries_alone_and_head_major(eq):
    """No keys; and heads that lie one after the other, each with all its tokens."""
    import torch
    plan = eq.eqlinear_rotary_plan(8, 3, 3, 8, 8, eq.EQL_ROTARY_HALF, eq.EQL_F32)
    x = torch.randn(3, 20, 8, 8).cuda()
    pos = torch.arange(20, dtype=torch.int32).cuda()
    y = torch.empty_like(x)
    eq.eqlinear_rotary(plan, x.transpose(0, 1), None, pos, y.transpose(0, 1), None)
    torch.cuda.synchronize()
    ref = ops.rotary(to_f64(x.transpose(0, 1)), np.arange(20.0), ops.rotary_frequencies(8), 8, False)
    assert np.max(np.abs(to_f64(y.transpose(0, 1)) - ref)) < 1e-5


def test_inverse_is_the_gradient(eq):
    """<R x, y> = <x, R^T y> to fp32 rounding."""
    import torch
    plan = eq.eqlinear_rotary_plan(7, 2, 2, 6, 4, eq.EQL_ROTARY_INTERLEAVED, eq.EQL_F32, magnitude=1.3)
    x, y = torch.randn(50, 2, 6, 7).cuda(), torch.randn(50, 2, 6, 7).cuda()
    pos = torch.arange(50, dtype=torch.int32).cuda() * 77
    rx, ry = torch.empty_like(x), torch.empty_like(y)
    eq.eqlinear_rotary(plan, x, None, pos, rx, None)
    eq.eqlinear_rotary(plan, y, None, pos, ry, None, inverse=True)
    a, b = (rx.double() * y.double()).sum().item(), (x.double() * ry.double()).sum().item()
    assert abs(a - b) <= 2.0 ** -20 * (rx.double() * y.double()).abs().sum().item()

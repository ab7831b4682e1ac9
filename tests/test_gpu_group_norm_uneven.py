"""Group norm over packed samples of which one is far longer than the rest (which choose the path), with a mean far
from 0 and gradients that add up.

Bounds, E = 2^-24.  Statistics are sums over short runs, merged or compensated, so they stand within 64 E of the
spread, and the mean within E of itself besides; a sum of gradients stands within 160 E of its absolute terms (64
in a run, one for each of the samples and workgroups joined behind it).  A chain of L additions would be off by up to
L E / 2 of the sum: half a million of them, by 2e-4 to 1e-2 where the terms are alike."""
import numpy as np
import pytest

import synthetic
from gpu_util import torch_dtype
from oracle import operators as ops
from test_gpu_group_norm import U, backward, build, eq, forward  # noqa: F401  (eq is the fixture)

pytestmark = pytest.mark.gpu

F32, BF16 = synthetic.F32, synthetic.BF16
E = 2.0 ** -24


def check(p, long, shift, what):
    """The long sample's outputs and the parameters' gradients (groups = 1)."""
    import torch
    torch.cuda.synchronize()
    u, s = U[p["dt"]], slice(int(p["off"][long]), int(p["off"][long + 1]))
    x, dy, gamma, beta = (p[n].double() for n in ("x", "dy", "gamma", "beta"))
    gamma, beta = gamma[None, :, None], beta[None, :, None]
    xl, g = x[s], dy[s] * gamma
    m = xl.mean()
    r = 1.0 / torch.sqrt(((xl - m) ** 2).mean() + p["eps"])
    xh = (xl - m) * r
    worst = lambda err, tol: float((err / tol).max())  # noqa: E731
    mean_err = E * abs(float(m)) + 64 * E / float(r)
    st = p["stats"][long, 0].double()
    assert abs(float(st[0] - m)) <= mean_err, (what, "mean", float(st[0] - m) / mean_err)
    assert abs(float(st[1] / r) - 1) <= 64 * E, (what, "rstd", (float(st[1] / r) - 1) / E)
    exh = mean_err * r + 72 * E * xh.abs()
    y = xh * gamma + beta
    tol = u * y.abs() + exh * gamma.abs() + 2 * E * (y.abs() + (xh * gamma).abs())
    assert worst((p["y"][s].double() - y).abs(), tol) <= 1, (what, "y", worst((p["y"][s].double() - y).abs(), tol))
    m1, m2 = g.mean(), (g * xh).mean()
    e1, e2 = 160 * E * g.abs().mean(), 160 * E * (g * xh).abs().mean() + (g.abs() * exh).mean()
    dx = (g - m1 - xh * m2) * r
    tol = u * dx.abs() + r * (e1 + xh.abs() * e2 + exh * m2.abs()) + 72 * E * r * (g.abs() + m1.abs() + (xh * m2).abs())
    err = (p["dx"][s].double() - dx).abs()
    assert worst(err, tol) <= 1, (what, "dx", worst(err, tol))
    db, size = dy.sum((0, 2)), dy.abs().sum((0, 2))
    err = (p["dbeta"].double() - db).abs()
    assert worst(err, 160 * E * size) <= 1, (what, "dbeta", worst(err, 160 * E * size))


# rows of one thread or of a few, pieces of 4, 8 and 1 numbers; samples before and after the long one
CASES = [(F32, 4, 33, 120000, 17200, False), (F32, 4, 8, 60000, 2200, False), (F32, 4, 11, 30000, 5000, True),
         (F32, 3, 40, 20000, 3000, False)]


@pytest.mark.parametrize("dt,N,C,length,others,odd", CASES)
@pytest.mark.parametrize("mean", [0.0, 1000.0])
def test_one_long_sample_among_many(eq, dt, N, C, length, others, odd, mean):
    lens = [1] * (others // 3) + [length] + [1] * (others - others // 3)
    p = build(eq, dt, N, C, 1, ops.NONE, lens, True, seed=C, mean=mean, wide=odd, odd=odd)
    p["dy"].mul_(0.01).add_(0.7)
    forward(p)
    backward(p)
    check(p, others // 3, mean, f"{dt} N={N} C={C} {length}")

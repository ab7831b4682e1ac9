"""Biases of the type's lowest number: finite, so rows that hold nothing else are means, not empty."""
import numpy as np
import pytest

from attention_util import BF16, E, F16, F32, Problem
from test_gpu_attention import eq  # noqa: F401
from test_gpu_attention_step import Step

pytestmark = pytest.mark.gpu
TYPES = [F32, BF16, F16]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("zero", ["q", "k"])
@pytest.mark.parametrize("causal,lens,d", [(True, [90, 200], 4), (False, [130], 8), (True, [150], 16)])
def test_rows_of_the_lowest_bias(eq, dt, zero, causal, lens, d):  # noqa: F811
    """Every key of head 0 under the lowest number, every key of head 3 under the largest; q or k all 0: o is the mean
    of the values, as without the number, and lse the number (held to 2.35e38 = log 2 times fp32's largest) plus log n."""
    import torch
    p = Problem(eq, dt, 8, 4, 2, d, d, lens, causal=causal, buckets=8, reach=40, seed=7)
    getattr(p, zero).zero_()
    p.bias.zero_()
    p.bias[0], p.bias[3] = torch.finfo(p.bias.dtype).min, torch.finfo(p.bias.dtype).max
    p.forward()
    n = np.array([i + 1 if causal else m for m in lens for i in range(m)])
    for h in (0, 3):
        c = float(p.bias[h, 0])
        want = np.sign(c) * min(abs(c), float(np.finfo(np.float32).max) * np.log(2)) + np.log(n)
        assert np.all(np.abs(p.lse[h].double().cpu().numpy() - want) <= 4 * E * abs(c) + 300 * E)
        p.lse[h] = torch.from_numpy(np.log(n)).float().cuda()
    p.bias.zero_()
    p.check(f"{dt}", backward=False)


@pytest.mark.parametrize("dt", TYPES)
def test_step_of_the_lowest_bias(eq, dt):  # noqa: F811
    """Every key under the type's lowest number: a mean, as of any other constant where the query is 0."""
    import torch
    a, b = (Step(eq, dt, 8, 2, 1, 8, 8, [300, 70, 1], 16, 32, 40) for _ in range(2))
    for s, c in ((a, torch.finfo(a.bias.dtype).min), (b, 0.0)):
        s.bias[:] = c
        s.q.zero_()
        s.run()
    assert torch.equal(a.o, b.o) and torch.isfinite(a.lse).all() and (a.lse < -6e4).all()

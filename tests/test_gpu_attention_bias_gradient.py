"""Gradients of biases whose distances no pair of a query and a key has."""
import pytest

from attention_util import BF16, F16, F32, Problem
from test_gpu_attention import eq  # noqa: F401

pytestmark = pytest.mark.gpu
TYPES = [F32, BF16, F16]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("causal,n", [(True, 100), (False, 200)])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["k", "v"])
def test_biases_of_distances_that_no_pair_has(eq, dt, causal, n, poison, what):  # noqa: F811
    """A NaN that every row sees is in the gradients of the distances that there are, 0 .. n - 1, and in no other."""
    import torch
    p = Problem(eq, dt, 8, 2, 1, 8, 8, [n], causal=causal, buckets=128 if causal else 256, reach=1000, seed=11)
    getattr(p, what)[0] = poison
    p.forward()
    p.backward()
    far = eq.eqlinear_attention_bucket(p.plan, n - 1)
    side = 128
    assert far + 1 < side and torch.isnan(p.dbias[:, :far + 1]).any()
    assert (p.dbias[:, far + 1:side] == 0).all()
    if not causal:
        assert (p.dbias[:, side + eq.eqlinear_attention_bucket(p.plan, n - 1) + 1:] == 0).all()

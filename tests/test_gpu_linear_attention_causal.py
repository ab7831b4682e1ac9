"""Linear attention: what a token does not see leaves its bits alone, NaN and infinities included.

Tokens from 50 on (before 50, in the gradients of keys and values) share a block of 16 scores and a
chunk of 64 with ones that do not see them.
"""
import pytest

import synthetic
from test_gpu_linear_attention import Problem, eq  # noqa: F401  (eq is the fixture)

pytestmark = pytest.mark.gpu

F32, BF16, F16 = synthetic.F32, synthetic.BF16, synthetic.F16


def run(p):
    import torch
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    return {n: getattr(p, n).clone() for n in ("o", "dq", "dk_", "dv_")}


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("lens", [[90], [90, 70], [900]], ids=str)
@pytest.mark.parametrize("a,b", [(float("nan"), float("inf")), (float("inf"), float("nan")), (-float("inf"), 6e4), (6e4, 6e4)])
def test_later_keys_and_values(eq, dt, lens, a, b):
    import torch
    p = Problem(eq, dt, 8, 4, 2, 8, 4, lens, len(lens) > 1, 41)
    first = run(p)
    p.k[50:90], p.v[50:90] = a, b
    got = run(p)
    for n in ("o", "dq"):
        assert torch.equal(first[n][:50], got[n][:50]), n
        assert torch.equal(first[n][lens[0]:], got[n][lens[0]:]), n


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("lens", [[90], [90, 70], [900]], ids=str)
@pytest.mark.parametrize("a,b", [(float("nan"), float("inf")), (float("inf"), float("nan")), (-float("inf"), 6e4), (6e4, 6e4)])
def test_earlier_queries(eq, dt, lens, a, b):
    import torch
    p = Problem(eq, dt, 8, 4, 2, 8, 4, lens, len(lens) > 1, 42)
    first = run(p)
    p.q[:50], p.d_o[:50] = a, b
    got = run(p)
    for n in ("dk_", "dv_"):
        assert torch.equal(first[n][50:], got[n][50:]), n

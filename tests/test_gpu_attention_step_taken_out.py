"""Single tokens over a paged cache whose heads take keys out by biases of -infinity, or hold them under the type's
lowest number: what a query does not see changes no bit of it (bounds: test_gpu_attention_step)."""
import pytest

from attention_util import BF16, F16, F32
from test_gpu_attention import eq  # noqa: F401
from test_gpu_attention_step import Step

pytestmark = pytest.mark.gpu
TYPES = [F32, BF16, F16]
NEAR = 8  # distances that keep their biases: below this


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("layout", ["apart", "odd"])
@pytest.mark.parametrize("d", [4, 8, 16])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_step_keys_taken_out(eq, dt, layout, d, poison):  # noqa: F811
    """Of heads that share their keys, one takes far ones out and one does not."""
    import torch
    make = lambda: Step(eq, dt, 8, 2, 1, d, d, [300, 100, 9, 1], 16, 32, 40, seed=d, layout=layout)  # noqa: E731
    a, b = make(), make()
    gone = sorted({eq.eqlinear_attention_bucket(a.plan, n) for n in range(NEAR, 400)})
    far = [(0, 5), (0, 130), (0, 299 - NEAR), (1, 40)]
    for s in (a, b):
        s.bias[0, gone] = -float("inf")
    for q, j in far:
        block = int(b.table[q, j // 16])
        b.kc[block, j % 16, :, 1, 1:] = poison
        b.vc[block, j % 16] = poison
        b.vc[block, j % 16, :, 0, 0] = -poison
    for s in (a, b):
        s.run()
    assert torch.isfinite(a.o.float()).all()
    assert torch.equal(a.o[:, 0], b.o[:, 0]) and torch.equal(a.lse[0], b.lse[0])
    assert torch.equal(a.o[2:], b.o[2:])
    assert not torch.isfinite(b.o[:2, 1].float()).all(-1).all(-1).any()
    # every bucket taken out: nothing is seen
    b.bias[0] = -float("inf")
    b.run()
    assert (b.o[:, 0] == 0).all() and (b.lse[0] == -float("inf")).all()
    a.bias[0, gone] = -200.0
    a.check(f"{dt}")


@pytest.mark.parametrize("dt", TYPES)
def test_step_an_infinity_where_it_is_seen(eq, dt):  # noqa: F811
    import torch
    s = Step(eq, dt, 8, 2, 1, 8, 8, [300], 16, 32, 40)
    gone = sorted({eq.eqlinear_attention_bucket(s.plan, n) for n in range(NEAR, 400)})
    s.bias[0, gone] = -float("inf")
    s.vc[int(s.table[0, 10]), 3, 0, 2, 3] = -float("inf")  # head 1 sees it
    s.vc[int(s.table[0, 18]), 10, 0, 1, 1] = float("inf")  # token 298: both do
    s.run()
    o = s.o[0].float()
    assert o[1, 2, 3] == -float("inf") and (o[:, 1, 1] == float("inf")).all()
    o[1, 2, 3] = o[0, 1, 1] = o[1, 1, 1] = 0
    assert torch.isfinite(o).all()

"""Keys that a bias of -infinity takes out of a row, and the type's lowest bias, which takes none out: what a query does
not see changes no bit of it, whatever stands there (bounds: attention_util)."""
import pytest

from attention_util import BF16, F16, F32, Problem
from test_gpu_attention import eq  # noqa: F401

pytestmark = pytest.mark.gpu
TYPES = [F32, BF16, F16]
NEAR = 8  # distances that keep their biases: below this


def pair(make, poison, keys):
    """Two equal problems, the second with `poison` in the keys and values of `keys`; both run."""
    a, b = make(), make()
    for p in (a, b):
        p.bias[:, p.cut] = -float("inf")
    for j in keys:
        b.k[j, :, 1, 1:] = poison
        b.v[j] = poison
        b.v[j, :, 0, 0] = -poison
    for p in (a, b):
        p.forward()
        p.backward()
    return a, b


def near_buckets(eq, p):  # noqa: F811
    """Marks in p.cut the buckets that hold no distance below NEAR; those that hold one hold no other."""
    keep = {eq.eqlinear_attention_bucket(p.plan, d) for d in range(0 if p.causal else 1 - NEAR, NEAR)}
    gone = {eq.eqlinear_attention_bucket(p.plan, s * d) for d in range(NEAR, 2000) for s in ((1,) if p.causal else (1, -1))}
    assert not keep & gone
    p.cut = sorted(gone)
    return p


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("N,d,lens,layout", [(8, 4, [200, 130], "apart"), (8, 4, [90], "odd"), (8, 8, [300], "apart"),
                                             (8, 12, [200], "apart"), (8, 16, [150], "fused"), (4, 4, [2100], "apart"),
                                             (8, 16, [2100], "apart")])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_keys_taken_out(eq, dt, causal, N, d, lens, layout, poison):  # noqa: F811
    """A key is seen from less than NEAR tokens away; farther rows keep their bits, on both sides of tiles' ends, and
    so do the gradients of keys that no row near it sees."""
    import torch
    make = lambda: near_buckets(eq, Problem(eq, dt, N, 4, 2, d, d, lens, causal=causal, buckets=32 if causal else 64,  # noqa: E731
                                            reach=40, layout=layout, seed=d))
    keys = [30, 63, 64] + ([129] if lens[0] > 130 else []) + ([1500, lens[0] - 1] if lens[0] > 1500 else [])
    a, b = pair(make, poison, keys)
    T = a.T
    ends = torch.tensor([i for i, n in enumerate(lens) for _ in range(n)])
    at = torch.arange(T)
    near = lambda x, y: (ends[x] == ends[y]) & ((y <= x) | (not causal)) & ((x - y).abs() < NEAR)  # noqa: E731  query x sees key y
    odd_rows = near(at[:, None], torch.tensor(keys)[None]).any(1)  # rows that see a poisoned key
    odd_keys = (near(at[:, None], at[None]) & odd_rows[:, None]).any(0)  # keys that such a row sees
    rows, keys_free = (~odd_rows).cuda(), (~odd_keys).cuda()
    assert rows.sum() > 40 and torch.isfinite(a.o.float()).all() and torch.isfinite(a.lse).all()
    for n in ("o", "dq"):
        assert torch.equal(getattr(a, n)[rows], getattr(b, n)[rows]), n
    assert torch.equal(a.lse[:, rows], b.lse[:, rows])
    for n in ("dk_", "dv_"):
        assert torch.equal(getattr(a, n)[keys_free], getattr(b, n)[keys_free]), n
    for p in (a, b):
        assert (p.dbias[:, p.cut] == 0).all()
    # the rows that see them are not spared
    assert not torch.isfinite(b.o[odd_rows.cuda()].float()).all(-1).all(-1).any()
    # the clean run is the attention of a band: -200 leaves e^-190 of a probability
    a.bias[:, a.cut] = -200.0
    if lens[0] < 1000:
        a.check(f"{dt}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("causal", [False, True])
def test_an_infinity_where_it_is_seen(eq, dt, causal):  # noqa: F811
    """A value of +infinity: one in the rows that see its key, and nothing in those from which it is taken out."""
    import torch
    p = near_buckets(eq, Problem(eq, dt, 8, 2, 2, 8, 8, [200], causal=causal, buckets=32 if causal else 64, reach=40, packed=False))
    p.bias[:, p.cut] = -float("inf")
    p.v[70, 0, 2, 3] = float("inf")
    p.v[71, 1, 2, 3] = -float("inf")
    p.forward()
    for h, j, x in ((0, 70, float("inf")), (1, 71, -float("inf"))):
        seen = torch.zeros(200, dtype=torch.bool)
        seen[(j if causal else j - NEAR + 1):j + NEAR] = True
        o = p.o[:, h].float().cpu()
        assert (o[seen, 2, 3] == x).all()
        assert torch.isfinite(o[~seen]).all()
        o[:, 2, 3] = 0
        assert torch.isfinite(o).all()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf")])
def test_heads_with_every_key_taken_out(eq, dt, causal, poison):  # noqa: F811
    """Rows that see nothing, over keys and values of anything: o = 0, lse = -infinity, no gradients."""
    import torch
    make = lambda: Problem(eq, dt, 8, 4, 4, 4, 4, [200, 60], causal=causal, buckets=8, reach=40, seed=3)  # noqa: E731
    a, b = make(), make()
    for p in (a, b):
        p.bias[1] = -float("inf")
    b.k[:, 1], b.v[:, 1] = poison, poison
    for p in (a, b):
        p.forward()
        p.backward()
        assert (p.o[:, 1] == 0).all() and (p.lse[1] == -float("inf")).all()
        for t in (p.dq[:, 1], p.dk_[:, 1], p.dv_[:, 1], p.dbias[1]):
            assert (t == 0).all()
    for n, t in a.outputs().items():
        assert torch.equal(t, b.outputs()[n]), n


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,d", [([90], 4), ([200, 130], 8), ([2100], 16)])
def test_the_lowest_bias_beside_others(eq, dt, causal, lens, d):  # noqa: F811
    """Biases of the type's lowest number beside others: nothing is left of such keys, in either direction, as of a
    bias of -200 (e^-190 of a probability)."""
    import torch
    p = Problem(eq, dt, 8, 2, 1, d, d, lens, causal=causal, buckets=8 if causal else 16, reach=40, seed=4)
    gone = [3, 4, 5, 6, 7] + ([] if causal else [10, 11, 12, 13, 14, 15])
    p.bias[:, gone] = torch.finfo(p.bias.dtype).min
    p.forward()
    p.backward()
    assert (p.dbias[:, gone] == 0).all()
    p.bias[:, gone] = -200.0
    p.check(f"{dt}")

"""Softmax attention at the ends of its lengths: lone keys, whose gradients are exactly 0, and sequences so long that
work is dealt to the card's parts in another order (bounds: attention_util)."""
import pytest

from attention_util import BF16, F16, F32, Problem
from test_gpu_attention import both, eq  # noqa: F401
from test_gpu_attention_step import Step

pytestmark = pytest.mark.gpu
TYPES = [F32, BF16, F16]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("buckets", [0, 8])
@pytest.mark.parametrize("N,dk,dv", [(8, 3, 3), (8, 12, 12), (4, 27, 27), (5, 3, 7)])
def test_a_lone_key(eq, dt, causal, buckets, N, dk, dv):  # noqa: F811
    """One key's probability is 1 whatever its score: dq, dk and the biases' gradients are 0, to the bit.  o is v and
    dv is d_o within their bounds only: the forward's exponentials are of a running maximum that need not be the
    score itself, so P is rounded (u), and lse is, which the probability of the backward is made from (e |lse|)."""
    p = Problem(eq, dt, N, 3, 3, dk, dv, [1] * 70, causal=causal, buckets=buckets, reach=20, bias_std=3.0, seed=dk)
    p.forward()
    p.backward()
    for t in (p.dq, p.dk_) + ((p.dbias,) if buckets else ()):
        assert (t == 0).all()
    p.check(f"{dt}")


@pytest.mark.parametrize("dt", TYPES)
def test_the_first_token_has_no_gradient(eq, dt):  # noqa: F811
    """A causal sequence's first query sees itself alone."""
    p = Problem(eq, dt, 8, 4, 2, 12, 12, [200, 130], causal=True, seed=2)
    both(p, f"{dt}")
    assert (p.dq[0] == 0).all() and (p.dq[200] == 0).all()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("H,K", [(2, 1), (9, 9)])
@pytest.mark.parametrize("causal", [False, True])
def test_long(eq, dt, H, K, causal):  # noqa: F811
    """Fewer (sequence, head) pairs than parts of the card, and one more than them."""
    both(Problem(eq, dt, 2, H, K, 4, 4, [2100], causal=causal, packed=False, seed=H), f"{dt} {H}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lens,kv_lens", [([2500, 1, 3650], None), ([2049, 2100], [2300, 1950]), ([2048, 2050], [70, 30]),
                                          ([60, 0], [2047, 2100])])
@pytest.mark.parametrize("causal", [False, True])
def test_long_and_packed(eq, dt, lens, kv_lens, causal):  # noqa: F811
    """Queries dealt and keys not, and the other way round, among them."""
    both(Problem(eq, dt, 2, 2, 1, 4, 8, lens, kv_lens, causal=causal, buckets=16, reach=300, behind=3, seed=len(lens)), f"{dt} {lens}")


@pytest.mark.parametrize("dt", TYPES)
def test_long_with_odd_rows(eq, dt):  # noqa: F811
    both(Problem(eq, dt, 7, 2, 1, 5, 5, [2200], causal=True, layout="odd", packed=False, seed=4), f"{dt}")


@pytest.mark.parametrize("dt", [BF16, F16])
def test_long_wide_heads(eq, dt):  # noqa: F811
    """128 numbers a head: dk and dv by kernels of their own."""
    both(Problem(eq, dt, 8, 2, 1, 16, 16, [2100], causal=True, buckets=8, reach=50, packed=False, seed=5), f"{dt}")


@pytest.mark.parametrize("dt", TYPES)
def test_nothing_seen_in_long_sequences(eq, dt):  # noqa: F811
    """NaN in queries, and their gradients, before a key leave its gradients' bits."""
    import torch
    a, b = (Problem(eq, dt, 4, 2, 1, 4, 4, [2300], causal=True, packed=False, seed=6) for _ in range(2))
    a.forward()
    a.backward()
    for t in (b.q, b.do):
        t[500, :, 3] = float("nan")
    b.forward()
    b.backward()
    for n in ("dk_", "dv_"):
        assert torch.equal(getattr(a, n)[501:], getattr(b, n)[501:]), n
        assert torch.isnan(getattr(b, n)[:501].float()).any()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("batch", [2047, 2048, 2049, 5000])
def test_a_step_of_thousands(eq, dt, batch):  # noqa: F811
    s = Step(eq, dt, 4, 2, 1, 2, 2, [(7 * b) % 150 for b in range(batch)], 16, 8, 20, seed=batch)
    s.run()
    s.check(f"{dt} {batch}")


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("low", [-1e8, -1e30])
def test_rows_under_large_negative_biases(eq, dt, low):  # noqa: F811
    """Every key of head 0 under one large number: o is a mean of v's rows, gradients are 0; head 1 is as ever."""
    import torch
    p, plain = (Problem(eq, dt, 8, 2, 2, 4, 4, [90, 200], causal=True, buckets=8, reach=40, seed=7) for _ in range(2))
    p.bias[0] = low
    for x in (p, plain):
        x.forward()
        x.backward()
    o = p.o.float()
    # a weighted mean, rounded: P and o by u each, and 16 e for the sums of up to 200 terms that are at most 1
    top = p.v[:, 0].float().abs().max() * (1 + 2.0 ** -6)
    assert torch.isfinite(o).all() and (o[:, 0].abs() <= top).all() and torch.isfinite(p.lse).all()
    for t in (p.dq[:, 0], p.dk_[:, 0], p.dv_[:, 0], p.dbias[0]):
        assert (t == 0).all()
    for a, b in ((p.o, plain.o), (p.dq, plain.dq), (p.dk_, plain.dk_), (p.dv_, plain.dv_)):
        assert torch.equal(a[:, 1], b[:, 1])
    assert torch.equal(p.dbias[1], plain.dbias[1])


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("scale", [2.0 ** -100, -2.0 ** -40])
def test_the_smallest_scales(eq, dt, scale):  # noqa: F811
    """Scores of nothing: the biases alone decide."""
    both(Problem(eq, dt, 8, 2, 1, 4, 4, [100], causal=True, buckets=8, reach=40, scale=scale, seed=8), f"{dt} {scale}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("what", ["no sequences", "no queries", "no keys"])
def test_nothing(eq, dt, what):  # noqa: F811
    """Gradients are written all the same, as zeros (offsets belong to one sequence at least: without any, batch = 0)."""
    lens, kv_lens = {"no sequences": ([], []), "no queries": ([0, 0], [70, 3]), "no keys": ([5, 40], [0, 0])}[what]
    p = Problem(eq, dt, 8, 2, 1, 4, 4, lens, kv_lens, buckets=8, reach=40, packed=bool(lens), seed=9)
    if not lens:
        with pytest.raises(eq.EqlError):
            Problem(eq, dt, 8, 2, 1, 4, 4, lens, kv_lens, buckets=8, reach=40, seed=9).forward()
    p.forward()
    p.backward()
    for t in (p.o, p.dq, p.dk_, p.dv_, p.dbias):
        assert (t == 0).all()
    if p.T:
        assert (p.lse == -float("inf")).all()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("d", [7, 12, 16])
@pytest.mark.parametrize("lens", [[300], [2050]])
def test_the_longest_reach_of_wide_heads(eq, dt, d, lens):  # noqa: F811
    """The most LDS that tiles and biases take together."""
    both(Problem(eq, dt, 8, 1, 1, d, d, lens, causal=True, buckets=256, reach=1024, packed=False, seed=d), f"{dt} {d}")


@pytest.mark.parametrize("dt", TYPES)
def test_a_step_of_thousands_with_wide_heads(eq, dt):  # noqa: F811
    s = Step(eq, dt, 8, 1, 1, 16, 16, [(11 * b) % 40 for b in range(2048)], 16, 256, 1024, seed=1)
    s.run()
    s.check(f"{dt}")

"""Softmax attention whose scores are large numbers: probabilities depend on their differences alone, and gradients
follow the forward at any size (bounds: attention_util, of the same scores without the number that they share)."""
import numpy as np
import pytest

from attention_util import BF16, E, F16, F32, Problem
from test_gpu_attention import eq  # noqa: F401

pytestmark = pytest.mark.gpu
TYPES = [F32, BF16, F16]


def seen(p):
    """Number of keys that each query sees."""
    n = []
    for q, k in zip(p.lens, p.kv_lens):
        n += [min(k, max(0, i + k - q + 1)) if p.causal else k for i in range(q)]
    return np.array(n)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("number", [-1e30, -1e9, -1e6, -3e4, -2500.0, 2500.0, 3e4, 1e6, 1e9, 1e30, "lowest"])
@pytest.mark.parametrize("zero", ["q", "k"])
@pytest.mark.parametrize("causal,lens,d", [(True, [90, 200], 4), (False, [130], 8)])
def test_one_bias_for_all(eq, dt, number, zero, causal, lens, d):  # noqa: F811
    """Every key of heads 0 and 3 under one number, and q or k all 0: P is 1 / n, as without the number."""
    import torch
    p = Problem(eq, dt, 8, 4, 2, d, d, lens, causal=causal, buckets=8, reach=40, seed=7)
    if number == "lowest":
        number = torch.finfo(p.bias.dtype).min
    if dt == F16 and abs(number) > 65504:
        pytest.skip("not an fp16 number")
    getattr(p, zero).zero_()
    p.bias.zero_()
    p.bias[0], p.bias[3] = number, number
    c = float(p.bias[0, 0])
    p.forward()
    p.backward()
    # (a number times log2 e is held to fp32's largest: 2.36e38 of them)
    want = max(c, -float(np.finfo(np.float32).max) * np.log(2)) + np.log(seen(p))
    for h in (0, 3):
        assert np.all(np.abs(p.lse[h].double().cpu().numpy() - want) <= 4 * E * abs(c) + 300 * E)
        p.lse[h] = torch.from_numpy(np.log(seen(p))).float().cuda()
    p.bias.zero_()
    p.check(f"{dt} {number}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("power", [12, 16, 20])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("causal,lens,d,layout", [(True, [90, 200], 8, "apart"), (False, [130], 4, "apart"), (True, [2200], 8, "apart"),
                                                  (True, [150], 16, "apart"), (False, [2100], 16, "apart"), (True, [140], 8, "fused"),
                                                  (True, [140], 5, "odd"), (False, [90], 3, "odd")])
def test_scores_that_share_a_large_number(eq, dt, power, sign, causal, lens, d, layout):  # noqa: F811
    """Scores of +-2^power and small multiples of 1/4: products of whole numbers below 2^24, exact in fp32."""
    import torch
    p = Problem(eq, dt, 8, 4, 2, d, d, lens, causal=causal, layout=layout, scale=0.25 * sign, seed=8)
    g = torch.Generator().manual_seed(9)
    for t in (p.q, p.k):
        t.copy_(torch.randint(-1, 2, t.shape, generator=g).to(t.dtype).cuda())
        t[:, :, 0, 0] = 2.0 ** ((power + 2) // 2)
    p.q[:, 1, 0, 0] = 0  # (beside heads with ordinary scores)
    p.forward()
    p.backward()
    lse = p.lse.double().cpu().numpy()
    for h in (0, 2, 3):
        assert np.all(np.abs(lse[h] - sign * 2.0 ** power) <= 64)
    # without the number: another lse, and no gradients of its factors
    for t in (p.q, p.k, p.dq, p.dk_):
        t[:, :, 0, 0] = 0
    q = Problem(eq, dt, 8, 4, 2, d, d, lens, causal=causal, layout=layout, scale=0.25 * sign, seed=8)
    q.q.copy_(p.q)
    q.k.copy_(p.k)
    q.forward()
    assert np.all(np.abs(lse[0] - sign * 2.0 ** power - q.lse[0].double().cpu().numpy()) <= 8 * E * 2.0 ** power)
    p.lse.copy_(q.lse)
    p.check(f"{dt} {power}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("number", [-3000.0, -800.0, 800.0, 3000.0])
def test_large_biases_and_scores(eq, dt, number):  # noqa: F811
    """A large number in every bias beside ordinary scores, and rows with and without it in one head."""
    p = Problem(eq, dt, 8, 2, 1, 8, 8, [150, 40], causal=True, buckets=8, reach=40, seed=10)
    p.bias[0] += number
    p.bias[1, 0] += 2 * number  # far rows have it in one key, the first row in its only one
    p.forward()
    p.backward()
    p.check(f"{dt} {number}")


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("number", [-1e8, -1e30, 1e8])
def test_a_head_under_a_large_number(eq, dt, number):  # noqa: F811
    """Every key of head 0 under a number whose fp32 neighbours are 8 and more away: whatever its probabilities are,
    they add up to 1, so that sum_j dv_j = sum_i d_o_i and sum dS = 0; head 1 keeps its bits.  (Each P is rounded by u
    and made of exponentials to 2^-20, each dv by u; dS likewise, of sizes P (|dP| + |delta|).)"""
    import torch
    from attention_util import U
    p, plain = (Problem(eq, dt, 8, 2, 2, 4, 4, [90, 200], causal=True, buckets=8, reach=40, seed=7) for _ in range(2))
    p.bias[0] = number
    for x in (p, plain):
        x.forward()
        x.backward()
    u = 0 if dt == F32 else U[dt]
    for a, b in ((0, 90), (90, 290)):
        do, dv = p.do[a:b, 0].double(), p.dv_[a:b, 0].double()
        bound = do.abs().sum(0) * (u + 2.0 ** -19) + dv.abs().sum(0) * max(u, E)
        assert ((dv.sum(0) - do.sum(0)).abs() <= bound).all()
        assert (dv.abs().sum(0) > 0.1 * do.sum(0).abs()).all()
    # |dP| and |delta| are at most sum |d_o| max |v|
    size = float((p.do[:, 0].double().abs().flatten(1).sum(1) * p.v[:, 0].double().abs().max()).sum())
    assert abs(float(p.dbias[0].double().sum())) <= 2 * size * 2.0 ** -19
    for x in (p.o[:, 0], p.dq[:, 0], p.dk_[:, 0], p.lse[0], p.dbias[0]):
        assert torch.isfinite(x.float()).all()
    for x, y in ((p.o, plain.o), (p.dq, plain.dq), (p.dk_, plain.dk_), (p.dv_, plain.dv_)):
        assert torch.equal(x[:, 1], y[:, 1])
    assert torch.equal(p.dbias[1], plain.dbias[1])


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("number", [-1e9, 1e9])
@pytest.mark.parametrize("causal,lens,d", [(True, [90, 200], 4), (False, [130], 8), (True, [2100], 8)])
def test_a_large_number_beside_keys_taken_out(eq, dt, number, causal, lens, d):  # noqa: F811
    """Biases of a large number or -infinity; q is 0, so that P is 1 / n of the keys that are left: a row's own and the two
    before it."""
    import torch
    p = Problem(eq, dt, 8, 2, 1, d, d, lens, causal=causal, buckets=8 if causal else 16, reach=40, seed=12)
    gone = [3, 4, 5, 6, 7] + ([] if causal else [9, 10, 11, 12, 13, 14, 15])
    p.q.zero_()
    p.bias[:] = number
    number = float(p.bias[0, 0])  # in the plan's type
    p.bias[:, gone] = -float("inf")
    p.forward()
    p.backward()
    assert (p.dbias[:, gone] == 0).all()
    n = torch.tensor([min(i + 1, 3) for m in lens for i in range(m)]).double()
    assert float((p.lse.double().cpu() - number - n.log()).abs().max()) <= 4 * E * abs(number)
    p.lse.copy_(n.log())
    p.bias.zero_()
    p.bias[:, gone] = -200.0
    p.check(f"{dt} {number}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("with_dbias", [True, False])
def test_captured_before_rows_are_steep(eq, dt, with_dbias):  # noqa: F811
    """A graph of both directions, replayed as its rows turn steep and back, against eager calls on another stream."""
    import torch
    p, q = (Problem(eq, dt, 8, 3, 1, 8, 8, [100, 229], causal=True, buckets=8, reach=40, seed=13) for _ in range(2))
    for x in (p, q):
        x.dbias = x.dbias if with_dbias else None
        x.ws = x.workspace(True)
        x.forward()
        x.backward(workspace=x.ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.forward()
        p.backward(workspace=p.ws)
    side = torch.cuda.Stream()
    for number in (0.0, -5000.0, 3000.0, -60000.0, 0.0):
        for x in (p, q):
            x.bias[:2] = number
            for t in x.outputs().values():
                t.fill_(7.0)
        side.wait_stream(torch.cuda.current_stream())
        g.replay()
        with torch.cuda.stream(side):
            q.forward()
            q.backward(workspace=q.ws)
        torch.cuda.synchronize()
        for n, t in p.outputs().items():
            assert torch.equal(t, q.outputs()[n]), (n, number)
            assert torch.isfinite(t.float()).all()

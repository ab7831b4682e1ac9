"""Softmax attention and its gradients against their fp64 definition: types, head widths, lengths, masks that
leave rows empty, shared heads, biases by distance, strides (bounds: attention_util)."""
import numpy as np
import pytest

from attention_util import BF16, F16, F32, Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import group_equivariant_linear_amd as eq
    eq.load_library()
    return eq


def both(p, what):
    p.forward()
    p.backward()
    return p.check(what)


TYPES = [F32, BF16, F16]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("N,dk,dv", [(8, 8, 8), (7, 16, 16), (8, 16, 16), (1, 1, 1), (5, 9, 9), (3, 11, 7), (4, 8, 24), (12, 2, 8),
                                     (16, 8, 2)])
@pytest.mark.parametrize("causal", [False, True])
def test_widths(eq, dt, N, dk, dv, causal):
    both(Problem(eq, dt, N, 4, 2, dk, dv, [70, 33], causal=causal, seed=N + dk), f"{dt} N={N} {dk} {dv}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lens", [[1], [2], [31], [32], [33], [63], [64], [65], [127], [128], [129], [197], [300]])
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(eq, dt, lens, causal):
    both(Problem(eq, dt, 8, 2, 2, 8, 8, lens, causal=causal, packed=False, seed=lens[0]), f"{dt} {lens}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lens,kv_lens", [([65, 0, 1, 130], None), ([3, 70, 5], [200, 70, 0]), ([0, 4, 9], [5, 0, 90]),
                                          ([130, 1], [2, 257]), ([1, 1, 1], [64, 128, 129])])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("buckets", [0, 8])
def test_packed_and_unlike_lengths(eq, dt, lens, kv_lens, causal, buckets):
    """Among them more queries than keys: causal rows that see nothing."""
    both(Problem(eq, dt, 8, 3, 1, 4, 8, lens, kv_lens, causal=causal, buckets=buckets, reach=20, behind=5, seed=len(lens)),
         f"{dt} {lens} {kv_lens}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("buckets,reach", [(4, 3), (8, 20), (32, 128), (64, 500), (256, 1024), (6, 1000)])
@pytest.mark.parametrize("causal", [False, True])
def test_biases(eq, dt, buckets, reach, causal):
    both(Problem(eq, dt, 8, 2, 1, 4, 4, [300, 50], causal=causal, buckets=buckets, reach=reach, seed=buckets), f"{dt} {buckets} {reach}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("causal", [False, True])
def test_biases_past_the_reach(eq, dt, causal):
    both(Problem(eq, dt, 4, 2, 2, 4, 4, [700], causal=causal, buckets=16, reach=60, packed=False), f"{dt}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("H,K", [(1, 1), (3, 1), (6, 2), (4, 4), (20, 1)])
def test_shared_heads(eq, dt, H, K):
    both(Problem(eq, dt, 8, H, K, 4, 4, [90, 41], causal=True, buckets=8, reach=30, seed=H), f"{dt} {H} {K}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("layout", ["fused", "odd"])
@pytest.mark.parametrize("N,dk,dv", [(8, 8, 8), (7, 16, 16), (5, 3, 4)])
def test_strides(eq, dt, layout, N, dk, dv):
    both(Problem(eq, dt, N, 4, 2, dk, dv, [100, 7, 64], causal=True, layout=layout, seed=N), f"{dt} {layout}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("std", [0.01, 8.0])
def test_flat_and_steep_scores(eq, dt, std):
    """Probabilities all alike, and ones that a single key takes."""
    both(Problem(eq, dt, 8, 2, 1, 8, 8, [150], causal=True, std=std, buckets=8, reach=40), f"{dt} {std}")


@pytest.mark.parametrize("dt", TYPES)
def test_negative_scale_and_large_biases(eq, dt):
    both(Problem(eq, dt, 8, 2, 1, 8, 8, [150], scale=-0.2, buckets=8, reach=40, bias_std=30.0), f"{dt}")


@pytest.mark.parametrize("do_std", [1e-6, 1e-3, 100.0])
def test_fp16_gradients_of_any_size(eq, do_std):
    """dS below and above fp16's range; dq, dk and dv are held to their own."""
    both(Problem(eq, F16, 8, 2, 1, 8, 8, [200], causal=True, do_std=do_std), f"{do_std}")


def test_fp16_one_large_probability_and_many_small(eq):
    """Thousands of probabilities near 2^-24 of the largest together weigh as much as a rounding."""
    import torch
    p = Problem(eq, F16, 8, 1, 1, 8, 8, [3000], scale=1.0)
    p.q.zero_()
    p.k.zero_()
    p.q[:, :, 0, 0] = 1.0
    p.k[1700, :, 0, 0] = 17.0
    p.v.copy_(torch.rand_like(p.v.float()) + 1.0)
    p.v[1700] = -1.0
    p.forward()
    p.check("spike", backward=False)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("low", ["lowest", "-inf"])
def test_biases_that_mask(eq, dt, low):
    """Buckets of the type's lowest value, or of -infinity: keys that vanish; rows whose every bucket is -infinity
    are empty."""
    import torch
    p = Problem(eq, dt, 8, 2, 1, 4, 4, [90], causal=True, buckets=8, reach=40)
    value = -float("inf") if low == "-inf" else torch.finfo(p.bias.dtype).min
    p.bias[0, 3:] = value
    p.bias[1, :] = value
    p.forward()
    o = p.o.float()
    assert torch.isfinite(o).all()
    if low == "-inf":
        assert (o[:, 1] == 0).all() and torch.isinf(p.lse[1]).all() and (p.lse[1] < 0).all()
        p.backward()
        for t in (p.dq, p.dk_, p.dv_, p.dbias):
            assert torch.isfinite(t.float()).all()
        assert (p.dq[:, 1] == 0).all() and (p.dbias[1] == 0).all() and (p.dbias[0, 3:] == 0).all()
    # head 0 equals a head whose far keys do not exist
    q, k, v = (t[:, 0].float().cpu().double().flatten(1).numpy() for t in (p.q, p.k, p.v))
    b = p.bias[0].float().cpu().double().numpy()
    for i in range(90):
        j0 = max(0, i - 2)  # buckets 0 .. 2 are the distances 0 .. 2
        s = p.scale * (k[j0:i + 1] @ q[i]) + b[i - np.arange(j0, i + 1)]
        w = np.exp(s - s.max())
        assert np.allclose(o[i, 0].flatten().cpu().numpy(), w @ v[j0:i + 1] / w.sum(), rtol=0.03, atol=0.03)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_seen_leaves_the_bits(eq, dt, bad):
    """NaN and infinities in tokens 60 and later change nothing before them, in any output, and none of the
    sequences beside; keys and values behind the last sequence are nobody's."""
    import torch
    a = Problem(eq, dt, 8, 2, 1, 8, 8, [100, 50], causal=True, buckets=8, reach=40, behind=3, seed=3)
    a.forward()
    a.backward()
    keep = {n: t.clone() for n, t in a.outputs().items()}
    b = Problem(eq, dt, 8, 2, 1, 8, 8, [100, 50], causal=True, buckets=8, reach=40, behind=3, seed=3)
    for t in (b.q, b.k, b.v):
        t[60, :, 1, 2] = bad
        t[75, :, 0] = bad
        t[150:] = bad
    b.do[150:] = bad
    b.forward()
    b.backward()
    for n, t in b.outputs().items():
        if n == "dbias":
            continue
        # gradients of keys before token 60 come from queries after it: only dq, o and lse of earlier tokens are free
        if n in ("dk", "dv"):
            assert torch.equal(t[100:150], keep[n][100:150]), n
            continue
        first = t[:, :60] if n == "lse" else t[:60]
        want = keep[n][:, :60] if n == "lse" else keep[n][:60]
        assert torch.equal(first, want), n
        rest, keep_rest = (t[:, 100:150], keep[n][:, 100:150]) if n == "lse" else (t[100:150], keep[n][100:150])
        assert torch.equal(rest, keep_rest), n


@pytest.mark.parametrize("dt", TYPES)
def test_queries_that_do_not_see_leave_a_keys_gradient(eq, dt):
    """NaN in the queries (and their d_o) before a key's token leave the bits of its gradients."""
    import torch
    make = lambda: Problem(eq, dt, 8, 2, 2, 8, 8, [140], causal=True, packed=False, seed=5)  # noqa: E731
    a, b = make(), make()
    a.forward()
    a.backward()
    for t in (b.q, b.do):
        t[20, :, 3] = float("nan")
        t[41, :, 2, 1] = float("inf")
    b.forward()
    b.backward()
    for n in ("dk_", "dv_"):
        assert torch.equal(getattr(a, n)[42:], getattr(b, n)[42:]), n
    assert torch.equal(a.dq[42:], b.dq[42:])
    assert torch.isnan(b.dk_[:21].float()).any()


@pytest.mark.parametrize("dt", TYPES)
def test_seen_infinities_arrive(eq, dt):
    """An infinite value is one in the rows that see it (and only there), a NaN a NaN."""
    import torch
    p = Problem(eq, dt, 8, 1, 1, 8, 8, [100], causal=True, packed=False, seed=6)
    p.v[30, 0, 1, 1] = float("inf")
    p.v[50, 0, 2, 2] = float("nan")
    p.forward()
    o = p.o.float()
    assert torch.isfinite(o[:30]).all() and torch.isfinite(o[:, :, 3:]).all()
    assert (o[30:, 0, 1, 1] == float("inf")).all() and torch.isfinite(o[:50, 0, 2]).all() and torch.isnan(o[50:, 0, 2, 2]).all()


@pytest.mark.parametrize("dt", TYPES)
def test_same_bits_every_time(eq, dt):
    import torch
    p = Problem(eq, dt, 8, 6, 2, 8, 8, [197, 3, 260], causal=False, buckets=32, reach=128, seed=7)
    first = None
    for _ in range(3):
        p.forward()
        p.backward()
        now = {n: t.clone() for n, t in p.outputs().items()}
        if first is not None:
            for n in now:
                assert torch.equal(now[n], first[n]), n
        first = now


def test_gradients_are_differences(eq):
    """fp32 gradients against differences of the forward: a step h of 2^-7 costs h^2 / 6 of a third derivative (of
    order 1 here) and 2^-24 times the outputs' sum over h, both below 1e-3 of gradients of order 1."""
    import torch
    p = Problem(eq, F32, 2, 2, 1, 4, 4, [20], causal=True, buckets=4, reach=9, packed=False, seed=8)

    def loss():
        p.forward()
        return (p.o.double() * p.do.double()).sum().item()

    p.forward()
    p.backward()
    for t, g in ((p.q, p.dq), (p.k, p.dk_), (p.v, p.dv_), (p.bias, p.dbias)):
        for i in range(0, t.numel(), max(1, t.numel() // 12)):
            flat = t.view(-1)
            x, h = flat[i].item(), 2.0 ** -7
            flat[i] = x + h
            up = loss()
            flat[i] = x - h
            down = loss()
            flat[i] = x
            assert abs((up - down) / (2 * h) - g.view(-1)[i].item()) < 2e-3


@pytest.mark.parametrize("dt", [BF16, F32])
def test_captured_and_on_another_stream(eq, dt):
    import torch
    p = Problem(eq, dt, 8, 3, 1, 8, 8, [100, 29], causal=True, buckets=8, reach=40, seed=9)
    ws = p.workspace(True)
    p.forward()
    p.backward(workspace=ws)
    want = {n: t.clone() for n, t in p.outputs().items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in p.outputs().values():
            t.fill_(7.0)
        p.forward()
        p.backward(workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    for n, t in p.outputs().items():
        assert torch.equal(t, want[n]), n
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.forward()
        p.backward(workspace=ws)
    for k in range(3):
        p.q.mul_(0.5)
        for t in p.outputs().values():
            t.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in p.outputs().items()}
        p.forward()
        p.backward(workspace=ws)
        torch.cuda.synchronize()
        for n, t in p.outputs().items():
            assert torch.equal(t, got[n]), (n, k)

"""The fp64 definitions of softmax attention and its cache, checked against loops, differences and the
symmetries they must have, and the plan's buckets against whole numbers (CPU)."""
import numpy as np
import pytest

from oracle import attention as att


def _head(rng, n_q, n_k, Dk, Dv):
    return rng.standard_normal((n_q, Dk)), rng.standard_normal((n_k, Dk)), rng.standard_normal((n_k, Dv))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n_q,n_k", [(5, 5), (3, 7), (6, 2), (1, 1)])
def test_forward_is_the_sum(causal, n_q, n_k):
    rng = np.random.default_rng(0)
    q, k, v = _head(rng, n_q, n_k, 3, 4)
    bias = rng.standard_normal(8)
    h = att.Head(q, k, v, 0.7, causal, bias, 6)
    for i in range(n_q):
        p = i + n_k - n_q
        w = {j: np.exp(0.7 * q[i] @ k[j] + bias[att.bucket(p - j, 8, 6, causal)]) for j in range(n_k) if not causal or j <= p}
        if not w:
            assert np.all(h.o[i] == 0) and h.lse[i] == -np.inf
            continue
        assert np.allclose(h.lse[i], np.log(sum(w.values())), rtol=1e-13)
        assert np.allclose(h.o[i], sum(w[j] * v[j] for j in w) / sum(w.values()), rtol=1e-12)


@pytest.mark.parametrize("causal", [False, True])
def test_gradients_are_differences(causal):
    rng = np.random.default_rng(1)
    q, k, v = _head(rng, 4, 6, 3, 2)
    bias, do = rng.standard_normal(8), rng.standard_normal((4, 2))
    loss = lambda q, k, v, b: (att.Head(q, k, v, 0.6, causal, b, 5).o * do).sum()  # noqa: E731
    h = att.Head(q, k, v, 0.6, causal, bias, 5).backward(do, 8)
    args = [q, k, v, bias]
    for i, g in enumerate((h.dq, h.dk, h.dv, h.dbias)):
        for at in np.ndindex(*args[i].shape):
            e = 1e-6
            up, down = [x.copy() for x in args], [x.copy() for x in args]
            up[i][at] += e
            down[i][at] -= e
            assert abs((loss(*up) - loss(*down)) / (2 * e) - g[at]) < 1e-7


def test_attention_commutes_with_a_shift_of_the_group_axis():
    rng = np.random.default_rng(2)
    N, d = 5, 3
    q, k, v = (rng.standard_normal((6, d, N)) for _ in range(3))
    run = lambda q, k, v: att.Head(*(x.reshape(6, -1) for x in (q, k, v)), 0.3, True, np.arange(4.0), 7).o  # noqa: E731
    roll = lambda x: np.roll(x, 2, axis=2)  # noqa: E731
    assert np.allclose(run(roll(q), roll(k), roll(v)), roll(run(q, k, v).reshape(6, d, N)).reshape(6, -1), rtol=1e-12)


def test_what_is_not_seen_is_no_term():
    rng = np.random.default_rng(3)
    q, k, v = _head(rng, 4, 4, 2, 2)
    a = att.Head(q, k, v, 1.0, True).o
    v[3], k[3] = np.nan, np.inf
    assert np.array_equal(att.Head(q, k, v, 1.0, True).o[:3], a[:3])


def test_step_is_the_last_row():
    rng = np.random.default_rng(4)
    k, v, q = rng.standard_normal((9, 2, 3)), rng.standard_normal((9, 2, 4)), rng.standard_normal((1, 4, 3))
    bias = rng.standard_normal((4, 6))
    kc, vc = np.full((5, 4, 2, 3), np.nan), np.full((5, 4, 2, 4), np.nan)
    table = np.array([[3, 0, 4, -1]])
    for j in range(9):
        kc[table[0, j // 4], j % 4], vc[table[0, j // 4], j % 4] = k[j], v[j]
    o, lse = att.step(q, kc, vc, table, [9], 0.5, bias, 7)
    for h in range(4):
        full = att.Head(q[:, h], k[:, h // 2], v[:, h // 2], 0.5, True, bias[h], 7)
        assert np.allclose(o[0, h], full.o[0], rtol=1e-12) and np.allclose(lse[h, 0], full.lse[0], rtol=1e-12)


def test_tables_by_hand():
    table = np.full((3, 3), 9, np.int32)
    table[0, 0], table[1, :2] = 5, (6, 2)
    out = att.tables([3, 8, 0], [2, 0, 5], [7, 1, 0, 3], 1, table, 4, 8)
    assert out[0].tolist() == [[5, 1, 9], [6, 2, 9], [0, 3, 9]]
    assert out[1].tolist() == [5, 8, 5] and out[2] == 4
    assert out[3].tolist() == [23, 4, 0, 1, 2, 3, 12, -1]
    assert out[4].tolist() == [3, 4, 0, 1, 2, 3, 4, 0]
    assert out[5].tolist() == [0, 2, 2, 7]


@pytest.fixture(scope="module")
def eq():
    import group_equivariant_linear_amd as eq
    from group_equivariant_linear_amd import _build
    if not eq.built():
        _build.build()
    eq.load_library()
    return eq


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("buckets,reach", [(4, 3), (6, 4), (8, 20), (8, 16), (16, 64), (32, 128), (32, 1024), (34, 129), (64, 500),
                                           (10, 1000), (128, 1024), (256, 1024), (256, 200), (18, 8 * 27)])
def test_buckets_of_a_plan(eq, causal, buckets, reach):
    p = eq.eqlinear_attention_plan(1, 1, 1, 4, 4, eq.EQL_F32, causal=causal, buckets=buckets, max_distance=reach)
    far = [2 * reach, 1 << 40, (1 << 63) - 1]
    for d in list(range(reach + 3)) + far:
        n = min(d, reach)  # all from the reach on are alike
        assert eq.eqlinear_attention_bucket(p, d) == att.bucket(n, buckets, reach, causal)
        assert eq.eqlinear_attention_bucket(p, -d) == (att.bucket(-n, buckets, reach, causal) if not causal or d == 0 else -1)
    assert eq.eqlinear_attention_bucket(p, -(1 << 63)) == (-1 if causal else buckets - 1)
    assert att.bucket(reach, buckets, reach, True) == buckets - 1

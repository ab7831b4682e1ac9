"""The fp64 definitions of the operators between the layers, checked against recurrences,
differences and the symmetries they must have (CPU)."""
import numpy as np
import pytest

from oracle import operators as ops


def _mix_inputs(rng, T, H, K, Dk, Dv, B):
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    return (n(T, H, Dk), n(T, K, Dk), n(T, K, Dv), -np.abs(n(K)) * 0.2, n(B, K, Dk, Dv), n(T, H, Dv),
            n(B, K, Dk, Dv))


def test_linear_attention_is_the_recurrence():
    rng = np.random.default_rng(0)
    q, k, v, la, S0, _, _ = _mix_inputs(rng, 9, 4, 2, 3, 5, 3)
    off = [0, 5, 5, 9]
    r = ops.linear_attention(q, k, v, la, 0.7, off, S0)
    for b in range(3):
        for h in range(4):
            g, S = h // 2, S0[b, h // 2].copy()
            for t in range(off[b], off[b + 1]):
                S = np.exp(la[g]) * S + np.outer(k[t, g], v[t, g])
                assert np.allclose(r["o"][t, h], 0.7 * q[t, h] @ S, rtol=1e-12, atol=1e-12)
            assert np.allclose(r["S1"][b, g], S, rtol=1e-12, atol=1e-12)


def test_linear_attention_gradients_are_differences():
    rng = np.random.default_rng(1)
    q, k, v, la, S0, do, dS1 = _mix_inputs(rng, 7, 4, 2, 3, 2, 2)
    off = [0, 4, 7]

    def loss(q, k, v, S0):
        r = ops.linear_attention(q, k, v, la, 0.6, off, S0)
        return (r["o"] * do).sum() + (r["S1"] * dS1).sum()

    r = ops.linear_attention(q, k, v, la, 0.6, off, S0, do, dS1)
    args = [q, k, v, S0]
    for i, name in enumerate(("dq", "dk", "dv", "dS0")):
        for _ in range(12):
            d = np.zeros_like(args[i])
            d[tuple(rng.integers(0, s) for s in d.shape)] = 1e-6
            num = (loss(*(a + d if j == i else a for j, a in enumerate(args)))
                   - loss(*(a - d if j == i else a for j, a in enumerate(args)))) / 2e-6
            assert abs(num - (r[name] * d).sum() / 1e-6) <= 1e-6 * (1 + abs(num)), name


def test_no_memory_is_the_token_alone():
    rng = np.random.default_rng(2)
    q, k, v, _, S0, _, _ = _mix_inputs(rng, 4, 1, 1, 3, 2, 1)
    r = ops.linear_attention(q, k, v, np.array([-np.inf]), 1.0, [0, 4], S0)
    for t in range(4):
        assert np.allclose(r["o"][t, 0], (q[t, 0] @ k[t, 0]) * v[t, 0])


@pytest.mark.parametrize("act", [ops.NONE, ops.GELU, ops.SILU])
def test_group_norm_gradients_are_differences(act):
    rng = np.random.default_rng(3)
    T, C, N, G, off = 7, 6, 3, 2, [0, 4, 4, 5, 7]
    x, dy = rng.standard_normal((T, C, N)), rng.standard_normal((T, C, N))
    gamma, beta = 1 + 0.3 * rng.standard_normal(C), 0.3 * rng.standard_normal(C)

    def loss(x, gamma, beta):
        return (ops.group_norm(x, gamma, beta, G, 1e-3, act, off)["y"] * dy).sum()

    r = ops.group_norm(x, gamma, beta, G, 1e-3, act, off, dy)
    args = [x, gamma, beta]
    for i, name in enumerate(("dx", "dgamma", "dbeta")):
        for _ in range(10):
            d = np.zeros_like(args[i])
            d[tuple(rng.integers(0, s) for s in d.shape)] = 1e-6
            num = (loss(*(a + d if j == i else a for j, a in enumerate(args)))
                   - loss(*(a - d if j == i else a for j, a in enumerate(args)))) / 2e-6
            assert abs(num - (r[name] * d).sum() / 1e-6) <= 2e-6 * (1 + abs(num)), name


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_scores_depend_on_the_distance(interleaved):
    rng = np.random.default_rng(4)
    x, y = rng.standard_normal((1, 1, 8, 3)), rng.standard_normal((1, 1, 8, 3))
    f = ops.rotary_frequencies(6)
    at = lambda z, p: ops.rotary(z, np.array([p]), f, 6, interleaved)  # noqa: E731
    assert np.isclose((at(x, 11) * at(y, 4)).sum(), (at(x, 1007) * at(y, 1000)).sum())
    z = ops.rotary(at(x, 5), np.array([5]), f, 6, interleaved, inverse=True)
    assert np.allclose(z, x) and np.array_equal(at(x, 5)[:, :, 6:], x[:, :, 6:])


def test_rotary_scalings():
    f = ops.rotary_frequencies(16)
    assert np.allclose(ops.rotary_frequencies(16, scaling="linear", factor=4.0), f / 4)
    g = ops.rotary_frequencies(16, scaling="raised", factor=4.0)
    assert np.isclose(g[0], f[0]) and np.isclose(g[-1], f[-1] / 4)
    g = ops.rotary_frequencies(16, scaling="banded", factor=4.0, context=4096.0)
    assert np.isclose(g[0], f[0]) and np.isclose(g[-1], f[-1] / 4) and np.all(g <= f) and np.all(g >= f / 4)


def test_operators_commute_with_the_group():
    """A cyclic shift of every record's group axis passes through each operator."""
    rng = np.random.default_rng(5)
    T, H, d, N = 6, 2, 4, 5
    q, k, v, dy = (rng.standard_normal((T, H, d, N)) for _ in range(4))
    roll = lambda z: np.roll(z, 2, axis=-1)  # noqa: E731
    f, pos = ops.rotary_frequencies(4), np.arange(T)
    assert np.allclose(ops.rotary(roll(q), pos, f, 4, True), roll(ops.rotary(q, pos, f, 4, True)))
    la = np.log([0.9, 0.7])

    def mix(q, k, v):
        return ops.linear_attention(*(z.reshape(T, H, d * N) for z in (q, k, v)), la, 1.0, [0, 2, 6])["o"].reshape(
            T, H, d, N)

    assert np.allclose(mix(roll(q), roll(k), roll(v)), roll(mix(q, k, v)))
    norm = lambda x: ops.group_norm(x.reshape(T, H * d, N), np.arange(8.0), np.ones(8), 2, 1e-5, ops.SILU,  # noqa: E731
                                    [0, 2, 6])["y"].reshape(T, H, d, N)
    assert np.allclose(norm(roll(dy)), roll(norm(dy)))

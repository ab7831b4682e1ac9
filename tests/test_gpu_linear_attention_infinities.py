"""Linear attention with infinities: the state that the formula gives, and no trace of them elsewhere.

A single infinite value v[t, c] makes column c of the state k_t times it, an infinity of k's sign in
every row, from token t on; a single infinite number of state_in stays one.  All else has the bits
that a 0 in its place gives: nothing here has a tolerance.
"""
import numpy as np
import pytest

import synthetic
from gpu_util import to_f64
from test_gpu_linear_attention import Problem, eq  # noqa: F401  (eq is the fixture)

pytestmark = pytest.mark.gpu

F32, BF16, F16 = synthetic.F32, synthetic.BF16, synthetic.F16
OUTPUTS = ("o", "S1", "dq", "dk_", "dv_", "dS0")

# (heads, kv heads, d_k, d_v, lengths): one chunk, several, packed; sums over segments; heads that fill no tile
SIZES = [(2, 2, 8, 8, [40]), (4, 2, 8, 4, [150]), (2, 1, 5, 11, [30, 0, 200, 9]), (2, 1, 8, 8, [1100])]


def problem(eq, dt, size, seed):
    H, K, dk, dv, lens = size
    return Problem(eq, dt, 8, H, K, dk, dv, lens, len(lens) > 1, seed, log_decay=[-0.01, -0.02][:K])


def results(p):
    import torch
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    return {n: getattr(p, n).flatten(2).clone() if n[0] != "S" and n != "dS0" else getattr(p, n).clone() for n in OUTPUTS}


def same_but(a, b, name, mask, what):
    """The bits of a and b alike outside mask."""
    import torch
    m = torch.broadcast_to(mask, a[name].shape)
    assert torch.equal(a[name][~m], b[name][~m]), f"{what}: {name} differs elsewhere"
    return b[name][m]


def sign_inf(x):
    return np.sign(x) * np.inf


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("which", ["v", "d_o"])
def test_an_infinite_row_number(eq, dt, size, sign, which):
    """v: state_out; d_o: d_state_in.  The token lies past the middle, in the longest sequence."""
    import torch
    p = problem(eq, dt, size, 31)
    seq = int(np.argmax(p.lens))
    t0, t1 = int(p.off[seq]), int(p.off[seq + 1])
    at, c = t0 + (t1 - t0) * 5 // 8, p.dv * p.N - 3
    g = p.K - 1
    h = g if which == "v" else p.H - 1  # d_o: the last query head, of the last kv head
    x = getattr(p, which)
    x[at, h, c // p.N, c % p.N] = 0
    clean = results(p)
    x[at, h, c // p.N, c % p.N] = sign * float("inf")
    got = results(p)
    what = f"{dt} {size} {which}"
    state, rows = ("S1", p.k[at, g]) if which == "v" else ("dS0", p.q[at, h])
    column = torch.zeros(p.S1.shape, dtype=torch.bool, device="cuda")
    column[seq, g, :, c] = True
    column = same_but(clean, got, state, column, what)
    rows = to_f64(rows).reshape(-1) * sign * np.sign(p.scale)
    assert np.all(rows != 0)
    assert np.array_equal(to_f64(column), sign_inf(rows)), f"{what}: {state}"
    # the rows of o (dv) that see it: the later (earlier) tokens of the sequence, this column
    name, heads = ("o", slice(g * (p.H // p.K), p.H)) if which == "v" else ("dv_", slice(g, g + 1))
    seen = torch.zeros(clean[name].shape, dtype=torch.bool, device="cuda")
    seen[slice(at, t1) if which == "v" else slice(t0, at + 1), heads, c] = True
    assert not torch.isfinite(same_but(clean, got, name, seen, what)).any(), f"{what}: {name}"


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("which", ["S0", "dS1"])
def test_an_infinite_state(eq, dt, size, which):
    import torch
    p = problem(eq, dt, size, 32)
    seq, g = int(np.argmax(p.lens)), p.K - 1
    s = slice(int(p.off[seq]), int(p.off[seq + 1]))
    i, c = 3, p.dv * p.N - 2
    x = getattr(p, which)
    x[seq, g, i, c] = 0
    clean = results(p)
    x[seq, g, i, c] = float("inf")
    got = results(p)
    what = f"{dt} {size} {which}"
    one = torch.zeros(p.S1.shape, dtype=torch.bool, device="cuda")
    one[seq, g, i, c] = True
    state = "S1" if which == "S0" else "dS0"
    assert same_but(clean, got, state, one, what).tolist() == [float("inf")], f"{what}: {state}"
    heads = slice(g * (p.H // p.K), p.H)
    kv = slice(g, g + 1)
    # a row of each output takes the infinite number times one of its own factor's
    for name, hs, col, factor in ((("o", heads, c, p.q.flatten(2)[s, heads, i]),
                                   ("dq", heads, i, p.d_o.flatten(2)[s, heads, c])) if which == "S0" else
                                  (("dv_", kv, c, p.k.flatten(2)[s, kv, i]), ("dk_", kv, i, p.v.flatten(2)[s, kv, c]))):
        mask = torch.zeros(clean[name].shape, dtype=torch.bool, device="cuda")
        mask[s, hs, col] = True
        y = same_but(clean, got, name, mask, what).view(-1, factor.shape[1])
        f = to_f64(factor)
        want = np.where(f == 0, np.nan, sign_inf(f * np.sign(p.scale)))
        assert np.array_equal(to_f64(y), want, equal_nan=True), f"{what}: {name}"

"""Linear attention where the numbers of a 16-bit plan leave the middle of its range, against the fp64 definition.

Error bound of every element, u = 2^-11 (fp16).  An output is rounded once: u |ref|, and below
fp16's normal range 2^-25.  A decayed score is rounded once: u of it, and where it lies far
below its row's largest an absolute 2^-17 of that (a row's scores enter the product times a power
of two that makes their largest 2^-8 or more: 2^-25 / 2^-8).  The state
and the decayed rows are two truncated terms of 11 bits: 4 u^2 of the sum of absolute products
(2^-21 each at most, and the floor 2^-24 under a column whose largest is 1 or more).  fp32 sums
add their length times 2^-24 of that sum.  Nothing else: no floor for the fp32 states.
"""
import numpy as np
import pytest

import synthetic
from gpu_util import to_f64
from oracle import operators as ops
from test_gpu_linear_attention import E32, U, Problem, eq  # noqa: F401  (eq is the fixture)

pytestmark = pytest.mark.gpu

F32, BF16, F16 = synthetic.F32, synthetic.BF16, synthetic.F16
CHUNK = 64


def sized(p, **factors):
    """The problem with its q, k, v, d_o, S0, dS1 multiplied (numbers, or arrays that broadcast)."""
    import torch
    for name, f in factors.items():
        t = getattr(p, name)
        t.copy_((t.double() * torch.as_tensor(f, dtype=torch.float64, device="cuda")).to(t.dtype))
    return p


def peaks(a):
    """Sums of |c| times the largest decayed score of the row, over the chunks' rows, for o, dq, dk, dv."""
    r = a["q"].shape[1] // a["k"].shape[1]
    out = {"o": np.zeros((*a["q"].shape[:2], a["v"].shape[2])), "dq": np.zeros(a["q"].shape),
           "dk": np.zeros(a["k"].shape), "dv": np.zeros(a["v"].shape)}
    for b in range(len(a["offsets"]) - 1):
        for h in range(a["q"].shape[1]):
            s, g = slice(int(a["offsets"][b]), int(a["offsets"][b + 1])), h // r
            q, k, v, do = a["q"][s, h], a["k"][s, g], a["v"][s, g], a["do"][s, h]
            t = np.arange(len(q))
            near = ops._powers(a["log_decay"][g], t[:, None] - t[None, :]) * abs(a["scale"])
            # chunks start at a multiple of 64 tokens of the sequence (segments too)
            near[t[:, None] // CHUNK != t[None, :] // CHUNK] = 0
            seen = near > 0
            P, dP = np.abs(q @ k.T) * near, np.abs(do @ v.T) * near
            most = lambda x, axis: x.max(axis=axis, initial=0, keepdims=True) * seen  # noqa: E731
            out["o"][s, h] = most(P, 1) @ np.abs(v)
            out["dq"][s, h] = most(dP, 1) @ np.abs(k)
            out["dk"][s, g] += most(dP, 0).T @ np.abs(q)
            out["dv"][s, g] += most(P, 0).T @ np.abs(do)
    return out


ROWS, STATES = ("o", "dq", "dk", "dv"), ("S1", "dS0")


def check(p, what, names):
    a = p.host()
    ref = ops.linear_attention(**a)
    scores = ops.linear_attention(**a, absolute="scores")
    every = ops.linear_attention(**a, absolute="all")
    peak, u = peaks(a), U[p.dt]
    got = {"o": p.o, "S1": p.S1, "dq": p.dq, "dk": p.dk_, "dv": p.dv_, "dS0": p.dS0}
    length = p.H // p.K * (max(p.lens) + 128) + 64
    for name in names:
        t = got[name]
        y = to_f64(t).reshape(ref[name].shape)
        tol = (E32 if name in ("S1", "dS0") else u) * np.abs(ref[name]) + (length * E32 + 4 * u * u) * every[name]
        if name not in ("S1", "dS0"):
            assert np.max(np.abs(ref[name])) < 60000, f"{what}: {name} would not fit"
            tol = tol + u * (1 + u) * scores[name] + 2.0 ** -17 * peak[name] + 2.0 ** -25
        assert np.all(np.isfinite(y)), f"{what}: {name} not finite"
        err = np.abs(y - ref[name])
        assert np.all(err <= tol), (f"{what}: {name} {int((err > tol).sum())} of {err.size} out of bounds, worst "
                                    f"{np.max(err / np.maximum(tol, 1e-300)):.3g} times")


def run(p, what, names=ROWS):
    import torch
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    check(p, what, names)


SIZES = [(1, 1, 1, 128, 128, [70]), (8, 4, 2, 8, 8, [1, 130, 0, 33]), (7, 2, 2, 9, 5, [100]), (8, 2, 1, 8, 8, [1100]),
         (8, 2, 2, 4, 16, [17, 64])]


def problem(eq, size, seed, **kw):
    N, H, K, dk, dv, lens = size
    return Problem(eq, F16, N, H, K, dk, dv, lens, len(set(lens)) > 1, seed, **kw)


# --- scores -----------------------------------------------------------------------------

@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("which", ["qk", "vd"])
def test_scores_past_the_range_of_fp16(eq, size, which):
    """Scores of up to about 1e5 in o and dv (or, of d_o and v, in dq and dk), outputs of a few thousand."""
    p = problem(eq, size, 21)
    big, small = (("q", "k"), ("v", "d_o")) if which == "qk" else (("v", "d_o"), ("q", "k"))
    sized(p, **{n: 160.0 for n in big}, **{n: 0.01 for n in small}, S0=0.01, dS1=0.01)
    run(p, f"{size} {which}")


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_one_row_past_the_range(eq, size):
    """One token's query (and d_o) far larger than the others'."""
    import torch
    p = problem(eq, size, 22)
    f = torch.ones(p.T, 1, 1, 1, dtype=torch.float64)
    f[0], f[p.T // 2], f[-1] = 9000.0, 2e-3, 2000.0
    sized(p, q=f, k=4.0, v=0.01, d_o=0.01)
    run(p, f"{size}")


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("f", [1e-3, 1e-5])
def test_small_scores(eq, size, f):
    """Scores of 1e-3 and 1e-5, values large enough for the outputs to be ordinary numbers."""
    p = problem(eq, size, 23)
    run(sized(p, q=f, v=300.0, S0=300.0), f"{size} q {f}")
    p = problem(eq, size, 24)
    run(sized(p, d_o=f, k=300.0, q=300.0, S0=1e-3, v=1e-3), f"{size} d_o {f}")


def test_scale_far_from_one(eq):
    run(sized(problem(eq, SIZES[1], 25, scale=2.0 ** -20), v=2000.0, k=100.0, S0=2000.0, dS1=0.1), "scale 2^-20")
    run(sized(problem(eq, SIZES[1], 26, scale=4096.0), q=0.01, v=0.01, S0=0.01, d_o=0.01, k=0.01, dS1=0.01), "scale 4096")


# --- states -----------------------------------------------------------------------------

@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("f", [1e-2, 1e-3, 1e-4, 1e-5, 100.0])
@pytest.mark.parametrize("which", ["v", "d_o"])
def test_states_of_small_and_large_rows(eq, size, f, which):
    """state_out is made of v, d_state_in of d_o: both keep fp32's accuracy whatever the size of either."""
    p = problem(eq, size, 27, state=False)
    p.dS1 = None
    run(sized(p, **{which: f}), f"{size} {which} {f}", STATES)


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_columns_of_unlike_sizes(eq, size):
    """Channels of v, q and d_o from 1 down to 1e-5 side by side, and states to match."""
    p = problem(eq, size, 28)
    channels = lambda d: 10.0 ** -(np.arange(d) % 6)[:, None]  # noqa: E731
    numbers = lambda d: np.repeat(10.0 ** -(np.arange(d) % 6), p.N)  # noqa: E731
    sized(p, v=channels(p.dv), d_o=channels(p.dv), S0=numbers(p.dv), dS1=numbers(p.dv))
    run(p, f"{size}", ROWS + STATES)


@pytest.mark.parametrize("lens", [[40, 100], [1100]], ids=str)
def test_large_state_with_small_rows(eq, lens):
    """A state of 1e30 keeps its size while rows of 1e-5 join it, and a state near fp32's top stays finite."""
    import torch
    for big in (1e30, 2.0 ** 119):
        p = Problem(eq, F16, 8, 2, 1, 8, 8, lens, len(lens) > 1, 29, log_decay=[-0.001])
        sized(p, v=1e-5)
        p.S0.fill_(big)
        p.forward()
        torch.cuda.synchronize()
        for b, n in enumerate(lens):
            want = big * np.exp(np.float64(np.float32(-0.001)) * n)
            assert np.all(np.abs(to_f64(p.S1[b]) / want - 1) <= (n + 64) * E32)

"""Linear attention with decays (prompt, gradients, single tokens) against its fp64 definition.

Error bound of every element, from the arithmetic.  With u the plan dtype's unit roundoff
(2^-24, 2^-8, 2^-11), an output is rounded once (u |ref|).  16-bit plans round each decayed
score once (u times the sum of |score| |value|) and carry the state and the decayed values as
two terms (u^2 of the sum of all absolute products, each); fp32 sums add at most their length
times 2^-24 of that sum.  fp16 has an absolute floor of 2^-25 per rounded term instead of u
below its normal range.
"""
import numpy as np
import pytest

import synthetic
from gpu_util import to_f64, torch_dtype
from oracle import operators as ops

pytestmark = pytest.mark.gpu

F32, BF16, F16 = synthetic.F32, synthetic.BF16, synthetic.F16
U = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
E32 = 2.0 ** -24


@pytest.fixture(scope="module")
def eq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import group_equivariant_linear_amd as eq
    eq.load_library()
    return eq


def _eqdt(eq, dt):
    return {F32: eq.EQL_F32, BF16: eq.EQL_BF16, F16: eq.EQL_F16}[dt]


class Problem:
    def __init__(self, eq, dt, N, H, K, dk, dv, lens, ragged, seed, fused=True, state=True, log_decay=None, scale=None,
                 odd=False):
        import torch
        self.eq, self.dt, self.lens, self.ragged = eq, dt, lens, ragged
        self.N, self.H, self.K, self.dk, self.dv = N, H, K, dk, dv
        self.B, self.T = len(lens), int(sum(lens))
        self.off = np.concatenate([[0], np.cumsum(lens)])
        self.scale = scale if scale is not None else float(np.float32(1 / np.sqrt(dk * N)))
        self.plan = eq.eqlinear_mixer_plan(N, H, K, dk, dv, _eqdt(eq, dt))
        g = torch.Generator().manual_seed(seed)
        self.g = g
        tdt = torch_dtype(dt)
        parts = [(H, dk), (K, dk), (K, dv)]
        W = sum(h * d for h, d in parts)

        def views(fill):
            if not fused:
                return [fill(self.T, h, d, N) for h, d in parts]
            # one element of slack before each row when odd: rows that start at no vector boundary
            buf = fill(self.T, W * N + (1 if odd else 0))
            at, out = (1 if odd else 0), []
            for h, d in parts:
                out.append(buf.as_strided((self.T, h, d, N), (buf.stride(0), d * N, N, 1), at))
                at += h * d * N
            self.keep = getattr(self, "keep", []) + [buf]
            return out

        rand = lambda *s: torch.randn(*s, generator=g).to(tdt).cuda()  # noqa: E731
        self.q, self.k, self.v = views(rand)
        self.d_o = rand(self.T, H, dv, N)
        self.dq, self.dk_, self.dv_ = views(lambda *s: torch.full(s, 7.0, dtype=tdt, device="cuda"))
        self.o = torch.full((self.T, H, dv, N), float("nan"), dtype=tdt, device="cuda")
        la = -np.abs(np.random.default_rng(seed).standard_normal(K)) * 0.2 if log_decay is None else log_decay
        self.la = torch.tensor(np.asarray(la, dtype=np.float32)).cuda()
        sh = (self.B, K, dk * N, dv * N)
        self.S0 = torch.randn(*sh, generator=g).cuda() if state else None
        self.dS1 = torch.randn(*sh, generator=g).cuda() if state else None
        self.S1 = torch.full(sh, float("nan"), device="cuda")
        self.dS0 = torch.full(sh, float("nan"), device="cuda")
        self.offsets = torch.tensor(self.off, dtype=torch.int64).cuda() if ragged else None

    def workspace(self, backward):
        import torch
        n = self.eq.eqlinear_linear_attention_workspace(self.plan, self.T, self.B, backward=backward)
        return torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") if n else None  # NaNs to whoever reads them

    def forward(self, stream=None):
        self.eq.eqlinear_linear_attention(self.plan, self.q, self.k, self.v, self.la, self.o, scale=self.scale,
                                          offsets=self.offsets, batch=self.B, state_in=self.S0, state_out=self.S1,
                                          workspace=self.workspace(False), stream=stream)

    def backward(self, stream=None):
        self.eq.eqlinear_linear_attention_backward(
            self.plan, self.q, self.k, self.v, self.d_o, self.la, self.dq, self.dk_, self.dv_, scale=self.scale,
            offsets=self.offsets, batch=self.B, state_in=self.S0, dstate_out=self.dS1, dstate_in=self.dS0,
            workspace=self.workspace(True), stream=stream)

    def host(self):
        f = lambda t: None if t is None else to_f64(t)  # noqa: E731
        flat = lambda t: to_f64(t).reshape(t.shape[0], t.shape[1], -1)  # noqa: E731
        return dict(q=flat(self.q), k=flat(self.k), v=flat(self.v), log_decay=f(self.la), scale=self.scale,
                    offsets=self.off, S0=f(self.S0), do=flat(self.d_o), dS1=f(self.dS1))

    def check(self, what, grads=True):
        a = self.host()
        ref = ops.linear_attention(**a)
        scores = ops.linear_attention(**a, absolute="scores")
        every = ops.linear_attention(**a, absolute="all")
        flat_one = dict(a, log_decay=np.zeros(self.K))
        for n in ("q", "k", "v", "do"):
            flat_one[n] = np.maximum(np.abs(a[n]), 1.0)
        most = ops.linear_attention(**flat_one, absolute="all")
        u = U[self.dt]
        got = {"o": self.o, "S1": self.S1}
        if grads:
            got |= {"dq": self.dq, "dk": self.dk_, "dv": self.dv_, "dS0": self.dS0}
        for name in ("S1", "dS0"):  # fp32 outputs: what lies below their range is 0
            if name in ref:
                ref[name] = ref[name].astype(np.float32).astype(np.float64)
        for name, t in got.items():
            y = to_f64(t).reshape(ref[name].shape)
            assert np.all(np.isfinite(y)), f"{what}: {name} not finite"
            out_u = E32 if name in ("S1", "dS0") else u
            # several query heads share the sums of dk, dv and dS0
            length = self.H // self.K * (max(self.lens, default=0) + 128) + 64
            tol = out_u * np.abs(ref[name]) + length * E32 * every[name]
            if self.dt != F32:
                tol = tol + u * (1 + u) * scores[name] + 4 * u * u * every[name]
            if self.dt == F16:
                tol = tol + 2.0 ** -25 * most[name]
            bad = np.abs(y - ref[name]) > tol
            assert not bad.any(), (f"{what}: {name} {int(bad.sum())} of {bad.size} out of bounds, worst "
                                   f"{np.max(np.abs(y - ref[name]) / np.maximum(tol, 1e-300)):.3g} times")


def run(p, what):
    import torch
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    p.check(what)


LENS = [[1], [5], [64], [65], [130, 130], [0, 1, 63, 64, 200], [17, 0, 0, 129]]


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_lengths(eq, dt, lens):
    run(Problem(eq, dt, 8, 4, 2, 4, 4, lens, len(set(lens)) > 1, seed=1), f"{dt} {lens}")


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("N,H,K,dk,dv", [(8, 2, 2, 8, 8), (8, 3, 1, 16, 16), (7, 2, 2, 16, 16), (1, 2, 1, 2, 3),
                                         (5, 2, 2, 7, 3), (1, 1, 1, 1, 128), (1, 1, 1, 128, 1), (16, 2, 1, 8, 2),
                                         (3, 2, 2, 11, 32), (6, 4, 4, 5, 21), (8, 12, 4, 8, 8), (1, 2, 2, 96, 72)])
def test_head_sizes(eq, dt, N, H, K, dk, dv):
    run(Problem(eq, dt, N, H, K, dk, dv, [70, 9, 130], True, seed=N + dk), f"{dt} N={N} {H}/{K} heads {dk} {dv}")


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("fused,odd,state", [(False, False, True), (True, True, True), (True, False, False),
                                             (False, False, False)])
def test_layouts_and_states(eq, dt, fused, odd, state):
    run(Problem(eq, dt, 7, 2, 1, 9, 5, [100, 100], False, seed=3, fused=fused, odd=odd, state=state),
        f"{dt} fused={fused} odd={odd} state={state}")


@pytest.mark.parametrize("dt", [F32, BF16, F16])
def test_long_sequences(eq, dt):
    """Few sequences and heads: the token axis is what there is to split."""
    run(Problem(eq, dt, 8, 2, 1, 8, 8, [3001], False, seed=5, log_decay=[-0.001]), f"{dt} one of 3001")
    run(Problem(eq, dt, 4, 1, 1, 5, 6, [1500, 0, 700, 3], True, seed=6, log_decay=[-0.003]), f"{dt} 1500, 0, 700, 3")


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("la", [0.0, -1e-4, -3.0, -200.0, -np.inf])
def test_decays(eq, dt, la):
    """From a plain running sum to no memory at all."""
    run(Problem(eq, dt, 8, 2, 2, 4, 4, [150, 40], True, seed=7, log_decay=[la, -0.05]), f"{dt} log decay {la}")


@pytest.mark.parametrize("dt", [BF16, F16])
def test_nothing_leaks_between_sequences_or_over_the_ends(eq, dt):
    """NaN in a sequence stays in it; padding that lies between rows is neither read nor written."""
    import torch
    p = Problem(eq, dt, 8, 2, 2, 4, 4, [70, 33, 64], True, seed=8)
    p.q[70:103] = float("nan")
    p.k[70:103] = float("inf")
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    for t in (p.o, p.dq, p.dk_, p.dv_):
        assert torch.isfinite(t[:70]).all() and torch.isfinite(t[103:]).all()
        assert not torch.isfinite(t[70:103]).all()
    assert torch.isfinite(p.S1[[0, 2]]).all() and torch.isfinite(p.dS0[[0, 2]]).all()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_later_tokens_do_not_reach_earlier_outputs(eq, dt):
    import torch
    p = Problem(eq, dt, 8, 2, 2, 8, 4, [90], False, seed=9)
    p.forward()
    first = p.o.clone()
    p.k[50:] = float("nan")
    p.v[50:] = float("inf")
    p.forward()
    torch.cuda.synchronize()
    assert torch.equal(first[:48], p.o[:48])


def test_outputs_only(eq):
    """Nothing but the output rows is written: the rest of a wide gradient buffer keeps its values."""
    import torch
    p = Problem(eq, BF16, 7, 2, 1, 3, 5, [77], False, seed=10, odd=True)
    p.backward()
    torch.cuda.synchronize()
    assert torch.all(p.keep[1][:, 0] == 7.0)  # the slack element of every row


def test_same_bits_every_time_and_on_another_stream(eq):
    import torch
    p = Problem(eq, BF16, 8, 6, 2, 8, 8, [300, 40, 511], True, seed=11)
    outs = []
    for _ in range(3):
        p.forward()
        p.backward()
        outs.append([t.clone() for t in (p.o, p.S1, p.dq, p.dk_, p.dv_, p.dS0)])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p.forward()
        p.backward(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    outs.append([p.o, p.S1, p.dq, p.dk_, p.dv_, p.dS0])
    torch.cuda.synchronize()
    for o in outs[1:]:
        for a, b in zip(outs[0], o):
            assert torch.equal(a, b)


def test_state_carries_a_prompt_over_calls(eq):
    """Two halves with the state between them give what the whole gives."""
    import torch
    p = Problem(eq, F32, 8, 2, 2, 8, 8, [128], False, seed=12)
    p.forward()
    S = torch.empty_like(p.S1)
    o = torch.empty_like(p.o)
    S2 = torch.empty_like(p.S1)
    for part, a, b in ((slice(0, 50), p.S0, S), (slice(50, 128), S, S2)):
        n = eq.eqlinear_linear_attention_workspace(p.plan, part.stop - part.start, 1)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        eq.eqlinear_linear_attention(p.plan, p.q[part], p.k[part], p.v[part], p.la, o[part], scale=p.scale, state_in=a,
                                     state_out=b, workspace=ws)
    torch.cuda.synchronize()
    scale = float(p.o.abs().max())
    assert float((o - p.o).abs().max()) <= 400 * E32 * scale * 64
    assert float((S2 - p.S1).abs().max()) <= 400 * E32 * float(p.S1.abs().max()) * 64


def test_no_tokens(eq):
    import torch
    p = Problem(eq, BF16, 8, 2, 1, 4, 4, [0, 0], True, seed=13)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    assert torch.equal(p.S1, p.S0) and torch.equal(p.dS0, p.dS1)


# --- one token ----------------------------------------------------------------------------

@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("B,N,H,K,dk,dv", [(1, 8, 2, 2, 8, 8), (7, 8, 12, 4, 16, 16), (3, 7, 4, 2, 16, 16),
                                           (2, 1, 2, 1, 3, 1), (5, 5, 3, 3, 7, 13), (33, 1, 1, 1, 128, 128),
                                           (2, 1, 4, 1, 1, 100)])
def test_step(eq, dt, B, N, H, K, dk, dv):
    import torch
    p = Problem(eq, dt, N, H, K, dk, dv, [1] * B, False, seed=B + N)
    a = p.host()
    ref = ops.linear_attention(**a)
    every = ops.linear_attention(**a, absolute="all")
    S = p.S0.clone()
    eq.eqlinear_linear_attention_step(p.plan, p.q, p.k, p.v, p.la, S, p.o, scale=p.scale)
    torch.cuda.synchronize()
    o, S = to_f64(p.o).reshape(ref["o"].shape), to_f64(S)
    # exp of the decay within 2 ulp, then one fused multiply-add; D_k terms
    assert np.all(np.abs(S - ref["S1"]) <= 8 * E32 * every["S1"])
    assert np.all(np.abs(o - ref["o"]) <= U[dt] * np.abs(ref["o"]) + (dk * N + 16) * E32 * every["o"])


def test_step_continues_a_prompt(eq):
    import torch
    p = Problem(eq, BF16, 8, 4, 2, 8, 8, [20], False, seed=14)
    p.forward()
    q, k, v = (torch.randn_like(t[:1]) for t in (p.q, p.k, p.v))
    S, o = p.S1.clone(), torch.empty_like(p.o[:1])
    eq.eqlinear_linear_attention_step(p.plan, q, k, v, p.la, S, o, scale=p.scale)
    both = Problem(eq, BF16, 8, 4, 2, 8, 8, [21], False, seed=14, fused=False)
    both.q, both.k, both.v = (torch.cat([a, b]) for a, b in ((p.q, q), (p.k, k), (p.v, v)))
    both.la, both.S0 = p.la, p.S0
    both.forward()
    torch.cuda.synchronize()
    # the prompt's last row rounds its scores; both round once at the end
    assert torch.allclose(o.float(), both.o[20:].float(), rtol=2 ** -6, atol=2 ** -6)
    both.check("prompt of 21", grads=False)

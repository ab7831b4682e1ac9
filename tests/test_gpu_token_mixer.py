"""The layers and the operators together (examples/token_mixer.py): values, shifts, gradients, single tokens, graphs.

Bounds.  Each of the block's five steps rounds its output once (2^-24 or 2^-8) and the steps'
gains are near one, so the error's root mean square is a few roundings': under 16 u of the
reference's, with room for the fp32 sums (u = 2^-20 stands for fp32: sums of up to 768 terms).
A derivative by differences of step e has a relative error of e^2 times ratios of derivatives
of order one, here 1e-4 times a few, and rounding 2^-20 / e: 1 % covers both.
"""
import numpy as np
import pytest

import synthetic
from gpu_util import to_f64
from oracle import operators as ops

pytestmark = pytest.mark.gpu

F32, BF16 = synthetic.F32, synthetic.BF16
U = {F32: 2.0 ** -20, BF16: 2.0 ** -8}


@pytest.fixture(scope="module")
def mixer():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from examples import token_mixer
    token_mixer.eq.load_library()
    return token_mixer


def block_of(m, dt, **kw):
    return m.TokenMixer(dtype={F32: m.eq.EQL_F32, BF16: m.eq.EQL_BF16}[dt], **kw)


def tokens(b, n, seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, b.C, b.N, generator=g).to(b.w_in.dtype).cuda()


def layer(w, x):
    """y[t,o,g] = sum w[o,i,(g-h) mod N] x[t,i,h]"""
    N = w.shape[2]
    return sum(np.einsum("oi,tih->toh", w[:, :, s], np.roll(x, s, axis=2)) for s in range(N))


def reference(b, x, lens, positions, state):
    w = {n: to_f64(getattr(b, n)) for n in ("w_in", "w_out", "gamma_x", "beta_x", "gamma_o", "beta_o", "log_decay")}
    x, T = to_f64(x), sum(lens)
    each, off = np.arange(T + 1), np.concatenate([[0], np.cumsum(lens)])
    h = ops.group_norm(x, w["gamma_x"], w["beta_x"], 1, 1e-5, ops.NONE, each)["y"]
    u = layer(w["w_in"], h).reshape(T, b.H + 2 * b.K, b.d, b.N)
    freq, pos = ops.rotary_frequencies(b.d), positions.cpu().numpy().astype(np.float64)
    q, k = (ops.rotary(a, pos, freq, b.d, False) for a in (u[:, :b.H], u[:, b.H:b.H + b.K]))
    D = b.d * b.N
    r = ops.linear_attention(q.reshape(T, b.H, D), k.reshape(T, b.K, D), u[:, b.H + b.K:].reshape(T, b.K, D),
                             w["log_decay"], b.scale, off, None if state is None else to_f64(state))
    n = ops.group_norm(r["o"].reshape(T, b.H * b.d, b.N), w["gamma_o"], w["beta_o"], b.H, 1e-5, ops.SILU, each)["y"]
    return x + layer(w["w_out"], n), r["S1"]


def rms(a):
    return float(np.sqrt(np.mean(np.square(a))))


def close(got, ref, dt, what):
    assert np.all(np.isfinite(got)), what
    assert rms(got - ref) <= 16 * U[dt] * rms(ref), (what, rms(got - ref) / rms(ref))


SIZES = [dict(), dict(N=7, C=20, heads=4, kv_heads=2, d=16), dict(N=4, C=8, heads=2, kv_heads=2, d=2)]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_prompt_and_tokens(mixer, dt, size):
    import torch
    b, lens = block_of(mixer, dt, **size), [70, 1, 130]
    off, pos = mixer.packed(lens)
    x = tokens(b, sum(lens), 1)
    y, state, _ = b.forward(x, off, pos)
    want, S = reference(b, x, lens, pos, None)
    close(to_f64(y), want, dt, "y")
    close(to_f64(state), S, dt, "state")
    # the next token by the step, and by a prompt of one token on the same state
    nxt, at = tokens(b, 3, 2), torch.tensor(lens, dtype=torch.int32).cuda()
    want, S = reference(b, nxt, [1, 1, 1], at, state)
    one, _ = mixer.packed([1, 1, 1])
    close(to_f64(b.forward(nxt, one, at, state)[0]), want, dt, "prompt of one")
    close(to_f64(b.step(nxt, at, state)), want, dt, "step")
    close(to_f64(state), S, dt, "state after the step")


@pytest.mark.parametrize("dt", [F32, BF16])
def test_shift_of_the_group_axis(mixer, dt):
    b, lens = block_of(mixer, dt), [64, 33]
    off, pos = mixer.packed(lens)
    x = tokens(b, sum(lens), 3)
    y = to_f64(b.forward(x, off, pos)[0])
    for s in (1, 5):
        close(to_f64(b.forward(x.roll(s, 2).contiguous(), off, pos)[0]), np.roll(y, s, axis=2), dt, s)


def test_gradients_by_differences(mixer):
    import torch
    b, lens = block_of(mixer, F32, **SIZES[1]), [40, 75]
    off, pos = mixer.packed(lens)
    x, weight = tokens(b, sum(lens), 4), to_f64(tokens(b, sum(lens), 5))
    S = torch.randn(b.new_state(2).shape, generator=torch.Generator().manual_seed(6)).cuda()
    _, _, saved = b.forward(x, off, pos, S)
    grads = b.backward(torch.from_numpy(weight).float().cuda(), saved)
    values = {n: getattr(b, n) for n in ("w_in", "w_out", "gamma_x", "beta_x", "gamma_o", "beta_o")}
    values |= {"x": x, "state": S}
    assert set(values) == set(grads)
    for name, p in values.items():
        g = grads[name].view(p.shape)
        size = float(g.double().norm())
        way = g / size * (1e-2 * max(float(p.norm()), 1e-2 * p.numel() ** 0.5))
        keep, loss = p.clone(), []
        for sign in (1, -1):
            p.copy_(keep + sign * way)
            b.update()
            loss.append(float((to_f64(b.forward(x, off, pos, S)[0]) * weight).sum()))
        p.copy_(keep)
        b.update()
        slope, want = (loss[0] - loss[1]) / 2, float((way.double() * g.double()).sum())
        assert abs(slope - want) <= 0.01 * want, (name, slope, want)


def test_steps_in_a_graph(mixer):
    import torch
    b = block_of(mixer, BF16)
    x, at, state = tokens(b, 8, 7), torch.zeros(8, dtype=torch.int32).cuda(), b.new_state(8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.step(x, at, state)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    state.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = b.step(x, at, state)
    mine = b.new_state(8)
    for i in range(5):
        x.copy_(tokens(b, 8, 10 + i))
        want = b.step(x, at, mine)  # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
        assert torch.equal(state, mine), i
        at += 1

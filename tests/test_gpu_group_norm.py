"""Group norm with an activation, and its gradients, against the fp64 definition.

Bounds.  fp32 statistics over n numbers of a group: the mean is within n 2^-24 of the mean
absolute value in the worst order; the tests' group means are a few spreads at most except
where a test says so, and sums run as trees of short chains, so 64 chained additions bound
every path.  xh then carries about 2^-24 (64 + 64 |mean| / spread) relative to its unit scale,
the activation and its slope (fractional error 1.2e-7 and the hardware reciprocal and exp2)
a few 2^-22 more, and the output its rounding u.  A gradient's sums add 64 2^-24 of the sum
of absolute terms.
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


def build(eq, dt, N, C, G, act, lens, ragged, seed=0, affine=True, wide=False, odd=False, mean=0.5, eps=1e-5):
    import torch
    g = torch.Generator().manual_seed(seed)
    T, B, tdt = int(sum(lens)), len(lens), torch_dtype(dt)
    plan = eq.eqlinear_norm_plan(N, C, G, act, {F32: eq.EQL_F32, BF16: eq.EQL_BF16, F16: eq.EQL_F16}[dt], eps=eps)

    def rows(fill):
        if not wide:
            return fill(T, C, N)
        W = C * N + (1 if odd else 16)
        return fill(T, W).as_strided((T, C, N), (W, N, 1), 1 if odd else 8)

    x = rows(lambda *s: (torch.randn(*s, generator=g) + mean).to(tdt).cuda())
    dy = rows(lambda *s: torch.randn(*s, generator=g).to(tdt).cuda())
    empty = lambda *s: torch.full(s, float("nan"), dtype=tdt, device="cuda")  # noqa: E731
    gamma = (1 + 0.3 * torch.randn(C, generator=g)).to(tdt).cuda() if affine else None
    beta = (0.3 * torch.randn(C, generator=g)).to(tdt).cuda() if affine else None
    off = np.concatenate([[0], np.cumsum(lens)])
    return dict(eq=eq, dt=dt, plan=plan, x=x, dy=dy, y=rows(empty), dx=rows(empty), gamma=gamma, beta=beta, off=off,
                B=B, T=T, G=G, C=C, N=N, act=act, eps=eps,
                offsets=torch.tensor(off, dtype=torch.int64).cuda() if ragged else None,
                stats=torch.full((B, G, 2), float("nan"), device="cuda"),
                dgamma=torch.full((C,), float("nan"), device="cuda"), dbeta=torch.full((C,), float("nan"), device="cuda"))


def workspace(p, backward):
    import torch
    n = p["eq"].eqlinear_group_norm_workspace(p["plan"], p["T"], p["B"], backward=backward)
    return torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") if n else None


def forward(p, y=None, stats=True):
    p["eq"].eqlinear_group_norm(p["plan"], p["x"], p["gamma"], p["beta"], p["y"] if y is None else y,
                                stats=p["stats"] if stats else None, offsets=p["offsets"], batch=p["B"],
                                workspace=workspace(p, False))


def backward(p, dx=None, params=True):
    p["eq"].eqlinear_group_norm_backward(p["plan"], p["dy"], p["x"], p["gamma"], p["beta"], p["stats"],
                                         p["dx"] if dx is None else dx, p["dgamma"] if params else None,
                                         p["dbeta"] if params else None, offsets=p["offsets"], batch=p["B"],
                                         workspace=workspace(p, True))


def check(p, what, lean=1.0):
    """lean: |mean| / spread of the groups, where it is more than a few."""
    import torch
    torch.cuda.synchronize()
    f = lambda t: None if t is None else to_f64(t)  # noqa: E731
    x, dy, gamma, beta = f(p["x"]), f(p["dy"]), f(p["gamma"]), f(p["beta"])
    r = ops.group_norm(x, gamma, beta, p["G"], p["eps"], p["act"], p["off"], dy)
    u, e = U[p["dt"]], 64 * E32 * (2 + lean)
    gm = np.ones(p["C"]) if gamma is None else np.abs(gamma)
    gmax = gm[None, :, None] * np.ones_like(x)
    assert np.all(np.isfinite(f(p["y"]))) and np.all(np.isfinite(f(p["dx"]))), what
    # |xh| <= sqrt(n) in principle; z = gamma xh + beta, and every activation's slope is below 1.2
    z = np.abs(ops.group_norm(x, gamma, beta, p["G"], p["eps"], ops.NONE, p["off"])["y"])
    tol = u * np.abs(r["y"]) + e * 1.2 * (gmax + z) + 2.0 ** -20 * z
    err = np.abs(f(p["y"]) - r["y"])
    assert np.all(err <= tol), f"{what}: y, worst {np.max(err / tol):.3g} times"
    st = f(p["stats"])
    for b in range(p["B"]):
        for j in range(p["G"]):
            m, s = r["stats"][b, j]
            if p["off"][b] == p["off"][b + 1]:
                assert tuple(st[b, j]) == (0.0, 0.0), what
            else:
                assert abs(st[b, j, 0] - m) <= 64 * E32 * (abs(m) + 1 / s) and abs(st[b, j, 1] / s - 1) <= 2 * e, what
    # the sums of absolute terms, group by group, through the same formula
    dz = np.abs(dy) * 1.2
    sizes = np.zeros_like(x)
    pa = np.zeros(p["C"]), np.zeros(p["C"])
    cg = p["C"] // p["G"]
    for b in range(p["B"]):
        s = slice(int(p["off"][b]), int(p["off"][b + 1]))
        if s.start == s.stop:
            continue
        for j in range(p["G"]):
            cs = slice(j * cg, (j + 1) * cg)
            m, rs = r["stats"][b, j]
            xh = np.abs(x[s, cs] - m) * rs
            g = dz[s, cs] * gmax[s, cs]
            sizes[s, cs] = (g + g.mean() + xh * (g * xh).mean() * 2 + g.mean()) * rs * (1 + xh)
            pa[0][cs] += (dz[s, cs] * (1 + xh) ** 2).sum((0, 2))
            pa[1][cs] += (dz[s, cs] * (1 + xh)).sum((0, 2))
    tol = u * np.abs(r["dx"]) + 4 * e * sizes
    err = np.abs(f(p["dx"]) - r["dx"])
    assert np.all(err <= tol), f"{what}: dx, worst {np.max(err / tol):.3g} times"
    for name, size in (("dgamma", pa[0]), ("dbeta", pa[1])):
        err = np.abs(f(p[name]) - r[name])
        assert np.all(err <= 4 * e * size + 1e-30), f"{what}: {name}, worst {np.max(err / (4 * e * size)):.3g} times"


def run(p, what, **kw):
    forward(p)
    backward(p)
    check(p, what, **kw)


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("act", [ops.NONE, ops.GELU, ops.SILU])
@pytest.mark.parametrize("lens", [[1] * 50, [197, 197], [0, 1, 33, 64, 300], [3, 0, 0]], ids=str)
def test_lengths_and_activations(eq, dt, act, lens):
    run(build(eq, dt, 8, 24, 3, act, lens, len(set(lens)) > 1), f"{dt} act {act} {lens}")


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("lens", [[1] * 33, [70, 70], [9, 120, 1]], ids=str)
@pytest.mark.parametrize("N,C,G", [(1, 16, 1), (7, 160, 10), (7, 5, 1), (3, 7, 7), (1, 1280, 4), (16, 80, 16), (5, 12, 2),
                                   (1, 40, 40), (2, 96, 3), (8, 160, 1), (12, 9, 3), (1, 5000, 1)])
def test_sizes(eq, dt, lens, N, C, G):
    if C // G * N < 2 and min(lens) == 1:
        lens = [n + 3 for n in lens]  # one number alone has no spread: test_groups_without_spread
    run(build(eq, dt, N, C, G, ops.SILU, lens, len(set(lens)) > 1, seed=C), f"{dt} N={N} C={C} G={G} {lens}")


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("lens", [[5000], [20000, 3], [4000, 0, 1, 2500]], ids=str)
def test_long_samples(eq, dt, lens):
    run(build(eq, dt, 4, 12, 2, ops.GELU, lens, len(set(lens)) > 1, seed=2), f"{dt} {lens}")


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("lens", [[1] * 40, [50, 50], [30, 700]], ids=str)
@pytest.mark.parametrize("wide,odd,affine", [(True, False, True), (True, True, True), (False, False, False)])
def test_strides_and_no_affine(eq, dt, lens, wide, odd, affine):
    run(build(eq, dt, 8, 16, 2, ops.GELU, lens, len(set(lens)) > 1, wide=wide, odd=odd, affine=affine),
        f"{dt} {lens} wide={wide} odd={odd} affine={affine}")
    run(build(eq, dt, 5, 6, 2, ops.SILU, lens, len(set(lens)) > 1, wide=wide, odd=odd, affine=affine),
        f"{dt} {lens} wide={wide} odd={odd} affine={affine}, N = 5")


@pytest.mark.parametrize("lens", [[1] * 20, [64, 64], [6000]], ids=str)
def test_mean_far_from_zero(eq, lens):
    """A mean 1000 spreads from 0: the variance must not come from differences of squares (relative error 1000^2 2^-24
    = 6 percent there; 64 2^-24 1000 = 0.4 percent of a spread bounds what the rounding of the mean leaves)."""
    run(build(eq, F32, 8, 32, 2, ops.NONE, lens, False, mean=1000.0), f"{lens}", lean=1000.0)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("lens", [[1] * 9, [40], [9000]], ids=str)
def test_groups_without_spread(eq, dt, lens):
    """All numbers equal: xh = 0, y = act(beta), dx finite; a group of a single number likewise."""
    import torch
    for N, C, G in ((8, 16, 2), (1, 4, 4)):
        p = build(eq, dt, N, C, G, ops.SILU, lens, False)
        p["x"].fill_(3.0)
        forward(p)
        backward(p)
        torch.cuda.synchronize()
        z = p["beta"].float()
        ref = (z * torch.sigmoid(z))[None, :, None].expand(p["y"].shape)
        assert float((p["y"].float() - ref).abs().max()) <= 2 * U[dt] + 1e-6
        assert torch.isfinite(p["dx"]).all() and torch.isfinite(p["dgamma"]).all()
        assert float(p["dgamma"].abs().max()) == 0.0


@pytest.mark.parametrize("lens", [[1] * 30, [60, 60], [30, 0, 9000]], ids=str)
def test_in_place(eq, lens):
    import torch
    p = build(eq, BF16, 8, 24, 3, ops.SILU, lens, len(set(lens)) > 1)
    forward(p)
    backward(p)
    y, dx, dg = p["y"].clone(), p["dx"].clone(), p["dgamma"].clone()
    backward(p, dx=p["dy"])  # dx in dy's place
    assert torch.equal(p["dy"], dx) and torch.equal(p["dgamma"], dg)
    forward(p, y=p["x"])
    torch.cuda.synchronize()
    assert torch.equal(p["x"], y)


@pytest.mark.parametrize("lens", [[1] * 1000, [60, 60], [30, 0, 5000]], ids=str)
def test_same_bits_every_time_and_optional_outputs(eq, lens):
    import torch
    p = build(eq, F32, 8, 24, 3, ops.GELU, lens, len(set(lens)) > 1)
    forward(p)
    backward(p)
    first = [p[n].clone() for n in ("y", "stats", "dx", "dgamma", "dbeta")]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            forward(p)
            backward(p)
    torch.cuda.current_stream().wait_stream(s)
    for a, n in zip(first, ("y", "stats", "dx", "dgamma", "dbeta")):
        assert torch.equal(a, p[n])
    forward(p, stats=False)
    backward(p, params=False)
    torch.cuda.synchronize()
    assert torch.equal(first[0], p["y"]) and torch.equal(first[2], p["dx"])


def test_nan_stays_in_its_sample_and_group(eq):
    import torch
    p = build(eq, BF16, 8, 24, 3, ops.SILU, [40, 50, 60], True)
    p["x"][45, 9, 3] = float("nan")  # sample 1, group 1
    forward(p)
    backward(p)
    torch.cuda.synchronize()
    for t in (p["y"], p["dx"]):
        bad = ~torch.isfinite(t)
        assert bad[40:90, 8:16].all()
        bad[40:90, 8:16] = False
        assert not bad.any()


def test_no_tokens(eq):
    import torch
    p = build(eq, F32, 4, 8, 2, ops.NONE, [0, 0], True)
    forward(p)
    backward(p)
    torch.cuda.synchronize()
    assert torch.count_nonzero(p["stats"]) == 0
    assert torch.count_nonzero(p["dgamma"]) == 0 and torch.count_nonzero(p["dbeta"]) == 0

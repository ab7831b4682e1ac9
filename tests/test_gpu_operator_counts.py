"""More sequences, tokens or samples than one launch of 2^32 threads takes: every one of them is answered.

(A larger grid starts its workgroups modulo 2^32 threads and reports no error.)"""
import pytest

pytestmark = pytest.mark.gpu

WGS = 1 << 24  # workgroups of 256 threads


@pytest.fixture(scope="module")
def eq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import group_equivariant_linear_amd as eq
    eq.load_library()
    return eq


@pytest.fixture(autouse=True)
def give_back():
    yield
    import torch
    torch.cuda.empty_cache()


def room(gib):
    import torch
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of free GPU memory")


def test_step(eq):
    import torch
    room(4)
    B, plan = WGS + 8, eq.eqlinear_mixer_plan(1, 1, 1, 1, 1, eq.EQL_F32)
    q, k, v, S = (torch.rand(B, 1, 1, 1, device="cuda") + 0.5 for _ in range(4))
    o, want = torch.zeros_like(q), S * 0.5 + k * v
    eq.eqlinear_linear_attention_step(plan, q, k, v, torch.log(torch.tensor([0.5])).cuda(), S, o, 2.0)
    assert torch.allclose(S, want, rtol=1e-5) and torch.allclose(o, 2 * q * want, rtol=1e-5)


def test_linear_attention(eq):
    """Sequences of one token each: o = scale q k v, and its gradients."""
    import torch
    room(8)
    B, plan = WGS + 9, eq.eqlinear_mixer_plan(1, 1, 1, 1, 1, eq.EQL_F32)
    q, k, v, do = (torch.rand(B, 1, 1, 1, device="cuda") + 0.5 for _ in range(4))
    o, dq, dk, dv = (torch.zeros_like(q) for _ in range(4))
    la = torch.tensor([-0.1]).cuda()
    n = eq.eqlinear_linear_attention_workspace(plan, B, B, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    eq.eqlinear_linear_attention(plan, q, k, v, la, o, 2.0, batch=B, workspace=ws)
    eq.eqlinear_linear_attention_backward(plan, q, k, v, do, la, dq, dk, dv, 2.0, batch=B, workspace=ws)
    for got, want in ((o, q * k * v), (dq, do * k * v), (dk, do * q * v), (dv, do * q * k)):
        assert torch.allclose(got, 2 * want, rtol=1e-5)


def test_rotary(eq):
    import torch
    room(80)
    T, D = 8 * WGS + 24, 256
    plan = eq.eqlinear_rotary_plan(1, 1, 1, D, D, eq.EQL_ROTARY_INTERLEAVED, eq.EQL_BF16)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") % 8
    x = torch.ones(T, 1, D, 1, dtype=torch.bfloat16, device="cuda")
    table = torch.ones(8, 1, D, 1, dtype=torch.bfloat16, device="cuda")
    eq.eqlinear_rotary(plan, table, None, pos[:8], table, None)
    eq.eqlinear_rotary(plan, x, None, pos, x, None)
    assert bool((x.view(T // 8, -1) == table.view(1, -1)).all(1).all())
    f = 10000.0 ** (-torch.arange(0, D, 2, device="cuda").double() / D)
    ang = torch.arange(8, device="cuda").double()[:, None] * f
    want = torch.stack([ang.cos() - ang.sin(), ang.cos() + ang.sin()], 2).view(8, 1, D, 1)
    assert float((table.double() - want).abs().max()) <= 2.0 ** -7


def test_group_norm(eq):
    """A norm per token, of rows that no workgroup holds."""
    import torch
    room(60)
    T, C = WGS + 40, 513
    plan = eq.eqlinear_norm_plan(1, C, 1, eq.EQL_ACT_NONE, eq.EQL_BF16)
    x, dy = (torch.empty(T, C, 1, dtype=torch.bfloat16, device="cuda").normal_() for _ in range(2))
    ends = [slice(0, 1000), slice(T - 1000, T)]
    xs, dys = ([t[s].double() for s in ends] for t in (x, dy))
    stats = torch.zeros(T, 1, 2, device="cuda")
    dg, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    ws = torch.empty(eq.eqlinear_group_norm_workspace(plan, T, T, True), dtype=torch.uint8, device="cuda")
    total = sum(p.double().sum((0, 2)) for p in dy.split(1 << 21))
    y = torch.empty_like(x)
    eq.eqlinear_group_norm(plan, x, None, None, y, stats=stats, batch=T, workspace=ws)
    eq.eqlinear_group_norm_backward(plan, dy, x, None, None, stats, dy, dg, db, batch=T, workspace=ws)
    for s, xe, g in zip(ends, xs, dys):
        m = xe.mean(1, keepdim=True)
        r = 1 / torch.sqrt(((xe - m) ** 2).mean(1, keepdim=True) + 1e-5)
        xh = (xe - m) * r
        assert float((y[s].double() - xh).abs().max()) <= 2.0 ** -8 * 5
        want = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * r
        assert float((dy[s].double() - want).abs().max()) <= 2.0 ** -8 * 6
    # 2^24 terms of size 1 and random sign, in fp32
    assert float((db.double() - total).abs().max()) <= 2.0 ** -24 * 2.0 ** 24
    assert int((stats[:, 0, 1] == 0).sum()) == 0

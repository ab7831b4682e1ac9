"""The operators on q, k and v whose heads alternate in one buffer, [token][head][q, k, v][d][N], with and without
numbers between the tokens: the bits that contiguous tensors give, and nothing else written."""
import pytest

pytestmark = pytest.mark.gpu

H, D, N = 3, 8, 8


@pytest.fixture(scope="module")
def eq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import group_equivariant_linear_amd as eq
    eq.load_library()
    return eq


def alternating(T, slack, first, seed):
    """A buffer of T rows and views of its q, k, v ([T, H, D, N])."""
    import torch
    buf = torch.randn(T, first + H * 3 * D * N + slack, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
    return buf, [buf.as_strided((T, H, D, N), (buf.stride(0), 3 * D * N, N, 1), first + i * D * N) for i in range(3)]


@pytest.mark.parametrize("T", [1, 2, 150])
@pytest.mark.parametrize("slack,first", [(0, 0), (64, 0), (200, 40)])
@pytest.mark.parametrize("swap", [False, True])
def test_rotary_in_place(eq, T, slack, first, swap):
    import torch
    plan = eq.eqlinear_rotary_plan(N, H, H, D, 6, eq.EQL_ROTARY_HALF, eq.EQL_BF16)
    buf, (a, b, v) = alternating(T, slack, first, T)
    q, k = (b, a) if swap else (a, b)
    pos = torch.arange(T, dtype=torch.int32).cuda() * 7
    qo, ko = torch.empty(T, H, D, N, dtype=q.dtype, device="cuda"), torch.empty(T, H, D, N, dtype=q.dtype, device="cuda")
    eq.eqlinear_rotary(plan, q.contiguous(), k.contiguous(), pos, qo, ko)
    keep = buf.clone()
    eq.eqlinear_rotary(plan, q, k, pos, q, k)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko)
    q.zero_(), k.zero_()
    for i, first_of in ((0, first), (1, first + D * N)):  # everything else as it was
        keep.as_strided((T, H, D, N), (buf.stride(0), 3 * D * N, N, 1), first_of).zero_()
    assert torch.equal(buf, keep)


@pytest.mark.parametrize("T", [1, 150])
@pytest.mark.parametrize("slack,first", [(0, 0), (200, 40)])
def test_attention_and_gradients(eq, T, slack, first):
    import torch
    plan = eq.eqlinear_mixer_plan(N, H, H, D, D, eq.EQL_BF16)
    _, (q, k, v) = alternating(T, slack, first, T)
    grad, views = alternating(T, slack, first, T + 1)
    la = torch.tensor([-0.1, -0.01, -0.3]).cuda()
    do = torch.randn(T, H, D, N, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    ws = torch.empty(eq.eqlinear_linear_attention_workspace(plan, T, 1, True) + 1, dtype=torch.uint8, device="cuda")
    out = []
    for ins, to in (([x.contiguous() for x in (q, k, v)], [torch.empty_like(do) for _ in "qkv"]), ((q, k, v), views)):
        o = torch.empty_like(do)
        eq.eqlinear_linear_attention(plan, *ins, la, o, 0.125, workspace=ws)
        eq.eqlinear_linear_attention_backward(plan, *ins, do, la, *to, 0.125, workspace=ws)
        torch.cuda.synchronize()
        out.append([o] + [t.contiguous() for t in to])
    for a, b in zip(*out):
        assert torch.equal(a, b)

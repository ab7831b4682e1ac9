"""The operators over buffers whose rows lie past 2^32 bytes and 2^32 elements: the bits of compact buffers.

Token strides of just under 2^24 bytes (whole 16-byte rows) and above, over a few hundred
tokens; only the tokens' own rows are touched.
"""
import pytest

pytestmark = pytest.mark.gpu

STRIDES = [8_388_600, 8_388_611]  # elements of 16 bits: 2^24 - 16 bytes; odd and past 2^24
T = 600


@pytest.fixture(scope="module")
def eq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.get_device_properties(0).total_memory < 64 << 30:
        pytest.skip("needs 64 GB of GPU memory")
    import group_equivariant_linear_amd as eq
    eq.load_library()
    return eq


def far(t, stride):
    """t [T, ...] at a token stride of `stride` elements."""
    import torch
    row = t[0].numel()
    buf = torch.empty((len(t) - 1) * stride + row, dtype=t.dtype, device="cuda")
    v = buf.as_strided(t.shape, (stride, *t.stride()[1:]))
    v.copy_(t)
    return v


def rows(*shape, seed):
    import torch
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def same(a, b):
    import torch
    torch.cuda.synchronize()
    return torch.equal(a.contiguous(), b.contiguous())


@pytest.mark.parametrize("stride", STRIDES)
def test_rotary(eq, stride):
    import torch
    plan = eq.eqlinear_rotary_plan(8, 2, 1, 8, 8, eq.EQL_ROTARY_HALF, eq.EQL_BF16)
    q, k = rows(T, 2, 8, 8, seed=1), rows(T, 1, 8, 8, seed=2)
    pos = torch.arange(T, dtype=torch.int32).cuda()
    fq, fk = far(q, stride), far(k, stride)
    eq.eqlinear_rotary(plan, q, k, pos, q, k)
    eq.eqlinear_rotary(plan, fq, fk, pos, fq, fk)
    assert same(fq, q) and same(fk, k)


@pytest.mark.parametrize("stride", STRIDES)
def test_linear_attention(eq, stride):
    import torch
    plan = eq.eqlinear_mixer_plan(8, 2, 1, 8, 8, eq.EQL_BF16)
    lens, u = torch.tensor([0, 130, 130, 131, T]).cuda(), rows(T, 4, 8, 8, seed=3)
    do = rows(T, 2, 8, 8, seed=4)
    la = torch.tensor([-0.01]).cuda()

    def run(u, do):
        o, du = torch.empty_like(do), torch.empty_like(u)  # (of an as_strided tensor: compact)
        if u.stride(0) == stride:
            o, du = far(o, stride), far(du, stride)
        S = torch.empty(4, 1, 64, 64, device="cuda")
        ws = torch.empty(eq.eqlinear_linear_attention_workspace(plan, T, 4, True) + 1, dtype=torch.uint8, device="cuda")
        q, k, v, dq, dk, dv = (x[:, i:j] for x in (u, du) for i, j in ((0, 2), (2, 3), (3, 4)))
        eq.eqlinear_linear_attention(plan, q, k, v, la, o, 0.125, offsets=lens, state_out=S, workspace=ws)
        eq.eqlinear_linear_attention_backward(plan, q, k, v, do, la, dq, dk, dv, 0.125, offsets=lens, workspace=ws)
        return o, S, du

    for a, b in zip(run(u, do), run(far(u, stride), far(do, stride))):
        assert same(a, b)


@pytest.mark.parametrize("stride", STRIDES)
@pytest.mark.parametrize("batch", [T, 12, 1])
def test_group_norm(eq, stride, batch):
    import torch
    plan = eq.eqlinear_norm_plan(8, 16, 2, eq.EQL_ACT_GELU, eq.EQL_BF16)
    x, dy = rows(T, 16, 8, seed=5), rows(T, 16, 8, seed=6)
    gamma, beta = rows(16, seed=7), rows(16, seed=8)
    ws = torch.empty(max(eq.eqlinear_group_norm_workspace(plan, T, batch, b) for b in (False, True)) + 1,
                     dtype=torch.uint8, device="cuda")

    def run(x, dy, y, dx):
        st, dg, db = torch.empty(batch, 2, 2, device="cuda"), torch.empty(16, device="cuda"), torch.empty(16, device="cuda")
        eq.eqlinear_group_norm(plan, x, gamma, beta, y, stats=st, batch=batch, workspace=ws)
        eq.eqlinear_group_norm_backward(plan, dy, x, gamma, beta, st, dx, dg, db, batch=batch, workspace=ws)
        return y, dx, st, dg, db

    near = run(x, dy, torch.empty_like(x), torch.empty_like(x))
    fx, fdy = far(x, stride), far(dy, stride)
    apart = run(fx, fdy, far(torch.zeros_like(x), stride), fdy)  # dx over dy
    for a, b in zip(near[:2], apart[:2]):
        if stride % 8 == 0:  # rows in pieces of 16 bytes, as the compact ones: the same sums in the same order
            assert same(a, b)
        else:  # another order of the fp32 sums: at most the next number of 8 bits
            a, b = a.float(), b.float()
            assert bool(((a - b).abs() <= 2.0 ** -7 * a.abs().clamp_min(2.0 ** -10)).all())

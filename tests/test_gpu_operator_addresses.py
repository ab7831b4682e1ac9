"""The operators given device addresses instead of tensors: the same bits.  And the stream they run on by default."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import group_equivariant_linear_amd as eq
    eq.load_library()
    return eq


def rand(*shape, seed):
    import torch
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def address(t):
    return None if t is None else t.data_ptr()


def both(call, ins, make, T):
    """call(as_given, *ins, *outs, T) with tensors and with addresses."""
    import torch
    outs = []
    for form in (lambda t: t, address):
        out = make()
        call(*(form(t) for t in ins), *(form(t) for t in out), T if form is address else None)
        torch.cuda.synchronize()
        outs.append(out)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 50])
def test_rotary_and_attention(eq, T):
    import torch
    rot = eq.eqlinear_rotary_plan(8, 2, 1, 8, 8, eq.EQL_ROTARY_HALF, eq.EQL_BF16)
    mix = eq.eqlinear_mixer_plan(8, 2, 1, 8, 8, eq.EQL_BF16)
    q, k, v, do = rand(T, 2, 8, 8, seed=1), rand(T, 1, 8, 8, seed=2), rand(T, 1, 8, 8, seed=3), rand(T, 2, 8, 8, seed=4)
    pos, la = torch.arange(T, dtype=torch.int32).cuda(), torch.tensor([-0.1]).cuda()
    new = lambda: [torch.empty_like(q), torch.empty_like(k)]  # noqa: E731
    both(lambda q, k, p, a, b, T: eq.eqlinear_rotary(rot, q, k, p, a, b, T=T), (q, k, pos), new, T)
    S = lambda: torch.empty(1, 1, 64, 64, device="cuda")  # noqa: E731
    both(lambda q, k, v, la, o, S, T: eq.eqlinear_linear_attention(mix, q, k, v, la, o, 0.1, state_out=S, T=T),
         (q, k, v, la), lambda: [torch.empty_like(q), S()], T)
    both(lambda q, k, v, do, la, a, b, c, T: eq.eqlinear_linear_attention_backward(mix, q, k, v, do, la, a, b, c, 0.1, T=T),
         (q, k, v, do, la), lambda: [torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)], T)
    both(lambda q, k, v, la, S, o, T: eq.eqlinear_linear_attention_step(mix, q, k, v, la, S, o, 0.1, batch=T),
         (q, k, v, la), lambda: [torch.ones(T, 1, 64, 64, device="cuda"), torch.empty_like(q)], T)


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("offsets", [False, True])
def test_group_norm(eq, strided, offsets):
    import torch
    T, plan = 60, eq.eqlinear_norm_plan(8, 16, 2, eq.EQL_ACT_GELU, eq.EQL_BF16)
    x, dy, gamma, beta = rand(T, 32, 8, seed=5)[:, 8:24], rand(T, 16, 8, seed=6), rand(16, seed=7), rand(16, seed=8)
    if not strided:
        x = x.contiguous()
    off, B = (torch.tensor([0, 20, 20, 60]).cuda(), 3) if offsets else (None, 4)
    ws = torch.empty(eq.eqlinear_group_norm_workspace(plan, T, B, True) + 1, dtype=torch.uint8, device="cuda")
    res = []
    for form in (lambda t: t, address):
        rows = form
        if strided and form is address:
            rows = lambda t: eq.eqlinear_heads(t.data_ptr(), t.stride(0), 0)  # noqa: E731
        n = T if form is address else None
        y, st, dx = torch.empty_like(dy), torch.empty(B, 2, 2, device="cuda"), torch.empty_like(dy)
        dg, db = torch.empty(16, device="cuda"), torch.empty(16, device="cuda")
        eq.eqlinear_group_norm(plan, rows(x), form(gamma), form(beta), rows(y), stats=form(st), offsets=form(off), batch=B,
                               workspace=ws, T=n)
        eq.eqlinear_group_norm_backward(plan, rows(dy), rows(x), form(gamma), form(beta), form(st), rows(dx), form(dg),
                                        form(db), offsets=form(off), batch=B, workspace=ws, T=n)
        torch.cuda.synchronize()
        res.append((y, st, dx, dg, db))
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_default_stream(eq):
    """No stream given: torch's current one, also where torch lacks its short way to it."""
    import torch
    s = torch.cuda.Stream()
    assert eq._raw_stream(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(s):
        assert eq._raw_stream(None) == s.cuda_stream == eq._raw_stream(s) == eq._raw_stream(s.cuda_stream)

"""Workspaces of the operators against the tensors they serve (host arithmetic: no GPU)."""
import pytest


@pytest.fixture(scope="module")
def eq():
    import group_equivariant_linear_amd as eq
    from group_equivariant_linear_amd import _build
    if not eq.built():
        _build.build()
    eq.load_library()
    return eq


SHAPES = [(1, 4096, 1), (8, 512, 1), (8, 96, 12), (1, 8191, 8191), (1, 8190, 4095), (7, 160, 10), (1, 1 << 20, 1),
          (1, 1 << 20, 1 << 20), (1, 1 << 20, 512), (1, 12288, 6), (1, 255 * 8, 255), (16, 1 << 16, 64), (3, 1001, 7),
          (1, 1920 * 8, 1920), (2, 5000, 8)]


@pytest.mark.parametrize("N,C,G", SHAPES)
@pytest.mark.parametrize("T,batch", [(1, 1), (100, 100), (4096, 4096), (131072, 131072), (32768, 1), (32768, 3), (50000, 64),
                                     (100000, 33333)])
def test_group_norm_workspace_is_bounded(eq, N, C, G, T, batch):
    """72 MiB for the sums of dgamma and dbeta (and no more than 16 tokens' worth of numbers where there are fewer than
    that), and for each block (16 tokens or more, one more a sample) 8 bytes per group and per 256 numbers of a row,
    for each sample 8 per group."""
    for dt in (eq.EQL_F32, eq.EQL_BF16):
        plan = eq.eqlinear_norm_plan(N, C, G, eq.EQL_ACT_NONE, dt)
        n = eq.eqlinear_group_norm_workspace(plan, T, batch, backward=True)
        parts = min(72 << 20, 8 * C * N * (T + batch) * 16)
        rest = 8 * ((T // 16 + batch) * (G + C * N // 256 + 1) + batch * G) + 1024
        assert n <= parts + rest, (dt, n, parts, rest)
        assert eq.eqlinear_group_norm_workspace(plan, T, batch) <= rest


def test_group_norm_workspace_of_wide_tokens(eq):
    """A norm per token of 131072 x 4096 bf16 numbers (1 GiB): less than a tenth of it."""
    plan = eq.eqlinear_norm_plan(1, 4096, 1, eq.EQL_ACT_NONE, eq.EQL_BF16)
    assert eq.eqlinear_group_norm_workspace(plan, 131072, 131072, backward=True) < 1 << 27
    plan = eq.eqlinear_norm_plan(8, 512, 1, eq.EQL_ACT_NONE, eq.EQL_BF16)
    assert eq.eqlinear_group_norm_workspace(plan, 32768, 32768, backward=True) < 1 << 27
    plan = eq.eqlinear_norm_plan(1, 8191, 8191, eq.EQL_ACT_NONE, eq.EQL_BF16)
    assert eq.eqlinear_group_norm_workspace(plan, 1, 1, backward=True) < 1 << 20

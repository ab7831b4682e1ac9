"""Group norm over rows and group counts that share or cap its workspace: groups that fill no workgroup, tokens
wider than one, more samples than workgroups.  Bounds as in test_gpu_group_norm.py."""
import pytest

import synthetic
from oracle import operators as ops
from test_gpu_group_norm import build, eq, run  # noqa: F401  (eq is the fixture)

pytestmark = pytest.mark.gpu

F32, BF16, F16 = synthetic.F32, synthetic.BF16, synthetic.F16


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("N,C,G,T", [(1, 2 * 1009, 1009, 1), (1, 2 * 1009, 1009, 40), (1, 4 * 255, 255, 33), (3, 255, 255, 7),
                                     (1, 17 * 264, 17, 9), (1, 6 * 2048, 6, 41), (1, 3 * 1024, 3, 300), (8, 12 * 32, 12, 50),
                                     (2, 5 * 700, 700, 12), (8, 1024, 1024, 3), (1, 15 * 1920, 1920, 6), (1, 12 * 300, 12, 2)])
def test_groups_of_tokens(eq, dt, N, C, G, T):
    run(build(eq, dt, N, C, G, ops.SILU, [1] * T, False, seed=G), f"{dt} N={N} C={C} G={G} T={T}")


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("lens", [[1] * 20, [3] * 7, [5, 0, 1, 9], [40]], ids=str)
@pytest.mark.parametrize("N,C,G", [(1, 4104, 1), (1, 20000, 2), (1, 6000, 3), (7, 1200, 1), (8, 2000, 5), (2, 4097, 1)])
def test_wide_tokens(eq, dt, lens, N, C, G):
    run(build(eq, dt, N, C, G, ops.GELU if C < 6000 else ops.NONE, lens, len(set(lens)) > 1, seed=C), f"{dt} N={N} C={C} G={G} {lens}")


@pytest.mark.parametrize("odd,T", [(False, 700), (True, 150)])
def test_more_samples_than_workgroups(eq, odd, T):
    run(build(eq, BF16, 1, 4104, 1, ops.SILU, [1] * T, False, wide=True, odd=odd), f"{T} tokens, odd={odd}")
    run(build(eq, BF16, 1, 4104, 3, ops.SILU, [2, 0, 1] * (T // 4), True, wide=True, odd=odd), f"{T} packed, odd={odd}")

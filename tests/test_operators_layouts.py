"""Which tensors may lie within each other's address range: the overlap check of the operators against a plain
count of elements.  The refusals come before any HIP call; what is accepted is run on a GPU in
test_gpu_operator_layouts.py."""
import pytest


@pytest.fixture(scope="module")
def eq():
    import group_equivariant_linear_amd as eq
    from group_equivariant_linear_amd import _build
    if not eq.built():
        _build.build()
    eq.load_library()
    return eq


BASE, APART = 1 << 20, 1 << 40


@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("heads,kv,hs_q,hs_k,ts,at", [
    (4, 4, 192, 192, 768, 32),     # k starts inside q's first run
    (4, 4, 192, 192, 768, 160),    # k's run ends in q's next
    (4, 4, 96, 96, 384, 48),       # runs that do not fit between
    (4, 4, 192, 128, 768, 64),     # head strides apart
    (4, 2, 128, 256, 512, 100),
    (4, 4, 192, 192, 800, 192),    # the same runs, one head later
])
def test_shared_elements_are_refused(eq, T, heads, kv, hs_q, hs_k, ts, at):
    """q turned in place, k over or beside it, heads of 64 numbers; every case shares an element by count."""
    q = {t * ts + h * hs_q + i for t in range(T) for h in range(heads) for i in range(64)}
    k = {at + t * ts + h * hs_k + i for t in range(T) for h in range(kv) for i in range(64)}
    assert q & k
    plan = eq.eqlinear_rotary_plan(8, heads, kv, 8, 8, 0, eq.EQL_BF16)
    hq, hk = eq.eqlinear_heads(BASE, ts, hs_q), eq.eqlinear_heads(BASE + 2 * at, ts, hs_k)
    f = eq.load_library().eqlinear_rotary
    assert f(plan.handle, hq, hk, APART, 0, hq, hk, T, None) == eq.EQL_ERR_INVALID
    other = eq.eqlinear_heads(APART, 4096, 64)
    assert f(plan.handle, hq, other, 2 * APART, 0, hq, hk, T, None) == eq.EQL_ERR_INVALID

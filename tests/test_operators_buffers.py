"""The operators' flat buffers (workspace, states, statistics, parameters, offsets): none that a call writes may share a
byte with another one of the call.  Every refusal comes before any HIP call, so the addresses are made up."""
import itertools

import pytest


@pytest.fixture(scope="module")
def eq():
    import group_equivariant_linear_amd as eq
    from group_equivariant_linear_amd import _build
    if not eq.built():
        _build.build()
    eq.load_library()
    return eq


def place(i):
    return (i + 1) << 32


def refuses(f, args, written, read, sizes):
    """Each written buffer moved onto each other one (its first byte on the other's last whole alignment)."""
    for w, r in itertools.chain(itertools.permutations(written, 2), itertools.product(written, read)):
        a = dict(args)
        a[w] = a[r] + (sizes[r] - 1) // 256 * 256
        assert f(*a.values()) == 1, (w, r)
        a = dict(args)
        a[r] = a[w] + (sizes[w] - 1) // 256 * 256
        assert f(*a.values()) == 1, (r, w)


def test_linear_attention(eq):
    lib = eq.load_library()
    plan = eq.eqlinear_mixer_plan(8, 4, 2, 8, 4, eq.EQL_BF16)  # D_k 64, D_v 32
    T, B = 4096, 2  # long enough for a workspace
    need = [lib.eqlinear_linear_attention_workspace(plan.handle, T, B, b) for b in (0, 1)]
    assert all(need)
    h = [eq.eqlinear_heads(place(20 + i), 256, 64) for i in range(8)]
    state = B * 2 * 64 * 32 * 4
    sizes = dict(la=8, off=8 * (B + 1), s0=state, s1=state, d0=state, d1=state)
    args = dict(p=plan.handle, q=h[0], k=h[1], v=h[2], la=place(0), scale=0.5, off=place(1), batch=B, s0=place(2),
                s1=place(3), o=h[3], T=T, ws=place(4), bytes=need[0], st=None)
    refuses(lib.eqlinear_linear_attention, args, ["s1", "ws"], ["la", "off", "s0"], sizes | {"ws": need[0]})
    for r in ("la", "off"):
        assert lib.eqlinear_linear_attention(*(args | {r: place(23)}).values()) == 1, r  # inside o
    args = dict(p=plan.handle, q=h[0], k=h[1], v=h[2], do=h[3], la=place(0), scale=0.5, off=place(1), batch=B,
                s0=place(2), d1=place(3), dq=h[4], dk=h[5], dv=h[6], d0=place(4), T=T, ws=place(5), bytes=need[1], st=None)
    refuses(lib.eqlinear_linear_attention_backward, args, ["d0", "ws"], ["la", "off", "s0", "d1"], sizes | {"ws": need[1]})
    for r in ("la", "off"):
        for out in (24, 25, 26):
            assert lib.eqlinear_linear_attention_backward(*(args | {r: place(out)}).values()) == 1, r
    args = dict(p=plan.handle, q=h[0], k=h[1], v=h[2], la=place(0), scale=0.5, state=place(1), o=h[3], batch=B, st=None)
    refuses(lib.eqlinear_linear_attention_step, args, ["state"], ["la"], sizes | {"state": state})
    assert lib.eqlinear_linear_attention_step(*(args | {"la": place(23)}).values()) == 1


def test_group_norm(eq):
    lib = eq.load_library()
    plan = eq.eqlinear_norm_plan(8, 24, 3, eq.EQL_ACT_SILU, eq.EQL_BF16)
    T, B = 4096, 2
    need = [lib.eqlinear_group_norm_workspace(plan.handle, T, B, b) for b in (0, 1)]
    assert all(need)
    sizes = dict(gamma=48, beta=48, off=8 * (B + 1), stats=B * 3 * 8, dg=96, db=96)
    args = dict(p=plan.handle, x=place(20), ldx=192, gamma=place(0), beta=place(1), off=place(2), batch=B, y=place(21),
                ldy=192, stats=place(3), T=T, ws=place(4), bytes=need[0], st=None)
    refuses(lib.eqlinear_group_norm, args, ["stats", "ws"], ["gamma", "beta", "off"], sizes | {"ws": need[0]})
    assert lib.eqlinear_group_norm(*(args | {"off": place(21)}).values()) == 1
    args = dict(p=plan.handle, dy=place(22), lddy=192, x=place(20), ldx=192, gamma=place(0), beta=place(1), stats=place(3),
                off=place(2), batch=B, dx=place(21), lddx=192, dg=place(4), db=place(5), T=T, ws=place(6), bytes=need[1],
                st=None)
    refuses(lib.eqlinear_group_norm_backward, args, ["dg", "db", "ws"], ["gamma", "beta", "off", "stats"],
            sizes | {"ws": need[1]})
    assert lib.eqlinear_group_norm_backward(*(args | {"off": place(21)}).values()) == 1

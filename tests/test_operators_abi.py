"""Refusals of the operators between the layers, through the C ABI with made-up addresses: every check
comes before any HIP call, so nothing here needs a GPU or launches anything."""
import pytest


@pytest.fixture(scope="module")
def eq():
    import group_equivariant_linear_amd as eq
    from group_equivariant_linear_amd import _build
    if not eq.built():
        _build.build()
    eq.load_library()
    return eq


A, B, C, D, E, F, G, S, W = (1 << k for k in (20, 30, 34, 36, 38, 40, 41, 42, 43))  # apart, aligned


def heads(eq, p, ts, hs):
    return eq.eqlinear_heads(p, ts, hs)


# --- plans ------------------------------------------------------------------------------

@pytest.mark.parametrize("kw", [dict(N=0), dict(N=17), dict(heads=0), dict(kv_heads=0), dict(d=1), dict(rot=0), dict(rot=3),
                                dict(rot=10), dict(layout=2), dict(layout=-1), dict(dtype=3), dict(base=0.0),
                                dict(base=float("nan")), dict(scaling=4), dict(scaling=1, factor=0.0),
                                dict(scaling=3, factor=2.0, context=0.0), dict(magnitude=0.0),
                                dict(scaling=3, factor=2.0, context=64.0, turns_slow=4.0, turns_fast=4.0),
                                dict(heads=1 << 18), dict(kv_heads=1 << 18)])
def test_rotary_plan_refusals(eq, kw):
    a = dict(N=8, heads=2, kv_heads=1, d=8, rot=8, layout=0, dtype=0) | kw
    with pytest.raises(eq.EqlError) as e:
        eq.eqlinear_rotary_plan(**a)
    assert e.value.status == eq.EQL_ERR_INVALID


@pytest.mark.parametrize("a", [(0, 2, 1, 4, 4, 0), (8, 0, 1, 4, 4, 0), (8, 3, 2, 4, 4, 0), (8, 2, 0, 4, 4, 0),
                               (8, 2, 1, 0, 4, 0), (8, 2, 1, 4, 0, 0), (8, 2, 1, 4, 4, 5), (17, 2, 1, 4, 4, 0)])
def test_mixer_plan_refusals(eq, a):
    with pytest.raises(eq.EqlError) as e:
        eq.eqlinear_mixer_plan(*a)
    assert e.value.status == eq.EQL_ERR_INVALID


def test_plans_past_the_limits_are_unsupported(eq):
    for f in (lambda: eq.eqlinear_mixer_plan(8, 2, 1, 17, 4, 0), lambda: eq.eqlinear_mixer_plan(1, 2, 1, 4, 129, 0),
              lambda: eq.eqlinear_rotary_plan(1, 1, 1, 300, 258, 0, 0)):
        with pytest.raises(eq.EqlError) as e:
            f()
        assert e.value.status == eq.EQL_ERR_UNSUPPORTED


@pytest.mark.parametrize("a", [(0, 8, 2, 0, 0), (8, 0, 1, 0, 0), (8, 8, 3, 0, 0), (8, 8, 0, 0, 0), (8, 8, 2, 3, 0),
                               (8, 8, 2, -1, 0), (8, 8, 2, 0, 7), (16, 1 << 17, 2, 0, 0)])
def test_norm_plan_refusals(eq, a):
    with pytest.raises(eq.EqlError) as e:
        eq.eqlinear_norm_plan(*a)
    assert e.value.status == eq.EQL_ERR_INVALID


@pytest.mark.parametrize("eps", [-1e-5, float("nan"), float("inf")])
def test_norm_plan_refuses_eps(eq, eps):
    with pytest.raises(eq.EqlError):
        eq.eqlinear_norm_plan(8, 8, 2, 0, 0, eps=eps)


def test_info_and_other_kinds(eq):
    lib = eq.load_library()
    r = eq.eqlinear_rotary_plan(8, 3, 1, 8, 4, 0, eq.EQL_BF16)
    m = eq.eqlinear_mixer_plan(8, 4, 2, 8, 4, eq.EQL_F16)
    n = eq.eqlinear_norm_plan(8, 24, 3, eq.EQL_ACT_SILU, eq.EQL_F32)
    assert (r.info["kind"], r.info["C_in"], r.info["N"]) == (eq.EQL_KIND_ROTARY, 24, 8)
    assert (m.info["kind"], m.info["C_in"], m.info["C_out"]) == (eq.EQL_KIND_MIXER, 32, 16)
    assert (n.info["kind"], n.info["params"], n.info["w_hat_elems"]) == (eq.EQL_KIND_NORM, 48, 0)
    layer = eq.eqlinear_plan(8, 8, 8, eq.EQL_F32)
    for p in (r, m, n):  # no layer call takes them
        assert lib.eqlinear_forward(p.handle, A, W, B, 5, None) == eq.EQL_ERR_INVALID
        assert lib.eqlinear_dense_forward(p.handle, A, W, B, 5, None) == eq.EQL_ERR_INVALID
        assert lib.eqlinear_expand_dense(p.handle, A, B, None) == eq.EQL_ERR_INVALID
        assert lib.eqlinear_backward_weight_workspace(p.handle, 5) == 0
    h = heads(eq, A, 64, 8)
    for p in (layer, m, n):
        assert lib.eqlinear_rotary(p.handle, h, None, B, 0, h, None, 5, None) == eq.EQL_ERR_INVALID
    for p in (layer, r, n):
        assert lib.eqlinear_linear_attention_workspace(p.handle, 100, 1, 1) == 0
        assert lib.eqlinear_linear_attention_step(p.handle, h, h, h, B, 1.0, C, h, 5, None) == eq.EQL_ERR_INVALID
    for p in (layer, r, m):
        assert lib.eqlinear_group_norm_workspace(p.handle, 100, 1, 1) == 0
        assert lib.eqlinear_group_norm(p.handle, A, 64, None, None, None, 1, B, 64, None, 5, None, 0,
                                       None) == eq.EQL_ERR_INVALID


# --- rotary -----------------------------------------------------------------------------

def test_rotary_refusals(eq):
    f = eq.load_library().eqlinear_rotary
    plan = eq.eqlinear_rotary_plan(8, 3, 1, 8, 4, 0, eq.EQL_BF16)  # rows: 192 and 64 elements
    p = plan.handle
    q, k = heads(eq, A, 256, 64), heads(eq, A + 384, 256, 64)
    qo, ko = heads(eq, B, 192, 64), heads(eq, C, 64, 64)
    bad = eq.EQL_ERR_INVALID
    assert f(p, q, k, S, 0, qo, ko, -1, None) == bad
    assert f(p, None, None, None, 0, None, None, 0, None) == eq.EQL_OK
    assert f(None, q, k, S, 0, qo, ko, 5, None) == bad
    assert f(p, None, k, S, 0, qo, ko, 5, None) == bad
    assert f(p, q, k, S, 0, None, ko, 5, None) == bad
    assert f(p, q, k, S, 0, qo, None, 5, None) == bad         # k without k_out
    assert f(p, q, None, S, 0, qo, ko, 5, None) == bad
    assert f(p, q, k, None, 0, qo, ko, 5, None) == bad
    assert f(p, q, k, S + 2, 0, qo, ko, 5, None) == bad       # positions misaligned
    assert f(p, heads(eq, A + 1, 256, 64), k, S, 0, qo, ko, 5, None) == bad  # half an element
    assert f(p, heads(eq, A, -256, 64), k, S, 0, qo, ko, 5, None) == bad
    assert f(p, q, k, S, 0, heads(eq, B, 100, 64), ko, 5, None) == bad       # rows of the output overlap
    assert f(p, q, k, S, 0, heads(eq, B, 192, 0), ko, 5, None) == bad        # heads of the output overlap
    assert f(p, q, k, S, 0, qo, heads(eq, B + 64, 64, 64), 5, None) == bad   # outputs over each other
    assert f(p, q, k, S, 0, heads(eq, A + 2, 256, 64), ko, 5, None) == bad   # q_out over q, shifted
    assert f(p, q, k, S, 0, k, ko, 5, None) == bad                           # q_out runs over k
    assert f(p, q, k, B + 128, 0, qo, ko, 5, None) == bad                    # positions inside q_out


# --- linear attention -------------------------------------------------------------------

def test_linear_attention_refusals(eq):
    lib = eq.load_library()
    plan = eq.eqlinear_mixer_plan(8, 4, 2, 8, 4, eq.EQL_BF16)  # D_k 64, D_v 32
    p, T = plan.handle, 6
    need = lib.eqlinear_linear_attention_workspace(p, T, 2, 1)
    row = 4 * 64 + 2 * 64 + 2 * 32
    q, k, v = heads(eq, A, row, 64), heads(eq, A + 512, row, 64), heads(eq, A + 768, row, 32)
    o = heads(eq, B, 128, 32)
    bad = eq.EQL_ERR_INVALID
    call = dict(p=p, q=q, k=k, v=v, la=C, scale=0.5, off=None, batch=2, s0=D, s1=E, o=o, T=T, ws=W,
                bytes=max(need, 256), st=None)

    def f(**kw):
        a = call | kw
        return lib.eqlinear_linear_attention(*(a[n] for n in call))

    assert f(p=None) == bad and f(T=-1) == bad and f(batch=-1) == bad and f(batch=4) == bad  # 6 tokens, 4 sequences
    assert f(batch=0) == bad                                     # tokens of no sequence
    assert f(batch=0, T=0) == eq.EQL_OK and f(T=0, s1=None) == eq.EQL_OK
    assert f(scale=0.0) == bad and f(scale=float("inf")) == bad and f(scale=float("nan")) == bad
    for n in ("q", "k", "v", "o", "la"):
        assert f(**{n: None}) == bad, n
    assert f(la=C + 2) == bad and f(s0=D + 8) == bad and f(s1=E + 4) == bad and f(off=S + 4) == bad
    assert f(s1=D) == bad and f(s1=D + 64) == bad                # the state is read while it is written
    assert f(o=heads(eq, B, 64, 32)) == bad                      # output rows overlap
    assert f(o=heads(eq, A, row, 64)) == bad                     # over q
    assert f(o=heads(eq, A + 768, row, 32)) == bad               # over v and the next row
    assert f(s1=B) == bad and f(s1=A) == bad                     # the state over o, over q
    if lib.eqlinear_linear_attention_workspace(p, T, 2, 0):
        assert f(ws=None) == bad and f(bytes=0) == bad and f(ws=W + 16) == bad and f(ws=A) == bad

    dq, dk, dv = heads(eq, F, row, 64), heads(eq, F + 512, row, 64), heads(eq, F + 768, row, 32)
    call = dict(p=p, q=q, k=k, v=v, do=o, la=C, scale=0.5, off=None, batch=2, s0=D, d1=E, dq=dq, dk=dk, dv=dv, d0=G,
                T=T, ws=W, bytes=max(need, 256), st=None)

    def g(**kw):
        a = call | kw
        return lib.eqlinear_linear_attention_backward(*(a[n] for n in call))

    assert g(p=None) == bad and g(T=-1) == bad and g(batch=4) == bad and g(scale=0.0) == bad
    assert g(batch=0, T=0) == eq.EQL_OK and g(T=0, d0=None) == eq.EQL_OK
    for n in ("q", "k", "v", "do", "la", "dq", "dk", "dv"):
        assert g(**{n: None}) == bad, n
    assert g(d0=E) == bad and g(d0=D) == bad and g(d0=F) == bad and g(d0=G + 4) == bad
    assert g(dk=heads(eq, F + 256, row, 64)) == bad              # over dq
    assert g(dq=q) == bad and g(dv=heads(eq, B, 128, 32)) == bad
    if need:
        assert g(ws=None) == bad and g(bytes=need - 1) == bad and g(ws=W + 128) == bad and g(ws=F) == bad


def test_step_refusals(eq):
    lib = eq.load_library()
    plan = eq.eqlinear_mixer_plan(8, 4, 2, 8, 4, eq.EQL_BF16)
    q, k, v, o = (heads(eq, x, 512, 64) for x in (A, B, C, D))
    call = dict(p=plan.handle, q=q, k=k, v=v, la=S, scale=0.5, state=E, o=o, batch=3, st=None)

    def f(**kw):
        a = call | kw
        return lib.eqlinear_linear_attention_step(*(a[n] for n in call))

    bad = eq.EQL_ERR_INVALID
    assert f(batch=-1) == bad and f(batch=0) == eq.EQL_OK and f(scale=0.0) == bad
    for n in ("p", "q", "k", "v", "la", "state", "o"):
        assert f(**{n: None}) == bad, n
    assert f(state=E + 4) == bad and f(state=D) == bad and f(state=A) == bad and f(o=q) == bad


# --- group norm -------------------------------------------------------------------------

def test_group_norm_refusals(eq):
    lib = eq.load_library()
    plan = eq.eqlinear_norm_plan(8, 24, 3, eq.EQL_ACT_SILU, eq.EQL_BF16)  # rows of 192 elements
    p, T = plan.handle, 6
    need = lib.eqlinear_group_norm_workspace(p, T, 2, 1)
    call = dict(p=p, x=A, ldx=192, gamma=B, beta=C, off=None, batch=2, y=D, ldy=192, stats=E, T=T, ws=W,
                bytes=max(need, 256), st=None)

    def f(**kw):
        a = call | kw
        return lib.eqlinear_group_norm(*(a[n] for n in call))

    bad = eq.EQL_ERR_INVALID
    assert f(p=None) == bad and f(T=-1) == bad and f(batch=4) == bad and f(batch=0) == bad
    assert f(batch=0, T=0) == eq.EQL_OK and f(T=0, stats=None) == eq.EQL_OK
    assert f(x=None) == bad and f(y=None) == bad and f(x=A + 1) == bad and f(y=D + 1) == bad
    assert f(ldy=100) == bad and f(ldx=-1) == bad and f(gamma=B + 1) == bad and f(stats=E + 4) == bad
    assert f(off=S + 4) == bad
    assert f(y=A + 64) == bad and f(y=A, ldy=256) == bad          # shifted, other stride
    assert f(gamma=D + 64) == bad and f(stats=D) == bad and f(stats=A) == bad

    call = dict(p=p, dy=F, lddy=192, x=A, ldx=192, gamma=B, beta=C, stats=E, off=None, batch=2, dx=D, lddx=192, dg=G,
                db=S, T=T, ws=W, bytes=max(need, 256), st=None)

    def g(**kw):
        a = call | kw
        return lib.eqlinear_group_norm_backward(*(a[n] for n in call))

    assert g(p=None) == bad and g(T=-1) == bad and g(batch=4) == bad
    for n in ("dy", "x", "dx", "stats"):
        assert g(**{n: None}) == bad, n
    assert g(dg=G + 4) == bad and g(db=G) == bad and g(db=S + 8) == bad
    assert g(dx=A) == bad and g(dx=F + 64) == bad and g(dg=D) == bad and g(stats=D) == bad and g(lddx=191) == bad
    assert g(dg=None, db=None, T=0) == eq.EQL_OK
    if need:
        assert g(ws=None) == bad and g(bytes=need - 1) == bad and g(ws=A) == bad and g(ws=W + 8) == bad


def test_binding_refusals(eq):
    """Host tensors, wrong shapes, dtypes and kinds never reach the C call."""
    import torch
    n = eq.eqlinear_norm_plan(8, 4, 2, 0, eq.EQL_F32)
    x = torch.zeros(3, 4, 8)
    with pytest.raises(ValueError):
        eq.eqlinear_group_norm(n, x, None, None, x)
    m = eq.eqlinear_mixer_plan(8, 2, 1, 4, 4, eq.EQL_F32)
    q = torch.zeros(3, 2, 4, 8)
    with pytest.raises(ValueError):
        eq.eqlinear_linear_attention(m, q, q, q, None, q, scale=1.0)
    with pytest.raises(eq.EqlError):
        eq.eqlinear_linear_attention(n, q, q, q, None, q, scale=1.0)
    r = eq.eqlinear_rotary_plan(8, 2, 1, 4, 4, 0, eq.EQL_F32)
    with pytest.raises(ValueError):
        eq.eqlinear_rotary(r, q, None, None, q, None)
    with pytest.raises(eq.EqlError):
        eq.eqlinear_rotary(m, q, None, None, q, None)

"""Refusals of softmax attention and its cache, through the C ABI with made-up addresses: every check comes before
any HIP call, so nothing here needs a GPU or launches anything."""
import ctypes

import pytest

Q, K, V, O, G, L, B, DQ, DK, DV, DB, OFF, KOFF, WS, TB, LN = (1 << 40 | (i + 1) << 32 for i in range(16))  # apart, aligned


@pytest.fixture(scope="module")
def eq():
    import group_equivariant_linear_amd as eq
    from group_equivariant_linear_amd import _build
    if not eq.built():
        _build.build()
    eq.load_library()
    return eq


@pytest.mark.parametrize("kw", [dict(N=0), dict(N=17), dict(heads=0), dict(kv_heads=0), dict(heads=3), dict(d_k=0), dict(d_v=0),
                                dict(dtype=3), dict(buckets=-1), dict(buckets=1), dict(buckets=8, max_distance=4),
                                dict(buckets=7, max_distance=40, causal=False), dict(buckets=2, max_distance=40, causal=False),
                                dict(buckets=8, max_distance=2, causal=False), dict(buckets=8, max_distance=-5),
                                dict(heads=1 << 20, kv_heads=1)])
def test_plan_refusals(eq, kw):
    a = dict(N=8, heads=4, kv_heads=2, d_k=8, d_v=8, dtype=0, causal=True) | kw
    with pytest.raises(eq.EqlError) as e:
        eq.eqlinear_attention_plan(**a)
    assert e.value.status == eq.EQL_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(d_k=17), dict(d_v=17), dict(buckets=257, max_distance=1000), dict(buckets=8, max_distance=1025)])
def test_plans_past_the_limits_are_unsupported(eq, kw):
    a = dict(N=8, heads=4, kv_heads=2, d_k=8, d_v=8, dtype=0, causal=True) | kw
    with pytest.raises(eq.EqlError) as e:
        eq.eqlinear_attention_plan(**a)
    assert e.value.status == eq.EQL_ERR_UNSUPPORTED


def test_plan_info(eq):
    p = eq.eqlinear_attention_plan(8, 12, 4, 8, 16, eq.EQL_BF16, causal=True)
    assert (p.info["kind"], p.info["N"], p.info["C_in"], p.info["C_out"]) == (eq.EQL_KIND_ATTENTION, 8, 96, 192)
    assert eq.eqlinear_attention_bucket(p, 3) == -1


@pytest.fixture(scope="module")
def plan(eq):
    return eq.eqlinear_attention_plan(8, 4, 2, 8, 8, eq.EQL_BF16, causal=True, buckets=8, max_distance=20)


def H(eq, p, heads=4, ts=None, hs=64):
    return eq.eqlinear_heads(p, heads * 64 if ts is None else ts, hs)


T, S = 100, 90


def call_forward(eq, plan, **kw):
    a = dict(q=H(eq, Q), k=H(eq, K, 2), v=H(eq, V, 2), scale=0.125, bias=B, off=OFF, koff=KOFF, batch=5, o=H(eq, O), lse=L,
             T=T, S=S, ws=WS, n=0) | kw
    ref = lambda h: None if h is None else ctypes.byref(h)  # noqa: E731
    return plan._lib.eqlinear_attention(plan.handle, ref(a["q"]), ref(a["k"]), ref(a["v"]), a["scale"], a["bias"], a["off"],
                                        a["koff"], a["batch"], ref(a["o"]), a["lse"], a["T"], a["S"], a["ws"], a["n"], None)


def bad_forward(eq):
    h = lambda *a, **k: H(eq, *a, **k)  # noqa: E731
    nan = float("nan")
    return [dict(scale=0.0), dict(scale=nan), dict(scale=float("inf")), dict(q=None), dict(k=None), dict(v=None), dict(o=None),
            dict(T=-1), dict(S=-1), dict(batch=-1), dict(batch=0), dict(off=OFF + 4), dict(koff=KOFF + 4),
            dict(off=None, batch=3), dict(koff=None, batch=4), dict(lse=L + 2), dict(bias=B + 1),
            dict(q=h(0)), dict(q=h(Q + 1)), dict(k=h(K, 2, ts=-8)), dict(v=h(V, 2, hs=-64)),
            dict(o=h(O, ts=0)), dict(o=h(O, hs=0)), dict(o=h(O, ts=255)), dict(o=h(Q)), dict(o=h(K)), dict(o=h(V + 64)),
            dict(o=h(Q + 4096)), dict(lse=Q), dict(lse=V), dict(lse=O), dict(lse=B), dict(lse=OFF), dict(lse=KOFF + 8),
            dict(o=h(B)), dict(o=h(OFF)), dict(o=h(KOFF)), dict(q=h(Q, ts=1 << 41))]


def test_forward_refusals(eq, plan):
    for kw in bad_forward(eq):
        assert call_forward(eq, plan, **kw) == eq.EQL_ERR_INVALID, kw
    other = eq.eqlinear_mixer_plan(8, 4, 2, 8, 8, eq.EQL_BF16)
    assert call_forward(eq, other) == eq.EQL_ERR_INVALID
    none = eq.eqlinear_attention_plan(8, 4, 2, 8, 8, eq.EQL_BF16)
    assert call_forward(eq, none) == eq.EQL_ERR_INVALID  # a bias without buckets
    assert call_forward(eq, plan, T=(1 << 30) + 5, off=OFF) == eq.EQL_ERR_UNSUPPORTED
    assert call_forward(eq, plan, S=(1 << 30) + 5) == eq.EQL_ERR_UNSUPPORTED
    assert call_forward(eq, plan, T=0, q=None, o=None) == eq.EQL_OK


def call_backward(eq, plan, **kw):
    need = eq.eqlinear_attention_workspace(plan, T, S, 5, backward=True) if plan.kind == eq.EQL_KIND_ATTENTION else 0
    a = dict(q=H(eq, Q), k=H(eq, K, 2), v=H(eq, V, 2), o=H(eq, O), g=H(eq, G), lse=L, scale=0.125, bias=B, off=OFF, koff=KOFF,
             batch=5, dq=H(eq, DQ), dk=H(eq, DK, 2), dv=H(eq, DV, 2), db=DB, T=T, S=S, ws=WS, n=need) | kw
    ref = lambda h: None if h is None else ctypes.byref(h)  # noqa: E731
    return plan._lib.eqlinear_attention_backward(
        plan.handle, ref(a["q"]), ref(a["k"]), ref(a["v"]), ref(a["o"]), ref(a["g"]), a["lse"], a["scale"], a["bias"], a["off"],
        a["koff"], a["batch"], ref(a["dq"]), ref(a["dk"]), ref(a["dv"]), a["db"], a["T"], a["S"], a["ws"], a["n"], None)


def test_backward_refusals(eq, plan):
    h = lambda *a, **k: H(eq, *a, **k)  # noqa: E731
    need = eq.eqlinear_attention_workspace(plan, T, S, 5, backward=True)
    assert need >= 2 * 4 * T * 4
    for kw in [dict(scale=0.0), dict(q=None), dict(o=None), dict(g=None), dict(lse=None), dict(dq=None), dict(dk=None),
               dict(dv=None), dict(k=None), dict(v=None), dict(bias=None), dict(db=DB + 2), dict(lse=L + 1), dict(T=-1),
               dict(ws=None), dict(ws=WS + 128), dict(n=need - 1), dict(off=OFF + 1), dict(batch=-2),
               dict(dq=h(DQ, ts=0)), dict(dk=h(DK, 2, ts=64)), dict(dq=h(Q)), dict(dq=h(DK)), dict(dv=h(DK, 2)), dict(dk=h(K, 2)),
               dict(dv=h(G, 2)), dict(dq=h(O)), dict(dq=h(L)), dict(dq=h(B)), dict(dk=h(DB, 2)), dict(dv=h(OFF, 2)),
               dict(db=L), dict(db=B), dict(db=OFF), dict(db=Q), dict(db=DQ), dict(db=WS), dict(ws=Q), dict(ws=DV), dict(ws=L),
               dict(ws=B), dict(ws=OFF), dict(ws=KOFF), dict(ws=DB)]:
        assert call_backward(eq, plan, **kw) == eq.EQL_ERR_INVALID, kw
    assert call_backward(eq, plan, T=(1 << 30) + 5) == eq.EQL_ERR_UNSUPPORTED
    assert call_backward(eq, plan, T=0, S=0, db=None, ws=None, n=0) == eq.EQL_OK


def pages(eq, p, bs=16 * 128, ts=128, hs=64):
    return eq.eqlinear_pages(p, bs, ts, hs)


def call_step(eq, plan, **kw):
    need = eq.eqlinear_attention_step_workspace(plan, 6) if plan.kind == eq.EQL_KIND_ATTENTION else 0
    a = dict(q=H(eq, Q), k=pages(eq, K), v=pages(eq, V), blocks=40, bs=16, table=TB, rows=9, lengths=LN, scale=0.125, bias=B,
             o=H(eq, O), lse=L, batch=6, ws=WS, n=need) | kw
    ref = lambda h: None if h is None else ctypes.byref(h)  # noqa: E731
    return plan._lib.eqlinear_attention_step(plan.handle, ref(a["q"]), ref(a["k"]), ref(a["v"]), a["blocks"], a["bs"], a["table"],
                                             a["rows"], a["lengths"], a["scale"], a["bias"], ref(a["o"]), a["lse"], a["batch"],
                                             a["ws"], a["n"], None)


def test_step_refusals(eq, plan):
    h = lambda *a, **k: H(eq, *a, **k)  # noqa: E731
    need = eq.eqlinear_attention_step_workspace(plan, 6)
    for kw in [dict(scale=0.0), dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(table=None), dict(lengths=None),
               dict(table=TB + 2), dict(lengths=LN + 1), dict(lse=L + 2), dict(bias=B + 1), dict(batch=-1), dict(blocks=-1),
               dict(bs=0), dict(rows=-1), dict(k=pages(eq, 0)), dict(k=pages(eq, K + 1)), dict(v=pages(eq, V, ts=-1)),
               dict(v=pages(eq, V, bs=1 << 41)), dict(o=h(O, ts=0)), dict(o=h(Q)), dict(o=h(K)), dict(o=h(V + 4096)), dict(o=h(TB)),
               dict(o=h(LN)), dict(o=h(B)), dict(o=h(L)), dict(lse=Q), dict(lse=K), dict(lse=TB), dict(lse=LN), dict(lse=B)]:
        assert call_step(eq, plan, **kw) == eq.EQL_ERR_INVALID, kw
    if need:
        for kw in [dict(ws=None), dict(ws=WS + 16), dict(n=need - 1), dict(ws=K), dict(ws=Q), dict(ws=O), dict(ws=TB), dict(ws=LN)]:
            assert call_step(eq, plan, **kw) == eq.EQL_ERR_INVALID, kw
    for kw in [dict(rows=(1 << 30) + 1), dict(rows=1 << 27, bs=16), dict(blocks=1 << 31)]:
        assert call_step(eq, plan, **kw) == eq.EQL_ERR_UNSUPPORTED, kw
    assert call_step(eq, plan, batch=0) == eq.EQL_OK
    none = eq.eqlinear_attention_plan(8, 4, 2, 8, 8, eq.EQL_BF16)
    assert call_step(eq, none) == eq.EQL_ERR_INVALID


def call_tables(eq, **kw):
    need = eq.eqlinear_cache_tables_workspace(6)
    a = dict(lengths=LN, added=Q, free=K, n_free=50, cursor=V, table=TB, rows=9, bs=16, out=O, cout=G, slots=L, pos=B, off=OFF,
             batch=6, T=30, ws=WS, n=need) | kw
    return eq.load_library().eqlinear_cache_tables(
        a["lengths"], a["added"], a["free"], a["n_free"], a["cursor"], a["table"], a["rows"], a["bs"], a["out"], a["cout"],
        a["slots"], a["pos"], a["off"], a["batch"], a["T"], a["ws"], a["n"], None)


def test_tables_refusals(eq):
    need = eq.eqlinear_cache_tables_workspace(6)
    assert need > 0
    for kw in [dict(batch=0), dict(batch=-1), dict(T=-1), dict(n_free=-1), dict(rows=-1), dict(bs=0), dict(lengths=None),
               dict(added=None), dict(free=None), dict(cursor=None), dict(table=None), dict(out=None), dict(cout=None),
               dict(slots=None), dict(pos=None), dict(off=None), dict(lengths=LN + 2), dict(added=Q + 1), dict(free=K + 2),
               dict(cursor=V + 1), dict(table=TB + 2), dict(out=O + 2), dict(cout=G + 2), dict(slots=L + 4), dict(pos=B + 2),
               dict(off=OFF + 4), dict(ws=None), dict(ws=WS + 8), dict(n=need - 1), dict(out=LN + 4), dict(out=Q), dict(out=V),
               dict(cout=LN), dict(cout=K), dict(table=K), dict(table=LN), dict(slots=TB), dict(pos=L), dict(off=L + 8),
               dict(ws=TB), dict(ws=Q), dict(cout=O + 8)]:
        assert call_tables(eq, **kw) == eq.EQL_ERR_INVALID, kw
    for kw in [dict(rows=1 << 27), dict(T=(1 << 30) + 1), dict(n_free=(1 << 30) + 1)]:
        assert call_tables(eq, **kw) == eq.EQL_ERR_UNSUPPORTED, kw


def call_store(eq, plan, **kw):
    a = dict(k=H(eq, Q, 2), v=H(eq, O, 2), slots=L, kc=pages(eq, K), vc=pages(eq, V), blocks=40, bs=16, T=30) | kw
    ref = lambda h: None if h is None else ctypes.byref(h)  # noqa: E731
    return plan._lib.eqlinear_cache_store(plan.handle, ref(a["k"]), ref(a["v"]), a["slots"], ref(a["kc"]), ref(a["vc"]),
                                          a["blocks"], a["bs"], a["T"], None)


def test_store_refusals(eq, plan):
    p = lambda *a, **k: pages(eq, *a, **k)  # noqa: E731
    for kw in [dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None), dict(slots=L + 4), dict(T=-1),
               dict(blocks=-1), dict(bs=0), dict(kc=p(0)), dict(kc=p(K + 1)), dict(kc=p(K, bs=0)), dict(kc=p(K, ts=0)),
               dict(kc=p(K, hs=0)), dict(kc=p(K, ts=127)), dict(kc=p(K, bs=16 * 128 - 1)), dict(vc=p(K)), dict(vc=p(K + 64)),
               dict(k=H(eq, K, 2)), dict(v=H(eq, K, 2)), dict(k=H(eq, V, 2)), dict(slots=K), dict(slots=V + 8),
               # one buffer, keys and values in turn, that do meet
               dict(kc=p(K, bs=4096), vc=p(K + 4000, bs=4096)), dict(kc=p(K, bs=4096, ts=256), vc=p(K + 2 * 120, bs=4096, ts=256))]:
        assert call_store(eq, plan, **kw) == eq.EQL_ERR_INVALID, kw
    assert call_store(eq, plan, T=0) == eq.EQL_OK
    assert call_store(eq, plan, T=(1 << 30) + 1) == eq.EQL_ERR_UNSUPPORTED


def test_sizes_of_refused_calls_are_zero(eq, plan):
    other = eq.eqlinear_mixer_plan(8, 4, 2, 8, 8, eq.EQL_BF16)
    for f in (lambda p: eq.eqlinear_attention_workspace(p, 10, 10, 1, True), lambda p: eq.eqlinear_attention_step_workspace(p, 10)):
        assert f(other) == 0
    assert eq.eqlinear_attention_workspace(plan, -1, 1, 1, True) == 0 == eq.eqlinear_attention_workspace(plan, 1 << 40, 1, 1, True)
    assert eq.eqlinear_attention_step_workspace(plan, -1) == 0 == eq.eqlinear_cache_tables_workspace(-1)


def test_calls_that_the_binding_refuses(eq, plan):
    import torch
    x = torch.zeros(4, 4, 8, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        eq.eqlinear_attention(plan, x, x, x, x, 0.1)
    with pytest.raises(TypeError):
        eq.eqlinear_cache_tables(1, 2, 3, 4, 5, 16, 6, 7, 8, 9, 10, workspace=None)
    h = eq.eqlinear_heads(Q, 256, 64)
    with pytest.raises(ValueError):
        eq.eqlinear_attention(plan, h, h, h, h, 0.1)  # T
    with pytest.raises(ValueError):
        eq.eqlinear_attention(plan, h, h, h, h, 0.1, T=4, T_kv=5, offsets=OFF, batch=2)  # keys' own offsets
    with pytest.raises(ValueError):
        eq.eqlinear_attention_step(plan, h, K, V, TB, LN, h, 0.1, batch=3)  # blocks of an address
    with pytest.raises(eq.EqlError):
        eq.eqlinear_attention(eq.eqlinear_mixer_plan(8, 4, 2, 8, 8, eq.EQL_BF16), h, h, h, h, 0.1, T=4, T_kv=4)


@pytest.mark.parametrize("scale", [2.0 ** -101, -2.0 ** -101, 1e-45])
def test_scales_that_lse_cannot_be_divided_by(eq, plan, scale):
    for call in (call_forward, call_backward, call_step):
        assert call(eq, plan, scale=scale) == eq.EQL_ERR_INVALID

"""Addresses in the operators' Python calls: what they need besides is asked for before any C call."""
import pytest


@pytest.fixture(scope="module")
def eq():
    import group_equivariant_linear_amd as eq
    from group_equivariant_linear_amd import _build
    if not eq.built():
        _build.build()
    eq.load_library()
    return eq


def test_addresses_need_the_token_count(eq):
    A = 1 << 32
    n = eq.eqlinear_norm_plan(8, 4, 2, 0, eq.EQL_F32)
    with pytest.raises(ValueError, match="T is required"):
        eq.eqlinear_group_norm(n, A, None, None, 2 * A)
    with pytest.raises(ValueError, match="T is required"):
        eq.eqlinear_group_norm_backward(n, A, 2 * A, None, None, 3 * A, 4 * A, None, None)
    r = eq.eqlinear_rotary_plan(8, 2, 1, 4, 4, 0, eq.EQL_F32)
    with pytest.raises(ValueError, match="T is required"):
        eq.eqlinear_rotary(r, A, None, A, 2 * A, None)


def test_addresses_pass_the_rows_strides(eq):
    """Contiguous rows of an address; an eqlinear_heads as it is."""
    n = eq.eqlinear_norm_plan(8, 4, 2, 0, eq.EQL_F32)
    assert eq._tokens_of(1 << 32, n, 5, "x") == (1 << 32, 32)
    assert eq._tokens_of(eq.eqlinear_heads(1 << 32, 48, 0), n, 5, "x") == (1 << 32, 48)
    r = eq.eqlinear_rotary_plan(8, 2, 1, 4, 4, 0, eq.EQL_F32)
    h = eq._heads(1 << 32, r, 5, 2, 4, "q")
    assert (h.ptr, h.token_stride, h.head_stride) == (1 << 32, 64, 32)


def test_current_stream_without_the_short_way(eq, monkeypatch):
    import torch
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    eq._current_stream.cache_clear()

    # (a fake: no GPU here)
    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    try:
        assert eq._raw_stream(None) == 77
    finally:
        eq._current_stream.cache_clear()

"""Limits of softmax attention's arguments that its C ABI answers before any HIP call (addresses are never read)."""
import ctypes

import pytest

from test_attention_abi import call_backward, call_forward, call_step, eq, plan  # noqa: F401


@pytest.mark.parametrize("call", [call_forward, call_backward, call_step])
def test_scales_whose_product_with_log2_e_is_no_number(eq, plan, call):  # noqa: F811
    """fp32 ends at 2^128; times log2 e, scales from 2.36e38 on were infinite."""
    largest = float.fromhex("0x1.fffffep127")
    for scale in (largest, -largest, 2.4e38, 2.0 ** 101, float("inf"), float("nan"), 2.0 ** -101):
        assert call(eq, plan, scale=scale) == eq.EQL_ERR_INVALID, scale


def test_step_counts_units_in_32_bits(eq, plan):  # noqa: F811
    """Up to 2048 sequences share their units of 128 keys out; with 2^38 keys and more in all, sums of them passed
    2^31.  (Short of a GPU, a call that is not refused ends in an error of HIP's.)"""
    for batch, rows in ((2048, 1024), (2048, 128), (257, 1024), (256, 1024)):
        need = eq.eqlinear_attention_step_workspace(plan, batch)
        got = call_step(eq, plan, batch=batch, rows=rows, bs=1 << 20, n=need)
        assert got == eq.EQL_ERR_UNSUPPORTED, (batch, rows)

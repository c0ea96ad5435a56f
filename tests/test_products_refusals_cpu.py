"""Calls of the product's gradients that are refused before any CUDA call: places that two results, or a result and an operand, share
(no GPU here)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def nat():
    import __graft_entry__ as g
    g.build()
    from asynchronous_expert_execution_gb300 import _native as N
    return N, N.load()


def args(N, **kw):
    at = {n: 4096 * (i + 1) for i, n in enumerate(("d_grad", "d_x", "d_w", "d_grad_x", "d_grad_w", "d_grad_bias"))}        # never looked at
    base = dict(x_dtype=N.MOE_BF16, w_dtype=N.MOE_F32, rows=4, fan_in=64, fan_out=32, grad_stride=32, x_stride=64, w_stride=64, residual_stride=64,
                grad_x_stride=64, grad_w_stride=64)
    return ctypes.byref(N.LinearBackwardArgs(**{**base, **at, **kw}))


def test_shared_places_are_refused(nat):
    N, lib = nat
    place = {n: 4096 * (i + 1) for i, n in enumerate(("d_grad", "d_x", "d_w", "d_grad_x", "d_grad_w", "d_grad_bias"))}
    for out in ("d_grad_x", "d_grad_w", "d_grad_bias"):
        for other in ("d_grad", "d_x", "d_w", "d_grad_x", "d_grad_w", "d_grad_bias"):
            if other != out:
                assert lib.moe_async_linear_backward(args(N, **{out: place[other]}), None) == N.MOE_ERR_INVALID, (out, other)
    assert lib.moe_async_linear_backward(args(N, d_residual=place["d_grad_w"]), None) == N.MOE_ERR_INVALID
    assert lib.moe_async_linear_backward(args(N, d_residual=place["d_x"], d_grad_x=place["d_x"]), None) == N.MOE_ERR_INVALID


def test_one_place_for_both_outputs_is_refused(nat):
    N, lib = nat
    P, Q = 256, 512
    assert lib.moe_async_act_mul_backward(N.MOE_BF16, 1, P, 8, P, 8, P, 8, 4, 8, Q, 8, Q, 8, None) == N.MOE_ERR_INVALID

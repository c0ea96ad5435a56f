"""Calls of the product's gradients that are refused before any CUDA call: places that two results, or a result and an operand, share,
and row counts whose walk would pass 32 bits (no GPU here)."""
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


def test_rows_whose_walk_would_pass_32_bits_are_refused(nat):
    """The bias's gradient walks rows in 32 bits: eight CTAs of eight warps with four rows each, eight of them in flight a lane, 2048 a turn.
    Its last turn looks up to two turns behind the last row; beyond 2^31 - 1 that would be a row before the matrix."""
    N, lib = nat
    turn = 8 * 8 * 4 * 8
    most = 2 ** 31 - 1 - 2 * turn
    for rows in (2 ** 31 - 1024 - 1, 2 ** 31 - 1 - turn, most + 1):
        a = args(N, rows=rows, fan_in=8, fan_out=8, grad_stride=8, x_stride=8, w_stride=8, grad_x_stride=8, grad_w_stride=8, d_x=None, d_grad_x=None, d_grad_w=None)
        assert lib.moe_async_linear_backward(a, None) == N.MOE_ERR_INVALID, rows
    # what is accepted: no index of the walk passes 2^31 - 1
    for n in (most, most - 1, most - turn):
        for first in (0, turn // 8 - 1):
            last = first + (n - 1 - first) // turn * turn                    # the last turn's first row
            assert last < n and last + turn <= 2 ** 31 - 1 and last + 7 * (turn // 8) <= 2 ** 31 - 1


def test_release_build_refuses_to_latch_a_word(nat):
    N, lib = nat
    if N.DEBUG_BOUNDS:
        pytest.skip("the bounds-checked build is loaded")
    assert lib.moe_async_debug_latch_ops_word(1, None) == N.MOE_ERR_UNSUPPORTED

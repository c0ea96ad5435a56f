"""Host-side checks of the stateless operators: every bad call is refused before any CUDA call (no GPU here)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def nat():
    import __graft_entry__ as g
    g.build()
    from asynchronous_expert_execution_gb300 import _native as N
    return N, N.load()


P = 256                                          # an address that is never looked at: every call returns early


def test_sort_and_merge_refusals(nat):
    N, lib = nat
    for T, K, E in ((-1, 2, 8), (4, 0, 8), (4, 33, 64), (4, 2, 0), (4, 2, 1025), (1 << 27, 32, 64)):
        assert lib.moe_async_sort_experts(P, T, K, E, P, P, P, None) == N.MOE_ERR_INVALID, (T, K, E)
    assert lib.moe_async_sort_experts(None, 4, 2, 8, P, P, P, None) == N.MOE_ERR_INVALID
    assert lib.moe_async_sort_experts(P, 4, 2, 8, None, P, P, None) == N.MOE_ERR_INVALID
    rows = lib.moe_async_sort_rows
    assert rows(N.MOE_BF16, P, 64, P, 0, 2, 64, P, 64, 8, None) == N.MOE_OK            # no tokens: nothing to do
    assert rows(N.MOE_BF16, P, 64, P, 4, 2, 64, P, 64, 0, None) == N.MOE_OK            # no rows
    for a in ((N.MOE_E4M3, P, 64, P, 4, 2, 64, P, 64, 8), (N.MOE_BF16, P, 63, P, 4, 2, 64, P, 64, 8), (N.MOE_BF16, P, 64, P, 4, 2, 64, P, 63, 8),
              (N.MOE_BF16, None, 64, P, 4, 2, 64, P, 64, 8), (N.MOE_BF16, P, 64, None, 4, 2, 64, P, 64, 8), (N.MOE_BF16, P, 64, P, 4, 2, 0, P, 64, 8),
              (N.MOE_BF16, P, 64, P, 4, 2, 64, P, 64, -1), (N.MOE_BF16, P, 64, P, 4, 2, 64, P, 64, 1 << 31)):
        assert rows(*a, None) == N.MOE_ERR_INVALID, a
    merge = lib.moe_async_merge_rows
    assert merge(N.MOE_F32, P, 8, 4, P, P, 0, 2, 8, None, 0, P, 8, None) == N.MOE_OK
    for a in ((N.MOE_F32, None, 8, 4, P, P, 2, 2, 8, None, 0, P, 8), (N.MOE_F32, P, 7, 4, P, P, 2, 2, 8, None, 0, P, 8),
              (N.MOE_F32, P, 8, 4, P, P, 2, 2, 8, P, 7, P, 8), (N.MOE_F32, P, 8, 4, P, P, 2, 2, 8, None, 0, None, 8),
              (N.MOE_F32, P, 8, 4, P, P, 2, 2, 8, None, 0, P, 7), (9, P, 8, 4, P, P, 2, 2, 8, None, 0, P, 8)):
        assert merge(*a, None) == N.MOE_ERR_INVALID, a
    back = lib.moe_async_merge_rows_backward
    assert back(N.MOE_F32, P, 8, P, 8, 4, P, P, 0, 2, 8, P, 8, P, None) == N.MOE_OK
    for a in ((N.MOE_F32, None, 8, P, 8, 4, P, P, 2, 2, 8, P, 8, P), (N.MOE_F32, P, 8, P, 8, 4, P, None, 2, 2, 8, P, 8, P),
              (N.MOE_F32, P, 8, P, 8, 4, P, P, 2, 2, 8, P, 8, None), (N.MOE_F32, P, 8, P, 8, 4, P, P, 2, 2, 8, None, 8, P)):
        assert back(*a, None) == N.MOE_ERR_INVALID, a
    rb = lib.moe_async_route_backward
    assert rb(P, P, P, 0, 8, 2, P, None) == N.MOE_OK
    for a in ((P, P, P, 4, 8, 9, P), (P, P, P, 4, 1025, 2, P), (None, P, P, 4, 8, 2, P), (P, P, P, 4, 8, 2, None)):
        assert rb(*a, None) == N.MOE_ERR_INVALID, a


def test_norm_refusals(nat):
    N, lib = nat
    f = lib.moe_async_add_rms_norm
    assert f(N.MOE_BF16, P, 64, None, 0, None, 1e-6, 0, 64, None, 0, P, 64, None, None) == N.MOE_OK
    for a in ((N.MOE_E4M3, P, 64, None, 0, None, 1e-6, 4, 64, None, 0, P, 64, None), (N.MOE_BF16, P, 64, None, 0, None, -1.0, 4, 64, None, 0, P, 64, None),
              (N.MOE_BF16, P, 64, None, 0, None, float("nan"), 4, 64, None, 0, P, 64, None), (N.MOE_BF16, P, 64, None, 0, None, 1e-6, 4, 0, None, 0, P, 64, None),
              (N.MOE_BF16, P, 63, None, 0, None, 1e-6, 4, 64, None, 0, P, 64, None), (N.MOE_BF16, P, 64, P, 63, None, 1e-6, 4, 64, P, 64, P, 64, None),
              (N.MOE_BF16, P, 64, None, 0, None, 1e-6, 4, 64, P, 64, P, 64, None), (N.MOE_BF16, P, 64, None, 0, None, 1e-6, 4, 64, None, 0, None, 64, None)):
        assert f(*a, None) == N.MOE_ERR_INVALID, a
    need = lib.moe_async_add_rms_norm_backward_workspace
    assert need(0, 64) == 0 and need(1, 64) >= 256 and need(100000, 7168) >= 4 * 7168
    b = lib.moe_async_add_rms_norm_backward
    size = need(4, 64)
    assert b(N.MOE_BF16, P, 64, P, 64, P, 1e-6, 4, 64, None, 0, P, 64, P, P, size - 1, None) == N.MOE_ERR_CAPACITY
    for a in ((N.MOE_BF16, P, 64, P, 64, P, 1e-6, 4, 64, None, 0, P, 64, P, None, size), (N.MOE_BF16, P, 64, P, 64, P, 1e-6, 4, 64, None, 0, P, 64, P, P + 4, size),
              (N.MOE_BF16, None, 64, P, 64, P, 1e-6, 4, 64, None, 0, P, 64, P, P, size), (N.MOE_BF16, P, 64, P, 64, P, 1e-6, 4, 64, P, 8, P, 64, P, P, size),
              (N.MOE_BF16, P, 64, P, 64, P, 1e-6, -1, 64, None, 0, P, 64, P, P, size)):
        assert b(*a, None) == N.MOE_ERR_INVALID, a


def test_linear_refusals(nat):
    N, lib = nat
    base = dict(dtype=N.MOE_BF16, out_dtype=N.MOE_BF16, act=0, rows=4, fan_in=64, fan_out=32, groups=0, d_x=P, d_w=P, d_y=P, x_stride=64,
                w_stride=64, mul_stride=32, residual_stride=32, y_stride=32)
    call = lambda **kw: lib.moe_async_linear(ctypes.byref(N.LinearArgs(**{**base, **kw})), None)   # noqa: E731
    assert lib.moe_async_linear(None, None) == N.MOE_ERR_INVALID
    assert call(rows=0) == N.MOE_OK
    for kw in (dict(rows=-1), dict(fan_in=0), dict(fan_out=0), dict(fan_in=2 ** 31 - 16, x_stride=2 ** 31, w_stride=2 ** 31),
               dict(fan_out=2 ** 31 - 1, y_stride=2 ** 31), dict(groups=-1), dict(groups=3), dict(groups=1025, d_offsets=P), dict(d_offsets=P),
               dict(act=4), dict(act=-1), dict(out_dtype=N.MOE_E4M3), dict(d_x=None), dict(d_w=None), dict(d_y=None), dict(x_stride=56),
               dict(w_stride=56), dict(y_stride=31), dict(d_mul=P, mul_stride=31), dict(d_residual=P, residual_stride=31), dict(d_x_scale=P),
               dict(d_w_scale=P), dict(dtype=N.MOE_E4M3), dict(dtype=N.MOE_E4M3, d_x_scale=P)):
        assert call(**kw) == N.MOE_ERR_INVALID, kw
    for kw in (dict(dtype=N.MOE_F32), dict(dtype=7), dict(fan_in=60), dict(d_x=P + 8), dict(d_w=P + 2), dict(x_stride=68), dict(w_stride=65),
               dict(dtype=N.MOE_E4M3, d_x_scale=P, d_w_scale=P, fan_in=56)):
        assert call(**kw) == N.MOE_ERR_UNSUPPORTED, kw


def test_tensors_off_the_gpu_are_refused(nat):
    import asynchronous_expert_execution_gb300 as moe
    x, pos, w = torch.zeros((2, 8)), torch.zeros((2, 1), dtype=torch.int32), torch.zeros((2, 1))
    for f in (lambda: moe.sort_experts(pos, 2), lambda: moe.sort_rows(x, pos), lambda: moe.merge_rows(x, pos, w), lambda: moe.add_rms_norm(x),
              lambda: moe.merge_rows_backward(x, x, pos, w), lambda: moe.route_backward(pos, w, w, 4), lambda: moe.add_rms_norm_backward(x, x),
              lambda: moe.sort_rows_backward(x, pos), lambda: moe.add_rms_norm_e4m3(x), lambda: moe.linear(x.bfloat16(), x.bfloat16())):
        with pytest.raises(moe.MoEError):
            f()

"""Host-side checks of the product's gradients, the block-scaled product and its quantisers: every bad call is refused before any
CUDA call (no GPU here)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 256                                          # an address that is never looked at: every call returns early


@pytest.fixture(scope="module")
def nat():
    import __graft_entry__ as g
    g.build()
    from asynchronous_expert_execution_gb300 import _native as N
    return N, N.load()


def test_linear_backward_refusals(nat):
    N, lib = nat
    base = dict(x_dtype=N.MOE_BF16, w_dtype=N.MOE_F32, rows=4, fan_in=64, fan_out=32, d_grad=P, d_x=P, d_w=P, d_grad_x=P, d_grad_w=P, grad_stride=32, x_stride=64,
                w_stride=64, residual_stride=64, grad_x_stride=64, grad_w_stride=64)
    args = lambda kw: ctypes.byref(N.LinearBackwardArgs(**{**base, **kw}))   # noqa: E731
    call = lambda **kw: lib.moe_async_linear_backward(args(kw), None)        # noqa: E731
    assert lib.moe_async_linear_backward(None, None) == N.MOE_ERR_INVALID
    assert call(rows=0, accumulate=1) == N.MOE_OK
    for kw in (dict(rows=-1), dict(fan_in=0), dict(fan_out=0), dict(groups=-1), dict(groups=3), dict(groups=1025, d_offsets=P), dict(d_offsets=P), dict(x_dtype=N.MOE_E4M3),
               dict(w_dtype=7), dict(d_grad=None), dict(d_x=None), dict(d_w=None), dict(grad_stride=31), dict(x_stride=56), dict(w_stride=56), dict(grad_x_stride=56),
               dict(grad_w_stride=56), dict(d_residual=P, residual_stride=63), dict(d_residual=P, d_grad_x=None), dict(d_grad=P + 2), dict(fan_in=2 ** 31 - 8)):
        assert call(**kw) == N.MOE_ERR_INVALID, kw
    for kw in (dict(fan_in=60), dict(d_x=P + 8), dict(d_w=P + 2), dict(x_stride=68), dict(w_stride=65), dict(fan_out=2 ** 30, grad_stride=2 ** 30, fan_in=2 ** 20, x_stride=2 ** 20,
                                                                                                          w_stride=2 ** 20, grad_x_stride=2 ** 20, grad_w_stride=2 ** 20)):
        assert call(**kw) == N.MOE_ERR_UNSUPPORTED, kw
    need = lambda **kw: lib.moe_async_linear_backward_workspace(args(kw))    # noqa: E731
    assert need() == 0 and need(rows=0) == 0 and need(fan_out=33, grad_stride=40) == 0
    assert need(fan_out=33, grad_stride=33) == 4 * 40 * 2 and need(d_grad=P + 2) == 4 * 32 * 2
    odd = dict(fan_out=33, grad_stride=33)
    assert call(**odd, d_workspace=P, workspace_bytes=4 * 40 * 2 - 1) == N.MOE_ERR_CAPACITY
    assert call(**odd, workspace_bytes=1 << 20) == N.MOE_ERR_INVALID and call(**odd, d_workspace=P + 4, workspace_bytes=1 << 20) == N.MOE_ERR_INVALID


def test_act_mul_backward_refusals(nat):
    N, lib = nat
    f = lib.moe_async_act_mul_backward
    assert f(N.MOE_BF16, 1, P, 8, P, 8, P, 8, 0, 8, P, 8, P, 8, None) == N.MOE_OK
    for a in ((N.MOE_E4M3, 1, P, 8, P, 8, P, 8, 4, 8, P, 8, P, 8), (N.MOE_BF16, 4, P, 8, P, 8, P, 8, 4, 8, P, 8, P, 8), (N.MOE_BF16, -1, P, 8, P, 8, P, 8, 4, 8, P, 8, P, 8),
              (N.MOE_BF16, 1, None, 8, P, 8, P, 8, 4, 8, P, 8, P, 8), (N.MOE_BF16, 1, P, 7, P, 8, P, 8, 4, 8, P, 8, P, 8), (N.MOE_BF16, 1, P, 8, P, 7, P, 8, 4, 8, P, 8, P, 8),
              (N.MOE_BF16, 1, P, 8, P, 8, P, 7, 4, 8, P, 8, P, 8), (N.MOE_BF16, 1, P, 8, P, 8, None, 8, 4, 8, P, 8, P, 8), (N.MOE_BF16, 1, P, 8, P, 8, P, 8, 4, 8, P, 8, None, 8),
              (N.MOE_BF16, 1, P, 8, P, 8, P, 8, 4, 8, P, 7, P, 8), (N.MOE_BF16, 1, P, 8, P, 8, P, 8, 4, 8, None, 8, P, 8), (N.MOE_BF16, 1, P, 8, P, 8, P, 8, -1, 8, P, 8, P, 8),
              (N.MOE_BF16, 1, P, 8, P, 8, P, 8, 4, 0, P, 8, P, 8), (N.MOE_F32, 1, P, 2 ** 31, P, 2 ** 31, P, 2 ** 31, 4, 2 ** 31 - 1, P, 2 ** 31, P, 2 ** 31)):
        assert f(*a, None) == N.MOE_ERR_INVALID, a


def test_linear_blocks_refusals(nat):
    N, lib = nat
    base = dict(dtype=N.MOE_E4M3, out_dtype=N.MOE_BF16, act=0, rows=4, fan_in=64, fan_out=32, groups=0, d_x=P, d_w=P, d_y=P, d_x_scale=P, d_w_scale=P, x_stride=64,
                w_stride=64, mul_stride=32, residual_stride=32, y_stride=32)
    call = lambda sr=1, sb=4, **kw: lib.moe_async_linear_blocks(ctypes.byref(N.LinearArgs(**{**base, **kw})), sr, sb, None)   # noqa: E731
    assert lib.moe_async_linear_blocks(None, 1, 4, None) == N.MOE_ERR_INVALID
    assert call(rows=0) == N.MOE_OK
    for kw in (dict(rows=-1), dict(fan_in=0), dict(fan_out=0), dict(groups=-1), dict(groups=3), dict(groups=1025, d_offsets=P), dict(d_offsets=P), dict(act=4), dict(act=-1),
               dict(out_dtype=N.MOE_E4M3), dict(d_x=None), dict(d_w=None), dict(d_y=None), dict(x_stride=56), dict(w_stride=56), dict(y_stride=31), dict(d_mul=P, mul_stride=31),
               dict(d_residual=P, residual_stride=31), dict(d_x_scale=None), dict(d_w_scale=None), dict(sr=-1), dict(sb=-1)):
        assert call(**kw) == N.MOE_ERR_INVALID, kw
    for kw in (dict(dtype=N.MOE_F32), dict(dtype=N.MOE_BF16), dict(fan_in=56), dict(d_x=P + 8), dict(d_w=P + 2), dict(x_stride=72), dict(w_stride=65)):
        assert call(**kw) == N.MOE_ERR_UNSUPPORTED, kw


def test_quantize_refusals(nat):
    N, lib = nat
    f = lib.moe_async_quantize_blocks
    assert f(N.MOE_BF16, P, 64, 1, 0, 64, 1, P, 64, P, 1, 4, None) == N.MOE_OK
    for a in ((N.MOE_E4M3, P, 64, 1, 4, 64, 1, P, 64, P, 1, 4), (N.MOE_BF16, P, 63, 1, 4, 64, 1, P, 64, P, 1, 4), (N.MOE_BF16, P, 64, 1, 4, 64, 1, P, 63, P, 1, 4),
              (N.MOE_BF16, None, 64, 1, 4, 64, 1, P, 64, P, 1, 4), (N.MOE_BF16, P, 64, 1, 4, 64, 1, None, 64, P, 1, 4), (N.MOE_BF16, P, 64, 1, 4, 64, 1, P, 64, None, 1, 4),
              (N.MOE_BF16, P, 64, 2, 4, 64, 1, P, 64, P, 1, 4), (N.MOE_BF16, P, 64, 0, 4, 64, 128, P, 64, P, 1, 4), (N.MOE_BF16, P, 64, 1, 4, 64, 64, P, 64, P, 1, 4),
              (N.MOE_BF16, P, 64, 1, -1, 64, 1, P, 64, P, 1, 4), (N.MOE_BF16, P, 64, 1, 4, 0, 1, P, 64, P, 1, 4), (N.MOE_BF16, P, 64, 1, 4, 64, 1, P, 64, P, -1, 4),
              (N.MOE_F32, P, 2 ** 31, 1, 4, 2 ** 31 - 1, 1, P, 2 ** 31, P, 1, 4)):
        assert f(*a, None) == N.MOE_ERR_INVALID, a


def test_tensors_off_the_gpu_are_refused(nat):
    import asynchronous_expert_execution_gb300 as moe
    x = torch.zeros((2, 8))
    for f in (lambda: moe.linear_backward(x.bfloat16(), x.bfloat16(), x.bfloat16()), lambda: moe.act_mul_backward(x, x), lambda: moe.quantize_blocks(x),
              lambda: moe.quantize_weight_blocks(x), lambda: moe.act_mul_backward(x, x, act="tanh")):
        with pytest.raises(moe.MoEError):
            f()


def test_one_shared_memory_limit_a_kernel():
    """A kernel's limit of dynamic shared memory belongs to the function: every place that sets it gives the same constant."""
    csrc = os.path.join(ROOT, "asynchronous_expert_execution_gb300", "csrc")
    for f in ("moe_linear_backward.cu", "moe_linear_blocks.cu"):
        limits = {}
        for name, size in re.findall(r"cudaFuncSetAttribute\((\w+)(?:<[^()]*?>)?,\s*cudaFuncAttributeMaxDynamicSharedMemorySize,\s*([^)]*(?:\([^)]*\)[^)]*)?)\)",
                                     open(os.path.join(csrc, f)).read()):
            limits.setdefault(name, set()).add(size)
        assert len(limits) >= 2 and all(len(s) == 1 and re.fullmatch(r"k[A-Z]\w*", next(iter(s))) for s in limits.values()), (f, limits)

"""Host-side checks of the stateless operators beyond their refusals (no GPU here)."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "asynchronous_expert_execution_gb300", "csrc")


def test_one_shared_memory_limit_a_kernel():
    """A kernel's limit of dynamic shared memory belongs to the function: host threads that set different ones take it
    away from each other between setting and launch.  Every place that sets an operator's limit gives the same constant."""
    limits = {}
    for f in ("moe_sort.cu", "moe_norm.cu", "moe_linear.cu"):
        src = open(os.path.join(CSRC, f)).read()
        local = dict(re.findall(r"const auto (\w+) = (\w+)<[^;]*>;", src))
        for name, size in re.findall(r"cudaFuncSetAttribute\((\w+)(?:<[^()]*?>)?,\s*cudaFuncAttributeMaxDynamicSharedMemorySize,\s*([^)]*(?:\([^)]*\)[^)]*)?)\)", src):
            limits.setdefault(local.get(name, name), set()).add(" ".join(size.split()))
    assert {"sort_experts_kernel", "rms_norm_backward_ring_kernel", "linear_split_kernel", "linear_pair_kernel"} <= set(limits)
    for name, sizes in limits.items():
        assert len(sizes) == 1, (name, sizes)
        assert re.fullmatch(r"(k[A-Z]\w*|\d+)( [*+] (k[A-Z]\w*|\d+))*", next(iter(sizes))), (name, sizes)


@pytest.fixture(scope="module")
def nat():
    import __graft_entry__ as g
    g.build()
    from asynchronous_expert_execution_gb300 import _native as N
    return N, N.load()


P = 256                                          # an address that is never looked at: every call returns early


@pytest.mark.parametrize("H", [2 ** 31 - 1, 2 ** 31 - 8, 2 ** 31 - 65536])
def test_widths_whose_columns_would_pass_32_bits_are_refused(nat, H):
    """Column indices are 32-bit and step past the row's end by up to a block's columns: a width near 2^31 would wrap there."""
    N, lib = nat
    for dt in (N.MOE_F32, N.MOE_BF16):
        assert lib.moe_async_add_rms_norm(dt, P, H, None, 0, None, 1e-6, 1, H, None, 0, P, H, None, None) == N.MOE_ERR_INVALID
        assert lib.moe_async_add_rms_norm_backward(dt, P, H, P, H, None, 1e-6, 1, H, None, 0, P, H, None, None, 0, None) == N.MOE_ERR_INVALID
        assert lib.moe_async_sort_rows(dt, P, H, P, 1, 1, H, P, H, 1, None) == N.MOE_ERR_INVALID
        assert lib.moe_async_merge_rows(dt, P, H, 1, P, P, 1, 1, H, None, 0, P, H, None) == N.MOE_ERR_INVALID
        assert lib.moe_async_merge_rows_backward(dt, P, H, P, H, 1, P, P, 1, 1, H, P, H, P, None) == N.MOE_ERR_INVALID


def test_release_build_refuses_to_latch_an_error(nat):
    """Only the bounds-checked build sets the operators' error word by hand."""
    N, lib = nat
    if N.DEBUG_BOUNDS:
        pytest.skip("the bounds-checked build is loaded")
    assert lib.moe_async_debug_latch_ops_error(None) == N.MOE_ERR_UNSUPPORTED


def test_binding_of_another_torch_is_rebuilt_and_not_loaded(nat, monkeypatch):
    """The binding uses torch's C++ classes: a binary of another version is stale whatever its file's time, and is refused."""
    import torch
    import asynchronous_expert_execution_gb300 as moe
    from asynchronous_expert_execution_gb300 import build as b, ops
    assert not b._binding_stale()
    monkeypatch.setattr(ops, "_bound", None)
    moe_error = None
    try:
        moe.add_rms_norm(torch.zeros((2, 8)))                                # binds, then refuses a CPU tensor
    except moe.MoEError as e:
        moe_error = e
    assert moe_error is not None
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    assert b._binding_stale()
    monkeypatch.setattr(ops, "_bound", None)
    with pytest.raises(RuntimeError, match="built for"):
        moe.add_rms_norm(torch.zeros((2, 8)))


def test_ops_sync_looks_at_the_device_of_its_stream(monkeypatch):
    """The error word is the device's: with a stream and no device, that is the stream's."""
    import contextlib
    import types
    import torch
    from asynchronous_expert_execution_gb300 import ops
    seen = []
    monkeypatch.setattr(ops.torch.cuda, "device", lambda d: seen.append(d) or contextlib.nullcontext())
    monkeypatch.setattr(ops.N, "load", lambda: types.SimpleNamespace(moe_async_ops_status=lambda s: seen.append(s) or 0))
    stream = types.SimpleNamespace(cuda_stream=7, device=torch.device("cuda", 1))
    ops.ops_sync(stream=stream)
    ops.ops_sync(0, stream)
    assert seen == [torch.device("cuda", 1), 7, 0, 7]

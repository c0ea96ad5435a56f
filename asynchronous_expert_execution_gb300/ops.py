"""Stateless operators around the expert path: thin functions over the C ABI, as in api.py.

For a caller that holds a whole routed batch (a prefill chunk, a training step):

    y, h = add_rms_norm(x, residual, gain)                 # or add_rms_norm_e4m3: 8 bits and a scale per row
    idx, w = route(linear(y, w_router, out_dtype=torch.float32), top_k)
    offsets, pos, pair = sort_experts(idx, num_experts)
    rows = sort_rows(y, pos)
    up = linear(rows, w3, offsets=offsets)                  # one product per expert
    act = linear(rows, w1, act="silu", mul=up, offsets=offsets)
    out = merge_rows(linear(act, w2, offsets=offsets), pos, w, residual=h)

Every function runs on the device of its first tensor, on that device's current stream unless
``stream`` is given, allocates only the outputs it is not handed, and raises ``MoEError``
(``MOE_ERR_INVALID``) for tensors that do not fit together.  Gradients are functions of their
own (``*_backward``), for an ``autograd.Function`` to call; nothing is recorded here, so a tensor
that requires grad is refused while grad mode is on.  Matrices are [rows, width] with adjacent
columns and any row stride.
"""
import ctypes

import torch

from . import _native as N

_ORDER = ("sort_experts", "sort_rows", "merge_rows", "merge_rows_backward", "route_backward", "add_rms_norm",
          "add_rms_norm_backward_workspace", "add_rms_norm_backward", "linear")
_bound = None


def _bind():
    """The binding (built beside the library), bound to the library that _native loaded."""
    global _bound
    from .build import binding_tag
    lib = N.load()
    try:
        from . import _ops
    except ImportError as e:
        raise RuntimeError("the operators' binding is missing or does not load: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`") from e
    if _ops.built_for != binding_tag():
        raise RuntimeError(f"the operators' binding was built for {_ops.built_for}, this is {binding_tag()}: build it again with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    _ops.bind(N.MoEError, *(ctypes.cast(getattr(lib, "moe_async_" + n), ctypes.c_void_p).value for n in _ORDER))
    _bound = _ops
    return _ops


def sort_experts(expert, num_experts, stream=None):
    """Order of a routed batch's pairs by expert, pairs of one expert in pair order.

    expert int32 [T, K] (ids outside [0, num_experts) get no row) -> (offsets int32 [E + 1]: the
    rows of expert e are offsets[e]:offsets[e + 1]; pos int32 [T, K]: the row of each pair, -1
    without one; pair int32 [T * K]: the pair t * K + k of each row, pairs without one last)."""
    return (_bound or _bind()).sort_experts(expert, num_experts, stream)


def sort_rows(x, pos, out=None, stream=None):
    """rows[pos[t, k]] = x[t]: x [T, H] fp32 or bf16, pos int32 [T, K] -> rows [T * K, H] (or
    `out` [R, H]); rows that no pair names are left as they were (in a new matrix: not set).  Each row
    is named by at most one pair, as sort_experts names them."""
    return (_bound or _bind()).sort_rows(x, pos, out, stream)


def merge_rows(rows, pos, w=None, residual=None, out=None, stream=None):
    """y[t] = sum_k w[t, k] rows[pos[t, k]] + residual[t] in fp32, ascending k, rounded once:
    rows [R, H], pos int32 [T, K], w fp32 [T, K] (None: plain sums), residual [T, H] or None ->
    y [T, H].  A pair without a row (pos outside [0, R)) adds nothing.  `out` may be `residual`."""
    return (_bound or _bind()).merge_rows(rows, pos, w, residual, out, stream)


def sort_rows_backward(grad_rows, pos, out=None, stream=None):
    """Gradient of sort_rows: grad_x[t] = sum_k grad_rows[pos[t, k]]."""
    return (_bound or _bind()).merge_rows(grad_rows, pos, None, None, out, stream)


def merge_rows_backward(grad, rows, pos, w, out=None, stream=None):
    """Gradients of merge_rows: (grad_rows, grad_w) with grad_rows[pos[t, k]] = w[t, k] grad[t]
    ([R, H] or `out`; rows that no pair names are left as they were, in a new matrix not set) and
    grad_w[t, k] = <rows[pos[t, k]], grad[t]> (fp32, 0 for a pair without a row).  The residual's is
    `grad`.  Each row is named by at most one pair."""
    return (_bound or _bind()).merge_rows_backward(grad, rows, pos, w, out, stream)


def route_backward(idx, w, grad_w, num_experts, stream=None):
    """Gradient of route's weights: idx int32 and w fp32 [T, K] as route returned them, grad_w
    fp32 [T, K] -> grad_logits fp32 [T, num_experts]."""
    return (_bound or _bind()).route_backward(idx, w, grad_w, num_experts, stream)


def add_rms_norm(x, residual=None, gain=None, eps=1e-6, out=None, out_h=None, stream=None):
    """(y, h): h = x + residual rounded to their type (x itself without a residual), y = h /
    sqrt(mean(h^2) + eps) * gain.  x, residual [T, H] fp32 or bf16, gain fp32 [H] or None.
    `out_h` may be x or residual."""
    y, _, h = (_bound or _bind()).add_rms_norm(x, residual, gain, eps, out, out_h, stream, False)
    return y, h


def add_rms_norm_e4m3(x, residual=None, gain=None, eps=1e-6, out=None, out_h=None, stream=None):
    """(q, scale, h): add_rms_norm with y in e4m3, one fp32 scale per row (y = q * scale, scale =
    max(max|y| / 448, 2^-126)): the operands x and x_scale of linear."""
    return (_bound or _bind()).add_rms_norm(x, residual, gain, eps, out, out_h, stream, True)


def add_rms_norm_backward(grad, h, gain=None, eps=1e-6, grad_h=None, out=None, stream=None):
    """Gradients of add_rms_norm at its h: (grad_x, grad_gain) from grad, the gradient of y, and
    grad_h, the gradient that arrives at h itself (or None).  grad_x is the gradient of x and of
    the residual alike; grad_gain is fp32 [H], None without a gain.  `out` may be `grad_h`."""
    return (_bound or _bind()).add_rms_norm_backward(grad, h, gain, eps, grad_h, out, stream)


def linear(x, weight, bias=None, act="none", mul=None, residual=None, offsets=None, x_scale=None, w_scale=None,
           out_dtype=None, out=None, stream=None):
    """act(x @ weight.T + bias) * mul + residual, products summed in fp32, rounded once.

    x [T, F] and weight [N, F], both bf16, or both e4m3 with x_scale fp32 [T] and w_scale fp32
    [N]; F a multiple of 16 bytes, rows of x and weight on 16-byte boundaries.  bias fp32 [N]; mul
    and residual [T, N] in the type of the result (out's, out_dtype or bf16; fp32 or bf16); act
    "none", "silu", "gelu" (the exact one) or "relu".  `out` may be mul or residual.
    With offsets (int32 [G + 1], as sort_experts gives them) weight is [G, N, F], bias and w_scale
    are [G, N], and rows offsets[g]:offsets[g + 1] of x meet weight[g]; other rows of `out` are
    left as they were (in a new matrix: not set)."""
    code = N.ACTS.get(act)
    if code is None:
        raise N.MoEError(N.MOE_ERR_INVALID, f"act: expected one of {tuple(N.ACTS)}, got {act!r}")
    return (_bound or _bind()).linear(x, weight, bias, code, mul, residual, offsets, x_scale, w_scale, out_dtype, out, stream)


def ops_sync(device=None, stream=None):
    """Wait for `stream` (default: the device's current one) and raise MoEError if a stateless
    operator found an error on the device since the last report, on any stream (a wait in linear that
    exceeded its bound).  Reported once: a call made after it starts clear."""
    with torch.cuda.device(getattr(stream, "device", None) if device is None else device):
        s = torch.cuda.current_stream() if stream is None else stream
        N.check(N.load().moe_async_ops_status(s.cuda_stream), "ops_sync")

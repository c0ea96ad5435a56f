"""Stateless operators around the expert path: argument marshalling only, as in api.py.

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
own (``*_backward``).  Matrices are [rows, width] with adjacent columns and any row stride.
"""
import ctypes

import torch

from . import _native as N

_DT = {torch.float32: N.MOE_F32, torch.bfloat16: N.MOE_BF16, torch.float8_e4m3fn: N.MOE_E4M3}
_ROWS = (torch.float32, torch.bfloat16)


def _need(ok, what):
    if not ok:
        raise N.MoEError(N.MOE_ERR_INVALID, what)


def _matrix(t, name, like, shape, dtype):
    """A [rows, width] operand on the device of `like`: adjacent columns, any row stride."""
    _need(t.device == like.device and t.dtype == dtype and tuple(t.shape) == shape
          and (shape[1] == 1 or t.stride(1) == 1) and (shape[0] <= 1 or t.stride(0) >= shape[1]),
          f"{name}: expected {shape} of {dtype} on {like.device} with adjacent columns, got {tuple(t.shape)} of "
          f"{t.dtype} on {t.device}, strides {t.stride()}")


def _vector(t, name, like, shape, dtype):
    _need(t.device == like.device and t.dtype == dtype and tuple(t.shape) == shape and t.is_contiguous(),
          f"{name}: expected contiguous {shape} of {dtype} on {like.device}, got {tuple(t.shape)} of {t.dtype} on "
          f"{t.device}")


def _first(t, name, dtypes):
    _need(t.is_cuda and t.dim() == 2 and t.dtype in dtypes, f"{name}: expected a CUDA matrix of {dtypes}, got "
          f"{tuple(t.shape)} of {t.dtype} on {t.device}")


def _ld(t):
    """Row stride in elements (a single row has none: its width)."""
    return max(t.stride(0), t.shape[1]) if t.shape[0] > 1 else t.shape[1]


def _p(t):
    return None if t is None else t.data_ptr()


class _On:
    """The call's device made current, and its stream."""
    __slots__ = ("dev", "prev", "stream")

    def __init__(self, t, stream):
        self.dev, self.stream = t.device.index, stream

    def __enter__(self):
        self.prev = torch.cuda.current_device()
        if self.prev != self.dev:
            torch.cuda.set_device(self.dev)
        s = torch.cuda.current_stream() if self.stream is None else self.stream
        return s.cuda_stream

    def __exit__(self, *_):
        if self.prev != self.dev:
            torch.cuda.set_device(self.prev)


def sort_experts(expert, num_experts, stream=None):
    """Order of a routed batch's pairs by expert, pairs of one expert in pair order.

    expert int32 [T, K] (ids outside [0, num_experts) get no row) -> (offsets int32 [E + 1]: the
    rows of expert e are offsets[e]:offsets[e + 1]; pos int32 [T, K]: the row of each pair, -1
    without one; pair int32 [T * K]: the pair t * K + k of each row, pairs without one last)."""
    _first(expert, "expert", (torch.int32,))
    _need(expert.is_contiguous(), "expert: expected contiguous")
    T, K = expert.shape
    with _On(expert, stream) as s:
        offsets = torch.empty(num_experts + 1 if num_experts > 0 else 1, dtype=torch.int32, device=expert.device)
        pos, pair = torch.empty_like(expert), torch.empty(T * K, dtype=torch.int32, device=expert.device)
        N.check(N.load().moe_async_sort_experts(_p(expert), T, K, num_experts, _p(offsets), _p(pos), _p(pair), s),
                "sort_experts")
    return offsets, pos, pair


def sort_rows(x, pos, out=None, stream=None):
    """rows[pos[t, k]] = x[t]: x [T, H] fp32 or bf16, pos int32 [T, K] -> rows [T * K, H] (or
    `out` [R, H]); rows that no pair names are left as they were."""
    _first(x, "x", _ROWS)
    T, H = x.shape
    _matrix(x, "x", x, (T, H), x.dtype)
    _need(pos.dim() == 2, "pos: expected [T, K]")
    K = pos.shape[1]
    _vector(pos, "pos", x, (T, K), torch.int32)
    with _On(x, stream) as s:
        if out is None:
            out = torch.empty((T * K, H), dtype=x.dtype, device=x.device)
        else:
            _matrix(out, "out", x, (out.shape[0], H), x.dtype)
        N.check(N.load().moe_async_sort_rows(_DT[x.dtype], _p(x), _ld(x), _p(pos), T, K, H, _p(out), _ld(out),
                                             out.shape[0], s), "sort_rows")
    return out


def merge_rows(rows, pos, w=None, residual=None, out=None, stream=None):
    """y[t] = sum_k w[t, k] rows[pos[t, k]] + residual[t] in fp32, ascending k, rounded once:
    rows [R, H], pos int32 [T, K], w fp32 [T, K] (None: plain sums), residual [T, H] or None ->
    y [T, H].  A pair without a row (pos outside [0, R)) adds nothing.  `out` may be `residual`."""
    _first(rows, "rows", _ROWS)
    R, H = rows.shape
    _matrix(rows, "rows", rows, (R, H), rows.dtype)
    _need(pos.dim() == 2, "pos: expected [T, K]")
    T, K = pos.shape
    _vector(pos, "pos", rows, (T, K), torch.int32)
    if w is not None:
        _vector(w, "w", rows, (T, K), torch.float32)
    if residual is not None:
        _matrix(residual, "residual", rows, (T, H), rows.dtype)
    with _On(rows, stream) as s:
        if out is None:
            out = torch.empty((T, H), dtype=rows.dtype, device=rows.device)
        else:
            _matrix(out, "out", rows, (T, H), rows.dtype)
        N.check(N.load().moe_async_merge_rows(_DT[rows.dtype], _p(rows), _ld(rows), R, _p(pos), _p(w), T, K, H,
                                              _p(residual), H if residual is None else _ld(residual), _p(out),
                                              _ld(out), s), "merge_rows")
    return out


def sort_rows_backward(grad_rows, pos, out=None, stream=None):
    """Gradient of sort_rows: grad_x[t] = sum_k grad_rows[pos[t, k]]."""
    return merge_rows(grad_rows, pos, out=out, stream=stream)


def merge_rows_backward(grad, rows, pos, w, out=None, stream=None):
    """Gradients of merge_rows: (grad_rows, grad_w) with grad_rows[pos[t, k]] = w[t, k] grad[t]
    ([R, H] or `out`; rows that no pair names are left as they were) and grad_w[t, k] =
    <rows[pos[t, k]], grad[t]> (fp32, 0 for a pair without a row).  The residual's is `grad`."""
    _first(rows, "rows", _ROWS)
    R, H = rows.shape
    _matrix(rows, "rows", rows, (R, H), rows.dtype)
    _need(pos.dim() == 2, "pos: expected [T, K]")
    T, K = pos.shape
    _vector(pos, "pos", rows, (T, K), torch.int32)
    _vector(w, "w", rows, (T, K), torch.float32)
    _matrix(grad, "grad", rows, (T, H), rows.dtype)
    with _On(rows, stream) as s:
        if out is None:
            out = torch.empty((R, H), dtype=rows.dtype, device=rows.device)
        else:
            _matrix(out, "out", rows, (R, H), rows.dtype)
        grad_w = torch.empty_like(w)
        N.check(N.load().moe_async_merge_rows_backward(_DT[rows.dtype], _p(grad), _ld(grad), _p(rows), _ld(rows), R,
                                                       _p(pos), _p(w), T, K, H, _p(out), _ld(out), _p(grad_w), s),
                "merge_rows_backward")
    return out, grad_w


def route_backward(idx, w, grad_w, num_experts, stream=None):
    """Gradient of route's weights: idx int32 and w fp32 [T, K] as route returned them, grad_w
    fp32 [T, K] -> grad_logits fp32 [T, num_experts]."""
    _first(w, "w", (torch.float32,))
    T, K = w.shape
    _vector(w, "w", w, (T, K), torch.float32)
    _vector(idx, "idx", w, (T, K), torch.int32)
    _vector(grad_w, "grad_w", w, (T, K), torch.float32)
    _need(num_experts >= 1, "num_experts: expected at least 1")
    with _On(w, stream) as s:
        out = torch.empty((T, num_experts), dtype=torch.float32, device=w.device)
        N.check(N.load().moe_async_route_backward(_p(idx), _p(w), _p(grad_w), T, num_experts, K, _p(out), s),
                "route_backward")
    return out


def _norm(x, residual, gain, eps, e4m3, out, out_h, stream):
    _first(x, "x", _ROWS)
    T, H = x.shape
    _matrix(x, "x", x, (T, H), x.dtype)
    if residual is not None:
        _matrix(residual, "residual", x, (T, H), x.dtype)
    if gain is not None:
        _vector(gain, "gain", x, (H,), torch.float32)
    _need(residual is not None or out_h is None, "out_h: there is no sum without a residual")
    dt = torch.float8_e4m3fn if e4m3 else x.dtype
    with _On(x, stream) as s:
        h = x
        if residual is not None:
            h = torch.empty((T, H), dtype=x.dtype, device=x.device) if out_h is None else out_h
            if out_h is not None:
                _matrix(out_h, "out_h", x, (T, H), x.dtype)
        if out is None:
            out = torch.empty((T, H), dtype=dt, device=x.device)
        else:
            _matrix(out, "out", x, (T, H), dt)
        scale = torch.empty(T, dtype=torch.float32, device=x.device) if e4m3 else None
        N.check(N.load().moe_async_add_rms_norm(_DT[x.dtype], _p(x), _ld(x), _p(residual),
                                                H if residual is None else _ld(residual), _p(gain), eps, T, H,
                                                None if residual is None else _p(h), _ld(h), _p(out), _ld(out),
                                                _p(scale), s), "add_rms_norm")
    return out, scale, h


def add_rms_norm(x, residual=None, gain=None, eps=1e-6, out=None, out_h=None, stream=None):
    """(y, h): h = x + residual rounded to their type (x itself without a residual), y = h /
    sqrt(mean(h^2) + eps) * gain.  x, residual [T, H] fp32 or bf16, gain fp32 [H] or None.
    `out_h` may be x or residual."""
    y, _, h = _norm(x, residual, gain, eps, False, out, out_h, stream)
    return y, h


def add_rms_norm_e4m3(x, residual=None, gain=None, eps=1e-6, out=None, out_h=None, stream=None):
    """(q, scale, h): add_rms_norm with y in e4m3, one fp32 scale per row (y = q * scale, scale =
    max(max|y| / 448, 2^-126)): the operands x and x_scale of linear."""
    return _norm(x, residual, gain, eps, True, out, out_h, stream)


def add_rms_norm_backward(grad, h, gain=None, eps=1e-6, grad_h=None, out=None, stream=None):
    """Gradients of add_rms_norm at its h: (grad_x, grad_gain) from grad, the gradient of y, and
    grad_h, the gradient that arrives at h itself (or None).  grad_x is the gradient of x and of
    the residual alike; grad_gain is fp32 [H], None without a gain.  `out` may be `grad_h`."""
    _first(h, "h", _ROWS)
    T, H = h.shape
    _matrix(h, "h", h, (T, H), h.dtype)
    _matrix(grad, "grad", h, (T, H), h.dtype)
    if grad_h is not None:
        _matrix(grad_h, "grad_h", h, (T, H), h.dtype)
    if gain is not None:
        _vector(gain, "gain", h, (H,), torch.float32)
    lib = N.load()
    with _On(h, stream) as s:
        if out is None:
            out = torch.empty((T, H), dtype=h.dtype, device=h.device)
        else:
            _matrix(out, "out", h, (T, H), h.dtype)
        grad_gain = ws = None
        size = 0
        if gain is not None:
            grad_gain = torch.empty_like(gain)
            size = lib.moe_async_add_rms_norm_backward_workspace(T, H)
            ws = torch.empty(size, dtype=torch.uint8, device=h.device)
            if stream is not None:
                ws.record_stream(stream)
        N.check(lib.moe_async_add_rms_norm_backward(_DT[h.dtype], _p(grad), _ld(grad), _p(h), _ld(h), _p(gain), eps, T,
                                                    H, _p(grad_h), H if grad_h is None else _ld(grad_h), _p(out),
                                                    _ld(out), _p(grad_gain), _p(ws), size, s),
                "add_rms_norm_backward")
    return out, grad_gain


def linear(x, weight, bias=None, act="none", mul=None, residual=None, offsets=None, x_scale=None, w_scale=None,
           out_dtype=None, out=None, stream=None):
    """act(x @ weight.T + bias) * mul + residual, products summed in fp32, rounded once.

    x [T, F] and weight [N, F], both bf16, or both e4m3 with x_scale fp32 [T] and w_scale fp32
    [N]; F a multiple of 16 bytes, rows of x and weight on 16-byte boundaries.  bias fp32 [N]; mul
    and residual [T, N] in the type of the result (out's, out_dtype or bf16; fp32 or bf16); act
    "none", "silu", "gelu" (erf) or "relu".  `out` may be mul or residual.
    With offsets (int32 [G + 1], as sort_experts gives them) weight is [G, N, F], bias and w_scale
    are [G, N], and rows offsets[g]:offsets[g + 1] of x meet weight[g]; other rows of `out` are
    left as they were."""
    _first(x, "x", (torch.bfloat16, torch.float8_e4m3fn))
    T, F = x.shape
    _matrix(x, "x", x, (T, F), x.dtype)
    G = 0
    if offsets is None:
        _need(weight.dim() == 2, f"weight: expected [N, {F}], got {tuple(weight.shape)}")
        n, per = weight.shape[0], (weight.shape[0],)
        _matrix(weight, "weight", x, (n, F), x.dtype)
        ldw = _ld(weight)
    else:
        _need(weight.dim() == 3, f"weight: expected [G, N, {F}], got {tuple(weight.shape)}")
        G, n = weight.shape[:2]
        per = (G, n)
        _vector(weight, "weight", x, (G, n, F), x.dtype)
        _vector(offsets, "offsets", x, (G + 1,), torch.int32)
        ldw = F
    _need(act in N.ACTS, f"act: expected one of {tuple(N.ACTS)}, got {act!r}")
    out_dtype = out_dtype if out_dtype is not None else out.dtype if out is not None else torch.bfloat16
    _need(out_dtype in _ROWS, f"out_dtype: expected fp32 or bf16, got {out_dtype}")
    if bias is not None:
        _vector(bias, "bias", x, per, torch.float32)
    e4m3 = x.dtype is torch.float8_e4m3fn
    _need((x_scale is not None) == e4m3 and (w_scale is not None) == e4m3, "x_scale, w_scale: both with e4m3, none with bf16")
    if e4m3:
        _vector(x_scale, "x_scale", x, (T,), torch.float32)
        _vector(w_scale, "w_scale", x, per, torch.float32)
    if mul is not None:
        _matrix(mul, "mul", x, (T, n), out_dtype)
    if residual is not None:
        _matrix(residual, "residual", x, (T, n), out_dtype)
    with _On(x, stream) as s:
        if out is None:
            out = torch.empty((T, n), dtype=out_dtype, device=x.device)
        else:
            _matrix(out, "out", x, (T, n), out_dtype)
        args = N.LinearArgs(_DT[x.dtype], _DT[out_dtype], N.ACTS[act], T, F, n, G, _p(x), _p(weight), _p(bias),
                            _p(x_scale), _p(w_scale), _p(mul), _p(residual), _p(offsets), _p(out), _ld(x), ldw,
                            n if mul is None else _ld(mul), n if residual is None else _ld(residual), _ld(out))
        N.check(N.load().moe_async_linear(ctypes.byref(args), s), "linear")
    return out

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
import struct

import torch

from . import _native as N

_DT = {torch.float32: N.MOE_F32, torch.bfloat16: N.MOE_BF16, torch.float8_e4m3fn: N.MOE_E4M3}
_F32, _BF16, _E4M3, _I32 = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.int32
_ROWS = (_F32, _BF16)
_LINEAR_ARGS = struct.Struct("7i9P5q")           # moe_async_linear_args

# A small call is bound by its host side (a decode step's norm runs 4 us on the GPU), so the
# checks below read each property once and build no message before one is needed.


def _bad(what, t=None):
    if isinstance(t, torch.Tensor):
        what += f"; got {tuple(t.shape)} of {t.dtype} on {t.device}, strides {t.stride()}"
    raise N.MoEError(N.MOE_ERR_INVALID, what)


def _leading(t, name, dtypes):
    """The matrix that names the call's device: (device, rows, width, row stride)."""
    if t.dim() != 2 or t.dtype not in dtypes or not t.is_cuda:
        _bad(f"{name}: expected a CUDA matrix of {dtypes}", t)
    rows, width = t.shape
    return t.get_device(), rows, width, _rows(t, name, t.get_device(), t.dtype, rows, width)


def _rows(t, name, dev, dtype, rows, width):
    """Row stride of a [rows, width] matrix with adjacent columns."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != (rows, width):
        _bad(f"{name}: expected ({rows}, {width}) of {dtype} on cuda:{dev}", t)
    if rows <= 1:
        if width > 1 and t.stride(1) != 1:
            _bad(f"{name}: expected adjacent columns", t)
        return width
    ld, step = t.stride()
    if (step != 1 and width > 1) or ld < width:
        _bad(f"{name}: expected adjacent columns and rows that do not overlap", t)
    return ld


def _whole(t, name, dev, dtype, shape):
    """A contiguous tensor."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _bad(f"{name}: expected contiguous {tuple(shape)} of {dtype} on cuda:{dev}", t)


def _pairs(pos, dev, T=None):
    """K of pos [T, K]."""
    if pos.dim() != 2:
        _bad("pos: expected [T, K]", pos)
    _whole(pos, "pos", dev, _I32, pos.shape if T is None else (T, pos.shape[1]))
    return pos.shape[1]


def _call(fn, what, dev, stream, *args):
    """fn(*args, stream) with the call's device current."""
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _call(fn, what, dev, stream, *args)
    status = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if status:
        raise N.MoEError(status, what)


def sort_experts(expert, num_experts, stream=None):
    """Order of a routed batch's pairs by expert, pairs of one expert in pair order.

    expert int32 [T, K] (ids outside [0, num_experts) get no row) -> (offsets int32 [E + 1]: the
    rows of expert e are offsets[e]:offsets[e + 1]; pos int32 [T, K]: the row of each pair, -1
    without one; pair int32 [T * K]: the pair t * K + k of each row, pairs without one last)."""
    dev, T, K, _ = _leading(expert, "expert", (_I32,))
    if not expert.is_contiguous():
        _bad("expert: expected contiguous", expert)
    if num_experts < 1:
        _bad(f"num_experts: expected at least 1, got {num_experts}")
    d = expert.device
    offsets = torch.empty(num_experts + 1, dtype=_I32, device=d)
    pos, pair = torch.empty_like(expert), torch.empty(T * K, dtype=_I32, device=d)
    _call(N.load().moe_async_sort_experts, "sort_experts", dev, stream, expert.data_ptr(), T, K, num_experts,
          offsets.data_ptr(), pos.data_ptr(), pair.data_ptr())
    return offsets, pos, pair


def sort_rows(x, pos, out=None, stream=None):
    """rows[pos[t, k]] = x[t]: x [T, H] fp32 or bf16, pos int32 [T, K] -> rows [T * K, H] (or
    `out` [R, H]); rows that no pair names are left as they were."""
    dev, T, H, ldx = _leading(x, "x", _ROWS)
    K = _pairs(pos, dev, T)
    if out is None:
        R, ldo = T * K, H
        out = torch.empty((R, H), dtype=x.dtype, device=x.device)
    else:
        R = out.shape[0]
        ldo = _rows(out, "out", dev, x.dtype, R, H)
    _call(N.load().moe_async_sort_rows, "sort_rows", dev, stream, _DT[x.dtype], x.data_ptr(), ldx, pos.data_ptr(), T, K,
          H, out.data_ptr(), ldo, R)
    return out


def merge_rows(rows, pos, w=None, residual=None, out=None, stream=None):
    """y[t] = sum_k w[t, k] rows[pos[t, k]] + residual[t] in fp32, ascending k, rounded once:
    rows [R, H], pos int32 [T, K], w fp32 [T, K] (None: plain sums), residual [T, H] or None ->
    y [T, H].  A pair without a row (pos outside [0, R)) adds nothing.  `out` may be `residual`."""
    dev, R, H, ldr = _leading(rows, "rows", _ROWS)
    dt = rows.dtype
    K = _pairs(pos, dev)
    T = pos.shape[0]
    if w is not None:
        _whole(w, "w", dev, _F32, (T, K))
    ldres = H if residual is None else _rows(residual, "residual", dev, dt, T, H)
    if out is None:
        ldo = H
        out = torch.empty((T, H), dtype=dt, device=rows.device)
    else:
        ldo = _rows(out, "out", dev, dt, T, H)
    _call(N.load().moe_async_merge_rows, "merge_rows", dev, stream, _DT[dt], rows.data_ptr(), ldr, R, pos.data_ptr(),
          None if w is None else w.data_ptr(), T, K, H, None if residual is None else residual.data_ptr(), ldres,
          out.data_ptr(), ldo)
    return out


def sort_rows_backward(grad_rows, pos, out=None, stream=None):
    """Gradient of sort_rows: grad_x[t] = sum_k grad_rows[pos[t, k]]."""
    return merge_rows(grad_rows, pos, out=out, stream=stream)


def merge_rows_backward(grad, rows, pos, w, out=None, stream=None):
    """Gradients of merge_rows: (grad_rows, grad_w) with grad_rows[pos[t, k]] = w[t, k] grad[t]
    ([R, H] or `out`; rows that no pair names are left as they were) and grad_w[t, k] =
    <rows[pos[t, k]], grad[t]> (fp32, 0 for a pair without a row).  The residual's is `grad`."""
    dev, R, H, ldr = _leading(rows, "rows", _ROWS)
    dt = rows.dtype
    K = _pairs(pos, dev)
    T = pos.shape[0]
    _whole(w, "w", dev, _F32, (T, K))
    ldg = _rows(grad, "grad", dev, dt, T, H)
    if out is None:
        ldo = H
        out = torch.empty((R, H), dtype=dt, device=rows.device)
    else:
        ldo = _rows(out, "out", dev, dt, R, H)
    grad_w = torch.empty_like(w)
    _call(N.load().moe_async_merge_rows_backward, "merge_rows_backward", dev, stream, _DT[dt], grad.data_ptr(), ldg,
          rows.data_ptr(), ldr, R, pos.data_ptr(), w.data_ptr(), T, K, H, out.data_ptr(), ldo, grad_w.data_ptr())
    return out, grad_w


def route_backward(idx, w, grad_w, num_experts, stream=None):
    """Gradient of route's weights: idx int32 and w fp32 [T, K] as route returned them, grad_w
    fp32 [T, K] -> grad_logits fp32 [T, num_experts]."""
    dev, T, K, _ = _leading(w, "w", (_F32,))
    _whole(w, "w", dev, _F32, (T, K))
    _whole(idx, "idx", dev, _I32, (T, K))
    _whole(grad_w, "grad_w", dev, _F32, (T, K))
    if num_experts < 1:
        _bad(f"num_experts: expected at least 1, got {num_experts}")
    out = torch.empty((T, num_experts), dtype=_F32, device=w.device)
    _call(N.load().moe_async_route_backward, "route_backward", dev, stream, idx.data_ptr(), w.data_ptr(),
          grad_w.data_ptr(), T, num_experts, K, out.data_ptr())
    return out


def _norm(x, residual, gain, eps, e4m3, out, out_h, stream):
    dev, T, H, ldx = _leading(x, "x", _ROWS)
    dt, d = x.dtype, x.device
    if gain is not None:
        _whole(gain, "gain", dev, _F32, (H,))
    h, ldr, ldh = x, H, H
    if residual is not None:
        ldr = _rows(residual, "residual", dev, dt, T, H)
        if out_h is None:
            h = torch.empty((T, H), dtype=dt, device=d)
        else:
            h, ldh = out_h, _rows(out_h, "out_h", dev, dt, T, H)
    elif out_h is not None:
        _bad("out_h: there is no sum without a residual")
    if out is None:
        ldo = H
        out = torch.empty((T, H), dtype=_E4M3 if e4m3 else dt, device=d)
    else:
        ldo = _rows(out, "out", dev, _E4M3 if e4m3 else dt, T, H)
    scale = torch.empty(T, dtype=_F32, device=d) if e4m3 else None
    _call(N.load().moe_async_add_rms_norm, "add_rms_norm", dev, stream, _DT[dt], x.data_ptr(), ldx,
          None if residual is None else residual.data_ptr(), ldr, None if gain is None else gain.data_ptr(), eps, T, H,
          None if residual is None else h.data_ptr(), ldh, out.data_ptr(), ldo, scale.data_ptr() if e4m3 else None)
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
    dev, T, H, ldh = _leading(h, "h", _ROWS)
    dt, d = h.dtype, h.device
    ldg = _rows(grad, "grad", dev, dt, T, H)
    ldgh = H if grad_h is None else _rows(grad_h, "grad_h", dev, dt, T, H)
    if out is None:
        ldo = H
        out = torch.empty((T, H), dtype=dt, device=d)
    else:
        ldo = _rows(out, "out", dev, dt, T, H)
    lib = N.load()
    grad_gain = ws = None
    size = 0
    if gain is not None:
        _whole(gain, "gain", dev, _F32, (H,))
        grad_gain = torch.empty_like(gain)
        size = lib.moe_async_add_rms_norm_backward_workspace(T, H)
        ws = torch.empty(size, dtype=torch.uint8, device=d)
        if stream is not None:
            ws.record_stream(stream)             # freed below, while the call may still run there
    _call(lib.moe_async_add_rms_norm_backward, "add_rms_norm_backward", dev, stream, _DT[dt], grad.data_ptr(), ldg,
          h.data_ptr(), ldh, None if gain is None else gain.data_ptr(), eps, T, H,
          None if grad_h is None else grad_h.data_ptr(), ldgh, out.data_ptr(), ldo,
          None if gain is None else grad_gain.data_ptr(), None if ws is None else ws.data_ptr(), size)
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
    dev, T, F, ldx = _leading(x, "x", (_BF16, _E4M3))
    dt = x.dtype
    G, po = 0, 0
    if offsets is None:
        if weight.dim() != 2:
            _bad(f"weight: expected [N, {F}]", weight)
        n = weight.shape[0]
        per = (n,)
        ldw = _rows(weight, "weight", dev, dt, n, F)
    else:
        if weight.dim() != 3:
            _bad(f"weight: expected [G, N, {F}]", weight)
        per = weight.shape[:2]
        G, n = per
        if G < 1:
            _bad("weight: expected at least one group", weight)
        _whole(weight, "weight", dev, dt, (G, n, F))
        _whole(offsets, "offsets", dev, _I32, (G + 1,))
        ldw, po = F, offsets.data_ptr()
    code = N.ACTS.get(act)
    if code is None:
        _bad(f"act: expected one of {tuple(N.ACTS)}, got {act!r}")
    if out_dtype is None:
        out_dtype = _BF16 if out is None else out.dtype
    if out_dtype not in _ROWS:
        _bad(f"out_dtype: expected fp32 or bf16, got {out_dtype}")
    psx = psw = pb = pm = pr = 0
    ldm = ldr = ldo = n
    if dt is _E4M3:
        if x_scale is None or w_scale is None:
            _bad("x_scale, w_scale: both are needed with e4m3")
        _whole(x_scale, "x_scale", dev, _F32, (T,))
        _whole(w_scale, "w_scale", dev, _F32, per)
        psx, psw = x_scale.data_ptr(), w_scale.data_ptr()
    elif x_scale is not None or w_scale is not None:
        _bad("x_scale, w_scale: bf16 operands have none")
    if bias is not None:
        _whole(bias, "bias", dev, _F32, per)
        pb = bias.data_ptr()
    if mul is not None:
        ldm, pm = _rows(mul, "mul", dev, out_dtype, T, n), mul.data_ptr()
    if residual is not None:
        ldr, pr = _rows(residual, "residual", dev, out_dtype, T, n), residual.data_ptr()
    if out is None:
        out = torch.empty((T, n), dtype=out_dtype, device=x.device)
    else:
        ldo = _rows(out, "out", dev, out_dtype, T, n)
    _call(N.load().moe_async_linear, "linear", dev, stream,
          _LINEAR_ARGS.pack(_DT[dt], _DT[out_dtype], code, T, F, n, G, x.data_ptr(), weight.data_ptr(), pb, psx, psw, pm,
                            pr, po, out.data_ptr(), ldx, ldw, ldm, ldr, ldo))
    return out


def ops_sync(device=None, stream=None):
    """Wait for `stream` (default: the device's current one) and raise MoEError if a stateless
    operator found an error on the device (a wait in linear that exceeded its bound)."""
    dev = torch.cuda.current_device() if device is None else torch.device(device).index
    _call(N.load().moe_async_ops_status, "ops_sync", dev, stream)

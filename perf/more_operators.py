"""The experts' products in training and in 8 bits with block scales, as a user's program calls them, and their plain forms.

Four operators: the gradients of the product, dense and per expert (`grad`: of the rows, the weights and the bias), the product of
e4m3 operands with a scale per 128 columns of a token and per 128 x 128 block of a weight (`blocks`), the quantiser that makes such
operands (`quantize`), and the gradient of the product's epilogue act(z) * mul (`act`).  Sizes are those of the layers in
workloads/configs.py (GPT-OSS: 2880 x 2880; DeepSeek-wide: 7168 x 2048, in 32-expert slices; the ragged test layers), or generic.
"""
import math

import torch

own = False

ACTS = ("none", "silu", "gelu", "relu")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
BLOCK = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -126           # smallest scale: a block of zeros has this one


def _grad(name, rows, fan_in, fan_out, groups=0, weight="f32", bias=False, add=False, drop=0.0):
    return {"name": name, "op": "grad", "rows": rows, "fan_in": fan_in, "fan_out": fan_out, "groups": groups, "weight": weight, "bias": bias,
            "add": add, "drop": drop}


def _blocks(name, rows, fan_in, fan_out, groups=0, out="bf16", act="none", bias=False, mul=False, residual=False, drop=0.0):
    return {"name": name, "op": "blocks", "rows": rows, "fan_in": fan_in, "fan_out": fan_out, "groups": groups, "out": out, "act": act, "bias": bias,
            "mul": mul, "residual": residual, "drop": drop}


def _quantize(name, rows, width, dtype="bf16", kind="rows", groups=0):
    return {"name": name, "op": "quantize", "rows": rows, "width": width, "dtype": dtype, "kind": kind, "groups": groups}


def _act(name, rows, width, act="silu", dtype="bf16", mul=True):
    return {"name": name, "op": "act", "rows": rows, "width": width, "act": act, "dtype": dtype, "mul": mul}


def listed():
    return [
        # a training step through the product of 32 GPT-OSS experts on sorted rows, weights' gradients kept in fp32
        _grad("grad_experts", 8192, 2880, 2880, groups=32),
        # the same through the down projection of a DeepSeek-wide slice, added to what earlier micro-batches left
        _grad("grad_wide_add", 4096, 2048, 7168, groups=32, weight="bf16", add=True),
        # the router's product: a long sum of few outputs
        _grad("grad_router", 2048, 7168, 256, bias=True),
        # one rank's share of a small ragged layer, some rows of no expert, outputs of an odd width
        _grad("grad_ragged", 200, 584, 997, groups=16, weight="bf16", bias=True, drop=0.25),
        # a decode step's projection
        _blocks("blocks_decode", 4, 7168, 2048, bias=True),
        # a decode step's experts: a few tokens each, the weights' bytes count
        _blocks("blocks_decode_experts", 64, 7168, 2048, groups=32),
        # a prefill chunk's projection into the residual stream
        _blocks("blocks_prefill", 4096, 7168, 7168, residual=True),
        # the gate product of a prefill chunk's experts
        _blocks("blocks_experts", 8192, 7168, 2048, groups=32, act="silu", mul=True),
        # a prefill chunk's rows on their way into 8-bit products
        _quantize("quantize_prefill", 4096, 7168),
        # a checkpoint's matrices on their way into memory
        _quantize("quantize_weights", 2048, 7168, kind="weights", groups=8),
        # the gradient of the gate of the experts' SwiGLU
        _act("act_experts", 8192, 2880),
        # a small layer's, odd rows
        _act("act_small", 99, 137, "gelu", "f32"),
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm; one in three as it comes, the others a multiple of 16."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v > 48 and rng.random() < 0.67:
        v = v // 16 * 16
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(("grad", "grad", "blocks", "blocks", "quantize", "act"))
    if op == "quantize":
        kind = rng.choice(("rows", "rows", "weights"))
        return {"op": op, "rows": _size(rng, 1, 4096), "width": 16 * max(1, _size(rng, 64, 7168) // 16), "dtype": rng.choice(("bf16", "bf16", "f32")), "kind": kind,
                "groups": rng.choice((0, 2, 5)) if kind == "weights" else 0}
    if op == "act":
        return {"op": op, "rows": _size(rng, 1, 8192), "width": _size(rng, 8, 2880), "act": rng.choice(ACTS), "dtype": rng.choice(("bf16", "bf16", "f32")),
                "mul": rng.random() < 0.7}
    groups = rng.choice((0, 0, _size(rng, 2, 64)))
    fan_out = _size(rng, 8, 7168)
    if op == "grad":
        fan_in = 8 * max(2, _size(rng, 16, 7168) // 8)
        if groups:
            fan_out = max(1, min(fan_out, 32 * 2880 * 2880 // (groups * fan_in)))
        most = 8192 * 2880 * 2880 // (fan_in * fan_out)
        return {"op": op, "rows": _size(rng, 1, max(1, min(8192, most))), "fan_in": fan_in, "fan_out": fan_out, "groups": groups,
                "weight": rng.choice(("f32", "bf16")), "bias": rng.random() < 0.4, "add": rng.random() < 0.3, "drop": rng.choice((0.0, 0.3)) if groups else 0.0}
    fan_in = 16 * max(1, _size(rng, 64, 7168) // 16)
    if groups:
        fan_out = max(1, min(fan_out, 32 * 7168 * 2048 // (groups * fan_in)))
    return {"op": op, "rows": _size(rng, 1, 4096), "fan_in": fan_in, "fan_out": fan_out, "groups": groups, "out": rng.choice(("bf16", "bf16", "f32")),
            "act": rng.choice(ACTS), "bias": rng.random() < 0.4, "mul": rng.random() < 0.3, "residual": rng.random() < 0.4,
            "drop": rng.choice((0.0, 0.3)) if groups else 0.0}


# ------------------------------------------------------------------ inputs


def _randn(shape, g, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _groups(c, g):
    """Sorted rows' offsets, and for the plain form each row's group and its place there (rows of no group lie behind the last)."""
    G, T = c["groups"], c["rows"]
    share = torch.softmax(0.5 * torch.randn(G, generator=g, device="cuda"), 0)      # a router trained for balance
    of = torch.multinomial(share, T, replacement=True, generator=g)
    n = torch.bincount(of[torch.rand(T, generator=g, device="cuda") >= c["drop"]], minlength=G)
    ends = n.cumsum(0)
    offsets = torch.cat([n.new_zeros(1), ends])
    live = int(offsets[-1])
    row = torch.arange(live, device="cuda")
    of = torch.searchsorted(ends, row, right=True)
    return offsets.to(torch.int32), of, row - offsets[of], max(1, int(n.max()))


def _blocked(t, rows):
    """A matrix (or several) padded to whole blocks of `rows` x 128, as [.., row blocks, rows, column blocks, 128]."""
    n, f = t.shape[-2:]
    t = torch.nn.functional.pad(t, (0, -f % BLOCK, 0, -n % rows))
    return t.reshape(*t.shape[:-2], t.shape[-2] // rows, rows, t.shape[-1] // BLOCK, BLOCK)


def _quantise(t, rows):
    """e4m3 and its scales per rows x 128, as the quantiser or a checkpoint gives them: scales [.., row blocks, column blocks]."""
    n, f = t.shape[-2:]
    v = _blocked(t.float(), rows)
    s = (v.abs().amax((-3, -1)) / E4M3_MAX).clamp(min=TINY)
    q = (v / s[..., :, None, :, None]).flatten(-4, -3).flatten(-2)[..., :n, :f]
    return q.to(torch.float8_e4m3fn).contiguous(), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, s = case, dict(case)
    T = c["rows"]
    s["offsets"] = None
    if c["op"] in ("grad", "blocks"):
        F, N, G = c["fan_in"], c["fan_out"], c["groups"]
        if G:
            s["offsets"], s["of"], s["at"], s["most"] = _groups(c, g)
    if c["op"] == "grad":
        s["x"], s["grad"] = _randn((T, F), g, torch.bfloat16), _randn((T, N), g, torch.bfloat16)
        s["w"] = _randn((G, N, F) if G else (N, F), g, torch.bfloat16, 1 / math.sqrt(F))
        s["grad_x"] = torch.zeros((T, F), dtype=torch.bfloat16, device="cuda")     # rows of no group stay zero
        s["residual"] = _randn((T, F), g, torch.bfloat16) if c["add"] else None    # what reaches the rows another way
        s["sum_w"] = s["sum_b"] = None
        if c["add"]:                                                               # what earlier micro-batches left, added to in place
            s["sum_w"] = _randn((G, N, F) if G else (N, F), g, DT[c["weight"]])
            s["sum_b"] = torch.randn((G, N) if G else (N,), generator=g, device="cuda") if c["bias"] else None
    elif c["op"] == "blocks":
        s["x"], sx = _quantise(_randn((T, F), g, torch.float32) * torch.exp(torch.randn((T, 1), generator=g, device="cuda")), 1)
        s["x_scale"] = sx.t().contiguous().t()                                     # tokens adjacent, as the quantiser leaves them
        s["w"], s["w_scale"] = _quantise(_randn((G, N, F) if G else (N, F), g, torch.float32, 1 / math.sqrt(F)), BLOCK)
        out = DT[c["out"]]
        s["bias_v"] = torch.randn((G, N) if G else (N,), generator=g, device="cuda") if c["bias"] else None
        s["mul_v"] = _randn((T, N), g, out) if c["mul"] else None
        s["residual_v"] = _randn((T, N), g, out) if c["residual"] else None
        s["y"] = torch.zeros((T, N), dtype=out, device="cuda")                     # rows of no group stay zero
    elif c["op"] == "quantize":
        shape = (c["groups"], T, c["width"]) if c["groups"] else (T, c["width"])
        v = _randn(shape, g, torch.float32) * torch.exp(torch.randn((*shape[:-1], 1), generator=g, device="cuda"))
        s["x"] = v.to(DT[c["dtype"]])
    else:
        dt = DT[c["dtype"]]
        s["grad"], s["z"] = _randn((T, c["width"]), g, dt), _randn((T, c["width"]), g, dt, 2.0)
        s["mul_v"] = _randn((T, c["width"]), g, dt) if c["mul"] else None
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    if own:
        return _run_own(s)
    return {"grad": _grad_plain, "blocks": _blocks_plain, "quantize": _quantize_plain, "act": _act_plain}[s["op"]](s)


def _run_own(s):
    import asynchronous_expert_execution_gb300 as moe
    if s["op"] == "grad":
        grad_x, grad_w, grad_b = moe.linear_backward(s["grad"], s["x"], s["w"], offsets=s["offsets"], bias=s["bias"], residual=s["residual"],
                                                     weight_dtype=DT[s["weight"]], out_x=s["grad_x"], out_weight=s["sum_w"], out_bias=s["sum_b"],
                                                     accumulate=s["add"])
        return {"grad_x": grad_x, "grad_w": grad_w, "grad_b": grad_b} if s["bias"] else {"grad_x": grad_x, "grad_w": grad_w}
    if s["op"] == "blocks":
        return moe.linear(s["x"], s["w"], s["bias_v"], act=s["act"], mul=s["mul_v"], residual=s["residual_v"], offsets=s["offsets"], x_scale=s["x_scale"],
                          w_scale=s["w_scale"], out=s["y"])
    if s["op"] == "quantize":
        q, scale = moe.quantize_blocks(s["x"]) if s["kind"] == "rows" else moe.quantize_weight_blocks(s["x"])
        return {"q": q, "scale": scale}
    grad_z, grad_mul = moe.act_mul_backward(s["grad"], s["z"], s["mul_v"], act=s["act"])
    return {"grad_z": grad_z, "grad_mul": grad_mul} if s["mul"] else grad_z


def _per_group(s, rows):
    """Sorted rows as [group, place, width], zeros behind each group's last."""
    t = rows.new_zeros((s["groups"], s["most"], rows.shape[1]))
    t[s["of"], s["at"]] = rows[:s["of"].numel()]
    return t


def _grad_plain(s):
    grad, x, w = s["grad"].float(), s["x"].float(), s["w"].float()
    if s["groups"]:
        grad, x = _per_group(s, grad), _per_group(s, x)
    gx, gw, gb = grad @ w, grad.mT @ x, grad.sum(-2)
    if s["groups"]:
        gx = gx[s["of"], s["at"]]
    live = gx.shape[0]
    if s["add"]:
        gx = gx + s["residual"][:live].float()
        gw = s["sum_w"].copy_(gw + s["sum_w"].float())
        gb = s["sum_b"].add_(gb) if s["bias"] else gb
    s["grad_x"][:live] = gx.to(torch.bfloat16)
    gw = gw.to(DT[s["weight"]])
    return {"grad_x": s["grad_x"], "grad_w": gw, "grad_b": gb} if s["bias"] else {"grad_x": s["grad_x"], "grad_w": gw}


def _act_of(v, act):
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    return v.clamp(min=0) if act == "relu" else v


def _spread(scale, rows, shape):
    """Scales per rows x 128 as a matrix of `shape`."""
    t = scale.repeat_interleave(BLOCK, -1)[..., :shape[-1]]
    return t if rows == 1 else t.repeat_interleave(rows, -2)[..., :shape[-2], :]


def _blocks_plain(s):
    x = s["x"].float() * _spread(s["x_scale"], 1, s["x"].shape)
    w = s["w"].float() * _spread(s["w_scale"], BLOCK, s["w"].shape)
    v = (_per_group(s, x) if s["groups"] else x) @ w.mT
    if s["bias"]:
        v = v + (s["bias_v"][:, None] if s["groups"] else s["bias_v"])
    if s["groups"]:
        v = v[s["of"], s["at"]]
    v, live = _act_of(v, s["act"]), v.shape[0]
    if s["mul"]:
        v = v * s["mul_v"][:live].float()
    if s["residual"]:
        v = v + s["residual_v"][:live].float()
    s["y"][:live] = v.to(s["y"].dtype)
    return s["y"]


def _quantize_plain(s):
    rows = 1 if s["kind"] == "rows" else BLOCK
    q, scale = _quantise(s["x"], rows)
    return {"q": q, "scale": scale}


def _act_plain(s):
    grad, z, act = s["grad"].float(), s["z"].float(), s["act"]
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        slope = p * (1.0 + z * (1.0 - p))
    elif act == "gelu":
        slope = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    else:
        slope = (z > 0).float() if act == "relu" else torch.ones_like(z)
    dt = s["z"].dtype
    if not s["mul"]:
        return (grad * slope).to(dt)
    return {"grad_z": (grad * s["mul_v"].float() * slope).to(dt), "grad_mul": (grad * _act_of(z, act)).to(dt)}


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    c, T = case, case["rows"]
    if c["op"] == "quantize":
        n = max(1, c["groups"]) * T * c["width"]
        per = BLOCK if c["kind"] == "rows" else BLOCK * BLOCK
        return {"bytes": n * SIZE[c["dtype"]] + n + 4 * n / per, "flops": 2.0 * n}
    if c["op"] == "act":
        return {"bytes": T * c["width"] * SIZE[c["dtype"]] * (5 if c["mul"] else 3), "flops": 10.0 * T * c["width"]}
    F, N, G = c["fan_in"], c["fan_out"], c["groups"]
    live = T * (1.0 - c["drop"])
    used = max(1, min(G, live))                       # weights of experts without a row are not read
    if c["op"] == "grad":
        moved = live * (N + F) * 2 + used * N * F * 2 + live * F * 2 * (1 + c["add"]) + max(1, G) * N * F * SIZE[c["weight"]] * (1 + c["add"])
        return {"bytes": moved + 4 * max(1, G) * N * c["bias"] * (1 + c["add"]), "flops": 4.0 * live * F * N}
    moved = live * F + used * N * F + 4 * (live + used * math.ceil(N / BLOCK)) * math.ceil(F / BLOCK)
    moved += live * N * SIZE[c["out"]] * (1 + c["mul"] + c["residual"]) + 4 * N * max(1, G) * c["bias"]
    return {"bytes": moved, "flops": 2.0 * live * F * N}


# ------------------------------------------------------------------ the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    d = lambda t: None if t is None else t.double()  # noqa: E731
    if s["op"] == "quantize":
        x, rows = d(s["x"]), 1 if s["kind"] == "rows" else BLOCK
        n, f = x.shape[-2:]
        scale = torch.zeros((*x.shape[:-2], -(-n // rows), -(-f // BLOCK)), dtype=torch.float64, device="cuda")
        q = torch.empty_like(x)
        for b in range(scale.shape[-1]):
            part = x[..., b * BLOCK:(b + 1) * BLOCK]
            most = part.abs().amax(-1)
            if rows > 1:
                most = torch.stack([m.amax(-1) for m in most.split(rows, -1)], -1)
            scale[..., b] = (most / E4M3_MAX).clamp(min=TINY)
            per_row = scale[..., b] if rows == 1 else scale[..., b].repeat_interleave(rows, -1)[..., :n]
            q[..., b * BLOCK:(b + 1) * BLOCK] = part / per_row[..., None]
        return {"q": q, "scale": scale}
    if s["op"] == "act":
        grad, z, m = d(s["grad"]), d(s["z"]), d(s["mul_v"])
        if s["act"] == "silu":
            y, slope = z * torch.sigmoid(z), torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
        elif s["act"] == "gelu":
            cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
            y, slope = z * cdf, cdf + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
        elif s["act"] == "relu":
            y, slope = torch.maximum(z, torch.zeros_like(z)), torch.where(z > 0, 1.0, 0.0).double()
        else:
            y, slope = z, torch.ones_like(z)
        return grad * slope if m is None else {"grad_z": grad * m * slope, "grad_mul": grad * y}
    T, F, N, G = s["rows"], s["fan_in"], s["fan_out"], s["groups"]
    if T * F * N > 3e11:
        return None
    at = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    if s["op"] == "grad":
        gx = d(s["grad_x"]).clone()
        gw = torch.zeros((len(at) - 1, N, F), dtype=torch.float64, device="cuda")
        gb = torch.zeros((len(at) - 1, N), dtype=torch.float64, device="cuda")
        for e in range(len(at) - 1):
            rows = slice(at[e], at[e + 1])
            grad, w = d(s["grad"][rows]), d(s["w"][e] if G else s["w"])
            gx[rows] = torch.einsum("tn,nf->tf", grad, w)
            gw[e] = torch.einsum("tn,tf->nf", grad, d(s["x"][rows]))
            gb[e] = grad.sum(0)
            if s["add"]:
                gx[rows] += d(s["residual"][rows])
        gw, gb = (gw, gb) if G else (gw[0], gb[0])
        if s["add"]:
            gw += s["sum_w"]
            gb = gb + s["sum_b"] if s["bias"] else gb
        return {"grad_x": gx, "grad_w": gw, "grad_b": gb} if s["bias"] else {"grad_x": gx, "grad_w": gw}
    y = d(s["y"]).clone()
    for e in range(len(at) - 1):
        rows = slice(at[e], at[e + 1])
        x, w = d(s["x"][rows]), d(s["w"][e] if G else s["w"])
        sx, sw = d(s["x_scale"][rows]), d(s["w_scale"][e] if G else s["w_scale"])
        n = torch.arange(N, device="cuda") // BLOCK
        k = torch.arange(F, device="cuda") // BLOCK
        v = torch.einsum("tf,nf->tn", x * sx[:, k], w * sw[n][:, k])
        if s["bias"]:
            v = v + d(s["bias_v"][e] if G else s["bias_v"])
        if s["act"] == "silu":
            v = v * torch.sigmoid(v)
        elif s["act"] == "gelu":
            v = v * 0.5 * torch.erfc(-v / math.sqrt(2.0))
        elif s["act"] == "relu":
            v = torch.maximum(v, torch.zeros_like(v))
        if s["mul"]:
            v = v * d(s["mul_v"][rows])
        if s["residual"]:
            v = v + d(s["residual_v"][rows])
        y[rows] = v
    return y

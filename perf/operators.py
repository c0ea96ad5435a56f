"""The stateless operators around the expert path, as a user's program calls them, and their plain forms.

Four of them: tokens sorted by expert and merged back (`dispatch`, forward and backward), the root-mean-square norm with
the residual's addition (`norm`: bf16 / fp32, e4m3 with a scale per row, backward), the matrix product with its epilogue
(`linear`: dense, e4m3, and per expert on sorted rows).  Sizes are those of the layers in workloads/configs.py
(GPT-OSS decode and prefill: 128 experts, top-4, 2880; DeepSeek-wide: 256 experts, top-8, 7168 x 2048; its 32-expert
slices; the ragged test layers), or generic.
"""
import math

import torch

own = False

ACTS = ("none", "silu", "gelu", "relu")
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0
TINY = 2.0 ** -126           # smallest scale: a row of zeros has this one
EPS = 1e-6


def _dispatch(name, direction, tokens, top_k, experts, hidden, dtype="bf16", drop=0.0, skew=0.0):
    return {"name": name, "op": "dispatch", "direction": direction, "tokens": tokens, "top_k": top_k, "experts": experts,
            "hidden": hidden, "dtype": dtype, "drop": drop, "skew": skew}


def _norm(name, direction, tokens, hidden, dtype="bf16", residual=True):
    return {"name": name, "op": "norm", "direction": direction, "tokens": tokens, "hidden": hidden, "dtype": dtype, "residual": residual}


def _linear(name, tokens, fan_in, fan_out, dtype="bf16", out="bf16", act="none", bias=False, mul=False, residual=False, groups=0, drop=0.0):
    return {"name": name, "op": "linear", "tokens": tokens, "fan_in": fan_in, "fan_out": fan_out, "dtype": dtype, "out": out, "act": act,
            "bias": bias, "mul": mul, "residual": residual, "groups": groups, "drop": drop}


def listed():
    return [
        # a decode step of the GPT-OSS layer: one token per request, where launches count
        _dispatch("dispatch_decode", "forward", 64, 4, 128, 2880),
        # the skewed prefill chunk: a few experts take most of the tokens
        _dispatch("dispatch_prefill_zipf", "forward", 4096, 4, 128, 2880, skew=1.2),
        # a training step's backward pass through the DeepSeek-wide layer's routing
        _dispatch("dispatch_wide_backward", "backward", 2048, 8, 256, 7168),
        # one rank's share of a small fp32 layer: a quarter of the pairs belong to other ranks
        _dispatch("dispatch_f32_backward", "backward", 999, 3, 12, 137, "f32", drop=0.25),
        # the norm before a decode step's layer
        _norm("norm_decode", "forward", 16, 7168),
        # the norm of a prefill chunk whose products run in 8 bits
        _norm("norm_prefill_e4m3", "e4m3", 4096, 7168),
        # a training step's backward pass through the norm
        _norm("norm_backward", "backward", 8192, 2880),
        # the projection of a decode step: its weights are read for four tokens
        _linear("linear_decode", 4, 2880, 2880, bias=True, residual=True),
        # router logits in fp32: many tokens, few outputs
        _linear("linear_router", 2048, 7168, 256, out="f32", bias=True),
        # an odd batch through a ragged layer's gate
        _linear("linear_ragged_gate", 777, 584, 997, act="silu", mul=True),
        # a prefill chunk's projection in 8 bits
        _linear("linear_prefill_e4m3", 4096, 7168, 7168, "e4m3", bias=True, residual=True),
        # the gate product of 32 GPT-OSS experts on sorted rows
        _linear("linear_experts", 8192, 2880, 2880, act="silu", mul=True, groups=32),
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm; one in three as it comes, the others a multiple of 16."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v > 48 and rng.random() < 0.67:
        v = v // 16 * 16
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(("dispatch", "norm", "linear"))
    if op == "dispatch":
        experts = _size(rng, 4, 256)
        top_k = rng.randint(1, min(8, experts))
        hidden = _size(rng, 64, 7168)
        dtype = rng.choice(("bf16", "bf16", "f32"))
        tokens = _size(rng, 1, max(1, min(8192, 2048 * 8 * 7168 * 2 // (max(2, top_k) * hidden * SIZE[dtype] * 5 // 4))))
        return {"op": op, "direction": rng.choice(("forward", "backward")), "tokens": tokens, "top_k": top_k, "experts": experts, "hidden": hidden,
                "dtype": dtype, "drop": rng.choice((0.0, 0.0, 0.25, 0.9)), "skew": rng.choice((0.0, 1.2))}
    if op == "norm":
        hidden = _size(rng, 64, 7168)
        return {"op": op, "direction": rng.choice(("forward", "e4m3", "backward")), "tokens": _size(rng, 1, 8192 if hidden <= 2880 else 4096),
                "hidden": hidden, "dtype": rng.choice(("bf16", "bf16", "f32")), "residual": rng.random() < 0.7}
    dtype = rng.choice(("bf16", "bf16", "e4m3"))
    fan_in = 16 * max(4, _size(rng, 64, 7168) // 16)
    fan_out = _size(rng, 8, 7168)
    groups = rng.choice((0, 0, _size(rng, 2, 64)))
    if groups:
        fan_out = min(fan_out, 2880, 32 * 2880 * 2880 // (groups * fan_in))
    return {"op": op, "tokens": _size(rng, 1, 4096), "fan_in": fan_in, "fan_out": fan_out, "dtype": dtype, "out": rng.choice(("bf16", "bf16", "f32")),
            "act": rng.choice(ACTS), "bias": rng.random() < 0.5, "mul": rng.random() < 0.3, "residual": rng.random() < 0.4, "groups": groups,
            "drop": rng.choice((0.0, 0.3)) if groups else 0.0}


# ------------------------------------------------------------------ inputs


def _route(c, g):
    """Router logits and their top-k choice with renormalised weights, as the forward pass left them; the expert ids with the
    pairs of other ranks marked -1; and the sorted order of those ids."""
    T, K, E = c["tokens"], c["top_k"], c["experts"]
    logits = torch.randn((T, E), generator=g, device="cuda")
    if c["skew"]:                                    # log of a Zipf popularity, in a random order of the experts
        order = torch.randperm(E, generator=g, device="cuda")
        logits = logits - c["skew"] * torch.log1p(order.float())
    top, idx = torch.topk(logits, K, dim=1)
    w = torch.softmax(top, dim=1)
    away = torch.rand((T, K), generator=g, device="cuda") < c["drop"]
    expert = torch.where(away, -1, idx).to(torch.int32)
    return idx.to(torch.int32).contiguous(), w.contiguous(), expert.contiguous()


def _order(expert, E):
    flat = expert.reshape(-1).long()
    here = (flat >= 0) & (flat < E)
    key = torch.where(here, flat, E)
    key, pair = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=key.device))
    pos = torch.empty_like(flat)
    pos[pair] = torch.arange(flat.numel(), device=key.device)
    pos = torch.where(here, pos, -1).reshape(expert.shape)
    return offsets.to(torch.int32), pos.to(torch.int32), pair.to(torch.int32)


def _randn(shape, g, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _quantise(x):
    """Rows in e4m3 and their scales, as the 8-bit norm or a checkpoint gives them."""
    s = x.abs().amax(-1) / E4M3_MAX
    return (x / s[..., None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, s = case, dict(case)
    if c["op"] == "dispatch":
        T, K, H, dt = c["tokens"], c["top_k"], c["hidden"], DT[c["dtype"]]
        s["idx"], s["w"], s["expert"] = _route(c, g)
        s["ys"] = _randn((T * K, H), g, dt)
        s["rows"] = torch.zeros((T * K, H), dtype=dt, device="cuda")      # rows behind the last pair stay zero
        if c["direction"] == "forward":
            s["x"], s["residual"] = _randn((T, H), g, dt), _randn((T, H), g, dt)
        else:
            s["offsets"], s["pos"], s["pair"] = _order(s["expert"], c["experts"])
            s["grad"], s["grad_rows"] = _randn((T, H), g, dt), _randn((T * K, H), g, dt)
    elif c["op"] == "norm":
        T, H, dt = c["tokens"], c["hidden"], DT[c["dtype"]]
        s["x"] = _randn((T, H), g, dt)
        s["other"] = _randn((T, H), g, dt, 4.0) if c["residual"] else None     # the residual stream, or the gradient that arrives through it
        s["gain"] = 1.0 + 0.1 * torch.randn(H, generator=g, device="cuda")
        if c["direction"] == "backward":
            s["grad"] = _randn((T, H), g, dt)
    else:
        T, F, N, G = c["tokens"], c["fan_in"], c["fan_out"], c["groups"]
        x = torch.randn((T, F), generator=g, device="cuda")
        w = torch.randn((G, N, F) if G else (N, F), generator=g, device="cuda") / math.sqrt(F)
        s["x_scale"] = s["w_scale"] = None
        if c["dtype"] == "e4m3":
            (s["x"], s["x_scale"]), (s["weight"], s["w_scale"]) = _quantise(x), _quantise(w)
        else:
            s["x"], s["weight"] = x.to(torch.bfloat16), w.to(torch.bfloat16)
        out = DT[c["out"]]
        s["bias_v"] = torch.randn((G, N) if G else (N,), generator=g, device="cuda") if c["bias"] else None
        s["mul_v"] = _randn((T, N), g, out) if c["mul"] else None
        s["residual_v"] = _randn((T, N), g, out) if c["residual"] else None
        s["y"] = torch.zeros((T, N), dtype=out, device="cuda")            # rows of no group stay zero
        s["offsets"] = None
        if G:
            share = torch.softmax(torch.randn(G, generator=g, device="cuda"), 0)
            of = torch.multinomial(share, T, replacement=True, generator=g)
            n = torch.bincount(of[torch.rand(T, generator=g, device="cuda") >= c["drop"]], minlength=G)
            s["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "dispatch":
        return _dispatch_forward(s) if s["direction"] == "forward" else _dispatch_backward(s)
    if s["op"] == "norm":
        return {"forward": _norm_forward, "e4m3": _norm_e4m3, "backward": _norm_backward}[s["direction"]](s)
    return _linear_plain(s)


def _run_own(s):
    import asynchronous_expert_execution_gb300 as moe
    if s["op"] == "dispatch":
        if s["direction"] == "forward":
            offsets, pos, pair = moe.sort_experts(s["expert"], s["experts"])
            rows = moe.sort_rows(s["x"], pos, out=s["rows"])
            y = moe.merge_rows(s["ys"], pos, s["w"], residual=s["residual"])
            return {"offsets": offsets, "pos": pos, "pair": pair, "rows": rows, "y": y}
        grad_ys, grad_w = moe.merge_rows_backward(s["grad"], s["ys"], s["pos"], s["w"], out=s["rows"])
        grad_x = moe.sort_rows_backward(s["grad_rows"], s["pos"])
        grad_logits = moe.route_backward(s["idx"], s["w"], grad_w, s["experts"])
        return {"grad_ys": grad_ys, "grad_w": grad_w, "grad_x": grad_x, "grad_logits": grad_logits}
    if s["op"] == "norm":
        if s["direction"] == "forward":
            y, h = moe.add_rms_norm(s["x"], s["other"], s["gain"], EPS)
            return {"y": y, "h": h}
        if s["direction"] == "e4m3":
            q, scale, h = moe.add_rms_norm_e4m3(s["x"], s["other"], s["gain"], EPS)
            return {"q": q, "scale": scale, "h": h}
        grad_x, grad_gain = moe.add_rms_norm_backward(s["grad"], s["x"], s["gain"], EPS, grad_h=s["other"])
        return {"grad_x": grad_x, "grad_gain": grad_gain}
    return moe.linear(s["x"], s["weight"], s["bias_v"], act=s["act"], mul=s["mul_v"], residual=s["residual_v"], offsets=s["offsets"],
                      x_scale=s["x_scale"], w_scale=s["w_scale"], out=s["y"])


def _dispatch_forward(s):
    T, K = s["expert"].shape
    offsets, pos, pair = _order(s["expert"], s["experts"])
    live = torch.arange(T * K, device=pair.device) < offsets[-1]
    rows = torch.where(live[:, None], s["x"][pair.long() // K], s["rows"])
    terms = s["ys"][pos.clamp(min=0).long()].float() * s["w"][:, :, None]
    y = torch.where((pos >= 0)[:, :, None], terms, 0.0).sum(1) + s["residual"].float()
    return {"offsets": offsets, "pos": pos, "pair": pair, "rows": rows, "y": y.to(s["ys"].dtype)}


def _dispatch_backward(s):
    T, K = s["pos"].shape
    pos, pair, dt = s["pos"].long(), s["pair"].long(), s["ys"].dtype
    here = pos >= 0
    live = torch.arange(T * K, device=pair.device) < s["offsets"][-1]
    grad = s["grad"].float()
    grad_ys = torch.where(live[:, None], (s["w"].reshape(-1)[pair, None] * grad[pair // K]).to(dt), s["rows"])
    grad_w = torch.where(here, (s["ys"][pos.clamp(min=0)].float() * grad[:, None]).sum(-1), 0.0)
    grad_x = torch.where(here[:, :, None], s["grad_rows"][pos.clamp(min=0)].float(), 0.0).sum(1)
    mean = (s["w"] * grad_w).sum(1, keepdim=True)
    grad_logits = torch.zeros((T, s["experts"]), device=pos.device).scatter(1, s["idx"].long(), s["w"] * (grad_w - mean))
    return {"grad_ys": grad_ys, "grad_w": grad_w, "grad_x": grad_x.to(dt), "grad_logits": grad_logits}


def _sum_and_norm(s):
    h = s["x"] if s["other"] is None else (s["x"].float() + s["other"].float()).to(s["x"].dtype)
    v = h.float()
    return h, v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * s["gain"]


def _norm_forward(s):
    h, y = _sum_and_norm(s)
    return {"y": y.to(h.dtype), "h": h}


def _norm_e4m3(s):
    h, y = _sum_and_norm(s)
    scale = (y.abs().amax(-1) / E4M3_MAX).clamp(min=TINY)
    return {"q": (y / scale[:, None]).to(torch.float8_e4m3fn), "scale": scale, "h": h}


def _norm_backward(s):
    h, grad = s["x"].float(), s["grad"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    n, u = h * r, grad * s["gain"]
    grad_x = r * (u - n * (u * n).mean(-1, keepdim=True))
    if s["other"] is not None:
        grad_x = grad_x + s["other"].float()
    return {"grad_x": grad_x.to(s["x"].dtype), "grad_gain": (grad * n).sum(0, dtype=torch.float64).float()}


def _act(v, act):
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    return v.clamp(min=0) if act == "relu" else v


def _epilogue(s, v, w_scale, bias, rows):
    if s["x_scale"] is not None:
        v = v * s["x_scale"][rows, None] * w_scale
    if bias is not None:
        v = v + bias
    v = _act(v, s["act"])
    if s["mul_v"] is not None:
        v = v * s["mul_v"][rows].float()
    if s["residual_v"] is not None:
        v = v + s["residual_v"][rows].float()
    return v.to(s["y"].dtype)


def _linear_plain(s):
    if s["offsets"] is None:
        return _epilogue(s, s["x"].float() @ s["weight"].float().T, s["w_scale"], s["bias_v"], slice(None))
    y, at = s["y"], s["offsets"].tolist()
    for e in range(s["groups"]):                      # one matrix product per expert: every expert has a number of rows of its own
        rows = slice(at[e], at[e + 1])
        if at[e] < at[e + 1]:
            y[rows] = _epilogue(s, s["x"][rows].float() @ s["weight"][e].float().T, None if s["w_scale"] is None else s["w_scale"][e],
                                None if s["bias_v"] is None else s["bias_v"][e], rows)
    return y


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    c = case
    if c["op"] == "dispatch":
        T, K, E, b = c["tokens"], c["top_k"], c["experts"], SIZE[c["dtype"]]
        P = T * K * (1.0 - c["drop"])
        row = c["hidden"] * b
        if c["direction"] == "forward":              # ids in, plan out; x in, its copies out; results, weights and residual in, y out
            return {"bytes": 4 * T * K * 3 + 4 * (E + 1) + T * row + P * row + P * row + 4 * T * K + 2 * T * row, "flops": 2.0 * P * c["hidden"]}
        return {"bytes": T * row + 2 * P * row + P * row + T * row + 4 * T * K * 4 + 4 * T * E, "flops": 4.0 * P * c["hidden"]}
    if c["op"] == "norm":
        T, H, b = c["tokens"], c["hidden"], SIZE[c["dtype"]]
        both = 2 if c["residual"] else 1
        if c["direction"] == "backward":             # grad and h (and the residual's grad) in, grad_x out; gain in, its gradient out
            return {"bytes": T * H * b * (2 + both) + 8 * H, "flops": 8.0 * T * H}
        y = T * H * b if c["direction"] == "forward" else T * H + 4 * T
        return {"bytes": T * H * b * (3 if c["residual"] else 1) + y + 4 * H, "flops": 5.0 * T * H}
    T, F, N, G = c["tokens"], c["fan_in"], c["fan_out"], c["groups"]
    live = T * (1.0 - c["drop"])
    b, o = SIZE[c["dtype"]], SIZE[c["out"]]
    moved = live * F * b + max(1, min(G, live)) * N * F * b + live * N * o * (1 + c["mul"] + c["residual"]) + 4 * N * max(1, G) * c["bias"]
    if c["dtype"] == "e4m3":
        moved += 4 * live + 4 * N * max(1, G)
    return {"bytes": moved, "flops": 2.0 * live * F * N}


# ------------------------------------------------------------------ the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    d = lambda t: None if t is None else t.double()  # noqa: E731
    if s["op"] == "dispatch":
        T, K = s["expert"].shape
        expert = s["expert"].cpu().tolist()
        ids = [(e, t, k) for t in range(T) for k, e in enumerate(expert[t]) if 0 <= e < s["experts"]]
        ids.sort(key=lambda v: v[0])
        P = len(ids)
        tok = torch.tensor([t for _, t, _ in ids], dtype=torch.long, device="cuda")
        kk = torch.tensor([k for _, _, k in ids], dtype=torch.long, device="cuda")
        if s["direction"] == "forward":
            rows = d(s["rows"]).clone()
            rows[:P] = d(s["x"])[tok]
            y = d(s["residual"]).clone()
            y.index_add_(0, tok, d(s["w"])[tok, kk, None] * d(s["ys"])[:P])
            return {"offsets": None, "pos": None, "pair": None, "rows": rows, "y": y}
        grad_ys = d(s["rows"]).clone()
        grad_ys[:P] = d(s["w"])[tok, kk, None] * d(s["grad"])[tok]
        grad_w = torch.zeros((T, K), dtype=torch.float64, device="cuda")
        grad_w[tok, kk] = (d(s["ys"])[:P] * d(s["grad"])[tok]).sum(1)
        grad_x = torch.zeros((T, s["hidden"]), dtype=torch.float64, device="cuda").index_add_(0, tok, d(s["grad_rows"])[:P])
        w = d(s["w"])
        jacobian = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
        grad_logits = torch.zeros((T, s["experts"]), dtype=torch.float64, device="cuda")
        grad_logits[torch.arange(T, device="cuda")[:, None], s["idx"].long()] = (jacobian @ grad_w[:, :, None])[:, :, 0]
        return {"grad_ys": grad_ys, "grad_w": grad_w, "grad_x": grad_x, "grad_logits": grad_logits}
    if s["op"] == "norm":
        if s["direction"] == "backward":
            h, grad, gain = d(s["x"]), d(s["grad"]), d(s["gain"])
            H = h.shape[1]
            q = (h * h).sum(1, keepdim=True) / H + EPS
            u = gain * grad
            grad_x = u / q.sqrt() - h * (u * h).sum(1, keepdim=True) / (H * q ** 1.5)
            if s["other"] is not None:
                grad_x = grad_x + d(s["other"])
            return {"grad_x": grad_x, "grad_gain": (grad * h / q.sqrt()).sum(0)}
        h = s["x"] if s["other"] is None else (d(s["x"]) + d(s["other"])).to(s["x"].dtype)
        y = d(h) / ((d(h) ** 2).sum(1, keepdim=True) / h.shape[1] + EPS).sqrt() * d(s["gain"])
        if s["direction"] == "forward":
            return {"y": y, "h": d(s["x"]) if s["other"] is None else d(s["x"]) + d(s["other"])}
        scale = (y.abs().amax(1) / E4M3_MAX).clamp(min=TINY)
        return {"q": y / scale[:, None], "scale": scale, "h": d(s["x"]) if s["other"] is None else d(s["x"]) + d(s["other"])}
    if 2.0 * s["tokens"] * s["fan_in"] * s["fan_out"] > 1e12:
        return None
    x = d(s["x"]) if s["x_scale"] is None else d(s["x"]) * d(s["x_scale"])[:, None]
    y = d(s["y"]).clone()
    at = [0, s["tokens"]] if s["offsets"] is None else s["offsets"].tolist()
    for e in range(len(at) - 1):
        pick = lambda t: t if s["offsets"] is None or t is None else t[e]  # noqa: E731
        w, i, j = d(pick(s["weight"])), at[e], at[e + 1]
        if s["w_scale"] is not None:
            w = w * d(pick(s["w_scale"]))[:, None]
        v = torch.einsum("tf,nf->tn", x[i:j], w)
        if s["bias_v"] is not None:
            v = v + d(pick(s["bias_v"]))
        if s["act"] == "silu":
            v = v * torch.sigmoid(v)
        elif s["act"] == "gelu":
            v = v * 0.5 * torch.erfc(-v / math.sqrt(2.0))
        elif s["act"] == "relu":
            v = torch.maximum(v, torch.zeros_like(v))
        if s["mul_v"] is not None:
            v = v * d(s["mul_v"][i:j])
        if s["residual_v"] is not None:
            v = v + d(s["residual_v"][i:j])
        y[i:j] = v
    return y

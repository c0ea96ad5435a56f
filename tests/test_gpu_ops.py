"""The stateless operators (sorted dispatch, norm, product) against their definitions in 64 bits.

Tolerances.  u = 2^-24 is half a step of fp32.  A sum of n fp32 terms in any order is off by at
most n u sum|terms|, an elementary operation by u of its result (2 u for a quotient or root used
here), a stored result by half a step of its type: 2^-8 (bf16), 2^-24 (fp32), 2^-4 (e4m3, and half
its smallest value, 2^-10, below the normal range) of its value.  Tensor-core sums may cut instead
of round: a whole step, 2^-23, per addition.
"""
import math

import numpy as np
import pytest
import torch

from oracle import moe_oracle as om

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BOTH = (torch.bfloat16, torch.float32)
NAN = float("nan")


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g
    g.build()
    import asynchronous_expert_execution_gb300 as pkg
    return pkg


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, g, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def strided(t, pad):
    """The same rows `pad` elements further apart, on a base `pad` elements into its buffer; what lies between is NaN."""
    if not pad:
        return t
    buf = torch.full((t.shape[0] + 1, t.shape[1] + 2 * pad), 0.0, device=t.device).to(t.dtype)
    if t.dtype != torch.float8_e4m3fn:
        buf.fill_(NAN)
    v = buf[:t.shape[0], pad:pad + t.shape[1]]
    v.copy_(t)
    return v


def close(got, want, tol, what):
    """Elementwise |got - want| <= tol in 64 bits."""
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((d / tol.clamp(min=1e-300)).nan_to_num(1e30).max()))


def ids(T, K, E, g, drop=0.0, skew=False):
    e = torch.rand((T, E), generator=g, device="cuda")
    if skew:
        e = e + 3.0 / (1 + torch.arange(E, device="cuda"))
    idx = torch.topk(e, K, dim=1).indices.to(torch.int32)
    away = torch.rand((T, K), generator=g, device="cuda") < drop
    return torch.where(away, torch.tensor(-1, dtype=torch.int32, device="cuda"), idx).contiguous()


def order(expert, E):
    """Offsets, pos, pair by numpy's stable sort."""
    flat = expert.cpu().numpy().reshape(-1)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    pair = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[pair], np.arange(E + 1))
    pos = np.empty(flat.size, dtype=np.int64)
    pos[pair] = np.arange(flat.size)
    pos[key == E] = -1
    return offsets, pos.reshape(expert.shape), pair


# ------------------------------------------------------------------ sorted dispatch

SORT_CASES = [(0, 1, 5), (1, 1, 1), (1, 8, 256), (2, 3, 3), (7, 5, 17), (33, 4, 128), (64, 32, 1024), (257, 8, 256), (1000, 3, 12),
              (2048, 8, 256), (4096, 4, 128), (5003, 7, 1023), (8192, 8, 64), (30011, 8, 257)]


@pytest.mark.parametrize("T,K,E", SORT_CASES)
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_sort_experts(moe, T, K, E, drop):
    expert = ids(T, K, E, gen(T + K), drop, skew=T % 2 == 1)
    if T > 2:
        expert[0], expert[1, 0], expert[-1] = E, -7, 2 ** 31 - 1         # outside on either side
    got = moe.sort_experts(expert, E)
    for g, w in zip(got, order(expert, E)):
        assert g.dtype == torch.int32 and np.array_equal(g.cpu().numpy(), w)


def test_sort_experts_one_expert_takes_all_and_repeats(moe):
    """Every pair on one expert, and the same expert twice in a token: still stable."""
    for E, e in ((1, 0), (300, 299), (1024, 512)):
        expert = torch.full((3001, 4), e, dtype=torch.int32, device="cuda")
        for g, w in zip(moe.sort_experts(expert, E), order(expert, E)):
            assert np.array_equal(g.cpu().numpy(), w)


ROW_CASES = [(1, 1, 4, 1), (1, 8, 64, 7168), (3, 2, 8, 7), (33, 4, 16, 64), (17, 9, 32, 137), (5, 32, 64, 520), (64, 4, 128, 2880),
             (301, 8, 256, 1000), (999, 3, 12, 137), (40, 2, 8, 20001)]


def dispatch_inputs(moe, T, K, E, H, dtype, drop, pad):
    g = gen(7 * T + K + H)
    expert = ids(T, K, E, g, drop)
    offsets, pos, pair = moe.sort_experts(expert, E)
    return g, pos, int(offsets[-1]), strided(randn((T, H), g, dtype), pad), strided(randn((T * K, H), g, dtype), pad)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T,K,E,H", ROW_CASES)
@pytest.mark.parametrize("drop,pad", [(0.0, 0), (0.4, 0), (0.0, 8), (0.4, 3), (1.0, 0)])
def test_rows_forward_and_back(moe, dtype, T, K, E, H, drop, pad):
    g, pos, P, x, ys = dispatch_inputs(moe, T, K, E, H, dtype, drop, pad)
    p = pos.cpu()
    here = p >= 0
    # sort_rows: copies, bit for bit; rows behind the last pair stay as they were
    out = strided(torch.full((T * K, H), 3.0, device="cuda").to(dtype), pad)
    rows = moe.sort_rows(x, pos, out=out)
    want = torch.full((T * K, H), 3.0, device="cuda").to(dtype)
    tok = torch.arange(T)[:, None].expand(T, K)
    want[p[here].long().cuda()] = x[tok[here].cuda()]
    assert rows is out and torch.equal(rows, want)
    # merge: what lies in rows of no pair, and the weights of pairs without a row, are not looked at
    ys[P:] = NAN
    w = torch.rand((T, K), generator=g, device="cuda")
    w_dirty = torch.where(pos >= 0, w, NAN)
    residual = strided(randn((T, H), g, dtype), pad)
    terms = torch.zeros((T, K, H), dtype=torch.float64, device="cuda")
    hc = here.cuda()
    terms[hc] = ys.double()[pos[hc].long()] * w.double()[hc][:, None]
    for weights, res in ((w_dirty, residual), (w_dirty, None), (None, None)):
        t = terms if weights is not None else torch.where(hc[:, :, None], terms / w.double()[:, :, None], 0.0)
        ref, mag = t.sum(1), t.abs().sum(1)
        if res is not None:
            ref, mag = ref + res.double(), mag + res.double().abs()
        y = moe.merge_rows(ys, pos, weights, res) if weights is not None else moe.sort_rows_backward(ys, pos)
        close(y, ref, (K + 2) * U * mag * 1.01 + HALF[dtype] * ref.abs() + 1e-300, "merge")
    if T:
        res2 = residual.clone()
        assert torch.equal(moe.merge_rows(ys, pos, w_dirty, res2, out=res2), moe.merge_rows(ys, pos, w_dirty, residual))
    # merge's gradients
    grad = strided(randn((T, H), g, dtype), pad)
    out = strided(torch.full((T * K, H), 3.0, device="cuda").to(dtype), pad)
    grad_rows, grad_w = moe.merge_rows_backward(grad, ys, pos, w_dirty, out=out)
    assert torch.equal(grad_rows[P:], want.new_full((T * K - P, H), 3.0))
    flat = (w.double()[:, :, None] * grad.double()[:, None]).reshape(T, K, H)
    ref = torch.zeros((P, H), dtype=torch.float64, device="cuda")
    ref[pos[hc].long()] = flat[hc]
    close(grad_rows[:P], ref, (U + HALF[dtype]) * ref.abs() * 1.01 + 1e-300, "grad_rows")
    prod = torch.zeros((T, K, H), dtype=torch.float64, device="cuda")
    prod[hc] = ys.double()[pos[hc].long()] * grad.double()[:, None].expand(T, K, H)[hc]
    close(grad_w, prod.sum(-1), (H + 1) * U * prod.abs().sum(-1) + 1e-300, "grad_w")


def test_merge_rows_equals_collect_bitwise(moe):
    """The sorted path's merge and the handle's collect: the same bits for the same results."""
    from workloads import get_config, make_workload
    spec = get_config("m4")
    L = spec.layer
    wl = make_workload(spec, seed=3)
    x = wl.x.cuda()
    idx, w = moe.route(wl.logits.cuda(), L.top_k)
    h = moe.MoEAsync(L.num_experts, L.top_k, L.hidden, L.inter, x.dtype, spec.tokens, expert_kind="identity")
    h.enqueue(0, x, idx, w)
    assert h.wait(0, moe.Policy("mtfs")) == 0
    y = torch.empty_like(x)
    slots = torch.empty(spec.tokens, dtype=torch.int32, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    h.collect(0, y, slots, n)
    assert h.sync() == 0 and int(n) == spec.tokens
    h.close()
    _, pos, _ = moe.sort_experts(idx, L.num_experts)
    mine = moe.merge_rows(moe.sort_rows(x, pos), pos, w)             # identity experts: E(x) = x
    assert torch.equal(mine[slots.long()], y)


@pytest.mark.parametrize("T,E,K", [(0, 8, 2), (1, 1, 1), (5, 33, 4), (100, 256, 8), (64, 1024, 32)])
def test_route_backward(moe, T, E, K):
    g = gen(T + E)
    logits = randn((T, E), g)
    idx, w = moe.route(logits, K)
    grad_w = randn((T, K), g)
    got = moe.route_backward(idx, w, grad_w, E)
    wd, gd = w.double(), grad_w.double()
    mag = (wd * gd).abs().sum(1, keepdim=True)
    ref = torch.zeros((T, E), dtype=torch.float64, device="cuda")
    ref.scatter_(1, idx.long(), wd * (gd - (wd * gd).sum(1, keepdim=True)))
    tol = torch.zeros_like(ref).scatter_(1, idx.long(), (K + 4) * U * wd * (gd.abs() + mag)) + 1e-300
    close(got, ref, tol, "grad_logits")


def test_route_backward_against_differences(moe):
    """The routing weights' own differences: steps of 2^-10 in 64 bits err by at most step^2 times the third derivative (< 1)."""
    g = gen(5)
    T, E, K = 6, 9, 3
    logits, grad_w = randn((T, E), g), randn((T, K), g)
    idx, w = moe.route(logits, K)
    got = moe.route_backward(idx, w, grad_w, E).double()
    f = lambda z: (torch.softmax(z.gather(1, idx.long()), 1) * grad_w.double()).sum(1)   # noqa: E731
    z, step = logits.double(), 2.0 ** -10
    for e in range(E):
        d = torch.zeros_like(z)
        d[:, e] = step
        diff = (f(z + d) - f(z - d)) / (2 * step)
        # 64-bit differences, their truncation, and the kernel's own error on weights off by 4 u
        assert float((got[:, e] - diff).abs().max()) <= (step ** 2 + 16 * K * U) * float(grad_w.abs().sum(1).max())


# ------------------------------------------------------------------ norm

NORM_CASES = [(1, 1), (1, 7168), (3, 7), (2, 8), (33, 64), (5, 137), (16, 997), (100, 2880), (7, 4104), (40, 8192), (3, 20001), (2, 40000),
              (1000, 584)]


def norm_parts(x, res, gain, eps):
    h = x if res is None else (x.double() + res.double()).to(x.dtype)        # 64 bits hold the sum of two such values
    v = h.double()
    r = 1.0 / (v.square().mean(1, keepdim=True) + eps).sqrt()
    return h, v * r * (1.0 if gain is None else gain.double()), r


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T,H", NORM_CASES)
@pytest.mark.parametrize("residual,gained,pad", [(True, True, 0), (False, True, 0), (True, False, 8), (True, True, 5)])
def test_add_rms_norm(moe, dtype, T, H, residual, gained, pad):
    g = gen(T * H)
    x = strided(randn((T, H), g, dtype), pad)
    res = strided(randn((T, H), g, dtype, 4.0), pad) if residual else None
    gain = 1 + 0.1 * randn((H,), g) if gained else None
    eps = 1e-6
    h, y, r = norm_parts(x, res, gain, eps)
    er = (H / 2 + 8) * U                                                     # of r: half the sum of squares' error, a mean, a root
    got, gh = moe.add_rms_norm(x, res, gain, eps)
    assert torch.equal(gh, h) and (residual or gh is x)
    close(got, y, (er + 2 * U + HALF[dtype]) * y.abs() * 1.01 + 1e-300, "y")
    q, scale, qh = moe.add_rms_norm_e4m3(x, res, gain, eps)
    assert torch.equal(qh, h) and q.dtype == torch.float8_e4m3fn
    want = (y.abs().amax(1) / 448).clamp(min=2.0 ** -126)
    close(scale, want, (er + 5 * U) * want * 1.01, "scale")
    s = scale.double()[:, None]
    close(q.double() * s, y, (2.0 ** -4 + 2 * er + 8 * U) * y.abs() + 1.01 * 2.0 ** -10 * s, "q")
    if residual:                                                             # the sum in place of either operand, in the same layout: the same bits
        for i in (0, 1):
            a = [strided(x.contiguous(), pad) if pad else x.clone(), strided(res.contiguous(), pad) if pad else res.clone()]
            y2, h2 = moe.add_rms_norm(a[0], a[1], gain, eps, out_h=a[i])
            assert h2 is a[i] and torch.equal(h2, h) and torch.equal(y2, got)


@pytest.mark.parametrize("dtype", BOTH)
def test_norm_of_zeros_nan_and_infinity(moe, dtype):
    """A row of zeros stays zeros with the smallest scale; one with a NaN or an infinity is NaN, alone."""
    x = randn((5, 264), gen(1), dtype)
    x[1], x[2, 9], x[3, 200] = 0.0, NAN, float("inf")
    y, _ = moe.add_rms_norm(x)
    q, scale, _ = moe.add_rms_norm_e4m3(x)
    assert not bool(y[[0, 1, 4]].isnan().any()) and not bool(y[1].any()) and bool(y[2].isnan().all())
    assert bool(y[3, 200].isnan()) and bool(scale[[2, 3]].isnan().all()) and float(scale[1]) == 2.0 ** -126
    assert not bool(q[1].float().any()) and bool(q[2].float().isnan().all()) and bool(torch.isfinite(scale[[0, 1, 4]]).all())
    tiny = torch.full((1, 64), 1e-38, device="cuda")                         # y / scale stays finite at the smallest scale
    q, scale, _ = moe.add_rms_norm_e4m3(tiny)
    assert bool(torch.isfinite(q.float()).all()) and float(scale[0]) >= 2.0 ** -126


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T,H", NORM_CASES + [(700, 200), (2500, 72)])
@pytest.mark.parametrize("arrives,gained,pad", [(True, True, 0), (False, True, 3), (True, False, 8)])
def test_add_rms_norm_backward(moe, dtype, T, H, arrives, gained, pad):
    g = gen(T + H)
    h, grad = strided(randn((T, H), g, dtype, 2.0), pad), strided(randn((T, H), g, dtype), pad)
    gh = strided(randn((T, H), g, dtype), pad) if arrives else None
    gain = 1 + 0.1 * randn((H,), g) if gained else None
    eps = 1e-6
    gx, gg = moe.add_rms_norm_backward(grad, h, gain, eps, grad_h=gh)
    v, d = h.double(), grad.double()
    r = 1.0 / (v.square().mean(1, keepdim=True) + eps).sqrt()
    n, u = v * r, d * (1.0 if gain is None else gain.double())
    m, mag = (u * n).mean(1, keepdim=True), (u * n).abs().mean(1, keepdim=True)
    ref = r * (u - n * m) + (0.0 if gh is None else gh.double())
    er = (H / 2 + 10) * U
    tol = r * ((u.abs() + n.abs() * m.abs()) * (2 * er + 8 * U) + n.abs() * mag * (H + 8) * U)
    close(gx, ref, tol + (HALF[dtype] + 2 * U) * (ref.abs() + tol) + (0.0 if gh is None else U * gh.double().abs()) + 1e-300, "grad_x")
    if gain is None:
        assert gg is None
    else:
        close(gg, (d * n).sum(0), (T + 2 + H / 2 + 10) * U * (d * n).abs().sum(0) * 1.01 + 1e-300, "grad_gain")
        again = moe.add_rms_norm_backward(grad, h, gain, eps, grad_h=gh)
        assert torch.equal(again[0], gx) and torch.equal(again[1], gg)
    if gh is not None:
        again = strided(torch.zeros((T, H), device="cuda").to(dtype), pad)
        moe.add_rms_norm_backward(grad, h, gain, eps, grad_h=gh, out=again)
        assert torch.equal(moe.add_rms_norm_backward(grad, h, gain, eps, grad_h=gh, out=gh)[0], again)


def test_norm_backward_against_differences(moe):
    """Central differences of the norm in 64 bits, step 2^-12: truncation below step^2 times a third derivative of at most 60."""
    g = gen(9)
    T, H, eps, step = 3, 11, 1e-6, 2.0 ** -12
    h, grad, gain = randn((T, H), g), randn((T, H), g), 1 + 0.1 * randn((H,), g)
    gx, gg = moe.add_rms_norm_backward(grad, h, gain, eps)
    f = lambda v, a: (v / (v.square().mean(1, keepdim=True) + eps).sqrt() * a * grad.double()).sum(1)   # noqa: E731
    v, a = h.double(), gain.double()
    bound = 60 * step ** 2 * float(grad.abs().sum(1).max()) / float(v.square().mean(1).sqrt().min()) ** 3 + 1e-5
    for c in range(H):
        d = torch.zeros_like(v)
        d[:, c] = step
        assert float((gx[:, c].double() - (f(v + d, a) - f(v - d, a)) / (2 * step)).abs().max()) <= bound
        e = torch.zeros_like(a)
        e[c] = step
        assert abs(float(gg[c]) - float(((f(v, a + e) - f(v, a - e)) / (2 * step)).sum())) <= bound


# ------------------------------------------------------------------ product

def act64(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * 0.5 * torch.erfc(-v * math.sqrt(0.5))
    return v.clamp(min=0) if act == "relu" else v


def linear_inputs(T, F, Nn, e4m3, out, extras, groups, g, pad=0):
    x, w = randn((T, F), g), randn((groups, Nn, F) if groups else (Nn, F), g, scale=1 / math.sqrt(F))
    kw, per = {}, (groups, Nn) if groups else (Nn,)
    if e4m3:
        kw["x_scale"] = x.abs().amax(1) / 448
        kw["w_scale"] = w.abs().amax(-1) / 448
        x, w = (x / kw["x_scale"][:, None]).to(torch.float8_e4m3fn), (w / kw["w_scale"][..., None]).to(torch.float8_e4m3fn)
    else:
        x, w = x.to(torch.bfloat16), w.to(torch.bfloat16)
    if "b" in extras:
        kw["bias"] = randn(per, g)
    if "m" in extras:
        kw["mul"] = strided(randn((T, Nn), g, out), pad)
    if "r" in extras:
        kw["residual"] = strided(randn((T, Nn), g, out), pad)
    return x, w, kw


def linear_ref(x, w, kw, act, out, start=None, at=None):
    """Result and tolerance in 64 bits."""
    G = 0 if at is None else len(at) - 1
    T, Nn, F = x.shape[0], w.shape[-2], x.shape[1]
    ref = torch.zeros((T, Nn), dtype=torch.float64, device="cuda") if start is None else start.double()
    tol = torch.zeros((T, Nn), dtype=torch.float64, device="cuda")
    for e in range(max(G, 1)):
        i, j = (0, T) if at is None else (at[e], at[e + 1])
        pick = lambda t: t if at is None or t is None else t[e]              # noqa: E731
        xe, we = x[i:j].double(), pick(w).double()
        if "x_scale" in kw:
            xe, we = xe * kw["x_scale"][i:j].double()[:, None], we * pick(kw["w_scale"]).double()[:, None]
        v, t = xe @ we.T, (F * 2.0 ** -23 + 4 * U) * (xe.abs() @ we.abs().T)
        if "bias" in kw:
            b = pick(kw["bias"]).double()
            v, t = v + b, t + U * (v.abs() + b.abs())
        v, t = act64(v, act), 1.13 * t + (8 * U * v.abs() if act != "none" else 0.0)     # slopes of silu and gelu stay below 1.13
        if "mul" in kw:
            m = kw["mul"][i:j].double()
            v, t = v * m, t * m.abs() + U * (v * m).abs()
        if "residual" in kw:
            r = kw["residual"][i:j].double()
            v, t = v + r, t + U * (v.abs() + r.abs())
        ref[i:j], tol[i:j] = v, t + HALF[out] * (v.abs() + t) + 1e-300
    return ref, tol


LINEAR_CASES = [  # tokens, fan_in, fan_out
    (1, 16, 1), (1, 2880, 2880), (2, 64, 7), (3, 48, 130), (4, 7168, 257), (7, 144, 997), (16, 1008, 128), (17, 512, 64), (33, 4112, 300),
    (64, 2880, 256), (65, 80, 1000), (127, 2064, 255), (128, 128, 128), (129, 256, 384), (200, 592, 416), (256, 1024, 512), (300, 992, 1000),
    (777, 592, 997), (1025, 320, 1111),
    # every width of the tiles over two SMs, and 128 tokens split one to six ways, on wide rows and others
    (412, 80, 2824), (963, 1040, 2680), (966, 1040, 3304), (2472, 336, 912), (1003, 1040, 3360), (2251, 592, 1760), (273, 144, 3864),
    (259, 6464, 3264), (2470, 2976, 1286), (1761, 1632, 1285), (1623, 1952, 1567), (2996, 6528, 137), (2529, 1152, 387),
    (138, 2688, 3693), (2997, 3424, 136), (2657, 1888, 131), (70, 4240, 3640), (2961, 4416, 39), (2314, 6368, 9), (1968, 1136, 1032)]


@pytest.mark.parametrize("T,F,Nn", LINEAR_CASES)
@pytest.mark.parametrize("e4m3,out,act,extras", [(False, torch.bfloat16, "none", ""), (False, torch.float32, "silu", "bm"),
                                                 (True, torch.bfloat16, "gelu", "br"), (True, torch.float32, "none", "bmr"),
                                                 (False, torch.bfloat16, "relu", "bmr")])
def test_linear(moe, T, F, Nn, e4m3, out, act, extras):
    g = gen(T + F + Nn)
    x, w, kw = linear_inputs(T, F, Nn, e4m3, out, extras, 0, g)
    got = moe.linear(x, w, act=act, out_dtype=out, **kw)
    ref, tol = linear_ref(x, w, kw, act, out)
    close(got, ref, tol, "linear")
    assert torch.equal(moe.linear(x, w, act=act, out_dtype=out, **kw), got)      # the same bits again


@pytest.mark.parametrize("T", [1, 3, 8, 9, 15, 16])
@pytest.mark.parametrize("F,Nn", [(16, 9), (64, 20011), (1056, 1235), (2064, 1200), (4128, 130), (208, 2500), (20000, 8), (7168, 6000)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_linear_of_few_tokens(moe, T, F, Nn, e4m3):
    """One to 16 rows, also on the sides of the sizes at which the kernel, its features a block and its warps change."""
    g = gen(T + F + Nn)
    out = torch.float32 if T % 2 else torch.bfloat16
    x, w, kw = linear_inputs(T, F, Nn, e4m3, out, "bmr", 0, g, pad=T % 3)
    got = moe.linear(strided(x, 32), strided(w, 16), act="silu", out_dtype=out, **kw)
    ref, tol = linear_ref(x, w, kw, "silu", out)
    close(got, ref, tol, "few tokens")
    assert torch.equal(moe.linear(x, w, act="silu", out_dtype=out, out=kw["residual"], **kw), got)


def test_linear_of_small_integers_is_exact(moe):
    """Integer operands whose sums stay below 2^24 leave no room for rounding: every product reaches its place."""
    g = gen(2)
    for T, F, Nn in ((1, 512, 300), (5, 2880, 200), (70, 1040, 130), (300, 2064, 520), (1030, 416, 777)):
        for dt in (torch.bfloat16, torch.float8_e4m3fn):
            x = torch.randint(-8, 9, (T, F), generator=g, device="cuda").float().to(dt)
            w = torch.randint(-8, 9, (Nn, F), generator=g, device="cuda").float().to(dt)
            one = {} if dt == torch.bfloat16 else {"x_scale": torch.ones(T, device="cuda"), "w_scale": torch.ones(Nn, device="cuda")}
            y = moe.linear(x, w, out_dtype=torch.float32, **one)
            assert torch.equal(y.double(), x.double() @ w.double().T), (T, F, Nn, dt)


@pytest.mark.parametrize("T,F,Nn,out", [(77, 160, 201, torch.float32), (11, 160, 201, torch.bfloat16), (963, 1040, 2680, torch.bfloat16),
                                        (963, 1040, 2680, torch.float32), (1623, 1952, 1567, torch.bfloat16), (1968, 1136, 1032, torch.bfloat16)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_linear_strides_and_outputs_in_place(moe, e4m3, T, F, Nn, out):
    g = gen(3)
    x, w, kw = linear_inputs(T, F, Nn, e4m3, out, "bmr", 0, g, pad=3)
    want = moe.linear(x, w, out_dtype=out, **kw)
    ref, tol = linear_ref(x, w, kw, "none", out)
    close(want, ref, tol, "contiguous")
    xs, ws = strided(x, 16), strided(w, 32)
    y = strided(torch.zeros((T, Nn), device="cuda").to(out), 5)
    assert torch.equal(moe.linear(xs, ws, out=y, **kw), want)
    for name in ("mul", "residual"):
        k2 = dict(kw)
        k2[name] = kw[name].clone()
        assert torch.equal(moe.linear(x, w, out=k2[name], **k2), want)


GROUP_CASES = [  # rows, fan_in, fan_out, rows of each group
    (10, 64, 40, [3, 0, 7]), (1, 128, 130, [0, 0, 1, 0]), (200, 592, 300, [0, 129, 1, 0, 64, 6]), (500, 256, 256, [256, 100, 144]),
    (300, 144, 257, [40] * 7), (64, 2880, 150, [1] * 64), (900, 320, 500, [600, 3, 0, 250]),
    (16, 320, 100, [0] * 40 + [3, 0, 9] + [0] * 50 + [4]), (13, 80, 33, [0, 13]), (8, 4128, 2000, [1, 0, 2, 0, 0, 5]), (16, 64, 1300, [1] * 16),
    (2000, 512, 2000, [700, 0, 3, 256, 255, 129, 600, 57]), (1500, 2064, 1000, [1, 900, 128, 127, 0, 300]), (3000, 592, 1040, [250] * 11 + [2])]


@pytest.mark.parametrize("T,F,Nn,counts", GROUP_CASES)
@pytest.mark.parametrize("e4m3,out,act,extras", [(False, torch.bfloat16, "silu", "m"), (True, torch.float32, "none", "bmr")])
def test_linear_per_expert(moe, T, F, Nn, counts, e4m3, out, act, extras):
    g = gen(T + F + Nn)
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    x, w, kw = linear_inputs(T, F, Nn, e4m3, out, extras, len(counts), g)
    if not e4m3:
        x[at[-1]:] = NAN                                                     # rows of no group are not looked at
    y = torch.full((T, Nn), 3.0, device="cuda").to(out)
    ref, tol = linear_ref(x, w, kw, act, out, y, at)
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    got = moe.linear(x, w, act=act, offsets=offsets, out=y, **kw)
    assert got is y
    close(y[:at[-1]], ref[:at[-1]], tol[:at[-1]], "per expert")
    assert bool((y[at[-1]:] == 3.0).all())


@pytest.mark.parametrize("T,F,Nn", [(1100, 1040, 520), (520, 2880, 300), (300, 208, 1000), (2600, 64, 96)])
@pytest.mark.parametrize("out", BOTH)
def test_linear_with_groups_of_every_size(moe, T, F, Nn, out):
    """70 groups, some large, most small or empty: the tiles are not taken in the groups' order."""
    g = gen(T + Nn)
    share = torch.rand(70, generator=g, device="cuda") ** 6
    at = torch.cat([torch.zeros(1, device="cuda"), (share.cumsum(0) / share.sum() * T)]).int()
    at[-1] = T
    x, w, kw = linear_inputs(T, F, Nn, False, out, "bmr", 70, g)
    ref, tol = linear_ref(x, w, kw, "silu", out, torch.zeros((T, Nn), device="cuda"), at.tolist())
    close(moe.linear(x, w, act="silu", offsets=at, out_dtype=out, **kw), ref, tol, "groups of every size")


def test_linear_rows_before_the_first_group_and_bad_offsets(moe):
    """Groups may start behind row 0; offsets outside the rows are clipped, descending ones hold no rows."""
    g = gen(4)
    x, w, _ = linear_inputs(50, 64, 24, False, torch.bfloat16, "", 4, g)
    y = torch.full((50, 24), 3.0, device="cuda").to(torch.bfloat16)
    moe.linear(x, w, offsets=torch.tensor([10, 20, 15, 45, 1000], dtype=torch.int32, device="cuda"), out=y)
    want = torch.full((50, 24), 3.0, device="cuda").to(torch.bfloat16)
    for e, (i, j) in ((0, (10, 20)), (2, (15, 45)), (3, (45, 50))):
        want[i:j] = moe.linear(x[i:j], w[e])
    # group 2 starts inside group 0's rows: the later of two writers of a row is not defined, the others are
    assert torch.equal(y[:15], want[:15]) and torch.equal(y[20:], want[20:])


@pytest.mark.parametrize("T,F,Nn", [(3, 1040, 700), (40, 592, 997), (300, 2064, 520), (512, 512, 3001), (1024, 1040, 2000), (2048, 592, 1999)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_linear_sums_do_not_depend_on_the_epilogue(moe, T, F, Nn, e4m3):
    """The same operands give the same sums, whatever is added, multiplied or skipped and wherever the rows lie."""
    g = gen(T + Nn)
    x, w, kw = linear_inputs(T, F, Nn, e4m3, torch.float32, "", 0, g)
    plain = moe.linear(x, w, out_dtype=torch.float32, **kw)
    assert torch.equal(moe.linear(x, w, out_dtype=torch.float32, act="relu", **kw), plain.clamp(min=0))
    one, zero = torch.ones((T, Nn), device="cuda"), torch.zeros((T, Nn), device="cuda")
    assert torch.equal(moe.linear(x, w, out_dtype=torch.float32, mul=one, residual=zero, **kw), plain)
    assert torch.equal(moe.linear(x, w, out=strided(zero, 3), mul=strided(one, 1), **kw), plain)


@pytest.mark.parametrize("e4m3", [False, True])
def test_linear_keeps_nan_and_infinity_in_their_rows(moe, e4m3):
    """A NaN in one row reaches that row's outputs only; inf * 0 of another row stays there; relu keeps NaN."""
    g = gen(6)
    x, w, kw = linear_inputs(40, 256, 130, e4m3, torch.float32, "", 0, g)
    clean = moe.linear(x, w, out_dtype=torch.float32, **kw)
    dirty = x.clone()
    dirty[7, 100] = torch.tensor(NAN).to(x.dtype)
    if not e4m3:
        dirty[9, 3] = float("inf")
    got = moe.linear(dirty, w, act="relu", out_dtype=torch.float32, **kw)
    keep = [i for i in range(40) if i not in (7, 9)]
    assert bool(got[7].isnan().all()) and torch.equal(got[keep], clean.clamp(min=0)[keep])
    if not e4m3:
        assert not bool(torch.isfinite(got[9][w[:, 3] > 0]).any())


# ------------------------------------------------------------------ together

def block(moe, x, res, p, K, E):
    """Norm in 8 bits -> router -> sorted experts -> merge with the residual."""
    q, s, h = moe.add_rms_norm_e4m3(x, res, p["gain"])
    idx, w = moe.route(moe.linear(q, p["router"][0], p["bias"], x_scale=s, w_scale=p["router"][1], out_dtype=torch.float32), K)
    offsets, pos, _ = moe.sort_experts(idx, E)
    y, _ = moe.add_rms_norm(x, res, p["gain"])
    rows = moe.sort_rows(y, pos)
    up = moe.linear(rows, p["w3"], offsets=offsets)
    act = moe.linear(rows, p["w1"], act="silu", mul=up, offsets=offsets)
    return y, h, idx, w, moe.merge_rows(moe.linear(act, p["w2"], offsets=offsets), pos, w, residual=h)


def block_params(E, H, I, g):
    r = randn((E, H), g, scale=1 / math.sqrt(H))
    rs = r.abs().amax(1) / 448
    return {"gain": 1 + 0.1 * randn((H,), g), "bias": randn((E,), g), "router": ((r / rs[:, None]).to(torch.float8_e4m3fn), rs),
            "w1": randn((E, I, H), g, torch.bfloat16, 1 / math.sqrt(H)), "w3": randn((E, I, H), g, torch.bfloat16, 1 / math.sqrt(H)),
            "w2": randn((E, H, I), g, torch.bfloat16, 1 / math.sqrt(I))}


@pytest.mark.parametrize("T", [1, 5, 64, 300])
def test_block_against_the_oracle(moe, T):
    """The operators in the order of use, against the oracle's dense layer on the same routing (the handle's own bound, 2e-2)."""
    E, K, H, I = 16, 4, 320, 192
    g = gen(T)
    p, x, res = block_params(E, H, I, g), randn((T, H), g, torch.bfloat16), randn((T, H), g, torch.bfloat16, 2.0)
    y, h, idx, w, out = block(moe, x, res, p, K, E)
    ex = lambda e: tuple(p[k][e].double().cpu().numpy().T for k in ("w1", "w3", "w2"))   # noqa: E731
    ref = om.dense_moe(y.double().cpu().numpy(), idx.cpu().numpy(), w.cpu().numpy(), ex) + h.double().cpu().numpy()
    assert np.abs(out.double().cpu().numpy() - ref).max() <= 2e-2 * np.abs(ref).max()


def test_block_captured_replayed_and_on_two_streams(moe):
    """One graph of the whole block, replayed on new inputs, equals direct calls; two streams at once give the same bits."""
    E, K, H, I, T = 16, 4, 320, 192, 100
    g = gen(11)
    p = block_params(E, H, I, g)
    xs = [randn((T, H), g, torch.bfloat16) for _ in range(4)]
    rs = [randn((T, H), g, torch.bfloat16, 2.0) for _ in range(4)]
    want = [block(moe, a, b, p, K, E)[-1] for a, b in zip(xs, rs)]
    x, r = xs[0].clone(), rs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(moe, x, r, p, K, E)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(moe, x, r, p, K, E)[-1]
    for i in (1, 2, 3, 0):
        x.copy_(xs[i])
        r.copy_(rs[i])
        graph.replay()
        assert torch.equal(out, want[i])
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(4)], [None] * 4
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = block(moe, xs[i], rs[i], p, K, E)[-1]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_backward_captured_and_replayed(moe):
    g = gen(13)
    T, K, E, H = 150, 4, 16, 264
    expert = ids(T, K, E, g, 0.2)
    gain = 1 + 0.1 * randn((H,), g)

    def step(grad, ys, w, h):
        _, pos, _ = moe.sort_experts(expert, E)
        grad_rows, grad_w = moe.merge_rows_backward(grad, ys, pos, w, out=torch.zeros_like(ys))
        gx = moe.sort_rows_backward(grad_rows, pos)
        return (grad_w, *moe.add_rms_norm_backward(gx, h, gain, grad_h=grad))

    def inputs():
        return [randn((T, H), g, torch.bfloat16), randn((T * K, H), g, torch.bfloat16), torch.rand((T, K), generator=g, device="cuda"),
                randn((T, H), g, torch.bfloat16)]
    a, b = inputs(), inputs()
    want = [step(*a), step(*b)]
    buf = [t.clone() for t in a]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*buf)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*buf)
    for i, src in ((1, b), (0, a), (1, b)):
        for d, s in zip(buf, src):
            d.copy_(s)
        graph.replay()
        for x, y in zip(out, want[i]):
            assert torch.equal(x, y)


def test_given_stream_is_used(moe):
    """stream=: the call is ordered behind that stream's work, not the current stream's."""
    s = torch.cuda.Stream()
    x = torch.zeros((64, 256), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        x.fill_(2.0)
    y, _ = moe.add_rms_norm(x, stream=s)
    gx, gg = moe.add_rms_norm_backward(x, x, torch.ones(256, device="cuda"), stream=s)
    s.synchronize()
    assert bool(((y.float() - 1).abs() < 1e-2).all()) and bool((gg > 0).all())


def test_outputs_of_a_given_stream_do_not_meet_the_current_stream(moe):
    """stream=: what the call allocates comes from that stream's memory, not from what the current stream has
    just given back while its kernels still read it."""
    s = torch.cuda.Stream()
    x = torch.ones((512, 4096), dtype=torch.bfloat16, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        victim = torch.full((512, 4096), 5.0, dtype=torch.bfloat16, device="cuda")
        torch.cuda._sleep(3_000_000)
        keep = victim.clone()                        # reads victim when the sleep is over
        del victim                                   # its memory is free again for the current stream only
        y, _ = moe.add_rms_norm(x, stream=s)
        s.synchronize()
        assert bool((y == 1).all())
        assert bool((keep == 5).all())


BIG = [(300_000, 7200)]                              # 2.16e9 elements: offsets pass 32 bits


@pytest.mark.parametrize("T,H", BIG)
def test_offsets_beyond_32_bits(moe, T, H):
    """The last rows of matrices of more than 2^31 elements."""
    g = gen(21)
    rows = torch.arange(T, device="cuda").remainder(97).to(torch.bfloat16)[:, None].expand(T, H).contiguous()
    pos = torch.arange(T, dtype=torch.int32, device="cuda").reshape(-1, 3)           # three pairs a token
    w = torch.rand(pos.shape, generator=g, device="cuda")
    y = moe.merge_rows(rows, pos, w)
    ref = (rows[:, 0].double().reshape(-1, 3) * w.double()).sum(1)
    assert float(((y[:, -1].double() - ref).abs() / (ref.abs() + 1e-9)).max()) < 2 ** -7 and torch.equal(y[:, 0], y[:, -1])
    back = moe.sort_rows(y, pos)
    assert torch.equal(back[:, -1], y[:, -1].repeat_interleave(3)) and torch.equal(back[-1], y[-1].clone())
    del back
    n, h = moe.add_rms_norm(rows, rows, out_h=rows)                                   # in place, twice the value
    assert float(h[-1, -1]) == 2 * ((T - 1) % 97) and abs(float(n[-1, -1]) - 1) < 2 ** -7
    del n, h, rows
    x, wt = randn((T, 64), g, torch.bfloat16), randn((H, 64), g, torch.bfloat16)
    out = moe.linear(x, wt)
    ref = x[-300:].double() @ wt.double().T
    close(out[-300:], ref, 65 * 2.0 ** -23 * (x[-300:].double().abs() @ wt.double().abs().T) + 2.0 ** -8 * 1.01 * ref.abs() + 1e-300, "far rows")
    offsets = torch.tensor([0, 5, T - 1000, T], dtype=torch.int32, device="cuda")
    w3 = torch.stack([wt, wt, 2 * wt])
    out.zero_()
    moe.linear(x, w3, offsets=offsets, out=out)
    close(out[-300:], 2 * ref, 65 * 2.0 ** -22 * (x[-300:].double().abs() @ wt.double().abs().T) + 2.0 ** -7 * 1.01 * ref.abs() + 1e-300, "far group")


def test_linear_with_many_groups(moe):
    """1024 experts, most of them without a row."""
    g = gen(22)
    T, F, Nn, G = 700, 64, 40, 1024
    of = torch.randint(0, G, (T,), generator=g, device="cuda").sort().values
    of[:300] = 5                                     # one group of several tiles
    of = of.sort().values
    at = torch.searchsorted(of, torch.arange(G + 1, device="cuda")).to(torch.int32)
    x, w = randn((T, F), g, torch.bfloat16), randn((G, Nn, F), g, torch.bfloat16)
    for out in BOTH:
        y = moe.linear(x, w, offsets=at, out_dtype=out)
        ref = torch.einsum("tf,tnf->tn", x.double(), w.double()[of])
        mag = torch.einsum("tf,tnf->tn", x.double().abs(), w.double().abs()[of])
        close(y, ref, F * 2.0 ** -23 * mag + HALF[out] * 1.01 * ref.abs() + 1e-300, "many groups")


@pytest.mark.parametrize("T,F,Nn", [(700, 7168, 2050), (1500, 2064, 1800), (300, 1040, 7168)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_long_fp32_sums_are_rounded_not_cut(moe, T, F, Nn, e4m3):
    """fp32 results of long sums: the error of the whole matrix stays at rounded sums' level.  A chunk of at most 14
    k-blocks is 56 matrix instructions, each of which may cut a whole step (2^-23) of its running sum: at most
    56 / 2 steps on average over a growing sum, towards zero, and chunks add with rounding."""
    g = gen(T)
    x, w, kw = linear_inputs(T, F, Nn, e4m3, torch.float32, "", 0, g)
    y = moe.linear(x, w, out_dtype=torch.float32, **kw)
    ref, _ = linear_ref(x, w, kw, "none", torch.float32)
    assert float((y.double() - ref).norm() / ref.norm()) <= 28 * 2.0 ** -23


def test_no_wait_ran_out(moe):
    """After everything above: the operators' sticky device error is clear."""
    moe.ops_sync()


# ------------------------------------------------------------------ refusals (nothing is launched)

def test_refusals(moe):
    g = gen(8)
    x, pos = randn((4, 32), g, torch.bfloat16), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    w, wt = torch.ones((4, 2), device="cuda"), randn((16, 32), g, torch.bfloat16)
    e8 = x.to(torch.float8_e4m3fn)
    bad = [
        lambda: moe.sort_experts(pos.long(), 4), lambda: moe.sort_experts(pos.cpu(), 4), lambda: moe.sort_experts(pos, 0),
        lambda: moe.sort_experts(pos, 1025), lambda: moe.sort_experts(pos[:, :1], 4), lambda: moe.sort_experts(pos[0], 4),
        lambda: moe.sort_experts(torch.zeros((2, 33), dtype=torch.int32, device="cuda"), 64),
        lambda: moe.sort_rows(x.half(), pos), lambda: moe.sort_rows(x, pos[:3]), lambda: moe.sort_rows(x.t(), pos),
        lambda: moe.sort_rows(x, pos, out=x.float()), lambda: moe.sort_rows(x, pos.cpu()), lambda: moe.sort_rows(x[:1].expand(4, 32), pos),
        lambda: moe.merge_rows(x, pos, w.double()), lambda: moe.merge_rows(x, pos, w[:, :1]), lambda: moe.merge_rows(x, pos, w, residual=x[:2]),
        lambda: moe.merge_rows_backward(x.float(), x, pos, w), lambda: moe.merge_rows_backward(x, x, pos, None if False else w.cpu()),
        lambda: moe.route_backward(pos, w, w, 1), lambda: moe.route_backward(pos, w, w.cpu(), 8), lambda: moe.route_backward(pos, w, w, 0),
        lambda: moe.add_rms_norm(x.half()), lambda: moe.add_rms_norm(x, x.float()), lambda: moe.add_rms_norm(x, gain=torch.ones(31, device="cuda")),
        lambda: moe.add_rms_norm(x, eps=-1.0), lambda: moe.add_rms_norm(x, eps=NAN), lambda: moe.add_rms_norm(x, out_h=x.clone()),
        lambda: moe.add_rms_norm(x, gain=torch.ones(32, device="cuda", dtype=torch.bfloat16)),
        lambda: moe.add_rms_norm_backward(x, x.float()), lambda: moe.add_rms_norm_backward(x[:, :16], x),
        lambda: moe.linear(x.float(), wt.float()), lambda: moe.linear(x, wt[:, :16]), lambda: moe.linear(x, wt, act="tanh"),
        lambda: moe.linear(x, wt, torch.ones(15, device="cuda")), lambda: moe.linear(e8, wt), lambda: moe.linear(e8, wt.to(e8.dtype)),
        lambda: moe.linear(x, wt, x_scale=torch.ones(4, device="cuda")), lambda: moe.linear(x, wt, out_dtype=torch.float16),
        lambda: moe.linear(x, wt, mul=torch.ones((4, 16), device="cuda")), lambda: moe.linear(x, wt, out=torch.ones((4, 15), device="cuda")),
        lambda: moe.linear(x, wt, offsets=torch.tensor([0, 4], dtype=torch.int32, device="cuda")),
        lambda: moe.linear(x, wt[None], offsets=torch.tensor([0, 4], device="cuda")), lambda: moe.linear(x, wt[None]),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(moe.MoEError):
            f()
            raise AssertionError(f"call {i} was accepted")
    # operands that cannot move in 16-byte units
    from asynchronous_expert_execution_gb300 import _native as N
    for f in (lambda: moe.linear(x[:, :20], wt[:, :20]), lambda: moe.linear(strided(x, 3), wt), lambda: moe.linear(x, strided(wt, 4))):
        with pytest.raises(moe.MoEError) as e:
            f()
        assert e.value.status == N.MOE_ERR_UNSUPPORTED


def test_empty_batches(moe):
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    pos, w = torch.empty((0, 2), dtype=torch.int32, device="cuda"), torch.empty((0, 2), device="cuda")
    offsets, p, pair = moe.sort_experts(pos, 5)
    assert offsets.tolist() == [0] * 6 and p.shape == (0, 2) and pair.shape == (0,)
    assert moe.sort_rows(x, pos).shape == (0, 64) and moe.merge_rows(x, pos, w).shape == (0, 64)
    assert moe.merge_rows_backward(x, x, pos, w)[1].shape == (0, 2) and moe.route_backward(pos, w, w, 4).shape == (0, 4)
    assert moe.add_rms_norm(x)[0].shape == (0, 64) and moe.add_rms_norm_e4m3(x)[1].shape == (0,)
    gx, gg = moe.add_rms_norm_backward(x, x, torch.ones(64, device="cuda"))
    assert gx.shape == (0, 64) and not bool(gg.any())
    wt = torch.ones((8, 64), dtype=torch.bfloat16, device="cuda")
    assert moe.linear(x, wt).shape == (0, 8)
    # tokens, but no rows to merge: the residual, or zeros
    pos1, r = torch.full((3, 2), -1, dtype=torch.int32, device="cuda"), torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")
    assert torch.equal(moe.merge_rows(x, pos1, torch.ones((3, 2), device="cuda"), r), r) and not bool(moe.merge_rows(x, pos1).any())

"""The gradients of the product and of its epilogue against their definitions in 64 bits.

Tolerances.  u = 2^-24 is half a step of fp32.  A tensor-core sum of n products may cut a whole step, 2^-23, per addition;
a rounded sum is off by n u of its terms' absolute values; a stored result by half a step of its type, 2^-8 (bf16) or
2^-24 (fp32) of its value.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BF16, F32 = torch.bfloat16, torch.float32
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


def randn(shape, g, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def strided(t, pad):
    """The same rows `pad` elements further apart, on a base `pad` elements into its buffer; what lies between is NaN."""
    if not pad:
        return t
    buf = torch.full((t.shape[0] + 1, t.shape[1] + 2 * pad), NAN, device=t.device, dtype=t.dtype)
    v = buf[:t.shape[0], pad:pad + t.shape[1]]
    v.copy_(t)
    return v


def close(got, want, tol, what):
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), tuple(bad.nonzero()[0].tolist()), float((d / tol.clamp(min=1e-300)).nan_to_num(1e30).max()))


def spans(T, G, g, kind):
    """Ascending offsets: some groups empty, some of one row, rows before the first and behind the last of no group."""
    if kind == "one":                                # every row in one group
        at = [0] * (G // 2 + 1) + [T] * (G - G // 2)
    else:
        cut = torch.randint(0, T + 1, (G + 1,), generator=g, device="cuda").sort().values.tolist()
        at = cut if kind == "gaps" else [0] + cut[1:-1] + [T]
    return at, torch.tensor(at, dtype=torch.int32, device="cuda")


def reference(grad, x, w, at, residual=None, old_w=None, old_b=None):
    """(value, tolerance before the last rounding) of the three gradients; rows of no group: None in `live`."""
    T, N = grad.shape
    F = x.shape[1]
    dense = at is None
    at = [0, T] if dense else at
    G = len(at) - 1
    gx, tx = (torch.zeros((T, F), dtype=torch.float64, device="cuda") for _ in range(2))
    gw, tw = (torch.zeros((G, N, F), dtype=torch.float64, device="cuda") for _ in range(2))
    gb, tb = (torch.zeros((G, N), dtype=torch.float64, device="cuda") for _ in range(2))
    live = torch.zeros(T, dtype=torch.bool, device="cuda")
    for e in range(G):
        i, j = at[e], at[e + 1]
        d, v, we = grad[i:j].double(), x[i:j].double(), (w if dense else w[e]).double()
        gx[i:j], tx[i:j] = d @ we, (N * 2.0 ** -23 + 4 * U) * (d.abs() @ we.abs())
        gw[e], tw[e] = d.T @ v, ((j - i) * 2.0 ** -23 + 4 * U) * (d.abs().T @ v.abs())
        gb[e], tb[e] = d.sum(0), (j - i) * U * d.abs().sum(0)
        live[i:j] = True
    if residual is not None:
        gx[live] += residual.double()[live]
        tx += U * gx.abs()
    if dense:
        gw, tw, gb, tb = gw[0], tw[0], gb[0], tb[0]
    if old_w is not None:
        gw = gw + old_w.double()
        tw = tw + U * gw.abs()
    if old_b is not None:
        gb = gb + old_b.double()
    return live, (gx, tx), (gw, tw), (gb, tb + 2 * U * gb.abs())


def check(moe, T, F, N, G, seed, kind="cover", out=BF16, wt=F32, bias=True, residual=False, add=False, pad=0, grad_pad=0):
    g = gen(seed)
    grad, x = randn((T, N), g, BF16), randn((T, F), g, BF16)
    w = randn((G, N, F) if G else (N, F), g, BF16, 1 / math.sqrt(N))
    at, offsets = spans(T, G, g, kind) if G else (None, None)
    res = randn((T, F), g, out) if residual else None
    old_w = randn((G, N, F) if G else (N, F), g, wt) if add else None
    old_b = randn((G, N) if G else (N,), g) if add and bias else None
    live, (gx, tx), (gw, tw), (gb, tb) = reference(grad, x, w, at, res, old_w, old_b)
    grad[~live], x[~live] = NAN, NAN                 # rows of no group are not read
    start = strided(torch.full((T, F), 3.0, device="cuda", dtype=out), pad)
    got_x, got_w, got_b = moe.linear_backward(
        strided(grad, grad_pad), strided(x, 8 * (pad > 0)), w if G else strided(w, 16 * (pad > 0)), offsets, bias, residual=strided(res, pad) if residual else None,
        weight_dtype=wt, out_x=start, out_weight=old_w.clone() if add else None, out_bias=old_b.clone() if old_b is not None else None, accumulate=add)
    assert got_x is start and got_w.dtype == wt and got_w.shape == w.shape
    close(got_x[live], gx[live], tx[live] + HALF[out] * 1.01 * (gx[live].abs() + tx[live]) + 1e-300, "grad_x")
    assert bool((got_x[~live] == 3.0).all())
    close(got_w, gw, tw + HALF[wt] * 1.01 * (gw.abs() + tw) + 1e-300, "grad_w")
    if bias:
        close(got_b, gb, tb * 1.01 + 1e-300, "grad_b")
    else:
        assert got_b is None
    return got_x, got_w, got_b


DENSE = [(1, 8, 1), (1, 2880, 2880), (2, 64, 7), (3, 48, 130), (16, 128, 128), (17, 512, 64), (63, 72, 129), (64, 64, 64), (65, 80, 1000), (127, 2064, 255),
         (128, 264, 136), (200, 584, 997), (256, 1024, 512), (300, 992, 1000), (777, 592, 997), (1025, 320, 1111), (2048, 7168, 256), (4099, 136, 40),
         (8192, 64, 200), (513, 1000, 2050), (40, 7168, 2048)]


@pytest.mark.parametrize("T,F,N", DENSE)
@pytest.mark.parametrize("out,wt,residual,add,pad,grad_pad", [(BF16, F32, False, False, 0, 0), (F32, BF16, True, True, 0, 8), (BF16, BF16, True, False, 3, 5),
                                                              (F32, F32, False, True, 8, 0)])
def test_dense(moe, T, F, N, out, wt, residual, add, pad, grad_pad):
    check(moe, T, F, N, 0, T + F + N, out=out, wt=wt, residual=residual, add=add, pad=pad, grad_pad=grad_pad)


GROUPED = [(1, 64, 64, 3), (5, 72, 33, 16), (64, 128, 256, 2), (200, 584, 997, 16), (333, 208, 584, 24), (700, 64, 40, 1024), (1000, 512, 384, 7), (1500, 2880, 160, 12),
           (4096, 256, 512, 32), (2500, 320, 2048, 5), (257, 2048, 7168, 4)]


@pytest.mark.parametrize("T,F,N,G", GROUPED)
@pytest.mark.parametrize("kind", ["cover", "gaps", "one"])
@pytest.mark.parametrize("out,wt,residual,add,grad_pad", [(BF16, F32, False, False, 0), (BF16, BF16, True, True, 3), (F32, F32, True, False, 8)])
def test_grouped(moe, T, F, N, G, kind, out, wt, residual, add, grad_pad):
    check(moe, T, F, N, G, T + F + N + G, kind, out, wt, residual=residual, add=add, grad_pad=grad_pad)


@pytest.mark.parametrize("T,F,N,G", [(70, 136, 200, 0), (333, 264, 520, 5), (1030, 416, 777, 0), (2100, 512, 130, 9)])
def test_small_integers_are_exact(moe, T, F, N, G):
    """Integer operands whose sums stay below 2^24 leave no room for rounding: every product reaches its place."""
    g = gen(T)
    grad, x, w = (torch.randint(-8, 9, s, generator=g, device="cuda").to(BF16) for s in ((T, N), (T, F), (G, N, F) if G else (N, F)))
    at, offsets = spans(T, G, g, "cover") if G else (None, None)
    gx, gw, gb = moe.linear_backward(grad, x, w, offsets, True, out_dtype=F32, weight_dtype=F32)
    _, (rx, _), (rw, _), (rb, _) = reference(grad, x, w, at)
    assert torch.equal(gx.double(), rx) and torch.equal(gw.double(), rw) and torch.equal(gb.double(), rb)


@pytest.mark.parametrize("G", [0, 6])
def test_each_alone_and_again(moe, G):
    """Any of the three without the others, and equal calls: the same bits; the residual in place."""
    g = gen(4)
    T, F, N = 600, 328, 450
    grad, x, w = randn((T, N), g, BF16), randn((T, F), g, BF16), randn((G, N, F) if G else (N, F), g, BF16)
    _, offsets = spans(T, G, g, "cover") if G else (None, None)
    gx, gw, gb = moe.linear_backward(grad, x, w, offsets, True)
    again = moe.linear_backward(grad, x, w, offsets, True)
    assert all(torch.equal(p, q) for p, q in zip((gx, gw, gb), again))
    only = moe.linear_backward(grad, None, w, offsets)
    assert torch.equal(only[0], gx) and only[1] is None and only[2] is None
    only = moe.linear_backward(grad, x, None, offsets)
    assert torch.equal(only[1], gw) and only[0] is None and only[2] is None
    only = moe.linear_backward(grad, offsets=offsets, bias=True)
    assert torch.equal(only[2], gb) and only[0] is None and only[1] is None
    res = randn((T, F), g, BF16)
    plain = moe.linear_backward(grad, None, w, offsets, residual=res)[0]
    assert moe.linear_backward(grad, None, w, offsets, residual=res, out_x=res)[0] is res and torch.equal(res, plain)


def test_what_lies_behind_a_group_does_not_reach_it(moe):
    """NaN and infinities in one group's rows stay in its gradient: sums end inside a tile of 64 rows, at every place of it."""
    g = gen(6)
    F, N = 136, 264
    for n in list(range(1, 18)) + [31, 33, 47, 48, 49, 63, 64, 65, 100, 129]:
        T = n + 70
        grad, x = randn((T, N), g, BF16), randn((T, F), g, BF16)
        clean = grad.clone(), x.clone()
        grad[n:], x[n:] = float("inf"), NAN
        offsets = torch.tensor([0, n, n, T], dtype=torch.int32, device="cuda")
        for wt in (F32, BF16):
            _, gw, gb = moe.linear_backward(grad, x, None, offsets, True, weight_dtype=wt)
            _, want, wb = moe.linear_backward(clean[0][:n], clean[1][:n], bias=True, weight_dtype=wt)
            assert bool(gw[2].isnan().all()) and not bool(gw[1].any()) and not bool(gb[1].any()) and bool(gb[2].isinf().all())
            ref = clean[0][:n].double().T @ clean[1][:n].double()
            tol = (n * 2.0 ** -23 + 4 * U) * (clean[0][:n].double().abs().T @ clean[1][:n].double().abs())
            close(gw[0], ref, tol + HALF[wt] * 1.01 * (ref.abs() + tol) + 1e-300, n)
            close(want, ref, tol + HALF[wt] * 1.01 * (ref.abs() + tol) + 1e-300, n)
            assert torch.equal(gb[0], wb) or float((gb[0] - wb).abs().max()) <= n * U * float(clean[0][:n].abs().sum(0).max())


@pytest.mark.parametrize("T,F,N", [(8192, 520, 384), (6000, 1040, 136), (5000, 264, 2056)])
def test_long_fp32_sums_are_rounded_not_cut(moe, T, F, N):
    """grad_weight in fp32 sums its rows in chunks of at most 14 x 64: 56 matrix instructions, each of which may cut a whole
    step (2^-23) of its running sum, at most 28 steps on average; the chunks add with rounding."""
    g = gen(T)
    grad, x = randn((T, N), g, BF16), randn((T, F), g, BF16)
    gw = moe.linear_backward(grad, x, weight_dtype=F32)[1]
    ref = grad.double().T @ x.double()
    assert float((gw.double() - ref).norm() / ref.norm()) <= 28 * 2.0 ** -23


def test_gradients_against_differences(moe):
    """Central differences of sum(y * c) in 64 bits: y is linear in x, w and bias, so they differ from the gradient by rounding only."""
    g = gen(11)
    T, F, N = 5, 16, 9
    x, w, c = randn((T, F), g, BF16), randn((N, F), g, BF16), randn((T, N), g, BF16)
    gx, gw, gb = moe.linear_backward(c, x, w, bias=True, out_dtype=F32, weight_dtype=F32)
    f = lambda x, w, b: float(((x @ w.T + b) * c.double()).sum())   # noqa: E731
    X, W, B, step = x.double(), w.double(), torch.zeros(N, dtype=torch.float64, device="cuda"), 0.5
    for got, leaf in ((gx, X), (gw, W), (gb, B)):
        flat = leaf.view(-1)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + step
            hi = f(X, W, B)
            flat[i] = keep - step
            lo = f(X, W, B)
            flat[i] = keep
            assert abs(float(got.reshape(-1)[i]) - (hi - lo) / (2 * step)) <= 20 * 2.0 ** -23 * float(c.abs().sum()) * 4


# ------------------------------------------------------------------ the epilogue's gradient

def act_parts(z, act):
    """act(z), act'(z), and the sum of the slope's terms' absolute values, in 64 bits."""
    if act == "silu":
        s, o = torch.sigmoid(z), torch.sigmoid(-z)
        return z * s, s * (1 + z * o), s * (1 + z.abs() * o)
    if act == "gelu":
        cdf, pdf = 0.5 * torch.erfc(-z * math.sqrt(0.5)), torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return z * cdf, cdf + z * pdf, cdf + z.abs() * pdf
    if act == "relu":
        return z.clamp(min=0), (z > 0).double(), (z > 0).double()
    return z, torch.ones_like(z), torch.ones_like(z)


@pytest.mark.parametrize("T,H", [(1, 1), (1, 4096), (3, 7), (2, 8), (33, 64), (99, 137), (16, 997), (100, 2880), (5, 20001), (1000, 584)])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu"])
@pytest.mark.parametrize("dtype,mul,pad", [(BF16, True, 0), (F32, True, 0), (BF16, False, 8), (F32, False, 3), (BF16, True, 5), (F32, True, 4)])
def test_act_mul_backward(moe, T, H, act, dtype, mul, pad):
    """act within 10 u (silu) and 20 u (gelu) of its value, or 2^-15 for bf16, as linear's; the slope's terms: s and 1 - s within 8 u
    each, the normal integral 20 u and density 8 u (a square's rounding put back to first order, an exponential, a factor), or 2^-15;
    two sums and products more."""
    g = gen(T + H)
    grad, z = strided(randn((T, H), g, dtype), pad), strided(randn((T, H), g, dtype, 3.0), pad)
    m = strided(randn((T, H), g, dtype), pad) if mul else None
    gz, gm = moe.act_mul_backward(grad, z, m, act)
    d, v, md = grad.double(), z.double(), m.double() if mul else 1.0
    y, slope, mag = act_parts(v, act)
    few = 0.0 if act in ("none", "relu") else 24 * U if dtype == F32 else 2.0 ** -14
    ref = d * md * slope
    tol = few * (d * md).abs() * mag + 3 * U * ref.abs()
    close(gz, ref, tol + HALF[dtype] * 1.01 * (ref.abs() + tol) + 1e-38, "grad_z")
    if not mul:
        assert gm is None
        return
    ref = d * y
    tol = (few + 2 * U) * ref.abs()
    close(gm, ref, tol + HALF[dtype] * 1.01 * (ref.abs() + tol) + 1e-38, "grad_mul")
    # in place of any operand, in the same layout: the same bits
    for i in range(3):
        a = [strided(t.contiguous(), pad) if pad else t.clone() for t in (grad, z, m)]
        z2, m2 = moe.act_mul_backward(*a, act, out_z=a[i], out_mul=a[(i + 1) % 3])
        assert z2 is a[i] and torch.equal(z2, gz) and torch.equal(m2, gm)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_slopes_at_the_ends_of_the_range(moe, dtype, act):
    """Far out every slope is 0 or 1, at infinities too; at 0 it is a half; NaN stays, alone."""
    z = torch.tensor([[-float("inf"), -1e30, -200.0, -50.0, 0.0, 50.0, 200.0, 1e30, float("inf"), NAN]], device="cuda").to(dtype)
    one = torch.ones_like(z)
    gz, gm = moe.act_mul_backward(one, z, one, act)
    assert gz[0, 4:9].tolist() == [0.5, 1.0, 1.0, 1.0, 1.0] and bool((gz[0, :4].abs() < 1e-19).all())
    assert bool(gz[0, 9].isnan()) and bool(gm[0, 9].isnan()) and bool((gm[0, 5:9] == z[0, 5:9]).all())


def test_act_against_differences(moe):
    """Central differences in 64 bits, step 2^-10: truncation below step^2 times a sixth of the third derivative (< 1)."""
    g = gen(3)
    z, grad, m = randn((4, 33), g, F32, 2.0), randn((4, 33), g), randn((4, 33), g)
    for act in ("silu", "gelu"):
        gz, gm = moe.act_mul_backward(grad, z, m, act)
        f = lambda v: act_parts(v, act)[0]   # noqa: E731
        step = 2.0 ** -10
        diff = (f(z.double() + step) - f(z.double() - step)) / (2 * step) * (grad * m.double())
        assert float((gz.double() - diff).abs().max()) <= (step ** 2 + 60 * U) * float((grad * m).abs().max())


# ------------------------------------------------------------------ together

def layer(moe, x, gain, wr, w1, w3, w2, idx_in=None):
    """A SwiGLU layer's forward pass on the operators, and what its backward pass keeps."""
    n, h = moe.add_rms_norm(x, None, gain)
    E = wr.shape[0]
    idx, w = moe.route(moe.linear(n, wr, out_dtype=F32), 2)
    offsets, pos, _ = moe.sort_experts(idx, E)
    rows = moe.sort_rows(n, pos)
    z, up = moe.linear(rows, w1, offsets=offsets), moe.linear(rows, w3, offsets=offsets)
    act = moe.linear(rows, w1, act="silu", mul=up, offsets=offsets)
    ys = moe.linear(act, w2, offsets=offsets)
    return moe.merge_rows(ys, pos, w, residual=h), (n, h, idx, w, offsets, pos, rows, z, up, act, ys)


def layer_backward(moe, grad, kept, gain, wr, w1, w3, w2):
    n, h, idx, w, offsets, pos, rows, z, up, act, ys = kept
    grad_ys, grad_w = moe.merge_rows_backward(grad, ys, pos, w)
    grad_act, grad_w2, _ = moe.linear_backward(grad_ys, act, w2, offsets, weight_dtype=F32)
    grad_z, grad_up = moe.act_mul_backward(grad_act, z, up)
    grad_rows, grad_w1, _ = moe.linear_backward(grad_z, rows, w1, offsets, weight_dtype=F32)
    grad_rows, grad_w3, _ = moe.linear_backward(grad_up, rows, w3, offsets, residual=grad_rows, weight_dtype=F32)
    grad_logits = moe.route_backward(idx, w, grad_w, wr.shape[0])
    grad_n, grad_wr, grad_br = moe.linear_backward(grad_logits.to(BF16), n, wr, bias=True, residual=moe.sort_rows_backward(grad_rows, pos), weight_dtype=F32)
    grad_x, grad_gain = moe.add_rms_norm_backward(grad_n, h, gain, grad_h=grad)
    return grad_x, grad_gain, grad_wr, grad_br, grad_w1, grad_w3, grad_w2


def test_training_step(moe):
    """One step through router, experts and merge against autograd in 64 bits on the same choice of experts.  What is kept between operators
    is rounded to bf16: twelve such roundings of 2^-8 at most lie on the longest path, and sums of many of them are compared by norm."""
    g = gen(20)
    T, H, I, E = 200, 136, 72, 6
    x, grad = randn((T, H), g, BF16), randn((T, H), g, BF16)
    gain = 1 + 0.1 * randn((H,), g)
    wr, w1, w3, w2 = (randn(s, g, BF16, 1 / math.sqrt(s[-1])) for s in ((E, H), (E, I, H), (E, I, H), (E, H, I)))
    y, kept = layer(moe, x, gain, wr, w1, w3, w2)
    got = layer_backward(moe, grad, kept, gain, wr, w1, w3, w2)
    leaf = [t.double().detach().requires_grad_() for t in (x, gain, wr, torch.zeros(E, device="cuda"), w1, w3, w2)]
    xd, gd, wrd, br, w1d, w3d, w2d = leaf
    n = xd / (xd.square().mean(1, keepdim=True) + 1e-6).sqrt() * gd
    idx = kept[2].long()
    w = torch.softmax((n @ wrd.T + br).gather(1, idx), 1)
    ref = xd
    for k in range(2):
        e = idx[:, k]
        a = torch.einsum("th,tih->ti", n, w1d[e])
        mid = a * torch.sigmoid(a) * torch.einsum("th,tih->ti", n, w3d[e])
        ref = ref + w[:, k, None] * torch.einsum("ti,thi->th", mid, w2d[e])
    assert float(((y.double() - ref).norm() / ref.norm()).detach()) <= 12 * 2.0 ** -8
    want = torch.autograd.grad((ref * grad.double()).sum(), leaf)
    for name, p, q in zip(("x", "gain", "wr", "br", "w1", "w3", "w2"), got, want):
        assert float((p.double() - q).norm() / q.norm()) <= 12 * 2.0 ** -8, name


def test_captured_step_replays(moe):
    """The whole backward pass in a graph: replays on new values give the eager call's bits."""
    g = gen(21)
    T, H, I, E = 300, 264, 136, 5
    x, grad = randn((T, H), g, BF16), randn((T, H), g, BF16)
    gain = 1 + 0.1 * randn((H,), g)
    wr, w1, w3, w2 = (randn(s, g, BF16, 1 / math.sqrt(s[-1])) for s in ((E, H), (E, I, H), (E, I, H), (E, H, I)))
    step = lambda: layer_backward(moe, grad, layer(moe, x, gain, wr, w1, w3, w2)[1], gain, wr, w1, w3, w2)   # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2):
        x.copy_(randn((T, H), gen(seed), BF16))
        grad.copy_(randn((T, H), gen(seed + 9), BF16))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, step()))


def test_streams_at_once(moe):
    """Calls on four streams that overlap: each gives its own result, grad of odd rows (a workspace each) too."""
    g = gen(30)
    T, F, N, G = 900, 264, 333, 4
    w = randn((G, N, F), g, BF16)
    sets = []
    for i in range(4):
        _, offsets = spans(T, G, g, "cover")
        sets.append((randn((T, N), g, BF16), randn((T, F), g, BF16), offsets))
    want = [moe.linear_backward(d, x, w, o, True) for d, x, o in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s, (d, x, o) in zip(streams, sets):
            got.append(moe.linear_backward(d, x, w, o, True, stream=s))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(p, q) for p, q in zip(r, want[i % 4]))


def test_offsets_beyond_32_bits(moe):
    """The last rows of matrices of more than 2^31 elements."""
    g = gen(40)
    T, F, N = 300_000, 7200, 64
    x = randn((1, F), g, BF16).expand(T, F).contiguous()
    grad = torch.zeros((T, N), dtype=BF16, device="cuda")
    grad[-40:] = randn((40, N), g, BF16)
    w = randn((N, F), g, BF16, 0.1)
    gx, gw, gb = moe.linear_backward(grad, x, w, bias=True, weight_dtype=F32)
    _, (rx, tx), (rw, tw), (rb, tb) = reference(grad[-40:], x[-40:], w, None)
    close(gx[-40:], rx, tx + 2.0 ** -8 * 1.01 * (rx.abs() + tx) + 1e-300, "far rows")
    assert not bool(gx[:-40].any())
    close(gw, rw, tw + 2.0 ** -24 * (rw.abs() + tw) + 1e-300, "far sum")
    close(gb, rb, tb + 1e-300, "far bias")


def test_many_far_matrices(moe):
    """grad_weight of more than 2^31 elements: the last groups' matrices."""
    g = gen(41)
    T, F, N, G = 640, 2048, 1100, 1000
    at = [0] * (G - 2) + [100, 300, T]
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    grad, x = randn((T, N), g, BF16), randn((T, F), g, BF16)
    gw = moe.linear_backward(grad, x, offsets=offsets)[1]
    assert not bool(gw[:G - 3].any())
    for e in (G - 3, G - 2, G - 1):
        d, v = grad[at[e]:at[e + 1]].double(), x[at[e]:at[e + 1]].double()
        ref, tol = d.T @ v, (d.shape[0] * 2.0 ** -23 + 4 * U) * (d.abs().T @ v.abs())
        close(gw[e], ref, tol + 2.0 ** -8 * 1.01 * (ref.abs() + tol) + 1e-300, e)


def test_refusals(moe):
    g = gen(8)
    x, w, grad = randn((4, 32), g, BF16), randn((16, 32), g, BF16), randn((4, 16), g, BF16)
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    out_w = torch.zeros((16, 32), device="cuda")
    bad = [
        lambda: moe.linear_backward(grad.float(), x, w), lambda: moe.linear_backward(grad, x.float(), w), lambda: moe.linear_backward(grad, x, w.float()),
        lambda: moe.linear_backward(grad), lambda: moe.linear_backward(grad, x[:3], w), lambda: moe.linear_backward(grad, x, w[:15]),
        lambda: moe.linear_backward(grad, x, w[:, :16]), lambda: moe.linear_backward(grad, x, w, off), lambda: moe.linear_backward(grad, x, w[None]),
        lambda: moe.linear_backward(grad, x, w[None], off.long()), lambda: moe.linear_backward(grad, x, w[None], off[:1]),
        lambda: moe.linear_backward(grad, x, w, accumulate=True), lambda: moe.linear_backward(grad, x, w, bias=True, out_weight=out_w, accumulate=True),
        lambda: moe.linear_backward(grad, x, w, out_weight=out_w.half()), lambda: moe.linear_backward(grad, x, w, out_weight=out_w[:, :16]),
        lambda: moe.linear_backward(grad, x, w, weight_dtype=torch.float16), lambda: moe.linear_backward(grad, x, w, out_dtype=torch.float64),
        lambda: moe.linear_backward(grad, x, w, residual=x.float()), lambda: moe.linear_backward(grad, x, residual=x), lambda: moe.linear_backward(grad, None, w, out_weight=out_w),
        lambda: moe.linear_backward(grad, x, w, out_bias=torch.zeros(16, device="cuda")), lambda: moe.linear_backward(grad, x.cpu(), w),
        lambda: moe.linear_backward(grad, x, w, out_x=torch.zeros((4, 31), device="cuda")),
        lambda: moe.act_mul_backward(grad, grad.float()), lambda: moe.act_mul_backward(grad, grad, grad[:2]), lambda: moe.act_mul_backward(grad, grad, act="tanh"),
        lambda: moe.act_mul_backward(grad, grad, out_mul=grad), lambda: moe.act_mul_backward(grad.half(), grad.half()),
        lambda: moe.act_mul_backward(grad, grad, out_z=grad.float()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(moe.MoEError):
            f()
            raise AssertionError(f"call {i} was accepted")
    from asynchronous_expert_execution_gb300 import _native as N
    for f in (lambda: moe.linear_backward(grad, x[:, :20], w[:, :20]), lambda: moe.linear_backward(grad, strided(x, 3), w),
              lambda: moe.linear_backward(grad, x, strided(w, 4))):
        with pytest.raises(moe.MoEError) as e:
            f()
        assert e.value.status == N.MOE_ERR_UNSUPPORTED


def test_no_rows(moe):
    x, w, grad = (torch.ones(s, dtype=BF16, device="cuda") for s in ((0, 32), (16, 32), (0, 16)))
    gx, gw, gb = moe.linear_backward(grad, x, w, bias=True)
    assert gx.shape == (0, 32) and gw.shape == (16, 32) and not bool(gw.any()) and not bool(gb.any())
    old_w, old_b = torch.ones((16, 32), device="cuda"), torch.ones(16, device="cuda")
    moe.linear_backward(grad, x, w, bias=True, out_weight=old_w, out_bias=old_b, accumulate=True)
    assert bool((old_w == 1).all()) and bool((old_b == 1).all())
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    _, gw, gb = moe.linear_backward(grad, x, torch.ones((3, 16, 32), dtype=BF16, device="cuda"), off, True, weight_dtype=F32)
    assert gw.shape == (3, 16, 32) and not bool(gw.any()) and not bool(gb.any())
    assert moe.act_mul_backward(grad, grad, grad)[1].shape == (0, 16)


def test_no_wait_ran_out(moe):
    moe.ops_sync()

"""The 8-bit product with a scale per block of 128, and its quantisers, against their definitions in 64 bits.

Tolerances.  u = 2^-24 is half a step of fp32.  A block's 128 products are summed by four matrix instructions, which may cut a
whole step, 2^-23, per addition; a block's sum is scaled by a rounded product of two scales and added with rounding: the whole is within
(128 * 2^-23 + (blocks + 3) u) of the terms' absolute values.  Stored results: half a step, 2^-8 (bf16), 2^-24 (fp32), 2^-4 (e4m3).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
NAN, INF = float("nan"), float("inf")


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
    buf = torch.full((t.shape[0] + 1, t.shape[1] + 2 * pad), NAN, device=t.device).to(t.dtype)
    v = buf[:t.shape[0], pad:pad + t.shape[1]]
    v.copy_(t)
    return v


def close(got, want, tol, what):
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), tuple(bad.nonzero()[0].tolist()), float((d / tol.clamp(min=1e-300)).nan_to_num(1e30).max()))


def act64(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * 0.5 * torch.erfc(-v * math.sqrt(0.5))
    return v.clamp(min=0) if act == "relu" else v


def spread(scale, rows, n, f):
    """Scales per rows x 128 as an [n, f] matrix in 64 bits."""
    t = scale.double().repeat_interleave(128, -1)[..., :f]
    return t if rows == 1 else t.repeat_interleave(rows, -2)[..., :n, :]


def operands(T, F, N, G, g, layout="tokens"):
    """e4m3 values and scales of their own (not the quantiser's): scales spread over five binary orders."""
    KB, NB = -(-F // 128), -(-N // 128)
    x, w = randn((T, F), g, scale=2.0).to(E4M3), randn((G, N, F) if G else (N, F), g, scale=2.0).to(E4M3)
    sx = torch.exp2(5 * torch.rand((T, KB), generator=g, device="cuda") - 3)
    sw = torch.exp2(5 * torch.rand((G, NB, KB) if G else (NB, KB), generator=g, device="cuda") - 3) / math.sqrt(F)
    if layout == "tokens":
        sx = sx.t().contiguous().t()
    elif layout == "strided":
        sx = torch.cat([sx, torch.full_like(sx, NAN)], 1).repeat_interleave(2, 0)[::2, :KB]
    return x, w, sx, sw


def extras(T, N, G, what, out, g, pad=0):
    kw = {}
    if "b" in what:
        kw["bias"] = randn((G, N) if G else (N,), g)
    if "m" in what:
        kw["mul"] = strided(randn((T, N), g, out), pad)
    if "r" in what:
        kw["residual"] = strided(randn((T, N), g, out), pad)
    return kw


def reference(x, w, sx, sw, kw, act, out, at=None):
    T, F = x.shape
    N, KB = w.shape[-2], sx.shape[1]
    ref, tol = (torch.zeros((T, N), dtype=torch.float64, device="cuda") for _ in range(2))
    live = torch.zeros(T, dtype=torch.bool, device="cuda")
    for e in range(1 if at is None else len(at) - 1):
        i, j = (0, T) if at is None else (at[e], at[e + 1])
        pick = lambda t: t if at is None or t is None else t[e]              # noqa: E731
        xe, we = x[i:j].double() * spread(sx[i:j], 1, j - i, F), pick(w).double() * spread(pick(sw), 128, N, F)
        v, t = xe @ we.T, (128 * 2.0 ** -23 + (KB + 3) * U) * (xe.abs() @ we.abs().T)
        if "bias" in kw:
            b = pick(kw["bias"]).double()
            v, t = v + b, t + U * (v.abs() + b.abs())
        v, t = act64(v, act), 1.13 * t + ((20 * U if out == F32 else 2.0 ** -15) * v.abs() if act in ("silu", "gelu") else 0.0)
        if "mul" in kw:
            m = kw["mul"][i:j].double()
            v, t = v * m, t * m.abs() + U * (v * m).abs()
        if "residual" in kw:
            r = kw["residual"][i:j].double()
            v, t = v + r, t + U * (v.abs() + r.abs())
        ref[i:j], tol[i:j], live[i:j] = v, t + HALF[out] * 1.01 * (v.abs() + t) + 1e-300, True
    return ref, tol, live


def check(moe, T, F, N, G, out, act, what, layout="tokens", kind="cover", pad=0, seed=0):
    g = gen(seed + T + F + N + G)
    x, w, sx, sw = operands(T, F, N, G, g, layout)
    kw = extras(T, N, G, what, out, g, pad)
    at = offsets = None
    if G:
        at = [0] * (G // 2 + 1) + [T] * (G - G // 2) if kind == "one" else torch.randint(0, T + 1, (G + 1,), generator=g, device="cuda").sort().values.tolist()
        if kind == "cover":
            at[0], at[-1] = 0, T
        offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    ref, tol, live = reference(x, w, sx, sw, kw, act, out, at)
    start = strided(torch.full((T, N), 3.0, device="cuda", dtype=out), pad)
    y = moe.linear(strided(x, 16 * (pad > 0)), w if G else strided(w, 32 * (pad > 0)), act=act, offsets=offsets, x_scale=sx, w_scale=sw, out=start, **kw)
    assert y is start
    close(y[live], ref[live], tol[live], "blocks")
    assert bool((y[~live] == 3.0).all())
    again = strided(torch.full((T, N), 3.0, device="cuda", dtype=out), pad)
    moe.linear(x, w, act=act, offsets=offsets, x_scale=sx.contiguous(), w_scale=sw, out=again, **kw)
    assert torch.equal(again, y)                                             # the same bits again, whatever the scales' layout


CASES = [(1, 16, 1), (1, 2880, 2880), (2, 64, 7), (3, 48, 130), (4, 7168, 257), (7, 144, 997), (16, 1008, 128), (17, 512, 64), (33, 4112, 300), (64, 2880, 256),
         (65, 80, 1000), (127, 2064, 255), (128, 128, 128), (129, 256, 384), (200, 592, 416), (256, 1024, 512), (300, 992, 1000), (777, 592, 997),
         (1025, 320, 1111), (412, 80, 2824), (2251, 592, 1760), (259, 6464, 3264), (2996, 6528, 137), (70, 4240, 3640), (9, 7168, 7168), (40, 3600, 129)]


@pytest.mark.parametrize("T,F,N", CASES)
@pytest.mark.parametrize("out,act,what,layout,pad", [(BF16, "none", "", "tokens", 0), (F32, "silu", "bm", "rows", 3), (BF16, "gelu", "br", "strided", 8),
                                                     (F32, "none", "bmr", "tokens", 0), (BF16, "relu", "bmr", "tokens", 5)])
def test_dense(moe, T, F, N, out, act, what, layout, pad):
    check(moe, T, F, N, 0, out, act, what, layout, pad=pad)


@pytest.mark.parametrize("T", [1, 3, 8, 9, 15, 16])
@pytest.mark.parametrize("F,N", [(16, 9), (64, 9000), (1056, 1235), (2064, 1200), (4128, 130), (208, 2500), (7168, 2048), (7168, 6000)])
def test_few_tokens(moe, T, F, N):
    """One to 16 rows, also on the sides of the sizes at which the kernel and its tiles change."""
    check(moe, T, F, N, 0, F32 if T % 2 else BF16, "silu", "bmr", ("tokens", "rows", "strided")[T % 3], pad=T % 3)


GROUPED = [(1, 64, 64, 3), (5, 80, 33, 16), (64, 2880, 256, 32), (64, 128, 256, 2), (200, 592, 997, 16), (333, 208, 584, 24), (700, 64, 40, 1024), (1000, 512, 384, 7),
           (1500, 2880, 160, 12), (4096, 256, 512, 32), (2500, 320, 2048, 5), (257, 2048, 1500, 4), (40, 7168, 520, 12), (16, 1040, 264, 5),
           (7, 7168, 300, 20)]


@pytest.mark.parametrize("T,F,N,G", GROUPED)
@pytest.mark.parametrize("kind", ["cover", "gaps", "one"])
@pytest.mark.parametrize("out,act,what,layout,pad", [(BF16, "none", "", "tokens", 0), (F32, "silu", "bm", "rows", 0), (BF16, "gelu", "bmr", "tokens", 3)])
def test_grouped(moe, T, F, N, G, kind, out, act, what, layout, pad):
    check(moe, T, F, N, G, out, act, what, layout, kind, pad)


def test_powers_of_two_are_exact(moe):
    """Small integers under scales of powers of two whose sums stay below 2^24 steps: nothing is rounded, every block meets its scale."""
    g = gen(2)
    for T, F, N, G in ((1, 512, 300, 0), (5, 2880, 200, 0), (70, 1040, 130, 3), (300, 2064, 520, 0), (1030, 416, 777, 5)):
        x, w = (torch.randint(-8, 9, s, generator=g, device="cuda").float().to(E4M3) for s in ((T, F), (G, N, F) if G else (N, F)))
        KB, NB = -(-F // 128), -(-N // 128)
        sx = torch.exp2(torch.randint(0, 3, (T, KB), generator=g, device="cuda").float())
        sw = torch.exp2(torch.randint(-2, 1, (G, NB, KB) if G else (NB, KB), generator=g, device="cuda").float())
        at = torch.linspace(0, T, G + 1).int().tolist() if G else None
        y = moe.linear(x, w, offsets=torch.tensor(at, dtype=torch.int32, device="cuda") if G else None, x_scale=sx, w_scale=sw, out_dtype=F32)
        ref, _, _ = reference(x, w, sx, sw, {}, "none", F32, at)
        assert torch.equal(y.double(), ref)


def test_equal_scales_give_the_row_scaled_product(moe):
    """One scale for all blocks of a token and of a feature block: the product with a scale a row, to both kernels' tolerances."""
    g = gen(3)
    T, F, N = 200, 1040, 384
    x, w, _, _ = operands(T, F, N, 0, g)
    a, b = torch.rand(T, generator=g, device="cuda") + 0.5, torch.rand(3, generator=g, device="cuda") + 0.5
    rows = moe.linear(x, w, x_scale=a, w_scale=b.repeat_interleave(128), out_dtype=F32)
    blocks = moe.linear(x, w, x_scale=a[:, None].expand(T, 9), w_scale=b[:, None].expand(3, 9).contiguous(), out_dtype=F32)
    mag = (x.double().abs() * a.double()[:, None]) @ (w.double().abs() * b.double().repeat_interleave(128)[:, None]).T
    close(rows, blocks.double(), (F * 2.0 ** -23 + 128 * 2.0 ** -23 + 16 * U) * mag, "equal scales")


def test_nan_stays_in_its_token_and_feature(moe):
    """A NaN or an infinity in x, in a scale, or in rows of another group reaches its own results only; rows behind the last group, none."""
    g = gen(4)
    for T, F, N in ((5, 400, 130), (90, 272, 260), (400, 256, 300)):
        x, w, sx, sw = operands(T, F, N, 0, g)
        clean = moe.linear(x, w, x_scale=sx, w_scale=sw)
        x2, sx2 = x.clone(), sx.clone()
        x2[1, 3], sx2[T - 1, 1], sx2[2, 0] = NAN, NAN, INF
        y = moe.linear(x2, w, x_scale=sx2, w_scale=sw)
        hit = torch.zeros(T, dtype=torch.bool, device="cuda")
        hit[[1, 2, T - 1]] = True
        assert torch.equal(y[~hit], clean[~hit]) and bool(y[1].isnan().all()) and bool(y[T - 1].isnan().all()) and not bool(torch.isfinite(y[2]).any())
        n = T - 3
        x3, sx3 = x.clone(), sx.clone()
        x3[n:], sx3[n:] = NAN, NAN
        at = torch.tensor([0, n, n], dtype=torch.int32, device="cuda")
        out = torch.full((T, N), 3.0, device="cuda", dtype=BF16)
        moe.linear(x3, torch.stack([w, w]), offsets=at, x_scale=sx3, w_scale=torch.stack([sw, sw]), out=out)
        ref, tol, _ = reference(x[:n], w, sx[:n], sw, {}, "none", BF16)
        close(out[:n], ref, tol, "beside NaN")
        assert bool((out[n:] == 3.0).all())


def test_in_place(moe):
    g = gen(5)
    for T, F, N in ((3, 512, 136), (70, 256, 129), (500, 384, 640)):
        x, w, sx, sw = operands(T, F, N, 0, g)
        m, r = randn((T, N), g, BF16), randn((T, N), g, BF16)
        want = moe.linear(x, w, mul=m, residual=r, act="silu", x_scale=sx, w_scale=sw)
        for t in (0, 1):
            a = [m.clone(), r.clone()]
            assert torch.equal(moe.linear(x, w, mul=a[0], residual=a[1], act="silu", x_scale=sx, w_scale=sw, out=a[t]), want)


# ------------------------------------------------------------------ quantisers

@pytest.mark.parametrize("T,F", [(1, 1), (1, 128), (3, 7), (2, 129), (33, 64), (16, 7168), (100, 2880), (257, 584), (1000, 136), (5, 20001), (4096, 1040)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_quantize_blocks(moe, T, F, dtype, pad):
    """scale within 2 u of max / 448 (a quotient and its rounding); q within half an e4m3 step, 2^-4, of x / scale or half the smallest
    value, 2^-10; 1 / scale and a product may move x / scale by 3 u before it is rounded."""
    g = gen(T + F)
    x = randn((T, F), g) * torch.exp(2 * randn((T, 1), g))
    x[0, 0] = 0.0
    x = strided(x.to(dtype), pad)
    q, scale = moe.quantize_blocks(x)
    KB = -(-F // 128)
    assert q.dtype == E4M3 and q.shape == (T, F) and scale.shape == (T, KB) and (T == 1 or scale.stride(0) == 1)
    v = torch.nn.functional.pad(x.double(), (0, KB * 128 - F)).reshape(T, KB, 128)
    want = (v.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
    close(scale, want, 2 * U * want, "scale")
    s = spread(scale, 1, T, F)
    close(q.double() * s, x.double(), (2.0 ** -4 + 8 * U) * x.double().abs() + 1.01 * 2.0 ** -10 * s, "q")
    assert float((q.float().abs().reshape(-1).max())) == 448.0 or not bool(x.any())          # every block's largest value takes the whole range
    out = strided(torch.zeros((T, F), device="cuda").to(E4M3), 16) if pad else torch.empty_like(q)
    q2, s2 = moe.quantize_blocks(x, out=out)
    assert q2 is out and torch.equal(q2.float(), q.float()) and torch.equal(s2, scale)


@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (127, 130), (128, 128), (129, 1000), (300, 584), (2048, 1040), (3, 40, 72), (5, 256, 384), (2, 130, 7)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_weight_blocks(moe, shape, dtype):
    g = gen(sum(shape))
    w = randn(shape, g, dtype)
    N, F = shape[-2:]
    q, scale = moe.quantize_weight_blocks(w)
    NB, KB = -(-N // 128), -(-F // 128)
    assert q.shape == w.shape and scale.shape == (*shape[:-2], NB, KB) and scale.is_contiguous()
    v = torch.nn.functional.pad(w.double(), (0, KB * 128 - F, 0, NB * 128 - N)).unflatten(-2, (NB, 128)).unflatten(-1, (KB, 128))
    want = (v.abs().amax((-3, -1)) / 448).clamp(min=2.0 ** -126)
    close(scale, want, 2 * U * want, "scale")
    s = spread(scale, 128, N, F)
    close(q.double() * s, w.double(), (2.0 ** -4 + 8 * U) * w.double().abs() + 1.01 * 2.0 ** -10 * s, "q")
    if len(shape) == 2:
        q2, s2 = moe.quantize_weight_blocks(strided(w, 8))
        assert torch.equal(q2.float(), q.float()) and torch.equal(s2, scale)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantisers_of_zeros_nan_and_infinity(moe, dtype):
    x = randn((4, 400), gen(1), dtype)
    x[0, :128], x[1, 130], x[2, 399], x[3, 128:256] = 0.0, NAN, -INF, 1e-38
    q, s = moe.quantize_blocks(x)
    f = q.float()
    assert float(s[0, 0]) == 2.0 ** -126 and not bool(f[0, :128].any())
    assert bool(f[1, 128:256].isnan().all()) and bool(s[1, 1].isnan()) and bool(f[2, 384:].isnan().all()) and bool(s[2, 3].isnan())
    assert int(f.isnan().sum()) == 128 + 16 and int(s.isnan().sum()) == 2
    q, s = moe.quantize_weight_blocks(x)
    assert s.shape == (1, 4) and s.isnan().tolist() == [[False, True, False, True]]
    assert int(q.float().isnan().sum()) == 4 * 128 + 4 * 16


# ------------------------------------------------------------------ together

def test_experts_in_blocks(moe):
    """A SwiGLU layer in 8 bits, quantised here, against 64 bits on the values that the quantised operands stand for.  What lies between
    operators is rounded to bf16 and to e4m3: three roundings of 2^-8 and one of 2^-4 on the longest path, sums compared by norm."""
    g = gen(20)
    T, H, I, E = 300, 400, 272, 6
    x = randn((T, H), g, BF16)
    idx = torch.rand((T, E), generator=g, device="cuda").topk(2).indices.to(torch.int32)
    wgt = torch.full((T, 2), 0.5, device="cuda")
    (w1, s1), (w3, s3), (w2, s2) = (moe.quantize_weight_blocks(randn(s, g, BF16, 1 / math.sqrt(s[-1]))) for s in ((E, I, H), (E, I, H), (E, H, I)))
    offsets, pos, _ = moe.sort_experts(idx, E)
    rows = moe.sort_rows(x, pos)

    def step():
        q, s = moe.quantize_blocks(rows)
        up = moe.linear(q, w3, offsets=offsets, x_scale=s, w_scale=s3)
        act = moe.linear(q, w1, act="silu", mul=up, offsets=offsets, x_scale=s, w_scale=s1)
        qa, sa = moe.quantize_blocks(act)
        return q, s, moe.merge_rows(moe.linear(qa, w2, offsets=offsets, x_scale=sa, w_scale=s2), pos, wgt, residual=x)

    q, s, y = step()
    d1, d3, d2 = w1.double() * spread(s1, 128, I, H), w3.double() * spread(s3, 128, I, H), w2.double() * spread(s2, 128, H, I)
    r = q.double() * spread(s, 1, 2 * T, H)
    ref = x.double()
    for k in range(2):
        v, e = r[pos[:, k].long()], idx[:, k].long()
        a = torch.einsum("th,tih->ti", v, d1[e])
        ref = ref + 0.5 * torch.einsum("ti,thi->th", a * torch.sigmoid(a) * torch.einsum("th,tih->ti", v, d3[e]), d2[e])
    assert float((y.double() - ref).norm() / ref.norm()) <= 3 * 2.0 ** -8 + 2.0 ** -4
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()[2]
    for seed in (1, 2):
        rows.copy_(moe.sort_rows(randn((T, H), gen(seed), BF16), pos))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step()[2])


def test_streams_at_once(moe):
    g = gen(30)
    sets = [operands(T, 528, 333, 0, g) for T in (5, 60, 400, 900)]
    want = [moe.linear(x, w, x_scale=sx, w_scale=sw) for x, w, sx, sw in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [moe.linear(x, w, x_scale=sx, w_scale=sw, stream=s) for _ in range(3) for s, (x, w, sx, sw) in zip(streams, sets)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 4]) for i, y in enumerate(got))


def test_offsets_beyond_32_bits(moe):
    """The last rows of matrices of more than 2^31 elements, of x, of y, and of what is quantised."""
    g = gen(41)
    T, F, N = 300_000, 7200, 40
    x, w, sx, sw = operands(600, F, N, 0, g)
    far = torch.zeros((T, F), dtype=torch.uint8, device="cuda").view(E4M3)
    far[-600:] = x
    scales = torch.ones((57, T), device="cuda").t()
    scales[-600:] = sx
    y = moe.linear(far, w, x_scale=scales, w_scale=sw)
    ref, tol, _ = reference(x, w, sx, sw, {}, "none", BF16)
    close(y[-600:], ref, tol, "far rows")
    assert not bool(y[:-600].any())
    del far, scales
    v = torch.zeros((T, F), dtype=BF16, device="cuda")
    v[-600:] = randn((600, F), g, BF16)
    q, s = moe.quantize_blocks(v)
    q2, s2 = moe.quantize_blocks(v[-600:])
    assert torch.equal(q[-600:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[-600:], s2)
    q, s = moe.quantize_weight_blocks(v)
    q2, s2 = moe.quantize_weight_blocks(v[-96:])                             # 300,000 = 2343 * 128 + 96
    assert torch.equal(q[-96:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[-1:], s2)


def test_refusals(moe):
    g = gen(8)
    x, w, sx, sw = operands(4, 256, 130, 0, g)
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    call = lambda **kw: moe.linear(**{**dict(x=x, weight=w, x_scale=sx, w_scale=sw), **kw})   # noqa: E731
    bad = [
        lambda: call(x_scale=sx[:, :1]), lambda: call(x_scale=sx[:3]), lambda: call(x_scale=sx.double()), lambda: call(x_scale=sx.cpu()), lambda: call(w_scale=sw[:1]),
        lambda: call(w_scale=sw[:, :1]), lambda: call(w_scale=sw[0]), lambda: call(w_scale=torch.ones(130, device="cuda")), lambda: call(x_scale=sx[:, 0]),
        lambda: call(w_scale=sw.t().contiguous().t()), lambda: call(weight=w[None], offsets=off), lambda: call(weight=w[None], w_scale=sw[None]),
        lambda: call(x_scale=sx[None]), lambda: call(x=x.to(BF16), weight=w.to(BF16)), lambda: call(act="tanh"), lambda: call(w_scale=None),
        lambda: moe.quantize_blocks(x), lambda: moe.quantize_blocks(torch.ones(4, 256, device="cuda", dtype=torch.float16)), lambda: moe.quantize_blocks(sx.cpu()),
        lambda: moe.quantize_blocks(torch.ones(4, 256, device="cuda"), out=torch.ones(4, 256, device="cuda")), lambda: moe.quantize_blocks(torch.ones(4, device="cuda")),
        lambda: moe.quantize_weight_blocks(torch.ones(4, device="cuda")), lambda: moe.quantize_weight_blocks(torch.ones((2, 4, 8), device="cuda")[:, :, :4]),
        lambda: moe.quantize_weight_blocks(torch.ones((4, 8))), lambda: moe.quantize_weight_blocks(torch.ones((4, 8), device="cuda", dtype=torch.float64)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(moe.MoEError):
            f()
            raise AssertionError(f"call {i} was accepted")
    from asynchronous_expert_execution_gb300 import _native as N
    for f in (lambda: call(x=x[:, :200], weight=w[:, :200]), lambda: call(x=strided(x, 8)), lambda: call(weight=strided(w, 8))):
        with pytest.raises(moe.MoEError) as e:
            f()
        assert e.value.status == N.MOE_ERR_UNSUPPORTED


def test_no_rows(moe):
    x, w = torch.zeros((0, 256), device="cuda").to(E4M3), torch.zeros((8, 256), device="cuda").to(E4M3)
    assert moe.linear(x, w, x_scale=torch.ones((0, 2), device="cuda"), w_scale=torch.ones((1, 2), device="cuda")).shape == (0, 8)
    q, s = moe.quantize_blocks(torch.ones((0, 256), device="cuda"))
    assert q.shape == (0, 256) and s.shape == (0, 2)


def test_no_wait_ran_out(moe):
    moe.ops_sync()

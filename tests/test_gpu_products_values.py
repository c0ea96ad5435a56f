"""Values of the products' companions where rounding or the ends of the range decide them."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


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


# ------------------------------------------------------------------ quantisers

def divided(x, rows):
    """What the quantisers document, by elementary operations: scale = max(max|x| / 448, 2^-126), q = x / scale, to nearest."""
    n, f = x.shape[-2:]
    v = torch.nn.functional.pad(x.float(), (0, -f % 128, 0, -n % rows))
    v = v.reshape(*v.shape[:-2], v.shape[-2] // rows, rows, v.shape[-1] // 128, 128)
    s = (v.abs().amax((-3, -1)) / torch.full((), 448.0, device="cuda")).clamp(min=2.0 ** -126)         # by a number torch multiplies
    q = (v / s[..., :, None, :, None]).flatten(-4, -3).flatten(-2)[..., :n, :f].to(E4M3)
    return q, s


def same(moe, x, rows):
    q, s = moe.quantize_blocks(x) if rows == 1 else moe.quantize_weight_blocks(x)
    want, ws = divided(x, rows)
    assert torch.equal(s, ws)
    off = q.view(torch.uint8) != want.view(torch.uint8)
    assert not bool(off.any()), (int(off.sum()), q[off][:4].tolist(), want[off][:4].tolist(), x[off][:4].tolist())


@pytest.mark.parametrize("shape,rows", [((300, 1040), 1), ((777, 2880), 1), ((5, 20001), 1), ((384, 1040), 128), ((3, 200, 584), 128), ((130, 257), 128)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantisers_divide(moe, shape, rows, dtype):
    """Bit for bit the quotient, rounded once to fp32 and then to e4m3, as whoever divides gets it.  Nothing is left to a tolerance."""
    g = gen(sum(shape) + rows)
    same(moe, (randn(shape, g) * torch.exp(randn((*shape[:-1], 1), g))).to(dtype), rows)


def test_quantisers_divide_every_bf16(moe):
    """Every bf16 mantissa of a block's largest value against every mantissa of another, at every exponent that reaches e4m3's range:
    448 = 7 * 64, so exact ties are common."""
    m = 1 + torch.arange(128, device="cuda") / 128.0
    down = torch.exp2(-torch.arange(0, 22, device="cuda").float())
    other = (m[:, None] * down).reshape(-1)                                  # 2816 values
    other = torch.nn.functional.pad(other, (0, -other.numel() % 127)).reshape(-1, 127)
    for exponent in (0, -60, 60, -110, 110, 126, -120):                      # the scales' own range too
        big = 2.0 * m * 2.0 ** exponent if exponent < 126 else m * 2.0 ** exponent
        x = torch.empty((128, other.shape[0], 128), device="cuda")
        x[:, :, 0] = big[:, None]
        x[:, :, 1:] = other * 2.0 ** exponent
        x = x.reshape(-1, 128).to(BF16)
        same(moe, x, 1)
        same(moe, x.float(), 1)
        w = x.reshape(128, -1, 128)[::9]                                     # one largest value a block of 128 rows
        for block in w:
            same(moe, block[:128].contiguous(), 128)


def test_quantisers_divide_beside_every_tie(moe):
    """fp32 values on both sides of every border between two e4m3 values, under scales of any mantissa, those next to powers of two
    and of few bits among them."""
    g = gen(4)
    values = torch.arange(0, 127, dtype=torch.uint8, device="cuda").view(E4M3).double()
    ties = (values[1:] + values[:-1]) / 2                                    # 126
    scale = torch.cat([torch.rand(3000, generator=g, device="cuda") + 1, 1 + torch.arange(0, 64, device="cuda") * 2.0 ** -23,
                       2 - torch.arange(1, 64, device="cuda") * 2.0 ** -23, 1 + torch.arange(0, 128, device="cuda") / 128.0])
    largest = (scale.double() * 448).float()
    s = (largest / torch.full((), 448.0, device="cuda")).double()
    for step in (-2, -1, 0, 1, 2):
        x = torch.zeros((scale.numel(), 128), device="cuda")
        near = (ties * s[:, None]).float()
        x[:, 1:127] = (near.view(torch.int32) + step).view(torch.float32)
        x[:, 0] = largest
        same(moe, x, 1)


# ------------------------------------------------------------------ the epilogue's gradient

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_products_beyond_the_range_on_the_way(moe, dtype, act):
    """grad * mul may lie outside the type where grad * mul * act'(z) does not: a slope of 0 gives 0, and small slopes or factors a finite
    result.  The slope's terms' absolute values are at most 2.1 times the slope here (silu at -3), and it is within 24 u of them, u = 2^-24, or
    2^-14 in bf16; two products and the last rounding more: 55 u < 2^-18, or 2^-8 + 2^-12 < 2^-7 of the value."""
    z = torch.tensor([[-3.0, -8.0, -60.0, 5.0, -3.0, -12.0, 2.0, -2000.0]], device="cuda")
    grad = torch.tensor([[1e30, 1e25, 1e30, 1e-30, 1e-30, 1e22, 3e38, 1e30]], device="cuda")
    mul = torch.tensor([[1e9, 1e14, 1e30, 1e-14, 1e-9, 1e18, 0.5, 1e30]], device="cuda")
    t = lambda v: v.to(dtype)   # noqa: E731
    for a, b in ((grad, mul), (mul, grad)):
        gz, gm = moe.act_mul_backward(t(a), t(z), t(b), act)
        zd, ab = t(z).double(), t(a).double() * t(b).double()
        if act == "silu":
            slope, big = torch.sigmoid(zd) * (1 + zd * torch.sigmoid(-zd)), zd.abs()
        elif act == "gelu":
            slope = 0.5 * torch.erfc(-zd * math.sqrt(0.5)) + zd * torch.exp(-0.5 * zd * zd) / math.sqrt(2 * math.pi)
        else:
            slope = (zd > 0).double()
        want = ab * slope
        inside = want.abs() < 3.3e38
        assert int(inside.sum()) >= 5 and not bool(gz.isnan().any())
        assert bool(gz[~inside].isinf().all()) and bool((gz[inside].sign() == want[inside].sign()).logical_or(want[inside].abs() < 1e-37).all())
        off = (gz[inside].double() - want[inside]).abs()
        assert bool((off <= (2.0 ** -7 if dtype == BF16 else 2.0 ** -18) * want[inside].abs() + 1e-37).all()), (gz.tolist(), want.tolist())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nan_and_infinity_in_either_factor(moe, dtype):
    """As the product of the three says: NaN from NaN, and from an infinity times 0, in either order."""
    nan, inf = float("nan"), float("inf")
    a = torch.tensor([[nan, 1.0, inf, inf, -inf, inf, -2.0, 0.0, -0.5]], device="cuda").to(dtype)
    b = torch.tensor([[1.0, nan, 0.0, -2.0, -inf, 3.0, 4.0, -3.0, -4.0]], device="cuda").to(dtype)
    z = torch.tensor([[1.0, 1.0, 1.0, 1.0, 1.0, -1.0, 1.0, 1.0, 1.0]], device="cuda").to(dtype)
    for x, y in ((a, b), (b, a)):
        gz, _ = moe.act_mul_backward(x, z, y, "relu")
        assert gz.isnan().tolist()[0] == [True, True, True, False, False, True, False, False, False]
        assert gz[0, 3:5].tolist() == [-inf, inf] and gz[0, 6:].tolist() == [-8.0, 0.0, 2.0]


def test_one_tensor_for_both_outputs_is_refused(moe):
    g = gen(3)
    grad, z, mul = (randn((40, 64), g, BF16) for _ in range(3))
    for t in (z, torch.empty_like(z)):
        with pytest.raises(moe.MoEError):
            moe.act_mul_backward(grad, z, mul, out_z=t, out_mul=t)
    both = torch.empty((40, 128), dtype=BF16, device="cuda")                 # two halves of one matrix are two outputs
    a, b = moe.act_mul_backward(grad, z, mul, out_z=both[:, :64], out_mul=both[:, 64:])
    c, d = moe.act_mul_backward(grad, z, mul)
    assert torch.equal(a, c) and torch.equal(b, d)


def test_gradients_over_operands_are_refused(moe):
    """The three gradients of a call run beside each other: none is written over what another reads."""
    g = gen(6)
    grad, x, w = randn((64, 64), g, BF16), randn((64, 64), g, BF16), randn((64, 64), g, BF16)
    kept = grad.clone(), x.clone(), w.clone()
    for kw in (dict(out_x=x), dict(out_x=grad), dict(out_x=w), dict(residual=x, out_x=x), dict(out_weight=x), dict(out_weight=grad), dict(out_weight=w),
               dict(residual=x.clone(), out_weight=w, accumulate=True)):
        with pytest.raises(moe.MoEError):
            moe.linear_backward(grad, x, w, **kw)
    same_place = torch.empty_like(x)
    with pytest.raises(moe.MoEError):
        moe.linear_backward(grad, x, w, out_x=same_place, out_weight=same_place)
    assert all(torch.equal(p, q) for p, q in zip(kept, (grad, x, w)))
    a = moe.linear_backward(grad, x, w, residual=x)                          # read by two is fine
    b = moe.linear_backward(x, x, w, residual=x)
    assert torch.equal(a[0], moe.linear_backward(grad, None, w, residual=x, out_x=x.clone())[0]) and torch.equal(b[1], moe.linear_backward(x, x.clone())[1])

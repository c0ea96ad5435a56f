"""The stateless operators at the edges of their ranges, against their definitions in 64 bits.

Tolerances count half steps: u = 2^-24 for fp32, 2^-8 for a stored bf16 value, 2^-4 for a stored e4m3 value (and half its
smallest value, 2^-10, below its normal range).
"""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BOTH = (torch.bfloat16, torch.float32)


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


def close(got, want, tol, what):
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((d / tol.clamp(min=1e-300)).nan_to_num(1e30).max()))


# ------------------------------------------------------------------ norm

def test_norm_of_a_gain_whose_product_with_the_row_passes_fp32(moe):
    """h / rms is near 1 whatever h's size: only its product with the gain has to fit."""
    for H in (64, 137, 2880, 20001):
        h = torch.full((3, H), 1e17, device="cuda")
        h[1] *= 1e-3
        gain = torch.full((H,), 1e22, device="cuda")
        y, _ = moe.add_rms_norm(h, gain=gain)
        v = h.double()
        ref = v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * gain.double()
        close(y, ref, (H / 2 + 10) * U * ref, "y")


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("H", [4, 64, 137, 2880, 20001])
@pytest.mark.parametrize("size", [3e-40, 6e-39, 1e-37, 1e-36, 2e-36, 1e-20])
def test_norm_in_8_bits_of_small_rows(moe, dtype, H, size):
    """Rows far below eps keep their ratios: zeros, halves and signs in 8 bits, with a scale down to 2^-126."""
    pattern = torch.tensor([1.0, 0.0, 0.5, -0.25], device="cuda").repeat(H // 4 + 1)[:H]
    x = (torch.stack([pattern, -pattern, pattern.flip(0)]) * size).to(dtype)
    gain = torch.full((H,), 1.5, device="cuda")
    eps = 1e-6
    q, scale, _ = moe.add_rms_norm_e4m3(x, gain=gain, eps=eps)
    v = x.double()
    y = v / (v.square().mean(1, keepdim=True) + eps).sqrt() * 1.5
    want = (y.abs().amax(1) / 448).clamp(min=2.0 ** -126)
    # a product h gain below 2^-126 is off by up to 2^-150, and 1 / rms is at most 1000
    tiny = 1000 * 2.0 ** -150
    close(scale, want, (H / 2 + 16) * U * want + tiny / 448 + 2.0 ** -149, "scale")
    s = scale.double()[:, None]
    close(q.double() * s, y, (2.0 ** -4 + (H + 24) * U) * y.abs() + 1.01 * 2.0 ** -10 * s + tiny, "q")
    assert bool((q.float()[x == 0] == 0).all())


@pytest.mark.parametrize("dtype", BOTH)
def test_norm_in_8_bits_of_rows_whose_squares_pass_fp32(moe, dtype):
    """A finite row whose sum of squares is not: zeros in its own type, in 8 bits a row and a scale of NaN, and no other row."""
    for H in (64, 137, 2880, 20001):
        x = torch.randn((4, H), generator=gen(H), device="cuda").to(dtype)
        x[1], x[2] = 1e20, -3e19
        y, _ = moe.add_rms_norm(x)
        assert not bool(y[1:3].any())
        q, scale, _ = moe.add_rms_norm_e4m3(x)
        assert bool(q[1:3].float().isnan().all()) and bool(scale[1:3].isnan().all())
        assert bool(torch.isfinite(q[[0, 3]].float()).all()) and bool(torch.isfinite(scale[[0, 3]]).all())
    x = torch.ones((2, 64), dtype=dtype, device="cuda")                      # likewise a product with the gain that passes fp32
    x[1] = 1e10
    q, scale, _ = moe.add_rms_norm_e4m3(x, gain=torch.full((64,), 1e30, device="cuda"))
    assert bool(q[1].float().isnan().all()) and bool(scale[1].isnan()) and bool((q[0].float() == 448).all())


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("H", [32, 64, 1024, 16384])
@pytest.mark.parametrize("power", [-74, -70, -65, -64, -30, 0, 40])
def test_norm_backward_without_eps(moe, dtype, H, power):
    """eps = 0 and rows of +-2^power: the mean square is a power of two (down to fp32's smallest value), so 1 / rms is
    exact, and its square may pass fp32 where grad_x does not."""
    g = gen(H)
    sign = torch.where(torch.rand((4, H), generator=g, device="cuda") < 0.5, -1.0, 1.0)
    h = (sign * 2.0 ** power).to(dtype)
    grad = torch.randn((4, H), generator=g, device="cuda").to(dtype)
    gain = 1 + 0.1 * torch.randn(H, generator=g, device="cuda")
    gx, gg = moe.add_rms_norm_backward(grad, h, gain, eps=0.0)
    n, u, r = sign.double(), grad.double() * gain.double(), 2.0 ** -power
    m, mag = (u * n).mean(1, keepdim=True), (u * n).abs().mean(1, keepdim=True)
    ref = r * (u - n * m)
    tol = r * ((u.abs() + m.abs()) * 16 * U + mag * (H + 16) * U)
    # u h below 2^-126 is off by up to 2^-150 a term: r times that in m
    close(gx, ref, tol + r * r * 2.0 ** -150 + HALF[dtype] * (ref.abs() + tol), "grad_x")
    close(gg, (grad.double() * n).sum(0), 16 * U * grad.double().abs().sum(0), "grad_gain")


# ------------------------------------------------------------------ product

def of_bias(moe, v, act, out, T):
    """act(v) by a product of zeros: the pre-activation is exactly the bias."""
    x, w = torch.zeros((T, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((v.numel(), 64), dtype=torch.bfloat16, device="cuda")
    y = moe.linear(x, w, v, act=act, out_dtype=out)
    assert all(torch.equal(y[0].nan_to_num(7.0), y[i].nan_to_num(7.0)) for i in (T // 2, T - 1))
    return y[0]


# For bf16 results the fast exponential may be used: it is off by at most 2 + 1.173 |argument| steps, each at most 2^-23.
def fast(argument):
    return (3 + 1.173 * argument.abs()) * 2 * U


@pytest.mark.parametrize("out", BOTH)
@pytest.mark.parametrize("T", [1, 16, 40, 300, 2500])
def test_silu_is_rounded_once(moe, out, T):
    """v / (1 + e^-v) to the smallest values: fp32 exponential 2 steps (4 u), sum u, quotient 2 steps (4 u), product u; an e^-|v|
    below 2^-126 is off by up to 2 steps of 2^-149, |v| times that in the result.  bf16's values below 2^-126 are the multiples of
    2^-133: half of that."""
    v = torch.cat([torch.linspace(-100, 30, 1999, device="cuda"), torch.zeros(1, device="cuda")])
    d = v.double()
    ref = d * torch.sigmoid(d)
    rel = 10.1 * U if out == torch.float32 else fast(d) + 6.1 * U + HALF[out]
    least = 110 * 2.0 ** -148 + (2.0 ** -134 if out == torch.bfloat16 else 0.0)
    close(of_bias(moe, v, "silu", out, T), ref, rel * ref.abs() + least, "silu")


@pytest.mark.parametrize("out", BOTH)
@pytest.mark.parametrize("T", [1, 16, 40, 300, 2500])
def test_gelu_keeps_its_negative_tail(moe, out, T):
    """v times the normal distribution's integral: fp32 exponential and its correction 6 u, the fit 0.6 u, its variable 5 u, nine steps
    of a polynomial whose terms stay below twice its value 5 u, three products 3 u.  In bf16 the exponent, v^2 / 2, keeps its
    rounding, and the fast exponential its error."""
    v = torch.cat([torch.linspace(-12, 8, 1999, device="cuda"), torch.zeros(1, device="cuda")])
    d = v.double()
    ref = 0.5 * d * torch.erfc(-d / math.sqrt(2.0))
    rel = 20 * U if out == torch.float32 else fast(d * d / 2) + (14 + d * d / 2) * U + HALF[out] * 1.01
    close(of_bias(moe, v, "gelu", out, T), ref, rel * ref.abs(), "gelu")


def test_activations_of_infinity_and_nan(moe):
    """relu, silu and gelu at the ends: infinity, 0 or NaN as the formulas give them."""
    inf, nan = float("inf"), float("nan")
    v = torch.tensor([inf, -inf, nan, 1e30, -1e30, -0.0, 1e-30, -1e-30], device="cuda")
    for T in (1, 40, 2500):
        for out in BOTH:
            y = {a: of_bias(moe, v, a, out, T).float() for a in ("relu", "silu", "gelu")}
            small = v[6:].to(out).float()
            for a in ("silu", "gelu"):
                assert float(y[a][0]) == inf and bool(y[a][1].isnan()) and bool(y[a][2].isnan()) and float(y[a][3]) == float(v[3].to(out))
                assert float(y[a][4]) == 0 and float(y[a][5]) == 0 and bool(((y[a][6:] - small / 2).abs() <= small.abs() * 2.0 ** -7).all())
            assert float(y["relu"][0]) == inf and float(y["relu"][1]) == 0 and bool(y["relu"][2].isnan()) and not bool(y["relu"][[4, 5]].any())


@pytest.mark.parametrize("T,F,Nn", [(1, 7168, 64), (16, 7168, 500), (40, 28672, 130), (300, 28672, 256), (900, 28672, 256), (700, 14336, 2050),
                                    (300, 7168, 2056)])
def test_fp32_sums_do_not_drift(moe, T, F, Nn):
    """Operands in [1, 2) with 6 bits behind the point: every sum of up to 1024 products is below 2^12 and a multiple of 2^-12, so
    the tensor cores hold the sums of 12 k-blocks (768 products) exactly, however they cut; what is left is fp32 rounding, u of the
    result for each addition on the longest way to it: the chunks, the partial sums of up to eight CTAs, or (up to 16 rows) four
    rounds of loads and 16 warps.  One sum over all of F would cut multiples of 2^-12 to the step of the running sum, always the
    same way (over two SMs it was off by 38 u at 7168 deep, 490 u at 14336)."""
    g = gen(F)
    six = lambda s: (1 + torch.randint(0, 64, s, generator=g, device="cuda") / 64).to(torch.bfloat16)   # noqa: E731
    x, w = six((T, F)), six((Nn, F))
    y = moe.linear(x, w, out_dtype=torch.float32)
    additions = math.ceil(F / 64 / 12) + 8 if T > 16 else 4 + 16
    close(y, x.double() @ w.double().T, additions * U * (x.double() @ w.double().T), "sums of one sign")


@pytest.mark.parametrize("T,F,Nn,groups", [(1, 7168, 300, 0), (16, 7168, 520, 0), (33, 7168, 300, 0), (300, 7168, 520, 0), (1030, 7168, 777, 0),
                                           (16, 4112, 130, 6), (200, 4112, 130, 6), (900, 7168, 264, 5), (3000, 592, 1040, 12)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("epilogue", [False, True])
def test_linear_of_integers_with_epilogue_and_groups_is_exact(moe, T, F, Nn, groups, dt, epilogue):
    """Integers whose sums stay below 2^24 leave no room for rounding: long sums, per expert, with bias, mul and residual."""
    g = gen(T + F)
    shape = (groups, Nn) if groups else (Nn,)
    ints = lambda s, n: torch.randint(-n, n + 1, s, generator=g, device="cuda").float()   # noqa: E731
    x, w = ints((T, F), 8).to(dt), ints((*shape, F), 8).to(dt)
    kw = {} if dt == torch.bfloat16 else {"x_scale": torch.full((T,), 2.0, device="cuda"), "w_scale": torch.full(shape, 0.5, device="cuda")}
    at = [0, T]
    if groups:
        cut = torch.sort(torch.randint(0, T + 1, (groups - 1,), generator=g, device="cuda")).values.tolist()
        at = [0, *cut, T]
        kw["offsets"] = torch.tensor(at, dtype=torch.int32, device="cuda")
    if epilogue:
        kw.update(bias=ints(shape, 50), mul=ints((T, Nn), 3), residual=ints((T, Nn), 100))
    y = moe.linear(x, w, out_dtype=torch.float32, **kw)
    ref = torch.zeros((T, Nn), dtype=torch.float64, device="cuda")
    for e in range(max(groups, 1)):
        i, j = at[e], at[e + 1]
        v = x[i:j].double() @ (w[e] if groups else w).double().T
        if epilogue:
            v = (v + (kw["bias"][e] if groups else kw["bias"]).double()) * kw["mul"][i:j].double() + kw["residual"][i:j].double()
        ref[i:j] = v
    assert float(ref.abs().max()) < 2 ** 24 and torch.equal(y.double(), ref)


# ------------------------------------------------------------------ tensors, streams and threads

def test_sort_experts_outputs_own_their_memory(moe):
    """Three tensors, three allocations: growing one in place leaves the others alone."""
    expert = torch.randint(0, 16, (200, 4), generator=gen(1), device="cuda").to(torch.int32)
    offsets, pos, pair = moe.sort_experts(expert, 16)
    assert len({t.untyped_storage().data_ptr() for t in (offsets, pos, pair)}) == 3
    for t in (offsets, pos, pair):
        assert t.storage_offset() == 0 and t.untyped_storage().nbytes() == t.numel() * 4
    keep = offsets.clone(), pair.clone()
    pos.resize_(2000, 4).fill_(-9)
    assert torch.equal(offsets, keep[0]) and torch.equal(pair, keep[1])


def on_threads(jobs, seconds=4.0):
    """Each job again and again on a host thread and a stream of its own; the first exception of any of them."""
    errors, stop = [], threading.Event()
    start = threading.Barrier(len(jobs))

    def work(job):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                while not stop.is_set():
                    job()
                torch.cuda.current_stream().synchronize()
        except Exception as e:                                               # noqa: BLE001
            errors.append(e)
            stop.set()
    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    stop.wait(seconds)
    stop.set()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


def test_sort_experts_of_different_sizes_on_two_threads(moe):
    """Two host threads whose calls need different amounts of shared memory."""
    jobs = []
    for E in (512, 1024):
        expert = torch.randint(0, E, (20000, 2), generator=gen(E), device="cuda").to(torch.int32)
        want = [t.clone() for t in moe.sort_experts(expert, E)]

        def job(expert=expert, E=E, want=want):
            for _ in range(50):
                got = moe.sort_experts(expert, E)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        jobs.append(job)
    torch.cuda.synchronize()
    assert not on_threads(jobs)


def test_linear_of_different_lengths_on_two_threads(moe):
    """Two host threads whose products take different kernels, tiles and amounts of shared memory, from the first call on."""
    code = ("import sys, threading, torch\n"
            "import asynchronous_expert_execution_gb300 as moe\n"
            "g = torch.Generator(device='cuda').manual_seed(1)\n"
            "r = lambda *s: torch.randn(s, generator=g, device='cuda').bfloat16()\n"
            "ops = [(r(512, 7168), r(256, 7168)), (r(40, 128), r(300, 128)), (r(600, 1024), r(4096, 1024)), (r(4, 512), r(64, 512))]\n"
            "want = [x.double() @ w.double().T for x, w in ops]\n"
            "torch.cuda.synchronize()\n"
            "bar, errors = threading.Barrier(4), []\n"
            "def work(i):\n"
            "    try:\n"
            "        with torch.cuda.stream(torch.cuda.Stream()):\n"
            "            bar.wait()\n"
            "            for _ in range(300):\n"
            "                y = moe.linear(*ops[i])\n"
            "            assert float((y.double() - want[i]).norm() / want[i].norm()) < 2 ** -8\n"
            "    except Exception as e:\n"
            "        errors.append(e)\n"
            "threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]\n"
            "[t.start() for t in threads]; [t.join() for t in threads]\n"
            "moe.ops_sync()\n"
            "assert not errors, errors\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_operators_refuse_to_drop_gradients(moe):
    """The operators record nothing: a call whose result would need a gradient is refused, one without grad mode runs."""
    x = torch.randn((4, 64), device="cuda").to(torch.bfloat16)
    w = torch.randn((16, 64), device="cuda").to(torch.bfloat16)
    gain, pos, wt = torch.ones(64, device="cuda"), torch.arange(8, dtype=torch.int32, device="cuda").reshape(4, 2), torch.ones((4, 2), device="cuda")
    rows = moe.sort_rows(x, pos)
    leaf = lambda t: t.clone().requires_grad_()                              # noqa: E731
    calls = [lambda f: moe.sort_rows(f(x), pos), lambda f: moe.merge_rows(f(rows), pos, wt), lambda f: moe.merge_rows(rows, pos, f(wt)),
             lambda f: moe.merge_rows(rows, pos, wt, f(x)), lambda f: moe.merge_rows_backward(f(x), rows, pos, wt),
             lambda f: moe.merge_rows_backward(x, rows, pos, f(wt)), lambda f: moe.route_backward(pos, f(wt), wt, 16),
             lambda f: moe.sort_rows_backward(f(rows), pos), lambda f: moe.add_rms_norm(f(x)), lambda f: moe.add_rms_norm(x, f(x)),
             lambda f: moe.add_rms_norm(x, None, f(gain)), lambda f: moe.add_rms_norm_e4m3(x, x, f(gain)),
             lambda f: moe.add_rms_norm_backward(f(x), x, gain), lambda f: moe.add_rms_norm_backward(x, x, f(gain)),
             lambda f: moe.add_rms_norm_backward(x, x, gain, grad_h=f(x)), lambda f: moe.linear(f(x), w), lambda f: moe.linear(x, f(w)),
             lambda f: moe.linear(x, w, f(torch.ones(16, device="cuda"))), lambda f: moe.linear(x, w, mul=f(x[:, :16].contiguous())),
             lambda f: moe.linear(x, w, residual=f(x[:, :16].contiguous())), lambda f: moe.linear(x, w, out=f(x[:, :16].contiguous())),
             lambda f: moe.add_rms_norm(x, x, out_h=f(x))]
    for i, call in enumerate(calls):
        with pytest.raises(moe.MoEError):
            call(leaf)
            raise AssertionError(f"call {i} was accepted")
        with torch.no_grad():
            call(leaf)
        with torch.inference_mode():
            call(lambda t: t.clone())
        call(lambda t: leaf(t).detach())


def test_outputs_in_place_raise_their_version(moe):
    """Autograd finds a saved tensor that an operator wrote over."""
    x = torch.randn((4, 64), device="cuda").to(torch.bfloat16)
    w = torch.randn((64, 64), device="cuda").to(torch.bfloat16)
    pos, wt = torch.arange(8, dtype=torch.int32, device="cuda").reshape(4, 2), torch.ones((4, 2), device="cuda")
    rows = torch.randn((8, 64), device="cuda").to(torch.bfloat16)
    for write in (lambda t: moe.sort_rows(x, pos, out=t[:8]), lambda t: moe.merge_rows(rows, pos, wt, out=t[:4]),
                  lambda t: moe.sort_rows_backward(rows, pos, out=t[:4]), lambda t: moe.merge_rows_backward(x, rows, pos, wt, out=t[:8]),
                  lambda t: moe.add_rms_norm(x, x, out=t[:4]), lambda t: moe.add_rms_norm(x, x, out_h=t[:4]),
                  lambda t: moe.add_rms_norm_backward(x, x, out=t[:4]), lambda t: moe.linear(x, w, out=t[:4])):
        t = torch.randn((8, 64), device="cuda").to(torch.bfloat16)
        a = t.clone().requires_grad_()
        y = (a * t).sum()                                                    # saves t for a's gradient
        write(t)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    with torch.inference_mode():
        t = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    assert bool(moe.linear(x, w, out=t).any())                               # made without a version


def test_a_stream_of_another_device_is_refused(moe):
    class Other:
        cuda_stream = torch.cuda.current_stream().cuda_stream
        device = torch.device("cuda", torch.cuda.current_device() + 1)
        device_index = device.index
    x = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoEError):
        moe.add_rms_norm(x, stream=Other())
    y, _ = moe.add_rms_norm(x, stream=torch.cuda.ExternalStream(torch.cuda.Stream().cuda_stream))
    torch.cuda.synchronize()
    assert bool((y == 1).all())


def test_a_reported_timeout_does_not_stay(moe):
    """The bounds-checked build can latch the operators' error word: it is reported once, then clear."""
    code = ("import torch, asynchronous_expert_execution_gb300 as moe\n"
            "from asynchronous_expert_execution_gb300 import _native as N\n"
            "x = torch.ones((4, 64), dtype=torch.bfloat16, device='cuda')\n"
            "moe.add_rms_norm(x); moe.ops_sync()\n"
            "for stream in (None, torch.cuda.Stream()):\n"
            "    N.check(N.load().moe_async_debug_latch_ops_error(None), 'latch')\n"
            "    torch.cuda.synchronize()\n"
            "    try:\n"
            "        moe.ops_sync(stream=stream)\n"
            "        raise SystemExit('not reported')\n"
            "    except moe.MoEError as e:\n"
            "        assert e.status == N.MOE_ERR_TIMEOUT\n"
            "    moe.ops_sync(); moe.ops_sync(stream=stream)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env={**os.environ, "MOE_DEBUG_BOUNDS": "1"}, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr

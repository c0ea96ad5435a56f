"""The product's gradients, the block-scaled product and its quantisers at the edges of what their documentation allows: outputs in
views, other streams, offsets outside the rows, long groups in fp32, versions, replayed graphs.  Tolerances as in the operators' own tests."""
import math

import pytest
import torch

from test_gpu_linear_backward import BF16, F32, HALF, NAN, U, close, gen, randn, reference
from test_gpu_linear_blocks import operands, spread

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g
    g.build()
    import asynchronous_expert_execution_gb300 as pkg
    return pkg


@pytest.mark.parametrize("wt", [BF16, F32])
@pytest.mark.parametrize("pad", [1, 4, 8, 24])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("T,F,N", [(300, 264, 520), (1000, 1032, 2050), (70, 2048, 2880)])
def test_weight_gradient_into_a_view(moe, wt, pad, add, T, F, N):
    """grad_weight into part of a larger matrix, on 16-byte boundaries or off them: what lies around it stays."""
    g = gen(T + pad)
    grad, x = randn((T, N), g, BF16), randn((T, F), g, BF16)
    buf = torch.full((N + 2, F + 2 * pad), 7.0, device="cuda", dtype=wt)
    view = buf[1:N + 1, pad:pad + F]
    old = randn((N, F), g, wt)
    view.copy_(old)
    got = moe.linear_backward(grad, x, out_weight=view, accumulate=add)[1]
    _, _, (gw, tw), _ = reference(grad, x, torch.zeros((N, F), dtype=BF16, device="cuda"), None, old_w=old if add else None)
    assert got is view
    close(view, gw, tw + HALF[wt] * 1.01 * (gw.abs() + tw) + 1e-300, "view")
    ring = buf.clone()
    ring[1:N + 1, pad:pad + F] = 7.0
    assert bool((ring == 7.0).all())


@pytest.mark.parametrize("wt", [BF16, F32])
def test_offsets_outside_the_rows_are_clipped(moe, wt):
    g = gen(3)
    T, F, N = 200, 144, 264
    grad, x, w = randn((T, N), g, BF16), randn((T, F), g, BF16), randn((3, N, F), g, BF16)
    wild = torch.tensor([-50, 70, 40, 100000], dtype=torch.int32, device="cuda")       # the second group descends: no rows
    tame = torch.tensor([0, 70, 70, T], dtype=torch.int32, device="cuda")
    a = moe.linear_backward(grad, x, w[:2].contiguous(), wild[:3].contiguous(), True, weight_dtype=wt)
    b = moe.linear_backward(grad, x, w[:2].contiguous(), tame[:3].contiguous(), True, weight_dtype=wt)
    assert torch.equal(a[0][:70], b[0][:70]) and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    assert not bool(a[1][1].any())
    q, sx = moe.quantize_blocks(x)
    v, sw = moe.quantize_weight_blocks(w)
    out = [torch.zeros((T, N), dtype=BF16, device="cuda") for _ in range(2)]
    for o, at in zip(out, (wild[:3], tame[:3])):
        moe.linear(q, v[:2].contiguous(), offsets=at.contiguous(), x_scale=sx, w_scale=sw[:2].contiguous(), out=o)
    assert torch.equal(out[0], out[1])


@pytest.mark.parametrize("wt,add", [(F32, False), (F32, True), (BF16, False), (BF16, True)])
def test_groups_of_every_length(moe, wt, add):
    """Groups of 0 to 3000 rows side by side, in no order of length: tiles of no k-block, of one, and of several chunks of a fp32 sum."""
    g = gen(9)
    sizes = [0, 3000, 1, 64, 0, 63, 65, 768, 769, 16, 1500, 0, 17, 833, 2, 48]
    T, F, N, G = sum(sizes), 520, 392, len(sizes)
    at = [0]
    for n in sizes:
        at.append(at[-1] + n)
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    grad, x = randn((T, N), g, BF16), randn((T, F), g, BF16)
    old = randn((G, N, F), g, wt) if add else None
    got = moe.linear_backward(grad, x, offsets=offsets, weight_dtype=wt, out_weight=old.clone() if add else None, accumulate=add)[1]
    _, _, (gw, tw), _ = reference(grad, x, torch.zeros((G, N, F), dtype=BF16, device="cuda"), at, old_w=old)
    close(got, gw, tw + HALF[wt] * 1.01 * (gw.abs() + tw) + 1e-300, "every length")
    if add:                                          # a group without rows: the same bits
        for e in (0, 4, 11):
            assert torch.equal(got[e], old[e])


def test_fp32_accumulation_over_micro_batches(moe):
    """Eight micro-batches added up: as the sum of their own gradients, each addition rounded once."""
    g = gen(12)
    F, N = 264, 520
    total = torch.zeros((N, F), device="cuda")
    bias = torch.zeros(N, device="cuda")
    ref, mag = torch.zeros((N, F), dtype=torch.float64, device="cuda"), torch.zeros((N, F), dtype=torch.float64, device="cuda")
    for T in (100, 257, 64, 1, 900, 33, 128, 500):
        grad, x = randn((T, N), g, BF16), randn((T, F), g, BF16)
        moe.linear_backward(grad, x, bias=True, out_weight=total, out_bias=bias, accumulate=True)
        ref += grad.double().T @ x.double()
        mag += (T * 2.0 ** -23 + 4 * U) * (grad.double().abs().T @ x.double().abs()) + U * ref.abs() * 1.01
    close(total, ref, mag, "micro-batches")


def test_views_versions_and_grad_mode(moe):
    """Outputs that are handed in raise their version; a tensor that requires grad is refused while grad mode is on."""
    g = gen(5)
    grad, x, w = randn((40, 72), g, BF16), randn((40, 64), g, BF16), randn((72, 64), g, BF16)
    outs = torch.empty((40, 64), dtype=BF16, device="cuda"), torch.empty((72, 64), device="cuda"), torch.empty(72, device="cuda")
    before = [t._version for t in outs]
    moe.linear_backward(grad, x, w, bias=True, out_x=outs[0], out_weight=outs[1], out_bias=outs[2])
    assert all(t._version > v for t, v in zip(outs, before))
    z = randn((40, 72), g, BF16)
    oz, om = torch.empty_like(z), torch.empty_like(z)
    moe.act_mul_backward(grad, z, z, out_z=oz, out_mul=om)
    q = torch.empty((40, 64), device="cuda").to(E4M3)
    v = q._version
    moe.quantize_blocks(x, out=q)
    assert oz._version > 0 and om._version > 0 and q._version > v
    w.requires_grad_()
    for f in (lambda: moe.linear_backward(grad, x, w), lambda: moe.quantize_weight_blocks(w), lambda: moe.act_mul_backward(w, w)):
        with pytest.raises(moe.MoEError):
            f()
        with torch.no_grad():
            f()


def test_streams_of_their_own(moe):
    """stream=: work and new outputs belong to that stream; events and stream contexts give the same."""
    g = gen(6)
    s = torch.cuda.Stream()
    grad, x, w = randn((500, 333), g, BF16), randn((500, 264), g, BF16), randn((333, 264), g, BF16)
    want = moe.linear_backward(grad, x, w, bias=True)
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.linear_backward(grad, x, w, bias=True, stream=s)
    q, sc = moe.quantize_blocks(x, stream=s)
    with torch.cuda.stream(s):
        again = moe.linear_backward(grad, x, w, bias=True)
        q2, sc2 = moe.quantize_blocks(x)
    s.synchronize()
    for a in (got, again):
        assert all(torch.equal(p, r) for p, r in zip(a, want))
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(sc, sc2)

    class Elsewhere:
        cuda_stream, device_index = 0, 7
    for f in (lambda: moe.linear_backward(grad, x, w, stream=Elsewhere()), lambda: moe.quantize_blocks(x, stream=Elsewhere()),
              lambda: moe.act_mul_backward(grad, grad, stream=Elsewhere()), lambda: moe.quantize_weight_blocks(w, stream=Elsewhere())):
        with pytest.raises(moe.MoEError):
            f()


def test_two_graphs_replayed_at_once(moe):
    """Two captured calls, each with its workspace, replayed on streams that overlap."""
    g = gen(7)
    sets = [(randn((700, 333), g, BF16), randn((700, 264), g, BF16), randn((333, 264), g, BF16)) for _ in range(2)]
    want = [moe.linear_backward(*t, bias=True, weight_dtype=F32) for t in sets]
    graphs, outs = [], []
    for t in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(moe.linear_backward(*t, bias=True, weight_dtype=F32))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for o, r in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(o, r))


@pytest.mark.parametrize("T,F,N,G", [(300, 264, 520, 0), (2048, 1024, 256, 0), (700, 520, 333, 5), (64, 2048, 2048, 0)])
def test_what_comes_before_and_after_in_the_stream(moe, T, F, N, G):
    """The three gradients of a call run beside each other, behind what made their inputs, and what follows finds all of them done: inputs
    written just before, and overwritten by other operators just after, eagerly and in a graph."""
    g = gen(T + N)
    src = [randn((T, N), g, BF16), randn((T, F), g, BF16)]
    w = randn((G, N, F) if G else (N, F), g, BF16)
    offsets = torch.linspace(0, T, G + 1).int().cuda() if G else None
    want = moe.linear_backward(*src, w, offsets, True, weight_dtype=F32)
    torch.cuda.synchronize()
    grad, x = (torch.zeros_like(t) for t in src)

    def step():
        for a, b in ((grad, src[0]), (x, src[1])):
            moe.act_mul_backward(b, b, act="none", out_z=a)                  # grad_z = grad: a copy, as the operator before
        r = moe.linear_backward(grad, x, w, offsets, True, weight_dtype=F32)
        for t in (grad, x):                                                  # in place, by the operator behind
            moe.act_mul_backward(t, torch.full_like(t, -1.0), act="relu", out_z=t)
        return r, [t.clone() for t in r]

    for _ in range(20):
        r, copies = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(r, want)) and all(torch.equal(p, q) for p, q in zip(copies, want))
        assert not bool(grad.any()) and not bool(x.any())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, copies = step()
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(r, want)) and all(torch.equal(p, q) for p, q in zip(copies, want))


@pytest.mark.parametrize("T", [1, 17, 64, 65, 129, 255, 256, 257, 300, 511, 513])
@pytest.mark.parametrize("N", [255, 256, 264, 384, 520, 2050])
def test_blocks_around_a_tile(moe, T, N):
    """Tokens and features on the sides of the tiles of either kernel, in fp32, where every feature block has a scale of its own."""
    g = gen(T + N)
    F = 720
    x, w, sx, sw = operands(T, F, N, 0, g)
    y = moe.linear(x, w, x_scale=sx, w_scale=sw, out_dtype=F32)
    xd, wd = x.double() * spread(sx, 1, T, F), w.double() * spread(sw, 128, N, F)
    close(y, xd @ wd.T, (128 * 2.0 ** -23 + 9 * U) * (xd.abs() @ wd.abs().T), "around a tile")


@pytest.mark.parametrize("out", [BF16, F32])
def test_blocks_with_many_groups(moe, out):
    """1024 experts, most of them without a row, one of several tiles."""
    g = gen(22)
    T, F, N, G = 900, 256, 130, 1024
    of = torch.randint(0, G, (T,), generator=g, device="cuda")
    of[:400] = 5
    of = of.sort().values
    at = torch.searchsorted(of, torch.arange(G + 1, device="cuda")).to(torch.int32)
    x, _, sx, _ = operands(T, F, N, 0, g)
    w = torch.randint(-8, 9, (G, N, F), generator=g, device="cuda").float().to(E4M3)
    sw = torch.exp2(torch.randint(-3, 1, (G, 2, 2), generator=g, device="cuda").float()) / 64
    y = moe.linear(x, w, offsets=at, x_scale=sx, w_scale=sw, out_dtype=out)
    xd = x.double() * spread(sx, 1, T, F)
    f = torch.repeat_interleave(torch.repeat_interleave(sw.double(), 128, 1)[:, :N], 128, 2)
    wd = (w.double() * f)[of]
    ref, mag = torch.einsum("tf,tnf->tn", xd, wd), torch.einsum("tf,tnf->tn", xd.abs(), wd.abs())
    t = (128 * 2.0 ** -23 + 5 * U) * mag
    close(y, ref, t + HALF[out] * 1.01 * (ref.abs() + t) + 1e-300, "many groups")


def test_blocks_scales_at_the_ends_of_the_range(moe):
    """Products of scales of 2^-126 and 2^100 stay finite; a block of zeros under the smallest scale adds nothing."""
    x, w = torch.ones((130, 256), device="cuda").to(E4M3), torch.ones((256, 256), device="cuda").to(E4M3)
    sx, sw = torch.full((130, 2), 2.0 ** -126, device="cuda"), torch.full((2, 2), 2.0 ** 100, device="cuda")
    y = moe.linear(x, w, x_scale=sx, w_scale=sw, out_dtype=F32)
    assert bool((y == 256 * 2.0 ** -26).all())
    z = torch.zeros((130, 256), device="cuda", dtype=BF16)
    q, s = moe.quantize_blocks(z)
    assert bool((s == 2.0 ** -126).all()) and not bool(moe.linear(q, w, x_scale=s, w_scale=sw).any())


def test_no_wait_ran_out(moe):
    moe.ops_sync()

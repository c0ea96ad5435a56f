"""grad_weight over many groups of every length, on the kernel whose two CTAs share an operand: what lies behind a group's end does not
reach it, whatever it is.

Tolerances as for the gradients themselves: u = 2^-24; a tensor-core sum of n products may cut a whole step, 2^-23, per addition; a stored
result is off by half a step of its type."""
import pytest
import torch

from test_gpu_linear_backward import BF16, F32, HALF, NAN, U, close, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g
    g.build()
    import asynchronous_expert_execution_gb300 as pkg
    return pkg


def lengths(G):
    """Every remainder of 16 and of 64 among them, empty groups too."""
    return [(7 * i + 3) % 131 for i in range(G)]


@pytest.mark.parametrize("wt,G,F,N", [(F32, 64, 264, 520), (BF16, 64, 264, 520), (F32, 56, 136, 1000), (BF16, 72, 520, 270)])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("fill", [NAN, float("inf"), 3e38])
def test_what_lies_behind_a_group_does_not_reach_it(moe, wt, G, F, N, add, fill):
    """Every other group holds NaN, infinities or the largest numbers: the others' gradients keep their bits, call after call.

    The sizes leave no other kernel: the tiles of 128 x 64 that a CTA of its own would take are more than the GPU has room for, with over
    3,072 rows, more than such a CTA's four sums in fp32, or, in bf16, twice as many rounds of dearer k-blocks."""
    g = gen(G + F + N)
    n = lengths(G)
    at = [0]
    for k in n:
        at.append(at[-1] + k)
    T = at[-1] + 5
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    grad, x = randn((T, N), g, BF16), randn((T, F), g, BF16)
    old = randn((G, N, F), g, wt) if add else None
    call = lambda d, v: moe.linear_backward(d, v, offsets=offsets, weight_dtype=wt, out_weight=old.clone() if add else None, accumulate=add)[1]   # noqa: E731
    clean = call(grad, x)
    for e in range(G):
        d, v = grad[at[e]:at[e + 1]].double(), x[at[e]:at[e + 1]].double()
        ref, tol = d.T @ v, (n[e] * 2.0 ** -23 + 4 * U) * (d.abs().T @ v.abs())
        if add:
            ref = ref + old[e].double()
            tol = tol + U * ref.abs()
        close(clean[e], ref, tol + HALF[wt] * 1.01 * (ref.abs() + tol) + 1e-300, ("clean", e))
    for odd in (0, 1):
        d, v = grad.clone(), x.clone()
        for e in range(odd, G, 2):
            d[at[e]:at[e + 1]], v[at[e]:at[e + 1]] = fill, -fill
        d[at[-1]:], v[at[-1]:] = fill, fill                                  # of no group
        for _ in range(10):
            got = call(d, v)
            for e in range(1 - odd, G, 2):
                assert torch.equal(got[e], clean[e]), (odd, e, n[e])


@pytest.mark.parametrize("wt", [F32, BF16])
def test_groups_of_every_remainder(moe, wt):
    """One to 64 rows behind two full blocks of 64, and alone, integers: exact."""
    g = gen(5)
    n = [128 * (i % 2) + i for i in range(1, 65)]
    G, F, N = len(n), 264, 300
    at = [0]
    for k in n:
        at.append(at[-1] + k)
    T = at[-1]
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    grad, x = (torch.randint(-3, 4, s, generator=g, device="cuda").to(BF16) for s in ((T, N), (T, F)))
    got = moe.linear_backward(grad, x, offsets=offsets, weight_dtype=wt)[1]
    for e in range(G):
        ref = grad[at[e]:at[e + 1]].double().T @ x[at[e]:at[e + 1]].double()
        assert torch.equal(got[e], ref.to(wt)), (e, n[e])


def test_no_wait_ran_out(moe):
    moe.ops_sync()

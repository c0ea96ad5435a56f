"""fp32 results of the products' gradients are summed in chunks of 12 k-blocks of 64, which add with rounding, because the tensor cores' own
sums cut: an unbroken sum's error grows with its length.

The limit.  Of the result's norm, a sum of 7168 in one piece is 2.6e-6 off, in chunks of 12 k-blocks 7.2e-7, and plain fp32 products are 2e-7 to 9e-7
(the figures beside the kernels' chunk length; 448 and 48 instructions, each of which cuts up to a step, 2^-23, of what it adds to).
Twice the chunked figure, 12 * 2^-23 = 1.43e-6, leaves out an unbroken sum of 8192 (448 instructions' 2.6e-6 times 512 / 448: 3.0e-6) and
one of 32768 (four times that); the chunks' own sum of 43 adds less than sqrt(43) * 2^-25 = 2e-7."""
import math

import pytest
import torch

from test_gpu_linear_backward import BF16, F32, gen, randn

pytestmark = pytest.mark.gpu
LIMIT = 12 * 2.0 ** -23


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g
    g.build()
    import asynchronous_expert_execution_gb300 as pkg
    return pkg


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("T,F,N", [(8192, 264, 136), (8192, 1040, 520), (24576, 264, 136), (32768, 264, 136), (32768, 2064, 1024), (65536, 136, 64)])
@pytest.mark.parametrize("groups", [0, 1, 3])
def test_weights(moe, T, F, N, groups):
    """Many rows, dense and all in one of several groups."""
    g = gen(T + F + groups)
    grad, x = randn((T, N), g, BF16), randn((T, F), g, BF16)
    offsets = torch.tensor([0] * (groups // 2 + 1) + [T] * (groups - groups // 2), dtype=torch.int32, device="cuda") if groups else None
    got = moe.linear_backward(grad, x, offsets=offsets, weight_dtype=F32)[1]
    if groups:
        assert not bool(got[:groups // 2].any()) and not bool(got[groups // 2 + 1:].any())
        got = got[groups // 2]
    assert off(got, grad.double().T @ x.double()) <= LIMIT


@pytest.mark.parametrize("T,F,N", [(64, 264, 8192), (300, 520, 8192), (40, 136, 24576), (300, 264, 32768), (2048, 1032, 32768)])
@pytest.mark.parametrize("groups", [0, 2])
def test_rows(moe, T, F, N, groups):
    """Many outputs."""
    g = gen(T + N + groups)
    grad, w = randn((T, N), g, BF16), randn((groups, N, F) if groups else (N, F), g, BF16, 1 / math.sqrt(N))
    offsets = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda") if groups else None
    got = moe.linear_backward(grad, None, w, offsets, out_dtype=F32)[0]
    want = grad.double() @ w.double() if not groups else torch.cat([grad[:T // 3].double() @ w[0].double(), grad[T // 3:].double() @ w[1].double()])
    assert off(got, want) <= LIMIT


@pytest.mark.parametrize("T,F,N", [(8192, 264, 136), (32768, 264, 136)])
def test_sums_of_one_sign(moe, T, F, N):
    """Where all terms are positive, cuts all go one way: in one piece a sum of 512 or 2048 instructions, whose running sum is half its end on
    average, loses half a step of it at a time, 128 or 512 steps of the end in all; in chunks of 48 that lose a whole step each time at most 24
    steps of a chunk's end, and the chunks' sum T / 768 roundings of u."""
    g = gen(T)
    grad, x = randn((T, N), g, BF16).abs(), randn((T, F), g, BF16).abs()
    want = grad.double().T @ x.double()
    got = moe.linear_backward(grad, x, weight_dtype=F32)[1]
    assert off(got, want) <= 48 * 2.0 ** -23 * 0.5 + math.ceil(T / 768) * 2.0 ** -24

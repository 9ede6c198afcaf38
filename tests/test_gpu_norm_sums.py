"""The block norms' sums over tokens, on inputs in which every token's share can be told."""
import pytest
import torch

import moe_grouped_gemm_02_amd as fg
from fgtest import dev
from normref import U32

pytestmark = pytest.mark.gpu


LONG = [(1, 8), (3, 128), (16390, 128), (16391, 120), (9001, 256), (4099, 64), (5001, 200), (2051, 1000), (1025, 512), (1100, 1032),
        (701, 2048), (530, 2304), (300, 7168), (70, 8200), (515, 16384)]


@pytest.mark.parametrize("T,N", LONG)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_token_is_in_a_channel_gates_gradient(T, N, dtype):
    """Without norms dgate = beta sum_t dr y. Whole numbers of a few bits: their sums stay below 2^24 and are exact in
    any order, so a token that is left out or taken twice shows."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    dr = torch.randint(-8, 9, (T, N), device=dev(), generator=gen)
    y = torch.randint(1, 5, (T, N), device=dev(), generator=gen)
    got = fg.block_norm_grad(y.to(dtype), dr=dr.to(dtype), y=y.to(dtype), gate=torch.ones(N, device=dev()), beta=0.5)[2]
    assert torch.equal(got.double(), 0.5 * (dr * y).sum(0).double())


def chain(T, N):
    """The roundings that a term of a sum over tokens goes through at most: the steps of a workgroup, whose rows follow
    one another (up to four a step, added across lanes at the end), then its own of 64 threads' parts, 16 of these, and
    2 last steps. The workspace holds two rows of N a workgroup."""
    groups = fg._block_norm_grad_workspace(T, N) // (8 * N)
    return -(-T // groups) + 2 + -(-groups // 64) + 16 + 2


@pytest.mark.parametrize("T,N", LONG)
def test_every_token_is_in_the_norms_weights_gradients(T, N):
    """r and y of +-1: rms 1, r / rms(r) = +-1 to the rounding of the statistics, so dpre = sum dh (+-1) and dpost = beta
    sum dr (+-1) of whole numbers from 1 to 8. Bound: the roundings of a term on its way (chain) and of its factors (a
    dozen: the sum of N ones is exact, 1 / N, the product, the root, the division and four products), of the terms' absolute
    sum. It is below 1, the least that a token adds."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    sign = lambda: torch.randint(0, 2, (T, N), device=dev(), generator=gen) * 2 - 1  # noqa: E731
    r, y = sign(), sign()
    dh, dr = (torch.randint(1, 9, (T, N), device=dev(), generator=gen) for _ in range(2))
    one = torch.ones(N, device=dev())
    f = lambda v: v.float()  # noqa: E731
    bound = (chain(T, N) + 12) * U32
    _, _, _, dpre, _ = fg.block_norm_grad(f(r), dh=f(dh), pre=one, eps=1e-30)
    tol = bound * dh.sum(0).double()
    assert float(tol.max()) < 1
    assert bool(((dpre.double() - (dh * r).sum(0)).abs() <= tol).all())
    _, _, _, _, dpost = fg.block_norm_grad(f(r), dr=f(dr), y=f(y), post=one, beta=1.0, eps=1e-30)
    tol = bound * dr.sum(0).double()
    assert float(tol.max()) < 1
    assert bool(((dpost.double() - (dr * y).sum(0)).abs() <= tol).all())


@pytest.mark.parametrize("T,N", [(16390, 128), (16389, 128), (9001, 256), (2051, 1000), (530, 2304), (70, 8200)])
def test_a_single_tokens_share(T, N):
    """dh of one token only: the sums are its terms, to the statistics' rounding (58 / 2 + 6 u of normref's rstd)."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    r = torch.randn(T, N, device=dev(), generator=gen)
    one = torch.ones(N, device=dev())
    for t in {0, 1, T // 2, T - 5, T - 4, T - 3, T - 2, T - 1}:
        dh = torch.zeros(T, N, device=dev())
        dh[t] = torch.rand(N, device=dev(), generator=gen) + 0.5
        dpre = fg.block_norm_grad(r, dh=dh, pre=one)[3].double()
        v = r[t].double()
        want = dh[t].double() * v * (v.square().mean() + 1e-6).rsqrt()
        assert bool(((dpre - want).abs() <= 40 * U32 * want.abs()).all()), t

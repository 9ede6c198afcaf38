"""The block norms' gradient where a block's output holds infinities and NaN and has no norm of its own."""
import pytest
import torch

import moe_grouped_gemm_02_amd as fg
from fgtest import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N", [(6, 64), (5, 256), (7, 1032), (3, 8200)])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_infinite_output_of_a_block_without_post(T, N, gate, dtype):
    """Without post dy = beta gate dR whatever y holds."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    new = lambda *s: torch.randn(*s, device=dev(), generator=gen)  # noqa: E731
    y, dr = new(T, N).to(dtype), new(T, N).to(dtype)
    g = {"none": None, "channel": new(N), "token": new(T, 1)}[gate]
    how = dict(dr=dr, gate=g, alpha=0.5, beta=2.0)
    want = fg.block_norm_grad(y, y=y, **how)
    bad = y.clone()
    bad[1, 3], bad[2, N - 1], bad[0, 0] = float("inf"), float("-inf"), float("nan")
    got = fg.block_norm_grad(y, y=bad, **how)
    assert torch.equal(got[0], want[0])
    assert torch.equal(got[1], want[1])
    if gate == "token":       # sum_n dR y: the rows of the three
        assert torch.equal(got[2][3:], want[2][3:]) and not bool(got[2][:3].isfinite().any())
    if gate == "channel":     # sum_t dR y: their columns
        rest = torch.ones(N, dtype=torch.bool, device=dev())
        rest[[0, 3, N - 1]] = False
        assert torch.equal(got[2][rest], want[2][rest]) and not bool(got[2][~rest].isfinite().any())

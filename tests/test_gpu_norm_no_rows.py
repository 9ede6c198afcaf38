"""The block norms' gradient of no tokens at all."""
import pytest
import torch

import moe_grouped_gemm_02_amd as fg
from fgtest import dev

pytestmark = pytest.mark.gpu


def test_no_rows_and_infinite_weights():
    """No tokens, no sums: zeros, whatever the weights hold."""
    x = torch.empty(0, 128, device=dev())
    w = torch.ones(128, device=dev())
    bad = w.clone()
    bad[3], bad[5] = float("inf"), float("nan")
    for pre, post, gate, beta in ((w, w, bad, 1.0), (w, bad, w, 1.0), (bad, bad, bad, 1.0), (w, w, w, float("inf"))):
        _, _, dgate, dpre, dpost = fg.block_norm_grad(x, dh=x.clone(), y=x.clone(), pre=pre, post=post, gate=gate, beta=beta)
        for v in (dgate, dpre, dpost):
            assert v.shape == (128,) and bool((v == 0).all())

"""Blocks whose largest value divided by its own scale amax / 448 is the float above 448 (amax / 448 was rounded down):
the row operators' encoder, which does not clamp its quotients, gives the same codes as the clamped division, of
both signs, with and without weights."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_02_amd as fg
import oracle
from fgtest import to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_largest_quotients(dtype, weighted):
    T, H = 512, 1024
    rng = np.random.default_rng(4)
    x = rng.standard_normal((T, H)).astype(np.float32)
    x = to_dev(x * 2.0 ** rng.integers(-60, 60, (T, 1)), torch.bfloat16 if dtype == "bf16" else torch.float32)
    h = x.float().cpu().numpy()
    w = rng.standard_normal((T, 1)).astype(np.float32) if weighted else None
    v = h if w is None else h * w
    blocks = v.reshape(T, H // 128, 128)
    amax = np.abs(blocks).max(2)
    top = amax / (amax / np.float32(448))
    above = top > 448
    assert above.mean() > 0.01 and np.all(top[above] == np.nextafter(np.float32(448), np.float32(449)))
    signs = np.take_along_axis(blocks, np.abs(blocks).argmax(2)[:, :, None], 2)[:, :, 0][above]
    assert (signs > 0).any() and (signs < 0).any()
    plan = fg.plan_contiguous(torch.zeros(T, 1, dtype=torch.int32, device=x.device), 1)
    Q, sa = fg.dispatch_quant(x, plan, w=None if w is None else to_dev(w))
    codes, scales = oracle.quantize_act_1x128(v, False)
    rows = plan.rows.view(-1).cpu().numpy()
    assert np.array_equal(sa.t().cpu().numpy()[rows], scales)
    assert np.array_equal(Q.cpu().numpy()[rows], codes)

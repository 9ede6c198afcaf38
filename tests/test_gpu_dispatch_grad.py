"""The gradients of dispatch's copies w x, without and with weights, against the formula in 64 bits and against the
transpose of the copies themselves."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_02_amd as fg
from fgtest import to_dev
from test_gpu_rows import PLANS, check_dw, host, make_plan, near

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


@pytest.mark.parametrize("layout,T,k,G", PLANS)
@pytest.mark.parametrize("H", [128, 2048])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_grad(layout, T, k, G, H, dtype, weighted):
    print(f"dispatch grad {layout} {T}x{k} G={G} H={H} {dtype} w={weighted}", flush=True)
    rng = np.random.default_rng(H + T)
    p = make_plan(layout, T, k, G)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    dA = to_dev(rng.standard_normal(p.lead + (H,)).astype(np.float32), td)
    x = to_dev(rng.standard_normal((T, H)).astype(np.float32), td)
    w = rng.standard_normal((T, k)).astype(np.float32) if weighted else None
    wd = None if w is None else to_dev(w)
    dx = fg.dispatch_grad(dA, p, w=wd)
    rows, d = host(p.rows), host(dA).reshape(-1, H).astype(np.float64)
    terms = d[np.maximum(rows, 0)] * np.where(rows >= 0, 1.0 if w is None else w.astype(np.float64), 0.0)[:, :, None]
    assert dx.dtype == td and np.all(near(host(dx), terms.sum(1), 2 * (k + 2) * U32 * np.abs(terms).sum(1), dtype))
    out = torch.empty_like(dx)
    assert fg.dispatch_grad(dA, p, out=out, w=wd) is out and torch.equal(out, dx)
    if weighted:     # the weights' gradient: <x[t], dA[row]>, which is combine_grad's dw
        _, dw = fg.combine_grad(x, dA, p, wd, with_dy=False)
        check_dw(host(dw), p, dA, x, H)


def test_weighted_dispatch_against_differences():
    """<copies of (x, w), dA> along random directions (bilinear: no truncation error), the copies written out in 64 bits."""
    T, k, G, H = 30, 3, 5, 128
    rng = np.random.default_rng(2)
    p = make_plan("contiguous", T, k, G)
    x, dirx = rng.standard_normal((2, T, H)).astype(np.float32)
    w, dirw = rng.standard_normal((2, T, k)).astype(np.float32)
    dA = rng.standard_normal(p.lead + (H,)).astype(np.float32)
    slots = host(p.slots)

    def value(x, w, dA):
        v = x.astype(np.float64)[np.maximum(slots, 0) // k] * w.astype(np.float64).reshape(-1)[np.maximum(slots, 0)][:, None]
        return (np.where((slots >= 0)[:, None], v, 0) * dA).sum()

    dx = host(fg.dispatch_grad(to_dev(dA), p, w=to_dev(w))).astype(np.float64)
    dw = host(fg.combine_grad(to_dev(x), to_dev(dA), p, to_dev(w), with_dy=False)[1]).astype(np.float64)
    x64, w64 = x.astype(np.float64), w.astype(np.float64)
    # the bounds of test_dispatch_grad, summed along the direction
    size = lambda x, w: value(np.abs(x), np.abs(w), np.abs(dA))  # noqa: E731
    diff = (value(x64 + dirx, w64, dA) - value(x64 - dirx, w64, dA)) / 2
    assert abs(diff - (dx * dirx).sum()) <= 2 * (k + 2) * U32 * size(dirx, w)
    diff = (value(x64, w64 + dirw, dA) - value(x64, w64 - dirw, dA)) / 2
    assert abs(diff - (dw * dirw).sum()) <= (H / 256 + 24) * U32 * size(x, dirw)

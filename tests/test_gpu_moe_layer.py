"""The example layer against the same layer in 64 bits with the experts' products taken from the library's own
operands: the routing, sorting, combining and adapters around the (separately tested) GEMMs fit together, and both
layouts give the same output."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import moe_grouped_gemm_02_amd as fg
import oracle

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs():
    out, same, dw, dlogits = example().main(["--tokens", "200", "--hidden", "512", "--inner", "256"])
    assert torch.equal(out, same)   # the GEMMs do not depend on the layout, nor does combine
    assert bool(dw.isfinite().all()) and bool(dlogits.isfinite().all())


@pytest.mark.parametrize("tokens", [1, 37, 300])
def test_layer_against_its_parts(tokens):
    """Each token's output is base + sum_j w_j expert_j(token) with the experts run densely, one by one, on all tokens:
    no sorting, no plan. The same kernels compute the products, so the sums differ by their fp32 rounding alone."""
    m = example()
    layer = m.Layer(512, 256, 8, 3, rank=16, seed=3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    x = torch.randn(tokens, 512, device="cuda", generator=gen).bfloat16()
    adapter_ids = torch.randint(-1, 3, (tokens,), device="cuda", generator=gen).to(torch.int32)
    out, (logits, ids, w, plan, y) = m.forward(layer, x, 2, adapter_ids)
    base = m.shared_with_adapters(layer, x, adapter_ids)
    A, sa = fg.quant_act_1x128(x.float())
    dense = []
    for e in range(8):
        Q, sq, _ = fg.gemm_fp8_nt_swiglu_quant(A, sa, layer.up[0][e], layer.up[1][e])
        D = torch.empty(tokens, 512, dtype=torch.bfloat16, device="cuda")
        fg.gemm_fp8_nt(Q, sq, layer.down[0][e], layer.down[1][e], D)
        dense.append(D)
    dense = torch.stack(dense).double()
    pick = dense[ids.long().t(), torch.arange(tokens, device="cuda")]          # [k, T, H]
    terms = pick * w.double().t()[:, :, None]
    ref = base.double() + terms.sum(0)
    size = base.double().abs() + terms.abs().sum(0)
    tol = 8 * 2.0 ** -24 * size
    lo, hi = (ref - tol).bfloat16(), (ref + tol).bfloat16()
    assert bool(((lo <= out) & (out <= hi)).all())
    assert np.array_equal(ids.cpu().numpy(), torch.sort(torch.sigmoid(logits) + 0.0, dim=1, descending=True, stable=True)
                          .indices[:, :2].cpu().numpy())
    # the sorted operand holds each token's own codes
    Q, _ = fg.dispatch_quant(x, plan)
    codes, _ = oracle.quantize_act_1x128(x.float().cpu().numpy())
    rows = plan.rows.cpu().numpy()
    for j in range(2):
        assert np.array_equal(Q.cpu().numpy()[rows[:, j]], codes)

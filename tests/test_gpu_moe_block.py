"""The example's block of a residual stream: it runs, its steps agree with the calls they are made of, and its
gradients are the formula's at the values that it saved."""
import os
import sys

import numpy as np
import pytest
import torch

import moe_grouped_gemm_02_amd as fg
import normref
from fgtest import dev

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu


def test_example_runs(capsys):
    moe_layer.main(["--tokens", "96", "--experts", "4", "--hidden", "512", "--inner", "256"])
    assert "block in 8-bit integers" in capsys.readouterr().out


def test_block_and_its_gradient():
    T, H, I, E = 70, 384, 256, 4
    gen = torch.Generator(device="cuda").manual_seed(2)
    new = lambda *s, fan=1: torch.randn(*s, device=dev(), generator=gen) * fan ** -0.5  # noqa: E731
    layer = moe_layer.Layer(H, I, E, 2, 8)
    up, down = fg.quant_int8(new(E, 2 * I, H, fan=H)), fg.quant_int8(new(E, H, I, fan=I))
    norms = [1 + 0.1 * new(H), 1 + 0.1 * new(H), new(H), 1 + 0.1 * new(H)]
    x = new(T, H).bfloat16()
    out, h, s, (saved, y) = moe_layer.block(layer, x, 2, norms, up, down)
    assert saved is out
    d = lambda t: t.double().cpu().numpy()  # noqa: E731
    (r, tol), (n, n_tol) = normref.forward(d(x), d(y), d(norms[3]), d(norms[1]), d(norms[2]), 1.0, 1.0, 1e-6)
    assert np.all(np.abs(d(out) - r) <= tol + np.abs(r) * 2.0 ** -8)          # one bf16 rounding
    scale = np.abs(n).max(1) / 127
    assert np.all(np.abs(d(s) - scale) <= (n_tol.max(1) / 127) + scale * 2.0 ** -23)
    assert np.all(np.abs(d(h) * d(s)[:, None] - n) <= 0.5001 * scale[:, None] + n_tol + scale[:, None] * 127 * 2.0 ** -22)
    dh, dout = new(T, H).bfloat16(), new(T, H).bfloat16()
    got = moe_layer.block_backward((saved, y), dh, dout, norms)
    ref = normref.backward(d(out), d(dh), d(dout), d(y), d(norms[3]), d(norms[1]), d(norms[2]), 1.0, 1.0, 1e-6)
    for name, v in zip(("dx", "dy", "dgate", "dpre", "dpost"), got):
        want, bound = ref[name]
        assert np.all(np.abs(d(v) - want) <= bound + np.abs(want) * (2.0 ** -8 if name in ("dx", "dy") else 2.0 ** -24)), name

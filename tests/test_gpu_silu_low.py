"""silu(gate) up as 8-bit integers where the gate's sigmoid is below the normal numbers."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_02_amd as fg
from fgtest import dev

pytestmark = pytest.mark.gpu


U32 = 2.0 ** -24


def as_values(h):
    """silu(gate) up of rows [T, 2 I] in 64 bits, where exp of 745 is the largest there is."""
    g, u = (v.reshape(len(h), -1) for v in np.split(h.astype(np.float64).reshape(len(h), -1, 2, 128), 2, axis=2))
    return g * np.exp(np.where(g < 0, g, 0)) / (1 + np.exp(-np.abs(g))) * u


# The value's error: exp2 of the hardware within 1 ulp (2 u) twice, its argument's low part and the correction's rounding
# (2 u), four products (4 u); 12 u leave room for the last steps near 1 + exp. The scale's division one more.
REL = 12 * U32


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("low,high", [(-86, -44), (-88, -86), (-90, -87), (-104, -88), (-127, -100), (-160, -120), (-172, -150)])
@pytest.mark.parametrize("I", [128, 640])
def test_gates_far_below_zero_with_large_ups(low, high, I, dtype):
    """Rows of nothing but such gates: what is left of them sets the scale."""
    rng = np.random.default_rng(int(-low))
    h = np.empty((9, I // 128, 2, 128), np.float32)
    h[:, :, 0] = rng.uniform(low, high, h[:, :, 0].shape)
    h[:, :, 1] = rng.uniform(0.1, 3.3, h[:, :, 1].shape) * 1e38 * rng.choice([-1, 1], h[:, :, 1].shape)
    t = torch.from_numpy(h.reshape(9, 2 * I)).to(dev(), dtype)
    v = as_values(t.float().cpu().numpy())
    Q, s = fg.swiglu_quant_int8(t)
    top = np.abs(v).max(1)
    scale = np.maximum(top / 127, 2.0 ** -126)
    assert np.all(np.abs(s.double().cpu().numpy() - scale) <= 2 * REL * scale)
    # half a code, the value's and the scale's errors of a quotient of at most 127, and below the normal numbers
    # half a unit of 2^-149 (2^-24 of the least scale)
    assert np.all(np.abs(Q.double().cpu().numpy() - v / scale[:, None]) <= 0.5 + 127 * 3 * REL + U32)


def test_gates_far_below_zero_beside_ordinary_ones():
    """A large product of a tiny sigmoid is the row's largest value; gate and up sit in every place of a unit."""
    for at in (0, 1, 15, 16, 63, 127):
        h = torch.zeros(2, 256)
        h[:, :128] = torch.linspace(-3, 3, 128)
        h[:, 128:] = 1.0
        h[1, at], h[1, 128 + at] = -88.0, 1e38
        Q, s = fg.swiglu_quant_int8(h.to(dev()))
        v = as_values(h.numpy())
        assert abs(v[1, at]) > 50                          # -88 exp(-88) 1e38
        for t in range(2):
            want = np.abs(v[t]).max() / 127
            assert abs(float(s[t]) - want) <= 2 * REL * want, at
            assert np.all(np.abs(Q[t].double().cpu().numpy() - v[t] / want) <= 0.5 + 127 * 3 * REL)


def test_gates_far_below_zero_at_the_ends():
    """Up infinite: so is the product, for any finite gate but zero. A gate of minus infinity: NaN, as inf / (1 + inf).
    Up zero or finite and the gate past all that 32 bits hold: zero."""
    inf, nan = float("inf"), float("nan")
    rows = [(-88.0, inf, inf), (-120.0, -inf, inf), (-300.0, inf, inf), (-3e38, inf, inf), (-inf, 1.0, nan), (-inf, 0.0, nan),
            (-88.0, nan, nan), (-500.0, nan, nan), (-300.0, 3e38, 1.0), (-3e38, 3e38, 1.0), (-200.0, 0.0, 1.0), (-88.0, 0.0, 1.0)]
    h = torch.zeros(len(rows), 256)
    for t, (g, u, _) in enumerate(rows):
        h[t, 5], h[t, 133] = g, u
    Q, s = fg.swiglu_quant_int8(h.to(dev()))
    for t, (g, u, want) in enumerate(rows):
        got = float(s[t])
        if want == 1.0:       # a row of zeros, or of nothing but a value below 2^-149
            assert got in (1.0, 2.0 ** -126) and not bool(Q[t].any()), (g, u, got)
        else:
            assert got == want or (got != got and want != want), (g, u, got)

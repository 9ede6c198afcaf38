"""Rows that hold infinities and NaN change nothing in the rows beside them, in a wave or a step: integer quantisers, block
norms and their gradient."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_02_amd as fg
from fgtest import dev

pytestmark = pytest.mark.gpu


BAD = [float("nan"), float("inf"), float("-inf")]


def spoil(v, seed):
    """v with a bad value in one row of three, and which rows those are; a step's rows hold bad and good ones."""
    rng = np.random.default_rng(seed)
    T, N = v.shape
    bad = np.zeros(T, bool)
    for t in range(1, T, 3):
        bad[t] = True
        v[t, int(rng.integers(N))] = BAD[t // 3 % len(BAD)]
    return torch.from_numpy(bad).to(v.device)


@pytest.mark.parametrize("T,N", [(31, 16), (30, 128), (29, 112), (23, 256), (22, 240), (13, 512), (9, 1024), (7, 4096)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("where", ["x", "y"])
def test_block_norms(T, N, dtype, where):
    gen = torch.Generator(device="cuda").manual_seed(N)
    new = lambda *s: torch.randn(*s, device=dev(), generator=gen)  # noqa: E731
    v = dict(x=new(T, N).to(dtype), y=new(T, N).to(dtype))
    how = dict(pre=new(N) + 2, post=new(N) + 2, gate=new(T, 1))
    dh, dr = new(T, N).to(dtype), new(T, N).to(dtype)
    w = {k: t.clone() for k, t in v.items()}
    bad = spoil(w[where], N)
    good = ~bad
    for quant in (None, "int8") + (("e4m3", "e4m3_pow2") if N % 128 == 0 else ()):
        clean, got = (fg.block_norm(a["x"], a["y"], quant=quant, **how) for a in (v, w))
        assert torch.equal(got[0][good], clean[0][good]) and torch.equal(got[1][good], clean[1][good]), quant
        if quant == "int8":
            assert torch.equal(got[2][good], clean[2][good]) and not bool(got[2][bad].isfinite().any())
        elif quant is not None:
            assert torch.equal(got[2][:, good], clean[2][:, good])
    clean, got = (fg.block_norm_grad(a["x"], dh=dh, dr=dr, y=a["y"], **how) for a in (v, w))
    for k in range(3):        # dx, dy and the tokens' gates
        assert torch.equal(got[k][good], clean[k][good]), k


@pytest.mark.parametrize("T,K", [(31, 16), (33, 128), (30, 112), (19, 256), (18, 208), (11, 512), (10, 400), (7, 1024), (5, 4096), (4, 16384)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantised_rows(T, K, dtype):
    x = torch.randn(T, K, device=dev(), generator=torch.Generator(device="cuda").manual_seed(K)).to(dtype)
    w = x.clone()
    bad = spoil(w, K)
    (q, s), (cq, cs) = fg.quant_int8(w), fg.quant_int8(x)
    assert torch.equal(q[~bad], cq[~bad]) and torch.equal(s[~bad], cs[~bad])
    assert not bool(s[bad].isfinite().any())
    if K % 128 == 0:
        up = torch.ones_like(x).view(T, -1, 128)
        both = lambda v: torch.stack([up, v.view(T, -1, 128)], 2).view(T, 2 * K)  # noqa: E731
        (q, s), (cq, cs) = fg.swiglu_quant_int8(both(w)), fg.swiglu_quant_int8(both(x))
        assert torch.equal(q[~bad], cq[~bad]) and torch.equal(s[~bad], cs[~bad]) and not bool(s[bad].isfinite().any())

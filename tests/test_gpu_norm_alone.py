"""The gradient of a norm without a block's output is the slope of its forward call, h = x / sqrt(mean x^2 + eps) pre
of x itself: alpha and beta, which belong to a block's output, are in neither."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_02_amd as fg
from fgtest import dev, to_dev
from normref import SUM, U32, rstd

pytestmark = pytest.mark.gpu

EPS = 1e-3


def definition(x, pre):
    """h in 64 bits."""
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * pre


def case(T, N, seed):
    rng = np.random.default_rng(seed)
    f32 = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    return dict(x=f32(T, N), pre=1 + 0.1 * f32(N), dh=f32(T, N), dr=f32(T, N))


@pytest.mark.parametrize("T,N", [(4, 64), (5, 200), (3, 520), (2, 2304), (3, 8200)])
@pytest.mark.parametrize("with_dr", [True, False])
def test_slope_of_the_forward_call(T, N, with_dr):
    """Central differences of the 64-bit definition, of the forward call's values as they come: the step's error is
    step^2 / 6 times a third derivative, of the gradient's own size for entries of size 1 (1e-8 of it with this step),
    and fp32's rounding of a gradient entry, normref's bound with a row's SUM roundings (some 70 u)."""
    v = case(T, N, T + N)
    g = {k: to_dev(a) for k, a in v.items()}
    how = dict(pre=g["pre"], alpha=0.75, beta=-1.5, eps=EPS)
    r, h, _ = fg.block_norm(g["x"], **how)
    d = {k: a.astype(np.float64) for k, a in v.items()}
    assert r is g["x"] and np.abs(h.double().cpu().numpy() - definition(d["x"], d["pre"])).max() < 1e-5
    dx, dy, dgate, dpre, dpost = fg.block_norm_grad(r, dh=g["dh"], dr=g["dr"] if with_dr else None, **how)
    assert dy is None and dgate is None and dpost is None
    dx, dpre = dx.double().cpu().numpy(), dpre.double().cpu().numpy()

    def loss(x, pre):
        return (definition(x, pre) * d["dh"]).sum() + ((x * d["dr"]).sum() if with_dr else 0.0)

    rng, step = np.random.default_rng(1), 1e-4
    for _ in range(20):
        t, n = rng.integers(T), rng.integers(N)
        e = np.zeros((T, N))
        e[t, n] = step
        slope = (loss(d["x"] + e, d["pre"]) - loss(d["x"] - e, d["pre"])) / (2 * step)
        assert abs(slope - dx[t, n]) <= 1e-5 * np.abs(dx[t]).max(), (t, n, slope, dx[t, n])
        e = np.zeros(N)
        e[n] = step
        slope = (loss(d["x"], d["pre"] + e) - loss(d["x"], d["pre"] - e)) / (2 * step)
        assert abs(slope - dpre[n]) <= 1e-5 * np.abs(dpre).max(), (n, slope, dpre[n])


@pytest.mark.parametrize("T,N", [(1, 8), (7, 128), (6, 256), (9, 512), (40, 1024), (70, 2048), (3, 4224), (20, 7168), (2, 16384)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_gradient_from_the_formula(T, N, dtype):
    """dx = dr + rx (z - rh mean(z rh)), z = dh pre, with normref's bound of fp32 arithmetic and the type's rounding."""
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    g = {k: to_dev(a) if k == "pre" else to_dev(a, dt) for k, a in case(T, N, N).items()}
    dx = fg.block_norm_grad(g["x"], dh=g["dh"], dr=g["dr"], pre=g["pre"], alpha=0.75, beta=3.0, eps=EPS)[0]
    d = {k: a.double().cpu().numpy() for k, a in g.items()}
    rx, e = rstd(d["x"], EPS)
    rh, z = d["x"] * rx, d["dh"] * d["pre"]
    want = d["dr"] + rx * (z - rh * (z * rh).mean(-1, keepdims=True))
    tol = rx * (np.abs(z) * (e + 4 * U32) + np.abs(rh) * np.abs(z * rh).mean(-1, keepdims=True) * (3 * e + (SUM + 8) * U32))
    tol = tol + 3 * U32 * np.abs(want) + (0 if dtype == "fp32" else 2.0 ** -8 * np.abs(want))
    assert np.all(np.abs(dx.double().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_alpha_and_beta_do_not_matter(dtype):
    g = {k: to_dev(a) if k == "pre" else to_dev(a, dtype) for k, a in case(33, 1032, 3).items()}
    for parts in (dict(dh=g["dh"], dr=g["dr"], pre=g["pre"]), dict(dh=g["dh"], pre=g["pre"]), dict(dr=g["dr"])):
        want = fg.block_norm_grad(g["x"], **parts)
        for alpha, beta in ((0.75, 1.0), (-3.0, 0.0), (0.0, 2.0)):
            got = fg.block_norm_grad(g["x"], alpha=alpha, beta=beta, **parts)
            assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(got, want)), (alpha, beta)
    assert torch.equal(want[0], g["dr"])          # without a norm the stream is x, and its gradient dr


def test_nothing_to_add_to_dr_in_place():
    dr = torch.randn(5, 136, device=dev())
    x, want = torch.randn(5, 136, device=dev()), dr.clone()
    got = fg.block_norm_grad(x, dr=dr, alpha=0.5, dx=dr)[0]
    assert got is dr and torch.equal(dr, want)

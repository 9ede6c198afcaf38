"""The sigmoid router's gradient where its scores are close to 1 or to 0. The tolerances are relative: with u = 2^-24 a
score and its complement are each off by at most 8 u of themselves (exp to 2 ulp, one sum, one division)."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_02_amd as fg
from fgtest import dev, to_dev
from test_gpu_rows import near

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


def logits_of(T, E, rng):
    """Logits of 10 to 30 and -30 to -10 beside ordinary ones."""
    l = rng.choice([-1.0, 1.0], (T, E)) * rng.uniform(10, 30, (T, E))
    return np.where(rng.random((T, E)) < 0.3, 2 * rng.standard_normal((T, E)), l).astype(np.float32)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(64, 32, 4), (40, 60, 6), (33, 256, 8), (8200, 64, 8), (16390, 128, 8)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_sigmoid_gradient_of_confident_experts(T, E, k, renorm, dtype):
    rng = np.random.default_rng(T + E)
    dl = to_dev(logits_of(T, E, rng), torch.bfloat16 if dtype == "bf16" else torch.float32)
    l = dl.double().cpu().numpy()
    # half of the choices are the best ones, half any: gradients of small scores too
    best = np.argsort(-l, axis=1, kind="stable")[:, :k]
    anyone = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    ids = np.where(np.arange(T)[:, None] % 2 == 0, best, anyone).astype(np.int32)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    got = fg.route_topk_grad(dl, to_dev(ids), to_dev(dw), score="sigmoid", renorm=renorm, scale=2.5).double().cpu().numpy()
    at = np.take_along_axis(l, ids.astype(np.int64), 1)
    s, slope = 1 / (1 + np.exp(-at)), 1 / ((1 + np.exp(-at)) * (1 + np.exp(at)))
    g = 2.5 * dw.astype(np.float64)
    if renorm:
        total = s.sum(1, keepdims=True)
        grad = (g - (g * s).sum(1, keepdims=True) / total) * slope / total
        tol = (4 * k + 60) * U32 * np.abs(g).max(1, keepdims=True) * slope / total
    else:
        grad = g * slope
        tol = 32 * U32 * np.abs(grad)
    ref, bound = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(ref, ids.astype(np.int64), grad, 1)
    np.put_along_axis(bound, ids.astype(np.int64), tol, 1)
    assert np.all(near(got, ref, bound, dtype))


def test_sigmoid_gradient_ends():
    """Logits at which the complement underflows, infinite ones and masked ones: 0, never NaN."""
    l = np.array([[85.0, 120.0, 3e38, np.inf, -np.inf, -3e38, -120.0, np.nan]], np.float32)
    ids = torch.arange(8, dtype=torch.int32, device=dev()).view(1, 8)
    got = fg.route_topk_grad(to_dev(l), ids, torch.ones(1, 8, device=dev()), score="sigmoid").cpu().numpy()[0]
    assert abs(got[0] - np.exp(-85.0)) <= 32 * U32 * np.exp(-85.0) and np.all(np.abs(got[1:]) <= 1e-38)

"""The adapters' numerics on the GPU. The inputs are whole numbers (and powers of two) of so few bits that every sum is exact in fp32
whatever its order, so an output has to be the bf16 rounding of the exact result, bit for bit."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_02_amd as fg
from fgtest import dev, to_dev

pytestmark = pytest.mark.gpu


def bf16(a):
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32))
    b = t.to(torch.bfloat16)
    assert torch.equal(b.float().isnan(), t.isnan()) and torch.equal(b.float().nan_to_num(1.5), t.nan_to_num(1.5))   # no rounding
    return b.to(dev())


def rounded(a):
    """fp64 values as bf16 values (through fp32, in which they have to be exact), NaN kept."""
    f = np.asarray(a, np.float64).astype(np.float32)
    return torch.from_numpy(f).to(torch.bfloat16).float().numpy()


def run(D, x, A, B, scales, ids, align, in_place=False):
    plan = fg.plan_contiguous(to_dev(ids.astype(np.int32).reshape(-1, 1)), A.shape[0], align)
    d = bf16(D)
    out = fg.adapters(d, bf16(x), bf16(A), bf16(B), to_dev(scales.astype(np.float32)), plan, out=d if in_place else None)
    return out.float().cpu().numpy(), plan


def reference(D, x, A, B, scales, ids):
    """h as fp32 holds it, the rest in 64 bits."""
    out = np.array(D, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        for a in range(A.shape[0]):
            t = np.flatnonzero(ids == a)
            h = (x[t].astype(np.float64) @ A[a].astype(np.float64).T).astype(np.float32)
            h = (h * np.float32(scales[a])).astype(np.float64)
            out[t] += (h[:, None, :] * B[a].astype(np.float64)[None]).sum(2) if not np.isfinite(h).all() or not np.isfinite(B[a]).all() \
                else h @ B[a].astype(np.float64).T
    return out


# ------------------------------------------------------------------ the inner result
@pytest.mark.parametrize("align", [16, 64])
@pytest.mark.parametrize("R", [8, 16, 32, 40, 64, 128])
def test_inner_result_keeps_32_bits(R, align):
    """Pairs of ranks whose h differ in the last eight of 24 bits alone: the output is that difference."""
    T, L, K, N = 70, 3, 128, 264
    rng = np.random.default_rng(R + align)
    ids = rng.integers(0, L, T)
    x = np.zeros((T, K))
    x[:, [5, 70, 100]] = np.array([65536.0, 256.0, 1.0]) * 2.0 ** rng.integers(-20, 21, (T, 1))
    byte = rng.integers(0, 256, (3, L, R // 2))
    byte[0] |= 128
    byte[2] |= 1
    sign = rng.choice([-1, 1], (L, R // 2))
    A, B = np.zeros((L, R, K)), np.zeros((L, N, R))
    A[:, 0::2, 5], A[:, 0::2, 70], A[:, 0::2, 100] = sign * byte
    A[:, 1::2, 5], A[:, 1::2, 70] = -sign * byte[:2]
    for n in range(N):
        i = n % (R // 2)
        B[:, n, 2 * i] = B[:, n, 2 * i + 1] = 1.0
    scales = np.array([1.0, 0.25, 8.0])
    out, _ = run(np.zeros((T, N)), x, A, B, scales, ids, align)
    want = (scales[:, None] * sign * byte[2])[ids][:, np.arange(N) % (R // 2)] * x[:, 100:101]
    assert np.array_equal(rounded(want), want) and np.all(want != 0)
    assert np.array_equal(out, want)

"""The adapters' numerics on the GPU: the inner result held in 32 bits, infinities, and both products' loops at the
depths of real sizes. The inputs are whole numbers (and powers of two) of so few bits that every sum is exact in fp32
whatever its order, so an output has to be the bf16 rounding of the exact result, bit for bit."""
import ctypes

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


# ------------------------------------------------------------------ infinities
@pytest.mark.parametrize("align", [16, 64])
@pytest.mark.parametrize("R", [8, 16, 32, 64, 72, 128])
def test_infinities_as_in_fp32(R, align):
    """A product that overflows, an infinite operand and the largest finite h give what fp32 gives: an infinity with
    its sign, NaN only for inf - inf, inf x 0 and NaN itself."""
    T, L, K, N = 24, 2, 128, 136
    rng = np.random.default_rng(R)
    ids = np.arange(T) % L
    x, A = np.zeros((T, K)), np.zeros((L, R, K))
    B = rng.integers(1, 5, (L, N, R)) * rng.choice([-1.0, 1.0], (L, N, R))
    D = rng.integers(-8, 9, (T, N)).astype(np.float64)
    D[6:8, 3], D[6:8, 4] = np.inf, -np.inf
    x[:, 2], A[:, :, 2] = 1.0, rng.integers(1, 100, (L, R))        # ordinary h everywhere
    # adapter 0: h overflows in rank 1 (both signs, by token); a column without that rank has inf x 0
    A[0, 1, 7] = 2.0 ** 100
    x[0, 7], x[2, 7] = 2.0 ** 100, -2.0 ** 100
    B[0, 9, 1] = 0.0
    # ranks 2 and 3 overflow together: inf - inf where their columns' signs differ
    A[0, 2, 11] = A[0, 3, 11] = 2.0 ** 90
    x[4, 11] = 2.0 ** 90
    # an infinite input
    x[8, 7] = np.inf
    # adapter 1: infinite weights; h of few bits, of 24 bits (both signs), and zero
    B[1, 5, 0], B[1, 6, 0], B[1, 7, R - 1] = np.inf, -np.inf, np.inf
    A[1, 0, 40:43] = 251.0, 253.0, 255.0
    x[3, 40:43] = 65536.0, 256.0, 1.0
    x[5, 40:43] = -65536.0, -256.0, -1.0
    x[7] = 0.0
    # adapter 1, rank 4: h above the largest bf16, below the largest fp32 (255.75 x 2^120)
    A[1, 4, 60:62] = 255 * 2.0 ** 20, 0.75 * 2.0 ** 20
    x[9, 60:62] = 2.0 ** 100
    A[1, 4, 2] = 0.0
    B[1, :, 4] = 2.0 ** -10 * rng.choice([-1.0, 1.0], N)
    out, _ = run(D, x, A, B, np.ones(L), ids, align)
    with np.errstate(over="ignore", invalid="ignore"):
        ref = rounded(reference(D, x, A, B, np.ones(L), ids))
    print("inf", int(np.isinf(ref).sum()), "nan", int(np.isnan(ref).sum()), flush=True)
    assert np.isinf(ref).sum() > 300 and 100 < np.isnan(ref).sum() < 0.25 * ref.size
    assert np.isfinite(ref[9, 8:]).all() and np.abs(ref[9, 8:]).min() >= 2.0 ** 117
    bad = ~((out == ref) | (np.isnan(out) & np.isnan(ref)))
    for t in (3, 5, 9):   # sums of a large h's products and ordinary ones are not exact: one bf16 step there
        with np.errstate(invalid="ignore"):
            bad[t] &= ~(np.abs(out[t] - ref[t]) <= 2.0 ** -7 * np.abs(ref[t]))
    assert not bad.any(), [(int(t), int(n), out[t, n], ref[t, n]) for t, n in np.argwhere(bad)[:8]]


# ------------------------------------------------------------------ depth of the loops
def shape_of_work(T, L, align, R, K, N):
    """What the size rules make of a call: parts of K (from the workspace they need), steps of 64 k for a wave's or
    workgroup's run, rounds of 128 columns in an expand workgroup, and whether the output is stored past the caches."""
    cap, size = fg.plan_capacity(T, 1, L, align), ctypes.c_size_t()
    assert fg.lib().fg_adapters_workspace(R, K, cap, align, ctypes.byref(size)) == 0
    groups = 1 if R <= 16 else 2 if R <= 32 else 4 if R <= 64 else 8
    parts, rest = divmod(size.value - 1024, cap * 16 * groups * 4)
    assert rest == 0
    rt = 64 if align % 64 == 0 else 16
    strip, tiles = 1024, cap // rt
    while strip > 128 and tiles * -(-N // strip) < (256 if rt == 64 else 512):
        strip //= 2
    return dict(parts=parts, steps=K // 64 // (parts * (1 if rt == 64 else 4)), rounds=-(-min(strip, N) // 128),
                stream=T * N * 2 > 32 << 20)


DEPTH = [
    # (T, L, align, R, K, N, what the case is here for)
    (1, 1, 16, 16, 7168, 4096, dict(parts=8)),
    (1, 1, 16, 64, 7168, 4096, dict(parts=8)),
    (1, 1, 16, 128, 7168, 4104, dict(parts=8)),
    (64, 64, 16, 16, 7168, 4096, dict(parts=4, steps=7, rounds=4)),
    (300, 200, 16, 64, 7168, 2056, dict(parts=2, steps=14)),
    (600, 500, 48, 32, 7168, 1000, dict(parts=1, steps=28)),
    (1024, 8, 64, 16, 7168, 4096, dict(parts=8, steps=14, rounds=2, stream=False)),
    (512, 8, 64, 128, 7168, 4096, dict(parts=4, steps=28)),
    (33, 1, 64, 40, 7168, 520, dict(parts=4, steps=28)),
    (8192, 8, 64, 8, 512, 1000, dict(rounds=4, stream=False)),
    (8192, 3, 64, 24, 512, 1000, dict(rounds=4, stream=False)),
    (8192, 3, 128, 64, 256, 1544, dict(rounds=8, stream=False)),
    (8192, 2, 64, 128, 256, 1000, dict(rounds=4, stream=False)),
    (4112, 8, 64, 8, 512, 4104, dict(rounds=8, stream=True)),
    (4112, 8, 64, 16, 512, 4104, dict(rounds=8, stream=True)),
    (4112, 8, 64, 40, 512, 4104, dict(rounds=8, stream=True)),
    (4112, 8, 64, 128, 1024, 4104, dict(rounds=8, stream=True)),
]


@pytest.mark.parametrize("T,L,align,R,K,N,what", DEPTH, ids=lambda v: str(v) if not isinstance(v, dict) else "")
def test_depth(T, L, align, R, K, N, what):
    got = shape_of_work(T, L, align, R, K, N)
    print(f"adapters T={T} L={L} align={align} R={R} K={K} N={N} {got}", flush=True)
    assert {k: got[k] for k in what} == what
    rng = np.random.default_rng(T + R + N)
    ids = rng.integers(-1 if T > 1 else 0, L, T)
    whole = lambda most, *shape: rng.integers(-most, most + 1, shape, dtype=np.int16).astype(np.float32)  # noqa: E731
    x, D, A, B = whole(4, T, K), whole(200, T, N), whole(2, L, R, K), whole(2, L, N, R)
    scales = 2.0 ** rng.integers(-2, 3, L)
    ref = reference(D, x, A, B, scales, ids)
    assert np.abs(ref).max() < 2 ** 21      # whole quarters below 2^24 of them
    for in_place in (False, True):
        out, _ = run(D, x, A, B, scales, ids, align, in_place)
        assert np.array_equal(out, rounded(ref))

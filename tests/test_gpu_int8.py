"""The integer products and their operands' quantisers on the GPU. The sums are exact, so a product's
outputs are compared bit for bit with the same three roundings (the sum to fp32, the two scales, bf16)
of the 64-bit sum; quantised codes and scales bit for bit with the same fp32 steps in numpy."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_02_amd as fg
from fgtest import SENTINEL, d_bits, dev, new_out, to_dev
from int8testing import forced_int8

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


def host(t):
    return (t.float() if t.is_floating_point() else t).cpu().numpy()


# ------------------------------------------------------------------ quantisers
def ref_quant(v):
    """(codes, scales) of fp32 rows, in the same fp32 steps."""
    amax = np.abs(v).max(-1)
    s = np.where(amax == 0, np.float32(1), np.maximum(amax / np.float32(127), np.float32(2.0 ** -126))).astype(np.float32)
    return np.rint(v / s[..., None]).astype(np.int8), s


def awkward_rows(T, K, seed):
    """Rows with outliers, zeros of both signs, subnormals, scales below 2^-90, ties, and the largest floats."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, K)).astype(np.float32)
    special = [lambda r: r * 50, lambda r: r * 0, lambda r: -0.0 * np.abs(r), lambda r: r * np.float32(1e-39),
               lambda r: r * np.float32(1e-30), lambda r: r * np.float32(6e37),
               lambda r: np.where(np.arange(K) == K // 2, 127, np.round(r) + 0.5)]
    for i, f in enumerate(special):
        if T > i + 1:
            x[i + 1] = f(x[i + 1])
    return x.astype(np.float32)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,K", [(1, 16), (9, 16), (8, 48), (5, 1024), (11, 1040), (8, 4096), (9, 4112), (8, 7168), (8, 8192),
                                 (9, 8208), (8, 16384), (3, 18432), (2, 65536), (2049, 128)])
def test_quant_rows(T, K, dtype):
    print(f"quant_int8 {T}x{K} {dtype}", flush=True)
    x = to_dev(awkward_rows(T, K, T + K), torch.bfloat16 if dtype == "bf16" else torch.float32)
    q, s = fg.quant_int8(x)
    rq, rs = ref_quant(host(x))
    assert np.array_equal(host(s), rs)
    assert np.array_equal(host(q), rq)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,K", [(8, 128), (33, 112), (31, 32), (14, 144), (130, 256), (67, 208), (9, 272), (13, 512), (131, 400)])
def test_quant_short_rows(T, K, dtype):
    """Several rows side by side in a wave, whole waves of them and not."""
    test_quant_rows(T, K, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,I", [(37, 128), (9, 256), (35, 384), (17, 512)])
def test_swiglu_short_rows(T, I, dtype):
    test_swiglu(T, I, dtype)


def test_quant_leading_dimensions_and_given_outputs():
    w = to_dev(awkward_rows(12, 256, 5).reshape(3, 4, 256))
    q = torch.empty(3, 4, 256, dtype=torch.int8, device=dev())
    s = torch.empty(3, 4, device=dev())
    got = fg.quant_int8(w, q=q, s=s)
    assert got[0] is q and got[1] is s
    rq, rs = ref_quant(host(w))
    assert np.array_equal(host(q), rq) and np.array_equal(host(s), rs)


def test_quant_rows_with_infinity_and_nan_say_so():
    x = torch.ones(5, 64, device=dev())
    x[1, 3] = float("inf")
    x[2, 60] = float("nan")
    x[3, 7], x[3, 8] = float("-inf"), float("nan")
    q, s = fg.quant_int8(x)
    s = host(s)
    assert np.isinf(s[1]) and np.isnan(s[2]) and np.isnan(s[3])
    assert s[0] == s[4] == np.float32(1) / np.float32(127)
    assert np.all(host(q)[[0, 4]] == 127)
    w, sw = fg.quant_int8(torch.ones(8, 64, device=dev()))
    D = fg.gemm_int8_nt(q, to_dev(s), w, sw, new_out((5, 8)))
    assert np.array_equal(np.isfinite(host(D)).all(1), [True, False, False, False, True])


def plans(T, k, E, G, M_max, seed):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[ids >= G] = np.where(rng.random((ids >= G).sum()) < 0.5, -1, E + 7)
    return fg.plan_contiguous(to_dev(ids), G), fg.plan_masked(to_dev(ids), G, M_max)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,k,E,G,H", [(1, 1, 1, 1, 16), (9, 2, 4, 3, 272), (33, 8, 24, 8, 1024), (40, 3, 8, 8, 7168),
                                       (7, 2, 6, 5, 8208), (3, 2, 4, 4, 18432)])
def test_dispatch(T, k, E, G, H, weighted, dtype):
    print(f"dispatch_quant_int8 T={T} k={k} E={E} G={G} H={H} weighted={weighted} {dtype}", flush=True)
    rng = np.random.default_rng(T + H)
    x = to_dev(awkward_rows(T, H, H), torch.bfloat16 if dtype == "bf16" else torch.float32)
    w = rng.standard_normal((T, k)).astype(np.float32) if weighted else None
    if weighted and T > 1:
        w[1] = 0.0
    for plan in plans(T, k, E, G, max(1, T // 2), T):
        Q = torch.full(plan.lead + (H,), 77, dtype=torch.int8, device=dev())
        s = torch.full(plan.lead, -3.0, device=dev())
        fg.dispatch_quant_int8(x, plan, w=None if w is None else to_dev(w), Q=Q, s=s)
        with np.errstate(over="ignore", invalid="ignore"):
            v = host(x)[:, None] * (np.ones((T, k, 1), np.float32) if w is None else w[:, :, None])
            rq, rs = ref_quant(v)
        wantQ, wantS = np.full((plan.capacity, H), 77, np.int8), np.full(plan.capacity, -3.0, np.float32)
        rows = host(plan.rows)
        wantQ[rows[rows >= 0]], wantS[rows[rows >= 0]] = rq[rows >= 0], rs[rows >= 0]
        assert np.array_equal(host(s).reshape(-1), wantS)
        finite = np.isfinite(wantS)                   # a weight may carry the largest floats past fp32
        assert np.array_equal(host(Q).reshape(-1, H)[finite], wantQ[finite])


@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_of_many_choices(weighted):
    """More choices than a wave has lanes."""
    test_dispatch(5, 70, 80, 80, 272, weighted, "fp32")


def test_swiglu_at_the_ends_of_the_range():
    """Gates so negative that exp overflows give 0, so positive that it vanishes give the gate itself."""
    g = torch.tensor([-3e38, -1e30, -1e5, -200.0, -104.0, -89.0, -80.0, 40.0, 90.0, 1e5] + [0.0] * 118)
    h = torch.cat([g, torch.ones(128)])[None].to(dev())
    h[0, 9] = 1e4
    Q, s = fg.swiglu_quant_int8(h)
    assert float(s) == float(np.float32(1e4) / np.float32(127))
    assert host(Q)[0].tolist() == [0] * 7 + [1, 1, 127] + [0] * 118


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_swiglu_of_gates_near_the_largest_float(dtype):
    """Their silu is the gate itself, an infinite one's infinity: the scale shows it."""
    g = torch.zeros(3, 128)
    g[0, :3] = torch.tensor([2.0 ** 127, 1.5 * 2.0 ** 127, -3e38])
    g[1, 0] = float("inf")
    g[2, 0] = float("nan")
    up = torch.full((3, 128), 0.5)
    Q, s = fg.swiglu_quant_int8(torch.cat([g, up], 1).to(dev(), torch.bfloat16 if dtype == "bf16" else torch.float32))
    assert float(s[0]) == float(np.float32(1.5 * 2.0 ** 126) / np.float32(127))
    assert host(Q)[0].tolist() == [85, 127] + [0] * 126    # 127 * 2 / 3 = 84.67
    assert float(s[1]) == float("inf") and bool(s[2].isnan())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,I", [(1, 128), (6, 384), (5, 1024), (4, 1152), (3, 4096), (3, 8192), (2, 18432)])
def test_swiglu(T, I, dtype):
    print(f"swiglu_quant_int8 {T}x{I} {dtype}", flush=True)
    rng = np.random.default_rng(I)
    h = (3 * rng.standard_normal((T, 2 * I))).astype(np.float32)
    h[-1] *= 40                                       # silu where exp overflows and where it vanishes
    h[0, :5] = [0.0, -0.0, -80.0, -200.0, 200.0]
    dh = to_dev(h, torch.bfloat16 if dtype == "bf16" else torch.float32)
    h = host(dh).astype(np.float64).reshape(T, -1, 2, 128)
    g = h[:, :, 0]
    v = (g / (1 + np.exp(-g)) * h[:, :, 1]).reshape(T, I)
    Q, s = fg.swiglu_quant_int8(dh)
    # v in fp32: exp within 2 ulp (4 u), the sum, the division and the product half an ulp (u) each; the scale one more
    rel = 8 * U32
    top = np.abs(v).max(1)
    assert np.all(np.abs(host(s) - top / 127) <= 2 * rel * top / 127)
    # half a code, and v's and the scale's errors of a quotient of at most 127
    assert np.all(np.abs(host(Q) - v / (top / 127)[:, None]) <= 0.5 + 127 * 3 * rel)


def test_swiglu_leaves_rows_without_a_slot():
    for plan in plans(20, 2, 6, 4, 6, 3):
        h = torch.full(plan.lead + (256,), float("nan"), device=dev(), dtype=torch.bfloat16)
        there = (plan.slots >= 0).view(plan.lead)
        h[there] = torch.randn(int(there.sum()), 256, device=dev()).bfloat16()
        Q = torch.full(plan.lead + (128,), 77, dtype=torch.int8, device=dev())
        s = torch.full(plan.lead, -3.0, device=dev())
        fg.swiglu_quant_int8(h, plan, Q=Q, s=s)
        full, fs = fg.swiglu_quant_int8(h[there])
        assert torch.equal(Q[there], full) and torch.equal(s[there], fs)
        assert bool((Q[~there] == 77).all()) and bool((s[~there] == -3.0).all())


# ------------------------------------------------------------------ products
def operands(lead, G, N, K, seed):
    """int8 operands over the whole range (-128 too) and scales from 2^-12 to 2^3."""
    rng = np.random.default_rng(seed)
    A = rng.integers(-128, 128, lead + (K,), dtype=np.int8)
    B = rng.integers(-128, 128, (G, N, K) if G else (N, K), dtype=np.int8)
    sa = np.exp2(rng.uniform(-12, 3, lead)).astype(np.float32)
    sb = np.exp2(rng.uniform(-12, 3, B.shape[:-1])).astype(np.float32)
    return A, sa, B, sb


def ref_product(A, sa, B, sb):
    """bf16 bits of (fp32(sum) * sa) * sb; the sum is exact in a double."""
    acc = (A.astype(np.float64) @ B.astype(np.float64).T).astype(np.float32)
    return d_bits(torch.from_numpy((acc * sa[:, None]) * sb).to(torch.bfloat16))


def on_gpu(*a):
    return tuple(to_dev(x) for x in a)


@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (1, 136, 48), (2, 24, 32), (15, 120, 112), (16, 128, 128), (17, 264, 144),
                                   (64, 520, 240), (65, 16, 256), (127, 136, 272), (129, 72, 1040), (300, 264, 2064),
                                   (1, 7168, 1024), (33, 2056, 7168), (520, 1032, 400)])
def test_dense(M, N, K):
    print(f"gemm_int8_nt {M}x{N}x{K}", flush=True)
    a = operands((M,), 0, N, K, M + N + K)
    D = fg.gemm_int8_nt(*on_gpu(*a), new_out((M, N)))
    assert np.array_equal(d_bits(D), ref_product(*a))


@pytest.mark.parametrize("kernel", ["256x256", "256x128", "128x256", "128x128", "64x128", "128x160", "split"])
@pytest.mark.parametrize("M,N,K", [(1, 520, 16), (70, 520, 128), (257, 776, 272), (300, 1032, 400), (513, 520, 1168)])
def test_dense_on_every_kernel(M, N, K, kernel):
    print(f"gemm_int8_nt {M}x{N}x{K} on {kernel}", flush=True)
    a = operands((M,), 0, N, K, M + N + K)
    want = ref_product(*a)
    a = on_gpu(*a)
    for grid in (1, 3, 0) if kernel == "split" else (0,):
        with forced_int8(kernel, grid):
            D = fg.gemm_int8_nt(*a, new_out((M, N)))
        assert np.array_equal(d_bits(D), want), grid


@pytest.mark.parametrize("M,N,K,columns", [
    (*size, columns) for columns in ("16 columns", "32 columns", "64 columns")
    for size in ((1, 8, 16), (16, 72, 2064), (31, 136, 128), (33, 64, 1040), (48, 200, 1024), (61, 128, 7168), (96, 264, 4112),
                 (80, 64, 272), (128, 72, 3088), (300, 136, 1168))
    if columns != "64 columns" or size[0] <= 96])                  # that width has kernels of up to 96 rows
def test_dense_streamed(M, N, K, columns):
    """The weight-streaming kernel at each width, K from less than one piece of one wave to many rounds of all."""
    print(f"gemm_int8_nt {M}x{N}x{K} streamed, {columns}", flush=True)
    a = operands((M,), 0, N, K, M + N + K)
    with forced_int8(columns):
        D = fg.gemm_int8_nt(*on_gpu(*a), new_out((M, N)))
    assert np.array_equal(d_bits(D), ref_product(*a))


@pytest.mark.parametrize("columns,rows", [(c, r) for r in (1, 2, 3, 4, 6, 8) for c in ("16 columns", "32 columns", "64 columns")
                                          if (c, r) != ("64 columns", 8)])
def test_streamed_on_every_block_of_rows(columns, rows):
    for M, N, K in [(5, 72, 48), (16 * rows, 264, 1040), (40 * rows + 3, 136, 2064), (300, 200, 7168)]:
        print(f"gemm_int8_nt {M}x{N}x{K} streamed, {16 * rows} rows, {columns}", flush=True)
        a = operands((M,), 0, N, K, M + N + K)
        with forced_int8(columns, rows):
            D = fg.gemm_int8_nt(*on_gpu(*a), new_out((M, N)))
        assert np.array_equal(d_bits(D), ref_product(*a))
    G, M_max, N, K, counts = 5, 70, 136, 528, [70, 0, 1, 33, -2]
    A, sa, B, sb = operands((G, M_max), G, N, K, rows)
    with forced_int8(columns, rows):
        D = fg.grouped_masked_int8(*on_gpu(A, sa, B, sb), new_out((G, M_max, N)), to_dev(np.array(counts, np.int32)))
    for g, n in enumerate(counts):
        n = max(n, 0)
        assert np.array_equal(d_bits(D[g, :n]), ref_product(A[g, :n], sa[g, :n], B[g], sb[g]))
        assert bool((D[g, n:].cpu().view(torch.int16) == new_out((1,)).cpu().view(torch.int16)).all())


def contiguous_rows(G, counts, seed, extra=128):
    """m_indices of experts with so many rows each, segments padded to 128, the tail all padding; a few rows
    inside the segments are padding too, and some padding ids are out of range."""
    rng = np.random.default_rng(seed)
    m = []
    for g, c in enumerate(counts):
        rows = np.full(-(-c // 128) * 128, -1)
        rows[:c] = g
        m.append(rows)
    m = np.concatenate(m + [np.full(extra, -1)]).astype(np.int32)
    at = np.flatnonzero(m >= 0)
    if at.size > 8:
        m[rng.choice(at, at.size // 8, replace=False)] = np.where(rng.random(at.size // 8) < 0.5, -1, G + 5)
    return m


def check_contiguous(G, N, K, counts, kernels):
    m = contiguous_rows(G, counts, sum(counts))
    A, sa, B, sb = operands((m.size,), G, N, K, N + K)
    want = np.full((m.size, N), SENTINEL, np.uint16)
    for g in range(G):
        at = m == g
        want[at] = ref_product(A[at], sa[at], B[g], sb[g])
    a, dm = on_gpu(A, sa, B, sb), to_dev(m)
    for kernel, grid in kernels:
        D = new_out((m.size, N))
        if kernel is None:
            fg.grouped_contiguous_int8(*a, D, dm)
        else:
            with forced_int8(kernel, grid):
                fg.grouped_contiguous_int8(*a, D, dm)
        assert np.array_equal(d_bits(D), want), (kernel, grid)


@pytest.mark.parametrize("G,N,K,counts", [(1, 8, 16, [1]), (3, 264, 272, [5, 0, 200]), (4, 520, 128, [130, 256, 1, 384]),
                                          (5, 136, 1040, [0, 0, 640, 7, 128]), (2, 1032, 400, [700, 300])])
def test_contiguous(G, N, K, counts):
    print(f"grouped_contiguous_int8 G={G} {N}x{K} {counts}", flush=True)
    check_contiguous(G, N, K, counts, [(None, 0), ("128x256", 0), ("128x128", 0), ("64x128", 0), ("128x160", 0), ("runs", 1), ("runs", 5),
                                       ("runs", 0)])


def test_contiguous_last_round_in_quarters():
    """A whole round of two-block tiles on 256 units, then 64 single blocks; the last columns' quarters are partly or
    wholly past N, the last rows' past the experts'."""
    for N, counts in [(2040, [1147, 1030, 1152, 1088, 1089, 1025, 1100, 1150]), (1800, [1147] * 8)]:
        check_contiguous(8, N, 144, counts, [("runs", 256)])


@pytest.mark.parametrize("rows", [1, 2, 4, 8])
@pytest.mark.parametrize("G,N,K,counts", [(1, 8, 16, [1]), (3, 136, 272, [5, 0, 200]), (4, 264, 1040, [130, 64, 1, 33]),
                                          (5, 72, 3088, [0, 0, 257, 7, 128])])
def test_contiguous_streamed(G, N, K, counts, rows):
    print(f"grouped_contiguous_int8 G={G} {N}x{K} {counts} streamed, {16 * rows} rows", flush=True)
    check_contiguous(G, N, K, counts, [(c, rows) for c in ("16 columns", "32 columns", "64 columns") if (c, rows) != ("64 columns", 8)])


def test_contiguous_all_padding():
    A, sa, B, sb = operands((256,), 2, 64, 64, 1)
    D = new_out((256, 64))
    fg.grouped_contiguous_int8(*on_gpu(A, sa, B, sb), D, to_dev(np.full(256, -1, np.int32)))
    assert np.all(d_bits(D) == SENTINEL)


@pytest.mark.parametrize("G,M_max,N,K,counts", [(1, 1, 8, 16, [1]), (3, 8, 264, 272, [0, 8, 3]), (4, 64, 520, 144, [64, -3, 99, 17]),
                                                (5, 256, 136, 1040, [256, 0, 129, 1, 65]), (2, 300, 1032, 400, [300, 257])])
def test_masked(G, M_max, N, K, counts):
    print(f"grouped_masked_int8 G={G} M_max={M_max} {N}x{K} {counts}", flush=True)
    A, sa, B, sb = operands((G, M_max), G, N, K, N + K)
    want = np.full((G, M_max, N), SENTINEL, np.uint16)
    for g, c in enumerate(counts):
        c = min(max(c, 0), M_max)
        want[g, :c] = ref_product(A[g, :c], sa[g, :c], B[g], sb[g])
    a, mm = on_gpu(A, sa, B, sb), to_dev(np.array(counts, np.int32))
    for kernel in (None, "256x256", "256x128", "128x256", "128x128", "64x128", "128x160", "16 columns", "32 columns", "64 columns"):
        if kernel == "64 columns" and M_max > 96:
            continue
        D = new_out((G, M_max, N))
        if kernel is None:
            fg.grouped_masked_int8(*a, D, mm)
        else:
            with forced_int8(kernel):
                fg.grouped_masked_int8(*a, D, mm)
        assert np.array_equal(d_bits(D), want), kernel


def test_largest_sums_are_exact():
    """The largest K, every product 128^2: the sum is 16384 K < 2^31, and one product less shows in fp32."""
    K = 131056
    A, B = np.full((17, K), -128, np.int8), np.full((8, K), -128, np.int8)
    A[3] = 127
    one = np.ones(17, np.float32), np.ones(8, np.float32)
    D = fg.gemm_int8_nt(*on_gpu(A, one[0], B, one[1]), new_out((17, 8)))
    assert np.array_equal(d_bits(D), ref_product(A, one[0], B, one[1]))


def test_operands_past_2_31_bytes():
    """Rows of A, of D and of the experts' weights whose byte offsets pass 2^31 and 2^32."""
    K, N, M = 16384, 24, 270000            # A: 4.4e9 bytes
    A = torch.zeros(M, K, dtype=torch.int8, device=dev())
    B = torch.zeros(N, K, dtype=torch.int8, device=dev())
    rows = torch.tensor([0, 1, 131071, 131072, 262143, 262144, 269998, 269999], device=dev())
    gen = torch.Generator(device="cuda").manual_seed(3)
    A[rows] = torch.randint(-128, 128, (rows.numel(), K), device=dev(), generator=gen).to(torch.int8)
    B[:] = torch.randint(-128, 128, (N, K), device=dev(), generator=gen).to(torch.int8)
    sa, sb = torch.rand(M, device=dev(), generator=gen), torch.rand(N, device=dev(), generator=gen)
    D = fg.gemm_int8_nt(A, sa, B, sb, new_out((M, N)))
    want = ref_product(host(A[rows]), host(sa[rows]), host(B), host(sb))
    assert np.array_equal(d_bits(D[rows]), want)
    zero = torch.ones(M, dtype=torch.bool, device=dev())
    zero[rows] = False
    assert bool((D[zero] == 0).all())
    q, s = fg.quant_int8(torch.ones(3, 16, device=dev()))   # nothing is left in flight that faults
    assert bool((q == 127).all())


def test_columns_up_to_the_limit():
    """The most columns there may be: 256 rows of D are just below 2^31 bytes, all 257 above."""
    M, N, K = 257, 4194296, 16
    gen = torch.Generator(device="cuda").manual_seed(6)
    A = torch.randint(-128, 128, (M, K), device=dev(), generator=gen).to(torch.int8)
    B = torch.randint(-128, 128, (N, K), device=dev(), generator=gen).to(torch.int8)
    sa, sb = torch.rand(M, device=dev(), generator=gen), torch.rand(N, device=dev(), generator=gen)
    D = fg.gemm_int8_nt(A, sa, B, sb, new_out((M, N)))
    at = torch.tensor([0, 1, 255, 4096, 2097152, N - 256, N - 9, N - 8, N - 1], device=dev())
    assert np.array_equal(d_bits(D[:, at].contiguous()), ref_product(host(A), host(sa), host(B[at]), host(sb[at])))
    one = fg.gemm_int8_nt(A[:1], sa[:1], B, sb, new_out((1, N)))     # the kernel of few rows
    assert torch.equal(one, D[:1])


def test_contiguous_rows_past_the_run_list():
    """More 128-row blocks than the run-following kernel lists: tiles of at most 128 rows."""
    G, N, K, M = 3, 24, 32, 2048 * 128 + 384
    m = torch.arange(M, device=dev()) // 128 % 4 - 1                  # every fourth block is padding
    gen = torch.Generator(device="cuda").manual_seed(7)
    A = torch.randint(-128, 128, (M, K), device=dev(), generator=gen).to(torch.int8)
    B = torch.randint(-128, 128, (G, N, K), device=dev(), generator=gen).to(torch.int8)
    sa, sb = torch.rand(M, device=dev(), generator=gen), torch.rand(G, N, device=dev(), generator=gen)
    D = host(fg.grouped_contiguous_int8(A, sa, B, sb, new_out((M, N)), m.to(torch.int32)).view(torch.int16)).view(np.uint16)
    m = host(m)
    assert np.all(D[m < 0] == SENTINEL)
    for g in range(G):
        assert np.array_equal(D[m == g], ref_product(host(A)[m == g], host(sa)[m == g], host(B)[g], host(sb)[g]))


def test_rows_past_a_launch():
    """More rows than one grid's threads can be (2^32, 64 a row): the last ones too."""
    T, K = (1 << 26) + 5, 16
    x = torch.zeros(T, K, dtype=torch.bfloat16, device=dev())
    x[-40:] = torch.randn(40, K, device=dev())
    q, s = fg.quant_int8(x)
    want, ws = fg.quant_int8(x[-40:].clone())
    assert torch.equal(q[-40:], want) and torch.equal(s[-40:], ws)
    assert int(q[:-40].count_nonzero()) == 0 and bool((s[:-40] == 1).all())


def test_experts_past_a_launch():
    """As many experts' tiles of 16 x 64, a few rows' choice, have more threads than a grid."""
    G, N, K = 6000000, 136, 16
    A = torch.ones(G, 1, K, dtype=torch.int8, device=dev())
    B = torch.zeros(G, N, K, dtype=torch.int8, device=dev())
    at = torch.tensor([0, 1, G // 2, G - 2, G - 1], device=dev())
    B[at] = torch.randint(-128, 128, (5, N, K), device=dev()).to(torch.int8)
    one = torch.ones(G, N, device=dev())
    D = torch.full((G, 1, N), 3.0, dtype=torch.bfloat16, device=dev())
    fg.grouped_masked_int8(A, one[:, :1].contiguous(), B, one, D, torch.ones(G, dtype=torch.int32, device=dev()))
    assert torch.equal(D[at, 0], B[at].int().sum(2).bfloat16())
    D[at] = 0.0
    assert int(D.count_nonzero()) == 0


def test_concurrent_streams():
    """Calls in flight together on several streams give bit for bit what they give one after another."""
    jobs = []
    for M, N, K in ((24, 2056, 2064), (300, 1032, 1040), (1001, 520, 528)):
        a = on_gpu(*operands((M,), 0, N, K, M))
        jobs.append((lambda D, a=a: fg.gemm_int8_nt(*a, D), (M, N)))
    want = [run(new_out(shape)) for run, shape in jobs]
    outs = [[new_out(shape) for _ in range(4)] for _, shape in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for r in range(4):
        for (run, _), o, stream in zip(jobs, outs, streams):
            with torch.cuda.stream(stream):
                run(o[r])
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, D) for D in o)


@pytest.mark.parametrize("M", [9, 300])
def test_scales_of_any_alignment(M):
    A, sa, B, sb = on_gpu(*operands((M,), 0, 264, 144, 9))
    odd = lambda v: torch.cat([v.new_zeros(1), v])[1:]  # noqa: E731
    assert torch.equal(fg.gemm_int8_nt(A, odd(sa), B, odd(sb), new_out((M, 264))), fg.gemm_int8_nt(A, sa, B, sb, new_out((M, 264))))
    mm = torch.tensor([7, M - 2], dtype=torch.int32, device=dev())[1:]
    got = fg.grouped_masked_int8(A[None], odd(sa)[None], B[None], odd(sb)[None], new_out((1, M, 264)), mm)
    want = fg.grouped_masked_int8(A[None], sa[None], B[None], sb[None], new_out((1, M, 264)), mm.clone())
    assert torch.equal(got, want)
    shifted = torch.zeros(M * 144 + 1, dtype=torch.int8, device=dev())[1:].view(M, 144)
    with pytest.raises(fg.FGError):
        fg.gemm_int8_nt(shifted, sa, B, sb, new_out((M, 264)))


def test_refusals():
    A, sa, B, sb = on_gpu(*operands((32,), 0, 64, 64, 1))
    D = new_out((32, 64))
    for bad, err in [((A.float(), sa, B, sb, D), TypeError), ((A.view(torch.uint8), sa, B, sb, D), TypeError),
                     ((A, sa[:31], B, sb, D), ValueError), ((A, sa, B, sb[:63], D), ValueError),
                     ((A, sa.double(), B, sb, D), TypeError), ((A, sa, B[:, :48], sb, D), ValueError),
                     ((A, sa, B, sb, D.float()), TypeError), ((A.cpu(), sa, B, sb, D), ValueError),
                     ((A, sa, B.t().contiguous().t(), sb, D), ValueError), ((A, sa, B[:60].contiguous(), sb[:60], D[:, :60]), ValueError),
                     ((A[:, :24].contiguous(), sa, B[:, :24].contiguous(), sb, D), ValueError)]:
        with pytest.raises(err):
            fg.gemm_int8_nt(*bad)
    assert np.all(d_bits(D) == SENTINEL)
    with pytest.raises(ValueError):
        fg.quant_int8(torch.ones(4, 24, device=dev()))
    with pytest.raises(TypeError):
        fg.quant_int8(torch.ones(4, 32, device=dev(), dtype=torch.float16))
    with pytest.raises(ValueError):
        fg.quant_int8(torch.ones(64, device=dev()))
    with pytest.raises(ValueError):
        fg.swiglu_quant_int8(torch.ones(4, 128, device=dev()))
    plan = fg.plan_masked(torch.zeros(4, 1, dtype=torch.int32, device=dev()), 2, 4)
    with pytest.raises(ValueError):
        fg.swiglu_quant_int8(torch.ones(2, 5, 256, device=dev()), plan)
    with pytest.raises(ValueError):
        fg.dispatch_quant_int8(torch.ones(3, 64, device=dev()), plan)


def test_no_rows():
    e = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device=dev())  # noqa: E731
    q, s = fg.quant_int8(e(0, 64))
    assert q.shape == (0, 64) and s.shape == (0,)
    D = fg.gemm_int8_nt(q, s, e(8, 64, dtype=torch.int8).zero_(), e(8).zero_(), e(0, 8, dtype=torch.bfloat16))
    assert D.shape == (0, 8)
    plan = fg.plan_contiguous(e(0, 2, dtype=torch.int32), 4)
    Q, s = fg.dispatch_quant_int8(e(0, 64), plan)
    assert Q.shape == (plan.capacity, 64)
    fg.swiglu_quant_int8(e(0, 256))


def test_captured_and_replayed():
    """A whole expert feed-forward in a graph, replayed on new contents of its inputs."""
    T, k, E, H, I, M_max = 24, 2, 4, 256, 128, 24
    gen = torch.Generator(device="cuda").manual_seed(4)
    new = lambda *s: torch.randn(*s, device=dev(), generator=gen)  # noqa: E731
    up, down = fg.quant_int8(new(E, 2 * I, H)), fg.quant_int8(new(E, H, I))
    x, ids = new(T, H).bfloat16(), torch.zeros(T, k, dtype=torch.int32, device=dev())

    def ffn():
        plan = fg.plan_masked(ids, E, M_max)
        A, sa = fg.dispatch_quant_int8(x, plan)
        h = torch.empty(E, M_max, 2 * I, dtype=torch.bfloat16, device=dev())
        fg.grouped_masked_int8(A, sa, *up, h, plan.masked_m)
        Q, sq = fg.swiglu_quant_int8(h, plan)
        y = torch.empty(E, M_max, H, dtype=torch.bfloat16, device=dev())
        fg.grouped_masked_int8(Q, sq, *down, y, plan.masked_m)
        return fg.combine(y, plan)

    ids.copy_(torch.randint(-1, E, (T, k), device=dev(), generator=gen).to(torch.int32))
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        ffn()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ffn()
    for i in range(4):
        x.copy_(new(T, H).bfloat16())
        ids.copy_(torch.randint(-1, E, (T, k), device=dev(), generator=gen).to(torch.int32))
        want = ffn()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_expert_feed_forward_in_both_layouts():
    """Tokens through routing, sorting, both projections and back: the two layouts agree bit for bit (the sums are
    exact), and the result is the unquantised one's to the quantisation's noise. A row's step is amax / 127; with
    amax up to 4.5 rms its rounding is 4.5 / 127 / sqrt(12) = 1% of a value; the four operands' add up to 2%, SiLU's
    slope (up to 1.1) and the bf16 roundings leave it below 3%."""
    T, k, E, H, I = 200, 3, 6, 512, 384
    gen = torch.Generator(device="cuda").manual_seed(5)
    new = lambda *s, fan=1: torch.randn(*s, device=dev(), generator=gen) * fan ** -0.5  # noqa: E731
    w_up, w_down = new(E, 2 * I, H, fan=H), new(E, H, I, fan=I)
    up, down = fg.quant_int8(w_up), fg.quant_int8(w_down)
    x = new(T, H).bfloat16()
    ids, w = fg.route_topk(new(T, E), k, renorm=True)
    plan = fg.plan_contiguous(ids, E)
    A, sa = fg.dispatch_quant_int8(x, plan)
    h = torch.empty(plan.capacity, 2 * I, dtype=torch.bfloat16, device=dev())
    fg.grouped_contiguous_int8(A, sa, *up, h, plan.m_indices)
    Q, sq = fg.swiglu_quant_int8(h, plan)
    y = torch.empty(plan.capacity, H, dtype=torch.bfloat16, device=dev())
    fg.grouped_contiguous_int8(Q, sq, *down, y, plan.m_indices)
    out = fg.combine(y, plan, w=w)
    plan = fg.plan_masked(ids, E, T)
    A, sa = fg.dispatch_quant_int8(x, plan)
    h = torch.empty(E, T, 2 * I, dtype=torch.bfloat16, device=dev())
    fg.grouped_masked_int8(A, sa, *up, h, plan.masked_m)
    Q, sq = fg.swiglu_quant_int8(h, plan)
    y = torch.empty(E, T, H, dtype=torch.bfloat16, device=dev())
    fg.grouped_masked_int8(Q, sq, *down, y, plan.masked_m)
    assert torch.equal(fg.combine(y, plan, w=w), out)
    xd, wd, ids = host(x).astype(np.float64), host(w).astype(np.float64), host(ids)
    up, down = host(w_up).astype(np.float64), host(w_down).astype(np.float64)
    want = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            v = (up[ids[t, j]] @ xd[t]).reshape(-1, 2, 128)
            act = (v[:, 0] / (1 + np.exp(-v[:, 0])) * v[:, 1]).reshape(-1)
            want[t] += wd[t, j] * (down[ids[t, j]] @ act)
    assert np.linalg.norm(host(out) - want) <= 0.03 * np.linalg.norm(want)

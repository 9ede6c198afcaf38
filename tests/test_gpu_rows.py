"""The row operators on the GPU against plain 64-bit references: routing and its
gradient, sorting, dispatch, combine and its gradient, adapters; at the sizes and
masks where they can go wrong. Tolerances are error bounds of fp32 arithmetic (u =
2^-24); a bf16 output has to be the bf16 rounding of some value within them."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_02_amd as fg
import oracle
import rowref
from fgtest import dev, to_dev

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
LOWEST = float(torch.finfo(torch.float32).min)


def host(t):
    return (t.float() if t.is_floating_point() else t).cpu().numpy()


def near(got, ref, tol, dtype):
    """got (fp32 or bf16 values) is ref to within tol, rounded to its type: rounding is monotone, so a bf16 value
    lies between the roundings of ref - tol and ref + tol."""
    if dtype == "fp32":
        return np.abs(got - ref) <= tol + 1e-38
    lo, hi = (torch.from_numpy(np.asarray(v, np.float64)).to(torch.bfloat16).double().numpy() for v in (ref - tol, ref + tol))
    return (lo <= got) & (got <= hi)


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16).to(dev())


# ------------------------------------------------------------------ route
def logits_of(T, E, seed, masks=True):
    rng = np.random.default_rng(seed)
    l = (2 * rng.standard_normal((T, E))).astype(np.float32)
    if masks and T >= 8:
        l[0] = -np.inf                                # nothing eligible
        l[1, 1:] = -np.inf                            # one left
        l[2, ::2] = np.nan                            # NaN is masked
        l[3] = LOWEST                                 # the type's lowest value is a logit like any other
        l[4] = 0.0
        l[4, ::3] = -0.0                              # equal logits, zeros of both signs: ties
        l[5, E // 2:] = LOWEST
        l[6] = np.round(l[6])                         # many ties
        l[7] = -np.inf
        l[7, E - 1] = 3.0
    return l


def check_route(l, dl, k, score, bias, renorm, scale, dtype):
    ids, w = fg.route_topk(dl, k, score=score, bias=None if bias is None else to_dev(bias), renorm=renorm, scale=scale)
    ids, w = host(ids), host(w)
    ref_ids, _, s = rowref.route(l, k, score, bias, renorm, scale)
    if bias is None:
        assert np.array_equal(ids, ref_ids)
    else:
        # ranks s + bias in fp32: each choice is as good as the 64-bit one of its place, to the rounding of s and the sum
        assert np.array_equal(ids < 0, ref_ids < 0)
        rank = s + bias.astype(np.float64)
        mine = np.take_along_axis(rank, np.maximum(ids, 0), 1)
        best = np.take_along_axis(rank, np.maximum(ref_ids, 0), 1)
        assert np.all(np.abs(mine - best)[ids >= 0] <= 70 * U32 * (1 + np.abs(bias).max()))
        for row in ids:
            got = row[row >= 0]
            assert len(set(got)) == len(got)
    # exp of a rounded difference of logits up to ~20 (20 u) and 2 ulp of exp, the sums' 32 terms, the divisions
    tol = (20 + 8 + 32 + 8) * U32
    ref_w = rowref.weights(s, ids, renorm, scale)
    assert np.all(np.abs(w - ref_w) <= tol * 2 * np.abs(ref_w) + 1e-30)
    assert np.all(w[ids < 0] == 0)
    return ids, s


@pytest.mark.parametrize("score,with_bias,renorm", [("softmax", False, False), ("softmax", False, True),
                                                    ("sigmoid", False, True), ("sigmoid", True, True),
                                                    ("sigmoid", True, False), ("softmax", True, True)])
@pytest.mark.parametrize("T,E,k", [(1, 8, 1), (9, 1, 1), (33, 60, 6), (130, 64, 8), (17, 65, 3), (64, 256, 8),
                                   (40, 257, 64), (12, 1024, 8), (21, 999, 13)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_route_and_gradient(T, E, k, score, with_bias, renorm, dtype):
    print(f"route {T}x{E} k={k} {score} bias={with_bias} renorm={renorm} {dtype}", flush=True)
    l = logits_of(T, E, 7 * E + k)
    dl = to_dev(l, torch.bfloat16 if dtype == "bf16" else torch.float32)
    l = host(dl)
    rng = np.random.default_rng(E + T)
    bias = (0.3 * rng.standard_normal(E)).astype(np.float32) if with_bias else None
    ids, s = check_route(l, dl, k, score, bias, renorm, 2.5, dtype)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    got = fg.route_topk_grad(dl, to_dev(ids.astype(np.int32)), to_dev(dw), score=score, renorm=renorm, scale=2.5)
    ref = rowref.route_grad(s, ids, dw, score, renorm, 2.5)
    # the terms' sizes: scale * |dw| times a score, each with the scores' relative error, sums of up to k + 16 terms
    size = 2.5 * np.abs(dw).sum(1, keepdims=True)
    tol = 4 * (70 + k) * U32 * size * np.maximum(s, 1e-12 if not renorm else 1.0) * (1 if not renorm else 1)
    assert np.all(near(host(got), ref, tol + 1e-30, dtype))


@pytest.mark.parametrize("score,with_bias,renorm", [("softmax", False, False), ("sigmoid", True, True)])
@pytest.mark.parametrize("T,E,k", [(8191, 64, 8), (8192, 64, 8), (8195, 21, 5), (16383, 128, 8), (16387, 128, 8),
                                   (16385, 77, 11)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_route_and_gradient_many_tokens(T, E, k, score, with_bias, renorm, dtype):
    """Batches long enough that several tokens share a wave, and the last shorter ones."""
    test_route_and_gradient(T, E, k, score, with_bias, renorm, dtype)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(score, renorm):
    T, E, k, h = 6, 24, 4, 2.0 ** -6
    rng = np.random.default_rng(3)
    l = np.stack([rng.permutation(E) for _ in range(T)]).astype(np.float32) / 4   # gaps of 1/4: the choice stays
    dw = rng.standard_normal((T, k)).astype(np.float32)
    how = dict(score=score, renorm=renorm, scale=1.5)
    ids, _ = fg.route_topk(to_dev(l), k, **how)
    grad = host(fg.route_topk_grad(to_dev(l), ids, to_dev(dw), **how))
    num = np.zeros((T, E))
    for e in range(E):
        w = []
        for sign in (1, -1):
            m = l.copy()
            m[:, e] += sign * np.float32(h)
            i, v = fg.route_topk(to_dev(m), k, **how)
            assert torch.equal(i, ids)
            w.append(host(v).astype(np.float64))
        num[:, e] = ((w[0] - w[1]) * dw).sum(1) / (2 * h)
    # third derivatives of a weight are below 1: h^2 / 6 each, and 2 * 140 u of noise over 2 h
    tol = 1.5 * np.abs(dw).sum(1, keepdims=True) * (h * h + 140 * U32 / h)
    assert np.all(np.abs(grad - num) <= tol)


def test_route_no_tokens():
    ids, w = fg.route_topk(torch.empty(0, 16, device=dev()), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    assert fg.route_topk_grad(torch.empty(0, 16, device=dev()), ids, w).shape == (0, 16)


# ------------------------------------------------------------------ plan
ID_KINDS = ["random", "one", "none", "wild", "sorted"]


def plan_ids(kind, T, k, G, seed):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full((T, k), G // 2, np.int32)
    if kind == "none":
        return np.full((T, k), -1, np.int32)
    ids = rng.integers(0, G, (T, k)).astype(np.int32)
    if kind == "wild":      # other devices' experts, padding and rubbish
        bad = rng.random((T, k)) < 0.5
        ids[bad] = rng.choice(np.array([-1, G, G + 1, 2 ** 31 - 1, -2 ** 31], np.int64), bad.sum()).astype(np.int32)
    if kind == "sorted":
        ids = np.sort(ids.reshape(-1))[::-1].reshape(T, k).copy()
    return ids


@pytest.mark.parametrize("kind", ID_KINDS)
@pytest.mark.parametrize("T,k,G,align,M_max", [(1, 1, 1, 128, 1), (5, 3, 7, 16, 2), (64, 8, 16, 128, 32),
                                               (511, 8, 256, 64, 16), (512, 8, 64, 128, 256), (513, 8, 1024, 16, 3),
                                               (4099, 2, 100, 128, 64), (9001, 7, 33, 1, 1000), (20000, 8, 64, 128, 4096)])
def test_plans(T, k, G, align, M_max, kind):
    print(f"plan {T}x{k} G={G} align={align} M_max={M_max} {kind}", flush=True)
    ids = plan_ids(kind, T, k, G, T + G)
    cap = fg.plan_capacity(T, k, G, align)
    p = fg.plan_contiguous(to_dev(ids), G, align)
    rows, slots, m, offsets = rowref.plan_contiguous(ids, G, align, cap)
    assert np.array_equal(host(p.offsets), offsets) and offsets[-1] <= cap and p.capacity == cap
    assert np.array_equal(host(p.rows), rows)
    assert np.array_equal(host(p.slots), slots)
    assert np.array_equal(host(p.m_indices), m)
    p = fg.plan_masked(to_dev(ids), G, M_max)
    rows, slots, n = rowref.plan_masked(ids, G, M_max)
    assert np.array_equal(host(p.masked_m), n)
    assert np.array_equal(host(p.rows), rows)
    assert np.array_equal(host(p.slots), slots)


def test_plan_no_tokens():
    p = fg.plan_contiguous(torch.empty(0, 4, dtype=torch.int32, device=dev()), 5)
    assert p.capacity == 0 and host(p.offsets).tolist() == [0] * 6
    p = fg.plan_masked(torch.empty(0, 4, dtype=torch.int32, device=dev()), 3, 4)
    assert host(p.masked_m).tolist() == [0] * 3 and np.all(host(p.slots) == -1)


# ------------------------------------------------------------------ dispatch, combine, gradient
PLANS = [("contiguous", 1, 1, 1), ("contiguous", 37, 3, 5), ("masked", 37, 3, 5), ("masked", 1, 2, 4),
         ("contiguous", 300, 9, 16), ("masked", 64, 8, 8)]


def make_plan(layout, T, k, G, seed=0, drop=True):
    """A plan over G experts of which a few slots have none, and (masked) buffers too short for all."""
    rng = np.random.default_rng(seed + 11)
    ids = rng.integers(-1 if drop and T > 1 else 0, G, (T, k)).astype(np.int32)
    if layout == "masked":
        return fg.plan_masked(to_dev(ids), G, max(1, (T * k * 3) // (4 * G)))
    return fg.plan_contiguous(to_dev(ids), G, 128)


def rows_input(rng, shape):
    x = rng.standard_normal(shape).astype(np.float32)
    if x.shape[0] > 3 and x.shape[1] >= 128:
        x[1] *= 50
        x[2, :128] = 0.0
        x[3, 0] = -1e-30
    return x


@pytest.mark.parametrize("layout,T,k,G", PLANS)
@pytest.mark.parametrize("H", [128, 640, 7168])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_quant(layout, T, k, G, H, pow2, dtype, weighted):
    """Codes and scales bit for bit those of the oracle's quantiser on each slot's fp32 row; other rows untouched."""
    print(f"dispatch {layout} {T}x{k} G={G} H={H} pow2={pow2} {dtype} w={weighted}", flush=True)
    rng = np.random.default_rng(H + T)
    p = make_plan(layout, T, k, G)
    x = to_dev(rows_input(rng, (T, H)), torch.bfloat16 if dtype == "bf16" else torch.float32)
    w = rng.standard_normal((T, k)).astype(np.float32) if weighted else None
    lead = p.lead
    Q = torch.full(lead + (H,), 0x55, dtype=torch.uint8, device=dev())
    sa = torch.full(lead[:-1] + (H // 128, lead[-1]), -7.0, device=dev())
    fg.dispatch_quant(x, p, w=None if w is None else to_dev(w), pow2=pow2, Q=Q, sa=sa)
    slots = host(p.slots)
    real = slots >= 0
    v = host(x)[np.maximum(slots, 0) // k]
    if weighted:
        v = v * w.reshape(-1)[np.maximum(slots, 0)][:, None]
    codes, scales = oracle.quantize_act_1x128(v, pow2)
    got_q = host(Q).reshape(-1, H)
    got_s = np.moveaxis(host(sa), -2, -1).reshape(-1, H // 128)
    assert np.array_equal(got_q[real], codes[real]) and np.array_equal(got_s[real], scales[real])
    assert np.all(got_q[~real] == 0x55) and np.all(got_s[~real] == -7.0)


@pytest.mark.parametrize("layout,T,k,G", PLANS)
@pytest.mark.parametrize("N", [8, 200, 2048, 7176])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("weighted,with_base", [(True, False), (True, True), (False, False)])
def test_combine(layout, T, k, G, N, dtype, weighted, with_base):
    print(f"combine {layout} {T}x{k} G={G} N={N} {dtype} w={weighted} base={with_base}", flush=True)
    rng = np.random.default_rng(N + T)
    p = make_plan(layout, T, k, G)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    y = torch.full(p.lead + (N,), float("nan"), dtype=td, device=dev())     # rows without a slot are never read into a sum
    real = to_dev((host(p.slots) >= 0))
    y.view(-1, N)[real] = torch.from_numpy(rng.standard_normal((int(real.sum()), N)).astype(np.float32)).to(dev(), td)
    w = rng.standard_normal((T, k)).astype(np.float32) if weighted else None
    base = to_dev(rng.standard_normal((T, N)).astype(np.float32), td) if with_base else None
    out = fg.combine(y, p, w=None if w is None else to_dev(w), base=base)
    ref, size = rowref.combine(host(y), host(p.rows), w, None if base is None else host(base))
    assert out.dtype == td and np.all(near(host(out), ref, 2 * (k + 2) * U32 * size, dtype))
    if with_base:   # in place on the base
        assert torch.equal(fg.combine(y, p, w=to_dev(w), base=base, out=base), out)
    if not weighted and not with_base:
        assert torch.equal(fg.dispatch_grad(y, p), out)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("weighted,with_base", [(True, True), (False, False)])
def test_combine_large_output(dtype, weighted, with_base):
    """An output past the size from which it is stored past the caches."""
    test_combine("contiguous", 2400, 2, 4, 7176, dtype, weighted, with_base)


def grad_inputs(layout, T, k, G, N, dtype):
    rng = np.random.default_rng(N + T + 1)
    p = make_plan(layout, T, k, G)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    y = to_dev(rng.standard_normal(p.lead + (N,)).astype(np.float32), td)
    dout = to_dev(rows_input(rng, (T, N)), td)
    w = rng.standard_normal((T, k)).astype(np.float32)
    return p, y, dout, w, td


def check_dw(dw, p, y, dout, N):
    rows, d = host(p.rows), host(dout).astype(np.float64)
    yy = host(y).reshape(-1, N).astype(np.float64)
    for t in range(rows.shape[0]):
        for j in range(rows.shape[1]):
            if rows[t, j] < 0:
                assert dw[t, j] == 0
            else:
                a = d[t] * yy[rows[t, j]]
                assert abs(dw[t, j] - a.sum()) <= (N / 256 + 24) * U32 * np.abs(a).sum()


@pytest.mark.parametrize("layout,T,k,G", PLANS)
@pytest.mark.parametrize("N", [8, 1000, 4096])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_combine_grad(layout, T, k, G, N, dtype):
    print(f"grad {layout} {T}x{k} G={G} N={N} {dtype}", flush=True)
    p, y, dout, w, td = grad_inputs(layout, T, k, G, N, dtype)
    dy = torch.full(p.lead + (N,), 9.0, dtype=td, device=dev())
    dy, dw = fg.combine_grad(dout, y, p, to_dev(w), dy=dy)
    check_dw(host(dw), p, y, dout, N)
    slots = host(p.slots)
    real = slots >= 0
    ref = host(dout)[np.maximum(slots, 0) // k].astype(np.float64) * w.reshape(-1)[np.maximum(slots, 0)][:, None]
    got = host(dy).reshape(-1, N)
    assert np.all(near(got, ref, U32 * np.abs(ref), dtype)[real]) and np.all(got[~real] == 9.0)
    none, dw2 = fg.combine_grad(dout, y, p, to_dev(w), with_dy=False)
    assert none is None and torch.equal(dw, dw2)


@pytest.mark.parametrize("layout,T,k,G", PLANS)
@pytest.mark.parametrize("N", [128, 4096])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_combine_grad_quant(layout, T, k, G, N, pow2, dtype):
    """The E4M3 gradient is dispatch_quant's of the weighted rows, bit for bit; the weights' gradient as in 64 bits."""
    print(f"grad quant {layout} {T}x{k} G={G} N={N} pow2={pow2} {dtype}", flush=True)
    p, y, dout, w, _ = grad_inputs(layout, T, k, G, N, dtype)
    lead = p.lead
    mk = lambda: (torch.full(lead + (N,), 0x55, dtype=torch.uint8, device=dev()),  # noqa: E731
                  torch.full(lead[:-1] + (N // 128, lead[-1]), -7.0, device=dev()))
    Q, sa = mk()
    Q2, sa2 = mk()
    Q, sa, dw = fg.combine_grad_quant(dout, y, p, to_dev(w), pow2=pow2, Q=Q, sa=sa)
    fg.dispatch_quant(dout, p, w=to_dev(w), pow2=pow2, Q=Q2, sa=sa2)
    assert torch.equal(Q, Q2) and torch.equal(sa, sa2)
    check_dw(host(dw), p, y, dout, N)


@pytest.mark.parametrize("layout", ["contiguous", "masked"])
@pytest.mark.parametrize("T", [511, 512])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_combine_grad_long_rows(layout, T, dtype):
    """Long rows on both sides of the number of tokens from which a token has fewer threads."""
    test_combine_grad(layout, T, 2, 4, 4104, dtype)
    test_combine_grad_quant(layout, T, 2, 4, 4224, False, dtype)


@pytest.mark.parametrize("dtype,T", [("bf16", 2400), ("fp32", 1201)])
def test_combine_grad_large_input(dtype, T):
    """More of y than the size from which it is read past the caches."""
    test_combine_grad("contiguous", T, 4, 6, 7176, dtype)


def test_combine_gradient_against_differences():
    """<dout, combine(y, w)> along random directions of y and w, in fp32 inputs (combine is bilinear: no truncation error)."""
    T, k, G, N = 20, 3, 4, 64
    rng = np.random.default_rng(5)
    p = make_plan("contiguous", T, k, G)
    y = to_dev(rng.standard_normal(p.lead + (N,)).astype(np.float32))
    dout = to_dev(rng.standard_normal((T, N)).astype(np.float32))
    w = to_dev(rng.standard_normal((T, k)).astype(np.float32))
    dy, dw = fg.combine_grad(dout, y, p, w, dy=torch.zeros_like(y))
    dirw = to_dev(rng.standard_normal((T, k)).astype(np.float32))
    diry = to_dev(rng.standard_normal(p.lead + (N,)).astype(np.float32))
    f = lambda y_, w_: (dout.double() * fg.combine(y_, p, w=w_).double()).sum()  # noqa: E731
    for num, ana in (((f(y, w + dirw) - f(y, w - dirw)) / 2, (dw.double() * dirw.double()).sum()),
                     ((f(y + diry, w) - f(y - diry, w)) / 2, (dy.double() * diry.double()).sum())):
        size = 8.0 * T * k * N     # every term of the two sums is of order one
        assert abs(float(num) - float(ana)) <= 8 * (k + 4) * U32 * size


def test_dispatch_gradient_is_the_copies_transpose():
    """<dispatch copies of x, dA> = <x, dispatch_grad(dA)>."""
    T, k, G, N = 50, 4, 6, 256
    rng = np.random.default_rng(6)
    p = make_plan("masked", T, k, G)
    dA = rng.standard_normal(p.lead + (N,)).astype(np.float32)
    x = rng.standard_normal((T, N)).astype(np.float32)
    slots = host(p.slots)
    copies = np.where((slots >= 0)[:, None], x[np.maximum(slots, 0) // k], 0)
    left = (copies.astype(np.float64) * dA.reshape(-1, N)).sum()
    dx = host(fg.dispatch_grad(to_dev(dA), p)).astype(np.float64)
    assert abs(left - (dx * x).sum()) <= 4 * (k + 2) * U32 * np.abs(copies * dA.reshape(-1, N)).sum()


def test_rows_past_32_bit_offsets():
    """A sorted layout of more than 2^32 bytes: its last rows are reached."""
    N, T, k = 7168, 64, 2
    n_rows = 2 ** 32 // (2 * N) + 1024
    if torch.cuda.mem_get_info()[0] < 8 * 2 * N * n_rows // 4:
        pytest.skip("not enough device memory")
    rng = np.random.default_rng(8)
    rows = torch.from_numpy(rng.permutation(np.arange(n_rows - 512, n_rows))[:T * k].reshape(T, k).astype(np.int32)).to(dev())
    slots = torch.full((n_rows,), -1, dtype=torch.int32, device=dev())
    slots[rows.view(-1).long()] = torch.arange(T * k, dtype=torch.int32, device=dev())
    p = fg.Plan.masked(rows, slots, torch.tensor([n_rows], dtype=torch.int32, device=dev()), n_rows)
    y = torch.zeros(1, n_rows, N, dtype=torch.bfloat16, device=dev())
    y[0, -512:] = torch.from_numpy(rng.standard_normal((512, N)).astype(np.float32)).to(dev(), torch.bfloat16)
    out = fg.combine(y, p)
    pair = y[0][rows.long()].float()
    assert torch.equal(out, (pair[:, 0] + pair[:, 1]).bfloat16())
    dout = torch.ones(T, N, dtype=torch.bfloat16, device=dev())
    w = torch.full((T, k), 2.0, device=dev())
    dy, dw = fg.combine_grad(dout, y, p, w, dy=y.clone())
    assert bool((dy[0][rows.long()] == 2.0).all())
    assert torch.equal(dy[0, :-512], y[0, :-512])
    s = y[0][rows.long()].double()
    assert bool(((dw.double() - s.sum(2)).abs() <= 64 * U32 * s.abs().sum(2)).all())


# ------------------------------------------------------------------ adapters
@pytest.mark.parametrize("T,L,align", [(1, 1, 16), (7, 3, 16), (64, 64, 16), (33, 5, 32), (200, 3, 64), (1000, 9, 64),
                                       (130, 2, 128), (50, 4, 48)])
@pytest.mark.parametrize("R,K,N", [(8, 128, 8), (16, 256, 200), (24, 384, 1000), (32, 128, 512), (64, 1024, 264),
                                   (72, 256, 2048), (128, 640, 136)])
def test_adapters(T, L, align, R, K, N):
    print(f"adapters T={T} L={L} align={align} R={R} K={K} N={N}", flush=True)
    rng = np.random.default_rng(T + R)
    ids = rng.integers(-1, L, T).astype(np.int32)
    x, D = bf16(rng.standard_normal((T, K))), bf16(rng.standard_normal((T, N)))
    A, B = bf16(rng.standard_normal((L, R, K)) * K ** -0.5), bf16(rng.standard_normal((L, N, R)))
    scales = (rng.random(L) + 0.5).astype(np.float32)
    p = fg.plan_contiguous(to_dev(ids.reshape(T, 1)), L, align)
    before = D.clone()
    out = fg.adapters(D, x, A, B, to_dev(scales), p)
    ref, d_size = rowref.adapters(host(D), host(x), host(A), host(B), scales, ids)
    # both products' fp32 sums and the 2^-16 of splitting h, and the addition
    tol = ((K + R + 16) * U32 + 2.0 ** -16) * d_size + U32 * np.abs(ref)
    got = host(out)
    assert torch.equal(D, before)
    assert np.all(near(got, ref, tol, "bf16"))
    assert np.array_equal(got[ids < 0], host(D)[ids < 0])
    assert fg.adapters(D, x, A, B, to_dev(scales), p, out=D) is D and torch.equal(D, out)


@pytest.mark.parametrize("R", [24, 64, 128])
def test_adapters_large_output(R):
    """An output past the size from which it is stored past the caches."""
    test_adapters(4112, 3, 64, R, 256, 4096)


def test_adapters_without_any():
    D, x = bf16(np.ones((5, 64))), bf16(np.ones((5, 128)))
    A, B = bf16(np.ones((2, 16, 128))), bf16(np.ones((2, 64, 16)))
    p = fg.plan_contiguous(torch.full((5, 1), -1, dtype=torch.int32, device=dev()), 2, 16)
    assert torch.equal(fg.adapters(D, x, A, B, torch.ones(2, device=dev()), p), D)


def test_adapters_other_rows_cannot_leak():
    """NaN and infinities in one token or one adapter stay there."""
    T, L, R, K, N = 40, 3, 16, 256, 96
    rng = np.random.default_rng(9)
    ids = rng.integers(0, L, T).astype(np.int32)
    x, D = rng.standard_normal((T, K)), rng.standard_normal((T, N))
    A, B = rng.standard_normal((L, R, K)), rng.standard_normal((L, N, R))
    p = fg.plan_contiguous(to_dev(ids.reshape(T, 1)), L, 64)
    s = torch.ones(L, device=dev())
    good = fg.adapters(bf16(D), bf16(x), bf16(A), bf16(B), s, p)
    x[0], A[2, 0, 0], B[2, 3, 1] = np.nan, np.inf, np.nan
    bad = fg.adapters(bf16(D), bf16(x), bf16(A), bf16(B), s, p)
    clean = to_dev((ids != 2) & (np.arange(T) != 0))
    assert torch.equal(bad[clean], good[clean]) and bool(clean.any())
    assert bool(bad[0].isnan().any())


# ------------------------------------------------------------------ streams, graphs, refusals
def whole_path(logits, x, w13, w2):
    """Route, sort, dispatch, two grouped GEMMs, combine, and the weights' gradient."""
    ids, w = fg.route_topk(logits, 3, renorm=True)
    p = fg.plan_contiguous(ids, w13[0].shape[0])
    zero = lambda *s, d=torch.uint8: torch.zeros(s, dtype=d, device=x.device)  # noqa: E731
    A, sa = fg.dispatch_quant(x, p)
    Q, sq, _ = fg.grouped_contiguous_swiglu_quant(A, sa, *w13, p.m_indices)
    D = zero(p.capacity, w2[0].shape[1], d=torch.bfloat16)
    fg.grouped_contiguous(Q, sq, *w2, D, p.m_indices)
    out = fg.combine(D, p, w=w)
    _, dw = fg.combine_grad(out, D, p, w, with_dy=False)
    dl = fg.route_topk_grad(logits, ids, dw, renorm=True)
    low = fg.plan_contiguous(ids[:, :1].contiguous(), w13[0].shape[0], align=16)
    out2 = fg.adapters(out, x, ADAPT["A"], ADAPT["B"], ADAPT["s"], low)
    return ids, w, p.rows, out, dw, dl, out2


ADAPT = {}


def path_inputs(T=100, E=6, H=256, I=128, seed=1):
    gen = torch.Generator(device=dev())
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device=dev(), generator=gen)  # noqa: E731
    w13, w2 = fg.quant_weight_128x128(rnd(E, 2 * I, H)), fg.quant_weight_128x128(rnd(E, H, I))
    ADAPT.update(A=rnd(E, 16, H).bfloat16(), B=rnd(E, H, 16).bfloat16(), s=rnd(E))
    return rnd(T, E), rnd(T, H).bfloat16(), w13, w2


def test_path_on_another_stream_and_in_a_graph():
    args = path_inputs()
    want = [t.clone() for t in whole_path(*args)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = whole_path(*args)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = whole_path(*args)
    for r in range(4):
        for t in got:
            t.zero_()
        whole_path(*args)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {r}"
    # new inputs in the same buffers: the replay follows them
    args[0].copy_(args[0].flip(0))
    args[1].copy_(args[1].flip(0))
    g.replay()
    torch.cuda.synchronize()
    again = [t.clone() for t in got]
    assert all(torch.equal(a, b) for a, b in zip(again, whole_path(*args)))
    assert not torch.equal(again[0], want[0])


def test_refusals():
    """Arguments the binding refuses before any launch."""
    d = dev()
    lg = torch.randn(4, 8, device=d)
    ids, w = fg.route_topk(lg, 2)
    p = fg.plan_contiguous(ids, 8)
    with pytest.raises(ValueError):
        fg.route_topk(lg, 9)
    with pytest.raises(ValueError):
        fg.route_topk(lg, 0)
    with pytest.raises(ValueError):
        fg.route_topk(lg, 2, score="tanh")
    with pytest.raises(TypeError):
        fg.route_topk(lg.half(), 2)
    with pytest.raises(ValueError, match="contiguous"):
        fg.route_topk(lg.t(), 2)
    with pytest.raises(ValueError):
        fg.route_topk(lg, 2, bias=torch.zeros(7, device=d))
    with pytest.raises(ValueError, match="device tensor"):
        fg.route_topk(lg.cpu(), 2, ids=ids)
    with pytest.raises(TypeError):
        fg.plan_contiguous(ids.long(), 8)
    with pytest.raises(ValueError):
        fg.plan_contiguous(ids, 1025)
    with pytest.raises(fg.FGError):
        fg.plan_contiguous(ids, 8, align=0)
    with pytest.raises(ValueError):
        fg.plan_masked(ids, 8, 0)
    x = torch.randn(4, 256, device=d)
    with pytest.raises(ValueError):
        fg.dispatch_quant(x[:3].contiguous(), p)
    with pytest.raises(ValueError):
        fg.dispatch_quant(torch.randn(4, 200, device=d), p)
    with pytest.raises(TypeError):
        fg.dispatch_quant(x, p, w=w.double())
    y = torch.randn(p.capacity, 64, device=d)
    with pytest.raises(ValueError):
        fg.combine(y[:128].contiguous() if p.capacity > 128 else y[:1].contiguous(), p)
    with pytest.raises(ValueError):
        fg.combine(y[:, :60].contiguous(), p)
    with pytest.raises(TypeError):
        fg.combine(y, p, base=torch.zeros(4, 64, device=d, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        fg.combine_grad_quant(torch.randn(4, 64, device=d), y, p, w)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=d)  # noqa: E731
    one = fg.plan_contiguous(ids[:, :1].contiguous(), 8, align=16)
    ok = dict(D=bf(4, 64), x=bf(4, 128), A=bf(8, 16, 128), B=bf(8, 64, 16), scales=torch.ones(8, device=d), plan=one)
    fg.adapters(**ok)
    for bad in (dict(plan=p), dict(x=bf(3, 128)), dict(A=bf(8, 20, 128)), dict(A=bf(7, 16, 128)), dict(B=bf(8, 16, 64)),
                dict(plan=fg.plan_contiguous(ids[:, :1].contiguous(), 8, align=8)),
                dict(plan=fg.plan_masked(ids[:, :1].contiguous(), 8, 4))):
        with pytest.raises(ValueError):
            fg.adapters(**{**ok, **bad})
    with pytest.raises(TypeError):
        fg.adapters(**{**ok, "D": torch.zeros(4, 64, device=d)})
    with pytest.raises(ValueError):
        fg.Plan.masked(p.rows, p.slots, ids.view(-1)[:3], 7)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("H", [128, 1024, 1152])
def test_dispatch_quant_extreme_blocks(H, pow2):
    """Signed zeros, blocks of tiny and of huge values, values that are exact ties of the code grid: bit for bit the oracle's."""
    T, k, G = 64, 2, 3
    rng = np.random.default_rng(H)
    x = rng.standard_normal((T, H)).astype(np.float32)
    for i, e in enumerate(range(-110, 120, 8)):      # scales from 2^-117 (below 2^-141 amax / 448 is no fp32 number)
        x[i] *= np.float32(2.0 ** e)
    x[40] = 0.0
    x[41] = -0.0
    x[42, ::2] = -0.0
    t = oracle.decode_table()[:0x7F]
    ties = ((t[:-1] + t[1:]) / 2).astype(np.float32)
    for i in range(43, 60):
        x[i, :126] = ties * rng.choice([-1, 1], 126)
        x[i, 126] = 448.0
        x[i] *= np.float32(1 + (i - 43) / 16)
    p = make_plan("contiguous", T, k, G, drop=False)
    w = (2.0 ** rng.integers(-3, 3, (T, k))).astype(np.float32)
    for weight in (None, w):
        Q, sa = fg.dispatch_quant(to_dev(x), p, w=None if weight is None else to_dev(weight), pow2=pow2)
        slots = host(p.slots)
        real = slots >= 0
        v = x[np.maximum(slots, 0) // k]
        if weight is not None:
            v = v * weight.reshape(-1)[np.maximum(slots, 0)][:, None]
        codes, scales = oracle.quantize_act_1x128(v, pow2)
        assert np.array_equal(host(sa).T[real], scales[real])
        assert np.array_equal(host(Q)[real], codes[real])


@pytest.mark.parametrize("layout", ["contiguous", "masked"])
def test_no_tokens_anywhere(layout):
    """An empty batch goes through every call and comes out empty."""
    ids, w = fg.route_topk(torch.empty(0, 8, device=dev()), 2)
    p = fg.plan_contiguous(ids, 8) if layout == "contiguous" else fg.plan_masked(ids, 8, 4)
    x = torch.empty(0, 256, dtype=torch.bfloat16, device=dev())
    Q, sa = fg.dispatch_quant(x, p)
    assert Q.shape == p.lead + (256,) and sa.shape[-1] == p.lead[-1]
    y = torch.zeros(p.lead + (256,), dtype=torch.bfloat16, device=dev())
    assert fg.combine(y, p, w=w).shape == (0, 256) and fg.dispatch_grad(y, p).shape == (0, 256)
    _, dw = fg.combine_grad(x, y, p, w)
    assert dw.shape == (0, 2)
    assert fg.combine_grad_quant(x, y, p, w)[2].shape == (0, 2)
    low = fg.plan_contiguous(torch.empty(0, 1, dtype=torch.int32, device=dev()), 3, align=64)
    A, B = (torch.zeros(s, dtype=torch.bfloat16, device=dev()) for s in ((3, 16, 256), (3, 64, 16)))
    D = torch.empty(0, 64, dtype=torch.bfloat16, device=dev())
    assert fg.adapters(D, x, A, B, torch.ones(3, device=dev()), low).shape == (0, 64)

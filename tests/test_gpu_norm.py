"""The norms around a block and their gradient on the GPU against their definitions in 64 bits, to the
bounds of fp32 arithmetic that normref.py derives; a bf16 output has to be the bf16 rounding of some value
within them. 8-bit outputs against the quantisers' rule on values within those bounds."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_02_amd as fg
import normref
import oracle
from fgtest import dev, to_dev
from normref import U32

pytestmark = pytest.mark.gpu

EPS = 1e-6
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
# N at the borders of the kernels' shapes, T from one row to more than there are workgroups
SIZES = [(1, 8), (3, 24), (7, 512), (5, 520), (4, 2048), (6, 2056), (9, 4096), (5, 4104), (6, 7168), (3, 8192), (3, 8200),
         (2, 16384), (4099, 64), (1100, 1032), (530, 2304)]
PARTS = [dict(y=True, pre=True, post=True, gate="channel"), dict(y=True, pre=True, post=True, gate="token"),
         dict(y=True, pre=True, post=False, gate="none"), dict(y=True, pre=False, post=True, gate="none"),
         dict(y=True, pre=True, post=False, gate="channel"), dict(y=True, pre=False, post=False, gate="token"),
         dict(y=False, pre=True, post=False, gate="none")]


def host(t):
    return None if t is None else t.double().cpu().numpy()


def near(got, ref, tol, dtype):
    """got is ref to within tol, rounded to its type: rounding is monotone, so a bf16 value lies between the
    roundings of ref - tol and ref + tol."""
    if dtype == "fp32":
        return np.abs(got - ref) <= tol + U32 * np.abs(ref) + 1e-38
    lo, hi = (torch.from_numpy(np.asarray(v, np.float64)).to(torch.bfloat16).double().numpy() for v in (ref - tol, ref + tol))
    return (lo <= got) & (got <= hi)


def inputs(T, N, dtype, y, pre, post, gate, seed, dr=True):
    rng = np.random.default_rng(seed)
    rows = lambda: rng.standard_normal((T, N)) * np.where(rng.random((T, 1)) < 0.1, 50.0, 1.0)  # noqa: E731
    d = lambda v: None if v is None else to_dev(v.astype(np.float32), DTYPES[dtype])  # noqa: E731
    f = lambda v: None if v is None else to_dev(v.astype(np.float32))  # noqa: E731
    x, b = rows(), rows() if y else None
    if T > 2:
        x[1] = 0.0                                   # a row of zeros, and one where the eps counts
        x[2] *= 1e-4
        if y:
            b[2] = 0.0
            b[1] *= 1e-3
    s = dict(x=d(x), y=d(b), pre=f(1 + 0.1 * rng.standard_normal(N)) if pre else None,
             post=f(1 + 0.1 * rng.standard_normal(N)) if post else None,
             gate={"none": None, "channel": f(rng.standard_normal(N)), "token": f(rng.standard_normal((T, 1)))}[gate],
             dh=d(rng.standard_normal((T, N))) if pre else None, dr=d(rng.standard_normal((T, N))) if dr or not pre else None)
    return s


@pytest.mark.parametrize("parts", PARTS, ids=lambda p: "-".join(f"{k}={v}" for k, v in p.items()))
@pytest.mark.parametrize("T,N", SIZES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_forward_and_gradient(T, N, dtype, parts):
    print(f"block_norm {T}x{N} {dtype} {parts}", flush=True)
    s = inputs(T, N, dtype, seed=T + N, **parts)
    how = dict(alpha=0.75, beta=-1.5, eps=EPS)
    r, h, sc = fg.block_norm(s["x"], s["y"], pre=s["pre"], post=s["post"], gate=s["gate"], **how)
    assert sc is None and (h is None) == (not parts["pre"])
    if not parts["y"]:
        assert r is s["x"]
    a = [host(s[n]) for n in ("x", "y", "pre", "post", "gate")]
    (rr, r_tol), rest = normref.forward(*a, 0.75 if parts["y"] else 1.0, -1.5, EPS)
    assert np.all(near(host(r), rr, r_tol, dtype))
    if parts["pre"]:
        assert np.all(near(host(h), *rest, dtype))
    got = fg.block_norm_grad(r, dh=s["dh"], dr=s["dr"], y=s["y"], pre=s["pre"], post=s["post"], gate=s["gate"], **how)
    check_gradient(got, r, s, 0.75, -1.5, dtype)


# rows side by side in a wave (four up to 128 columns, two up to 256), whole steps of them and not, and rows
# of two waves, several a workgroup
SHORT = [(1, 128), (2, 136), (3, 120), (4, 16), (5, 128), (6, 256), (7, 248), (1030, 128), (1027, 264), (2051, 200), (16390, 128),
         (9001, 72), (9001, 256), (701, 528), (2051, 1000), (5000, 1024)]


@pytest.mark.parametrize("parts", PARTS, ids=lambda p: "-".join(f"{k}={v}" for k, v in p.items()))
@pytest.mark.parametrize("T,N", SHORT)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_short_rows(T, N, dtype, parts):
    test_forward_and_gradient(T, N, dtype, parts)


@pytest.mark.parametrize("T,N", [(1, 128), (3, 128), (4, 128), (5, 256), (6, 256), (1001, 128), (7001, 256), (26001, 128)])
@pytest.mark.parametrize("quant", ["e4m3", "e4m3_pow2", "int8"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("y", [True, False])
def test_short_rows_quantised(T, N, dtype, quant, y):
    test_quantised_output(T, N, dtype, quant, y)


@pytest.mark.parametrize("T,N", [(2, 16), (5, 48), (9, 112), (11, 144), (33, 240)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_short_rows_of_odd_lengths_as_integers(T, N, dtype):
    for y in (True, False):
        test_quantised_output(T, N, dtype, "int8", y)


def check_gradient(got, r, s, alpha, beta, dtype):
    ref = normref.backward(host(r), host(s["dh"]), host(s["dr"]), *[host(s[n]) for n in ("y", "pre", "post", "gate")],
                           alpha, beta, EPS)
    for name, v in zip(("dx", "dy", "dgate", "dpre", "dpost"), got):
        assert (v is None) == (name not in ref), name
        if v is not None:
            ok = near(host(v), *ref[name], dtype if name in ("dx", "dy") else "fp32")
            assert np.all(ok), (name, int((~ok).sum()), ok.size)


@pytest.mark.parametrize("T,N", [(1, 128), (5, 512), (9, 640), (70, 2048), (3, 4224), (20, 7168), (2, 16384)])
@pytest.mark.parametrize("quant", ["e4m3", "e4m3_pow2", "int8"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("y", [True, False])
def test_quantised_output(T, N, dtype, quant, y):
    print(f"block_norm {T}x{N} {dtype} to {quant}, y {y}", flush=True)
    s = inputs(T, N, dtype, y, True, y, "channel" if y else "none", seed=N)
    how = dict(pre=s["pre"], post=s["post"], gate=s["gate"], alpha=0.5, beta=2.0, eps=EPS)
    r, h, sc = fg.block_norm(s["x"], s["y"], quant=quant, **how)
    plain = fg.block_norm(s["x"], s["y"], **how)
    assert torch.equal(r, plain[0])
    # the same arithmetic in fp32 rows gives the values that were quantised
    exact = fg.block_norm(s["x"].float(), None if s["y"] is None else s["y"].float(), **how)[1].cpu().numpy()
    if quant == "int8":
        amax = np.abs(exact).max(1)
        want = np.where(amax == 0, np.float32(1), np.maximum(amax / np.float32(127), np.float32(2.0 ** -126)))
        assert h.dtype == torch.int8 and np.array_equal(sc.cpu().numpy(), want)
        assert np.array_equal(h.cpu().numpy(), np.rint(exact / want[:, None]).astype(np.int8))
        return
    codes, scales = oracle.quantize_act_1x128(exact, quant == "e4m3_pow2")
    assert np.array_equal(sc.cpu().numpy().T, scales)
    assert np.array_equal(h.cpu().numpy(), codes)


def test_tiny_streams_quantise():
    """h below the normal numbers and scales below 2^-90: the paths beside the three-step quotient."""
    N = 256
    x = torch.randn(4, N, device=dev())
    for size in (1e-42, 1e-36, 1e-30):
        pre = torch.full((N,), size, device=dev())
        want = fg.block_norm(x, pre=pre)[1]
        q, s = fg.block_norm(x, pre=pre, quant="int8")[1:]
        rq, rs = fg.quant_int8(want)
        assert torch.equal(q, rq) and torch.equal(s, rs)
        for quant, alone in (("e4m3", fg.quant_act_1x128), ("e4m3_pow2", fg.quant_act_1x128_pow2)):
            q, s = fg.block_norm(x, pre=pre, quant=quant)[1:]
            rq, rs = alone(want)
            assert torch.equal(q, rq) and torch.equal(s, rs), quant


def test_vectors_of_any_alignment():
    """Weights, gates and scales start at any float; rows at 16 bytes, or the call is refused."""
    s = inputs(9, 264, "bf16", True, True, True, "channel", 4)
    odd = lambda v: torch.cat([v.new_zeros(1), v])[1:]  # noqa: E731
    how = dict(pre=s["pre"], post=s["post"], gate=s["gate"])
    shifted = {k: odd(v) for k, v in how.items()}
    want, got = fg.block_norm(s["x"], s["y"], **how), fg.block_norm(s["x"], s["y"], **shifted)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    rest = dict(dh=s["dh"], dr=s["dr"], y=s["y"])
    assert all(torch.equal(a, b) for a, b in zip(fg.block_norm_grad(want[0], **rest, **how),
                                                 fg.block_norm_grad(want[0], **rest, **shifted)))
    scales = torch.zeros(10, device=dev())[1:]
    q, got = fg.block_norm(s["x"][:, :256].contiguous(), pre=odd(s["pre"][:256]), quant="int8", s=scales)[1:]
    want = fg.block_norm(s["x"][:, :256].contiguous(), pre=s["pre"][:256].contiguous(), quant="int8")
    assert got is scales and torch.equal(got, want[2]) and torch.equal(q, want[1])
    x = torch.zeros(9 * 264 + 1, dtype=torch.bfloat16, device=dev())[1:].view(9, 264)
    with pytest.raises(fg.FGError):
        fg.block_norm(x, pre=s["pre"])
    with pytest.raises(fg.FGError):
        fg.block_norm_grad(s["x"], dr=x)


@pytest.mark.parametrize("parts", PARTS[:4], ids=lambda p: "-".join(f"{k}={v}" for k, v in p.items()))
def test_gradient_against_differences(parts):
    """Central differences of the 64-bit forward against the kernels' gradient: the step's error is h^2 times a third
    derivative of about 1, the tolerance 2e-4 of the gradient's size above fp32's own."""
    T, N, step = 5, 64, 1e-4
    s = inputs(T, N, "fp32", seed=9, **parts)
    how = dict(alpha=0.75, beta=-1.5, eps=1e-2)       # an eps that keeps the small rows' slopes small
    v = {n: host(s[n]) for n in ("x", "y", "pre", "post", "gate")}
    args = dict(v)

    def loss(**change):
        a = {**args, **change}
        (r, _), rest = normref.forward(a["x"], a["y"], a["pre"], a["post"], a["gate"], 0.75, -1.5, 1e-2)
        total = 0.0 if s["dr"] is None else (r * host(s["dr"])).sum()
        return total + (0.0 if rest is None else (rest[0] * host(s["dh"])).sum())

    r = normref.forward(*v.values(), 0.75, -1.5, 1e-2)[0][0]
    if not parts["y"]:
        r = v["x"]
    got = fg.block_norm_grad(to_dev(r.astype(np.float32)), dh=s["dh"], dr=s["dr"], y=s["y"], pre=s["pre"], post=s["post"],
                             gate=s["gate"], **how)
    rng = np.random.default_rng(1)
    for name, g in zip(("x", "y", "gate", "pre", "post"), got):
        if g is None:
            continue
        g = host(g)
        size = np.abs(g).max()
        for _ in range(12):
            at = tuple(rng.integers(n) for n in g.shape)
            up, down = v[name].copy(), v[name].copy()
            up[at] += step
            down[at] -= step
            slope = (loss(**{name: up}) - loss(**{name: down})) / (2 * step)
            if name == "x" and not parts["y"]:
                slope *= 0.75                         # without y the stream is x, and alpha is dx's factor alone
            assert abs(slope - g[at]) <= 2e-4 * size + 1e-6, (name, at, slope, g[at])


def test_in_place():
    s = inputs(40, 1032, "bf16", True, True, True, "channel", 5)
    how = dict(pre=s["pre"], post=s["post"], gate=s["gate"])
    r, h, _ = fg.block_norm(s["x"], s["y"], **how)
    dx, dy, *vectors = fg.block_norm_grad(r, dh=s["dh"], dr=s["dr"], y=s["y"], **how)
    x2, y2 = s["x"].clone(), s["y"].clone()
    r2, h2, _ = fg.block_norm(x2, y2, r=x2, h=y2, **how)
    assert r2 is x2 and h2 is y2 and torch.equal(x2, r) and torch.equal(y2, h)
    for into in ("dr", "dh"):
        t = {n: s[n].clone() for n in ("dr", "dh", "y")}
        got = fg.block_norm_grad(r, dh=t["dh"], dr=t["dr"], y=t["y"], dx=t[into], dy=t["y"], **how)
        assert got[0] is t[into] and torch.equal(got[0], dx) and torch.equal(got[1], dy)
        assert all(torch.equal(a, b) for a, b in zip(got[2:], vectors))


def test_norm_alone_in_place():
    s = inputs(20, 520, "fp32", False, True, False, "none", 3)
    want = fg.block_norm(s["x"], pre=s["pre"])[1]
    x = s["x"].clone()
    r, h, _ = fg.block_norm(x, pre=s["pre"], h=x)
    assert r is x and h is x and torch.equal(h, want)


def test_rows_past_4_gib():
    """Byte offsets past 2^32: sampled rows against the same rows alone, the sums over all rows against theirs in
    blocks (fp32 sums of 300000 terms in another order: (T + 40) u of the terms' absolute sum, normref's bound)."""
    T, N = 300000, 8192
    gen = torch.Generator(device="cuda").manual_seed(8)
    base = torch.randn(1000, N, device=dev(), generator=gen).bfloat16()
    x = base.repeat(T // 1000, 1)
    pre = torch.rand(N, device=dev(), generator=gen) + 0.5
    _, h, s = fg.block_norm(x, pre=pre, quant="e4m3")
    _, h0, s0 = fg.block_norm(base, pre=pre, quant="e4m3")
    for t in (0, 1, 131071, 262143, 262144, 299999):
        assert torch.equal(h[t], h0[t % 1000]) and torch.equal(s[:, t], s0[:, t % 1000]), t
    del h, s
    dx, _, _, dpre, _ = fg.block_norm_grad(x, dh=x, pre=pre)
    dx0, _, _, dpre0, _ = fg.block_norm_grad(base, dh=base, pre=pre)
    for t in (0, 1, 131071, 262143, 262144, 299999):
        assert torch.equal(dx[t], dx0[t % 1000]), t
    assert bool((dpre / (T // 1000) - dpre0).abs().le((T + 1100) * U32 * dpre0).all())    # dh = x: all terms positive


def test_infinities_and_nan_stay_in_their_rows():
    s = inputs(30, 520, "fp32", True, True, True, "token", 6)
    how = dict(pre=s["pre"], post=s["post"], gate=s["gate"])
    clean = fg.block_norm(s["x"], s["y"], **how)
    x, y = s["x"].clone(), s["y"].clone()
    x[3, 0], x[7, 519], y[11, 5], y[20, 519] = float("nan"), float("inf"), float("nan"), float("-inf")
    r, h, _ = fg.block_norm(x, y, **how)
    bad = torch.zeros(30, dtype=torch.bool, device=dev())
    bad[[3, 7, 11, 20]] = True
    assert torch.equal(r[~bad], clean[0][~bad]) and torch.equal(h[~bad], clean[1][~bad])
    assert bool(h[bad].isnan().any(1).all())
    got, want = (fg.block_norm_grad(a, dh=s["dh"], dr=s["dr"], y=b, **how) for a, b in ((r, y), (clean[0], s["y"])))
    assert torch.equal(got[0][~bad], want[0][~bad]) and torch.equal(got[1][~bad], want[1][~bad])


def test_no_rows():
    x = torch.empty(0, 128, device=dev())
    w = torch.ones(128, device=dev())
    r, h, s = fg.block_norm(x, x.clone(), pre=w, post=w, gate=w, quant="int8")
    assert r.shape == h.shape == (0, 128) and s.shape == (0,)
    dx, dy, dgate, dpre, dpost = fg.block_norm_grad(x, dh=x.clone(), y=x.clone(), pre=w, post=w, gate=w)
    assert dx.shape == dy.shape == (0, 128)
    for v in (dgate, dpre, dpost):
        assert bool((v == 0).all())


def test_captured_and_replayed():
    """Forward and gradient in a graph, replayed on new contents, with eager calls between the replays."""
    s = inputs(300, 2304, "bf16", True, True, True, "channel", 8)
    how = dict(pre=s["pre"], post=s["post"], gate=s["gate"])

    def both():
        r, h, sc = fg.block_norm(s["x"], s["y"], quant="e4m3", **how)
        return (r, h, sc) + fg.block_norm_grad(r, dh=s["dh"], dr=s["dr"], y=s["y"], **how)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    gen = torch.Generator(device="cuda").manual_seed(9)
    for i in range(4):
        for n in ("x", "y", "dh", "dr"):
            s[n].copy_(torch.randn(s[n].shape, device=dev(), generator=gen).bfloat16())
        want = both()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_concurrent_streams():
    jobs = [inputs(T, N, "bf16", True, True, True, "channel", T) for T, N in ((700, 1032), (33, 7168), (2000, 512))]
    run = lambda s: fg.block_norm_grad(s["x"], dh=s["dh"], dr=s["dr"], y=s["y"], pre=s["pre"], post=s["post"], gate=s["gate"])  # noqa: E731
    want = [run(s) for s in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[] for _ in jobs]
    for _ in range(4):
        for s, stream, g in zip(jobs, streams, got):
            with torch.cuda.stream(stream):
                g.append(run(s))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for once in g:
            assert all(torch.equal(a, b) for a, b in zip(once, w))


def test_refusals():
    x = torch.ones(4, 128, device=dev())
    w = torch.ones(128, device=dev())
    for err, call in [(ValueError, lambda: fg.block_norm(x)), (ValueError, lambda: fg.block_norm(x, pre=w, post=w)),
                      (ValueError, lambda: fg.block_norm(x, pre=w, gate=w)), (ValueError, lambda: fg.block_norm(x, pre=w[:64])),
                      (TypeError, lambda: fg.block_norm(x, pre=w.bfloat16())), (TypeError, lambda: fg.block_norm(x.half(), pre=w)),
                      (TypeError, lambda: fg.block_norm(x, x.bfloat16(), pre=w)), (ValueError, lambda: fg.block_norm(x, x[:3], pre=w)),
                      (ValueError, lambda: fg.block_norm(x, pre=w, eps=0.0)), (ValueError, lambda: fg.block_norm(x, pre=w, quant="fp8")),
                      (ValueError, lambda: fg.block_norm(x, x, quant="int8")), (ValueError, lambda: fg.block_norm(x.t(), pre=w)),
                      (ValueError, lambda: fg.block_norm(x[:, :64], pre=w[:64])), (ValueError, lambda: fg.block_norm(x, x, gate=torch.ones(5, 1, device=dev()))),
                      (ValueError, lambda: fg.block_norm(x.cpu(), pre=w)), (ValueError, lambda: fg.block_norm(x, pre=w, r=x.clone())),
                      (ValueError, lambda: fg.block_norm(x[:, :64].contiguous(), pre=w[:64].contiguous(), quant="e4m3")),
                      (ValueError, lambda: fg.block_norm_grad(x)), (ValueError, lambda: fg.block_norm_grad(x, dh=x)),
                      (ValueError, lambda: fg.block_norm_grad(x, pre=w, dr=x)), (ValueError, lambda: fg.block_norm_grad(x, dr=x, dy=x)),
                      (ValueError, lambda: fg.block_norm_grad(x, dr=x, post=w)), (TypeError, lambda: fg.block_norm_grad(x, dr=x.bfloat16()))]:
        with pytest.raises(err):
            call()


def test_outputs_that_would_not_be_written_are_refused():
    x, w = torch.ones(4, 128, device=dev()), torch.ones(128, device=dev())
    s = torch.ones(4, device=dev())
    for call in [lambda: fg.block_norm(x, x, h=x.clone()), lambda: fg.block_norm(x, pre=w, s=s), lambda: fg.block_norm(x, x, s=s)]:
        with pytest.raises(ValueError):
            call()

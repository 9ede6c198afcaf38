"""8-bit integer projections and the norms around a block, as cases that can be timed and compared.

Four operators, each with its plain form in elementary torch operations (32-bit arithmetic, one rounding at the end)
and its call of the library:

    quant      rows as 8-bit integers with one scale each: activations or weights as they are, token rows sorted
               by a plan, or the gated activation of a first projection
    gemm       D = A . B^T of 8-bit integers with a scale per token and per channel: dense, contiguous, masked
    norm       a block's output normed, gated and added to the scaled residual stream, and the stream's norm as the
               next block's operand
    norm_grad  its gradient: stream, block output, gate and both norms' weights

`own` chooses the side: False computes the plain form, True calls the library.
"""
import torch

own = False

DEVICE = "cuda"
TINY = 2.0 ** -126


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode batch's rows into one device's masked buffers: latency
        dict(name="quant_dispatch_decode", op="quant", mode="dispatch", layout="masked", T=128, k=8, E=16, G=16, M_max=256,
             H=7168, dtype="bf16", weighted=False),
        # a prefill batch's activations before a dense projection
        dict(name="quant_rows_prefill", op="quant", mode="rows", T=8192, H=7168, dtype="bf16"),
        # the gated activation between an expert's two projections, a ragged batch, a third of the experts elsewhere
        dict(name="quant_swiglu_ragged", op="quant", mode="swiglu", layout="contiguous", T=1001, k=3, E=24, G=16, align=128,
             H=2048, dtype="bf16"),
        # one decode step of a small batch through a dense projection: the weights are the traffic
        dict(name="gemm_decode", op="gemm", layout="dense", M=16, N=7168, K=7168),
        # odd sizes in every direction
        dict(name="gemm_ragged", op="gemm", layout="dense", M=1001, N=4104, K=2064),
        # a training-sized feed-forward projection: matrix cores
        dict(name="gemm_ffn", op="gemm", layout="dense", M=8192, N=7168, K=18432),
        # 8 experts' rows of a prefill batch
        dict(name="gemm_contiguous", op="gemm", layout="contiguous", T=8192, G=8, N=4096, K=7168),
        # 16 experts' buffers of a decode batch
        dict(name="gemm_masked", op="gemm", layout="masked", G=16, M_max=256, N=7168, K=2048),
        # one decode step between two blocks, both norms, a gate per channel: latency
        dict(name="norm_decode", op="norm", T=32, N=7168, dtype="bf16", y=True, pre=True, post=True, gate="channel", quant="none"),
        # a prefill batch between two blocks, the next block's operand in E4M3
        dict(name="norm_prefill", op="norm", T=8192, N=7168, dtype="bf16", y=True, pre=True, post=True, gate="none", quant="e4m3"),
        # the gradient of a ragged fp32 batch with a gate per token
        dict(name="grad_ragged", op="norm_grad", T=1001, N=2048, dtype="fp32", y=True, pre=True, post=True, gate="token", dr=True),
        # the gradient of a training batch
        dict(name="grad_train", op="norm_grad", T=8192, N=7168, dtype="bf16", y=True, pre=True, post=True, gate="channel",
             dr=True),
    ]


def log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quant", "gemm", "norm", "norm_grad"])
    if op == "quant":
        mode = rng.choice(["rows", "dispatch", "swiglu"])
        c = dict(op=op, mode=mode, dtype=rng.choice(["bf16", "fp32"]))
        if mode == "rows":
            c.update(T=log_int(rng, 1, 8192), H=16 * log_int(rng, 1, 448))
            return c
        E = log_int(rng, 8, 128)
        G = E if rng.random() < 0.5 else max(1, E // 4)
        layout = rng.choice(["contiguous", "masked"])
        c.update(layout=layout, T=log_int(rng, 1, 2048 if layout == "contiguous" else 512), k=rng.randint(1, 8), E=E, G=G)
        c.update(dict(align=128) if layout == "contiguous" else dict(M_max=rng.choice([64, 128, 256])))
        if mode == "dispatch":
            c.update(H=16 * log_int(rng, 4, 448), weighted=rng.random() < 0.3)
        else:
            c.update(H=128 * log_int(rng, 1, 16))
        return c
    if op == "gemm":
        layout = rng.choice(["dense", "dense", "contiguous", "masked"])
        N, K = 8 * log_int(rng, 8, 896), 16 * log_int(rng, 4, 448)
        if layout == "dense":
            return dict(op=op, layout=layout, M=log_int(rng, 1, 4096), N=N, K=K)
        G = log_int(rng, 1, 16)
        if layout == "contiguous":
            return dict(op=op, layout=layout, T=log_int(rng, 1, 2048), G=G, N=N, K=K)
        return dict(op=op, layout=layout, G=G, M_max=rng.choice([8, 64, 256]), N=N, K=K)
    y = rng.random() < 0.8
    c = dict(op=op, T=log_int(rng, 1, 8192), N=8 * log_int(rng, 8, 896), dtype=rng.choice(["bf16", "fp32"]), y=y,
             pre=not y or rng.random() < 0.8, post=y and rng.random() < 0.7,
             gate=rng.choice(["none", "channel", "token"]) if y else "none")
    if op == "norm_grad":
        c["dr"] = not c["pre"] or rng.random() < 0.7
        return c
    c["quant"] = rng.choice(["none", "e4m3", "int8"]) if c["pre"] else "none"
    if c["quant"] == "e4m3":
        c["N"] = -(-c["N"] // 128) * 128
    elif c["quant"] == "int8":
        c["N"] = -(-c["N"] // 16) * 16
    return c


# ------------------------------------------------------------------ inputs
def dtype_of(c):
    return torch.bfloat16 if c.get("dtype", "bf16") == "bf16" else torch.float32


def capacity(c):
    """Rows of the sorted layout, from sizes alone: every expert's segment may need align - 1 rows of padding."""
    if c["layout"] == "masked":
        return c["G"] * c["M_max"]
    slots, G, align = c["T"] * c["k"], c["G"], c["align"]
    return -(-(slots + min(slots, G) * (align - 1)) // align) * align


def rows_like(gen, *shape, dtype=torch.bfloat16):
    """Activations: N(0, 1), one row in a hundred scaled by 50."""
    x = torch.randn(*shape, device=DEVICE, generator=gen)
    x *= torch.where(torch.rand(*shape[:-1], 1, device=DEVICE, generator=gen) < 0.01, 50.0, 1.0)
    return x.to(dtype)


def expert_choice(c, gen):
    """Distinct experts per token, popular ones more often; experts of other devices come out of range (>= G)."""
    pull = torch.randn(c["E"], device=DEVICE, generator=gen)
    gumbel = -torch.log(-torch.log(torch.rand(c["T"], c["E"], device=DEVICE, generator=gen).clamp(1e-9, 1 - 1e-7)))
    return (0.5 * pull + gumbel).argsort(dim=1, descending=True)[:, :c["k"]].to(torch.int32).contiguous()


def sort_slots(c, ids):
    """The plan a program keeps: rows [T, k] (-1: none), slots [rows] (-1: none), and the layout's own index."""
    flat = ids.reshape(-1).long()
    G, cap, S = c["G"], capacity(c), flat.numel()
    key = torch.where((flat >= 0) & (flat < G), flat, G)
    key, order = torch.sort(key, stable=True)
    counts = torch.bincount(key, minlength=G + 1)
    rank = torch.arange(S, device=DEVICE) - (torch.cumsum(counts, 0) - counts)[key]
    if c["layout"] == "masked":
        start = torch.arange(G + 1, device=DEVICE) * c["M_max"]
        there = (key < G) & (rank < c["M_max"])
    else:
        padded = -(-counts // c["align"]) * c["align"]
        start = torch.cumsum(padded, 0) - padded
        there = key < G
    row = torch.where(there, start[key] + rank, cap)
    new = lambda n: torch.full((n,), -1, dtype=torch.int32, device=DEVICE)  # noqa: E731
    rows = new(S).scatter_(0, order, torch.where(there, row, -1).to(torch.int32)).view(ids.shape)
    slots = new(cap + 1).scatter_(0, row, order.to(torch.int32))[:cap].contiguous()
    p = dict(rows=rows, slots=slots)
    if c["layout"] == "masked":
        p["masked_m"] = counts[:G].clamp(max=c["M_max"]).to(torch.int32)
    else:
        p["m_indices"] = new(cap + 1).scatter_(0, row, key.to(torch.int32))[:cap].contiguous()
        p["offsets"] = start.to(torch.int32)
    return p


def int8_rows(gen, *shape):
    """8-bit operands as a program has them: normal rows quantised to their largest value, and their scales."""
    x = torch.randn(*shape, device=DEVICE, generator=gen)
    s = x.abs().amax(-1) / 127
    return torch.round(x / s[..., None]).to(torch.int8), s * torch.exp(0.5 * torch.randn(s.shape, device=DEVICE, generator=gen))


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "quant":
        if c["mode"] == "rows":
            s["x"] = rows_like(gen, c["T"], c["H"], dtype=dtype_of(c))
            return s
        s["ids"] = expert_choice(c, gen)
        s["plan"] = sort_slots(c, s["ids"])
        lead = (c["G"], c["M_max"]) if c["layout"] == "masked" else (capacity(c),)
        # the product's operand buffers, kept by the program; rows that hold no token stay as they are
        s["Q"] = torch.zeros(lead + (c["H"],), dtype=torch.int8, device=DEVICE)
        s["s"] = torch.zeros(lead, device=DEVICE)
        if c["mode"] == "dispatch":
            s["x"] = rows_like(gen, c["T"], c["H"], dtype=dtype_of(c))
            s["w"] = torch.rand(s["ids"].shape, device=DEVICE, generator=gen) + 0.05 if c["weighted"] else None
        else:
            s["h"] = rows_like(gen, *lead, 2 * c["H"], dtype=dtype_of(c))
        return s
    if c["op"] == "gemm":
        N, K = c["N"], c["K"]
        if c["layout"] == "dense":
            s["A"], s["sa"] = int8_rows(gen, c["M"], K)
            s["B"], s["sb"] = int8_rows(gen, N, K)
            s["D"] = torch.zeros(c["M"], N, dtype=torch.bfloat16, device=DEVICE)
            return s
        G = c["G"]
        s["B"], s["sb"] = int8_rows(gen, G, N, K)
        if c["layout"] == "masked":
            s["masked_m"] = torch.randint(0, c["M_max"] + 1, (G,), device=DEVICE, generator=gen).to(torch.int32)
            lead = (G, c["M_max"])
        else:
            share = torch.rand(G, device=DEVICE, generator=gen) + 0.15
            counts = (share / share.sum() * c["T"]).long()
            counts[0] += c["T"] - counts.sum()
            blocks = -(-counts // 128)
            M = -(-c["T"] // 128) * 128 + 128 * (G - 1)         # the most that any counts can need
            which = torch.repeat_interleave(torch.arange(G, device=DEVICE), blocks)
            first = torch.cumsum(blocks, 0) - blocks
            at = torch.arange(M, device=DEVICE)
            block = at // 128
            g = torch.nn.functional.pad(which, (0, M // 128 - which.numel()), value=-1)[block]
            within = at - first[g.clamp(min=0)] * 128
            s["m_indices"] = torch.where((g >= 0) & (within < counts[g.clamp(min=0)]), g, -1).to(torch.int32)
            lead = (M,)
        s["A"], s["sa"] = int8_rows(gen, *lead, K)
        s["D"] = torch.zeros(lead + (N,), dtype=torch.bfloat16, device=DEVICE)
        return s
    T, N, dt = c["T"], c["N"], dtype_of(c)
    vector = lambda spread, at: torch.randn(N, device=DEVICE, generator=gen) * spread + at  # noqa: E731
    s["x"] = rows_like(gen, T, N, dtype=dt)                    # the stream (its new value in the gradient)
    s["y"] = rows_like(gen, T, N, dtype=dt) if c["y"] else None
    s["pre"] = vector(0.1, 1.0) if c["pre"] else None
    s["post"] = vector(0.1, 1.0) if c["post"] else None
    s["gate"] = {"none": None, "channel": vector(0.2, 0.5), "token": torch.rand(T, 1, device=DEVICE, generator=gen)}[c["gate"]]
    if c["op"] == "norm_grad":
        s["dh"] = torch.randn(T, N, device=DEVICE, generator=gen).to(dt) if c["pre"] else None
        s["dr"] = torch.randn(T, N, device=DEVICE, generator=gen).to(dt) if c["dr"] else None
    return s


ALPHA, BETA, EPS = 0.875, 0.22, 1e-6     # residual scale, block scale


# ------------------------------------------------------------------ plain forms
def plain_int8(v):
    """Codes and scales of fp32 rows."""
    amax = v.abs().amax(-1)
    s = torch.where(amax == 0, 1.0, (amax / torch.full_like(amax, 127.0)).clamp(min=TINY))
    return torch.round(v / s[..., None]), s


def plain_quant(s):
    c = s["case"]
    if c["mode"] == "rows":
        q, sc = plain_int8(s["x"].float())
        return dict(q=q.to(torch.int8), s=sc)
    if c["mode"] == "dispatch":
        rows = s["plan"]["rows"].long()
        v = s["x"].float()[:, None].expand(-1, rows.shape[1], -1)
        v = v if s["w"] is None else v * s["w"][:, :, None]
        q, sc = plain_int8(v)
        cap = capacity(c)
        at = torch.where(rows >= 0, rows, cap).reshape(-1)     # slots without a row go to one past the end
        Q = torch.zeros(cap + 1, c["H"], dtype=torch.int8, device=DEVICE)
        Q[at] = q.reshape(-1, c["H"]).to(torch.int8)
        S = torch.zeros(cap + 1, device=DEVICE)
        S[at] = sc.reshape(-1)
        return dict(q=Q[:cap].view(s["Q"].shape), s=S[:cap].view(s["s"].shape))
    h = s["h"].float().reshape(-1, c["H"] // 128, 2, 128)
    v = h[:, :, 0] / (1 + torch.exp(-h[:, :, 0])) * h[:, :, 1]
    q, sc = plain_int8(v.reshape(-1, c["H"]))
    there = s["plan"]["slots"] >= 0
    # near a border between two codes the side goes by the last bit of exp: the codes come as values
    return dict(q=torch.where(there[:, None], q, 0.0).to(torch.bfloat16).view(s["Q"].shape),
                s=torch.where(there, sc, 0.0).view(s["s"].shape))


def plain_gemm(s):
    c = s["case"]
    if c["layout"] == "dense":
        return (s["A"].float() @ s["B"].float().t() * s["sa"][:, None] * s["sb"]).bfloat16()
    if c["layout"] == "masked":
        D = torch.bmm(s["A"].float(), s["B"].float().transpose(1, 2)) * s["sa"][:, :, None] * s["sb"][:, None]
        there = torch.arange(c["M_max"], device=DEVICE) < s["masked_m"][:, None]
        return torch.where(there[:, :, None], D, 0.0).bfloat16()
    # every 128 rows are one expert's: a batched product over the blocks
    mi = s["m_indices"].view(-1, 128)
    g = mi.amax(1).clamp(min=0).long()
    D = torch.bmm(s["A"].float().view(-1, 128, c["K"]), s["B"].float()[g].transpose(1, 2))
    D = D * s["sa"].view(-1, 128, 1) * s["sb"][g][:, None]
    return torch.where((mi >= 0)[:, :, None], D, 0.0).bfloat16().view(-1, c["N"])


def plain_norm(s):
    c = s["case"]
    out, r = {}, s["x"].float()
    if c["y"]:
        u = s["y"].float()
        if c["post"]:
            u = u / torch.sqrt((u * u).mean(1, keepdim=True) + EPS) * s["post"]
        if s["gate"] is not None:
            u = u * s["gate"]
        r = ALPHA * r + BETA * u
        out["r"] = r.to(s["x"].dtype)
    if not c["pre"]:
        return out
    h = r / torch.sqrt((r * r).mean(1, keepdim=True) + EPS) * s["pre"]     # of the stream before its rounding
    if c["quant"] == "none":
        out["h"] = h.to(s["x"].dtype)
    elif c["quant"] == "int8":
        q, out["s"] = plain_int8(h)
        out["h"] = q.to(torch.bfloat16)     # the values of the codes
    else:
        h = h.view(c["T"], -1, 128)
        amax = h.abs().amax(2)
        sc = torch.where(amax == 0, 1.0, amax / torch.full_like(amax, 448.0))
        out["h"] = (h / sc[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(c["T"], c["N"])
        out["s"] = sc.t().contiguous()
    return out


def plain_grad(s):
    c = s["case"]
    out = {}
    dR = s["dr"].float() if c["dr"] else torch.zeros(c["T"], c["N"], device=DEVICE)
    if c["pre"]:
        r, dh = s["x"].float(), s["dh"].float()
        rstd = 1 / torch.sqrt((r * r).mean(1, keepdim=True) + EPS)
        rh = r * rstd
        out["dpre"] = (dh * rh).sum(0)
        z = dh * s["pre"]
        dR = dR + rstd * (z - rh * (z * rh).mean(1, keepdim=True))
    out["dx"] = (ALPHA * dR).to(s["x"].dtype)
    if not c["y"]:
        return out
    yh = s["y"].float()
    if c["post"]:
        ystd = 1 / torch.sqrt((yh * yh).mean(1, keepdim=True) + EPS)
        yh = yh * ystd
    u = yh * s["post"] if c["post"] else yh
    d = BETA * dR
    if c["gate"] == "channel":
        out["dgate"] = (d * u).sum(0)
    elif c["gate"] == "token":
        out["dgate"] = (d * u).sum(1, keepdim=True)
    if s["gate"] is not None:
        d = d * s["gate"]
    if c["post"]:
        out["dpost"] = (d * yh).sum(0)
        d = d * s["post"]
        d = ystd * (d - yh * (d * yh).mean(1, keepdim=True))
    out["dy"] = d.to(s["x"].dtype)
    return out


def run_plain(s):
    op = s["case"]["op"]
    if op == "quant":
        return plain_quant(s)
    if op == "gemm":
        return dict(D=plain_gemm(s))
    return plain_norm(s) if op == "norm" else plain_grad(s)


# ------------------------------------------------------------------ the library's calls
def the_plan(fg, s):
    c, p = s["case"], s["plan"]
    if c["layout"] == "masked":
        return fg.Plan.masked(p["rows"], p["slots"], p["masked_m"], c["M_max"])
    return fg.Plan.contiguous(p["rows"], p["slots"], p["m_indices"], p["offsets"], c["align"])


def run_own(s):
    import moe_grouped_gemm_02_amd as fg
    c = s["case"]
    if c["op"] == "quant":
        if c["mode"] == "rows":
            q, sc = fg.quant_int8(s["x"])
        elif c["mode"] == "dispatch":
            q, sc = fg.dispatch_quant_int8(s["x"], the_plan(fg, s), w=s["w"], Q=s["Q"], s=s["s"])
        else:
            q, sc = fg.swiglu_quant_int8(s["h"], the_plan(fg, s), Q=s["Q"], s=s["s"])
            q = q.to(torch.bfloat16)        # the values of the codes
        return dict(q=q, s=sc)
    if c["op"] == "gemm":
        a = s["A"], s["sa"], s["B"], s["sb"], s["D"]
        if c["layout"] == "dense":
            return dict(D=fg.gemm_int8_nt(*a))
        if c["layout"] == "masked":
            return dict(D=fg.grouped_masked_int8(*a, s["masked_m"]))
        return dict(D=fg.grouped_contiguous_int8(*a, s["m_indices"]))
    how = dict(pre=s["pre"], post=s["post"], gate=s["gate"], alpha=ALPHA, beta=BETA, eps=EPS)
    if c["op"] == "norm":
        quant = None if c["quant"] == "none" else c["quant"]
        r, h, sc = fg.block_norm(s["x"], s["y"], quant=quant, **how)
        out = dict(r=r) if c["y"] else {}
        if c["pre"]:
            out["h"] = h
        if quant:
            out["s"] = sc
            out["h"] = h.view(torch.float8_e4m3fn) if quant == "e4m3" else h.to(torch.bfloat16)
        return out
    # alpha is the factor of a stream that a block's output is added to (alpha x + beta y): where the case has no such
    # output the call gets the stream in its place, whose gradient dy is not asked for
    y = s["y"] if c["y"] else s["x"]
    dx, dy, dgate, dpre, dpost = fg.block_norm_grad(s["x"], dh=s["dh"], dr=s["dr"], y=y, **how)
    out = dict(dx=dx, dy=dy if c["y"] else None, dgate=dgate, dpre=dpre, dpost=dpost)
    return {name: v for name, v in out.items() if v is not None}


def run(state):
    return run_own(state) if own else run_plain(state)


# ------------------------------------------------------------------ costs
def work(case):
    """Each input read once, each output written once; masked and contiguous rows taken as in the mean, experts as all in use."""
    c = case
    b = 2 if c.get("dtype", "bf16") == "bf16" else 4
    if c["op"] == "quant":
        if c["mode"] == "rows":
            return dict(bytes=c["T"] * (c["H"] * (b + 1) + 4), flops=3 * c["T"] * c["H"])
        here = c["T"] * min(c["k"], c["E"]) * c["G"] // c["E"]
        here = min(here, capacity(c)) if c["layout"] == "masked" else here
        rows_in = c["T"] * c["H"] if c["mode"] == "dispatch" else 2 * here * c["H"]
        return dict(bytes=rows_in * b + here * (c["H"] + 4) + 4 * c["T"] * c["k"], flops=(3 if c["mode"] == "dispatch" else 7) * here * c["H"])
    if c["op"] == "gemm":
        N, K, G = c["N"], c["K"], c.get("G", 1)
        rows = c["M"] if c["layout"] == "dense" else c["T"] if c["layout"] == "contiguous" else max(1, G * c["M_max"] // 2)
        return dict(bytes=rows * (K + 4) + G * N * (K + 4) + 2 * rows * N, flops=2 * rows * N * K)
    n = c["T"] * c["N"]
    if c["op"] == "norm":
        wide = 0 if not c["pre"] else b if c["quant"] == "none" else 1
        return dict(bytes=n * (b * (3 if c["y"] else 1) + wide) + 4 * c["N"] * (c["pre"] + c["post"]), flops=n * (5 * c["pre"] + 7 * c["y"]))
    return dict(bytes=n * b * (1 + 2 * c["y"] + 2 * c["pre"] + c["dr"]) + 8 * c["N"] * (c["pre"] + c["post"]), flops=n * (9 * c["pre"] + 9 * c["y"]))


# ------------------------------------------------------------------ 64 bits
def exact_scale(v):
    top = v.abs().amax(-1)
    return torch.where(top > 0, (top / 127).clamp(min=TINY), torch.ones_like(top))


def exact_norm(v, w):
    n = v * torch.rsqrt(v.pow(2).mean(-1, keepdim=True) + EPS)
    return n if w is None else n * w.double()


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "quant":
        if c["mode"] == "rows":
            return dict(q=None, s=exact_scale(s["x"].double()))
        slots = s["plan"]["slots"].long()
        real = slots >= 0
        slot = slots.clamp(min=0)
        if c["mode"] == "dispatch":
            v = s["x"].double()[slot // c["k"]]
            if s["w"] is not None:
                v = v * s["w"].double().view(-1)[slot][:, None]
            return dict(q=None, s=torch.where(real, exact_scale(v), 0.0).view(s["s"].shape))
        h = s["h"].double().view(-1, c["H"] // 128, 256)
        v = (torch.sigmoid(h[..., :128]) * h[..., :128] * h[..., 128:]).flatten(1)
        sc = exact_scale(v)
        q = torch.round(v / sc[:, None])
        return dict(q=torch.where(real[:, None], q, 0.0).view(s["Q"].shape), s=torch.where(real, sc, 0.0).view(s["s"].shape))
    if c["op"] == "gemm":
        if c["layout"] == "dense":
            A, B = s["A"].double() * s["sa"].double()[:, None], s["B"].double() * s["sb"].double()[:, None]
            return dict(D=A @ B.t())
        D = torch.zeros(s["D"].shape, dtype=torch.float64, device=DEVICE)
        for g in range(c["G"]):
            B = s["B"][g].double() * s["sb"][g].double()[:, None]
            if c["layout"] == "masked":
                m = int(s["masked_m"][g])
                D[g, :m] = (s["A"][g, :m].double() * s["sa"][g, :m].double()[:, None]) @ B.t()
            else:
                at = (s["m_indices"] == g).nonzero().view(-1)
                D[at] = (s["A"][at].double() * s["sa"][at].double()[:, None]) @ B.t()
        return dict(D=D)
    d = lambda t: None if t is None else t.double()  # noqa: E731
    x, y, gate = d(s["x"]), d(s["y"]), d(s["gate"])
    if c["op"] == "norm":
        out, r = {}, x
        if c["y"]:
            u = exact_norm(y, s["post"]) if c["post"] else y
            r = ALPHA * x + BETA * (u if gate is None else gate * u)
            out["r"] = r
        if c["pre"]:
            h = exact_norm(r, s["pre"])
            out["h"] = h
            if c["quant"] == "int8":
                out["s"] = exact_scale(h)
                out["h"] = torch.round(h / out["s"][:, None])
            elif c["quant"] == "e4m3":
                h = h.view(c["T"], -1, 128)
                top = h.abs().amax(2)
                sc = torch.where(top > 0, top / 448, torch.ones_like(top))
                out["h"], out["s"] = (h / sc[:, :, None]).view(c["T"], c["N"]), sc.t().contiguous()
        return out
    # the derivative by automatic differentiation of the definition
    with torch.enable_grad():
        leaf = lambda t: None if t is None else t.detach().double().requires_grad_()  # noqa: E731
        pre, post, gate, y, r = (leaf(s[n]) for n in ("pre", "post", "gate", "y", "x"))
        total = r * 0
        if c["y"]:
            u = y if post is None else y / (y.square().mean(1, keepdim=True) + EPS).sqrt() * post
            total = total + BETA * (u if gate is None else u * gate)
        stream = r.detach() + (total - total.detach()) + (r - r.detach())    # its value is r, its slope in y is total's
        loss = torch.zeros((), dtype=torch.float64, device=DEVICE)
        if c["pre"]:
            loss = loss + (stream / (stream.square().mean(1, keepdim=True) + EPS).sqrt() * pre * d(s["dh"])).sum()
        if c["dr"]:
            loss = loss + (stream * d(s["dr"])).sum()
        names = [n for n, v in (("dx", r), ("dy", y), ("dgate", gate), ("dpre", pre), ("dpost", post)) if v is not None]
        got = torch.autograd.grad(loss, [v for v in (r, y, gate, pre, post) if v is not None])
    out = dict(zip(names, got))
    out["dx"] = ALPHA * out["dx"]
    return out

"""The operators around the grouped GEMMs of a mixture-of-experts layer, as cases that can be timed and compared.

Six operators, each with its plain form in elementary torch operations (32-bit arithmetic, one rounding at the end) and
its call of the library:

    route      top-k expert choice from router logits (softmax or sigmoid scores), its weights, and their gradient
    plan       stable sort of the (token, slot) pairs by expert into the GEMM's contiguous or masked layout
    dispatch   token rows copied into the sorted layout as E4M3 codes with 1x128 scales
    combine    weighted sum of the experts' output rows back into token order
    grad       gradient of combine: the sorted rows' gradient (bf16 or E4M3 with scales) and the weights' gradient
    adapters   low-rank adapters of many requests added to a shared projection

`own` chooses the side: False computes the plain form, True calls the library.
"""
import torch

own = False

DEVICE = "cuda"
INF = float("inf")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a small batch through a sigmoid router with a balancing bias: latency
        dict(name="route_decode", op="route", T=32, E=256, k=8, dtype="bf16", score="sigmoid", bias=True, renorm=True,
             masked=False, grad=False),
        # a training batch through a softmax router, forward and gradient, with experts masked out for some tokens
        dict(name="route_train", op="route", T=16384, E=64, k=8, dtype="fp32", score="softmax", bias=False, renorm=False,
             masked=True, grad=True),
        # a decode batch sorted for one device's 16 of 256 experts, fixed buffers of 256 rows: most slots are elsewhere
        dict(name="plan_decode", op="plan", layout="masked", T=256, k=8, E=256, G=16, M_max=256),
        # a prefill batch sorted for all of its experts, segments padded to the GEMM's 128-row blocks
        dict(name="plan_prefill", op="plan", layout="contiguous", T=16384, k=8, E=64, G=64, align=128),
        # decode rows into the masked layout, power-of-two scales
        dict(name="dispatch_decode", op="dispatch", layout="masked", T=128, k=8, E=16, G=16, M_max=256, H=7168,
             dtype="bf16", pow2=True, weighted=False),
        # prefill rows into the contiguous layout, 8 experts, fp32 scales
        dict(name="dispatch_prefill", op="dispatch", layout="contiguous", T=8192, k=4, E=8, G=8, align=128, H=7168,
             dtype="bf16", pow2=False, weighted=False),
        # decode rows back from the masked layout
        dict(name="combine_decode", op="combine", layout="masked", T=64, k=8, E=16, G=16, M_max=256, N=7168, weighted=True,
             base=False),
        # prefill rows back, added to a shared expert's output
        dict(name="combine_prefill", op="combine", layout="contiguous", T=8192, k=4, E=8, G=8, align=128, N=7168,
             weighted=True, base=True),
        # a ragged batch's gradient, some slots on other devices, kept in bf16
        dict(name="grad_ragged", op="grad", layout="contiguous", T=1001, k=3, E=24, G=16, align=128, N=2048, quant=False,
             pow2=False),
        # a training batch's gradient as the backward GEMM's E4M3 operand
        dict(name="grad_train", op="grad", layout="contiguous", T=8192, k=4, E=8, G=8, align=128, N=4096, quant=True,
             pow2=False),
        # one token each of 64 requests over 64 adapters
        dict(name="adapters_decode", op="adapters", T=64, L=64, R=16, K=7168, N=4096, align=16),
        # whole prompts of a few requests over 8 adapters
        dict(name="adapters_prefill", op="adapters", T=8192, L=8, R=64, K=7168, N=4096, align=64),
    ]


def log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["route", "plan", "dispatch", "combine", "grad", "adapters"])
    if op == "route":
        E = log_int(rng, 8, 256)
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, T=log_int(rng, 1, 16384), E=E, k=rng.randint(1, 8), dtype=rng.choice(["bf16", "fp32"]),
                    score=score, bias=score == "sigmoid" and rng.random() < 0.5, renorm=rng.random() < 0.5,
                    masked=rng.random() < 0.5, grad=rng.random() < 0.5)
    if op == "adapters":
        T = log_int(rng, 1, 8192)
        L = log_int(rng, 1, 64 if T <= 512 else 8)
        K, N = 128 * log_int(rng, 4, 56), 8 * log_int(rng, 64, 512)
        return dict(op=op, T=T, L=L, R=rng.choice([8, 16, 32, 64]), K=K, N=N, align=64 if T >= 32 * L else 16)
    layout = rng.choice(["contiguous", "masked"])
    E = log_int(rng, 8, 128)
    G = E if rng.random() < 0.5 else max(1, E // 4)
    c = dict(op=op, layout=layout, T=log_int(rng, 1, 4096 if layout == "contiguous" else 512), k=rng.randint(1, 8), E=E, G=G)
    c.update(dict(align=128) if layout == "contiguous" else dict(M_max=rng.choice([64, 128, 256])))
    if op == "dispatch":
        c.update(H=128 * log_int(rng, 1, 56), dtype=rng.choice(["bf16", "fp32"]), pow2=rng.random() < 0.5,
                 weighted=rng.random() < 0.3)
    elif op == "combine":
        c.update(N=8 * log_int(rng, 16, 896), weighted=rng.random() < 0.7, base=rng.random() < 0.5)
    elif op == "grad":
        quant = rng.random() < 0.5
        c.update(N=128 * log_int(rng, 1, 32) if quant else 8 * log_int(rng, 16, 512), quant=quant,
                 pow2=quant and rng.random() < 0.5)
    return c


# ------------------------------------------------------------------ inputs
def dtype_of(c):
    return torch.bfloat16 if c.get("dtype", "bf16") == "bf16" else torch.float32


def capacity(c):
    """Rows of the sorted layout, from sizes alone: every expert's segment may need align - 1 rows of padding."""
    if c.get("layout") == "masked":
        return c["G"] * c["M_max"]
    slots, G, align = c["T"] * c.get("k", 1), c.get("G", c.get("L")), c["align"]
    return -(-(slots + min(slots, G) * (align - 1)) // align) * align


def expert_choice(c, gen):
    """Distinct experts per token, popular ones more often; experts of other devices come out of range (>= G)."""
    pull = torch.randn(c["E"], device=DEVICE, generator=gen)
    gumbel = -torch.log(-torch.log(torch.rand(c["T"], c["E"], device=DEVICE, generator=gen).clamp(1e-9, 1 - 1e-7)))
    return (0.5 * pull + gumbel).argsort(dim=1, descending=True)[:, :c["k"]].to(torch.int32).contiguous()


def rows_like(gen, *shape, dtype=torch.bfloat16):
    """Activations: N(0, 1), one row in a hundred scaled by 50."""
    x = torch.randn(*shape, device=DEVICE, generator=gen)
    x *= torch.where(torch.rand(*shape[:-1], 1, device=DEVICE, generator=gen) < 0.01, 50.0, 1.0)
    return x.to(dtype)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "route":
        logits = torch.randn(c["T"], c["E"], device=DEVICE, generator=gen) * 2
        if c["masked"]:
            some = torch.rand(c["T"], 1, device=DEVICE, generator=gen)
            first = torch.arange(c["E"], device=DEVICE)
            logits.masked_fill_((some < 0.5) & (first < c["E"] // 4), -INF)   # a quarter masked for half of the tokens
            logits.masked_fill_((some > 0.99) & (first > 2), -INF)            # few experts left for some
        s["logits"] = logits.to(dtype_of(c))
        s["bias"] = torch.randn(c["E"], device=DEVICE, generator=gen) * 0.1 if c["bias"] else None
        s["dw"] = torch.randn(c["T"], c["k"], device=DEVICE, generator=gen)
        return s
    if c["op"] == "adapters":
        T, L, R, K, N = c["T"], c["L"], c["R"], c["K"], c["N"]
        # requests in the batch one after another; about one in sixteen uses no adapter
        request = torch.randint(0, max(1, min(T, 2 * L)), (T,), device=DEVICE, generator=gen).sort().values
        adapter = torch.randint(0, L, (max(1, min(T, 2 * L)),), device=DEVICE, generator=gen)
        plain = torch.rand(adapter.shape, device=DEVICE, generator=gen) < 1 / 16
        ids = torch.where(plain, -1, adapter)[request].to(torch.int32)
        s.update(ids=ids.view(T, 1), x=rows_like(gen, T, K), D=torch.randn(T, N, device=DEVICE, generator=gen).bfloat16(),
                 A=(torch.randn(L, R, K, device=DEVICE, generator=gen) * K ** -0.5).bfloat16(),
                 B=(torch.randn(L, N, R, device=DEVICE, generator=gen) * R ** -0.5).bfloat16(),
                 scales=torch.rand(L, device=DEVICE, generator=gen) + 0.5)
        s["plan"] = plain_plan(c, s["ids"])
        return s
    s["ids"] = expert_choice(c, gen)
    if c["op"] == "plan":
        return s
    s["plan"] = plain_plan(c, s["ids"])
    w = torch.rand(s["ids"].shape, device=DEVICE, generator=gen)
    s["w"] = w / w.sum(1, keepdim=True)
    lead = (c["G"], c["M_max"]) if c["layout"] == "masked" else (capacity(c),)
    if c["op"] == "dispatch":
        s["x"] = rows_like(gen, c["T"], c["H"], dtype=dtype_of(c))
        s["Q"], s["sa"] = sorted_buffers(c, c["H"])
        s["w"] = s["w"] if c["weighted"] else None
    elif c["op"] == "combine":
        s["y"] = rows_like(gen, *lead, c["N"])
        s["w"] = s["w"] if c["weighted"] else None
        s["base"] = rows_like(gen, c["T"], c["N"]) if c["base"] else None
    else:
        s["y"] = rows_like(gen, *lead, c["N"])
        s["dout"] = rows_like(gen, c["T"], c["N"])
        if c["quant"]:
            s["Q"], s["sa"] = sorted_buffers(c, c["N"])
        else:
            s["dy"] = torch.zeros(*lead, c["N"], dtype=torch.bfloat16, device=DEVICE)
    return s


def sorted_buffers(c, H):
    """The GEMM's operand buffers, kept by the program; rows that hold no token stay as they are."""
    if c["layout"] == "masked":
        q, sa = (c["G"], c["M_max"], H), (c["G"], H // 128, c["M_max"])
    else:
        q, sa = (capacity(c), H), (H // 128, capacity(c))
    return torch.zeros(q, dtype=torch.uint8, device=DEVICE), torch.zeros(sa, device=DEVICE)


# ------------------------------------------------------------------ plain forms
def plain_route(s):
    c = s["case"]
    l = s["logits"].float()
    ok = l > -INF
    if c["score"] == "softmax":
        e = torch.where(ok, torch.exp(l - torch.where(ok, l, -INF).amax(1, keepdim=True)), 0.0)
        total = e.sum(1, keepdim=True)
        p = torch.where(total > 0, e / total, 0.0)
    else:
        p = torch.where(ok, 1 / (1 + torch.exp(-l)), 0.0)
    key = l if s["bias"] is None else p + s["bias"]
    key = torch.where(ok, key, -INF)
    key, order = torch.sort(key, dim=1, descending=True, stable=True)
    key, order = key[:, :c["k"]], order[:, :c["k"]]
    there = key > -INF
    ids = torch.where(there, order, -1).to(torch.int32)
    chosen = torch.where(there, p.gather(1, order), 0.0)
    total = chosen.sum(1, keepdim=True)
    share = torch.where(total > 0, chosen / total, 0.0)
    w = (share if c["renorm"] else chosen) * 2.5
    out = dict(ids=ids, w=w)
    if c["grad"]:
        g = torch.where(there, s["dw"] * 2.5, 0.0)
        if c["score"] == "softmax" and not c["renorm"]:
            full = torch.zeros_like(l).scatter_add_(1, order, g)
            out["dlogits"] = p * (full - (full * p).sum(1, keepdim=True))
        else:
            if c["renorm"]:
                g = g - (g * share).sum(1, keepdim=True)
            if c["score"] == "softmax":
                g = share * g
            else:
                g = g * chosen * (1 - chosen)
                g = torch.where(total > 0, g / total, 0.0) if c["renorm"] else g
            out["dlogits"] = torch.zeros_like(l).scatter_add_(1, order, torch.where(there, g, 0.0))
        out["dlogits"] = out["dlogits"].to(dtype_of(c))
    return out


def plain_plan(c, ids):
    """Sorted layout of the slots: rows [T, k] (-1: no row), slots [rows] (-1: padding), and the layout's own index."""
    flat = ids.reshape(-1).long()
    G, cap, S = c.get("G", c.get("L")), capacity(c), flat.numel()
    key = torch.where((flat >= 0) & (flat < G), flat, G)
    key, order = torch.sort(key, stable=True)
    counts = torch.zeros(G + 1, dtype=torch.long, device=DEVICE).scatter_add_(0, key, torch.ones_like(key))
    rank = torch.arange(S, device=DEVICE) - (torch.cumsum(counts, 0) - counts)[key]
    if c.get("layout") == "masked":
        start = torch.arange(G + 1, device=DEVICE) * c["M_max"]
        there = (key < G) & (rank < c["M_max"])
    else:
        padded = -(-counts // c["align"]) * c["align"]
        start = torch.cumsum(padded, 0) - padded
        there = key < G
    row = torch.where(there, start[key] + rank, cap)      # slots without a row go to one past the end
    new = lambda n: torch.full((n,), -1, dtype=torch.int32, device=DEVICE)  # noqa: E731
    rows = new(S).scatter_(0, order, torch.where(there, row, -1).to(torch.int32)).view(ids.shape)
    slots = new(cap + 1).scatter_(0, row, order.to(torch.int32))[:cap].contiguous()
    if c.get("layout") == "masked":
        return dict(rows=rows, slots=slots, masked_m=counts[:G].clamp(max=c["M_max"]).to(torch.int32))
    m_indices = new(cap + 1).scatter_(0, row, key.to(torch.int32))[:cap].contiguous()
    return dict(rows=rows, slots=slots, m_indices=m_indices, offsets=start.to(torch.int32))


def slot_rows(s):
    """Each slot's row of the sorted layout as an index, one past the end where it has none."""
    rows = s["plan"]["rows"].long()
    return torch.where(rows >= 0, rows, capacity(s["case"])), rows >= 0


def plain_sort_quant(s, x, w, H):
    """Rows of w * x (w: none or [T, k]) in the sorted layout as E4M3 values with a scale for each 128 of a row."""
    c = s["case"]
    at, _ = slot_rows(s)
    v = x.float()[:, None].expand(-1, at.shape[1], -1)
    v = v if w is None else v * w[:, :, None]
    v = v.reshape(-1, H // 128, 128)
    amax = v.abs().amax(2)
    scale = torch.where(amax == 0, 1.0, amax / torch.full_like(amax, 448.0))
    if c["pow2"]:
        m, e = torch.frexp(scale)
        scale = torch.ldexp(torch.ones_like(scale), torch.where(m == 0.5, e - 1, e)).clamp(min=2.0 ** -126)
    code = (v / scale[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1, H)
    cap = capacity(c)
    Q = torch.zeros(cap + 1, H, dtype=torch.uint8, device=DEVICE)
    Q[at.reshape(-1)] = code
    sa = torch.zeros(cap + 1, H // 128, device=DEVICE)
    sa[at.reshape(-1)] = scale
    Q, sa = Q[:cap], sa[:cap]
    if c["layout"] == "masked":
        Q = Q.view(c["G"], c["M_max"], H)
        sa = sa.view(c["G"], c["M_max"], H // 128).transpose(1, 2).contiguous()
    else:
        sa = sa.t().contiguous()
    return Q.view(torch.float8_e4m3fn), sa


def plain_combine(s):
    c = s["case"]
    at, there = slot_rows(s)
    y = s["y"].reshape(-1, c["N"])
    v = y[at.clamp(max=y.shape[0] - 1)].float()
    weight = there.float() if s["w"] is None else torch.where(there, s["w"], 0.0)
    out = (torch.where(there[:, :, None], v, 0.0) * weight[:, :, None]).sum(1)
    return (out if s["base"] is None else out + s["base"].float()).bfloat16()


def plain_grad(s):
    c = s["case"]
    at, there = slot_rows(s)
    y = s["y"].reshape(-1, c["N"])
    dout = s["dout"].float()
    dw = (y[at.clamp(max=y.shape[0] - 1)].float() * dout[:, None]).sum(2)
    out = dict(dw=torch.where(there, dw, 0.0))
    if c["quant"]:
        out["Q"], out["sa"] = plain_sort_quant(s, s["dout"], s["w"], c["N"])
        return out
    dy = torch.zeros(capacity(c) + 1, c["N"], dtype=torch.bfloat16, device=DEVICE)
    dy[at.reshape(-1)] = (dout[:, None] * s["w"][:, :, None]).reshape(-1, c["N"]).bfloat16()
    out["dy"] = dy[:capacity(c)].view(s["y"].shape)
    return out


def plain_adapters(s):
    """All adapters at once: a token's products with the others are left out by a mask between the two products."""
    c = s["case"]
    ids = s["ids"].long()
    h = (s["x"].float() @ s["A"].float().view(-1, c["K"]).t()).view(c["T"], c["L"], c["R"])
    mine = (ids == torch.arange(c["L"], device=DEVICE)).float() * s["scales"]
    h = (h * mine[:, :, None]).view(c["T"], -1)
    return (s["D"].float() + h @ s["B"].float().transpose(1, 2).reshape(-1, c["N"])).bfloat16()


def run_plain(s):
    c = s["case"]
    if c["op"] == "route":
        return plain_route(s)
    if c["op"] == "plan":
        return plain_plan(c, s["ids"])
    if c["op"] == "dispatch":
        Q, sa = plain_sort_quant(s, s["x"], s["w"], c["H"])
        return dict(Q=Q, sa=sa)
    if c["op"] == "combine":
        return dict(out=plain_combine(s))
    if c["op"] == "grad":
        return plain_grad(s)
    return dict(D=plain_adapters(s))


# ------------------------------------------------------------------ the library's calls
def the_plan(fg, s):
    c, p = s["case"], s["plan"]
    if c.get("layout") == "masked":
        return fg.Plan.masked(p["rows"], p["slots"], p["masked_m"], c["M_max"])
    return fg.Plan.contiguous(p["rows"], p["slots"], p["m_indices"], p["offsets"], c["align"])


def run_own(s):
    import moe_grouped_gemm_02_amd as fg
    c = s["case"]
    if c["op"] == "route":
        how = dict(score=c["score"], renorm=c["renorm"], scale=2.5)
        ids, w = fg.route_topk(s["logits"], c["k"], bias=s["bias"], **how)
        out = dict(ids=ids, w=w)
        if c["grad"]:
            out["dlogits"] = fg.route_topk_grad(s["logits"], ids, s["dw"], **how)
        return out
    if c["op"] == "plan":
        if c["layout"] == "masked":
            p = fg.plan_masked(s["ids"], c["G"], c["M_max"])
            return dict(rows=p.rows, slots=p.slots, masked_m=p.masked_m)
        p = fg.plan_contiguous(s["ids"], c["G"], align=c["align"])
        return dict(rows=p.rows, slots=p.slots, m_indices=p.m_indices, offsets=p.offsets)
    plan = the_plan(fg, s)
    if c["op"] == "dispatch":
        Q, sa = fg.dispatch_quant(s["x"], plan, w=s["w"], pow2=c["pow2"], Q=s["Q"], sa=s["sa"])
        return dict(Q=Q.view(torch.float8_e4m3fn), sa=sa)
    if c["op"] == "combine":
        return dict(out=fg.combine(s["y"], plan, w=s["w"], base=s["base"]))
    if c["op"] == "grad":
        if c["quant"]:
            Q, sa, dw = fg.combine_grad_quant(s["dout"], s["y"], plan, s["w"], pow2=c["pow2"], Q=s["Q"], sa=s["sa"])
            return dict(dw=dw, Q=Q.view(torch.float8_e4m3fn), sa=sa)
        dy, dw = fg.combine_grad(s["dout"], s["y"], plan, s["w"], dy=s["dy"])
        return dict(dw=dw, dy=dy)
    return dict(D=fg.adapters(s["D"], s["x"], s["A"], s["B"], s["scales"], plan))


def run(state):
    return run_own(state) if own else run_plain(state)


# ------------------------------------------------------------------ costs
def work(case):
    """Each input read once, each output written once; slots taken as all having a row, adapters as all in use."""
    c = case
    T = c["T"]
    if c["op"] == "route":
        b = 2 if c["dtype"] == "bf16" else 4
        n = T * c["E"] * b + T * c["k"] * 8
        return dict(bytes=n + (T * c["E"] * b + T * c["k"] * 4 if c["grad"] else 0), flops=T * c["E"] * (5 if c["grad"] else 3))
    if c["op"] == "adapters":
        used = min(T, c["L"])
        return dict(bytes=2 * (T * c["K"] + 2 * T * c["N"] + used * c["R"] * (c["K"] + c["N"])),
                    flops=2 * T * c["R"] * (c["K"] + c["N"]))
    S = T * min(c["k"], c["E"])
    here = S * c["G"] // c["E"]            # slots of this device's experts
    if c["layout"] == "masked":
        here = min(here, capacity(c))
    if c["op"] == "plan":
        return dict(bytes=8 * S + (4 if c["layout"] == "masked" else 8) * capacity(c) + 4 * c["G"], flops=0)
    if c["op"] == "dispatch":
        b = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=T * c["H"] * b + here * (c["H"] + c["H"] // 32 + 4), flops=3 * here * c["H"])
    if c["op"] == "combine":
        return dict(bytes=2 * c["N"] * (here + T * (2 if c["base"] else 1)) + here * 8, flops=2 * here * c["N"])
    wide = c["N"] + c["N"] // 32 if c["quant"] else 2 * c["N"]
    return dict(bytes=2 * c["N"] * (T + here) + here * wide + here * 12, flops=(5 if c["quant"] else 3) * here * c["N"])


# ------------------------------------------------------------------ 64 bits
def exact_route(s):
    c = s["case"]
    l = s["logits"].double()
    l = torch.where(l > -INF, l, torch.full_like(l, -INF))
    if c["score"] == "softmax":
        p = torch.nan_to_num(torch.softmax(l, dim=1), nan=0.0)
    else:
        p = torch.sigmoid(l)
    rank_by = l if s["bias"] is None else torch.where(l > -INF, p + s["bias"].double(), l)
    best = rank_by.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    picked = torch.zeros_like(l).scatter_(1, best, 1.0) * (rank_by > -INF)
    q = p * picked
    if c["renorm"]:
        norm = q.sum(1, keepdim=True)
        q = q / torch.where(norm > 0, norm, torch.ones_like(norm))
    w = 2.5 * q
    out = dict(ids=None, w=w.gather(1, best))
    if c["grad"]:
        # derivative of sum(dw * w) by the chain rule over the full rows
        g = torch.zeros_like(l).scatter_(1, best, 2.5 * s["dw"].double()) * picked
        if c["renorm"]:
            g = picked * (g - (g * q).sum(1, keepdim=True)) / torch.where(norm > 0, norm, torch.full_like(norm, INF))
        slope = p * (g - (g * p).sum(1, keepdim=True)) if c["score"] == "softmax" else g * p * (1 - p)
        out["dlogits"] = slope
    return out


def exact_quant(s, x, H):
    """The values before their rounding to E4M3, and the scales."""
    c = s["case"]
    slots = s["plan"]["slots"].long()
    real = (slots >= 0)[:, None]
    slot = slots.clamp(min=0)
    v = x.double()[slot // s["ids"].shape[1]]
    if s["w"] is not None:
        v = v * s["w"].double().reshape(-1)[slot][:, None]
    v = torch.where(real, v, 0.0).view(slots.numel(), H // 128, 128)
    top = v.abs().amax(2)
    sa = torch.where(top > 0, top / 448, torch.ones_like(top))
    if c["pow2"]:
        # the smallest power of two that is not below the scale as 32 bits hold it
        sa = torch.exp2(torch.ceil(torch.log2(sa.float().double()) - 1e-12))
    Q = (v / sa[:, :, None]).view(slots.numel(), H)
    sa = torch.where(real, sa, 0.0)
    if c["layout"] == "masked":
        return Q.view(c["G"], c["M_max"], H), sa.view(c["G"], c["M_max"], -1).transpose(1, 2).contiguous()
    return Q, sa.t().contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "plan":
        return None                       # whole numbers only
    if c["op"] == "route":
        return exact_route(s)
    if c["op"] == "dispatch":
        Q, sa = exact_quant(s, s["x"], c["H"])
        return dict(Q=Q, sa=sa)
    if c["op"] == "adapters":
        D = s["D"].double()
        for a in range(c["L"]):
            t = (s["ids"].view(-1) == a).nonzero().view(-1)
            h = s["x"][t].double() @ s["A"][a].double().t()
            D[t] += s["scales"][a].double() * (h @ s["B"][a].double().t())
        return dict(D=D)
    slots = s["plan"]["slots"].long()
    mine = (slots >= 0).nonzero().view(-1)
    slot = slots[mine]
    token = slot // s["ids"].shape[1]
    y = s["y"].view(-1, c["N"])[mine].double()
    if c["op"] == "combine":
        out = torch.zeros(c["T"], c["N"], dtype=torch.float64, device=DEVICE)
        if s["base"] is not None:
            out += s["base"].double()
        if s["w"] is not None:
            y = y * s["w"].double().view(-1)[slot][:, None]
        return dict(out=out.index_add_(0, token, y))
    d = s["dout"].double()[token]
    dw = torch.zeros(s["w"].numel(), dtype=torch.float64, device=DEVICE)
    dw[slot] = (d * y).sum(1)
    out = dict(dw=dw.view(s["w"].shape))
    if c["quant"]:
        out["Q"], out["sa"] = exact_quant(s, s["dout"], c["N"])
        return out
    dy = torch.zeros(slots.numel(), c["N"], dtype=torch.float64, device=DEVICE)
    dy[mine] = d * s["w"].double().view(-1)[slot][:, None]
    out["dy"] = dy.view(s["y"].shape)
    return out

"""One mixture-of-experts layer on the library's calls: forward in the contiguous layout
(training, prefill) with the backward of its routing, forward in the masked layout (decode),
and a shared projection with the low-rank adapters of many requests beside it.

    python examples/moe_layer.py [--tokens 512] [--experts 8] [--hidden 1024] [--inner 512]

needs an MI355X. Weights are random; every step prints what it made.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_grouped_gemm_02_amd as fg  # noqa: E402

ROUTER = dict(score="sigmoid", renorm=True, scale=2.5)


class Layer:
    """Weights of one layer: a router, E experts (gate and up rows interleaved every 128, then down), a shared
    projection and L adapters of rank R for it."""

    def __init__(self, hidden, inner, experts, adapters, rank, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        new = lambda *s, fan: torch.randn(*s, device="cuda", generator=gen) * fan ** -0.5  # noqa: E731
        self.experts = experts
        self.router = new(experts, hidden, fan=hidden)
        self.balance = torch.zeros(experts, device="cuda")
        self.up = fg.quant_weight_128x128(new(experts, 2 * inner, hidden, fan=hidden))
        self.down = fg.quant_weight_128x128(new(experts, hidden, inner, fan=inner))
        self.shared = fg.quant_weight_128x128(new(hidden, hidden, fan=hidden))
        self.A = new(adapters, rank, hidden, fan=hidden).bfloat16()
        self.B = new(adapters, hidden, rank, fan=rank).bfloat16()
        self.adapter_scales = torch.ones(adapters, device="cuda")


def shared_with_adapters(layer, x, adapter_ids):
    """The shared projection of x, each token's own adapter added: many tokens an adapter go in tiles of 64 rows."""
    A, sa = fg.quant_act_1x128(x.float())
    D = torch.empty(x.shape[0], layer.shared[0].shape[0], dtype=torch.bfloat16, device=x.device)
    fg.gemm_fp8_nt(A, sa, *layer.shared, D)
    n = layer.A.shape[0]
    plan = fg.plan_contiguous(adapter_ids.view(-1, 1), n, align=64 if x.shape[0] >= 32 * n else 16)
    return fg.adapters(D, x, layer.A, layer.B, layer.adapter_scales, plan, out=D)


def forward(layer, x, k, adapter_ids):
    """Contiguous layout. Returns the output and what the backward needs."""
    logits = (x.float() @ layer.router.t()).contiguous()
    ids, w = fg.route_topk(logits, k, bias=layer.balance, **ROUTER)
    plan = fg.plan_contiguous(ids, layer.experts)
    A, sa = fg.dispatch_quant(x, plan)
    Q, sq, _ = fg.grouped_contiguous_swiglu_quant(A, sa, *layer.up, plan.m_indices)
    y = torch.empty(plan.capacity, x.shape[1], dtype=torch.bfloat16, device=x.device)
    fg.grouped_contiguous(Q, sq, *layer.down, y, plan.m_indices)
    out = fg.combine(y, plan, w=w, base=shared_with_adapters(layer, x, adapter_ids))
    return out, (logits, ids, w, plan, y)


def backward(saved, dout):
    """Gradient of the layer's output into the experts' outputs (as the backward GEMM's E4M3 operand), the
    router's weights and its logits."""
    logits, ids, w, plan, y = saved
    dyq, dys, dw = fg.combine_grad_quant(dout, y, plan, w)
    return dyq, dys, dw, fg.route_topk_grad(logits, ids, dw, **ROUTER)


def decode(layer, x, k, adapter_ids, M_max):
    """Masked layout: fixed buffers of M_max rows per expert, nothing read back to the host."""
    logits = (x.float() @ layer.router.t()).contiguous()
    ids, w = fg.route_topk(logits, k, bias=layer.balance, **ROUTER)
    plan = fg.plan_masked(ids, layer.experts, M_max)
    A, sa = fg.dispatch_quant(x, plan)
    Q, sq, _ = fg.grouped_masked_swiglu_quant(A, sa, *layer.up, plan.masked_m)
    y = torch.empty(layer.experts, M_max, x.shape[1], dtype=torch.bfloat16, device=x.device)
    fg.grouped_masked(Q, sq, *layer.down, y, plan.masked_m)
    return fg.combine(y, plan, w=w, base=shared_with_adapters(layer, x, adapter_ids))


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=512)
    ap.add_argument("--choices", type=int, default=2)
    ap.add_argument("--adapters", type=int, default=4)
    a = ap.parse_args(argv)
    layer = Layer(a.hidden, a.inner, a.experts, a.adapters, rank=16)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn(a.tokens, a.hidden, device="cuda", generator=gen).bfloat16()
    adapter_ids = torch.randint(-1, a.adapters, (a.tokens,), device="cuda", generator=gen).to(torch.int32)
    out, saved = forward(layer, x, a.choices, adapter_ids)
    print(f"contiguous: {a.tokens} tokens, {int(saved[3].offsets[-1])} of {saved[3].capacity} rows in use, "
          f"output rms {float(out.float().square().mean().sqrt()):.3f}")
    dyq, _, dw, dlogits = backward(saved, torch.randn_like(out))
    print(f"backward: gradient operand {tuple(dyq.shape)}, weights' rms {float(dw.square().mean().sqrt()):.3f}, "
          f"logits' rms {float(dlogits.square().mean().sqrt()):.3f}")
    same = decode(layer, x, a.choices, adapter_ids, M_max=a.tokens)
    print(f"masked: largest difference from the contiguous layout {float((same.float() - out.float()).abs().max()):.1e}")
    return out, same, dw, dlogits


if __name__ == "__main__":
    main()

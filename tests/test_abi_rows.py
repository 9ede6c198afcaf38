"""The row operators' C entry points refuse bad arguments before touching the
device (no GPU needed), and the host-only sizes are what they should be."""
import ctypes

import pytest

import moe_grouped_gemm_02_amd as fg

EINVAL, OK = -1, 0
P = ctypes.c_void_p(0x100000)    # aligned, never dereferenced
ODD = ctypes.c_void_p(0x100001)


def call(name, good, **changes):
    args = dict(good)
    assert not set(changes) - set(args)
    args.update(changes)
    return getattr(fg.lib(), name)(*args.values())


ROUTE = dict(logits=P, dtype=0, bias=None, ids=P, w=P, T=4, E=16, k=2, score=0, renorm=0, scale=1.0, stream=None)
ROUTE_GRAD = dict(logits=P, dtype=0, ids=P, dw=P, dlogits=P, T=4, E=16, k=2, score=0, renorm=0, scale=1.0, stream=None)
PLAN_C = dict(ids=P, rows=P, slots=P, m_indices=P, offsets=P, ws=None, T=4, k=2, G=4, align=128, stream=None)
PLAN_M = dict(ids=P, rows=P, slots=P, masked_m=P, ws=None, T=4, k=2, G=4, M_max=8, stream=None)
DISPATCH = dict(x=P, dtype=0, rows=P, w=None, Q=P, sa=P, T=4, k=2, H=256, G=1, M=128, scales=0, stream=None)
COMBINE = dict(y=P, dtype=0, rows=P, w=None, base=None, out=P, T=4, k=2, N=64, n_rows=128, stream=None)
GRAD = dict(dout=P, y=P, dtype=0, rows=P, w=P, dy=None, dw=P, T=4, k=2, N=64, n_rows=128, stream=None)
GRAD_Q = dict(dout=P, y=P, dtype=0, rows=P, w=P, Q=P, sq=P, dw=P, T=4, k=2, N=128, G=2, M=64, scales=0, stream=None)
ADAPTERS = dict(D=P, x=P, A=P, B=P, scales=P, rows=P, slots=P, m_indices=P, offsets=P, out=P, ws=P, T=4, L=2, R=16, K=128, N=64,
                cap=32, align=16, stream=None)


@pytest.mark.parametrize("name,good,changes", [
    (n, g, c) for n, g, cs in [
        ("fg_route_topk", ROUTE, [dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=17), dict(k=65, E=100),
                                  dict(dtype=2), dict(score=2), dict(logits=None), dict(logits=ODD), dict(ids=None),
                                  dict(w=ODD), dict(bias=ODD)]),
        ("fg_route_topk_grad", ROUTE_GRAD, [dict(T=-1), dict(E=0), dict(k=17), dict(dw=None), dict(dlogits=None),
                                            dict(dlogits=ODD), dict(ids=ODD), dict(dtype=-1)]),
        ("fg_plan_contiguous", PLAN_C, [dict(T=-1), dict(k=0), dict(G=0), dict(G=1025), dict(align=0), dict(ids=None),
                                        dict(rows=ODD), dict(slots=None), dict(offsets=None), dict(m_indices=None),
                                        dict(T=1 << 30, k=2)]),
        ("fg_plan_masked", PLAN_M, [dict(T=-1), dict(k=0), dict(G=0), dict(M_max=0), dict(G=1024, M_max=1 << 22),
                                    dict(ids=None), dict(slots=None), dict(masked_m=None), dict(rows=ODD)]),
        ("fg_dispatch_quant", DISPATCH, [dict(T=-1), dict(k=0), dict(H=100), dict(H=0), dict(G=0), dict(M=0),
                                         dict(scales=2), dict(dtype=2), dict(x=None), dict(x=ODD), dict(Q=ODD),
                                         dict(sa=None), dict(rows=None), dict(w=ODD), dict(G=1 << 16, M=1 << 16)]),
        ("fg_combine", COMBINE, [dict(T=-1), dict(k=0), dict(N=60), dict(N=0), dict(n_rows=-1), dict(dtype=5),
                                 dict(y=None), dict(y=ODD), dict(out=None), dict(base=ODD), dict(w=ODD)]),
        ("fg_combine_grad", GRAD, [dict(T=-1), dict(N=4), dict(w=None), dict(dw=None), dict(dout=None), dict(dy=ODD),
                                   dict(y=ODD)]),
        ("fg_combine_grad_quant", GRAD_Q, [dict(N=64), dict(Q=None), dict(sq=ODD), dict(dw=None), dict(G=0),
                                           dict(scales=-1), dict(y=None)]),
        ("fg_adapters", ADAPTERS, [dict(T=-1), dict(L=0), dict(R=4), dict(R=12), dict(R=136), dict(K=64), dict(N=12),
                                   dict(align=8), dict(align=24), dict(cap=20), dict(cap=0), dict(ws=None), dict(D=None),
                                   dict(x=ODD), dict(out=ODD), dict(slots=None), dict(scales=ODD), dict(offsets=None)]),
    ] for c in cs], ids=lambda v: v if isinstance(v, str) else ",".join(v) if isinstance(v, dict) and len(v) < 4 else "")
def test_bad_arguments_are_refused(name, good, changes):
    assert call(name, good, **changes) == EINVAL


def test_no_tokens_is_a_no_op():
    assert call("fg_route_topk", ROUTE, T=0, logits=None, ids=None, w=None) == OK
    assert call("fg_dispatch_quant", DISPATCH, T=0, x=None) == OK
    assert call("fg_combine", COMBINE, T=0, y=None, out=None) == OK
    assert call("fg_combine_grad", GRAD, T=0, dout=None) == OK
    assert call("fg_combine_grad_quant", GRAD_Q, T=0, dout=None) == OK
    assert call("fg_adapters", ADAPTERS, T=0, cap=0, D=None) == OK


def test_plan_capacity():
    # every expert that can have a slot may waste align - 1 rows
    assert fg.plan_capacity(1, 1, 8) == 128
    assert fg.plan_capacity(1, 8, 8) == 8 * 128
    assert fg.plan_capacity(8192, 4, 8) == 32768 + 8 * 127 + 8   # rounded up to 128
    assert fg.plan_capacity(0, 4, 8) == 0
    assert fg.plan_capacity(100, 1, 3, align=16) == 160
    assert fg.plan_capacity(5, 2, 4, align=1) == 10
    with pytest.raises(fg.FGError):
        fg.plan_capacity(1 << 24, 127, 1024, align=65536)


@pytest.mark.parametrize("T,k,G,align", [(1, 1, 1, 16), (7, 3, 5, 16), (100, 8, 16, 128), (37, 2, 64, 64)])
def test_plan_capacity_is_reached_and_enough(T, k, G, align):
    S, cap = T * k, fg.plan_capacity(T, k, G, align)
    # worst split: one slot for all experts that get any, the rest on one of them
    most = 0
    for used in range(1, min(S, G) + 1):
        for extra in range(align):
            big = S - (used - 1) - extra
            if big >= 1:
                most = max(most, (used - 1) * align + -(-big // align) * align)
    assert most <= cap < most + 2 * align


def test_adapters_workspace():
    L, size = fg.lib(), ctypes.c_size_t()
    assert L.fg_adapters_workspace(16, 7168, 1024, 16, ctypes.byref(size)) == OK and size.value >= 1024 * 16 * 4
    assert L.fg_adapters_workspace(16, 7168, 1000, 16, ctypes.byref(size)) == EINVAL
    assert L.fg_adapters_workspace(16, 7168, 1024, 16, None) == EINVAL
    assert L.fg_plan_workspace(4, 8, 16, ctypes.byref(size)) == OK and size.value == 0
    assert L.fg_plan_workspace(100000, 8, 16, ctypes.byref(size)) == OK and size.value > 0

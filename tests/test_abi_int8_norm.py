"""The integer products', their quantisers' and the block norms' C entry points refuse bad
arguments before touching the device (no GPU needed)."""
import ctypes

import pytest

import moe_grouped_gemm_02_amd as fg

EINVAL, OK = -1, 0
P = ctypes.c_void_p(0x100000)    # aligned, never dereferenced
P2 = ctypes.c_void_p(0x200000)
ODD = ctypes.c_void_p(0x100001)


def call(name, good, **changes):
    args = dict(good)
    assert not set(changes) - set(args)
    args.update(changes)
    return getattr(fg.lib(), name)(*args.values())


DENSE = dict(A=P, sa=P, B=P, sb=P, D=P, M=4, N=64, K=128, stream=None)
CONTIGUOUS = dict(A=P, sa=P, B=P, sb=P, D=P, m_indices=P, M=128, N=64, K=128, G=2, stream=None)
MASKED = dict(A=P, sa=P, B=P, sb=P, D=P, masked_m=P, G=2, M_max=8, N=64, K=128, stream=None)
QUANT = dict(x=P, dtype=0, q=P, s=P, M=4, K=128, stream=None)
DISPATCH = dict(x=P, dtype=0, rows=P, w=None, Q=P, s=P, T=4, k=2, H=128, n_rows=16, stream=None)
SWIGLU = dict(h=P, dtype=0, slots=None, Q=P, s=P, rows=4, I=128, stream=None)
NORM = dict(x=P, y=P, dtype=0, pre=P, post=P, gate=P, gate_kind=1, r=P, h=P2, s=P, out=0, T=4, N=128, alpha=1.0, beta=1.0,
            eps=1e-6, stream=None)
GRAD = dict(r=P, dh=P, dr=P, y=P, dtype=0, pre=P, post=P, gate=P, gate_kind=1, dx=P, dy=P2, dgate=P, dpre=P, dpost=P, ws=P,
            T=4, N=128, alpha=1.0, beta=1.0, eps=1e-6, stream=None)
SIZES = [dict(N=-8), dict(N=60), dict(N=4194304), dict(K=0), dict(K=8), dict(K=24), dict(K=131072), dict(A=None), dict(A=ODD),
         dict(sa=None), dict(sa=ODD), dict(B=None), dict(B=ODD), dict(sb=None), dict(sb=ODD), dict(D=None), dict(D=ODD)]


@pytest.mark.parametrize("name,good,changes", [
    (n, g, c) for n, g, cs in [
        ("fg_gemm_int8_nt", DENSE, SIZES + [dict(M=-1), dict(M=2147483647, N=4194296)]),
        ("fg_grouped_contiguous_int8", CONTIGUOUS, SIZES + [dict(M=-1), dict(G=0), dict(m_indices=None), dict(m_indices=ODD)]),
        ("fg_grouped_masked_int8", MASKED, SIZES + [dict(M_max=-1), dict(G=0), dict(masked_m=None), dict(masked_m=ODD),
                                                    dict(G=1 << 20, M_max=1 << 20)]),
        ("fg_quant_int8", QUANT, [dict(M=-1), dict(K=0), dict(K=120), dict(K=65552), dict(dtype=2), dict(x=None), dict(x=ODD),
                                  dict(q=None), dict(q=ODD), dict(s=None), dict(s=ODD)]),
        ("fg_dispatch_quant_int8", DISPATCH, [dict(T=-1), dict(k=0), dict(H=100), dict(n_rows=-1), dict(dtype=-1), dict(x=None),
                                              dict(rows=None), dict(rows=ODD), dict(w=ODD), dict(Q=None), dict(Q=ODD),
                                              dict(s=None)]),
        ("fg_swiglu_quant_int8", SWIGLU, [dict(rows=-1), dict(I=0), dict(I=64), dict(I=144), dict(I=65664), dict(h=None),
                                          dict(h=ODD), dict(slots=ODD), dict(Q=None), dict(s=ODD)]),
        ("fg_block_norm", NORM, [dict(T=-1), dict(N=0), dict(N=100), dict(N=16392), dict(dtype=2), dict(out=4), dict(out=-1),
                                 dict(out=1, N=64), dict(out=3, N=72), dict(out=1, s=None), dict(eps=0.0), dict(eps=-1.0),
                                 dict(eps=float("nan")), dict(x=None), dict(x=ODD), dict(y=None), dict(y=ODD), dict(r=None),
                                 dict(r=ODD), dict(h=None), dict(h=ODD), dict(gate=None), dict(gate_kind=0), dict(gate_kind=3),
                                 dict(pre=ODD), dict(post=ODD), dict(gate=ODD), dict(s=ODD), dict(h=P),
                                 dict(y=None, post=None, gate=None, gate_kind=0, pre=None)]),
        ("fg_block_norm_grad", GRAD, [dict(T=-1), dict(N=100), dict(N=16392), dict(dtype=3), dict(eps=0.0), dict(r=None),
                                      dict(dh=None), dict(pre=None), dict(y=None), dict(dy=None), dict(dx=None), dict(dpre=None),
                                      dict(dpost=None), dict(dgate=None), dict(gate=None), dict(gate_kind=0), dict(ws=None),
                                      dict(r=ODD), dict(dh=ODD), dict(dr=ODD), dict(y=ODD), dict(dx=ODD), dict(dy=ODD),
                                      dict(ws=ODD), dict(dpre=ODD), dict(dh=None, pre=None, dr=None), dict(dy=P)]),
    ] for c in cs], ids=lambda v: v if isinstance(v, str) else ",".join(v) if isinstance(v, dict) and len(v) < 4 else "")
def test_bad_arguments_are_refused(name, good, changes):
    assert call(name, good, **changes) == EINVAL


@pytest.mark.parametrize("name,good,changes", [
    ("fg_gemm_int8_nt", DENSE, dict(M=2147483647, N=8)), ("fg_gemm_int8_nt", DENSE, dict(M=1 << 30, N=1024)),
    ("fg_grouped_contiguous_int8", CONTIGUOUS, dict(M=1 << 30, N=8)),
    ("fg_grouped_masked_int8", MASKED, dict(G=1 << 23, M_max=1, N=8)), ("fg_grouped_masked_int8", MASKED, dict(G=1 << 22, M_max=300, N=8)),
    ("fg_grouped_masked_int8", MASKED, dict(G=2147483647, M_max=2147483647, N=4194296)),
    ("fg_grouped_masked_int8", MASKED, dict(G=1 << 29, M_max=1 << 30, N=1 << 21))],
    ids=lambda v: v if isinstance(v, str) else "")
def test_products_of_more_tiles_than_a_grid_are_refused(name, good, changes):
    assert call(name, good, **changes) == EINVAL


def test_nothing_to_do_is_a_no_op():
    assert call("fg_gemm_int8_nt", DENSE, M=0, A=None, D=None) == OK
    assert call("fg_gemm_int8_nt", DENSE, N=0, B=None, D=None) == OK
    assert call("fg_grouped_contiguous_int8", CONTIGUOUS, M=0, A=None, m_indices=None) == OK
    assert call("fg_grouped_masked_int8", MASKED, M_max=0, A=None) == OK
    assert call("fg_quant_int8", QUANT, M=0, x=None, q=None) == OK
    assert call("fg_dispatch_quant_int8", DISPATCH, T=0, x=None) == OK
    assert call("fg_dispatch_quant_int8", DISPATCH, n_rows=0, Q=None, s=None) == OK
    assert call("fg_swiglu_quant_int8", SWIGLU, rows=0, h=None) == OK
    assert call("fg_block_norm", NORM, T=0, x=None, r=None, h=None) == OK


def test_gradient_workspace():
    L, size = fg.lib(), ctypes.c_size_t()
    assert L.fg_block_norm_grad_workspace(1, 8, ctypes.byref(size)) == OK and size.value >= 2 * 8 * 4
    assert L.fg_block_norm_grad_workspace(0, 8, ctypes.byref(size)) == OK
    assert L.fg_block_norm_grad_workspace(8192, 7168, ctypes.byref(size)) == OK and size.value >= 2 * 7168 * 4
    # the most rows there may be: no more partial sums than there are workgroups
    assert L.fg_block_norm_grad_workspace(2147483647, 8, ctypes.byref(size)) == OK and 0 < size.value <= 2048 * 2 * 8 * 4
    assert L.fg_block_norm_grad_workspace(4, 12, ctypes.byref(size)) == EINVAL
    assert L.fg_block_norm_grad_workspace(-1, 8, ctypes.byref(size)) == EINVAL
    assert L.fg_block_norm_grad_workspace(4, 8, None) == EINVAL

"""FP8 (OCP E4M3) block-scaled GEMM for AMD MI355X (gfx950).

Thin Python binding over the C ABI of ``libfg.so`` (see ``include/fg.h``):
argument checking and marshalling only. Every step of the computation runs in
the library's HIP kernels; there is no CPU or PyTorch fallback, and calls fail
loudly when the library is missing or the device is not gfx950.

torch is used for device memory and the current HIP stream only.

    D = A . B^T,  D[m, n] = sum_kb sa[m, kb] sb[n // 128, kb] sum_{k in kb} a[m, k] b[n, k]

Tensor conventions (all on the same CUDA/HIP device, contiguous):
    A   uint8 or float8_e4m3fn  [M, K]        (masked: [G, M_max, K])
    sa  float32                 [K/128, M]    (masked: [G, K/128, M_max])
    B   uint8 or float8_e4m3fn  [N, K]        (grouped: [G, N, K])
    sb  float32                 [ceil(N/128), K/128] (grouped: [G, ceil(N/128), K/128])
    D   bfloat16                [M, N]        (masked: [G, M_max, N])

Row operators around the grouped calls (route_topk, plan_contiguous, plan_masked,
dispatch_quant, combine and their gradients) and beside the dense one (adapters):
see their own docstrings; token rows are [T, columns] in bfloat16 or float32,
choices [T, k] int32, weights [T, k] float32.

The same products in 8-bit integers (gemm_int8_nt, grouped_contiguous_int8,
grouped_masked_int8): A and B int8, sa [M] and sb [N] float32, one scale per token and
per output channel (masked: sa [G, M_max]; grouped: sb [G, N]); quant_int8,
dispatch_quant_int8 and swiglu_quant_int8 make their operands. block_norm and
block_norm_grad: the norms before and after a block with its gate and residual scales,
their output in the row's type or as either product's operand.
"""
import ctypes
import functools
import math
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfg.so")

LAYOUT_DENSE, LAYOUT_CONTIGUOUS, LAYOUT_MASKED = 0, 1, 2
SELECT_SWIGLU_QUANT = 0x100      # fg_select_config: the tile of the fused SiLU-gate epilogue
SCALES_FP32, SCALES_POW2 = 0, 1

_lib = None


class FGError(RuntimeError):
    pass


def _declare(L):
    """Argument and return types of every entry point of include/fg.h."""
    vp, fp, ip, i = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int
    ipp = ctypes.POINTER(ctypes.c_int)
    L.fg_gemm_fp8_nt.argtypes = [vp, fp, vp, fp, vp, i, i, i, vp]
    L.fg_grouped_contiguous.argtypes = [vp, fp, vp, fp, vp, ip, i, i, i, i, vp]
    L.fg_grouped_masked.argtypes = [vp, fp, vp, fp, vp, ip, i, i, i, i, vp]
    L.fg_select_config.argtypes = [i, i, i, i, i, i, ipp, ipp]
    L.fg_select_grid.argtypes = [i, i, i, i, i, i, ipp]
    L.fg_quant_act_1x128.argtypes = [vp, vp, vp, i, i, i, vp]
    L.fg_quant_weight_128x128.argtypes = [vp, vp, vp, i, i, i, vp]
    L.fg_gemm_fp8_nt_pow2.argtypes = L.fg_gemm_fp8_nt.argtypes
    L.fg_grouped_contiguous_pow2.argtypes = L.fg_grouped_contiguous.argtypes
    L.fg_grouped_masked_pow2.argtypes = L.fg_grouped_masked.argtypes
    L.fg_quant_act_1x128_pow2.argtypes = L.fg_quant_act_1x128.argtypes
    L.fg_quant_weight_128x128_pow2.argtypes = L.fg_quant_weight_128x128.argtypes
    L.fg_gemm_fp8_nt_swiglu_quant.argtypes = [vp, fp, vp, fp, vp, fp, fp, i, i, i, i, vp]
    L.fg_grouped_contiguous_swiglu_quant.argtypes = [vp, fp, vp, fp, vp, fp, fp, ip, i, i, i, i, i, vp]
    L.fg_grouped_masked_swiglu_quant.argtypes = [vp, fp, vp, fp, vp, fp, fp, ip, i, i, i, i, i, vp]
    sz, f = ctypes.POINTER(ctypes.c_size_t), ctypes.c_float
    L.fg_route_topk.argtypes = [vp, i, fp, ip, fp, i, i, i, i, i, f, vp]
    L.fg_route_topk_grad.argtypes = [vp, i, ip, fp, vp, i, i, i, i, i, f, vp]
    L.fg_plan_capacity.argtypes = [i, i, i, i, ipp]
    L.fg_plan_workspace.argtypes = [i, i, i, sz]
    L.fg_plan_contiguous.argtypes = [ip, ip, ip, ip, ip, vp, i, i, i, i, vp]
    L.fg_plan_masked.argtypes = [ip, ip, ip, ip, vp, i, i, i, i, vp]
    L.fg_dispatch_quant.argtypes = [vp, i, ip, fp, vp, fp, i, i, i, i, i, i, vp]
    L.fg_combine.argtypes = [vp, i, ip, fp, vp, vp, i, i, i, i, vp]
    L.fg_combine_grad.argtypes = [vp, vp, i, ip, fp, vp, fp, i, i, i, i, vp]
    L.fg_combine_grad_quant.argtypes = [vp, vp, i, ip, fp, vp, fp, fp, i, i, i, i, i, i, vp]
    L.fg_adapters_workspace.argtypes = [i, i, i, i, sz]
    L.fg_adapters.argtypes = [vp, vp, vp, vp, fp, ip, ip, ip, ip, vp, vp, i, i, i, i, i, i, i, vp]
    L.fg_gemm_int8_nt.argtypes = [vp, fp, vp, fp, vp, i, i, i, vp]
    L.fg_grouped_contiguous_int8.argtypes = L.fg_grouped_contiguous.argtypes
    L.fg_grouped_masked_int8.argtypes = L.fg_grouped_masked.argtypes
    L.fg_quant_int8.argtypes = [vp, i, vp, fp, i, i, vp]
    L.fg_dispatch_quant_int8.argtypes = [vp, i, ip, fp, vp, fp, i, i, i, i, vp]
    L.fg_swiglu_quant_int8.argtypes = [vp, i, ip, vp, fp, i, i, vp]
    L.fg_block_norm.argtypes = [vp, vp, i, fp, fp, fp, i, vp, vp, fp, i, i, i, f, f, f, vp]
    L.fg_block_norm_grad_workspace.argtypes = [i, i, sz]
    L.fg_block_norm_grad.argtypes = [vp, vp, vp, vp, i, fp, fp, fp, i, vp, vp, fp, fp, fp, vp, i, i, f, f, f, vp]
    L.fg_strerror.argtypes = [i]
    L.fg_strerror.restype = ctypes.c_char_p
    for name in ENTRY_POINTS:
        if name != "fg_strerror":
            getattr(L, name).restype = ctypes.c_int
    return L


ENTRY_POINTS = ("fg_gemm_fp8_nt", "fg_grouped_contiguous", "fg_grouped_masked",
                "fg_select_config", "fg_select_grid", "fg_quant_act_1x128",
                "fg_quant_weight_128x128", "fg_gemm_fp8_nt_pow2", "fg_grouped_contiguous_pow2",
                "fg_grouped_masked_pow2", "fg_quant_act_1x128_pow2",
                "fg_quant_weight_128x128_pow2", "fg_gemm_fp8_nt_swiglu_quant",
                "fg_grouped_contiguous_swiglu_quant", "fg_grouped_masked_swiglu_quant",
                "fg_route_topk", "fg_route_topk_grad", "fg_plan_capacity", "fg_plan_workspace",
               "fg_plan_contiguous", "fg_plan_masked", "fg_dispatch_quant", "fg_combine",
               "fg_combine_grad", "fg_combine_grad_quant", "fg_adapters_workspace", "fg_adapters",
               "fg_gemm_int8_nt", "fg_grouped_contiguous_int8", "fg_grouped_masked_int8", "fg_quant_int8",
               "fg_dispatch_quant_int8", "fg_swiglu_quant_int8", "fg_block_norm", "fg_block_norm_grad_workspace",
               "fg_block_norm_grad",
               "fg_strerror")


def load(path):
    """ctypes handle of a build of the library at `path`, with its entry points
    declared (raises ImportError if the file is missing)."""
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m moe_grouped_gemm_02_amd.build`")
    return _declare(ctypes.CDLL(path))


def lib():
    """Load libfg.so (built in-tree by ``moe_grouped_gemm_02_amd.build``)."""
    global _lib
    if _lib is None:
        _lib = load(LIB_PATH)
    return _lib


def strerror(code):
    return lib().fg_strerror(int(code)).decode()


def _check(code, what):
    if code != 0:
        raise FGError(f"{what}: {strerror(code)} (code {code})")


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_raw_stream = None


_current_device = None


def _stream(t):
    """The current HIP stream of t's device as an address. torch's raw getter takes 0.1 us;
    a Stream object, where a torch has no such getter, 1.9 us, a third of a small call."""
    if _raw_stream is None:
        _getters()
    return _raw_stream(t.device.index)


def _getters():
    """torch's raw getters of the current stream and device (its public ones where it has
    no such), set once CUDA is initialised by the first tensor on a device."""
    global _raw_stream, _current_device
    torch = _torch()
    lib()
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(fn, dev, *args):
    """Calls entry point `fn` with `dev` as the current device (the library
    launches on the current device, on the stream passed last) and raises
    FGError on a nonzero return code."""
    if _current_device is not None and _current_device() == dev.index:
        code = getattr(_lib, fn)(*args)
    else:
        with _torch().cuda.device(dev):
            code = getattr(lib(), fn)(*args)
    if code:
        _check(code, fn)


def _fp8(t, name, shape, device=None):
    torch = _torch()
    if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise TypeError(f"{name} must be uint8 or float8_e4m3fn E4M3 bytes, got {t.dtype}")
    _dev(t, name, shape, device=device)


def _dev(t, name, shape, dtype=None, device=None):
    """Checks a tensor argument: on a GPU (on `device` if given), of `dtype`
    (if given), of `shape`, contiguous."""
    if (t.is_cuda and t.shape == shape and (dtype is None or t.dtype is dtype)
            and (device is None or t.device == device) and t.is_contiguous()):
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's operands on {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _ptr(t):
    return t.data_ptr()


def gemm_fp8_nt(A, sa, B, sb, D):
    """Dense D[M, N] = A[M, K] . B[N, K]^T with block scales; writes D in place."""
    return _dense("fg_gemm_fp8_nt", A, sa, B, sb, D)


def gemm_fp8_nt_pow2(A, sa, B, sb, D):
    """gemm_fp8_nt with power-of-two scales applied by the matrix core (every sa
    and sb entry must be a power of two in [2^-126, 2^127])."""
    return _dense("fg_gemm_fp8_nt_pow2", A, sa, B, sb, D)


def _dense(fn, A, sa, B, sb, D):
    torch = _torch()
    M, K = A.shape
    N = B.shape[0]
    dev = A.device
    _fp8(A, "A", (M, K))
    _fp8(B, "B", (N, K), dev)
    if K % 128 or N % 8:
        raise ValueError("K must be a multiple of 128 and N of 8")
    _dev(sa, "sa", (K // 128, M), torch.float32, dev)
    _dev(sb, "sb", (-(-N // 128), K // 128), torch.float32, dev)
    _dev(D, "D", (M, N), torch.bfloat16, dev)
    _call(fn, dev, _ptr(A), _ptr(sa), _ptr(B), _ptr(sb), _ptr(D), M, N, K, _stream(A))
    return D


def grouped_contiguous(A, sa, B, sb, D, m_indices):
    """MoE contiguous layout: rows of A belong to expert m_indices[row] (-1 = padding,
    not written); B is [G, N, K]."""
    return _contiguous("fg_grouped_contiguous", A, sa, B, sb, D, m_indices)


def grouped_contiguous_pow2(A, sa, B, sb, D, m_indices):
    """grouped_contiguous with power-of-two scales applied by the matrix core."""
    return _contiguous("fg_grouped_contiguous_pow2", A, sa, B, sb, D, m_indices)


def _contiguous(fn, A, sa, B, sb, D, m_indices):
    torch = _torch()
    M, K = A.shape
    G, N = B.shape[0], B.shape[1]
    dev = A.device
    _fp8(A, "A", (M, K))
    _fp8(B, "B", (G, N, K), dev)
    if K % 128 or N % 8:
        raise ValueError("K must be a multiple of 128 and N of 8")
    _dev(sa, "sa", (K // 128, M), torch.float32, dev)
    _dev(sb, "sb", (G, -(-N // 128), K // 128), torch.float32, dev)
    _dev(D, "D", (M, N), torch.bfloat16, dev)
    _dev(m_indices, "m_indices", (M,), torch.int32, dev)
    _call(fn, dev, _ptr(A), _ptr(sa), _ptr(B), _ptr(sb), _ptr(D), _ptr(m_indices), M, N, K, G, _stream(A))
    return D


def grouped_masked(A, sa, B, sb, D, masked_m):
    """MoE masked layout: expert g has masked_m[g] valid rows of A[g]; only those rows
    of D[g] are written. masked_m stays on the device."""
    return _masked("fg_grouped_masked", A, sa, B, sb, D, masked_m)


def grouped_masked_pow2(A, sa, B, sb, D, masked_m):
    """grouped_masked with power-of-two scales applied by the matrix core."""
    return _masked("fg_grouped_masked_pow2", A, sa, B, sb, D, masked_m)


def _masked(fn, A, sa, B, sb, D, masked_m):
    torch = _torch()
    G, M_max, K = A.shape
    N = B.shape[1]
    dev = A.device
    _fp8(A, "A", (G, M_max, K))
    _fp8(B, "B", (G, N, K), dev)
    if K % 128 or N % 8:
        raise ValueError("K must be a multiple of 128 and N of 8")
    _dev(sa, "sa", (G, K // 128, M_max), torch.float32, dev)
    _dev(sb, "sb", (G, -(-N // 128), K // 128), torch.float32, dev)
    _dev(D, "D", (G, M_max, N), torch.bfloat16, dev)
    _dev(masked_m, "masked_m", (G,), torch.int32, dev)
    _call(fn, dev, _ptr(A), _ptr(sa), _ptr(B), _ptr(sb), _ptr(D), _ptr(masked_m), G, M_max, N, K, _stream(A))
    return D


def _fused_outputs(lead, I, M, dev, Q, sq, act, with_act):
    """Allocate (or check) the fused epilogue's outputs: Q [*lead, M, I] uint8,
    sq [*lead, I/128, M] fp32, act [*lead, M, I] fp32 or None."""
    torch = _torch()
    if Q is None:
        Q = torch.empty(lead + (M, I), dtype=torch.uint8, device=dev)
    if sq is None:
        sq = torch.empty(lead + (I // 128, M), dtype=torch.float32, device=dev)
    if act is None and with_act:
        act = torch.empty(lead + (M, I), dtype=torch.float32, device=dev)
    _fp8(Q, "Q", lead + (M, I), dev)
    _dev(sq, "sq", lead + (I // 128, M), torch.float32, dev)
    if act is not None:
        _dev(act, "act", lead + (M, I), torch.float32, dev)
    return Q, sq, act


def _opt_ptr(t):
    return None if t is None else t.data_ptr()


def gemm_fp8_nt_swiglu_quant(A, sa, B, sb, Q=None, sq=None, act=None, pow2=False, with_act=False):
    """Dense first projection with the fused epilogue: H = A . B^T (B's rows
    interleave gate and up every 128), act = silu(gate) * up, quantised per 1x128
    block. Returns (Q [M, N/2] E4M3, sq [N/256, M] fp32, act [M, N/2] fp32 or None).
    pow2: power-of-two input scales and output scales."""
    torch = _torch()
    M, K = A.shape
    N = B.shape[0]
    dev = A.device
    _fp8(A, "A", (M, K))
    _fp8(B, "B", (N, K), dev)
    if K % 128 or N % 256:
        raise ValueError("K must be a multiple of 128 and N of 256")
    _dev(sa, "sa", (K // 128, M), torch.float32, dev)
    _dev(sb, "sb", (N // 128, K // 128), torch.float32, dev)
    Q, sq, act = _fused_outputs((), N // 2, M, dev, Q, sq, act, with_act)
    _call("fg_gemm_fp8_nt_swiglu_quant", dev, _ptr(A), _ptr(sa), _ptr(B), _ptr(sb), _ptr(Q), _ptr(sq),
          _opt_ptr(act), M, N, K, int(bool(pow2)), _stream(A))
    return Q, sq, act


def grouped_contiguous_swiglu_quant(A, sa, B, sb, m_indices, Q=None, sq=None, act=None, pow2=False,
                                    with_act=False):
    """MoE contiguous first projection with the fused epilogue (see
    gemm_fp8_nt_swiglu_quant); padding rows (m_indices = -1) are not written."""
    torch = _torch()
    M, K = A.shape
    G, N = B.shape[0], B.shape[1]
    dev = A.device
    _fp8(A, "A", (M, K))
    _fp8(B, "B", (G, N, K), dev)
    if K % 128 or N % 256:
        raise ValueError("K must be a multiple of 128 and N of 256")
    _dev(sa, "sa", (K // 128, M), torch.float32, dev)
    _dev(sb, "sb", (G, N // 128, K // 128), torch.float32, dev)
    _dev(m_indices, "m_indices", (M,), torch.int32, dev)
    Q, sq, act = _fused_outputs((), N // 2, M, dev, Q, sq, act, with_act)
    _call("fg_grouped_contiguous_swiglu_quant", dev, _ptr(A), _ptr(sa), _ptr(B), _ptr(sb), _ptr(Q), _ptr(sq),
          _opt_ptr(act), _ptr(m_indices), M, N, K, G, int(bool(pow2)), _stream(A))
    return Q, sq, act


def grouped_masked_swiglu_quant(A, sa, B, sb, masked_m, Q=None, sq=None, act=None, pow2=False,
                                with_act=False):
    """MoE masked first projection with the fused epilogue; only rows
    r < masked_m[g] of each expert are written. Q [G, M_max, N/2],
    sq [G, N/256, M_max], act [G, M_max, N/2]."""
    torch = _torch()
    G, M_max, K = A.shape
    N = B.shape[1]
    dev = A.device
    _fp8(A, "A", (G, M_max, K))
    _fp8(B, "B", (G, N, K), dev)
    if K % 128 or N % 256:
        raise ValueError("K must be a multiple of 128 and N of 256")
    _dev(sa, "sa", (G, K // 128, M_max), torch.float32, dev)
    _dev(sb, "sb", (G, N // 128, K // 128), torch.float32, dev)
    _dev(masked_m, "masked_m", (G,), torch.int32, dev)
    Q, sq, act = _fused_outputs((G,), N // 2, M_max, dev, Q, sq, act, with_act)
    _call("fg_grouped_masked_swiglu_quant", dev, _ptr(A), _ptr(sa), _ptr(B), _ptr(sb), _ptr(Q), _ptr(sq),
          _opt_ptr(act), _ptr(masked_m), G, M_max, N, K, int(bool(pow2)), _stream(A))
    return Q, sq, act


def select_config(M, N, K, G=1, layout=LAYOUT_DENSE, num_cus=0):
    """(bm, bn): the tile the library would launch for the problem (layout
    optionally | SELECT_SWIGLU_QUANT); host-only, no device access."""
    bm, bn = ctypes.c_int(), ctypes.c_int()
    _check(lib().fg_select_config(M, N, K, G, layout, num_cus, ctypes.byref(bm), ctypes.byref(bn)),
           "fg_select_config")
    return bm.value, bn.value


def select_grid(M, N, K, G=1, layout=LAYOUT_DENSE, num_cus=0):
    """Workgroups the launch for the problem would use; host-only."""
    grid = ctypes.c_int()
    _check(lib().fg_select_grid(M, N, K, G, layout, num_cus, ctypes.byref(grid)), "fg_select_grid")
    return grid.value


def quant_act_1x128(x, q=None, sa=None):
    """fp32 activations [M, K] (or [batch, M, K]) -> (E4M3 codes, sa) with one scale per
    1x128 block; sa comes out in the GEMM's layout [K/128, M] ([batch, K/128, M])."""
    return _quant_act("fg_quant_act_1x128", x, q, sa)


def quant_act_1x128_pow2(x, q=None, sa=None):
    """quant_act_1x128 with each scale rounded up to a power of two (>= 2^-126)."""
    return _quant_act("fg_quant_act_1x128_pow2", x, q, sa)


def _quant_act(fn, x, q, sa):
    torch = _torch()
    if x.dim() not in (2, 3):
        raise ValueError("x must be [M, K] or [batch, M, K]")
    batch = x.shape[0] if x.dim() == 3 else 1
    M, K = x.shape[-2], x.shape[-1]
    if K % 128:
        raise ValueError("K must be a multiple of 128")
    _dev(x, "x", tuple(x.shape), torch.float32)
    if q is None:
        q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    sa_shape = (batch, K // 128, M) if x.dim() == 3 else (K // 128, M)
    if sa is None:
        sa = torch.empty(sa_shape, dtype=torch.float32, device=x.device)
    _fp8(q, "q", tuple(x.shape), x.device)
    _dev(sa, "sa", sa_shape, torch.float32, x.device)
    _call(fn, x.device, _ptr(x), _ptr(q), _ptr(sa), batch, M, K, _stream(x))
    return q, sa


def quant_weight_128x128(w, q=None, sb=None):
    """fp32 weights [N, K] (or [G, N, K]) -> (E4M3 codes, sb) with one scale per
    128x128 block; sb is [ceil(N/128), K/128] ([G, ceil(N/128), K/128]). N need
    not be a multiple of 128: the last row block then holds N mod 128 rows."""
    return _quant_weight("fg_quant_weight_128x128", w, q, sb)


def quant_weight_128x128_pow2(w, q=None, sb=None):
    """quant_weight_128x128 with each scale rounded up to a power of two (>= 2^-126)."""
    return _quant_weight("fg_quant_weight_128x128_pow2", w, q, sb)


def _quant_weight(fn, w, q, sb):
    torch = _torch()
    if w.dim() not in (2, 3):
        raise ValueError("w must be [N, K] or [G, N, K]")
    G = w.shape[0] if w.dim() == 3 else 1
    N, K = w.shape[-2], w.shape[-1]
    if K % 128:
        raise ValueError("K must be a multiple of 128")
    _dev(w, "w", tuple(w.shape), torch.float32)
    sb_shape = tuple(w.shape[:-2]) + (-(-N // 128), K // 128)
    if q is None:
        q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    if sb is None:
        sb = torch.empty(sb_shape, dtype=torch.float32, device=w.device)
    _fp8(q, "q", tuple(w.shape), w.device)
    _dev(sb, "sb", sb_shape, torch.float32, w.device)
    _call(fn, w.device, _ptr(w), _ptr(q), _ptr(sb), G, N, K, _stream(w))
    return q, sb


# ---------------------------------------------------------------- row operators
SCORES = {"softmax": 0, "sigmoid": 1}


def _elem(t, name):
    """fg.h element type of an activation tensor."""
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return 0
    if t.dtype == torch.float32:
        return 1
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _score(score):
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    return SCORES[score]


def _new(t, name, shape, dtype, dev):
    """An output: the caller's, checked, or a new one."""
    if t is None:
        return _torch().empty(shape, dtype=dtype, device=dev)
    _dev(t, name, shape, dtype, dev)
    return t


def route_topk(logits, k, score="softmax", bias=None, renorm=False, scale=1.0, ids=None, w=None):
    """Each token's k best experts from router logits [T, E] (bf16 or fp32; -inf or NaN
    masks an expert): (ids [T, k] int32, best first, -1 where fewer are left, w [T, k]
    fp32). score: "softmax" or "sigmoid"; bias [E] fp32 is added to the scores for the
    ranking only; renorm divides the chosen scores by their sum; scale multiplies w.
    Ties go to the lower index."""
    torch = _torch()
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    dev = logits.device
    dt, sc = _elem(logits, "logits"), _score(score)
    if not 1 <= k <= min(E, 64):
        raise ValueError(f"k must be in 1 .. min(E, 64), got {k} for E = {E}")
    _dev(logits, "logits", (T, E))
    if bias is not None:
        _dev(bias, "bias", (E,), torch.float32, dev)
    ids = _new(ids, "ids", (T, k), torch.int32, dev)
    w = _new(w, "w", (T, k), torch.float32, dev)
    _call("fg_route_topk", dev, _ptr(logits), dt, _opt_ptr(bias), _ptr(ids), _ptr(w), T, E, k, sc, int(bool(renorm)),
          scale, _stream(logits))
    return ids, w


def route_topk_grad(logits, ids, dw, score="softmax", renorm=False, scale=1.0, dlogits=None):
    """Gradient of route_topk's w [T, k] with respect to its logits, the choice ids taken as
    given; the other arguments as in the forward call. Returns dlogits, in logits' type."""
    torch = _torch()
    if logits.dim() != 2 or ids.dim() != 2:
        raise ValueError("logits must be [T, E] and ids [T, k]")
    T, E = logits.shape
    k = ids.shape[1]
    dev = logits.device
    dt, sc = _elem(logits, "logits"), _score(score)
    _dev(logits, "logits", (T, E))
    _dev(ids, "ids", (T, k), torch.int32, dev)
    _dev(dw, "dw", (T, k), torch.float32, dev)
    dlogits = _new(dlogits, "dlogits", (T, E), logits.dtype, dev)
    _call("fg_route_topk_grad", dev, _ptr(logits), dt, _ptr(ids), _ptr(dw), _ptr(dlogits), T, E, k, sc,
          int(bool(renorm)), scale, _stream(logits))
    return dlogits


class Plan:
    """Where each (token, choice) slot's row is in a grouped GEMM's layout; made by
    plan_contiguous or plan_masked, or from tensors of the same meaning.

    rows [T, k] int32: the slot's row, -1 if none; slots int32: each row's slot t * k + j,
    -1 if none. Contiguous: m_indices (per row, as grouped_contiguous takes it), offsets
    [G + 1], align. Masked: masked_m [G], M_max; row g * M_max + r is row r of expert g."""
    __slots__ = ("layout", "rows", "slots", "m_indices", "offsets", "align", "masked_m", "M_max", "G",
                 "T", "k", "device", "capacity", "lead", "_blocks")

    def __init__(self, layout, rows, slots, m_indices, offsets, align, masked_m, M_max, G):
        self.layout, self.rows, self.slots, self.G = layout, rows, slots, G
        self.m_indices, self.offsets, self.align = m_indices, offsets, align
        self.masked_m, self.M_max = masked_m, M_max
        self.T, self.k = rows.shape
        self.device = rows.device
        self.capacity = slots.shape[0]          # rows of the layout (masked: G * M_max)
        # leading dimensions of the layout's tensors: (capacity,) or (G, M_max)
        self.lead = (G, M_max) if layout == LAYOUT_MASKED else (self.capacity,)
        self._blocks = self.lead if layout == LAYOUT_MASKED else (1, self.capacity)   # the library's G, M

    @classmethod
    def contiguous(cls, rows, slots, m_indices, offsets, align):
        cap, G = _plan_rows(rows, slots), offsets.shape[0] - 1
        _index(m_indices, "m_indices", rows.device, cap)
        _index(offsets, "offsets", rows.device, G + 1)
        if align < 1 or cap % align or G < 1:
            raise ValueError("a contiguous plan has G + 1 >= 2 offsets and a multiple of align rows")
        return cls(LAYOUT_CONTIGUOUS, rows, slots, m_indices, offsets, align, None, 0, G)

    @classmethod
    def masked(cls, rows, slots, masked_m, M_max):
        cap, G = _plan_rows(rows, slots), masked_m.shape[0]
        _index(masked_m, "masked_m", rows.device, G)
        if cap != G * M_max or M_max < 1 or G < 1:
            raise ValueError("a masked plan has G * M_max slots")
        return cls(LAYOUT_MASKED, rows, slots, None, None, 1, masked_m, M_max, G)


def _index(t, name, device, n):
    """Checks an int32 vector of n entries on `device`."""
    if t.dtype is not _torch().int32 or t.device != device or t.shape != (n,) or not t.is_contiguous():
        _dev(t, name, (n,), _torch().int32, device)


def _plan_rows(rows, slots):
    if rows.dim() != 2 or slots.dim() != 1:
        raise ValueError("rows must be [T, k] and slots [rows]")
    _dev(rows, "rows", rows.shape, _torch().int32)
    cap = slots.shape[0]
    _index(slots, "slots", rows.device, cap)
    return cap


def _plan_args(ids, G):
    torch = _torch()
    if ids.dim() != 2:
        raise ValueError("ids must be [T, k]")
    T, k = ids.shape
    _dev(ids, "ids", (T, k), torch.int32)
    if not 1 <= G <= 1024 or k < 1:
        raise ValueError("G must be in 1 .. 1024 and k at least 1")
    size = _plan_workspace(T, k, G)
    return T, k, torch.empty(size, dtype=torch.uint8, device=ids.device) if size else None


@functools.lru_cache(maxsize=1024)
def _plan_workspace(T, k, G):
    size = ctypes.c_size_t()
    _check(lib().fg_plan_workspace(T, k, G, ctypes.byref(size)), "fg_plan_workspace")
    return size.value


@functools.lru_cache(maxsize=1024)
def plan_capacity(T, k, G, align=128):
    """Rows of a contiguous plan, the most that any ids [T, k] can need; host-only."""
    rows = ctypes.c_int()
    _check(lib().fg_plan_capacity(T, k, G, align, ctypes.byref(rows)), "fg_plan_capacity")
    return rows.value


def _int32_parts(dev, *sizes):
    """New int32 vectors of these sizes in one allocation."""
    torch = _torch()
    return torch.empty(sum(sizes), dtype=torch.int32, device=dev).split_with_sizes(sizes)


def plan_contiguous(ids, G, align=128):
    """Stable sort of the slots by expert (ids [T, k] int32; outside [0, G): no row) into the
    contiguous layout, segments starting at multiples of align rows. Returns a Plan."""
    torch = _torch()
    T, k, ws = _plan_args(ids, G)
    dev = ids.device
    cap = plan_capacity(T, k, G, align)
    m_indices, slots, rows, offsets = _int32_parts(dev, cap, cap, T * k, G + 1)
    rows = rows.view(T, k)
    _call("fg_plan_contiguous", dev, _ptr(ids), _ptr(rows), _ptr(slots), _ptr(m_indices), _ptr(offsets),
          _opt_ptr(ws), T, k, G, align, _stream(ids))
    return Plan(LAYOUT_CONTIGUOUS, rows, slots, m_indices, offsets, align, None, 0, G)


def plan_masked(ids, G, M_max):
    """The same into the masked layout: at most M_max rows per expert, later slots get no row."""
    torch = _torch()
    T, k, ws = _plan_args(ids, G)
    if M_max < 1 or G * M_max > 0x7fffffff:
        raise ValueError("M_max must be at least 1 and G * M_max below 2^31")
    dev = ids.device
    slots, rows, masked_m = _int32_parts(dev, G * M_max, T * k, G)
    rows = rows.view(T, k)
    _call("fg_plan_masked", dev, _ptr(ids), _ptr(rows), _ptr(slots), _ptr(masked_m), _opt_ptr(ws), T, k, G, M_max,
          _stream(ids))
    return Plan(LAYOUT_MASKED, rows, slots, None, None, 1, masked_m, M_max, G)


def _quant_rows(plan, H, Q, sa):
    """The sorted E4M3 operand: Q [*lead, H], sa [H/128, capacity] or [G, H/128, M_max]."""
    torch = _torch()
    lead = plan.lead
    if H % 128 or H < 128:
        raise ValueError("rows must be a positive multiple of 128 long")
    if Q is None:
        Q = torch.empty(lead + (H,), dtype=torch.uint8, device=plan.device)
    else:
        _fp8(Q, "Q", lead + (H,), plan.device)
    sa = _new(sa, "sa", lead[:-1] + (H // 128, lead[-1]), torch.float32, plan.device)
    return Q, sa


def dispatch_quant(x, plan, w=None, pow2=False, Q=None, sa=None):
    """Token rows x [T, H] (bf16 or fp32), times w [T, k] if given, into the plan's layout as
    the grouped GEMM's A operand: E4M3 codes Q ([capacity, H] or [G, M_max, H]) and scales sa
    ([H/128, capacity] or [G, H/128, M_max]). Rows without a slot are not written."""
    dt = _elem(x, "x")
    dev, T, k = plan.device, plan.T, plan.k
    if x.dim() != 2:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [{T}, columns]")
    H = x.shape[1]
    _dev(x, "x", (T, H), None, dev)
    if w is not None:
        _dev(w, "w", (T, k), _torch().float32, dev)
    Q, sa = _quant_rows(plan, H, Q, sa)
    G, M = plan._blocks
    _call("fg_dispatch_quant", dev, _ptr(x), dt, _ptr(plan.rows), _opt_ptr(w), _ptr(Q), _ptr(sa), T, k, H, G, M,
          int(bool(pow2)), _stream(x))
    return Q, sa


def _sorted_rows(y, plan):
    if y.dim() != len(plan.lead) + 1:
        raise ValueError(f"y has shape {tuple(y.shape)}, expected {plan.lead} + (N,)")
    N = y.shape[-1]
    _dev(y, "y", plan.lead + (N,), None, plan.device)
    if N % 8 or N < 8:
        raise ValueError("N must be a positive multiple of 8")
    return N


def combine(y, plan, w=None, base=None, out=None):
    """out[t] = base[t] + sum_j w[t, j] y[row of slot (t, j)]: the experts' rows back in token
    order ([T, N], y's type). w None: all ones, which is unweighted dispatch's gradient. out may be base."""
    dt = _elem(y, "y")
    N = _sorted_rows(y, plan)
    dev, T, k = plan.device, plan.T, plan.k
    if w is not None:
        _dev(w, "w", (T, k), _torch().float32, dev)
    if base is not None:
        _dev(base, "base", (T, N), y.dtype, dev)
    out = _new(out, "out", (T, N), y.dtype, dev)
    _call("fg_combine", dev, _ptr(y), dt, _ptr(plan.rows), _opt_ptr(w), _opt_ptr(base), _ptr(out), T, k, N,
          plan.capacity, _stream(y))
    return out


def dispatch_grad(dA, plan, out=None, w=None):
    """Gradient of dispatch's copies with respect to x: the sum of each token's sorted rows, times
    w [T, k] where dispatch_quant was given it. The weights' own gradient <x[t], dA[row]> is the dw of
    combine_grad(x, dA, plan, w, with_dy=False). The rounding to E4M3 is passed over."""
    return combine(dA, plan, w=w, out=out)


def _combine_grad_args(dout, y, plan, w, dw):
    dt = _elem(y, "y")
    N = _sorted_rows(y, plan)
    dev, T, k = plan.device, plan.T, plan.k
    f32 = _torch().float32
    _dev(dout, "dout", (T, N), y.dtype, dev)
    _dev(w, "w", (T, k), f32, dev)
    return dt, N, _new(dw, "dw", (T, k), f32, dev)


def combine_grad(dout, y, plan, w, dy=None, dw=None, with_dy=True):
    """Gradient of combine: (dy in y's shape and type, rows without a slot not written, or None
    with with_dy=False; dw [T, k] fp32)."""
    dt, N, dw = _combine_grad_args(dout, y, plan, w, dw)
    if dy is not None or with_dy:
        dy = _new(dy, "dy", y.shape, y.dtype, plan.device)
    _call("fg_combine_grad", plan.device, _ptr(dout), _ptr(y), dt, _ptr(plan.rows), _ptr(w), _opt_ptr(dy), _ptr(dw),
          plan.T, plan.k, N, plan.capacity, _stream(dout))
    return dy, dw


def combine_grad_quant(dout, y, plan, w, pow2=False, Q=None, sa=None, dw=None):
    """combine_grad with dy as the backward GEMM's operand: (Q E4M3 codes, sa scales, dw)."""
    dt, N, dw = _combine_grad_args(dout, y, plan, w, dw)
    Q, sa = _quant_rows(plan, N, Q, sa)
    G, M = plan._blocks
    _call("fg_combine_grad_quant", plan.device, _ptr(dout), _ptr(y), dt, _ptr(plan.rows), _ptr(w), _ptr(Q), _ptr(sa),
          _ptr(dw), plan.T, plan.k, N, G, M, int(bool(pow2)), _stream(dout))
    return Q, sa, dw


@functools.lru_cache(maxsize=1024)
def _adapters_workspace(R, K, cap, align):
    size = ctypes.c_size_t()
    _check(lib().fg_adapters_workspace(R, K, cap, align, ctypes.byref(size)), "fg_adapters_workspace")
    return size.value


def adapters(D, x, A, B, scales, plan, out=None):
    """Low-rank adapters of many requests beside a shared projection: out[t] = D[t] +
    scales[a] (x[t] . A[a]^T) . B[a]^T for token t's adapter a, D[t] for a token without one.
    D [T, N], x [T, K], A [L, R, K], B [L, N, R] bf16, scales [L] fp32; plan: plan_contiguous of
    the tokens' adapter ids [T, 1] with align 64 (prompts) or 16 (decode). out may be D (in place)."""
    torch = _torch()
    if D.dim() != 2 or x.dim() != 2 or A.dim() != 3:
        raise ValueError("D must be [T, N], x [T, K] and A [L, R, K]")
    if plan.layout != LAYOUT_CONTIGUOUS or plan.k != 1 or plan.align % 16:
        raise ValueError("adapters need a contiguous plan of ids [T, 1] with align a multiple of 16")
    T, N = D.shape
    L, R, K = A.shape
    dev = D.device
    bf = torch.bfloat16
    if plan.T != T or plan.G != L or plan.device != dev:
        raise ValueError(f"the plan is of {plan.T} tokens and {plan.G} adapters on {plan.device}, "
                         f"the call of {T} and {L} on {dev}")
    if R % 8 or not 8 <= R <= 128 or K % 128 or N % 8:
        raise ValueError("R must be a multiple of 8 up to 128, K of 128 and N of 8")
    _dev(D, "D", (T, N), bf, dev)
    _dev(x, "x", (T, K), bf, dev)
    _dev(A, "A", (L, R, K), bf, dev)
    _dev(B, "B", (L, N, R), bf, dev)
    _dev(scales, "scales", (L,), torch.float32, dev)
    out = _new(out, "out", (T, N), bf, dev)
    ws = torch.empty(_adapters_workspace(R, K, plan.capacity, plan.align), dtype=torch.uint8, device=dev)
    _call("fg_adapters", dev, _ptr(D), _ptr(x), _ptr(A), _ptr(B), _ptr(scales), _ptr(plan.rows), _ptr(plan.slots),
          _ptr(plan.m_indices), _ptr(plan.offsets), _ptr(out), _ptr(ws), T, L, R, K, N, plan.capacity, plan.align, _stream(D))
    return out


# ---------------------------------------------------------------- 8-bit integers
# These calls check their tensors in one expression of plain attributes (a third of the time of a
# check each, and a quarter of a small call); where it fails, _dev names the tensor and what is wrong.
def _is(t, dtype, shape, index):
    """Whether t is a contiguous tensor of this type and shape on GPU `index`."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()


_INT_MAX = 2 ** 31 - 1


def _too_large(*sizes):
    """Raised by the calls below for sizes past a C int, of which ctypes would pass on the low 32 bits."""
    raise ValueError(f"every size must be below 2^31, got {max(sizes)}")


def _int8_product(fn, A, sa, B, sb, D, lead, N, K, index, *sizes):
    """Checks and makes the call of an integer product; lead: the leading dimensions of A and D, index: the
    layout's tensor with its name and shape (None: dense), sizes: the call's."""
    torch = _torch()
    d = A.get_device()
    i8, f32 = torch.int8, torch.float32
    if not (d >= 0 and A.dtype is i8 and A.is_contiguous() and _is(B, i8, B.shape, d) and _is(sa, f32, lead, d)
            and _is(sb, f32, B.shape[:-1], d) and _is(D, torch.bfloat16, lead + (N,), d)
            and (index is None or _is(index[0], torch.int32, index[2], d))):
        dev = A.device
        _dev(A, "A", lead + (K,), i8)
        _dev(B, "B", B.shape, i8, dev)
        _dev(sa, "sa", lead, f32, dev)
        _dev(sb, "sb", B.shape[:-1], f32, dev)
        _dev(D, "D", lead + (N,), torch.bfloat16, dev)
        if index is not None:
            _dev(index[0], index[1], index[2], torch.int32, dev)
    if K % 16 or not 16 <= K <= 131056 or N % 8:
        raise ValueError("K must be a multiple of 16 from 16 to 131056 and N of 8")
    if max(sizes) > _INT_MAX:
        _too_large(*sizes)
    stream = _raw_stream(d) if _raw_stream is not None else _stream(A)
    if index is None:
        _call(fn, A.device, A.data_ptr(), sa.data_ptr(), B.data_ptr(), sb.data_ptr(), D.data_ptr(), *sizes, stream)
    else:
        _call(fn, A.device, A.data_ptr(), sa.data_ptr(), B.data_ptr(), sb.data_ptr(), D.data_ptr(), index[0].data_ptr(),
              *sizes, stream)
    return D


def gemm_int8_nt(A, sa, B, sb, D):
    """Dense D[m, n] = sa[m] sb[n] sum_k A[m, k] B[n, k]: A [M, K] and B [N, K] int8, sa [M] and
    sb [N] float32, the sum exact in 32-bit integers; writes D [M, N] bfloat16 in place."""
    a, b = A.shape, B.shape
    if len(a) != 2 or len(b) != 2 or a[1] != b[1]:
        raise ValueError(f"A must be [M, K] and B [N, K], got {tuple(a)} and {tuple(b)}")
    (M, K), N = a, b[0]
    return _int8_product("fg_gemm_int8_nt", A, sa, B, sb, D, (M,), N, K, None, M, N, K)


def grouped_contiguous_int8(A, sa, B, sb, D, m_indices):
    """gemm_int8_nt in the contiguous layout: rows of A belong to expert m_indices[row] (-1 =
    padding, not written); B [G, N, K], sb [G, N]."""
    a, b = A.shape, B.shape
    if len(a) != 2 or len(b) != 3 or a[1] != b[2]:
        raise ValueError(f"A must be [M, K] and B [G, N, K], got {tuple(a)} and {tuple(b)}")
    (M, K), (G, N, _) = a, b
    return _int8_product("fg_grouped_contiguous_int8", A, sa, B, sb, D, (M,), N, K, (m_indices, "m_indices", (M,)),
                         M, N, K, G)


def grouped_masked_int8(A, sa, B, sb, D, masked_m):
    """gemm_int8_nt in the masked layout: expert g has masked_m[g] valid rows of A[g], and only
    those of D[g] are written; A [G, M_max, K], sa [G, M_max], B [G, N, K], sb [G, N]."""
    a, b = A.shape, B.shape
    if len(a) != 3 or len(b) != 3 or a[2] != b[2] or a[0] != b[0]:
        raise ValueError(f"A must be [G, M_max, K] and B [G, N, K], got {tuple(a)} and {tuple(b)}")
    (G, M_max, K), N = a, b[1]
    return _int8_product("fg_grouped_masked_int8", A, sa, B, sb, D, (G, M_max), N, K, (masked_m, "masked_m", (G,)),
                         G, M_max, N, K)


def _int8_rows(x, lead, K, q, s):
    """Outputs of an integer quantiser on x's device: codes [*lead, K] and scales lead."""
    torch = _torch()
    if K % 16 or not 16 <= K <= 65536:
        raise ValueError("rows must be a multiple of 16 long, from 16 to 65536")
    rows = math.prod(lead)
    if rows > _INT_MAX:
        _too_large(rows)
    shape = tuple(lead) + (K,)
    if q is None:
        q = torch.empty_like(x, dtype=torch.int8) if x.shape == shape else torch.empty(shape, dtype=torch.int8, device=x.device)
    else:
        _dev(q, "q", shape, torch.int8, x.device)
    return q, _new(s, "s", tuple(lead), torch.float32, x.device)


def quant_int8(x, q=None, s=None):
    """Rows of x [..., K] (bf16 or fp32; activations, or weights whose rows are output channels) as
    8-bit integers with one scale each: (q int8 in x's shape, s [...] fp32), x about q * s."""
    dt = _elem(x, "x")
    if x.dim() < 2:
        raise ValueError("x must be [..., rows, K]")
    lead, K = x.shape[:-1], x.shape[-1]
    _dev(x, "x", x.shape)
    q, s = _int8_rows(x, lead, K, q, s)
    _call("fg_quant_int8", x.device, _ptr(x), dt, _ptr(q), _ptr(s), s.numel(), K, _stream(x))
    return q, s


def dispatch_quant_int8(x, plan, w=None, Q=None, s=None):
    """Token rows x [T, H] (bf16 or fp32), times w [T, k] if given, into the plan's layout as the
    grouped integer product's A operand: Q int8 ([capacity, H] or [G, M_max, H]) and s ([capacity]
    or [G, M_max]). Rows without a slot are not written."""
    dt = _elem(x, "x")
    dev, T, k = plan.device, plan.T, plan.k
    if x.dim() != 2:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [{T}, columns]")
    H = x.shape[1]
    _dev(x, "x", (T, H), None, dev)
    if T > _INT_MAX or k > _INT_MAX:
        _too_large(T, k)
    if w is not None:
        _dev(w, "w", (T, k), _torch().float32, dev)
    Q, s = _int8_rows(x, plan.lead, H, Q, s)
    _call("fg_dispatch_quant_int8", dev, _ptr(x), dt, _ptr(plan.rows), _opt_ptr(w), _ptr(Q), _ptr(s), T, k, H,
          plan.capacity, _stream(x))
    return Q, s


def swiglu_quant_int8(h, plan=None, Q=None, s=None):
    """silu(gate) * up of a first projection's output h [..., 2 I] (bf16 or fp32; gate and up
    interleaved every 128 columns) as the next integer product's operand: Q int8 [..., I], s [...].
    With a plan h is in its layout, and rows without a slot are neither read nor written."""
    dt = _elem(h, "h")
    if h.dim() < 2 or h.shape[-1] % 256:
        raise ValueError("h must be [..., rows, 2 I] with 2 I a multiple of 256")
    lead, I = h.shape[:-1], h.shape[-1] // 2
    _dev(h, "h", h.shape)
    if plan is not None and (lead != plan.lead or h.device != plan.device):
        raise ValueError(f"h has shape {tuple(h.shape)} on {h.device}, the plan's rows are {plan.lead} on {plan.device}")
    Q, s = _int8_rows(h, lead, I, Q, s)
    _call("fg_swiglu_quant_int8", h.device, _ptr(h), dt, None if plan is None else _ptr(plan.slots), _ptr(Q), _ptr(s),
          s.numel(), I, _stream(h))
    return Q, s


# ---------------------------------------------------------------- norms around a block
def _new_like(t, name, like):
    """An output of a checked (contiguous) tensor's shape, type and device; empty_like costs half of empty."""
    if t is None:
        return _torch().empty_like(like)
    _dev(t, name, like.shape, like.dtype, like.device)
    return t


NORM_OUTPUTS = {None: 0, "e4m3": 1, "e4m3_pow2": 2, "int8": 3}


def _norm_args(x, name, y, pre, post, gate, eps):
    """Checks what block_norm and its gradient share: (element type, T, N, gate kind, GPU)."""
    torch = _torch()
    dt, shape, f32, d = _elem(x, name), x.shape, torch.float32, x.get_device()
    if len(shape) != 2:
        raise ValueError(f"{name} must be [T, N], got {tuple(shape)}")
    T, N = shape
    if not (d >= 0 and x.is_contiguous()):
        _dev(x, name, shape)
    if T > _INT_MAX:
        _too_large(T)
    if N % 8 or not 8 <= N <= 16384:
        raise ValueError("N must be a multiple of 8 from 8 to 16384")
    if not eps > 0:
        raise ValueError("eps must be positive")
    if y is not None:
        if not _is(y, x.dtype, shape, d):
            _dev(y, "y", shape, x.dtype, x.device)
    elif post is not None or gate is not None:
        raise ValueError("post and gate belong to a block's output y")
    if pre is not None and not _is(pre, f32, (N,), d):
        _dev(pre, "pre", (N,), f32, x.device)
    if post is not None and not _is(post, f32, (N,), d):
        _dev(post, "post", (N,), f32, x.device)
    if gate is None:
        return dt, T, N, 0, d
    kind = 1 if gate.dim() == 1 else 2
    if not _is(gate, f32, (N,) if kind == 1 else (T, 1), d):
        _dev(gate, "gate", (N,) if kind == 1 else (T, 1), f32, x.device)
    return dt, T, N, kind, d


def block_norm(x, y=None, pre=None, post=None, gate=None, alpha=1.0, beta=1.0, eps=1e-6, quant=None, r=None, h=None, s=None):
    """The norms around a block in one pass, x [T, N] the residual stream and y [T, N] the block's
    output (both bf16 or both fp32):

        u = y / sqrt(mean y^2 + eps) * post       (y itself without post [N] fp32)
        r = alpha x + beta gate u                 (x itself without y, whatever alpha; gate fp32 [N] or [T, 1], or none)
        h = r / sqrt(mean r^2 + eps) * pre        (None without pre [N] fp32), of r before its rounding

    Returns (r, h, s). quant None: h in x's type, s None; "e4m3" or "e4m3_pow2": h the E4M3 product's
    operand (uint8 codes) with its scales s [N/128, T]; "int8": the integer product's (int8 codes, s [T]).
    r may be x or y (in place)."""
    torch = _torch()
    if quant not in NORM_OUTPUTS:
        raise ValueError(f"quant must be one of {list(NORM_OUTPUTS)}, got {quant!r}")
    if y is None and pre is None:
        raise ValueError("block_norm needs a block's output y, the next norm's weight pre, or both")
    dt, T, N, kind, d = _norm_args(x, "x", y, pre, post, gate, eps)
    out = NORM_OUTPUTS[quant]
    if pre is None and quant is not None:
        raise ValueError("quant is for h, which needs pre")
    if (h is not None and pre is None) or (s is not None and out == 0):
        raise ValueError("h is written where there is pre, s where there is quant")
    if y is not None:
        r = _new_like(r, "r", x)
    elif r is not None and r is not x:
        raise ValueError("without y the stream is x itself")
    if pre is None:
        h = s = None
    elif out == 0:
        h, s = _new_like(h, "h", x), None
    elif out == 3:
        h, s = _int8_rows(x, (T,), N, h, s)
    else:
        if N % 128:
            raise ValueError("E4M3 rows must be a multiple of 128 long")
        if h is None:
            h = torch.empty_like(x, dtype=torch.uint8)
        else:
            _fp8(h, "h", (T, N), x.device)
        s = _new(s, "s", (N // 128, T), torch.float32, x.device)
    _call("fg_block_norm", x.device, _ptr(x), _opt_ptr(y), dt, _opt_ptr(pre), _opt_ptr(post), _opt_ptr(gate), kind,
          None if y is None else _ptr(r), _opt_ptr(h), _opt_ptr(s), out, T, N, alpha, beta, eps,
          _raw_stream(d) if _raw_stream is not None else _stream(x))
    return (x if y is None else r), h, s


@functools.lru_cache(maxsize=1024)
def _block_norm_grad_workspace(T, N):
    size = ctypes.c_size_t()
    _check(lib().fg_block_norm_grad_workspace(T, N, ctypes.byref(size)), "fg_block_norm_grad_workspace")
    return size.value


def block_norm_grad(r, dh=None, dr=None, y=None, pre=None, post=None, gate=None, alpha=1.0, beta=1.0, eps=1e-6,
                    dx=None, dy=None):
    """Gradient of block_norm at the stream r it returned: dh the gradient of h (with pre), dr that of r from
    what else reads it (None: none), the other arguments as in the forward call (pre None if h was not used).
    Returns (dx, dy, dgate, dpre, dpost): dx and dy in r's type, the vectors fp32; None where the forward call
    had no such input. Without y, r is x: alpha and beta are not used. dx may be dr or dh, dy may be y (in place)."""
    torch = _torch()
    if (dh is None) != (pre is None):
        raise ValueError("dh and pre belong together")
    if dh is None and dr is None:
        raise ValueError("block_norm_grad needs dh, dr, or both")
    dt, T, N, kind, d = _norm_args(r, "r", y, pre, post, gate, eps)
    if dh is not None and not _is(dh, r.dtype, (T, N), d):
        _dev(dh, "dh", (T, N), r.dtype, r.device)
    if dr is not None and not _is(dr, r.dtype, (T, N), d):
        _dev(dr, "dr", (T, N), r.dtype, r.device)
    dx = _new_like(dx, "dx", r)
    if y is not None:
        dy = _new_like(dy, "dy", r)
    elif dy is not None:
        raise ValueError("dy is y's gradient, and there is no y")
    dgate, dpre, dpost = (None if v is None else torch.empty_like(v) for v in (gate, pre, post))
    dev = r.device
    ws = torch.empty(_block_norm_grad_workspace(T, N), dtype=torch.uint8, device=dev)
    _call("fg_block_norm_grad", dev, _ptr(r), _opt_ptr(dh), _opt_ptr(dr), _opt_ptr(y), dt, _opt_ptr(pre), _opt_ptr(post),
          _opt_ptr(gate), kind, _ptr(dx), _opt_ptr(dy), _opt_ptr(dgate), _opt_ptr(dpre), _opt_ptr(dpost), _ptr(ws), T, N,
          alpha, beta, eps, _raw_stream(d) if _raw_stream is not None else _stream(r))
    return dx, dy, dgate, dpre, dpost

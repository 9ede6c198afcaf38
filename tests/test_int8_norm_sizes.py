"""Sizes that a C int does not hold are refused by the integer and norm calls instead of being cut to its 32 bits
(tensors without memory; no GPU needed)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import moe_grouped_gemm_02_amd as fg

MANY = 2 ** 32 + 8     # 8 in 32 bits


@pytest.fixture
def no_calls(monkeypatch):
    def reached(fn, *args):
        raise AssertionError(f"{fn} was called")
    monkeypatch.setattr(fg, "_call", reached)
    monkeypatch.setattr(fg, "_raw_stream", lambda index: 0)
    with FakeTensorMode():
        yield


def new(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="cuda")


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
@pytest.mark.parametrize("M", [2 ** 31, MANY])
def test_rows(no_calls, M):
    bf16, i8 = torch.bfloat16, torch.int8
    x, w = new(M, 16, dtype=bf16), new(16)
    some = new(8, 16, dtype=i8), new(8)
    for call in [lambda: fg.quant_int8(x), lambda: fg.quant_int8(new(2, M // 2, 16)), lambda: fg.block_norm(x, pre=w),
                 lambda: fg.block_norm(x, x, pre=w, quant="int8"), lambda: fg.block_norm_grad(x, dh=x, pre=w),
                 lambda: fg.block_norm_grad(x, dr=x, y=x, gate=new(M, 1)), lambda: fg.swiglu_quant_int8(new(M, 256)),
                 lambda: fg.gemm_int8_nt(new(M, 16, dtype=i8), new(M), *some, new(M, 8, dtype=bf16)),
                 lambda: fg.gemm_int8_nt(*some, new(M, 16, dtype=i8), new(M), new(8, M, dtype=bf16)),
                 lambda: fg.grouped_masked_int8(new(1, M, 16, dtype=i8), new(1, M), new(1, 8, 16, dtype=i8), new(1, 8),
                                                new(1, M, 8, dtype=bf16), new(1, dtype=torch.int32)),
                 lambda: fg.grouped_contiguous_int8(new(M, 16, dtype=i8), new(M), new(1, 8, 16, dtype=i8), new(1, 8),
                                                    new(M, 8, dtype=bf16), new(M, dtype=torch.int32))]:
        with pytest.raises(ValueError):
            call()


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
@pytest.mark.parametrize("T,k,rows", [(MANY, 1, 16), (4, 1, MANY), (4, MANY, 16)])
def test_plans(no_calls, T, k, rows):
    """Tokens or choices of a plan that the caller made, or its rows."""
    plan = fg.Plan.contiguous(new(T, k, dtype=torch.int32), new(rows, dtype=torch.int32), new(rows, dtype=torch.int32),
                              new(2, dtype=torch.int32), 8)
    with pytest.raises(ValueError):
        fg.dispatch_quant_int8(new(T, 16), plan)

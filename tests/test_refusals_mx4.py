"""What the MXFP4 and decoding entry points refuse, on the host, before any
device call."""

import ctypes

import pytest
import torch

import fp8_quantized_moe_gb300 as moe


@pytest.fixture(scope="module")
def lib():
    return moe.lib()


P = ctypes.c_void_p(256)  # a 16-byte aligned dummy address (never dereferenced)
ODD = ctypes.c_void_p(264)


def test_quantisers(lib):
    assert lib.moe_quantize_rows_mx4(None, 4, 128, P, P, None) == 1
    assert lib.moe_quantize_rows_mx4(P, 4, 128, P, None, None) == 1
    assert lib.moe_quantize_rows_mx4(P, 4, 96, P, P, None) == 1          # cols % 128
    assert lib.moe_quantize_rows_mx4(P, 4, 32896, P, P, None) == 1       # cols > 32768
    assert lib.moe_quantize_rows_mx4(P, -1, 128, P, P, None) == 1
    assert lib.moe_quantize_rows_mx4(P, 1 << 31, 128, P, P, None) == 1
    assert lib.moe_quantize_rows_mx4(ODD, 4, 128, P, P, None) == 1
    assert lib.moe_quantize_rows_mx4(P, 4, 128, P, ctypes.c_void_p(258), None) == 1
    assert lib.moe_quantize_rows_mx4(P, 0, 128, P, P, None) == 0         # nothing to do
    assert lib.moe_dequantize_rows_mx4(P, P, 4, 96, P, None) == 1
    assert lib.moe_dequantize_rows_mx4(P, P, 4, 128, None, None) == 1
    assert lib.moe_dequantize_rows_mx4(P, P, 4, 128, ODD, None) == 1
    assert lib.moe_swiglu_quant_mx4(P, 4, 96, P, P, None) == 1
    assert lib.moe_swiglu_quant_mx4(P, 4, 128, ODD, P, None) == 1
    assert lib.moe_quantize_sort_mx4(P, P, 4, 2, 4, 96, P, P, P, P, P, P, P, 1 << 20, None) == 1
    assert lib.moe_quantize_sort_mx4(P, P, 4, 2, 4, 32896, P, P, P, P, P, P, P, 1 << 20, None) == 1
    assert lib.moe_quantize_sort_mx4(P, P, 4, 33, 4, 128, P, P, P, P, P, P, P, 1 << 20, None) == 1
    assert lib.moe_quantize_sort_mx4(P, P, 4, 2, 4, 128, P, P, P, P, P, P, P, 0, None) == 1
    assert lib.moe_quantize_sort_mx4(P, P, 4, 2, 4, 128, P, P, P, P, P, None, P, 1 << 20, None) == 1


def test_binding_checks_types_and_shapes():
    x = torch.zeros(4, 256)
    with pytest.raises(moe.MoEError):
        moe.quantize_rows_mx4(x)                               # fp32
    with pytest.raises(moe.MoEError):
        moe.quantize_rows_mx4(x.bfloat16()[0])                 # one dimension
    with pytest.raises(moe.MoEError):
        moe.quantize_rows_mx4(x.bfloat16())                    # not on the GPU
    with pytest.raises(moe.MoEError):
        moe.dequantize_rows_mx4(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(1, 4, 4, dtype=torch.uint8))
    with pytest.raises(moe.MoEError):
        moe.quantize_rows_mx4(x.bfloat16(), q=torch.zeros(4, 256, dtype=torch.uint8))
    with pytest.raises(moe.MoEError):
        moe.quantize_sort_mx4(x.bfloat16(), torch.zeros(3, 2, dtype=torch.int32), 4)   # T differs
    with pytest.raises(moe.MoEError):
        moe.quantize_sort_mx4(x.bfloat16(), torch.zeros(4, 2, dtype=torch.int64), 4)   # ids not int32
    with pytest.raises(moe.MoEError):
        moe.swiglu_quant_mx4(x)


def test_product(lib):
    def call(lq=P, ls=P, rq=P, rs=P, sz=P, E=4, g0=0, El=4, M=8, K=256, N=64, out=P):
        return lib.gmm_fp4_mx(lq, ls, rq, rs, sz, E, g0, El, M, K, N, out, None)

    for bad in (dict(lq=None), dict(ls=None), dict(rq=None), dict(rs=None), dict(sz=None), dict(out=None), dict(E=0),
                dict(E=1025), dict(g0=-1), dict(El=0), dict(g0=1), dict(E=2, g0=1, El=2), dict(M=-1), dict(M=1 << 31),
                dict(K=0), dict(K=192), dict(K=1 << 30), dict(N=0), dict(N=24), dict(N=1 << 30), dict(lq=ODD),
                dict(rq=ODD), dict(out=ODD), dict(ls=ctypes.c_void_p(258)), dict(rs=ctypes.c_void_p(258)),
                dict(El=2147483647, E=1024)):
        assert call(**bad) == 1, bad


def test_product_binding():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    sizes = torch.tensor([3, 5], dtype=torch.int32)
    good = [u8(8, 128), u8(2, 8, 4), u8(2, 32, 128), u8(2, 64, 4), sizes]
    for i, bad in ((0, u8(8, 64)), (0, u8(8, 128).to(torch.int8)), (1, u8(8, 2, 4)), (2, u8(2, 32, 64)), (3, u8(2, 32, 4)),
                   (4, sizes.long())):
        with pytest.raises(moe.MoEError):
            moe.gmm_mx4(*good[:i], bad, *good[i + 1:])
    with pytest.raises(moe.MoEError):
        moe.gmm_mx4(*good, E_local=1)
    with pytest.raises(moe.MoEError):
        moe.gmm_mx4(*good)  # not on the GPU

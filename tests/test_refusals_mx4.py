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
                dict(rq=ODD), dict(out=ODD), dict(ls=ctypes.c_void_p(258)), dict(rs=ctypes.c_void_p(260)),
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


def test_decode(lib):
    def call(x=P, ids=P, w=P, T=4, k=2, E=8, g0=0, El=8, D=256, F=128, kind=0, wi=P, si=P, mi=0, wo=P, so=P, mo=0, y=P,
             ws=P, nws=1 << 30):
        return lib.moe_ffn_decode(x, ids, w, T, k, E, g0, El, D, F, kind, wi, si, mi, wo, so, mo, y, ws, nws, None)

    need = lib.moe_ffn_decode_workspace_bytes(4, 2, 256, 128)
    assert need >= 4 * 8 * (256 + 128)
    for bad in (dict(x=None), dict(ids=None), dict(wi=None), dict(si=None), dict(wo=None), dict(so=None), dict(y=None),
                dict(ws=None), dict(T=-1), dict(T=65), dict(k=0), dict(k=33), dict(T=64, k=17), dict(D=0), dict(D=24),
                dict(F=24), dict(D=32784), dict(F=32784), dict(E=0), dict(E=1025), dict(g0=-1), dict(g0=1), dict(El=0),
                dict(El=9), dict(kind=4), dict(kind=-1), dict(mi=3), dict(mi=4), dict(mo=7), dict(nws=need - 1),
                dict(mi=1, D=144), dict(mo=1, D=144), dict(mi=1, F=144), dict(kind=2, D=144), dict(kind=3, F=144),
                dict(x=ODD), dict(wi=ODD), dict(wo=ODD), dict(si=ODD), dict(so=ODD), dict(y=ODD), dict(ws=ODD),
                dict(E=1024, El=1024, F=32768, D=32768, T=1, nws=1 << 40, g0=1)):
        assert call(**bad) == 1, bad
    for shape in ((65, 2, 256, 128), (4, 0, 256, 128), (4, 2, 250, 128), (64, 17, 256, 128), (-1, 2, 256, 128)):
        assert lib.moe_ffn_decode_workspace_bytes(*shape) == 0


def test_decode_binding():
    u8, f32 = (lambda *s: torch.zeros(*s, dtype=torch.uint8)), torch.zeros
    x, ids, w = torch.zeros(2, 256, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32), f32(2, 2)
    W = moe.ExpertWeights(u8(4, 256, 256), f32(4, 256), moe.PER_ROW, u8(4, 256, 128), f32(4, 256), moe.PER_ROW)
    with pytest.raises(moe.MoEError):
        moe.ffn_decode(x, ids, w, W)  # not on the GPU
    with pytest.raises(moe.MoEError):
        moe.ffn_decode(x.float(), ids, w, W)
    with pytest.raises(moe.MoEError):
        moe.ffn_decode(x, ids.long(), w, W)
    with pytest.raises(moe.MoEError):
        moe.DecodeBuffers(65, 256, 4, 2, 128, "cpu")
    with pytest.raises(moe.MoEError):
        moe.DecodeBuffers(4, 250, 4, 2, 128, "cpu")

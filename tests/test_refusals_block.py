"""Calls that the operators on block-scaled 8-bit experts and the balance loss refuse, on
the host: nothing is launched, so no GPU is needed."""

import ctypes

import pytest
import torch

moe = pytest.importorskip("fp8_quantized_moe_gb300")

P = ctypes.c_void_p(256)      # a 16-byte aligned address, never dereferenced
ODD = ctypes.c_void_p(264)
INVALID = 1


@pytest.fixture(scope="module")
def lib():
    return moe.lib()


def gmm(lib, a=P, sa=P, b=P, sb=P, g=P, E=1, g0=0, El=1, M=8, K=128, N=256, out=P):
    return lib.gmm_fp8_block(a, sa, b, sb, g, E, g0, El, M, K, N, out, None)


@pytest.mark.parametrize("bad", [
    dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(out=None), dict(g=None, E=2),
    dict(a=ODD), dict(sa=ODD), dict(b=ODD), dict(sb=ODD), dict(out=ODD),
    dict(E=0), dict(E=1025), dict(E=2, g0=1, El=2), dict(g0=-1), dict(El=0), dict(M=-1), dict(M=(1 << 31) - 100),
    dict(K=0), dict(K=144), dict(K=64), dict(N=0), dict(N=24), dict(N=1 << 31), dict(E=1024, El=1024, N=1 << 22),
    dict(M=1 << 30, N=1 << 30),
])
def test_gmm_block(lib, bad):
    assert gmm(lib, **bad) == INVALID


def tgmm(lib, x=P, L=8, idx=None, k=1, d=P, g=P, E=1, g0=0, El=1, M=8, K=16, N=16, out=P, ws=P, n=1 << 30):
    return lib.tgmm_fp8_mx(x, L, idx, k, d, g, E, g0, El, M, K, N, out, ws, n, None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(d=None), dict(g=None), dict(out=None), dict(ws=None), dict(x=ODD), dict(d=ODD), dict(out=ODD),
    dict(ws=ODD), dict(E=0), dict(E=1025), dict(E=2, g0=1, El=2), dict(g0=-1), dict(El=0), dict(M=-1), dict(L=7),
    dict(k=2), dict(k=0, idx=P), dict(L=-1, idx=P), dict(K=0), dict(K=24), dict(N=24), dict(N=0), dict(n=1000),
    dict(M=(1 << 31) - 8, L=(1 << 31) - 8), dict(M=1 << 24, L=1 << 24, K=1 << 20), dict(K=1 << 20, N=1 << 20, E=1024, El=1024),
])
def test_tgmm_mx(lib, bad):
    assert tgmm(lib, **bad) == INVALID


def test_tgmm_mx_workspace(lib):
    n = lib.tgmm_fp8_mx_workspace_bytes
    assert n(1000, 256, 512, 8) >= (1000 + 8 * 127) // 128 * 128 * (256 + 512)
    assert n(8, 16, 16, 1) >= 128 * 32 and n(0, 16, 16, 1) > 0
    assert n(8, 24, 16, 1) == n(8, 16, 24, 1) == n(-1, 16, 16, 1) == n(8, 16, 16, 0) == n(8, 16, 16, 1025) == 0
    assert tgmm(lib, n=n(8, 16, 16, 1) - 1) == INVALID


@pytest.mark.parametrize("bad", [
    dict(w=None), dict(q=None), dict(s=None), dict(q_t=P), dict(s_t=P), dict(w=ODD), dict(q=ODD), dict(s=ODD),
    dict(q_t=ODD, s_t=P, N=128), dict(q_t=P, s_t=ODD, N=128), dict(q_t=P, s_t=P, N=144), dict(E=0), dict(N=0),
    dict(K=0), dict(K=64), dict(E=1 << 30, N=1 << 20),
])
def test_quantize_weights_block(lib, bad):
    a = dict(dict(w=P, E=1, N=16, K=128, q=P, s=P, q_t=None, s_t=None), **bad)
    assert lib.moe_quantize_weights_block(a["w"], a["E"], a["N"], a["K"], a["q"], a["s"], a["q_t"], a["s_t"], None) == INVALID


def test_backward_helpers(lib):
    f = lib.moe_gather_scale_quant_block
    assert f(None, P, P, 1, 1, 128, P, P, P, None) == INVALID
    assert f(P, P, P, 1, 1, 144, P, P, P, None) == INVALID       # D % 128
    assert f(P, P, P, 1, 0, 128, P, P, P, None) == INVALID
    assert f(P, P, P, 1 << 30, 2, 128, P, P, P, None) == INVALID
    assert f(P, P, P, 1, 1, 128, P, P, ODD, None) == INVALID
    f = lib.moe_swiglu_bwd_quant_block
    assert f(P, P, 1, 144, P, P, P, P, None) == INVALID          # F % 128
    assert f(P, P, 1, 128, P, P, P, None, None) == INVALID
    assert f(P, P, -1, 128, P, P, P, P, None) == INVALID
    assert f(P, P, 1, 16512, P, P, P, P, None) == INVALID        # 2F > 32768
    assert f(P, ODD, 1, 128, P, P, P, P, None) == INVALID


def balance(lib, x=P, i=P, v=None, T=8, E=4, k=2, S=1, out=P, ws=P, n=1 << 20):
    return lib.moe_router_balance(x, i, v, T, E, k, S, 1.0, out, P, P, P, ws, n, None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(i=None), dict(out=None), dict(ws=None), dict(x=ODD), dict(ws=ODD), dict(T=-1), dict(S=0),
    dict(S=3), dict(S=16), dict(E=0), dict(E=1025), dict(k=0), dict(k=33), dict(T=1 << 30, k=2), dict(n=8),
])
def test_balance(lib, bad):
    assert balance(lib, **bad) == INVALID
    if "n" not in bad and "x" not in bad and "i" not in bad and "out" not in bad and "ws" not in bad:
        a = dict(dict(T=8, E=4, k=2, S=1), **bad)
        assert lib.moe_router_balance_workspace_bytes(a["T"], a["E"], a["k"], a["S"]) == 0
        assert lib.moe_router_balance_backward(P, None, a["T"], a["E"], a["k"], a["S"], 1.0, P, P, None, P, None) == INVALID


def test_balance_backward(lib):
    f = lib.moe_router_balance_backward
    assert f(None, None, 8, 4, 2, 1, 1.0, P, P, None, P, None) == INVALID
    assert f(P, None, 8, 4, 2, 1, 1.0, None, P, None, P, None) == INVALID
    assert f(P, None, 8, 4, 2, 1, 1.0, P, None, None, P, None) == INVALID
    assert f(P, None, 8, 4, 2, 1, 1.0, P, P, None, None, None) == INVALID
    assert f(P, None, 8, 4, 2, 1, 1.0, P, P, None, ODD, None) == INVALID


def test_tensors_of_another_device_or_type_are_refused_by_name():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    u8, f32, i32 = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 1), torch.zeros(1, dtype=torch.int32)
    w, sw = torch.zeros(1, 16, 128, dtype=torch.uint8), torch.zeros(1, 1, 1)
    for call in (lambda: moe.gmm_block(u8, f32, w, sw), lambda: moe.gmm_block(x, f32, w, sw),
                 lambda: moe.gmm_block(u8, f32, w, sw, i32.long()),
                 lambda: moe.tgmm_mx(x, x, i32), lambda: moe.tgmm_mx(x.float(), x, i32), lambda: moe.tgmm_mx(x, x[:3], i32),
                 lambda: moe.quantize_weights_block(x[None]), lambda: moe.quantize_weights_block(x),
                 lambda: moe.gather_scale_quant_block(x, None, i32, 1), lambda: moe.swiglu_bwd_quant_block(x, x),
                 lambda: moe.router_balance_loss(f32, i32[:, None]), lambda: moe.router_balance_loss(x, i32[:, None])):
        with pytest.raises(moe.MoEError):
            call()

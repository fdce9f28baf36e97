"""GPU tests of scales below 2^-125, whose reciprocals are past fp32 (or next to it): codes are
e4m3 of the exact quotient, and zeros stay zeros.  All bit-exact against the oracle, and the
fused forms against the separate ones."""

import numpy as np
import pytest
import torch

import oracle
from tests.gpu_helpers import assert_close, dev, host, rand_codes, ragged_sizes
from tests.test_gpu_gmm import GC, R0, RB, RT
from tests.test_gpu_w8 import make_w8_case, w8_args, w8_both

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("fp8_quantized_moe_gb300")


def tiny(rng, shape):
    """bf16 bits of values near 2^-122, a third of them zero, columns of unequal size."""
    v = rng.standard_normal(shape) * np.exp2(rng.integers(-126, -112, (1, shape[1])).astype(np.float64))
    v[:, 1::7] = 0
    return oracle.bf16_bits(torch.from_numpy(np.where(rng.random(shape) < 0.3, 0.0, v)).to(torch.bfloat16))


@pytest.mark.parametrize("M,N,E,g0,El", [(1, 16, 1, 0, 1), (300, 256, 9, 0, 9), (500, 96, 8, 2, 4)])
def test_quantize_group_cols(M, N, E, g0, El):
    rng = np.random.default_rng(M)
    sizes = ragged_sizes(rng, E, M)
    g = tiny(rng, (M, N))
    q_ref, s_ref = oracle.quantize_group_cols(g, sizes, g0, El)
    q, s = moe.quantize_group_cols(dev(g), dev(sizes), g0, El)
    assert np.array_equal(host(s), s_ref) and (M < 10 or s_ref.min() < 2.0 ** -128)
    starts = np.concatenate([[0], np.cumsum(sizes)])
    lo, hi = starts[g0], starts[g0 + El]
    assert np.array_equal(host(q)[lo:hi], q_ref[lo:hi])


@pytest.mark.parametrize("M,K,N,E", [(200, 64, 96, 3), (1000, 128, 272, 7)])
def test_gradient_codes_made_in_the_transposed_layout(M, K, N, E):
    rng = np.random.default_rng(M)
    sizes = ragged_sizes(rng, E, M)
    x, g = rand_codes(rng, (M, K)), tiny(rng, (M, N))
    sx = dev(np.array([2.0 ** 100], np.float32))  # the products are ordinary numbers again
    gq, gs = moe.quantize_group_cols(dev(g), dev(sizes))
    want = moe.tgmm(dev(x), sx, RT, gq, gs, GC, dev(sizes))
    out = moe.tgmm_gcq(dev(x), sx, RT, dev(g), gs, dev(sizes))
    assert moe.device_error() == 0
    assert out.isfinite().all() and out.any() and torch.equal(out, want)


@pytest.mark.parametrize("M,K,F,E,amode,wmode,hmode", [
    (300, 256, 256, 4, R0, R0, R0), (300, 256, 256, 4, R0, R0, RB), (300, 256, 256, 4, R0, R0, RT),
    (200, 4096, 256, 3, R0, R0, R0), (200, 4096, 256, 3, R0, R0, RB), (200, 4096, 256, 3, RT, RT, RT),
    (300, 384, 256, 3, RB, RB, R0), (300, 384, 256, 3, RB, RB, RB), (300, 384, 256, 3, RB, R0, RT),
])
def test_fused_swiglu_of_tiny_activations(M, K, F, E, amode, wmode, hmode):
    rng = np.random.default_rng(M + K + hmode)
    sizes = ragged_sizes(rng, E, M)
    a, w = rand_codes(rng, (M, K)), rand_codes(rng, (E, 2 * F, K))
    w[:, 3::5] = 0  # a0 or a1, and so h, is zero in these columns
    a[::9] = 0
    nb = oracle.nblocks(K)
    # a0 and a1 of some 2^-60, h of some 2^-121, rows of unequal size
    top = 2.0 ** -60 / (150.0 ** 2 * np.sqrt(K))
    row = np.exp2(rng.integers(-4, 5, M).astype(np.float64))
    sa = {R0: row * top, RB: np.repeat(row[:, None] * top, nb, 1), RT: [top]}[amode]
    sw = {R0: np.ones((E, 2 * F)), RB: np.ones((E, nb, 2 * F)), RT: [1.0]}[wmode]
    sa, sw = np.asarray(sa, np.float32), np.asarray(sw, np.float32)
    hs = dev(np.array([2.0 ** -130], np.float32))
    args = (dev(a), dev(sa), amode, dev(w), dev(sw), wmode, dev(sizes))
    a_ref = moe.gmm(*args)
    hq, hsc, a_out = moe.gmm_swiglu(*args, hmode, hs, keep_a=True)
    assert moe.device_error() == 0 and torch.equal(a_out, a_ref)
    hq_ref, hs_ref = moe.swiglu_quant(a_ref, hmode, hs)
    q_or, s_or, hb = oracle.swiglu_quant(host(a_ref), hmode, 2.0 ** -130)
    assert 0.2 < (hb & 0x7FFF == 0).mean() < 0.9
    assert np.array_equal(host(hq_ref), q_or) and np.array_equal(host(hq), q_or)
    if hmode != RT:
        assert (s_or < 2.0 ** -128).any()
        assert np.array_equal(host(hs_ref), s_or) and np.array_equal(host(hsc), s_or)


@pytest.mark.parametrize("M,K,N,E", [(200, 256, 512, 3), (700, 768, 384, 2)])
def test_int8_weights_with_tiny_block_scales(M, K, N, E):
    sizes, a, sa, q, sw = make_w8_case(M, M, K, N, E, w_mode=RB, spread=4)
    sw = np.ldexp(sw, -118).astype(np.float32)
    sw[:, :, ::2] = np.ldexp(sw[:, :, ::2], 40)  # beside ordinary channels
    sa = np.ldexp(sa, 90).astype(np.float32)
    assert 0 < sw.min() < 2.0 ** -130
    ref = oracle.gmm_w8(a, sa, R0, q, sw, RB, sizes)
    out = w8_both(w8_args(a, sa, R0, q, sw, RB, sizes), M, K)
    assert moe.device_error() == 0
    # each channel by itself: the tolerance of blockwise int8 weights
    for part in (slice(0, None, 2), slice(1, None, 2)):
        assert_close(np.ascontiguousarray(out[:, part]), np.ascontiguousarray(ref[:, part]), "tiny block scales")

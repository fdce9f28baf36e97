"""The failure paths of the MXFP4 product and of the decoding step: the warps that
consume are held on a barrier that nothing arrives on (a test hook, 200 us), so
that their wait runs out.  The kernel stops, lets its copies and products finish,
returns and reports MOE_DEVERR_TIMEOUT; the context stays usable."""

import contextlib

import pytest

from tests.gpu_helpers import dev
from tests.mx4_helpers import pack, sf_kmajor
from tests.test_gpu_decode import KINDS, case, check, make_weights
from tests.test_gpu_mx4 import assert_product, mx4_case

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("fp8_quantized_moe_gb300")

TIMEOUT = 0x4


@contextlib.contextmanager
def consumers_held():
    assert moe.device_error() == 0
    moe.lib().moe_test_stall_consumers(200_000)
    try:
        yield
    finally:
        moe.lib().moe_test_stall_consumers(0)


@pytest.mark.parametrize("M,K,N,E", [
    (100, 256, 256, 1),    # the producer has issued all it has and is done
    (4096, 512, 1024, 8),  # several tiles a CTA: every role waits
    (2048, 4096, 512, 4),  # a long K loop
    (65, 384, 48, 3),      # odd K blocks, an N tail
])
def test_product(M, K, N, E):
    sizes, a, asf, w, wsf = mx4_case(M + K, M, K, N, E)
    args = (dev(pack(a)), dev(sf_kmajor(asf)), dev(pack(w)), dev(sf_kmajor(wsf.reshape(E * N, K // 32))), dev(sizes))
    with consumers_held():
        moe.gmm_mx4(*args)
        assert moe.device_error() == TIMEOUT
    out = moe.gmm_mx4(*args)
    assert moe.device_error() == 0
    assert_product(out, sizes, a, asf, w, wsf)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,k,E,D,F", [
    (1, 1, 2, 128, 128),     # a CTA's weights of both phases fit the ring
    (16, 4, 8, 1024, 1280),  # the producer waits for its ring
])
def test_decoding_step(kind, T, k, E, D, F):
    rng, x, ids, w = case(T + D, T, k, E, D)
    W = make_weights(kind, E, D, F, rng)
    buf = moe.DecodeBuffers(T, D, E, k, F, "cuda")
    idd, wd = dev(ids), dev(w)
    with consumers_held():
        moe.ffn_decode(x, idd, wd, W, buf)
        assert moe.device_error() == TIMEOUT
    buf.reset()
    check(moe.ffn_decode(x, idd, wd, W, buf), x, ids, w, W)


@pytest.mark.parametrize("kind", ["e4m3-block", "mx4"])
def test_steps_after_one_that_timed_out(kind):
    """What it left in the workspace gives no wrong result in silence: steps report
    the error until the buffers are reset; steps on other buffers go on."""
    rng, x, ids, w = case(3, 9, 4, 8, 512)
    W = make_weights(kind, 8, 512, 256, rng)
    buf, other = (moe.DecodeBuffers(9, 512, 8, 4, 256, "cuda") for _ in range(2))
    idd, wd = dev(ids), dev(w)
    with consumers_held():
        moe.ffn_decode(x, idd, wd, W, buf)
        assert moe.device_error() == TIMEOUT
    for n in (9, 2):
        moe.ffn_decode(x[:n], idd[:n], wd[:n], W, buf)
        assert moe.device_error() == TIMEOUT
    check(moe.ffn_decode(x, idd, wd, W, other), x, ids, w, W)
    buf.reset()
    for _ in range(2):
        check(moe.ffn_decode(x, idd, wd, W, buf), x, ids, w, W)

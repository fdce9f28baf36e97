"""The failure path of the MXFP4 product: its consumers are held on a barrier
that nothing arrives on (a test hook, 200 us), so that their wait runs out.  The
kernel stops, lets its copies and products finish, returns and reports
MOE_DEVERR_TIMEOUT; the context stays usable."""

import contextlib

import pytest

from tests.gpu_helpers import dev
from tests.mx4_helpers import pack, sf_kmajor
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

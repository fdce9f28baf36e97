"""The workspace of a decoding step: what is asked for a batch of T tokens serves
every smaller batch (host arithmetic, no GPU)."""

import pytest

import fp8_quantized_moe_gb300 as moe


@pytest.mark.parametrize("D,F", [(16, 16), (128, 32768), (4096, 14336), (7168, 2048), (32768, 128)])
def test_never_less_for_more_tokens(D, F):
    need = moe.lib().moe_ffn_decode_workspace_bytes
    for k in range(1, 33):
        last = min(64, 1024 // k)
        sizes = [need(T, k, D, F) for T in range(0, last + 1)]
        assert all(sizes) and sizes == sorted(sizes), (k, sizes)
        # and not more than the largest batch's sums or a few pairs' sums of segments take
        assert sizes[-1] <= 16384 + max(4 * last * k * (D + F), 512 * (D + 2 * F)), (k, sizes[-1])


def test_buffers_serve_every_smaller_batch():
    need = moe.lib().moe_ffn_decode_workspace_bytes
    for T, k in ((64, 2), (63, 1), (28, 8), (17, 1), (12, 8)):
        buf = moe.DecodeBuffers(T, 256, 40, k, 384, "cpu")
        assert all(need(t, k, 256, 384) <= buf.ws_bytes for t in range(T + 1)), (T, k)

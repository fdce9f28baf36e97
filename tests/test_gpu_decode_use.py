"""Decoding steps as a server runs them: batches that grow and shrink on the same
buffers.  Values against the float64 oracle, in the bound that
test_gpu_decode.py derives."""

import pytest
import torch

from tests.gpu_helpers import dev
from tests.test_gpu_decode import case, check, make_weights

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("fp8_quantized_moe_gb300")


@pytest.mark.parametrize("kind", ["e4m3-block", "mx4"])
@pytest.mark.parametrize("T,k,steps", [(64, 2, (64, 33, 32, 16, 8, 5, 1)), (16, 8, (16, 8, 7, 2, 1)), (63, 1, (63, 32, 16, 1))])
def test_a_batch_that_drains(kind, T, k, steps):
    rng, x, ids, w = case(T, T, k, 12, 512)
    W = make_weights(kind, 12, 512, 256, rng)
    buf = moe.DecodeBuffers(T, 512, 12, k, 256, "cuda")
    for n in steps + steps[::-1]:
        y = moe.ffn_decode(x[:n], dev(ids[:n]), dev(w[:n]), W, buf)
        assert y.data_ptr() == buf.y.data_ptr()
        check(y, x[:n], ids[:n], w[:n], W)


@pytest.mark.parametrize("T,k,E", [(8, 2, 8), (16, 4, 8), (64, 8, 16)])
@pytest.mark.parametrize("D,F", [(256, 768), (1536, 128), (2304, 1280)])
def test_mx4_ring_goes_round(T, k, E, D, F):
    """Two groups on alternate stages: rings of both chunk widths, units of one
    stage, of odd and of even numbers, one after the other; 200 calls alike."""
    rng, x, ids, w = case(T + D, T, k, E, D)
    W = make_weights("mx4", E, D, F, rng)
    idd, wd, buf = dev(ids), dev(w), moe.DecodeBuffers(T, D, E, k, F, "cuda")
    first = moe.ffn_decode(x, idd, wd, W, buf).clone()
    check(first, x, ids, w, W)
    differs = torch.zeros((), dtype=torch.bool, device="cuda")
    for _ in range(200):
        differs |= (moe.ffn_decode(x, idd, wd, W, buf) != first).any()
    assert not differs.item() and moe.device_error() == 0


def test_buffers_are_ready_on_any_stream():
    """The workspace is zero when the constructor returns, whatever the creating
    stream still has to do and whatever the memory held before."""
    n = moe.DecodeBuffers(8, 1024, 4, 2, 1024, "cuda").ws_bytes
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    junk = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    del junk  # (its memory is the next to be handed out for this size)
    torch.cuda._sleep(200_000_000)  # some 0.1 s of work on the creating stream
    buf = moe.DecodeBuffers(8, 1024, 4, 2, 1024, "cuda")
    with torch.cuda.stream(side):
        seen = buf.ws.any()
    side.synchronize()
    assert not seen.item()
    rng, x, ids, w = case(50, 8, 2, 4, 1024)
    W = make_weights("e4m3-channel", 4, 1024, 1024, rng)
    idd, wd = dev(ids), dev(w)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    buf = moe.DecodeBuffers(8, 1024, 4, 2, 1024, "cuda")
    with torch.cuda.stream(side):
        y = moe.ffn_decode(x, idd, wd, W, buf)
    side.synchronize()
    check(y, x, ids, w, W)


def test_captured_without_buffers():
    """The buffers of a call without any are made, and zeroed, in the graph."""
    rng, x, ids, w = case(51, 5, 2, 4, 256)
    W = make_weights("mx8", 4, 256, 128, rng)
    idd, wd = dev(ids), dev(w)
    moe.ffn_decode(x, idd, wd, W)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = moe.ffn_decode(x, idd, wd, W)
        z = moe.ffn_decode(x, idd, wd, W, moe.DecodeBuffers(8, 256, 4, 2, 128, "cuda"))
    for _ in range(3):
        y.fill_(7.0), z.fill_(7.0)
        g.replay()
        check(y, x, ids, w, W)
        check(z, x, ids, w, W)

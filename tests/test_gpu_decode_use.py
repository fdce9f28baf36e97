"""Decoding steps as a server runs them: batches that grow and shrink on the same
buffers, tokens alone and in a batch, shards, layers one after the other.  Values
against the float64 oracle, in the bound that test_gpu_decode.py derives."""

import numpy as np
import pytest
import torch

import oracle
from tests.gpu_helpers import dev
from tests.test_gpu_decode import KINDS, bound, case, check, make_weights, values

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


def tolerance(x, ids, w, W, g0=0):
    """(the float64 result, how far a bf16 one may be from it)."""
    w_in, w_out = values(W.w_in, W.s_in, W.in_mode), values(W.w_out, W.s_out, W.out_mode)
    xf = x.double().cpu().numpy()
    want = oracle.ffn_decode(xf, ids, w, w_in, w_out, g0)
    return want, bound(xf, ids, w, w_in, w_out, g0) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)


@pytest.mark.parametrize("kind", ["e4m3-block", "mx4"])
def test_a_token_alone_and_in_its_batch(kind):
    """Every token of a batch, and the same tokens in steps of their own (whose K is
    split into segments): each within its bound, so within both of one another."""
    rng, x, ids, w = case(60, 40, 2, 4, 512)
    W = make_weights(kind, 4, 512, 256, rng)
    batch = moe.ffn_decode(x, dev(ids), dev(w), W).double().cpu().numpy()
    want, tol = tolerance(x, ids, w, W)
    assert (np.abs(batch - want) <= tol).all()
    for t in (0, 17, 39):
        one = slice(t, t + 1)
        alone = moe.ffn_decode(x[one], dev(ids[one]), dev(w[one]), W).double().cpu().numpy()
        assert (np.abs(alone - want[one]) <= tol[one]).all()
        assert (np.abs(alone - batch[one]) <= 2 * tol[one]).all()


@pytest.mark.parametrize("T", [2, 40])
@pytest.mark.parametrize("kind", ["e4m3-block", "mx8", "mx4"])
def test_shards_add_up(kind, T):
    """The sum over shards that divide the experts between them is the whole."""
    rng, x, ids, w = case(T + 61, T, 3, 6, 256)
    W = make_weights(kind, 6, 256, 128, rng)
    want, _ = tolerance(x, ids, w, W)
    total, tol = np.zeros_like(want), np.zeros_like(want)
    for g0, El in ((0, 2), (2, 3), (5, 1)):
        part = lambda t, n: t[n * g0:n * (g0 + El)].contiguous()  # noqa: E731
        rows = lambda s, n: s[:, n * g0:n * (g0 + El)].contiguous() if kind[:2] == "mx" else part(s, 1)  # noqa: E731
        Ws = moe.ExpertWeights(part(W.w_in, 1), rows(W.s_in, 256), W.in_mode, part(W.w_out, 1), rows(W.s_out, 256), W.out_mode)
        y = moe.ffn_decode(x, dev(ids), dev(w), Ws, E=6, group_offset=g0)
        total += y.double().cpu().numpy()
        tol += tolerance(x, ids, w, Ws, g0)[1]
    assert moe.device_error() == 0
    assert (np.abs(total - want) <= tol).all()


@pytest.mark.parametrize("kind", KINDS)
def test_layers_one_after_the_other_on_the_same_buffers(kind):
    """A step's result, which lies in the buffers, is the next layer's input."""
    rng, x, ids, w = case(62, 12, 2, 4, 256)
    layers = [make_weights(kind, 4, 256, 384, rng, std=0.2) for _ in range(3)]
    idd, wd = dev(ids), dev(w)
    buf, y = moe.DecodeBuffers(12, 256, 4, 2, 384, "cuda"), x
    for W in layers:
        before = y.clone()
        y = moe.ffn_decode(y, idd, wd, W, buf)
        check(y, before, ids, w, W)
    assert y.data_ptr() == buf.y.data_ptr()


@pytest.mark.parametrize("kind", ["int8-channel", "e4m3-channel"])
def test_every_code(kind):
    """Weights of all int8 codes, -128 too, and of all e4m3 codes but NaN."""
    rng, x, ids, w = case(63, 7, 2, 3, 256)
    W = make_weights(kind, 3, 256, 512, rng)
    for t in (W.w_in, W.w_out):
        codes = rng.permutation(np.arange(t.numel()) % 256).astype(np.uint8)
        if kind == "e4m3-channel":
            codes[(codes & 127) == 127] = 0x76
        t.copy_(dev(codes.view(np.int8) if kind == "int8-channel" else codes).view_as(t))
    check(moe.ffn_decode(x, dev(ids), dev(w), W), x, ids, w, W)


@pytest.mark.parametrize("kind", ["mx8", "mx4"])
@pytest.mark.parametrize("far", [104, -96])
def test_far_mx_weights(kind, far):
    """wo's scales moved so that its largest magnitude lies in [2^(far - 1), 2^far],
    the choices' weights the other way."""
    rng, x, ids, w = case(64, 5, 2, 3, 256)
    W = make_weights(kind, 3, 256, 384, rng)
    top = np.abs(values(W.w_out, W.s_out, W.out_mode)).max()
    by = far - int(np.ceil(np.log2(top)))
    W.s_out.copy_((W.s_out.int() + by).to(torch.uint8))
    assert 2.0 ** (far - 1) <= np.abs(values(W.w_out, W.s_out, W.out_mode)).max() <= 2.0 ** far
    w = (w * 2.0 ** -far).astype(np.float32)
    check(moe.ffn_decode(x, dev(ids), dev(w), W), x, ids, w, W)

"""The expert FFN of a decoding step against the float64 oracle, on the values
that the weights' codes stand for.

Tolerance, derived.  Write u = 2^-24.  x is bf16 and reaches the products as
f16, exactly but for values below 2^-28 of the largest of their span, which are
off by at most 2^-39 of it; the weights' codes are exact in f16.  Each of the K
additions (and the few scalings by block) is off by at most 2 u of the mass of
its sum, m_a = sum |x||w|: d_a <= 2 K u m_a + 2^-39 max|x| sum |w|.  h =
silu(a0) a1 has |silu'| <= 1.1 and |silu(z)| <= |z|, so it is off by d_h <= 1.1
d_a0 |a1| + |silu(a0)| d_a1 + 1.1 d_a0 d_a1 + 8 u |h|, and f16 (half a step,
2^-11) holds it while it is multiplied: o = Wo h is off by at most sum |wo| (d_h
+ 2^-11 |h|) + 2 K u sum |wo||h|, y by sum_j |w| times that plus (k + 1) u of
its mass, and one rounding to bf16, 2^-8 |y|."""

import numpy as np
import pytest
import torch

import oracle
from tests.gpu_helpers import dev
from tests.mx4_helpers import bf16, sf_rows, unpack

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("fp8_quantized_moe_gb300")

KINDS = ["e4m3-channel", "e4m3-block", "e4m3-static", "int8-channel", "int8-block", "mx8", "mx4"]


def make_weights(kind, E, D, F, rng, std=0.05):
    w_in = dev(bf16(rng.standard_normal((E, 2 * F, D)).astype(np.float32) * std))
    w_out = dev(bf16(rng.standard_normal((E, D, F)).astype(np.float32) * std))
    if kind == "mx8":
        return moe.prepare_weights(w_in, w_out, moe.MX32)
    if kind == "mx4":
        return moe.prepare_weights(w_in, w_out, moe.MX4)
    if kind == "e4m3-static":
        return moe.prepare_weights(w_in, w_out, moe.PER_TENSOR, {"w0": 0.001, "w1": 0.0007, "wo": 0.0008})
    mode = moe.PER_ROW if kind.endswith("channel") else moe.PER_ROW_BLOCK128
    return (moe.prepare_weights_w8 if kind.startswith("int8") else moe.prepare_weights)(w_in, w_out, mode)


def values(q, s, mode):
    """The float64 weights [E, N, K] that codes and scales stand for."""
    q, s = q.cpu().numpy(), s.cpu().numpy()
    E, N = q.shape[:2]
    if mode in (moe.MX32, moe.MX4):
        rows = sf_rows(s).reshape(E, N, -1)
        v = oracle.E2M1[unpack(q).astype(int)] if mode == moe.MX4 else oracle.e4m3_to_f64(q)
        return v * np.repeat(oracle.e8m0_to_f64(rows), 32, -1)
    v = q.astype(np.float64) if q.dtype == np.int8 else oracle.e4m3_to_f64(q)
    s = s.astype(np.float64)
    if mode == moe.PER_ROW:
        return v * s[:, :, None]
    if mode == moe.PER_TENSOR:
        return v * s[0]
    return v * np.repeat(s.transpose(0, 2, 1), 128, -1)


def bound(x, ids, w, w_in, w_out, g0=0):
    """The tolerance of the file's head, without the last rounding."""
    T, k = ids.shape
    F, D = w_out.shape[2], w_out.shape[1]
    u, f16 = 2.0 ** -24, 2.0 ** -11
    tol = np.zeros((T, D))
    for t in range(T):
        mass = np.zeros(D)
        for j in range(k):
            e = int(ids[t, j]) - g0
            if not 0 <= e < w_in.shape[0]:
                continue
            a = w_in[e] @ x[t]
            da = 2 * len(x[t]) * u * (np.abs(w_in[e]) @ np.abs(x[t])) + 2.0 ** -39 * np.abs(x[t]).max() * np.abs(w_in[e]).sum(1)
            with np.errstate(over="ignore"):
                si = a[:F] / (1 + np.exp(-a[:F]))
            h = si * a[F:]
            dh = 1.1 * da[:F] * np.abs(a[F:]) + np.abs(si) * da[F:] + 1.1 * da[:F] * da[F:] + 8 * u * np.abs(h)
            wj = 1.0 if w is None else abs(float(w[t, j]))
            tol[t] += wj * (np.abs(w_out[e]) @ (dh + (f16 + 2 * F * u) * np.abs(h)))
            mass += wj * (np.abs(w_out[e]) @ np.abs(h))
        tol[t] += (k + 1) * u * mass
    return tol


def check(y, x, ids, w, W, g0=0):
    assert moe.device_error() == 0
    w_in, w_out = values(W.w_in, W.s_in, W.in_mode), values(W.w_out, W.s_out, W.out_mode)
    xf = x.double().cpu().numpy()
    want = oracle.ffn_decode(xf, ids, w, w_in, w_out, g0)
    got = y.double().cpu().numpy()
    tol = bound(xf, ids, w, w_in, w_out, g0) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    worst = np.max(np.abs(got - want) / np.maximum(tol, 1e-300)) if got.size else 0
    assert np.all(np.abs(got - want) <= tol), worst


def case(seed, T, k, E, D):
    rng = np.random.default_rng(seed)
    x = dev(bf16(rng.standard_normal((T, D)).astype(np.float32)))
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    return rng, x, ids, rng.random((T, k)).astype(np.float32)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,k,E,D,F", [(1, 1, 1, 128, 128), (1, 8, 16, 512, 384), (3, 2, 4, 384, 256), (9, 2, 5, 256, 640),
                                       (33, 4, 8, 256, 256), (64, 2, 3, 128, 256)])
def test_matches_the_oracle(kind, T, k, E, D, F):
    rng, x, ids, w = case(T * 100 + E, T, k, E, D)
    W = make_weights(kind, E, D, F, rng)
    check(moe.ffn_decode(x, dev(ids), dev(w), W), x, ids, w, W)


@pytest.mark.parametrize("kind", ["e4m3-channel", "e4m3-static", "int8-channel"])
@pytest.mark.parametrize("T,D,F", [(1, 16, 16), (5, 48, 1040), (20, 1040, 80), (2, 2064, 144)])
def test_sizes_that_fill_no_tile(kind, T, D, F):
    rng, x, ids, w = case(T + D, T, 2, 3, D)
    W = make_weights(kind, 3, D, F, rng)
    check(moe.ffn_decode(x, dev(ids), dev(w), W), x, ids, w, W)


@pytest.mark.parametrize("kind", ["e4m3-block", "int8-channel", "mx4"])
@pytest.mark.parametrize("T,k,E", [(8, 4, 2), (64, 4, 3), (20, 32, 40), (40, 3, 200), (64, 16, 9)])
def test_routing_that_repeats_crowds_and_scatters(kind, T, k, E):
    """The same expert twice for a token, every pair on one expert (several
    chunks of it), more than 32 pairs and more than 32 chunks."""
    rng = np.random.default_rng(T * k + E)
    D, F = 128, 256
    x = dev(bf16(rng.standard_normal((T, D)).astype(np.float32)))
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    if E == 3:
        ids[:] = 1
    w = rng.random((T, k)).astype(np.float32)
    W = make_weights(kind, E, D, F, rng)
    check(moe.ffn_decode(x, dev(ids), dev(w), W), x, ids, w, W)


@pytest.mark.parametrize("kind", ["e4m3-channel", "mx8", "mx4"])
@pytest.mark.parametrize("T,k,D,F", [(1, 1, 4096, 128), (2, 1, 128, 4096), (1, 3, 2048, 2176), (17, 2, 640, 1408)])
def test_long_contractions(kind, T, k, D, F):
    """K in several segments (one or a few pairs), an odd number of boxes, the
    ring going round."""
    rng, x, ids, w = case(D + F, T, k, 4, D)
    W = make_weights(kind, 4, D, F, rng)
    check(moe.ffn_decode(x, dev(ids), dev(w), W), x, ids, w, W)


def test_without_weights_of_the_choices():
    rng, x, ids, w = case(3, 5, 2, 4, 256)
    W = make_weights("e4m3-block", 4, 256, 128, rng)
    check(moe.ffn_decode(x, dev(ids), None, W), x, ids, None, W)


@pytest.mark.parametrize("T", [2, 40])
@pytest.mark.parametrize("kind", ["e4m3-block", "mx4"])
def test_shards(kind, T):
    """Experts of other shards add nothing; a token with none of its experts here
    gets zeros; the sum over the shards is the whole."""
    rng, x, ids, w = case(T, T, 2, 6, 256)
    ids[0] = [4, 5]
    W = make_weights(kind, 6, 256, 128, rng)
    wi, wo = values(W.w_in, W.s_in, W.in_mode), values(W.w_out, W.s_out, W.out_mode)
    for g0, El in ((0, 2), (2, 3), (0, 1)):
        part = lambda t, n: t[n * g0:n * (g0 + El)].contiguous()  # noqa: E731
        if kind == "mx4":
            sl = lambda s, n: s[:, n * g0:n * (g0 + El)].contiguous()  # noqa: E731
            Ws = moe.ExpertWeights(part(W.w_in, 1), sl(W.s_in, 256), W.in_mode, part(W.w_out, 1), sl(W.s_out, 256), W.out_mode)
        else:
            Ws = moe.ExpertWeights(part(W.w_in, 1), part(W.s_in, 1), W.in_mode, part(W.w_out, 1), part(W.s_out, 1), W.out_mode)
        y = moe.ffn_decode(x, dev(ids), dev(w), Ws, E=6, group_offset=g0)
        check(y, x, ids, w, Ws, g0)
        if g0 + El <= 4:
            assert (y[0] == 0).all()
    assert wi.shape[0] == wo.shape[0] == 6


def test_no_expert_here_at_all():
    rng, x, _, w = case(4, 7, 2, 2, 128)
    W = make_weights("int8-channel", 2, 128, 256, rng)
    buf = moe.DecodeBuffers(7, 128, 9, 2, 256, "cuda")
    buf.y.fill_(3.0)
    y = moe.ffn_decode(x, dev(np.full((7, 2), 8, np.int32)), dev(w), W, buf, E=9, group_offset=3)
    assert (y == 0).all() and moe.device_error() == 0


def test_bad_ids_add_nothing_and_are_reported():
    rng, x, ids, w = case(5, 9, 3, 4, 128)
    W = make_weights("e4m3-channel", 4, 128, 128, rng)
    bad = ids.copy()
    bad[0, 1], bad[4, 0], bad[8, 2] = -1, 4, 2147483647
    y = moe.ffn_decode(x, dev(bad), dev(w), W)
    assert moe.device_error() == 0x1
    check(y, x, bad, w, W)


@pytest.mark.parametrize("kind", KINDS)
def test_infinities_and_nan_stay_in_their_token(kind):
    rng, x, ids, w = case(6, 11, 2, 3, 256)
    W = make_weights(kind, 3, 256, 128, rng)
    clean = moe.ffn_decode(x, dev(ids), dev(w), W).clone()
    x2 = x.clone()
    x2[3, 17], x2[7, 200] = float("nan"), float("inf")
    y = moe.ffn_decode(x2, dev(ids), dev(w), W)
    assert not torch.isfinite(y[3]).any() and not torch.isfinite(y[7]).any()
    keep = [t for t in range(11) if t not in (3, 7)]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("kind", ["mx8", "mx4", "e4m3-channel"])
def test_nan_weights_reach_the_outputs_they_feed(kind):
    rng, x, ids, w = case(7, 5, 1, 3, 256)
    ids[:] = [[0], [1], [2], [1], [0]]
    W = make_weights(kind, 3, 256, 128, rng)
    clean = moe.ffn_decode(x, dev(ids), dev(w), W).clone()
    if kind == "e4m3-channel":
        W.w_out[1, 9, 100] = 0x7F
    else:
        W.s_out[0, 256 + 9, 3] = 255  # expert 1, channel 9, values 96..127
    y = moe.ffn_decode(x, dev(ids), dev(w), W)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[1, 9] = bad[3, 9] = True
    assert y[bad].isnan().all() and torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("scale", [2.0 ** -45, 2.0 ** 60])
@pytest.mark.parametrize("kind", ["e4m3-block", "mx4"])
def test_far_magnitudes(kind, scale):
    """Rows far outside f16's range, beside ordinary ones, and spans of one row
    2^20 apart: the span scales carry them."""
    rng, x, ids, w = case(8, 6, 2, 3, 512)
    x[1] *= scale
    x[4, 128:256] *= 2.0 ** -20
    W = make_weights(kind, 3, 512, 128, rng)
    check(moe.ffn_decode(x, dev(ids), dev(w), W), x, ids, w, W)


@pytest.mark.parametrize("kind", KINDS)
def test_repeats_bit_for_bit(kind):
    rng, x, ids, w = case(9, 33, 4, 8, 512)
    W = make_weights(kind, 8, 512, 256, rng)
    ids_d, w_d = dev(ids), dev(w)
    first = moe.ffn_decode(x, ids_d, w_d, W)
    buf = moe.DecodeBuffers(64, 512, 8, 4, 256, "cuda")
    for _ in range(20):
        assert torch.equal(moe.ffn_decode(x, ids_d, w_d, W, buf), first)


def test_the_batch_around_a_token_does_not_change_it():
    """A token alone and in a batch: the same sums up to the K segments that few
    pairs are split into, so within both bounds of the oracle."""
    rng, x, ids, w = case(10, 40, 2, 4, 256)
    W = make_weights("e4m3-block", 4, 256, 256, rng)
    for t in (0, 39):
        check(moe.ffn_decode(x[t:t + 1].contiguous(), dev(ids[t:t + 1]), dev(w[t:t + 1]), W), x[t:t + 1], ids[t:t + 1],
              w[t:t + 1], W)


def test_empty_and_shorter_batches():
    rng, x, ids, w = case(11, 16, 2, 4, 256)
    W = make_weights("mx8", 4, 256, 128, rng)
    buf = moe.DecodeBuffers(16, 256, 4, 2, 128, "cuda")
    assert moe.ffn_decode(x[:0], dev(ids[:0]), dev(w[:0]), W, buf).shape == (0, 256)
    moe.ffn_decode(x, dev(ids), dev(w), W, buf)
    rest = buf.y[5:].clone()
    y = moe.ffn_decode(x[:5], dev(ids[:5]), dev(w[:5]), W, buf)
    check(y, x[:5], ids[:5], w[:5], W)
    assert torch.equal(buf.y[5:], rest)  # rows behind the batch stay as they were


@pytest.mark.parametrize("kind", ["e4m3-block", "int8-channel", "mx8", "mx4"])
def test_most_pairs_and_experts(kind):
    """1024 pairs over 1024 experts: full tables, and units of a single stage."""
    rng, x, ids, w = case(40, 64, 16, 1024, 128)
    W = make_weights(kind, 1024, 128, 128, rng)
    check(moe.ffn_decode(x, dev(ids), dev(w), W), x, ids, w, W)


@pytest.mark.parametrize("kind", ["e4m3-channel", "mx8", "mx4"])
@pytest.mark.parametrize("D,F", [(1280, 640), (256, 1792)])
def test_a_hundred_calls_alike(kind, D, F):
    """Odd numbers of stages: the ring's rounds fall on every slot and group."""
    rng, x, ids, w = case(41, 16, 8, 64, D)
    W = make_weights(kind, 64, D, F, rng)
    idd, wd, buf = dev(ids), dev(w), moe.DecodeBuffers(16, D, 64, 8, F, "cuda")
    first = moe.ffn_decode(x, idd, wd, W, buf).clone()
    check(first, x, ids, w, W)
    differs = torch.zeros((), dtype=torch.bool, device="cuda")
    for _ in range(100):
        differs |= (moe.ffn_decode(x, idd, wd, W, buf) != first).any()
    assert not differs.item() and moe.device_error() == 0


def test_shapes_that_follow_on_one_workspace():
    """A model whose layers differ: the counters of one shape may not lie in
    another's sums."""
    shapes = [(7, 3, 256, 1024, "mx4"), (2, 2, 2048, 128, "e4m3-block"), (64, 4, 128, 512, "mx8"), (1, 1, 8192, 256, "int8-channel")]
    bufs = [moe.DecodeBuffers(T, D, 4, k, F, "cuda") for T, k, D, F, _ in shapes]
    ws = torch.zeros(max(b.ws_bytes for b in bufs), dtype=torch.uint8, device="cuda")
    for b in bufs:
        b.ws, b.ws_bytes = ws, ws.numel()
    for seed in (30, 31):
        for (T, k, D, F, kind), buf in zip(shapes, bufs):
            rng, x, ids, w = case(seed, T, k, 4, D)
            W = make_weights(kind, 4, D, F, rng)
            check(moe.ffn_decode(x, dev(ids), dev(w), W, buf), x, ids, w, W)


def test_captured_and_replayed():
    """Two graphs on the same buffers, replayed in turn with new inputs."""
    rng, x, ids, w = case(12, 6, 2, 4, 256)
    W = make_weights("e4m3-block", 4, 256, 128, rng)
    W4 = make_weights("mx4", 4, 256, 128, rng)
    buf = moe.DecodeBuffers(6, 256, 4, 2, 128, "cuda")
    xd, idd, wd = x.clone(), dev(ids), dev(w)
    graphs = []
    for weights in (W, W4):
        moe.ffn_decode(xd, idd, wd, weights, buf)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.ffn_decode(xd, idd, wd, weights, buf)
        graphs.append((g, weights))
    for seed in (20, 21, 22):
        _, x2, ids2, w2 = case(seed, 6, 2, 4, 256)
        xd.copy_(x2), idd.copy_(dev(ids2)), wd.copy_(dev(w2))
        for g, weights in graphs:
            g.replay()
            check(buf.y.clone(), x2, ids2, w2, weights)


def test_on_two_streams_at_once():
    rng, x, ids, w = case(13, 8, 2, 4, 1024)
    W = make_weights("e4m3-channel", 4, 1024, 1024, rng)
    idd, wd = dev(ids), dev(w)
    want = moe.ffn_decode(x, idd, wd, W).clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    bufs = [moe.DecodeBuffers(8, 1024, 4, 2, 1024, "cuda") for _ in streams]
    for _ in range(10):
        for s, b in zip(streams, bufs):
            with torch.cuda.stream(s):
                moe.ffn_decode(x, idd, wd, W, b)
    torch.cuda.synchronize()
    assert all(torch.equal(b.y, want) for b in bufs) and moe.device_error() == 0


def test_a_prompt_and_its_decoding_steps():
    """As a server uses them: weights quantised once to MXFP4, the prompt through
    ffn_forward, then steps routed by router_topk through ffn_decode."""
    rng = np.random.default_rng(14)
    T, D, E, k, F = 96, 256, 8, 2, 256
    W = make_weights("mx4", E, D, F, rng)
    gate = dev(bf16(rng.standard_normal((E, D)).astype(np.float32) * 0.1))
    x = dev(bf16(rng.standard_normal((T, D)).astype(np.float32)))
    _, ids, w = moe.router_topk(x, gate, k)
    prompt = moe.ffn_forward(x, ids, w, W, moe.MX4, moe.FFNBuffers(T, D, E, k, F, moe.MX4, "cuda"))
    assert torch.isfinite(prompt).all() and moe.device_error() == 0
    buf = moe.DecodeBuffers(4, D, E, k, F, "cuda")
    step = x[:4].contiguous()
    for _ in range(3):
        _, ids, w = moe.router_topk(step, gate, k)
        y = moe.ffn_decode(step, ids, w, W, buf)
        check(y, step, ids.cpu().numpy(), w.cpu().numpy(), W)
        step = (step + y).contiguous()

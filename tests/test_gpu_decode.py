"""The expert FFN of a decoding step against the float64 oracle, on the values
that the weights' codes stand for.

Tolerance, derived.  Write u = 2^-24.  Every activation reaches the products
as f16 within 2^-12 relative (2^-39 of its span's largest at least), so a is
off by at most (2^-12 + 2 K u) of its mass m_a = sum |x||w| (x itself is bf16
and exact unless its span covers over 2^14; the bound does not use that).  h =
silu(a0) a1 has |silu'| <= 1.1 and |silu(z)| <= |z|, so it is off by d_h <= 1.1
d_a0 |a1| + |silu(a0)| d_a1 + d_a0 d_a1 * 1.1 + 8 u |h|.  o = Wo h is off by
at most sum |wo| (d_h + 2^-12 |h|) + 2 K u sum |wo||h|, y by sum_j |w| times
that plus (k + 1) u of its mass, and one rounding to bf16, 2^-8 |y|."""

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
    u, f16 = 2.0 ** -24, 2.0 ** -12
    tol = np.zeros((T, D))
    for t in range(T):
        mass = np.zeros(D)
        for j in range(k):
            e = int(ids[t, j]) - g0
            if not 0 <= e < w_in.shape[0]:
                continue
            a = w_in[e] @ x[t]
            da = (f16 + 2 * D * u) * (np.abs(w_in[e]) @ np.abs(x[t]))
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

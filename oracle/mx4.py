"""The oracle's MXFP4 path and its decoding step, in numpy float64.

MXFP4 is the OCP "Microscaling Formats (MX) Specification" v1.0 with e2m1
elements: blocks of 32 values along the contracted dimension share the scale
2^X, X = floor(log2(amax)) - 2 (at least -127), stored as X + 127; the codes
are e2m1(x / 2^X), ties to even, at most 6 in magnitude.  A block with an
infinity or a NaN takes scale code 255 (NaN).

Layouts here are row-major: codes one a byte [rows, cols] (values 0..15),
scale codes [rows, cols/32].
"""

from __future__ import annotations

import numpy as np

# the sixteen e2m1 values by code: sign, two exponent bits (bias 1), one
# mantissa bit; exponent 0 is subnormal (0 and 0.5)
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def _bf16_to_f64(bits):
    return (np.ascontiguousarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f64_to_e2m1(v):
    """Nearest e2m1 code of each value (ties to the even code, saturating), by
    distance to the eight magnitudes."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(v), 6.0)
    d = np.abs(a[..., None] - E2M1[:8])
    best = d.min(-1, keepdims=True)
    hit = d == best  # one magnitude, or two neighbours at a tie
    low = hit.argmax(-1)
    tie = hit.sum(-1) == 2
    code = np.where(tie & (low % 2 == 1), low + 1, low)
    return (code | (np.signbit(v).astype(np.int64) << 3)).astype(np.uint8)


def e8m0_to_f64(codes):
    c = np.asarray(codes, np.int64)
    return np.where(c == 255, np.nan, np.ldexp(1.0, c - 127))


def quantize_rows_mx4(x_bits):
    """bf16 bits [rows, cols] -> (codes [rows, cols], scale codes [rows, cols/32])."""
    x = _bf16_to_f64(x_bits)
    rows, cols = x.shape
    assert cols % 32 == 0
    b = x.reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(bad, 1.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1))
    X = np.where(amax > 0, np.frexp(np.where(amax > 0, amax, 1.0))[1] - 1 - 2, -127)
    X = np.maximum(X, -127)
    q = f64_to_e2m1(np.ldexp(np.where(bad[..., None], np.copysign(0.0, b), b), -X[..., None]))
    sf = np.where(bad, 255, X + 127).astype(np.uint8)
    return q.reshape(rows, cols), sf


def quantize_weights_mx4(w_bits):
    """bf16 bits [E, N, K] -> (codes [E, N, K], scale codes [E, N, K/32])."""
    E, N, K = w_bits.shape
    q, sf = quantize_rows_mx4(np.asarray(w_bits).reshape(E * N, K))
    return q.reshape(E, N, K), sf.reshape(E, N, K // 32)


def mx4_to_f64(q, sf):
    """Values of codes [..., cols] with scale codes [..., cols/32]."""
    return E2M1[np.asarray(q, np.int64)] * np.repeat(e8m0_to_f64(sf), 32, axis=-1)


def grouped_matmul(a, w, group_sizes, group_offset=0):
    """out[m] = a[m] w[g(m) - group_offset]^T for rows of the E_local = len(w)
    local groups, zero for the others; everything float64."""
    out = np.zeros((a.shape[0], w.shape[1]))
    row = 0
    for g, n in enumerate(int(v) for v in group_sizes):
        if n and 0 <= g - group_offset < w.shape[0]:
            out[row:row + n] = a[row:row + n] @ w[g - group_offset].T
        row += n
    return out


def gmm_mx4(lhs, lhs_sf, rhs, rhs_sf, group_sizes, group_offset=0):
    """MXFP4 grouped matmul in float64 (unrounded)."""
    return grouped_matmul(mx4_to_f64(lhs, lhs_sf), mx4_to_f64(rhs, rhs_sf), group_sizes, group_offset)


def ffn_decode(x, topk_ids, topk_w, w_in, w_out, group_offset=0):
    """The expert FFN of a decoding step in float64: x [T, D], weights w_in
    [E_local, 2F, D] (wi_0 rows, then wi_1 rows) and w_out [E_local, D, F] as
    the values that their codes stand for; experts outside
    [group_offset, group_offset + E_local) add nothing."""
    T, k = topk_ids.shape
    F = w_out.shape[2]
    y = np.zeros((T, w_out.shape[1]))
    for t in range(T):
        for j in range(k):
            e = int(topk_ids[t, j]) - group_offset
            if 0 <= e < w_in.shape[0]:
                a = w_in[e] @ x[t]
                with np.errstate(over="ignore"):
                    h = a[:F] / (1.0 + np.exp(-a[:F])) * a[F:]
                y[t] += (1.0 if topk_w is None else float(topk_w[t, j])) * (w_out[e] @ h)
    return y

"""Pins of the oracle's MXFP4 path and decoding step (CPU only): blocks derived
by hand from the e2m1 and E8M0 encodings, the bracket 4 * 2^X <= amax < 8 *
2^X, the half-step error bound of the grid, equivariance under powers of two,
the MXFP8 oracle on shared values, and the reduction of the decoding step to
the grouped products it is made of."""

import numpy as np
import pytest

import oracle
from tests.mx4_helpers import bf16, pack, sf_kmajor, sf_rows, special_rows, unpack


def row(vals):
    x = np.zeros(32, np.float32)
    x[:len(vals)] = vals
    return x


# (values, scale code, element codes of the listed values)
HAND = [
    # amax 3 = 1.5 * 2^1: X = 1 - 2 = -1 (126).  x * 2: 2 -> code 4; -1 -> 8 + 2;
    # 0.5 -> 1; 6 -> 7
    ([1.0, -0.5, 0.25, 3.0], 126, [4, 10, 1, 7]),
    # amax 7.75: X = 0 (127); 7.75 and -6.5 saturate to 6
    ([7.75, -6.5, 4.0], 127, [7, 15, 6]),
    # the midpoints at X = 0 go to the even code: 0.25 -> 0, 0.75 -> 1.0 (2), 1.25 -> 1.0 (2),
    # 1.75 -> 2.0 (4), 2.5 -> 2.0 (4), 3.5 -> 4.0 (6), 5 -> 4.0 (6), -0.25 -> -0
    ([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25], 127, [6, 0, 2, 2, 4, 4, 6, 6, 8]),
    # amax 2^-126: X = -128 clamps to -127 (code 0); 2^-126 * 2^127 = 2 -> 4
    ([2.0 ** -126], 0, [4]),
    ([0.0, -0.0], 0, [0, 8]),
    # the largest bf16 (255/128 * 2^127): X = 125 (252), 7.97 saturates
    ([3.3895313892515355e38], 252, [7]),
]


@pytest.mark.parametrize("vals,code,codes", HAND)
def test_hand_derived_blocks(vals, code, codes):
    q, sf = oracle.quantize_rows_mx4(bf16(row(vals)[None]))
    assert sf[0, 0] == code and list(q[0, :len(codes)]) == codes


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_a_block_with_no_finite_maximum_is_nan(bad):
    x = np.ones((1, 64), np.float32)
    x[0, 3] = bad
    q, sf = oracle.quantize_rows_mx4(bf16(x))
    assert list(sf[0]) == [255, 125]
    v = oracle.mx4_to_f64(q, sf)
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 1).all()


def test_bracket_and_half_step():
    rng = np.random.default_rng(5)
    x = oracle.bf16_to_f64(special_rows(rng, 70, 256)).reshape(70, 8, 32)
    q, sf = oracle.quantize_rows_mx4(special_rows(np.random.default_rng(5), 70, 256))
    amax, s = np.abs(x).max(-1), oracle.e8m0_to_f64(sf)
    normal = sf > 0
    assert ((4 * s <= amax) & (amax < 8 * s))[normal].all()
    assert (amax < 8 * s)[~normal].all()
    v = oracle.mx4_to_f64(q, sf).reshape(x.shape)
    m = np.minimum(np.abs(x) / s[..., None], 6)
    step = np.where(m < 2, 0.5, np.where(m < 4, 1, 2))
    assert (np.abs(np.abs(v) / s[..., None] - m) <= step / 2).all()
    assert (np.signbit(v) == np.signbit(x)).all()


def test_powers_of_two_move_only_the_scale():
    x = np.random.default_rng(1).standard_normal((3, 64)).astype(np.float32)
    q, sf = oracle.quantize_rows_mx4(bf16(x))
    q2, sf2 = oracle.quantize_rows_mx4(bf16(x * 32))
    assert np.array_equal(q, q2) and np.array_equal(sf.astype(int) + 5, sf2)


def test_layout_moves_round_trip():
    rng = np.random.default_rng(2)
    q, sf = rng.integers(0, 16, (5, 256)).astype(np.uint8), rng.integers(0, 255, (5, 8)).astype(np.uint8)
    assert np.array_equal(unpack(pack(q)), q) and np.array_equal(sf_rows(sf_kmajor(sf)), sf)


def test_product_against_the_mxfp8_oracle():
    """e4m3 holds every e2m1 value, so the pinned MXFP8 product on the same
    values and scales is the MXFP4 product."""
    rng = np.random.default_rng(3)
    sizes = np.array([3, 0, 5], np.int32)
    a, w = rng.integers(0, 16, (8, 64)).astype(np.uint8), rng.integers(0, 16, (2, 6, 64)).astype(np.uint8)
    asf, wsf = rng.integers(120, 130, (8, 2)).astype(np.uint8), rng.integers(120, 130, (2, 6, 2)).astype(np.uint8)
    to8 = {float(v): c for c, v in reversed(list(enumerate(oracle.e4m3_table()))) if np.isfinite(v)}
    conv = np.array([to8[abs(float(v))] | (0x80 if c > 7 else 0) for c, v in enumerate(oracle.E2M1)], np.uint8)
    want = oracle.gmm_mx(conv[a], asf, conv[w], wsf, sizes, group_offset=1, E_local=2, want="f64")
    got = oracle.gmm_mx4(a, asf, w, wsf, sizes, group_offset=1)
    assert np.allclose(got, want, rtol=1e-13, atol=0)
    assert (got[:3] == 0).all()


def test_decoding_step_is_the_products_it_is_made_of():
    rng = np.random.default_rng(4)
    T, k, E, D, F = 3, 2, 4, 16, 8
    x, w_in, w_out = rng.standard_normal((T, D)), rng.standard_normal((E, 2 * F, D)), rng.standard_normal((E, D, F))
    ids = np.array([[0, 3], [3, 3], [1, 0]], np.int32)
    w = rng.random((T, k)).astype(np.float32)
    src, pos, sizes, _ = oracle.ragged_sort(ids, E)
    h = oracle.swiglu_f64(oracle.grouped_matmul(x[src // k], w_in, sizes))
    want = oracle.combine_f64(oracle.grouped_matmul(h, w_out, sizes), pos, w, k)
    assert np.allclose(oracle.ffn_decode(x, ids, w, w_in, w_out), want, rtol=1e-12)
    shards = sum(oracle.ffn_decode(x, ids, w, w_in[g:g + 2], w_out[g:g + 2], g) for g in (0, 2))
    assert np.allclose(shards, want, rtol=1e-12)

"""GPU parity of the MXFP4 variant against the oracle.

- the quantisers (rows, weights, fused into the sort, SwiGLU) and the reading
  back are bit-exact: 2^X is a power of two, so nothing rounds but the codes;
- the grouped product: every product of two e2m1 values and two powers of two
  is exact in fp32, so what is left is the fp32 accumulation of K terms and
  one rounding to bf16."""

import numpy as np
import pytest
import torch

import oracle
from tests.gpu_helpers import dev, host, ragged_sizes
from tests.mx4_helpers import bf16, pack, sf_kmajor, sf_rows, special_rows, unpack

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("fp8_quantized_moe_gb300")


@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 128), (37, 4096), (65, 7168), (9, 14336), (301, 384), (5, 32768)])
def test_quantize_rows_and_back(rows, cols):
    xb = special_rows(np.random.default_rng(rows * 7 + cols), rows, cols)
    q_ref, sf_ref = oracle.quantize_rows_mx4(xb)
    q, sf = moe.quantize_rows_mx4(dev(xb))
    assert tuple(q.shape) == (rows, cols // 2) and tuple(sf.shape) == (cols // 128, rows, 4)
    assert np.array_equal(host(q), pack(q_ref))
    assert np.array_equal(sf_rows(host(sf)), sf_ref)
    v = moe.dequantize_rows_mx4(q, sf)
    assert np.array_equal(host(v), bf16(oracle.mx4_to_f64(q_ref, sf_ref)))


def test_blocks_without_a_finite_maximum_read_back_as_nan():
    x = np.ones((4, 256), np.float32)
    x[0, 5], x[1, 40], x[3, 255] = np.inf, np.nan, -np.inf
    q_ref, sf_ref = oracle.quantize_rows_mx4(bf16(x))
    q, sf = moe.quantize_rows_mx4(dev(bf16(x)))
    assert np.array_equal(host(q), pack(q_ref)) and np.array_equal(sf_rows(host(sf)), sf_ref)
    v = moe.dequantize_rows_mx4(q, sf).float().cpu().numpy()
    bad = np.repeat(sf_ref == 255, 32, axis=1)
    assert np.isnan(v[bad]).all() and (v[~bad] == 1).all() and bad.sum() == 96


def test_reading_back_every_code_at_every_scale():
    q = np.tile(np.arange(16, dtype=np.uint8), (256, 8))  # row r: all codes in each of its blocks, scale code r
    sf = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 4, axis=1)
    v = moe.dequantize_rows_mx4(dev(pack(q)), dev(sf_kmajor(sf))).float().cpu().numpy()
    with np.errstate(over="ignore"):
        want = oracle.mx4_to_f64(q, sf)
        want32 = torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16).float().numpy()
    assert np.array_equal(v, want32, equal_nan=True)
    assert np.isnan(v[255]).all() and np.array_equal(np.signbit(v[:255]), np.signbit(want[:255]))


def test_quantize_weights_layout():
    w = bf16(np.random.default_rng(3).standard_normal((5, 48, 256)).astype(np.float32) * 0.02)
    q_ref, sf_ref = oracle.quantize_weights_mx4(w)
    q, sf = moe.quantize_weights_mx4(dev(w))
    assert tuple(q.shape) == (5, 48, 128) and tuple(sf.shape) == (2, 240, 4)
    assert np.array_equal(host(q), pack(q_ref)) and np.array_equal(sf_rows(host(sf)).reshape(5, 48, 8), sf_ref)


@pytest.mark.parametrize("T,k,E,D", [(1, 1, 1, 128), (256, 2, 4, 128), (333, 8, 64, 7168), (1023, 6, 24, 2048)])
def test_quantize_sort(T, k, E, D):
    rng = np.random.default_rng(T + k + E + D)
    xb = special_rows(rng, T, D)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    src, pos, sizes, offsets = oracle.ragged_sort(ids, E)
    xq, xsf = oracle.quantize_rows_mx4(xb)
    o = moe.quantize_sort_mx4(dev(xb), dev(ids), E)
    assert moe.device_error() == 0
    assert np.array_equal(host(o["sorted_src"]), src) and np.array_equal(host(o["pos"]), pos)
    assert np.array_equal(host(o["group_sizes"]), sizes) and np.array_equal(host(o["group_offsets"]), offsets)
    assert np.array_equal(host(o["xs_q"]), pack(xq[src // k]))
    assert np.array_equal(sf_rows(host(o["xs_scale"])), xsf[src // k])


@pytest.mark.parametrize("R,F", [(1, 128), (300, 128), (77, 2048), (16, 14336)])
def test_swiglu_quant(R, F):
    rng = np.random.default_rng(R + F)
    a = rng.standard_normal((R, 2 * F)).astype(np.float32) * 3
    a[rng.random((R, 2 * F)) < 0.05] = 0.0
    a[:, :32] *= np.float32(1e-3)
    hq_ref, hsf_ref, _ = oracle.swiglu_quant_mx4(bf16(a))
    hq, hsf = moe.swiglu_quant_mx4(dev(bf16(a)))
    assert np.array_equal(unpack(host(hq)), hq_ref) and np.array_equal(sf_rows(host(hsf)), hsf_ref)


def test_empty_rows():
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    q, sf = moe.quantize_rows_mx4(x)
    assert tuple(q.shape) == (0, 128) and tuple(moe.dequantize_rows_mx4(q, sf).shape) == (0, 256)
    o = moe.quantize_sort_mx4(x, torch.empty(0, 2, dtype=torch.int32, device="cuda"), 4)
    assert o["group_sizes"].tolist() == [0] * 4 and o["group_offsets"].tolist() == [0] * 5


# ---------------------------------------------------------------- the product

def mx4_case(seed, M, K, N, E, g0=0, El=None, zero_frac=0.25):
    rng = np.random.default_rng(seed)
    El = E - g0 if El is None else El
    sizes = ragged_sizes(rng, E, M, zero_frac)
    a, w = rng.integers(0, 16, (M, K)).astype(np.uint8), rng.integers(0, 16, (El, N, K)).astype(np.uint8)
    asf = rng.integers(118, 130, (M, K // 32)).astype(np.uint8)
    wsf = rng.integers(112, 124, (El, N, K // 32)).astype(np.uint8)
    return sizes, a, asf, w, wsf


def run_gmm(sizes, a, asf, w, wsf, g0=0):
    El, N, K = w.shape
    out = moe.gmm_mx4(dev(pack(a)), dev(sf_kmajor(asf)), dev(pack(w)), dev(sf_kmajor(wsf.reshape(El * N, K // 32))),
                      dev(sizes), group_offset=g0, E_local=El)
    assert moe.device_error() == 0
    return out


def assert_product(out, sizes, a, asf, w, wsf, g0=0):
    """|out - exact| <= half a bf16 step of the result + K fp32 additions,
    each off by at most 2^-23 of the sum of the magnitudes."""
    av, wv = oracle.mx4_to_f64(a, asf), oracle.mx4_to_f64(w, wsf)
    want = oracle.grouped_matmul(av, wv, sizes, g0)
    mass = oracle.grouped_matmul(np.abs(av), np.abs(wv), sizes, g0)
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + a.shape[1] * 2.0 ** -23 * mass * (1 + 2.0 ** -8)).all()
    rows = np.repeat(np.arange(len(sizes)), sizes)
    outside = (rows < g0) | (rows >= g0 + w.shape[0])
    assert (got[outside] == 0).all()


@pytest.mark.parametrize("M,K,N,E", [
    (1, 128, 16, 1),          # the smallest: half a stage, one row, 16 channels
    (128, 256, 256, 1),       # one tile, one stage
    (129, 384, 272, 2),       # an odd number of 128-wide K blocks, a one-row second tile, an N tail of 16
    (300, 128, 144, 4),
    (200, 512, 512, 3),
    (1000, 1024, 784, 7),
    (257, 7168, 512, 3),      # 28 stages: the ring wraps
    (64, 14336, 48, 2),
    (2048, 2048, 512, 128),   # many empty or short groups
    (700, 640, 2048, 5),
])
def test_gmm(M, K, N, E):
    c = mx4_case(M + K + N + E, M, K, N, E)
    assert_product(run_gmm(*c), *c)


@pytest.mark.parametrize("M,K,N,E,g0,El", [(300, 256, 256, 8, 2, 3), (513, 384, 144, 6, 0, 1), (77, 128, 512, 4, 3, 1),
                                          (40, 256, 256, 1024, 500, 24)])
def test_gmm_shard(M, K, N, E, g0, El):
    c = mx4_case(M + K + E, M, K, N, E, g0, El)
    assert_product(run_gmm(*c, g0=g0), *c, g0=g0)


def test_gmm_every_code_and_extreme_scales():
    """One-hot rows read single weights: every e2m1 code, at scale codes whose
    product leaves fp32's normal range on neither side."""
    K, N = 256, 256
    a = np.zeros((N, K), np.uint8)
    a[np.arange(N), np.arange(N) % K] = 2  # 1.0
    asf = np.full((N, K // 32), 127, np.uint8)
    rng = np.random.default_rng(0)
    w = rng.integers(0, 16, (1, N, K)).astype(np.uint8)
    wsf = rng.integers(10, 240, (1, N, K // 32)).astype(np.uint8)
    out = run_gmm(np.array([N], np.int32), a, asf, w, wsf).double().cpu().numpy()
    want = oracle.mx4_to_f64(w, wsf)[0].T[np.arange(N) % K]  # one product, exact in bf16
    assert np.array_equal(out, want)


def test_gmm_a_nan_scale_stays_in_its_row():
    c = mx4_case(9, 140, 256, 256, 2, zero_frac=0)
    sizes, a, asf, w, wsf = c
    clean = run_gmm(*c)
    asf2, wsf2 = asf.copy(), wsf.copy()
    asf2[7, 3] = 255
    wsf2[1, 30, 0] = 255
    out = run_gmm(sizes, a, asf2, w, wsf2)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[7] = True
    bad[int(sizes[0]):, 30] = True
    assert out[bad].isnan().all() and torch.equal(out[~bad], clean[~bad])


def test_gmm_repeats_bit_for_bit():
    c = mx4_case(11, 1500, 2048, 1024, 9)
    first = run_gmm(*c)
    for _ in range(20):
        assert torch.equal(run_gmm(*c), first)


def test_gmm_bad_group_sizes():
    sizes, a, asf, w, wsf = mx4_case(2, 64, 128, 64, 4)
    args = (dev(pack(a)), dev(sf_kmajor(asf)), dev(pack(w)), dev(sf_kmajor(wsf.reshape(-1, 4))))
    for bad in (sizes + 1, np.array([-1, 65, 0, 0], np.int32)):
        moe.gmm_mx4(*args, dev(bad.astype(np.int32)))
        assert moe.device_error() == 0x2
    out = moe.gmm_mx4(*args, dev(sizes))
    assert_product(out, sizes, a, asf, w, wsf)


# ---------------------------------------------------------------- the forward

@pytest.mark.parametrize("T,k,E,D,F", [(1, 1, 2, 128, 128), (96, 2, 4, 256, 128), (200, 4, 16, 512, 384)])
def test_forward(T, k, E, D, F):
    """Every step of ffn_forward against the oracle fed what the GPU made one
    step before, so that no rounding is counted twice."""
    rng = np.random.default_rng(T)
    w_in = bf16(rng.standard_normal((E, 2 * F, D)).astype(np.float32) * 0.05)
    w_out = bf16(rng.standard_normal((E, D, F)).astype(np.float32) * 0.05)
    xb = bf16(rng.standard_normal((T, D)).astype(np.float32))
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    W = moe.prepare_weights(dev(w_in), dev(w_out), moe.MX4)
    buf = moe.FFNBuffers(T, D, E, k, F, moe.MX4, "cuda")
    y = moe.ffn_forward(dev(xb), dev(ids), dev(w), W, moe.MX4, buf)
    assert moe.device_error() == 0
    qin, sin = oracle.quantize_weights_mx4(w_in)
    qo, so = oracle.quantize_weights_mx4(w_out)
    ref = oracle.ffn_forward_mx4(xb, ids, w, (qin, sin, qo, so), E)
    assert np.array_equal(unpack(host(buf.sort["xs_q"])), ref["xs_q"])
    assert_product(buf.a, ref["sizes"], ref["xs_q"], ref["xs_sf"], qin, sin)
    hq, hsf, _ = oracle.swiglu_quant_mx4(host(buf.a))
    assert np.array_equal(unpack(host(buf.h_q)), hq) and np.array_equal(sf_rows(host(buf.h_s)), hsf)
    assert_product(buf.o, ref["sizes"], hq, hsf, qo, so)
    want = oracle.combine(host(buf.o), ref["pos"], w, k, want="f64")
    mass = oracle.combine_f64(np.abs(buf.o.double().cpu().numpy()), ref["pos"], w, k)
    # k fp32 multiply-adds and one rounding to bf16
    assert (np.abs(y.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + (k + 1) * 2.0 ** -24 * mass).all()


def test_forward_refuses_mixed_weights():
    W = moe.prepare_weights(torch.zeros(2, 256, 128, dtype=torch.bfloat16, device="cuda"),
                            torch.zeros(2, 128, 128, dtype=torch.bfloat16, device="cuda"), moe.MX4)
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    ids, w = torch.zeros(4, 1, dtype=torch.int32, device="cuda"), torch.ones(4, 1, device="cuda")
    with pytest.raises(moe.MoEError):
        moe.ffn_forward(x, ids, w, W, moe.PER_ROW, moe.FFNBuffers(4, 128, 2, 1, 128, moe.PER_ROW, "cuda"))
    W8 = moe.ExpertWeights(W.w_in, W.s_in, moe.MX32, W.w_out, W.s_out, moe.MX32)
    with pytest.raises(moe.MoEError):
        moe.ffn_forward(x, ids, w, W8, moe.MX4, moe.FFNBuffers(4, 128, 2, 1, 128, moe.MX4, "cuda"))

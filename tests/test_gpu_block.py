"""GPU tests of the products on block-scaled 8-bit experts against 64-bit forms.

- the quantisers' codes and scales are bit-exact: every step is one fp32 rounding;
- gmm_block: products of e4m3 values are exact in fp32.  The tensor core adds 128 of
  them, each addition off by 2^-23 of the magnitudes' sum S at most (a truncated addend
  counts as a whole step), one rounding of the scale product and one a block of the
  fold: |error| <= S (128 * 2^-23 + (K/128 + 2) 2^-24), then bf16's half step 2^-8;
- tgmm_mx: the codes are exact (powers of two), so |error| <= S * rows * 2^-23, and
  fp32's half step."""

import numpy as np
import pytest
import torch

from tests import block_helpers as ref
from tests.gpu_helpers import ragged_sizes

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("fp8_quantized_moe_gb300")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand_codes(g, *shape):
    """Finite e4m3 codes of every magnitude and both signs."""
    c = torch.randint(0, 0x7F, shape, generator=g, device="cuda", dtype=torch.uint8)
    return c | (torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.uint8) << 7)


def rand_scales(g, *shape):
    return torch.exp2(torch.rand(shape, generator=g, device="cuda") * 12 - 12)


def product_case(seed, M, K, N, El):
    g = gen(seed)
    return (rand_codes(g, M, K), rand_scales(g, M, K // 128), rand_codes(g, El, N, K),
            rand_scales(g, El, -(-N // 128), K // 128))


def check_product(out, want, mag, K):
    tol = mag * (128 * 2.0 ** -23 + (K // 128 + 2) * 2.0 ** -24) + want.abs() * 2.0 ** -8
    err = (out.double() - want).abs()
    assert (err <= tol).all(), f"{(err / tol.clamp(min=1e-300)).max().item()} times the bound"
    # as a whole: bf16's rounding, uniform in half a step, is 2^-8 / sqrt(3) of a value at most
    assert err.norm() <= 2.0 ** -8 * want.norm() + 1e-30


def sizes_tensor(sizes):
    return torch.tensor([int(v) for v in sizes], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("M,K,N", [
    (1, 128, 16), (1, 2048, 1536), (2, 384, 144), (127, 256, 256), (128, 128, 128), (129, 640, 272), (257, 1024, 400),
    (300, 7168, 1296), (1000, 896, 16), (5, 14336, 272),
])
def test_dense_product(M, K, N):
    a = product_case(M + K + N, M, K, N, 1)
    out = moe.gmm_block(*a)
    assert moe.device_error() == 0
    check_product(out, *ref.gmm(*a, [M]), K)
    # the same through group sizes, and into a given output
    out2 = moe.gmm_block(*a, sizes_tensor([M]), out=torch.full_like(out, 7))
    assert torch.equal(out, out2)


@pytest.mark.parametrize("M,K,N,E,g0,El", [
    (129, 1024, 1296, 4, 0, 4), (700, 512, 528, 9, 2, 5), (2000, 256, 768, 130, 0, 130), (64, 128, 32, 1024, 0, 1024),
    (999, 1152, 4096, 16, 15, 1), (1, 256, 512, 7, 0, 7), (40, 256, 512, 7, 3, 2), (3000, 384, 176, 3, 0, 3),
])
def test_ragged_groups(M, K, N, E, g0, El):
    a = product_case(M + K + N + E, M, K, N, El)
    sizes = ragged_sizes(np.random.default_rng(M + E), E, M)
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.gmm_block(*a, sizes_tensor(sizes), group_offset=g0, out=out)
    assert moe.device_error() == 0
    check_product(out, *ref.gmm(*a, sizes.tolist(), g0), K)


def test_groups_at_tile_borders():
    sizes = [0, 128, 256, 1, 255, 0, 129, 127, 257, 0]
    M = sum(sizes)
    a = product_case(5, M, 256, 272, len(sizes))
    out = moe.gmm_block(*a, sizes_tensor(sizes))
    assert moe.device_error() == 0
    check_product(out, *ref.gmm(*a, sizes), 256)


def test_rows_without_a_group_in_this_shard_are_zero():
    a = product_case(6, 300, 256, 144, 2)
    for sizes in ([300, 0, 0, 0], [0, 0, 0, 300], [150, 0, 0, 150]):
        out = torch.full((300, 144), 3.0, dtype=torch.bfloat16, device="cuda")
        moe.gmm_block(*a, sizes_tensor(sizes), group_offset=1, out=out)
        assert moe.device_error() == 0 and not out.any()


def test_nan_codes_stay_in_their_rows_and_columns():
    lhs_q, lhs_s, rhs_q, rhs_s = product_case(7, 200, 256, 144, 2)
    lhs_q[130, 5] = 0x7F          # a NaN activation of the second group
    rhs_q[0, 100, 200] = 0xFF     # and a NaN weight of the first expert
    out = moe.gmm_block(lhs_q, lhs_s, rhs_q, rhs_s, sizes_tensor([90, 110])).float()
    nan = torch.zeros_like(out, dtype=torch.bool)
    nan[130] = True
    nan[:90, 100] = True
    assert torch.equal(out.isnan(), nan)


def test_scales_of_every_size():
    lhs_q, _, rhs_q, _ = product_case(8, 150, 512, 256, 1)
    g = gen(9)
    lhs_s = torch.exp2(torch.randint(-60, 40, (150, 4), generator=g, device="cuda").float())
    rhs_s = torch.exp2(torch.randint(-40, 40, (1, 2, 4), generator=g, device="cuda").float())
    lhs_s[3] = 0
    out = moe.gmm_block(lhs_q, lhs_s, rhs_q, rhs_s)
    check_product(out, *ref.gmm(lhs_q, lhs_s, rhs_q, rhs_s, [150]), 512)
    assert not out[3].any()


def test_group_sizes_that_do_not_add_up():
    a = product_case(10, 100, 128, 64, 2)
    for sizes in ([50, 49], [120, -20], [60, 60]):
        moe.gmm_block(*a, sizes_tensor(sizes))
        assert moe.device_error() & 0x2
    assert moe.device_error() == 0


def test_product_on_16_byte_aligned_output():
    a = product_case(11, 70, 256, 272, 1)
    buf = torch.zeros(70 * 272 + 8, dtype=torch.bfloat16, device="cuda")
    out = buf[8:].view(70, 272)
    assert out.data_ptr() % 32 == 16
    moe.gmm_block(*a, out=out)
    assert torch.equal(out, moe.gmm_block(*a)) and not buf[:8].any()


@pytest.mark.parametrize("E,N,K", [(1, 128, 128), (3, 256, 384), (2, 144, 256), (1, 16, 128), (5, 1408, 512), (2, 130, 256)])
def test_quantize_weights_block(E, N, K):
    g = gen(E * N + K)
    w = torch.randn(E, N, K, generator=g, device="cuda")
    w *= torch.exp2(torch.randint(-20, 10, (E, N, 1), generator=g, device="cuda").float())
    w[0, :128, :128] = 0
    w = w.bfloat16()
    q, s = moe.quantize_weights_block(w)
    vq, vs = ref.quantise_blocks(w)
    assert torch.equal(s.double(), vs) and torch.equal(ref.e4m3(q), vq)
    if N % 128 == 0:
        q2, s2, q_t, s_t = moe.quantize_weights_block(w, transposed=True)
        assert torch.equal(q2, q) and torch.equal(s2, s)
        assert torch.equal(q_t, q.transpose(1, 2)) and torch.equal(s_t, s.transpose(1, 2))


def test_quantize_weights_block_of_tiny_values():
    w = (torch.randn(1, 128, 128, generator=gen(1), device="cuda") * 2.0 ** -122).bfloat16()
    q, s = moe.quantize_weights_block(w)
    vq, vs = ref.quantise_blocks(w)
    assert torch.equal(s.double(), vs) and torch.equal(ref.e4m3(q), vq)


def test_input_gradient_is_the_product_on_the_transposed_weights():
    g = gen(12)
    w = (torch.randn(3, 256, 384, generator=g, device="cuda") * 0.02).bfloat16()
    q, s, q_t, s_t = moe.quantize_weights_block(w, transposed=True)
    d = torch.randn(500, 256, generator=g, device="cuda").bfloat16()
    sizes = [200, 0, 300]
    dq, ds = moe.quantize_rows(d, moe.PER_ROW_BLOCK128)
    dx = moe.gmm_block(dq, ds, q_t, s_t, sizes_tensor(sizes))
    wv, dv = ref.weight_value(q, s), ref.rows_value(dq, ds)
    want = torch.cat([dv[:200] @ wv[0], dv[200:] @ wv[2]])
    mag = torch.cat([dv[:200].abs() @ wv[0].abs(), dv[200:].abs() @ wv[2].abs()])
    check_product(dx, want, mag, 256)


# ---------------------------------------------------------------- weight gradient

def check_gradient(out, want, mag, rows):
    tol = mag * rows * 2.0 ** -23 + want.abs() * 2.0 ** -24
    err = (out.double() - want).abs()
    assert (err <= tol).all(), f"{(err / tol.clamp(min=1e-300)).max().item()} times the bound"


def gradient_case(seed, T, M, K, N):
    g = gen(seed)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    d = torch.randn(M, N, generator=g, device="cuda") * torch.exp(2 * torch.randn(M, 1, generator=g, device="cuda") - 6)
    return x, d.bfloat16()


@pytest.mark.parametrize("M,K,N,E,g0,El", [
    (1, 16, 16, 1, 0, 1), (77, 256, 400, 3, 0, 3), (128, 128, 256, 1, 0, 1), (129, 144, 272, 2, 0, 2), (700, 384, 528, 9, 2, 5),
    (1500, 64, 48, 130, 0, 130), (200, 32, 32, 1024, 0, 1024), (33, 2048, 16, 4, 1, 2), (2500, 272, 1040, 3, 0, 3),
    (0, 32, 48, 2, 0, 2),
])
def test_weight_gradient(M, K, N, E, g0, El):
    x, d = gradient_case(M + K + N, M, M, K, N)
    sizes = ragged_sizes(np.random.default_rng(M + E), E, M) if M else np.zeros(E, np.int32)
    out = torch.full((El, K, N), float("nan"), device="cuda")
    moe.tgmm_mx(x, d, sizes_tensor(sizes), group_offset=g0, E_local=El, out=out)
    assert moe.device_error() == 0
    check_gradient(out, *ref.tgmm(x, d, sizes.tolist(), g0, El), max(1, int(sizes.max())))


def test_weight_gradient_of_groups_at_block_borders():
    sizes = [0, 31, 32, 33, 128, 0, 1, 127, 129, 96, 256, 0]
    x, d = gradient_case(3, sum(sizes), sum(sizes), 80, 304)
    out = moe.tgmm_mx(x, d, sizes_tensor(sizes))
    assert moe.device_error() == 0
    check_gradient(out, *ref.tgmm(x, d, sizes, 0, len(sizes)), 256)


def test_weight_gradient_with_picked_rows():
    T, k, E = 150, 3, 5
    g = gen(4)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    src = torch.argsort(ids.flatten(), stable=True).to(torch.int32)
    sizes = torch.bincount(ids.flatten(), minlength=E).to(torch.int32)
    x, d = gradient_case(5, T, T * k, 128, 272)
    out = moe.tgmm_mx(x, d, sizes, lhs_rows=src, k=k)
    picked = x[src.long() // k].contiguous()
    assert moe.device_error() == 0
    assert torch.equal(out, moe.tgmm_mx(picked, d, sizes))
    check_gradient(out, *ref.tgmm(picked, d, sizes.tolist(), 0, E), T)


def test_weight_gradient_picked_row_out_of_range_is_zero():
    x, d = gradient_case(6, 40, 90, 32, 48)
    rows = torch.arange(90, device="cuda", dtype=torch.int32) % 40
    for bad in (40, -1, 2 ** 31 - 1, -2 ** 31):
        rows[17] = bad
        out = moe.tgmm_mx(x, d, sizes_tensor([50, 40]), lhs_rows=rows)
        assert moe.device_error() == 0x10
        picked = x[(torch.arange(90, device="cuda") % 40)].clone()
        picked[17] = 0
        check_gradient(out, *ref.tgmm(picked, d, [50, 40], 0, 2), 50)


def test_rounding_is_exact():
    """One-hot lhs rows read the rounded rhs back: 1 is a code, so every entry is r(rhs)."""
    n = 128
    x = torch.eye(n, device="cuda").bfloat16()
    g = gen(7)
    d = torch.randn(n, 512, generator=g, device="cuda") * torch.exp2(torch.randint(-90, 60, (1, 512), generator=g, device="cuda").float())
    d[:, :64] *= torch.exp2(torch.randint(-12, 1, (n, 64), generator=g, device="cuda").float())  # subnormal codes
    d[32:64, 100:110] = 0
    d[5, 200], d[6, 200], d[40, 201] = 448.0, 450.0, 449.0  # the border of a scale
    d = d.bfloat16()
    out = moe.tgmm_mx(x, d, sizes_tensor([n]))
    assert moe.device_error() == 0
    assert torch.equal(out[0].double(), ref.round_rows(d))
    # the other operand's side
    out = moe.tgmm_mx(d, x, sizes_tensor([n]))
    assert torch.equal(out[0].t().double(), ref.round_rows(d))


def test_infinity_and_nan_in_a_gradient():
    x = torch.eye(64, device="cuda").bfloat16()
    d = torch.ones(64, 48, device="cuda").bfloat16()
    d[3, 5], d[40, 7] = float("inf"), float("nan")
    out = moe.tgmm_mx(x, d, sizes_tensor([64]))[0]
    # the infinity's code stands for 448 * 2^120, above fp32's range; beside it 1 rounds to zero
    assert out[3, 5] == float("inf") and out[:, 5].isfinite().sum() == 63
    assert not out[:3, 5].any() and (out[32:, 5] == 1).all()
    # every product of column 7 with the second block's NaN is NaN, through rows that are zero there as well
    assert out[:, 7].isnan().all()
    rest = torch.ones(48, dtype=torch.bool, device="cuda")
    rest[5] = rest[7] = False
    assert torch.equal(out[:, rest], torch.ones(64, 46, device="cuda"))
    assert (out[4:32, 5] == 0).all()


def test_weight_gradient_group_sizes_that_do_not_add_up():
    x, d = gradient_case(8, 100, 100, 32, 32)
    for sizes in ([50, 49], [120, -20], [60, 60]):
        moe.tgmm_mx(x, d, sizes_tensor(sizes))
        assert moe.device_error() & 0x2
    assert moe.device_error() == 0


def test_weight_gradient_against_differences():
    """d/dW of sum(D * (X W)) along a direction, X and D being e4m3 values: exact operands."""
    g = gen(9)
    x = torch.randint(-8, 9, (96, 32), generator=g, device="cuda").float()
    d = torch.randint(-8, 9, (96, 48), generator=g, device="cuda").float()
    w = torch.randn(32, 48, generator=g, device="cuda").double()
    v = torch.randn(32, 48, generator=g, device="cuda").double()
    out = moe.tgmm_mx(x.bfloat16(), d.bfloat16(), sizes_tensor([96]))[0].double()
    f = lambda w: (d.double() * (x.double() @ w)).sum()  # noqa: E731
    slope = (f(w + v) - f(w - v)) / 2
    # sums of 96 integers below 64 are exact in fp32
    assert abs((out * v).sum() - slope) <= 1e-9 * (out * v).abs().sum()


# ---------------------------------------------------------------- graphs, streams, both at once

def test_captured_and_replayed():
    a = product_case(20, 300, 256, 272, 3)
    sizes = sizes_tensor([100, 0, 200])
    x, d = gradient_case(21, 300, 300, 64, 272)
    ws = torch.empty(moe.tgmm_mx_workspace_bytes(300, 64, 272, 3), dtype=torch.uint8, device="cuda")
    y, dw = moe.gmm_block(*a, sizes), moe.tgmm_mx(x, d, sizes, workspace=ws)
    y0, dw0 = torch.zeros_like(y), torch.zeros_like(dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.gmm_block(*a, sizes, out=y0)
        moe.tgmm_mx(x, d, sizes, out=dw0, workspace=ws)
    for new in ([100, 0, 200], [0, 300, 0], [1, 298, 1]):
        sizes.copy_(sizes_tensor(new))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y0, moe.gmm_block(*a, sizes)) and torch.equal(dw0, moe.tgmm_mx(x, d, sizes))
    assert moe.device_error() == 0


def test_on_two_streams_at_once():
    a, b = product_case(22, 900, 512, 528, 2), product_case(23, 700, 1024, 272, 2)
    x, d = gradient_case(24, 700, 700, 256, 272)
    sa, sb = sizes_tensor([400, 500]), sizes_tensor([699, 1])
    want = moe.gmm_block(*a, sa), moe.gmm_block(*b, sb), moe.tgmm_mx(x, d, sb)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            y1 = moe.gmm_block(*a, sa)
        with torch.cuda.stream(s2):
            y2 = moe.gmm_block(*b, sb)
            w2 = moe.tgmm_mx(x, d, sb)
        torch.cuda.synchronize()
        assert torch.equal(y1, want[0]) and torch.equal(y2, want[1]) and torch.equal(w2, want[2])
    assert moe.device_error() == 0


@pytest.mark.parametrize("M,K,N,E", [
    (300, 256, 272, 1),     # the producer has issued all it has and is done
    (4096, 512, 1024, 8),   # several tiles a CTA: every role waits
    (1, 4096, 512, 1),      # a tile shared by eight CTAs
    (65, 2048, 48, 1),      # by two, an N tail
])
def test_a_wait_that_runs_out_is_reported(M, K, N, E):
    a = product_case(25, M, K, N, E)
    x, d = gradient_case(26, M, M, K, N)
    sizes = sizes_tensor(ragged_sizes(np.random.default_rng(M), E, M))
    y, dw = moe.gmm_block(*a, sizes), moe.tgmm_mx(x, d, sizes)
    assert moe.device_error() == 0
    for call in (lambda: moe.gmm_block(*a, sizes), lambda: moe.tgmm_mx(x, d, sizes)):
        moe.lib().moe_test_stall_consumers(200_000)
        try:
            call()
            assert moe.device_error() == 0x4
        finally:
            moe.lib().moe_test_stall_consumers(0)
    assert torch.equal(moe.gmm_block(*a, sizes), y) and torch.equal(moe.tgmm_mx(x, d, sizes), dw)
    assert moe.device_error() == 0


@pytest.mark.parametrize("M", [1, 3, 40, 64, 100, 128, 129])
@pytest.mark.parametrize("K", [1024, 2048, 4096, 7168])
def test_tiles_shared_by_several_ctas(M, K):
    """Few tiles and many K blocks: one, two, four and eight CTAs a tile."""
    a = product_case(M + K, M, K, 528, 1)
    check_product(moe.gmm_block(*a), *ref.gmm(*a, [M]), K)
    assert moe.device_error() == 0
    a = product_case(M + K + 1, M, K, 272, 2)
    for sizes in ([M, 0], [0, M], [M // 2, M - M // 2]):
        out = moe.gmm_block(*a, sizes_tensor(sizes))
        check_product(out, *ref.gmm(*a, sizes), K)
    # and as the only local one of three groups, the others' rows zeroed
    a = product_case(M + K + 2, M + 50, K, 144, 1)
    out = torch.full((M + 50, 144), 5.0, dtype=torch.bfloat16, device="cuda")
    moe.gmm_block(*a, sizes_tensor([20, M, 30]), group_offset=1, out=out)
    check_product(out, *ref.gmm(*a, [20, M, 30], 1), K)
    # or with no row at all
    out.fill_(5)
    moe.gmm_block(*a, sizes_tensor([M + 20, 0, 30]), group_offset=1, out=out)
    assert not out.any() and moe.device_error() == 0


def test_shared_tiles_with_sizes_that_do_not_add_up():
    a = product_case(40, 8, 7168, 272, 2)
    for sizes in ([4, 3], [9, -1], [8, 1]):
        moe.gmm_block(*a, sizes_tensor(sizes))
        assert moe.device_error() & 0x2
    assert moe.device_error() == 0


def test_two_graphs_at_once():
    """Two captured steps with workspaces of their own, replayed on two streams."""
    cases = [gradient_case(41 + i, 500, 500, 128, 272) for i in range(2)]
    sizes = [sizes_tensor([300, 0, 200]), sizes_tensor([0, 499, 1])]
    want = [moe.tgmm_mx(x, d, s) for (x, d), s in zip(cases, sizes)]
    graphs, outs = [], []
    for (x, d), s in zip(cases, sizes):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(moe.tgmm_mx(x, d, s))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want)) and moe.device_error() == 0


def test_offsets_past_32_bits():
    # 2.4e9 outputs and 2.2e9 lhs codes of a product
    M, K, N = 300_000, 7296, 8192
    g = gen(30)
    a = torch.randint(0, 0x70, (M, K), generator=g, device="cuda", dtype=torch.uint8)
    sa = rand_scales(g, M, K // 128)
    w, sw = rand_codes(g, 1, N, K), rand_scales(g, 1, N // 128, K // 128)
    out = moe.gmm_block(a, sa, w, sw)
    rows = torch.tensor([0, 131_071, 262_143, 262_144, 294_000, 299_999], device="cuda")
    check_product(out[rows], *ref.gmm(a[rows].contiguous(), sa[rows].contiguous(), w, sw, [len(rows)]), K)
    del a, out
    # 2.3e9 gradients, and 2.6e9 weight codes
    El, K, N = 9, 16384, 15680
    x, d = gradient_case(31, 70, 70, K, N)
    out = moe.tgmm_mx(x, d, sizes_tensor([5, 0, 30, 0, 0, 0, 0, 0, 35]))
    assert moe.device_error() == 0
    last = ref.round_rows(x[35:]).t()[-200:] @ ref.round_rows(d[35:])
    assert ((out[8, -200:].double() - last).abs() <= 1e-5 * last.abs() + 1e-5 * last.abs().amax()).all()
    assert not out[1].any() and not out[7].any()
    del out
    E, N, K = 10, 16000, 16384
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    w[9, 15872:] = torch.randn(128, K, generator=g, device="cuda").bfloat16()
    q, s, q_t, s_t = moe.quantize_weights_block(w, transposed=True)
    vq, vs = ref.quantise_blocks(w[9:, 15872:].contiguous())
    assert torch.equal(ref.e4m3(q[9, 15872:])[None], vq) and torch.equal(s[9, 124:].double()[None], vs)
    assert torch.equal(q_t[9, :, 15872:], q[9, 15872:].t()) and torch.equal(s_t[9, :, 124], s[9, 124])

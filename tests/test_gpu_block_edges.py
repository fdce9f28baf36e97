"""GPU tests of calls next to the ordinary ones: products repeat their bits over many K blocks and
calls in flight, gradients do not depend on what their workspace held, on the output's
alignment or on whether an infinity was there when a graph was captured, and one expert may
hold all rows.  Tolerances are those of test_gpu_block."""

import pytest
import torch

from tests import block_helpers as ref
from tests.test_gpu_block import check_gradient, check_product, gen, product_case, sizes_tensor

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("fp8_quantized_moe_gb300")


@pytest.mark.parametrize("M,K,N,sizes", [(300, 28672, 528, [100, 0, 200]), (40, 14336, 272, [40])])
def test_a_long_product_repeats_its_bits(M, K, N, sizes):
    a = product_case(M + K, M, K, N, len(sizes))
    s = sizes_tensor(sizes)
    first = moe.gmm_block(*a, s)
    want, mag = ref.gmm(*a, sizes)
    check_product(first, want, mag, K)
    # bf16's nearest to 64 bits but where fp32's error, mag (128 * 2^-23 + (K/128 + 2) 2^-24) at the most,
    # reaches over a border between two: that error counted twice in a step of 2^-7 of the value
    tol = mag * (128 * 2.0 ** -23 + (K // 128 + 2) * 2.0 ** -24)
    near = (2 * tol / (want.abs() * 2.0 ** -8).clamp(min=1e-300)).clamp(max=1).mean()
    assert (first != want.float().bfloat16()).double().mean() <= near
    outs = [moe.gmm_block(*a, s) for _ in range(20)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        outs += [moe.gmm_block(*a, s) for _ in range(20)]
    outs += [moe.gmm_block(*a, s) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)
    assert moe.device_error() == 0


def gradient_operands(seed, M, K, N):
    g = gen(seed)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    return x, (1e-3 * torch.randn(M, N, generator=g, device="cuda")).bfloat16()


@pytest.mark.parametrize("M,K,N,sizes", [(77, 48, 80, [30, 0, 47]), (900, 400, 528, [33, 500, 367])])
def test_gradients_whatever_the_workspace_held(M, K, N, sizes):
    x, d = gradient_operands(M, M, K, N)
    n, s = moe.tgmm_mx_workspace_bytes(M, K, N, len(sizes)), sizes_tensor(sizes)
    outs = []
    for fill in (0, 1, 0x7F, 0xFD, 0xFF):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        outs.append(moe.tgmm_mx(x, d, s, workspace=ws))
        d2 = d.clone()
        d2[M // 2, 3] = float("inf")  # a call that leaves its mark in the workspace
        moe.tgmm_mx(x, d2, s, workspace=ws)
        outs.append(moe.tgmm_mx(x, d, s, workspace=ws))
    assert moe.device_error() == 0 and outs[0].isfinite().all()
    assert all(torch.equal(outs[0], o) for o in outs)


def test_gradients_into_16_byte_aligned_outputs():
    M, K, N = 200, 272, 400
    x, d = gradient_operands(4, M, K, N)
    d[7, 9] = float("inf")
    s = sizes_tensor([120, 80])
    want = moe.tgmm_mx(x, d, s)
    room = torch.full((2 * K * N + 12,), 7.0, device="cuda")
    out = room[4:4 + 2 * K * N].view(2, K, N)
    assert out.data_ptr() % 32 == 16
    moe.tgmm_mx(x, d, s, out=out)
    assert moe.device_error() == 0 and torch.equal(out.nan_to_num(3.0), want.nan_to_num(3.0))
    assert (room[:4] == 7).all() and (room[4 + 2 * K * N:] == 7).all()


def test_an_infinity_that_appears_after_the_capture():
    M, K, N = 300, 128, 272
    x, d = gradient_operands(5, M, K, N)
    s = sizes_tensor([100, 200])
    ws = torch.empty(moe.tgmm_mx_workspace_bytes(M, K, N, 2), dtype=torch.uint8, device="cuda")
    plain = moe.tgmm_mx(x, d, s, workspace=ws).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.tgmm_mx(x, d, s, workspace=ws)
    keep = d.clone()
    for bad in (False, True, False):
        d.copy_(keep)
        if bad:
            d[150, 11] = -float("inf")
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], plain[0])
        if bad:
            col = torch.where(x[150] == 0, 0.0, -x[150].float().sign() * float("inf"))
            m = x[150] != 0
            assert torch.equal(out[1, m, 11], col[m]) and torch.equal(out[1, :, 12:], plain[1, :, 12:])
        else:
            assert torch.equal(out, plain)
    assert moe.device_error() == 0


def test_all_rows_in_one_expert():
    M, K, N = 16384, 144, 272
    x, d = gradient_operands(6, M, K, N)
    sizes = [0, M, 0]
    out = moe.tgmm_mx(x, d, sizes_tensor(sizes))
    assert moe.device_error() == 0
    want, mag = ref.tgmm(x, d, sizes, 0, 3)
    check_gradient(out, want, mag, M)
    # as a whole: 512 additions of 32 products to one fp32 accumulator, each off by 2^-23 of it at the
    # most, and its size grows to the sum's own
    assert (out.double() - want).norm() <= (M / 32 + 32) * 2.0 ** -23 * want.norm()


def test_products_of_scales_below_the_normal_numbers():
    """The scales' product is an fp32 number: below 2^-126 it is off by 2^-150 at the most, a block of 128
    products by 128 * 448^2 * 2^-150 < 2^-125."""
    M, K, N = 130, 640, 272
    lhs_q, lhs_s, rhs_q, rhs_s = product_case(9, M, K, N, 1)
    for up in (-100, -110, -118, -126):
        a = (lhs_q, lhs_s * 2.0 ** up, rhs_q, rhs_s * 2.0 ** -20)
        out = moe.gmm_block(*a)
        want, mag = ref.gmm(*a, [M])
        tol = mag * (128 * 2.0 ** -23 + (K // 128 + 2) * 2.0 ** -24) + want.abs() * 2.0 ** -8
        # (and bf16's own half step below its normal numbers, 2^-134)
        assert ((out.double() - want).abs() <= tol + K // 128 * 2.0 ** -125 + 2.0 ** -134).all()
    assert moe.device_error() == 0

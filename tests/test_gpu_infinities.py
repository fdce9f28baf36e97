"""GPU tests of infinities in the operands of tgmm_mx: a sum that an infinity enters with a
value other than zero is that infinity, however small the value (a row's code may round to
zero beside larger ones), and NaN where both signs meet.  Columns without one keep their bits."""

import pytest
import torch

from tests import block_helpers as ref
from tests.test_gpu_block import gen, sizes_tensor
from tests.test_gpu_block_ffn import layer

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("fp8_quantized_moe_gb300")

INF = float("inf")


def operands(seed, M, K, N):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    return r(M, K), r(M, N)


@pytest.mark.parametrize("v", [0.1, -3.0, 2.0 ** -20, -2.0 ** -100, 2.0 ** -133])
@pytest.mark.parametrize("side,row", [("rhs", 45), ("lhs", 45), ("rhs", 129), ("lhs", 0)])
def test_an_infinity_never_comes_out_finite(side, row, v):
    x, d = operands(3, 130, 80, 272)
    (x if side == "rhs" else d)[row] = v
    sizes = sizes_tensor([70, 60])
    plain = moe.tgmm_mx(x, d, sizes)
    (d if side == "rhs" else x)[row, 37] = INF
    out = moe.tgmm_mx(x, d, sizes)
    assert moe.device_error() == 0
    e = int(row >= 70)
    hit = torch.zeros_like(out, dtype=torch.bool)
    if side == "rhs":
        hit[e, :, 37] = True
    else:
        hit[e, 37] = True
    assert (out[hit] == (INF if v > 0 else -INF)).all()
    assert torch.equal(out[~hit], plain[~hit])


def hits(x, d, rows):
    """Sums of the products of these rows that an infinity enters with a value other than zero (else 0)."""
    out = torch.zeros(x.shape[1], d.shape[1], dtype=torch.float64, device="cuda")
    for m in rows:
        p = x[m].double().unsqueeze(1) * d[m].double()
        zero = (x[m] == 0).unsqueeze(1) | (d[m] == 0)
        out += torch.where(p.isfinite() | zero, 0.0, p)
    return out


@pytest.mark.parametrize("M,K,N,sizes,g0,El,picked", [
    (64, 16, 16, [64], 0, 1, False), (1000, 400, 528, [3, 0, 600, 397], 0, 4, False),
    (1000, 400, 528, [3, 0, 600, 397], 2, 1, False), (600, 272, 304, [1, 299, 0, 300], 1, 3, True),
    (5000, 1040, 784, [2000, 3000], 0, 2, True),
])
def test_infinities_among_zeros_and_both_signs(M, K, N, sizes, g0, El, picked):
    g = gen(M + K)
    x, d = operands(M + N, M // 2 if picked else M, K, N)[0], operands(M + N, M, K, N)[1]
    x[torch.rand(x.shape, generator=g, device="cuda") < 0.2] = 0
    d[torch.rand(d.shape, generator=g, device="cuda") < 0.2] = 0
    for t in (x, d):
        n = max(2, t.shape[0] // 100)
        r = torch.randint(0, t.shape[0], (n,), generator=g, device="cuda")
        c = torch.randint(0, t.shape[1], (n,), generator=g, device="cuda")
        t[r, c] = torch.where(torch.rand(n, generator=g, device="cuda") < 0.5, INF, -INF).bfloat16()
    src = torch.randint(0, M, (M,), generator=g, device="cuda", dtype=torch.int32) if picked else None
    args = (sizes_tensor(sizes), g0, El) + ((src, 2) if picked else ())
    out = moe.tgmm_mx(x, d, *args)
    assert moe.device_error() == 0
    xs = x[src.long() // 2] if picked else x
    bad = xs.isinf().any(1) | d.isinf().any(1)
    some = False
    for e, r, n in ref.groups(sizes, g0, El):
        want = hits(xs, d, (torch.nonzero(bad[r:r + n]).flatten() + r).tolist())
        m = want != 0  # (NaN too)
        some = some or bool(m.any())
        assert torch.equal(out[e][m].isnan(), want[m].isnan())
        k = m & ~want.isnan()
        assert torch.equal(out[e][k].double(), want[k])
        # columns and rows without an infinity: as without any
        a, b = xs[r:r + n].isinf().any(0), d[r:r + n].isinf().any(0)
        free = ~(a.unsqueeze(1) | b)
        got, mag = (t[0] for t in ref.tgmm(torch.where(xs[r:r + n].isinf(), 0, xs[r:r + n]),
                                           torch.where(d[r:r + n].isinf(), 0, d[r:r + n]), [n], 0, 1))
        tol = mag * n * 2.0 ** -23 + got.abs() * 2.0 ** -24  # as check_gradient's
        assert ((out[e].double() - got).abs() <= tol)[free].all()
        assert out[e][~m].isfinite().all()
    assert some
    assert torch.equal(out.nan_to_num(7.0), moe.tgmm_mx(x, d, *args).nan_to_num(7.0))


def test_nothing_but_infinities():
    """A step whose gradient has overflowed everywhere."""
    x, d = operands(12, 3000, 528, 784)
    x[:, ::5] = 0
    d[:] = torch.where(d > 0, INF, -INF)
    d[:, 3] = INF
    x[:, 7] = x[:, 7].abs() + 1
    out = moe.tgmm_mx(x, d, sizes_tensor([1000, 0, 2000]))
    assert moe.device_error() == 0
    assert not out[1].any()
    for e, r, n in ((0, 0, 1000), (2, 1000, 2000)):
        assert out[e][7, 3] == INF and not out[e][::5].any()
        rest = torch.ones(528, dtype=torch.bool, device="cuda")
        rest[::5] = False
        assert not out[e][rest].isfinite().any()
        assert out[e][rest].isnan().float().mean() > 0.99  # both signs meet nearly everywhere


def test_infinities_of_other_shards_do_nothing():
    x, d = operands(9, 300, 64, 64)
    sizes = sizes_tensor([100, 100, 100])
    plain = moe.tgmm_mx(x, d, sizes, 1, 1)
    d[:100, 3] = INF
    x[200:, 5] = -INF
    assert torch.equal(moe.tgmm_mx(x, d, sizes, 1, 1), plain)


def test_an_infinity_in_the_output_gradient_reaches_the_weight_gradients():
    T, D, E, k, F = 200, 256, 8, 2, 128
    x, dY, w_in, w_out, w_gate = layer(11, T, D, E, k, F)
    W = moe.prepare_weights(w_in, w_out, moe.PER_BLOCK128, for_backward=True)
    buf = moe.FFNBuffers(T, D, E, k, F, moe.PER_ROW_BLOCK128, "cuda", backward=True)
    _, ids, w = moe.router_topk(x, w_gate, k)
    moe.ffn_forward(x, ids, w, W, moe.PER_ROW_BLOCK128, buf)
    dY[5, 7] = INF
    keep = {}
    _, dW_in, dW_out = moe.ffn_backward(dY, w, W, buf, x=x, keep=keep)
    assert moe.device_error() == 0
    rows = [int(torch.nonzero(buf.sort["sorted_src"] == 5 * k + j)) for j in range(k)]
    for j, e in enumerate(ids[5].tolist()):
        assert not dW_out[e, :, 7][keep["h"][rows[j]] != 0].isfinite().any()
        assert not dW_in[e].isfinite().any()  # dH's row is NaN

"""GPU tests of the router's balance loss and its gradient against 64-bit forms.

Counts are exact.  With R the logits' range in a row, e^(x - max) is off by R + 5 half
steps of fp32 relative (the subtraction; the exponential's 2^-22 and a rounding), their sum
by E more, the reciprocal and the product by 2: a probability by u = (2 R + E + 8) 2^-24 at the most, a mean over n
rows by u + n 2^-24 (sums in order, at the worst), the loss likewise."""

import pytest
import torch

from tests import block_helpers as ref

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("fp8_quantized_moe_gb300")


def case(seed, T, E, k, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = spread * torch.randn(T, E, generator=g, device="cuda")
    ids = torch.topk(logits, min(k, E), -1)[1].to(torch.int32)
    if k > E:
        ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    return logits, ids.contiguous()


def check(logits, ids, coef=0.01, seqs=1, valid=None, grad=3.0):
    T, E = logits.shape
    b = moe.router_balance_loss(logits, ids, coef, seqs=seqs, valid=valid)
    d = moe.router_balance_loss_backward(logits, b, torch.tensor([grad], device="cuda"))
    loss, counts, mean, tokens, dl = ref.balance(logits.cpu(), ids.cpu(), coef, seqs, None if valid is None else valid.cpu(), grad)
    finite = logits[torch.isfinite(logits)]
    R = float(finite.max() - finite.min()) if finite.numel() else 0.0
    u = (2 * R + E + 8) * 2.0 ** -24
    n = max(1, T // seqs)
    assert torch.equal(b.counts.cpu().long(), counts) and torch.equal(b.tokens.cpu().long(), tokens)
    tiny = 2.0 ** -120
    assert ((b.mean.cpu().double() - mean).abs() <= (u + n * 2.0 ** -24) * mean + tiny).all()
    assert abs(float(b.loss) - loss) <= (u + (n + E + seqs + 8) * 2.0 ** -24) * abs(loss) + tiny
    # p (c - c* - sum p (c - c*)): p's error, and that of the difference, E + 4 roundings and E errors u of
    # numbers up to C, the largest difference of two c
    f = counts.double() * E / (ids.shape[1] * tokens.clamp(min=1).double().unsqueeze(1))
    c = (grad * coef / seqs / tokens.clamp(min=1).double().unsqueeze(1) * f).repeat_interleave(T // seqs, 0)
    C = c.amax(1, keepdim=True) - c.amin(1, keepdim=True)
    x = logits.cpu().double()
    p = torch.nan_to_num(torch.softmax(x, 1))
    tol = p * C * (2 * u + (E + 12) * 2.0 ** -24) + dl.abs() * (u + 8 * 2.0 ** -24) + tiny
    err = (d.cpu().double() - dl).abs()
    if valid is not None:
        assert not d[~valid].any()
        err, tol = err[valid.cpu()], tol[valid.cpu()]
    assert (err <= tol).all(), float((err / tol).max())
    return b, d


@pytest.mark.parametrize("T,E,k,seqs", [
    (1, 1, 1, 1), (1, 8, 2, 1), (24, 128, 8, 1), (64, 4, 2, 1), (65, 256, 8, 1), (1000, 64, 6, 4), (4096, 256, 8, 2),
    (777, 13, 3, 7), (513, 130, 5, 1), (300, 512, 8, 3), (130, 1024, 32, 2), (90, 1023, 1, 1), (2000, 33, 33 - 1, 1000),
    (20000, 16, 2, 1), (700, 2, 5, 700),
])
def test_loss_and_gradient(T, E, k, seqs):
    logits, ids = case(T + E + k, T, E, k)
    check(logits, ids, seqs=seqs)
    assert moe.device_error() == 0


@pytest.mark.parametrize("E", [31, 65, 95, 96, 97, 129, 191, 192, 193, 257, 320, 384, 385, 513, 701, 768, 769, 1024])
def test_every_width_at_its_edges(E):
    for T, seqs in ((6, 2), (3 * 701, 3)):
        logits, ids = case(E, T, E, 4)
        valid = torch.arange(T, device="cuda") % 5 != 2
        check(logits, ids, seqs=seqs)
        check(logits, ids, seqs=seqs, valid=valid)
    assert moe.device_error() == 0


def test_padded_rows_count_nowhere_whatever_they_hold():
    S, L, E = 5, 70, 40
    logits, ids = case(1, S * L, E, 4)
    length = torch.tensor([70, 0, 1, 33, 69], device="cuda")  # a whole one, an empty one, a single row
    valid = (torch.arange(L, device="cuda") < length.unsqueeze(1)).flatten()
    b, d = check(logits, ids, seqs=S, valid=valid)
    logits2, ids2 = logits.clone(), ids.clone()
    logits2[~valid] = float("nan")
    ids2[~valid] = -1
    b2 = moe.router_balance_loss(logits2, ids2, 0.01, seqs=S, valid=valid)
    d2 = moe.router_balance_loss_backward(logits2, b2, torch.tensor([3.0], device="cuda"))
    assert moe.device_error() == 0
    assert torch.equal(b.loss, b2.loss) and torch.equal(b.counts, b2.counts) and torch.equal(b.mean, b2.mean)
    assert torch.equal(d, d2) and b2.tokens.tolist() == length.tolist()


def test_no_valid_row_at_all():
    logits, ids = case(2, 12, 8, 2)
    valid = torch.zeros(12, dtype=torch.bool, device="cuda")
    for seqs in (1, 3):
        b = moe.router_balance_loss(logits, ids, 1.0, seqs=seqs, valid=valid)
        d = moe.router_balance_loss_backward(logits, b)
        assert float(b.loss) == 0 and not b.counts.any() and not b.mean.any() and not d.any()


def test_no_rows():
    logits, ids = torch.zeros(0, 8, device="cuda"), torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    b = moe.router_balance_loss(logits, ids, 1.0, seqs=3)
    assert float(b.loss) == 0 and not b.counts.any() and not b.mean.any() and not b.tokens.any()
    assert moe.router_balance_loss_backward(logits, b).shape == (0, 8)


def test_closed_experts_and_rows_of_minus_infinity():
    logits, ids = case(3, 300, 96, 4)
    logits[:, 7] = logits[:, 90] = -torch.inf
    logits[20:40, 50:] = torch.finfo(torch.float32).min
    logits[100] = -torch.inf
    b = moe.router_balance_loss(logits, ids, 0.5)
    d = moe.router_balance_loss_backward(logits, b)
    loss, counts, mean, _, dl = ref.balance(logits.cpu(), ids.cpu(), 0.5, 1, None)
    assert torch.equal(b.counts.cpu()[0].long(), counts[0])
    assert torch.allclose(b.mean.cpu().double(), mean, rtol=3e-5, atol=1e-30) and abs(float(b.loss) / loss - 1) < 3e-5
    assert not b.mean[0, 7] and not d[100].any() and not d[:, 7].any()
    scale = dl.abs().amax()
    assert torch.isfinite(d).all() and ((d.cpu().double() - dl).abs() <= 3e-5 * scale).all()


def test_a_dominant_expert_loses_no_digits():
    """p near 1: the gradient there is a small difference, still relatively exact."""
    logits = torch.zeros(40, 3, device="cuda")
    logits[:, 1] = torch.linspace(5, 30, 40)
    ids = torch.tensor([[1], [0]], device="cuda", dtype=torch.int32).repeat(20, 1)
    b = moe.router_balance_loss(logits, ids, 1.0)
    d = moe.router_balance_loss_backward(logits, b).cpu().double()
    # in 64 bits, with the same regrouping: p* (c* - sum) = -p* sum_j p_j (c_j - c*)
    x = logits.cpu().double()
    p = torch.softmax(x, 1)
    c = b.counts.cpu().double()[0] * 3 / 40 / 40
    want = p * ((c - c[1]) - (p * (c - c[1])).sum(1, keepdim=True))
    assert ((d - want).abs() <= 1e-5 * want.abs()).all()


def test_ids_out_of_range_are_reported_and_not_counted():
    logits, ids = case(4, 200, 16, 2)
    ids[3, 0], ids[150, 1] = 16, -1
    b = moe.router_balance_loss(logits, ids)
    assert moe.device_error() == 0x1
    assert int(b.counts.sum()) == 398


def test_the_same_expert_twice_counts_twice():
    logits, ids = case(5, 50, 8, 2)
    ids[:, 1] = ids[:, 0]
    check(logits, ids)


def test_nan_logits_reach_the_loss():
    logits, ids = case(6, 30, 8, 2)
    logits[4, 2] = float("nan")
    b = moe.router_balance_loss(logits, ids)
    d = moe.router_balance_loss_backward(logits, b)
    assert b.loss.isnan().all() and d[4].isnan().all() and torch.isfinite(d[5]).all()


def test_gradient_against_differences():
    logits, ids = case(7, 6, 5, 2)
    b = moe.router_balance_loss(logits, ids, 1.0, seqs=2)
    d = moe.router_balance_loss_backward(logits, b).cpu().double()
    x, h = logits.cpu().double(), 1e-5
    for t in range(6):
        for e in range(5):
            up, down = x.clone(), x.clone()
            up[t, e] += h
            down[t, e] -= h
            slope = (ref.balance(up, ids.cpu(), 1.0, 2, None)[0] - ref.balance(down, ids.cpu(), 1.0, 2, None)[0]) / (2 * h)
            # central differences: h^2 of the third derivative, 1e-10, and 64-bit rounding over h, 1e-11
            assert abs(float(d[t, e]) - slope) <= 1e-6 * d.abs().max() + 1e-9


def test_the_same_bits_every_time_and_in_a_graph():
    logits, ids = case(8, 8192, 256, 8)
    valid = torch.rand(8192, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0)) < 0.8
    b = moe.router_balance_loss(logits, ids, 0.1, seqs=4, valid=valid)
    d = moe.router_balance_loss_backward(logits, b)
    for _ in range(10):
        c = moe.router_balance_loss(logits, ids, 0.1, seqs=4, valid=valid)
        assert torch.equal(b.loss, c.loss) and torch.equal(b.mean, c.mean)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = moe.router_balance_loss(logits, ids, 0.1, seqs=4, valid=valid)
        gd = moe.router_balance_loss_backward(logits, g)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(g.loss, b.loss) and torch.equal(g.counts, b.counts) and torch.equal(gd, d)


def test_gradient_into_the_logits_own_memory():
    logits, ids = case(9, 100, 24, 2)
    b, d = check(logits, ids, grad=1.0, coef=1.0)
    assert torch.equal(moe.router_balance_loss_backward(logits, b, torch.ones(1, device="cuda"), out=logits), d)


def test_router_backward_adds_the_loss_gradient():
    g = torch.Generator(device="cuda").manual_seed(10)
    T, D, E, k = 200, 128, 16, 2
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, wg, G, o = r(T, D), r(E, D) * 0.1, r(T, D), r(T * k, D)
    pos = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
    logits, ids, _ = moe.router_topk(x, wg, k)
    b = moe.router_balance_loss(logits, ids, 200.0)
    aux = moe.router_balance_loss_backward(logits, b)
    dw0, dl0, gg0, sg0 = moe.router_backward(G, o, pos, x, wg, logits, ids)
    dw, dl, gg, sg = moe.router_backward(G, o, pos, x, wg, logits, ids, dlogits_aux=aux)
    assert torch.equal(dw, dw0)
    # the sum is rounded once; dl0 is within half a bf16 step of the router's own part
    err = (dl.double() - (dl0.double() + aux.double())).abs()
    assert (err <= 2.0 ** -8 * (dl0.double().abs() + (dl0.double() + aux.double()).abs()) + 1e-30).all()
    assert (aux.abs().max() > 0.01 * dl0.abs().max())
    # the gate's gradients are those of the sum
    want = dl.double().t() @ x.double()
    assert (gg.double() - want).norm() <= 2e-3 * want.norm()
    want = dl.double() @ wg.double()
    assert (sg.double() - want).norm() <= (2.0 ** -8 + 1e-5) * want.norm()


def test_on_two_streams_at_once():
    a, b = case(12, 6000, 64, 4), case(13, 3000, 300, 8)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    want = []
    for x, ids in (a, b):
        r = moe.router_balance_loss(x, ids, 0.1, seqs=3)
        want.append((r, moe.router_balance_loss_backward(x, r)))
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for (x, ids), st in zip((a, b), streams):
            with torch.cuda.stream(st):
                r = moe.router_balance_loss(x, ids, 0.1, seqs=3)
                got.append((r, moe.router_balance_loss_backward(x, r)))
        torch.cuda.synchronize()
        for (r, d), (r0, d0) in zip(got, want):
            assert torch.equal(r.loss, r0.loss) and torch.equal(r.counts, r0.counts) and torch.equal(d, d0)


def test_offsets_past_32_bits():
    T, E = 2_200_000, 1000
    g = torch.Generator(device="cuda").manual_seed(11)
    logits = torch.empty(T, E, device="cuda")
    for part in logits.split(200_000):
        part.normal_(generator=g)
    ids = torch.randint(0, E, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    b = moe.router_balance_loss(logits, ids, 1.0, seqs=11)
    d = moe.router_balance_loss_backward(logits, b)
    assert moe.device_error() == 0 and int(b.counts.sum()) == T
    p = torch.softmax(logits[-200_000:].double(), 1)
    mean = p.mean(0)
    assert ((b.mean[10].double() - mean).abs() <= 1e-5 * mean).all()
    c = b.counts[10].double() * E / 11 / 200_000 / 200_000
    want = p[-100:] * (c - (p[-100:] @ c).unsqueeze(1))
    assert ((d[-100:].double() - want).abs() <= 1e-5 * want.abs().amax()).all()

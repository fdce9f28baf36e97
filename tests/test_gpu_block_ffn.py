"""GPU tests of a training step of the MoE layer on PER_BLOCK128 weights: router, balance
loss, experts forward and backward, router backward.

Each step is checked against its 64-bit form on the GPU's own inputs of that step; the
whole is compared with 64-bit arithmetic without any rounding.  There an e4m3 operand is
off by half a step, uniform: 2^-4 / sqrt(3) of its value, 3.6 %, at most (root mean
square); up to eight independent such operands meet in an output (dW_in: x twice, w_in, dO,
w_out, h's two factors, dA), sqrt(8) * 3.6 % = 10.2 %."""

import pytest
import torch

from tests import block_helpers as ref
from tests.test_gpu_block import check_gradient, check_product, gen

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("fp8_quantized_moe_gb300")


def layer(seed, T, D, E, k, F):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, dY = r(T, D).bfloat16(), r(T, D).bfloat16()
    w_in, w_out = (0.05 * r(E, 2 * F, D)).bfloat16(), (0.05 * r(E, D, F)).bfloat16()
    w_gate = (r(E, D) / D ** 0.5).bfloat16()
    return x, dY, w_in, w_out, w_gate


def bf16_step(got, want, parts=None):
    """got = bf16(want) up to half a step (want: 64 bits)."""
    tol = want.abs() * 2.0 ** -8 + (0 if parts is None else parts * 2.0 ** -20) + 1e-30
    assert ((got.double() - want).abs() <= tol).all()


def exact_step(x, ids, w, w_in, w_out, dY):
    """(y, dX, dW_in [E, D, 2F], dW_out [E, F, D]) in 64 bits, nothing rounded."""
    F = w_out.shape[2]
    x, w, dY = x.double(), w.double(), dY.double()
    y, dX = torch.zeros_like(x), torch.zeros_like(x)
    dWi = torch.zeros(w_in.shape[0], w_in.shape[2], 2 * F, dtype=torch.float64, device=x.device)
    dWo = torch.zeros(w_in.shape[0], F, w_in.shape[2], dtype=torch.float64, device=x.device)
    for e in range(w_in.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        a = x[t] @ w_in[e].double().t()
        a0, a1 = a[:, :F], a[:, F:]
        sg = torch.sigmoid(a0)
        h = a0 * sg * a1
        y.index_add_(0, t, (h @ w_out[e].double().t()) * w[t, j].unsqueeze(1))
        dO = dY[t] * w[t, j].unsqueeze(1)
        dH = dO @ w_out[e].double()
        dA = torch.cat([dH * a1 * sg * (1 + a0 * (1 - sg)), dH * a0 * sg], 1)
        dX.index_add_(0, t, dA @ w_in[e].double())
        dWi[e], dWo[e] = x[t].t() @ dA, h.t() @ dO
    return y, dX, dWi, dWo


def close(got, want, bound=0.102):
    err = (got.double() - want).norm() / want.norm()
    assert err <= bound, float(err)


@pytest.mark.parametrize("T,D,E,k,F", [(200, 256, 8, 2, 128), (1, 128, 4, 2, 256), (515, 384, 16, 6, 256), (300, 128, 3, 1, 384)])
def test_training_step(T, D, E, k, F):
    x, dY, w_in, w_out, w_gate = layer(T + D, T, D, E, k, F)
    W = moe.prepare_weights(w_in, w_out, moe.PER_BLOCK128, for_backward=True)
    buf = moe.FFNBuffers(T, D, E, k, F, moe.PER_ROW_BLOCK128, "cuda", backward=True)
    logits, ids, w = moe.router_topk(x, w_gate, k)
    b = moe.router_balance_loss(logits, ids, 0.01)
    y = moe.ffn_forward(x, ids, w, W, moe.PER_ROW_BLOCK128, buf).clone()
    keep = {}
    dX, dW_in, dW_out = moe.ffn_backward(dY, w, W, buf, x=x, keep=keep)
    aux = moe.router_balance_loss_backward(logits, b, torch.tensor([2.0], device="cuda"))
    dw, dl, gg, sg = moe.router_backward(dY, buf.o, buf.sort["pos"], x, w_gate, logits, ids, dlogits_aux=aux)
    assert moe.device_error() == 0
    s = buf.sort
    sizes, src = s["group_sizes"].tolist(), s["sorted_src"].long()

    # forward products on the codes that they were given
    check_product(buf.a, *ref.gmm(s["xs_q"], s["xs_scale"], W.w_in, W.s_in, sizes), D)
    check_product(buf.o, *ref.gmm(buf.h_q, buf.h_s, W.w_out, W.s_out, sizes), F)
    # dO: one product, one rounding; its codes
    dO = dY.double()[src // k] * w.double().flatten()[src].unsqueeze(1)
    bf16_step(keep["dO"], dO, dO.abs())
    vq, vs = ref.quantise_rows128(keep["dO"])
    assert torch.equal(ref.e4m3(keep["dO_q"]), vq) and torch.equal(keep["dO_s"].double(), vs)
    check_product(buf.dH, *ref.gmm(keep["dO_q"], keep["dO_s"], W.w_out_t, W.s_out_t, sizes), D)
    # SwiGLU backward: a few fp32 roundings of each factor, one bf16 rounding
    a, dH = buf.a.double(), buf.dH.double()
    a0, a1 = a[:, :F], a[:, F:]
    sig = torch.sigmoid(a0)
    bf16_step(keep["h"], a0 * sig * a1, (a0 * a1).abs())
    d0 = dH * a1 * sig
    bf16_step(keep["dA"], torch.cat([d0 * (1 + a0 * (1 - sig)), dH * a0 * sig], 1), torch.cat([d0.abs() * (1 + a0.abs()), (dH * a0).abs()], 1))
    vq, vs = ref.quantise_rows128(keep["dA"])
    assert torch.equal(ref.e4m3(keep["dA_q"]), vq) and torch.equal(keep["dA_s"].double(), vs)
    check_product(buf.dXs, *ref.gmm(keep["dA_q"], keep["dA_s"], W.w_in_t, W.s_in_t, sizes), 2 * F)
    xs = x[src // k]
    check_gradient(dW_in, *ref.tgmm(xs, keep["dA"], sizes, 0, E), max(sizes))
    check_gradient(dW_out, *ref.tgmm(keep["h"], keep["dO"], sizes, 0, E), max(sizes))

    # the whole against arithmetic without rounding
    ey, edX, edWi, edWo = exact_step(x, ids, w, w_in, w_out, dY)
    close(y, ey)
    close(dX, edX)
    close(dW_in, edWi)
    close(dW_out, edWo)
    # both losses in the router's gradients
    bf16_step(dl, ref_dlogits(logits, ids, dw) + aux.double(), 64 * (aux.double().abs() + dw.double().abs().amax(1, keepdim=True)))
    close(gg, dl.double().t() @ x.double(), 2e-3)


def ref_dlogits(logits, ids, dw):
    p = torch.softmax(logits.double(), 1)
    g = torch.zeros_like(p).scatter_(1, ids.long(), dw.double())
    return p * (g - (p * g).sum(1, keepdim=True))


def test_steps_repeat_on_the_same_buffers():
    T, D, E, k, F = 150, 256, 6, 2, 128
    x, dY, w_in, w_out, w_gate = layer(7, T, D, E, k, F)
    W = moe.prepare_weights(w_in, w_out, moe.PER_BLOCK128, for_backward=True)
    buf = moe.FFNBuffers(T, D, E, k, F, moe.PER_ROW_BLOCK128, "cuda", backward=True)
    _, ids, w = moe.router_topk(x, w_gate, k)

    def step():
        y = moe.ffn_forward(x, ids, w, W, moe.PER_ROW_BLOCK128, buf).clone()
        dX, a, b = moe.ffn_backward(dY, w, W, buf, x=x)
        return y, dX.clone(), a, b

    first = step()
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, step()))
    # captured: the same values from new inputs in the same places
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x2, dY2, *_ = layer(8, T, D, E, k, F)
    x.copy_(x2)
    dY.copy_(dY2)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in got]
    assert all(torch.equal(p, q) for p, q in zip(got, step()))
    assert not torch.equal(got[0], first[0])


def test_decoding_on_the_same_weights():
    T, D, E, k, F = 5, 256, 8, 2, 256
    x, _, w_in, w_out, w_gate = layer(9, T, D, E, k, F)
    W = moe.prepare_weights(w_in, w_out, moe.PER_BLOCK128)
    _, ids, w = moe.router_topk(x, w_gate, k)
    y = moe.ffn_decode(x, ids, w, moe.decode_weights(W))
    wi, wo = ref.weight_value(W.w_in, W.s_in), ref.weight_value(W.w_out, W.s_out)
    want = exact_step(x, ids, w, wi, wo, torch.zeros_like(x))[0]
    # bf16's half step and h's 2^-11 (activations are not rounded in a decoding step)
    assert moe.device_error() == 0 and (y.double() - want).norm() <= 2.0 ** -8 * want.norm()


def test_refusals():
    T, D, E, k, F = 4, 128, 2, 1, 128
    x, dY, w_in, w_out, _ = layer(10, T, D, E, k, F)
    W = moe.prepare_weights(w_in, w_out, moe.PER_BLOCK128)
    buf = moe.FFNBuffers(T, D, E, k, F, moe.PER_ROW_BLOCK128, "cuda", backward=True)
    ids, w = torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda")
    with pytest.raises(moe.MoEError, match="PER_ROW_BLOCK128"):
        moe.ffn_forward(x, ids, w, W, moe.PER_ROW, moe.FFNBuffers(T, D, E, k, F, moe.PER_ROW, "cuda"))
    moe.ffn_forward(x, ids, w, W, moe.PER_ROW_BLOCK128, buf)
    with pytest.raises(moe.MoEError, match="for_backward"):
        moe.ffn_backward(dY, w, W, buf, x=x)
    W = moe.prepare_weights(w_in, w_out, moe.PER_BLOCK128, for_backward=True)
    with pytest.raises(moe.MoEError, match="and x"):
        moe.ffn_backward(dY, w, W, buf)
    small = moe.FFNBuffers(T, D, E, k, F, moe.PER_ROW_BLOCK128, "cuda")
    moe.ffn_forward(x, ids, w, W, moe.PER_ROW_BLOCK128, small)
    with pytest.raises(moe.MoEError, match="backward=True"):
        moe.ffn_backward(dY, w, W, small, x=x)
    with pytest.raises(moe.MoEError, match="static"):
        moe.ffn_backward(dY, w, moe.prepare_weights(w_in, w_out, moe.PER_ROW), buf)
    with pytest.raises(moe.MoEError, match="expected 4 values"):
        moe.gather_scale_quant_block(dY, w[:2], torch.zeros(T, dtype=torch.int32, device="cuda"), 1)
    with pytest.raises(moe.MoEError, match="decode_weights"):
        moe.ffn_decode(x, ids, w, W)
    with pytest.raises(moe.MoEError):
        moe.prepare_weights(w_in[:, :, :64].contiguous(), w_out[:, :64].contiguous(), moe.PER_BLOCK128)


def test_rows_of_tiny_values_with_zeros_among_them():
    """Block scales whose reciprocals are past fp32: exact quotients, and zeros stay zeros."""
    g = torch.Generator(device="cuda").manual_seed(31)
    x = torch.randn(9, 512, generator=g, device="cuda") * 2.0 ** -122
    x[:, ::3] = 0
    x[3] *= 2.0 ** 100
    x[4, 128:256] *= 2.0 ** 121
    x = x.bfloat16()
    vq, vs = ref.quantise_rows128(x)
    src = torch.arange(9, dtype=torch.int32, device="cuda")
    dO, q, s = moe.gather_scale_quant_block(x, None, src, 1)
    assert torch.equal(dO, x) and torch.equal(s.double(), vs) and torch.equal(ref.e4m3(q), vq)
    q, s = moe.quantize_rows(x, moe.PER_ROW_BLOCK128)
    assert torch.equal(s.double(), vs) and torch.equal(ref.e4m3(q), vq)
    # dA1 = dH silu(a0), a0 = 1; dA0 = 0 (a1 = 0), scale 1
    a = torch.zeros(9, 1024, device="cuda", dtype=torch.bfloat16)
    a[:, :512] = 1
    dA, q, s, h = moe.swiglu_bwd_quant_block(x, a)
    vq, vs = ref.quantise_rows128(dA)
    assert not dA[:, :512].any() and not h.any()
    assert torch.equal(s.double(), vs) and torch.equal(ref.e4m3(q), vq)

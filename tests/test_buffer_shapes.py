"""Buffers that were made for another shape are refused by name before anything is launched
(their kernels would write past them).  On the CPU: every refusal comes before the first
look at a device."""

import pytest
import torch

moe = pytest.importorskip("fp8_quantized_moe_gb300")

T, D, E, k, F = 6, 256, 4, 2, 128
MODES = [moe.PER_ROW, moe.PER_ROW_BLOCK128, moe.PER_TENSOR, moe.MX32, moe.MX4]


def inputs(T=T, D=D, k=k):
    return (torch.zeros(T, D, dtype=torch.bfloat16), torch.zeros(T, k, dtype=torch.int32),
            torch.zeros(T, k, dtype=torch.float32))


def weights(mode, E=E, D=D, F=F):
    half = 2 if mode == moe.MX4 else 1
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    W = moe.ExpertWeights(u8(E, 2 * F, D // half), torch.zeros(1), mode, u8(E, D, F // half), torch.zeros(1), mode)
    W.w_in_t, W.w_out_t = u8(E, D, 2 * F), u8(E, F, D)
    return W


def act(w_mode):
    return moe.PER_ROW_BLOCK128 if w_mode == moe.PER_BLOCK128 else w_mode


def sorted_as(mode, T=T, D=D, E=E, k=k):
    """What a sort of this shape leaves in a dict."""
    R = T * k
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(R, D // 2 if mode == moe.MX4 else D, dtype=torch.uint8)
    return dict(sorted_src=i32(R), pos=i32(R), group_sizes=i32(E), group_offsets=i32(E + 1), xs_q=q,
                xs_scale=moe._scale_buf(mode, R, D, "cpu"))


def buffers(mode, filled=True, **kw):
    buf = moe.FFNBuffers(T, D, E, k, F, mode, "cpu", **kw)
    if filled:
        buf.sort.update(sorted_as(mode))
    return buf


@pytest.mark.parametrize("w_mode", MODES + [moe.PER_BLOCK128])
def test_forward_on_buffers_of_another_shape(w_mode):
    mode = act(w_mode)
    W, st = weights(w_mode), torch.ones(1)
    for filled in (False, True):
        for x, ids, w in (inputs(T=T + 1), inputs(T=T - 1), inputs(k=k + 1), inputs(T=3 * T)):
            with pytest.raises(moe.MoEError, match="made for 6 tokens of 2 experts"):
                moe.ffn_forward(x, ids, w, W, mode, buffers(mode, filled), st, st)
        x, ids, w = inputs()
        with pytest.raises(moe.MoEError, match="made for D = 256 and F = 128"):
            moe.ffn_forward(x, ids, w, weights(w_mode, F=2 * F), mode, buffers(mode, filled), st, st)
        with pytest.raises(moe.MoEError, match="ffn_forward x"):
            moe.ffn_forward(inputs(D=2 * D)[0], ids, w, W, mode, buffers(mode, filled), st, st)
        with pytest.raises(moe.MoEError, match="ffn_forward x"):
            moe.ffn_forward(x[:3], ids, w, W, mode, buffers(mode, filled), st, st)
        with pytest.raises(moe.MoEError, match="ffn_forward topk_w"):
            moe.ffn_forward(x, ids, w[:3], W, mode, buffers(mode, filled), st, st)
        with pytest.raises(moe.MoEError, match="topk_ids"):
            moe.ffn_forward(x, ids.long(), w, W, mode, buffers(mode, filled), st, st)


def test_forward_on_buffers_of_another_scale_mode():
    x, ids, w = inputs()
    for made, mode in ((moe.PER_ROW, moe.PER_ROW_BLOCK128), (moe.PER_TENSOR, moe.PER_ROW), (moe.MX4, moe.PER_TENSOR),
                       (moe.PER_ROW, moe.MX32)):
        with pytest.raises(moe.MoEError, match=f"made for scale mode {made}"):
            moe.ffn_forward(x, ids, w, weights(mode), mode, buffers(made), torch.ones(1), torch.ones(1))


@pytest.mark.parametrize("w_mode", [moe.PER_ROW, moe.PER_TENSOR, moe.MX32, moe.PER_BLOCK128])
@pytest.mark.parametrize("experts", [E + 1, 1024, 1])
def test_forward_with_another_number_of_experts(w_mode, experts):
    """The sort's dict holds the group sizes of the experts it was first called with."""
    mode = act(w_mode)
    x, ids, w = inputs()
    with pytest.raises(moe.MoEError, match="made for another shape: group_sizes"):
        moe.ffn_forward(x, ids, w, weights(w_mode, E=experts), mode, buffers(mode), torch.ones(1), torch.ones(1))


@pytest.mark.parametrize("was", [dict(T=T - 1), dict(T=T + 1), dict(k=1), dict(E=E - 1), dict(D=128)])
@pytest.mark.parametrize("mode", [moe.PER_ROW, moe.PER_ROW_BLOCK128, moe.PER_TENSOR, moe.MX32])
def test_sorts_into_a_dict_of_another_shape(mode, was):
    x, ids, _ = inputs()
    q = torch.zeros(T, D, dtype=torch.uint8)
    calls = [lambda o: moe.quantize_sort_mx(x, ids, E, out=o)] if mode == moe.MX32 else \
        [lambda o: moe.quantize_sort(x, ids, E, mode, torch.ones(1), out=o),
         lambda o: moe.ragged_sort(ids, E, q, torch.ones(T, 2), mode, out=o)]
    for call in calls:
        with pytest.raises(moe.MoEError, match="made for another shape"):
            call(sorted_as(mode, **was))


def test_sort_of_another_mode_and_of_too_few_rows():
    x, ids, _ = inputs()
    with pytest.raises(moe.MoEError, match="made for another shape: xs_scale"):
        moe.quantize_sort(x, ids, E, moe.PER_ROW_BLOCK128, out=sorted_as(moe.PER_ROW))
    with pytest.raises(moe.MoEError, match="made for another shape: xs_scale is nothing"):
        moe.quantize_sort(x, ids, E, moe.PER_ROW, out=sorted_as(moe.PER_TENSOR))
    with pytest.raises(moe.MoEError, match="topk_ids are of 6 tokens"):
        moe.quantize_sort(x[:5], ids, E, moe.PER_ROW)
    with pytest.raises(moe.MoEError, match="topk_ids"):
        moe.quantize_sort_mx(x, ids.long(), E)


def test_backward_on_what_does_not_belong_together():
    dY, _, w = inputs()
    x, W, st = dY.clone(), weights(moe.PER_BLOCK128), torch.ones(1)
    made = lambda **kw: buffers(moe.PER_ROW_BLOCK128, backward=True, **kw)  # noqa: E731
    with pytest.raises(moe.MoEError, match="ffn_backward dY"):
        moe.ffn_backward(dY[:5], w, W, made(), x=x)
    with pytest.raises(moe.MoEError, match="ffn_backward x"):
        moe.ffn_backward(dY, w, W, made(), x=x[:5])
    with pytest.raises(moe.MoEError, match="ffn_backward topk_w"):
        moe.ffn_backward(dY, w[:5], W, made(), x=x)
    with pytest.raises(moe.MoEError, match="made for D = 256 and F = 128"):
        moe.ffn_backward(dY, w, weights(moe.PER_BLOCK128, F=2 * F), made(), x=x)
    for bad in (made(filled=False), made()):
        with pytest.raises(moe.MoEError, match="has to run on these buffers first"):
            moe.ffn_backward(dY, w, W if not bad.sort else weights(moe.PER_BLOCK128, E=E - 1), bad, x=x)
    static = buffers(moe.PER_TENSOR, backward=True)
    with pytest.raises(moe.MoEError, match="ffn_backward dY"):
        moe.ffn_backward(dY[:5], w, weights(moe.PER_TENSOR), static, st, st)
    with pytest.raises(moe.MoEError, match="backward=True"):
        moe.ffn_backward(dY, w, weights(moe.PER_TENSOR), buffers(moe.PER_TENSOR), st, st)


def test_gradient_workspace_grows_with_the_experts():
    buf = moe.FFNBuffers(T, D, E, k, F, moe.PER_ROW_BLOCK128, "cpu", backward=True)
    need = lambda n: max(moe.tgmm_mx_workspace_bytes(T * k, D, 2 * F, n), moe.tgmm_mx_workspace_bytes(T * k, F, D, n))  # noqa: E731
    small = buf.tgmm_workspace(2)
    assert small.numel() >= need(2) and buf.tgmm_workspace(2) is small
    large = buf.tgmm_workspace(1024)
    assert large.numel() >= need(1024) > need(2)
    assert buf.tgmm_workspace(2) is large

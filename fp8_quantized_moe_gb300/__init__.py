"""GB300 (sm_103a) FP8-quantized MoE expert FFN.

Python binding of libmoefp8.so (C ABI in include/moefp8.h).  Every function
here only marshals arguments: it allocates outputs with PyTorch, passes raw
device pointers and the current CUDA stream, and checks the status.  All
arithmetic runs in the library's CUDA kernels; there is no fallback.

Forward path (the order of "Quantize activations before EP all gather"):
quantize_rows -> ragged_sort -> gmm (wi_0 | wi_1) -> swiglu_quant ->
gmm (wo) -> ragged_gather_reduce.  With int8 expert weights ("Keep qwix out
of tpu-inference's fused MoE kernel and pre-quantize weights": float8_e4m3fn
or int8 weights) both contractions run gmm_w8.  The backward pass of the static scheme
("Support quantization for tokamax gmm v2": fp8_static_wa) adds
gather_scale_quant, swiglu_bwd_quant, quantize_group_cols and tgmm.

The MXFP8 variant (MX32: OCP MX v1.0 blocks of 32 e4m3 values sharing one
E8M0 power-of-two scale along the contracted dimension) runs the same
forward path on the block-scaled tensor-core MMA: quantize_sort_mx ->
gmm_mx_swiglu (or gmm_mx + swiglu_quant_mx) -> gmm_mx -> ragged_gather_reduce.
The MXFP4 variant (MX4: the same blocks of e2m1 values, two a byte) runs
quantize_sort_mx4 -> gmm_mx4 -> swiglu_quant_mx4 -> gmm_mx4 ->
ragged_gather_reduce.

Expert weights with one scale for each 128 x 128 block (PER_BLOCK128) are for training as
well: gmm_block contracts them with activations that carry one scale per row and 128 columns
and, transposed, gives the input gradient; tgmm_mx the weight gradient from bf16 operands;
ffn_forward and ffn_backward run on them, and router_balance_loss with its gradient joins
router_backward.

Single decoding steps (up to 64 tokens) take ffn_decode: the whole expert FFN in
one kernel, on bf16 activations and the same expert weights of any type.
"""

from __future__ import annotations

import ctypes
import dataclasses
import functools
from typing import Optional

import torch

from . import _native
from ._native import MoEError, check

PER_ROW = 0
PER_ROW_BLOCK128 = 1
PER_TENSOR = 2
PER_GROUP_COL = 3
MX32 = 4  # MXFP8: uint8 E8M0 codes, K-block-major [cols/128, rows, 4]
MX4 = 5  # MXFP4: packed e2m1 codes, two a byte, with scale codes as MX32
PER_BLOCK128 = 6  # weights: one fp32 scale for each 128 x 128 block, [E, ceil(N/128), K/128]

__all__ = [
    "PER_ROW", "PER_ROW_BLOCK128", "PER_TENSOR", "PER_GROUP_COL", "MoEError", "lib", "device_error",
    "quantize_rows", "quantize_weights", "ragged_sort", "gmm", "gmm_swiglu", "swiglu_fusable", "swiglu_fuse_pays", "swiglu_quant", "ragged_gather_reduce",
    "gather_scale_quant", "swiglu_bwd_quant", "quantize_group_cols", "tgmm", "transpose_u8",
    "router_topk", "router_backward", "MX32", "quantize_rows_mx", "quantize_weights_mx", "quantize_sort_mx",
    "gmm_mx", "gmm_mx_swiglu", "swiglu_quant_mx", "MX4", "quantize_rows_mx4", "quantize_weights_mx4",
    "dequantize_rows_mx4", "quantize_sort_mx4", "swiglu_quant_mx4", "gmm_mx4", "quantize_weights_int8", "gmm_w8", "gmm_w8_workspace_bytes",
    "prepare_weights_w8",
    "ExpertWeights", "prepare_weights", "FFNBuffers", "ffn_forward", "ffn_backward", "DecodeBuffers", "ffn_decode",
    "PER_BLOCK128", "decode_weights", "quantize_weights_block", "gmm_block", "tgmm_mx", "tgmm_mx_workspace_bytes",
    "gather_scale_quant_block", "swiglu_bwd_quant_block", "BalanceLoss", "router_balance_loss",
    "router_balance_loss_backward",
]


def lib():
    return _native.load()


def _lib():
    """lib() without its lock once the library is loaded."""
    return _native._lib or _native.load()


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise MoEError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise MoEError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _s():
    # (the raw handle: building a torch.cuda.Stream object takes longer than a launch)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _stream(dev: int) -> int:
    """The raw handle of the current stream of `dev`, the current CUDA device."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _arg(what: str, t, dtype, ndim: int):
    """`t`, checked to be a tensor of this type and number of dimensions (its
    shape is then read off it)."""
    if t.dtype is not dtype or t.dim() != ndim:
        raise MoEError(f"{what}: expected {dtype} of {ndim} dimensions, got {t.dtype} {list(t.shape)}")
    return t


def _ptr(what: str, t: torch.Tensor, dtype, shape: tuple, dev: int) -> int:
    """The address of `t`, checked against the type, shape and device that the call `what` takes."""
    if t.dtype is not dtype or t.shape != shape:
        raise MoEError(f"{what}: expected {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.get_device() != dev:
        raise MoEError(f"{what}: expected a tensor on the current CUDA device {dev}, got one on {t.device}")
    if not t.is_contiguous():
        raise MoEError(f"{what}: expected a contiguous tensor")
    return t.data_ptr()


def _dev(what: str, t: torch.Tensor) -> int:
    """The device of `t`, which has to be the current CUDA device (its stream is the one launched on)."""
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise MoEError(f"{what}: expected a tensor on the current CUDA device, got one on {t.device}")
    return dev


def _nb(cols: int) -> int:
    return (cols + 127) // 128


def device_error() -> int:
    """Synchronise the current stream and return (and clear) the device error word."""
    code = ctypes.c_int(0)
    st = lib().moe_get_device_error(_s(), ctypes.byref(code))
    if st not in (0, 4):
        check(st, "moe_get_device_error")
    return code.value


def _scale_shape(mode: int, rows: int, cols: int):
    """Type and shape of the scales of [rows, cols] in this mode, or None for one scale."""
    if mode == PER_ROW:
        return torch.float32, (rows,)
    if mode == PER_ROW_BLOCK128:
        return torch.float32, (rows, _nb(cols))
    if mode in (MX32, MX4):
        return torch.uint8, (cols // 128, rows, 4)
    return None


def _scale_buf(mode: int, rows: int, cols: int, device, out=None):
    if out is not None:
        return out
    made = _scale_shape(mode, rows, cols)
    return None if made is None else torch.empty(made[1], dtype=made[0], device=device)


def _sort_buffers(what: str, out: Optional[dict], x: torch.Tensor, topk_ids: torch.Tensor, E: int, mode: int):
    """The dict of a sort: `out`, or a new one.  Its tensors are allocated where it is empty; those that it holds
    have to be of this call's shapes (a captured graph may write them, so they are not replaced)."""
    T, k = _arg(f"{what} topk_ids", topk_ids, torch.int32, 2).shape
    if x.dim() != 2 or x.shape[0] < T:
        raise MoEError(f"{what}: topk_ids are of {T} tokens, x is {list(x.shape)}")
    R, D, dev = T * k, x.shape[1], x.device
    o = out if out is not None else {}
    if "sorted_src" not in o:
        o["sorted_src"] = torch.empty(R, dtype=torch.int32, device=dev)
        o["pos"] = torch.empty(R, dtype=torch.int32, device=dev)
        o["group_sizes"] = torch.empty(E, dtype=torch.int32, device=dev)
        o["group_offsets"] = torch.empty(E + 1, dtype=torch.int32, device=dev)
        o["xs_q"] = torch.empty(R, D, dtype=torch.uint8, device=dev)
        o["xs_scale"] = _scale_buf(mode, R, D, dev)
        return o
    i32 = torch.int32
    for key, want in (("sorted_src", (i32, (R,))), ("pos", (i32, (R,))), ("group_sizes", (i32, (E,))),
                      ("group_offsets", (i32, (E + 1,))), ("xs_q", (torch.uint8, (R, D))),
                      ("xs_scale", _scale_shape(mode, R, D))):
        t = o[key]
        if want is not None and (t is None or t.shape != want[1] or t.dtype is not want[0] or t.device != dev):
            held = "nothing" if t is None else f"{t.dtype} {list(t.shape)} on {t.device}"
            raise MoEError(f"{what}: the given buffers were made for another shape: {key} is {held}, "
                           f"expected {want[0]} {list(want[1])} on {dev}")
    return o


def quantize_rows(x: torch.Tensor, mode: int, static_scale: Optional[torch.Tensor] = None, q=None, scale=None):
    """bf16 [rows, cols] -> (e4m3 codes uint8 [rows, cols], fp32 scales or None)."""
    rows, cols = x.shape
    q = torch.empty(rows, cols, dtype=torch.uint8, device=x.device) if q is None else q
    scale = _scale_buf(mode, rows, cols, x.device, scale)
    check(lib().moe_quantize_rows(_p(x), rows, cols, mode, _p(static_scale), _p(q), _p(scale), _s()),
          "moe_quantize_rows")
    return q, scale


def quantize_weights(w: torch.Tensor, mode: int, static_scale: Optional[torch.Tensor] = None):
    """bf16 [E, N, K] -> (codes [E, N, K], scales [E, N] | [E, K/128, N] | None)."""
    E, N, K = w.shape
    q = torch.empty(E, N, K, dtype=torch.uint8, device=w.device)
    if mode == PER_ROW:
        s = torch.empty(E, N, dtype=torch.float32, device=w.device)
    elif mode == PER_ROW_BLOCK128:
        s = torch.empty(E, _nb(K), N, dtype=torch.float32, device=w.device)
    else:
        s = None
    check(lib().moe_quantize_weights(_p(w), E, N, K, mode, _p(static_scale), _p(q), _p(s), _s()),
          "moe_quantize_weights")
    return q, s


def quantize_weights_int8(w: torch.Tensor, mode: int, static_scale: Optional[torch.Tensor] = None):
    """bf16 [E, N, K] -> (int8 codes [E, N, K], scales [E, N] | [E, K/128, N] | None)."""
    E, N, K = w.shape
    q = torch.empty(E, N, K, dtype=torch.int8, device=w.device)
    if mode == PER_ROW:
        s = torch.empty(E, N, dtype=torch.float32, device=w.device)
    elif mode == PER_ROW_BLOCK128:
        s = torch.empty(E, _nb(K), N, dtype=torch.float32, device=w.device)
    else:
        s = None
    check(lib().moe_quantize_weights_int8(_p(w), E, N, K, mode, _p(static_scale), _p(q), _p(s), _s()),
          "moe_quantize_weights_int8")
    return q, s


def quantize_rows_mx(x: torch.Tensor, q=None, sf=None):
    """MXFP8: bf16 [rows, cols] -> (e4m3 codes [rows, cols], E8M0 codes uint8 [cols/128, rows, 4])."""
    rows, cols = x.shape
    q = torch.empty(rows, cols, dtype=torch.uint8, device=x.device) if q is None else q
    sf = _scale_buf(MX32, rows, cols, x.device, sf)
    check(lib().moe_quantize_rows_mx(_p(x), rows, cols, _p(q), _p(sf), _s()), "moe_quantize_rows_mx")
    return q, sf


def quantize_weights_mx(w: torch.Tensor):
    """MXFP8 weights: bf16 [E, N, K] -> (codes [E, N, K], E8M0 codes [K/128, E*N, 4])."""
    E, N, K = w.shape
    q, sf = quantize_rows_mx(w.reshape(E * N, K))
    return q.view(E, N, K), sf


def ragged_sort(topk_ids: torch.Tensor, E: int, x_q: torch.Tensor, x_scale: Optional[torch.Tensor], mode: int,
                out: Optional[dict] = None):
    """Returns dict(sorted_src, pos, group_sizes, group_offsets, xs_q, xs_scale)."""
    T, k = topk_ids.shape
    D, dev = x_q.shape[1], x_q.device
    o = _sort_buffers("ragged_sort", out, x_q, topk_ids, E, mode)
    nws = lib().moe_ragged_sort_workspace_bytes(T, k, E)
    if "sort_ws" not in o or o["sort_ws"].numel() < nws:
        o["sort_ws"] = torch.empty(max(nws, 16), dtype=torch.uint8, device=dev)
    xs_scale = o["xs_scale"]
    check(lib().moe_ragged_sort(_p(topk_ids), T, k, E, _p(x_q), _p(x_scale), D, mode, _p(o["sorted_src"]),
                                _p(o["pos"]), _p(o["group_sizes"]), _p(o["group_offsets"]), _p(o["xs_q"]),
                                _p(xs_scale), _p(o["sort_ws"]), o["sort_ws"].numel(), _s()), "moe_ragged_sort")
    return o


def quantize_sort(x: torch.Tensor, topk_ids: torch.Tensor, E: int, mode: int,
                  static_scale: Optional[torch.Tensor] = None, out: Optional[dict] = None):
    """Steps 1 + 2 fused: sort indices and the gathered codes/scales of x.
    Returns the same dict as ragged_sort (bit-identical xs_q / xs_scale)."""
    T, k = topk_ids.shape
    D, dev = x.shape[1], x.device
    o = _sort_buffers("quantize_sort", out, x, topk_ids, E, mode)
    nws = lib().moe_ragged_sort_workspace_bytes(T, k, E)
    if "sort_ws" not in o or o["sort_ws"].numel() < nws:
        o["sort_ws"] = torch.empty(max(nws, 16), dtype=torch.uint8, device=dev)
    xs_scale = o["xs_scale"] if mode != PER_TENSOR else None
    check(lib().moe_quantize_sort(_p(x), _p(topk_ids), T, k, E, D, mode, _p(static_scale), _p(o["sorted_src"]),
                                  _p(o["pos"]), _p(o["group_sizes"]), _p(o["group_offsets"]), _p(o["xs_q"]),
                                  _p(xs_scale), _p(o["sort_ws"]), o["sort_ws"].numel(), _s()), "moe_quantize_sort")
    return o


def quantize_sort_mx(x: torch.Tensor, topk_ids: torch.Tensor, E: int, out: Optional[dict] = None):
    """MXFP8 steps 1 + 2: the dict of quantize_sort with xs_scale = E8M0 codes [D/128, T*k, 4]."""
    T, k = topk_ids.shape
    D, dev = x.shape[1], x.device
    o = _sort_buffers("quantize_sort_mx", out, x, topk_ids, E, MX32)
    nws = lib().moe_ragged_sort_workspace_bytes(T, k, E)
    if "sort_ws" not in o or o["sort_ws"].numel() < nws:
        o["sort_ws"] = torch.empty(max(nws, 16), dtype=torch.uint8, device=dev)
    check(lib().moe_quantize_sort_mx(_p(x), _p(topk_ids), T, k, E, D, _p(o["sorted_src"]), _p(o["pos"]),
                                     _p(o["group_sizes"]), _p(o["group_offsets"]), _p(o["xs_q"]), _p(o["xs_scale"]),
                                     _p(o["sort_ws"]), o["sort_ws"].numel(), _s()), "moe_quantize_sort_mx")
    return o


def gmm_mx(lhs_q, lhs_sf, rhs_q, rhs_sf, group_sizes, group_offset: int = 0, E_local: Optional[int] = None,
           out=None):
    """MXFP8 grouped matmul -> bf16 [M, N]; lhs_sf [K/128, M, 4], rhs_sf [K/128, E_local*N, 4]."""
    M, K = lhs_q.shape
    El, N, K2 = rhs_q.shape
    if K2 != K:
        raise MoEError("lhs/rhs K mismatch")
    E = group_sizes.numel()
    E_local = El if E_local is None else E_local
    out = torch.empty(M, N, dtype=torch.bfloat16, device=lhs_q.device) if out is None else out
    check(lib().gmm_fp8_mx(_p(lhs_q), _p(lhs_sf), _p(rhs_q), _p(rhs_sf), _p(group_sizes), E, group_offset, E_local,
                           M, K, N, _p(out), _s()), "gmm_fp8_mx")
    return out


def gmm_mx_swiglu(lhs_q, lhs_sf, rhs_q, rhs_sf, group_sizes, group_offset: int = 0, E_local: Optional[int] = None,
                  keep_a: bool = False, a_out=None, h_q=None, h_sf=None):
    """MXFP8 gmm with [wi_0 | wi_1] fused with SwiGLU and the MXFP8
    requantisation of h.  Returns (h_q [M, F], h_sf [F/128, M, 4], a [M, 2F] bf16 or None)."""
    M, K = lhs_q.shape
    El, F2, K2 = rhs_q.shape
    if K2 != K:
        raise MoEError("lhs/rhs K mismatch")
    F = F2 // 2
    dev = lhs_q.device
    E = group_sizes.numel()
    E_local = El if E_local is None else E_local
    h_q = torch.empty(M, F, dtype=torch.uint8, device=dev) if h_q is None else h_q
    h_sf = _scale_buf(MX32, M, F, dev, h_sf)
    if keep_a and a_out is None:
        a_out = torch.empty(M, F2, dtype=torch.bfloat16, device=dev)
    check(lib().gmm_fp8_mx_swiglu(_p(lhs_q), _p(lhs_sf), _p(rhs_q), _p(rhs_sf), _p(group_sizes), E, group_offset,
                                  E_local, M, K, F, _p(a_out), _p(h_q), _p(h_sf), _s()), "gmm_fp8_mx_swiglu")
    return h_q, h_sf, a_out


def swiglu_quant_mx(a: torch.Tensor, h_q=None, h_sf=None):
    """MXFP8 step 4: a = [a0 | a1] bf16 [R, 2F] -> (h codes [R, F], h E8M0 codes [F/128, R, 4])."""
    R, F2 = a.shape
    F = F2 // 2
    h_q = torch.empty(R, F, dtype=torch.uint8, device=a.device) if h_q is None else h_q
    h_sf = _scale_buf(MX32, R, F, a.device, h_sf)
    check(lib().moe_swiglu_quant_mx(_p(a), R, F, _p(h_q), _p(h_sf), _s()), "moe_swiglu_quant_mx")
    return h_q, h_sf


def quantize_rows_mx4(x: torch.Tensor, q=None, sf=None):
    """MXFP4: bf16 [rows, cols] -> (packed e2m1 codes uint8 [rows, cols/2], E8M0 codes uint8 [cols/128, rows, 4])."""
    rows, cols = _arg("quantize_rows_mx4", x, torch.bfloat16, 2).shape
    dev = _dev("quantize_rows_mx4", x)
    px = _ptr("quantize_rows_mx4", x, torch.bfloat16, (rows, cols), dev)
    q = torch.empty(rows, cols // 2, dtype=torch.uint8, device=x.device) if q is None else q
    sf = _scale_buf(MX4, rows, cols, x.device, sf)
    pq = _ptr("quantize_rows_mx4 q", q, torch.uint8, (rows, cols // 2), dev)
    ps = _ptr("quantize_rows_mx4 sf", sf, torch.uint8, (cols // 128, rows, 4), dev)
    if rows:
        check(lib().moe_quantize_rows_mx4(px, rows, cols, pq, ps, _s()), "moe_quantize_rows_mx4")
    return q, sf


def quantize_weights_mx4(w: torch.Tensor):
    """MXFP4 weights: bf16 [E, N, K] -> (codes [E, N, K/2], E8M0 codes [K/128, E*N, 4])."""
    E, N, K = _arg("quantize_weights_mx4", w, torch.bfloat16, 3).shape
    if not w.is_contiguous():
        raise MoEError("quantize_weights_mx4: expected a contiguous tensor")
    q, sf = quantize_rows_mx4(w.view(E * N, K))
    return q.view(E, N, K // 2), sf


def dequantize_rows_mx4(q: torch.Tensor, sf: torch.Tensor, out=None) -> torch.Tensor:
    """MXFP4 codes [rows, cols/2] and scale codes [cols/128, rows, 4] -> their bf16 values [rows, cols]."""
    rows, half = _arg("dequantize_rows_mx4", q, torch.uint8, 2).shape
    cols, dev = 2 * half, _dev("dequantize_rows_mx4", q)
    pq = _ptr("dequantize_rows_mx4", q, torch.uint8, (rows, half), dev)
    ps = _ptr("dequantize_rows_mx4 sf", sf, torch.uint8, (cols // 128, rows, 4), dev)
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device=q.device) if out is None else out
    po = _ptr("dequantize_rows_mx4 out", out, torch.bfloat16, (rows, cols), dev)
    if rows:
        check(lib().moe_dequantize_rows_mx4(pq, ps, rows, cols, po, _s()), "moe_dequantize_rows_mx4")
    return out


def quantize_sort_mx4(x: torch.Tensor, topk_ids: torch.Tensor, E: int, out: Optional[dict] = None):
    """MXFP4 steps 1 + 2: the dict of quantize_sort with xs_q = packed codes [T*k, D/2] and
    xs_scale = E8M0 codes [D/128, T*k, 4]."""
    T, k = _arg("quantize_sort_mx4 topk_ids", topk_ids, torch.int32, 2).shape
    D = _arg("quantize_sort_mx4 x", x, torch.bfloat16, 2).shape[1]
    R, dev, at = T * k, _dev("quantize_sort_mx4", x), x.device
    px = _ptr("quantize_sort_mx4 x", x, torch.bfloat16, (T, D), dev)
    pi = _ptr("quantize_sort_mx4 topk_ids", topk_ids, torch.int32, (T, k), dev)
    o = out if out is not None else {}
    if "sorted_src" not in o:
        o["sorted_src"] = torch.empty(R, dtype=torch.int32, device=at)
        o["pos"] = torch.empty(R, dtype=torch.int32, device=at)
        o["group_sizes"] = torch.empty(E, dtype=torch.int32, device=at)
        o["group_offsets"] = torch.empty(E + 1, dtype=torch.int32, device=at)
        o["xs_q"] = torch.empty(R, D // 2, dtype=torch.uint8, device=at)
        o["xs_scale"] = _scale_buf(MX4, R, D, at)
    p = [_ptr(f"quantize_sort_mx4 {key}", o[key], torch.int32, (n,), dev)
         for key, n in (("sorted_src", R), ("pos", R), ("group_sizes", E), ("group_offsets", E + 1))]
    pq = _ptr("quantize_sort_mx4 xs_q", o["xs_q"], torch.uint8, (R, D // 2), dev)
    ps = _ptr("quantize_sort_mx4 xs_scale", o["xs_scale"], torch.uint8, (D // 128, R, 4), dev)
    if not R:
        o["group_sizes"].zero_()
        o["group_offsets"].zero_()
        return o
    L = lib()
    nws = L.moe_ragged_sort_workspace_bytes(T, k, E)
    ws = o.get("sort_ws")
    if ws is None or ws.numel() < nws:
        ws = o["sort_ws"] = torch.empty(max(nws, 16), dtype=torch.uint8, device=at)
    check(L.moe_quantize_sort_mx4(px, pi, T, k, E, D, *p, pq, ps, ws.data_ptr(), ws.numel(), _s()),
          "moe_quantize_sort_mx4")
    return o


def gmm_mx4(lhs_q, lhs_sf, rhs_q, rhs_sf, group_sizes, group_offset: int = 0, E_local: Optional[int] = None,
            out=None):
    """MXFP4 grouped matmul of packed codes lhs_q [M, K/2] and rhs_q [E_local, N, K/2] -> bf16 [M, N];
    lhs_sf [K/128, M, 4], rhs_sf [K/128, E_local*N, 4]."""
    M, half = _arg("gmm_mx4 lhs_q", lhs_q, torch.uint8, 2).shape
    El, N, _ = _arg("gmm_mx4 rhs_q", rhs_q, torch.uint8, 3).shape
    E = _arg("gmm_mx4 group_sizes", group_sizes, torch.int32, 1).shape[0]
    K, dev = 2 * half, _dev("gmm_mx4", lhs_q)
    if E_local is not None and E_local != El:
        raise MoEError(f"gmm_mx4: E_local is {E_local}, but rhs_q holds {El} experts")
    pl = _ptr("gmm_mx4 lhs_q", lhs_q, torch.uint8, (M, half), dev)
    pls = _ptr("gmm_mx4 lhs_sf", lhs_sf, torch.uint8, (K // 128, M, 4), dev)
    pr = _ptr("gmm_mx4 rhs_q", rhs_q, torch.uint8, (El, N, half), dev)
    prs = _ptr("gmm_mx4 rhs_sf", rhs_sf, torch.uint8, (K // 128, El * N, 4), dev)
    pg = _ptr("gmm_mx4 group_sizes", group_sizes, torch.int32, (E,), dev)
    out = torch.empty(M, N, dtype=torch.bfloat16, device=lhs_q.device) if out is None else out
    po = _ptr("gmm_mx4 out", out, torch.bfloat16, (M, N), dev)
    if M:
        check(lib().gmm_fp4_mx(pl, pls, pr, prs, pg, E, group_offset, El, M, K, N, po, _s()), "gmm_fp4_mx")
    return out


def swiglu_quant_mx4(a: torch.Tensor, h_q=None, h_sf=None):
    """MXFP4 step 4: a = [a0 | a1] bf16 [R, 2F] -> (h codes [R, F/2], h E8M0 codes [F/128, R, 4])."""
    R, F2 = _arg("swiglu_quant_mx4", a, torch.bfloat16, 2).shape
    F, dev = F2 // 2, _dev("swiglu_quant_mx4", a)
    pa = _ptr("swiglu_quant_mx4", a, torch.bfloat16, (R, 2 * F), dev)
    h_q = torch.empty(R, F // 2, dtype=torch.uint8, device=a.device) if h_q is None else h_q
    h_sf = _scale_buf(MX4, R, F, a.device, h_sf)
    pq = _ptr("swiglu_quant_mx4 h_q", h_q, torch.uint8, (R, F // 2), dev)
    ps = _ptr("swiglu_quant_mx4 h_sf", h_sf, torch.uint8, (F // 128, R, 4), dev)
    if R:
        check(lib().moe_swiglu_quant_mx4(pa, R, F, pq, ps, _s()), "moe_swiglu_quant_mx4")
    return h_q, h_sf


def quantize_weights_block(w: torch.Tensor, transposed: bool = False, q=None, s=None, q_t=None, s_t=None):
    """bf16 [E, N, K] -> (e4m3 codes [E, N, K], fp32 scales [E, ceil(N/128), K/128]), one scale for each 128 x 128
    block; with `transposed` also the transposed weights' (codes [E, K, N], scales [E, K/128, N/128]), N % 128 == 0."""
    what = "quantize_weights_block"
    E, N, K = _arg(what, w, torch.bfloat16, 3).shape
    dev, at = _dev(what, w), w.device
    pw = _ptr(what, w, torch.bfloat16, (E, N, K), dev)
    q = torch.empty(E, N, K, dtype=torch.uint8, device=at) if q is None else q
    s = torch.empty(E, _nb(N), K // 128, dtype=torch.float32, device=at) if s is None else s
    pq = _ptr(what + " q", q, torch.uint8, (E, N, K), dev)
    ps = _ptr(what + " s", s, torch.float32, (E, _nb(N), K // 128), dev)
    pqt = pst = None
    if transposed:
        q_t = torch.empty(E, K, N, dtype=torch.uint8, device=at) if q_t is None else q_t
        s_t = torch.empty(E, K // 128, N // 128, dtype=torch.float32, device=at) if s_t is None else s_t
        pqt = _ptr(what + " q_t", q_t, torch.uint8, (E, K, N), dev)
        pst = _ptr(what + " s_t", s_t, torch.float32, (E, K // 128, N // 128), dev)
    check(lib().moe_quantize_weights_block(pw, E, N, K, pq, ps, pqt, pst, _s()), "moe_quantize_weights_block")
    return (q, s, q_t, s_t) if transposed else (q, s)


def gmm_block(lhs_q: torch.Tensor, lhs_s: torch.Tensor, rhs_q: torch.Tensor, rhs_s: torch.Tensor,
              group_sizes: Optional[torch.Tensor] = None, group_offset: int = 0, out=None) -> torch.Tensor:
    """Grouped matmul of codes lhs_q [M, K] (scales lhs_s [M, K/128], as quantize_rows gives them with
    PER_ROW_BLOCK128) and rhs_q [E_local, N, K] (scales rhs_s [E_local, ceil(N/128), K/128], as
    quantize_weights_block gives them) -> bf16 [M, N].  The experts are [group_offset, group_offset + E_local)
    of group_sizes' E; without group_sizes (and with one expert) every row is the expert's: a dense product."""
    what = "gmm_block"
    M, K = _arg("gmm_block lhs_q", lhs_q, torch.uint8, 2).shape
    El, N, _ = _arg("gmm_block rhs_q", rhs_q, torch.uint8, 3).shape
    dev = _dev(what, lhs_q)
    if group_sizes is None:
        E, pg = 1, None
        if El != 1 or group_offset:
            raise MoEError("gmm_block: without group_sizes, rhs_q holds one expert")
    else:
        E = _arg("gmm_block group_sizes", group_sizes, torch.int32, 1).shape[0]
        pg = _ptr("gmm_block group_sizes", group_sizes, torch.int32, (E,), dev)
    pl = _ptr("gmm_block lhs_q", lhs_q, torch.uint8, (M, K), dev)
    pls = _ptr("gmm_block lhs_s", lhs_s, torch.float32, (M, K // 128), dev)
    pr = _ptr("gmm_block rhs_q", rhs_q, torch.uint8, (El, N, K), dev)
    prs = _ptr("gmm_block rhs_s", rhs_s, torch.float32, (El, _nb(N), K // 128), dev)
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
        po = out.data_ptr()
    else:
        po = _ptr("gmm_block out", out, torch.bfloat16, (M, N), dev)
    if M:
        check(_lib().gmm_fp8_block(pl, pls, pr, prs, pg, E, group_offset, El, M, K, N, po, _stream(dev)), "gmm_fp8_block")
    return out


def tgmm_mx_workspace_bytes(M: int, K: int, N: int, E_local: int) -> int:
    """Bytes of tgmm_mx's workspace (0 for a shape that it does not take)."""
    return int(lib().tgmm_fp8_mx_workspace_bytes(M, K, N, E_local))


def tgmm_mx(lhs: torch.Tensor, rhs: torch.Tensor, group_sizes: torch.Tensor, group_offset: int = 0,
            E_local: Optional[int] = None, lhs_rows: Optional[torch.Tensor] = None, k: int = 1, out=None,
            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Weight gradient of a grouped matmul: fp32 [E_local, K, N], the sum over each expert's rows of lhs [M, K]
    times rhs [M, N] (bf16 both), each rounded to e4m3 with a power-of-two scale for every 32 rows of an expert and
    column.  With lhs_rows (int32 [M], sorted_src of a sort of T tokens) row m of the lhs is lhs[lhs_rows[m] // k],
    lhs then being [T, K].  A sum that an infinity enters with a value other than zero is that infinity (NaN where
    both signs meet).  workspace: tgmm_mx_workspace_bytes(M, K, N, E_local) bytes; calls that may overlap on the GPU
    need workspaces of their own."""
    what = "tgmm_mx"
    L, K = _arg("tgmm_mx lhs", lhs, torch.bfloat16, 2).shape
    M, N = _arg("tgmm_mx rhs", rhs, torch.bfloat16, 2).shape
    E = _arg("tgmm_mx group_sizes", group_sizes, torch.int32, 1).shape[0]
    dev = _dev(what, lhs)
    El = E - group_offset if E_local is None else E_local
    if lhs_rows is None and (k != 1 or L != M):
        raise MoEError(f"tgmm_mx: lhs has {L} rows and rhs {M}; lhs_rows picks rows of lhs, k at a time")
    px = _ptr("tgmm_mx lhs", lhs, torch.bfloat16, (L, K), dev)
    pd = _ptr("tgmm_mx rhs", rhs, torch.bfloat16, (M, N), dev)
    pg = _ptr("tgmm_mx group_sizes", group_sizes, torch.int32, (E,), dev)
    pi = None if lhs_rows is None else _ptr("tgmm_mx lhs_rows", lhs_rows, torch.int32, (M,), dev)
    if El <= 0:
        raise MoEError(f"tgmm_mx: E_local is {El}")
    if out is None:
        out = torch.empty(El, K, N, dtype=torch.float32, device=dev)
        po = out.data_ptr()
    else:
        po = _ptr("tgmm_mx out", out, torch.float32, (El, K, N), dev)
    if not M:
        return out.zero_()
    L_ = _lib()
    if workspace is None:
        workspace = torch.empty(max(16, L_.tgmm_fp8_mx_workspace_bytes(M, K, N, El)), dtype=torch.uint8, device=dev)
    pw = _ptr("tgmm_mx workspace", workspace, torch.uint8, (workspace.numel(),), dev)
    check(L_.tgmm_fp8_mx(px, L, pi, k, pd, pg, E, group_offset, El, M, K, N, po, pw, workspace.numel(),
                         _stream(dev)), "tgmm_fp8_mx")
    return out


def gmm(lhs_q, lhs_scale, lhs_mode, rhs_q, rhs_scale, rhs_mode, group_sizes, group_offset: int = 0,
        E_local: Optional[int] = None, out=None):
    """Grouped matmul -> bf16 [M, N]."""
    M, K = lhs_q.shape
    El, N, K2 = rhs_q.shape
    if K2 != K:
        raise MoEError("lhs/rhs K mismatch")
    E = group_sizes.numel()
    E_local = El if E_local is None else E_local
    out = torch.empty(M, N, dtype=torch.bfloat16, device=lhs_q.device) if out is None else out
    check(lib().gmm_fp8(_p(lhs_q), _p(lhs_scale), lhs_mode, _p(rhs_q), _p(rhs_scale), rhs_mode, _p(group_sizes),
                        E, group_offset, E_local, M, K, N, _p(out), _s()), "gmm_fp8")
    return out


def gmm_w8(lhs_q, lhs_scale, lhs_mode, rhs_q, rhs_scale, rhs_mode, group_sizes, group_offset: int = 0,
           E_local: Optional[int] = None, out=None, workspace=None):
    """Grouped matmul with int8 weights rhs_q [E_local, N, K] -> bf16 [M, N].

    workspace: optional uint8 device buffer of gmm_w8_workspace_bytes(M, K)
    bytes or more; with it the activations are decoded to f16 there first
    (the same result, faster where the tensor pipe binds)."""
    M, K = lhs_q.shape
    El, N, K2 = rhs_q.shape
    if K2 != K:
        raise MoEError("lhs/rhs K mismatch")
    if rhs_q.dtype != torch.int8:
        raise MoEError("gmm_w8 takes int8 weight codes")
    E = group_sizes.numel()
    E_local = El if E_local is None else E_local
    out = torch.empty(M, N, dtype=torch.bfloat16, device=lhs_q.device) if out is None else out
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(lib().gmm_fp8_w8(_p(lhs_q), _p(lhs_scale), lhs_mode, _p(rhs_q), _p(rhs_scale), rhs_mode,
                           _p(group_sizes), E, group_offset, E_local, M, K, N, _p(out), _p(workspace), ws_bytes,
                           _s()), "gmm_fp8_w8")
    return out


def gmm_w8_workspace_bytes(M: int, K: int) -> int:
    return int(lib().gmm_fp8_w8_workspace_bytes(M, K))


def gmm_ksplit(lhs_q, lhs_scale, lhs_mode, rhs_q, rhs_scale2, K_split: int, group_sizes, group_offset: int = 0,
               E_local: Optional[int] = None, out=None):
    """Grouped matmul over two K segments with one static weight scale each
    (rhs_scale2 = [s0, s1]) -> bf16 [M, N]."""
    M, K = lhs_q.shape
    El, N, K2 = rhs_q.shape
    if K2 != K:
        raise MoEError("lhs/rhs K mismatch")
    E = group_sizes.numel()
    E_local = El if E_local is None else E_local
    out = torch.empty(M, N, dtype=torch.bfloat16, device=lhs_q.device) if out is None else out
    check(lib().gmm_fp8_ksplit(_p(lhs_q), _p(lhs_scale), lhs_mode, _p(rhs_q), _p(rhs_scale2), K_split,
                               _p(group_sizes), E, group_offset, E_local, M, K, N, _p(out), _s()), "gmm_fp8_ksplit")
    return out


def gmm_swiglu(lhs_q, lhs_scale, lhs_mode, rhs_q, rhs_scale, rhs_mode, group_sizes, h_mode: int,
               h_static: Optional[torch.Tensor] = None, group_offset: int = 0, E_local: Optional[int] = None,
               keep_a: bool = False, a_out=None, h=None, h_q=None, h_scale=None):
    """gmm with [wi_0 | wi_1] fused with SwiGLU and the requantisation of h.

    Returns (h_q uint8 [M, F], h_scale or None, a [M, 2F] bf16 or None)."""
    M, K = lhs_q.shape
    El, F2, K2 = rhs_q.shape
    if K2 != K:
        raise MoEError("lhs/rhs K mismatch")
    F = F2 // 2
    dev = lhs_q.device
    E = group_sizes.numel()
    E_local = El if E_local is None else E_local
    h_q = torch.empty(M, F, dtype=torch.uint8, device=dev) if h_q is None else h_q
    h_scale = _scale_buf(h_mode, M, F, dev, h_scale)
    if h_mode == PER_ROW and h is None:
        h = torch.empty(M, F, dtype=torch.bfloat16, device=dev)
    if keep_a and a_out is None:
        a_out = torch.empty(M, F2, dtype=torch.bfloat16, device=dev)
    check(lib().gmm_fp8_swiglu(_p(lhs_q), _p(lhs_scale), lhs_mode, _p(rhs_q), _p(rhs_scale), rhs_mode,
                               _p(group_sizes), E, group_offset, E_local, M, K, F, h_mode, _p(h_static), _p(a_out),
                               _p(h), _p(h_q), _p(h_scale), _s()), "gmm_fp8_swiglu")
    return h_q, h_scale, a_out


def swiglu_fusable(act_mode: int, w_mode: int, F: int) -> bool:
    """gmm_fp8_swiglu covers every operand scale mode (per row, per row and
    128 columns, per tensor) when F % 128 == 0."""
    modes = (PER_ROW, PER_ROW_BLOCK128, PER_TENSOR)
    return act_mode in modes and w_mode in modes and F % 128 == 0


def swiglu_fuse_pays(act_mode: int, w_mode: int, F: int) -> bool:
    """Whether the forward runs steps 3 and 4 as one gmm_fp8_swiglu call.

    With a blockwise operand scale the contraction's epilogue is already the
    bound (it folds every 128-wide K block into fp32 registers), and the
    SwiGLU tail cannot overlap the next tile there, so gmm_fp8 followed by
    moe_swiglu_quant is faster (measured on the DeepSeek-V3-shaped layer:
    5.1 + 0.4 ms against 6.0 ms); the two are bit-identical."""
    blockwise = act_mode == PER_ROW_BLOCK128 or w_mode == PER_ROW_BLOCK128
    return swiglu_fusable(act_mode, w_mode, F) and not blockwise


def swiglu_quant(a: torch.Tensor, mode: int, static_scale: Optional[torch.Tensor] = None, h_q=None, h_scale=None):
    R, F2 = a.shape
    F = F2 // 2
    h_q = torch.empty(R, F, dtype=torch.uint8, device=a.device) if h_q is None else h_q
    h_scale = _scale_buf(mode, R, F, a.device, h_scale)
    check(lib().moe_swiglu_quant(_p(a), R, F, mode, _p(static_scale), _p(h_q), _p(h_scale), _s()),
          "moe_swiglu_quant")
    return h_q, h_scale


def ragged_gather_reduce(rows: torch.Tensor, pos: torch.Tensor, weights: Optional[torch.Tensor], k: int,
                         out=None):
    R, D = rows.shape
    T = R // k
    out = torch.empty(T, D, dtype=torch.bfloat16, device=rows.device) if out is None else out
    check(lib().ragged_gather_reduce(_p(rows), _p(pos), _p(weights), T, k, D, _p(out), _s()),
          "ragged_gather_reduce")
    return out


def gather_scale_quant(G: torch.Tensor, w: Optional[torch.Tensor], sorted_src: torch.Tensor, k: int):
    T, D = G.shape
    R = T * k
    dev = G.device
    dO = torch.empty(R, D, dtype=torch.bfloat16, device=dev)
    dO_q = torch.empty(R, D, dtype=torch.uint8, device=dev)
    dO_s = torch.empty(R, dtype=torch.float32, device=dev)
    check(lib().moe_gather_scale_quant(_p(G), _p(w), _p(sorted_src), T, k, D, _p(dO), _p(dO_q), _p(dO_s), _s()),
          "moe_gather_scale_quant")
    return dO, dO_q, dO_s


def swiglu_bwd_quant(dH: torch.Tensor, a: torch.Tensor):
    R, F = dH.shape
    dev = dH.device
    dA = torch.empty(R, 2 * F, dtype=torch.bfloat16, device=dev)
    dA_q = torch.empty(R, 2 * F, dtype=torch.uint8, device=dev)
    dA_s = torch.empty(R, dtype=torch.float32, device=dev)
    check(lib().moe_swiglu_bwd_quant(_p(dH), _p(a), R, F, _p(dA), _p(dA_q), _p(dA_s), _s()), "moe_swiglu_bwd_quant")
    return dA, dA_q, dA_s


def gather_scale_quant_block(G: torch.Tensor, w: Optional[torch.Tensor], sorted_src: torch.Tensor, k: int):
    """gather_scale_quant with one scale per row and 128 columns: (dO bf16 [T*k, D], codes, scales [T*k, D/128])."""
    what = "gather_scale_quant_block"
    T, D = _arg(what, G, torch.bfloat16, 2).shape
    R, dev, at = T * k, _dev(what, G), G.device
    pG = _ptr(what, G, torch.bfloat16, (T, D), dev)
    if w is not None and w.numel() != R:
        raise MoEError(f"{what} w: expected {R} values, got {list(w.shape)}")
    pw = None if w is None else _ptr(what + " w", w, torch.float32, w.shape, dev)
    ps = _ptr(what + " sorted_src", sorted_src, torch.int32, (R,), dev)
    dO = torch.empty(R, D, dtype=torch.bfloat16, device=at)
    dO_q = torch.empty(R, D, dtype=torch.uint8, device=at)
    dO_s = torch.empty(R, D // 128, dtype=torch.float32, device=at)
    if R:
        check(lib().moe_gather_scale_quant_block(pG, pw, ps, T, k, D, dO.data_ptr(), dO_q.data_ptr(), dO_s.data_ptr(),
                                                 _s()), "moe_gather_scale_quant_block")
    return dO, dO_q, dO_s


def swiglu_bwd_quant_block(dH: torch.Tensor, a: torch.Tensor):
    """swiglu_bwd_quant with one scale per row and 128 columns, and h = bf16(silu(a0) a1):
    (dA bf16 [R, 2F], codes, scales [R, 2F/128], h bf16 [R, F])."""
    what = "swiglu_bwd_quant_block"
    R, F = _arg(what, dH, torch.bfloat16, 2).shape
    dev, at = _dev(what, dH), dH.device
    pd = _ptr(what, dH, torch.bfloat16, (R, F), dev)
    pa = _ptr(what + " a", a, torch.bfloat16, (R, 2 * F), dev)
    dA = torch.empty(R, 2 * F, dtype=torch.bfloat16, device=at)
    dA_q = torch.empty(R, 2 * F, dtype=torch.uint8, device=at)
    dA_s = torch.empty(R, 2 * F // 128, dtype=torch.float32, device=at)
    h = torch.empty(R, F, dtype=torch.bfloat16, device=at)
    if R:
        check(lib().moe_swiglu_bwd_quant_block(pd, pa, R, F, dA.data_ptr(), dA_q.data_ptr(), dA_s.data_ptr(),
                                               h.data_ptr(), _s()), "moe_swiglu_bwd_quant_block")
    return dA, dA_q, dA_s, h


def quantize_group_cols(g: torch.Tensor, group_sizes: torch.Tensor, group_offset: int = 0,
                        E_local: Optional[int] = None, scales_only: bool = False):
    """Per-(expert, column) e4m3 codes and scales of g; (None, scales) with scales_only."""
    M, N = g.shape
    E = group_sizes.numel()
    E_local = E - group_offset if E_local is None else E_local
    # rows of other experts stay unwritten
    q = None if scales_only else torch.empty(M, N, dtype=torch.uint8, device=g.device)
    s = torch.empty(E_local, N, dtype=torch.float32, device=g.device)
    check(lib().moe_quantize_group_cols(_p(g), M, N, _p(group_sizes), E, group_offset, E_local, _p(q), _p(s), _s()),
          "moe_quantize_group_cols")
    return q, s


def tgmm(lhs_q, lhs_scale, lhs_mode, rhs_q, rhs_scale, rhs_mode, group_sizes, group_offset: int = 0,
         E_local: Optional[int] = None, out=None, workspace=None):
    """Transposed grouped matmul -> fp32 [E_local, K, N]."""
    M, K = lhs_q.shape
    M2, N = rhs_q.shape
    if M2 != M:
        raise MoEError("lhs/rhs M mismatch")
    E = group_sizes.numel()
    E_local = E - group_offset if E_local is None else E_local
    out = torch.empty(E_local, K, N, dtype=torch.float32, device=lhs_q.device) if out is None else out
    nws = lib().tgmm_fp8_workspace_bytes(M, K, N, E_local)
    if workspace is None or workspace.numel() < nws:
        workspace = torch.empty(nws, dtype=torch.uint8, device=lhs_q.device)
    check(lib().tgmm_fp8(_p(lhs_q), _p(lhs_scale), lhs_mode, _p(rhs_q), _p(rhs_scale), rhs_mode, _p(group_sizes), E,
                         group_offset, E_local, M, K, N, _p(out), _p(workspace), workspace.numel(), _s()), "tgmm_fp8")
    return out


def tgmm_gcq(lhs_q, lhs_scale, lhs_mode, rhs_g, rhs_scale, group_sizes, group_offset: int = 0,
             E_local: Optional[int] = None, out=None, workspace=None):
    """tgmm with the rhs as a bf16 gradient and its per-(expert, column) scales
    -> fp32 [E_local, K, N] (the codes are made in the contraction's layout)."""
    M, K = lhs_q.shape
    M2, N = rhs_g.shape
    if M2 != M:
        raise MoEError("lhs/rhs M mismatch")
    E = group_sizes.numel()
    E_local = E - group_offset if E_local is None else E_local
    out = torch.empty(E_local, K, N, dtype=torch.float32, device=lhs_q.device) if out is None else out
    nws = lib().tgmm_fp8_workspace_bytes(M, K, N, E_local)
    if workspace is None or workspace.numel() < nws:
        workspace = torch.empty(nws, dtype=torch.uint8, device=lhs_q.device)
    check(lib().tgmm_fp8_gcq(_p(lhs_q), _p(lhs_scale), lhs_mode, _p(rhs_g), _p(rhs_scale), _p(group_sizes), E,
                             group_offset, E_local, M, K, N, _p(out), _p(workspace), workspace.numel(), _s()),
          "tgmm_fp8_gcq")
    return out


def router_topk(x: torch.Tensor, w_gate: torch.Tensor, k: int):
    """Gate layer + softmax top-k: (logits fp32 [T, E], ids int32 [T, k], w fp32 [T, k])."""
    T, D = x.shape
    E = w_gate.shape[0]
    dev = x.device
    logits = torch.empty(T, E, dtype=torch.float32, device=dev)
    ids = torch.empty(T, k, dtype=torch.int32, device=dev)
    w = torch.empty(T, k, dtype=torch.float32, device=dev)
    check(lib().moe_router_topk(_p(x), _p(w_gate), T, D, E, k, _p(logits), _p(ids), _p(w), _s()), "moe_router_topk")
    return logits, ids, w


@dataclasses.dataclass
class BalanceLoss:
    """What router_balance_loss computed, and what its gradient needs."""
    loss: torch.Tensor    # fp32 [1]
    counts: torch.Tensor  # int32 [seqs, E]: pairs of valid rows routed to each expert
    mean: torch.Tensor    # fp32 [seqs, E]: mean probability over valid rows
    state: torch.Tensor   # the call's workspace, its last words the sequences' valid rows
    k: int
    coef: float
    valid: Optional[torch.Tensor] = None

    @property
    def tokens(self) -> torch.Tensor:
        """int32 [seqs]: valid rows."""
        return self.state.view(torch.int32)[-self.counts.shape[0]:]


@functools.lru_cache(maxsize=256)
def _balance_workspace(T: int, E: int, k: int, seqs: int) -> int:
    return int(lib().moe_router_balance_workspace_bytes(T, E, k, seqs))


def router_balance_loss(logits: torch.Tensor, topk_ids: torch.Tensor, coef: float = 1.0, seqs: int = 1,
                        valid: Optional[torch.Tensor] = None) -> BalanceLoss:
    """Balance loss of router logits fp32 [T, E] and their choices int32 [T, k], the T rows being `seqs` sequences
    of equal length: coef times the mean over sequences of sum_e (E counts_e / (k n)) mean_e, with n the
    sequence's valid rows.  valid: bool [T]; a row that is not counts nowhere (padding), whatever it holds."""
    what = "router_balance_loss"
    T, E = _arg("router_balance_loss logits", logits, torch.float32, 2).shape
    k = _arg("router_balance_loss topk_ids", topk_ids, torch.int32, 2).shape[1]
    dev = _dev(what, logits)
    pl = _ptr("router_balance_loss logits", logits, torch.float32, (T, E), dev)
    pi = _ptr("router_balance_loss topk_ids", topk_ids, torch.int32, (T, k), dev)
    pv = None if valid is None else _ptr("router_balance_loss valid", valid, torch.bool, (T,), dev)
    nws = _balance_workspace(T, E, k, seqs)
    if not nws:
        raise MoEError(f"router_balance_loss does not take T = {T}, E = {E}, k = {k}, seqs = {seqs}")
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    counts = torch.empty(seqs, E, dtype=torch.int32, device=dev)
    mean = torch.empty(seqs, E, dtype=torch.float32, device=dev)
    state = torch.empty(nws + 4 * seqs, dtype=torch.uint8, device=dev)
    ws = state.data_ptr()
    check(_lib().moe_router_balance(pl, pi, pv, T, E, k, seqs, coef, loss.data_ptr(), counts.data_ptr(),
                                    mean.data_ptr(), ws + nws, ws, nws, _stream(dev)), "moe_router_balance")
    return BalanceLoss(loss, counts, mean, state, k, coef, valid)


def router_balance_loss_backward(logits: torch.Tensor, b: BalanceLoss, grad: Optional[torch.Tensor] = None,
                                 out=None) -> torch.Tensor:
    """Gradient of router_balance_loss in the logits it was given, fp32 [T, E] (zero in rows that are not valid);
    grad: fp32 [1], the loss's own gradient (None: 1).  Counts are constants.  router_backward takes it as
    dlogits_aux."""
    what = "router_balance_loss_backward"
    T, E = _arg("router_balance_loss_backward logits", logits, torch.float32, 2).shape
    seqs, dev = b.counts.shape[0], _dev(what, logits)
    pl = _ptr("router_balance_loss_backward logits", logits, torch.float32, (T, E), dev)
    pc = _ptr("router_balance_loss_backward counts", b.counts, torch.int32, (seqs, E), dev)
    ns = b.state.numel()
    pt = _ptr(what + " state", b.state, torch.uint8, (ns,), dev) + ns - 4 * seqs
    pv = None if b.valid is None else _ptr("router_balance_loss_backward valid", b.valid, torch.bool, (T,), dev)
    pg = None if grad is None else _ptr("router_balance_loss_backward grad", grad, torch.float32, (1,), dev)
    if out is None:
        out = torch.empty(T, E, dtype=torch.float32, device=dev)
        po = out.data_ptr()
    else:
        po = _ptr("router_balance_loss_backward out", out, torch.float32, (T, E), dev)
    check(_lib().moe_router_balance_backward(pl, pv, T, E, b.k, seqs, b.coef, pc, pt, pg, po, _stream(dev)),
          "moe_router_balance_backward")
    return out


def router_backward(G: torch.Tensor, o: torch.Tensor, pos: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor,
                    logits: torch.Tensor, ids: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                    dlogits_aux: Optional[torch.Tensor] = None):
    """Router gradient: (dw fp32 [T, k], dlogits bf16 [T, E], grad_gate fp32 [E, D], state_grad bf16 [T, D]).
    dlogits_aux: fp32 [T, E], another loss's gradient in the logits (router_balance_loss_backward), added to theirs."""
    T, D = x.shape
    E = w_gate.shape[0]
    k = ids.shape[1]
    dev = x.device
    dw = torch.empty(T, k, dtype=torch.float32, device=dev)
    dl = torch.empty(T, E, dtype=torch.bfloat16, device=dev)
    gg = torch.empty(E, D, dtype=torch.float32, device=dev)
    sg = torch.empty(T, D, dtype=torch.bfloat16, device=dev)
    nws = lib().moe_router_backward_workspace_bytes(T, D, E)
    if workspace is None or workspace.numel() < nws:
        workspace = torch.empty(max(nws, 16), dtype=torch.uint8, device=dev)
    aux = None if dlogits_aux is None else _ptr("router_backward dlogits_aux", dlogits_aux, torch.float32, (T, E),
                                                _dev("router_backward", x))
    check(lib().moe_router_backward_aux(_p(G), _p(o), _p(pos), _p(x), _p(w_gate), _p(logits), _p(ids), aux, T, D, E, k,
                                        _p(dw), _p(dl), _p(gg), _p(sg), _p(workspace), workspace.numel(), _s()),
          "moe_router_backward")
    return dw, dl, gg, sg


def transpose_u8(x: torch.Tensor) -> torch.Tensor:
    """Batched byte transpose [B, R, C] -> [B, C, R] (weight layout preparation)."""
    B, R, C = x.shape
    out = torch.empty(B, C, R, dtype=torch.uint8, device=x.device)
    check(lib().moe_transpose_u8(_p(x), B, R, C, _p(out), _s()), "moe_transpose_u8")
    return out


# ---------------------------------------------------------------------------
# The expert FFN
# ---------------------------------------------------------------------------

@dataclasses.dataclass
class ExpertWeights:
    """Pre-quantised expert weights in the device layout.

    w_in  [E, 2F, D] codes (wi_0 rows, then wi_1 rows), scales per in_mode;
    w_out [E, D, F] codes, scales per out_mode.  For the backward pass the
    transposed codes w_in_t [E, D, 2F] and w_out_t [E, F, D] are kept too."""
    w_in: torch.Tensor
    s_in: torch.Tensor
    in_mode: int
    w_out: torch.Tensor
    s_out: torch.Tensor
    out_mode: int
    w_in_t: Optional[torch.Tensor] = None
    s_in_t: Optional[torch.Tensor] = None
    w_out_t: Optional[torch.Tensor] = None
    s_in_split: Optional[torch.Tensor] = None  # [s_w0, s_w1]: the two K halves of w_in_t
    s_out_t: Optional[torch.Tensor] = None  # PER_BLOCK128: the block scales of w_out_t


def prepare_weights(w_in: torch.Tensor, w_out: torch.Tensor, w_mode: int, static: Optional[dict] = None,
                    for_backward: bool = False) -> ExpertWeights:
    """Quantise the bf16 expert weights once (outside the timed FFN).

    Static scheme: wi_0, wi_1 and wo each carry one fixed scale; the wi_0 |
    wi_1 concatenation then has a per-channel scale vector.  The backward pass takes
    PER_TENSOR (static) or PER_BLOCK128 weights."""
    dev = w_in.device
    E, F2, D = w_in.shape
    F = F2 // 2
    if w_mode == PER_BLOCK128:
        if not for_backward:
            qin, sin = quantize_weights_block(w_in)
            qo, so = quantize_weights_block(w_out)
            return ExpertWeights(qin, sin, PER_BLOCK128, qo, so, PER_BLOCK128)
        if D % 128 != 0 or F % 128 != 0:
            raise MoEError("the backward pass needs D % 128 == 0 and F % 128 == 0")
        qin, sin, qin_t, sin_t = quantize_weights_block(w_in, transposed=True)
        qo, so, qo_t, so_t = quantize_weights_block(w_out, transposed=True)
        return ExpertWeights(qin, sin, PER_BLOCK128, qo, so, PER_BLOCK128, w_in_t=qin_t, s_in_t=sin_t, w_out_t=qo_t,
                             s_out_t=so_t)
    if w_mode == MX32:
        qin, sin = quantize_weights_mx(w_in)
        qo, so = quantize_weights_mx(w_out)
        return ExpertWeights(qin, sin, MX32, qo, so, MX32)
    if w_mode == MX4:
        qin, sin = quantize_weights_mx4(w_in)
        qo, so = quantize_weights_mx4(w_out)
        return ExpertWeights(qin, sin, MX4, qo, so, MX4)
    if w_mode == PER_TENSOR:
        s0 = torch.tensor([static["w0"]], dtype=torch.float32, device=dev)
        s1 = torch.tensor([static["w1"]], dtype=torch.float32, device=dev)
        so = torch.tensor([static["wo"]], dtype=torch.float32, device=dev)
        q0, _ = quantize_weights(w_in[:, :F].contiguous(), PER_TENSOR, s0)
        q1, _ = quantize_weights(w_in[:, F:].contiguous(), PER_TENSOR, s1)
        qin = torch.cat([q0, q1], dim=1).contiguous()
        sin = torch.empty(E, F2, dtype=torch.float32, device=dev)
        sin[:, :F] = static["w0"]
        sin[:, F:] = static["w1"]
        qo, _ = quantize_weights(w_out, PER_TENSOR, so)
        W = ExpertWeights(qin, sin, PER_ROW, qo, so, PER_TENSOR)
        if for_backward:
            if F2 % 128 != 0 or F % 128 != 0:
                raise MoEError("the backward pass needs F % 128 == 0")
            W.w_in_t = transpose_u8(qin)
            nb = F2 // 128
            st = torch.empty(E, nb, D, dtype=torch.float32, device=dev)
            st[:, : F // 128] = static["w0"]
            st[:, F // 128:] = static["w1"]
            W.s_in_t = st
            W.s_in_split = torch.tensor([static["w0"], static["w1"]], dtype=torch.float32, device=dev)
            W.w_out_t = transpose_u8(qo)
        return W
    qin, sin = quantize_weights(w_in, w_mode)
    qo, so = quantize_weights(w_out, w_mode)
    return ExpertWeights(qin, sin, w_mode, qo, so, w_mode)


def prepare_weights_w8(w_in: torch.Tensor, w_out: torch.Tensor, w_mode: int) -> ExpertWeights:
    """int8 expert weights (per channel or blockwise), quantised once outside
    the timed FFN; ffn_forward then runs both contractions with gmm_w8."""
    if w_mode not in (PER_ROW, PER_ROW_BLOCK128):
        raise MoEError("int8 weights take per-channel or blockwise scales")
    qin, sin = quantize_weights_int8(w_in, w_mode)
    qo, so = quantize_weights_int8(w_out, w_mode)
    return ExpertWeights(qin, sin, w_mode, qo, so, w_mode)


def decode_weights(W: ExpertWeights) -> ExpertWeights:
    """PER_BLOCK128 weights as ffn_decode takes them: the same codes, each block's scale repeated for its 128
    channels ([E, K/128, N], a 32nd of the codes' bytes).  To be made once, as prepare_weights' result is."""
    if W.in_mode != PER_BLOCK128:
        raise MoEError("decode_weights: expected PER_BLOCK128 weights")
    wide = lambda s, N: s.transpose(1, 2).repeat_interleave(128, 2)[..., :N].contiguous()  # noqa: E731
    return ExpertWeights(W.w_in, wide(W.s_in, W.w_in.shape[1]), PER_ROW_BLOCK128, W.w_out,
                         wide(W.s_out, W.w_out.shape[1]), PER_ROW_BLOCK128)


class FFNBuffers:
    """Every intermediate of one forward (and backward) pass, allocated once."""

    def __init__(self, T, D, E, k, F, act_mode, device, backward=False):
        R = T * k
        f = lambda *s, dt=torch.uint8: torch.empty(*s, dtype=dt, device=device)
        self.T, self.D, self.E, self.k, self.F, self.act_mode = T, D, E, k, F, act_mode
        self.x_q = f(T, D)
        self.x_s = _scale_buf(act_mode, T, D, device)
        self.sort = {}
        self.a = f(R, 2 * F, dt=torch.bfloat16)
        self.h = f(R, F, dt=torch.bfloat16)  # scratch of the fused per-row path
        self.keep_a = backward
        self.h_q = f(R, F // 2 if act_mode == MX4 else F)
        self.h_s = _scale_buf(act_mode, R, F, device)
        self.o = f(R, D, dt=torch.bfloat16)
        self.y = f(T, D, dt=torch.bfloat16)
        self._w8_ws = None
        self._tgmm_ws = None
        if backward:
            self.dH = f(R, F, dt=torch.bfloat16)
            self.dXs = f(R, D, dt=torch.bfloat16)
            self.dX = f(T, D, dt=torch.bfloat16)

    def w8_workspace(self) -> torch.Tensor:
        """The int8-weight contractions' f16 activation workspace, allocated on
        first use: 2 bytes per element of the larger of their two lhs,
        [T*k, D] and [T*k, F]."""
        if self._w8_ws is None:
            n = gmm_w8_workspace_bytes(self.T * self.k, max(self.D, self.F))
            self._w8_ws = torch.empty(n, dtype=torch.uint8, device=self.y.device)
        return self._w8_ws

    def tgmm_workspace(self, E: int) -> torch.Tensor:
        """tgmm_mx's workspace for either weight gradient of E experts, allocated on first use (and again for
        more experts)."""
        R = self.T * self.k
        n = max(tgmm_mx_workspace_bytes(R, self.D, 2 * self.F, E), tgmm_mx_workspace_bytes(R, self.F, self.D, E), 16)
        if self._tgmm_ws is None or self._tgmm_ws.numel() < n:
            self._tgmm_ws = torch.empty(n, dtype=torch.uint8, device=self.y.device)
        return self._tgmm_ws

    def check(self, what: str, W: "ExpertWeights", topk_w: Optional[torch.Tensor], T: int, k: int):
        """Refuse a call of T tokens and k choices, or weights, that these buffers were not made for."""
        if T != self.T or k != self.k:
            raise MoEError(f"{what}: the buffers were made for {self.T} tokens of {self.k} experts, got {T} of {k}")
        half = 2 if W.in_mode == MX4 else 1
        E, D, F = W.w_in.shape[0], self.D, self.F
        if W.w_in.shape != (E, 2 * F, D // half) or W.w_out.shape != (E, D, F // half):
            raise MoEError(f"{what}: the buffers were made for D = {D} and F = {F}, got weights {list(W.w_in.shape)} "
                           f"and {list(W.w_out.shape)}")
        if topk_w is not None and (topk_w.dtype is not torch.float32 or topk_w.numel() != T * k):
            raise MoEError(f"{what} topk_w: expected {torch.float32} {[T, k]}, got {topk_w.dtype} {list(topk_w.shape)}")


def ffn_forward(x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor, W: ExpertWeights, act_mode: int,
                buf: FFNBuffers, static_x: Optional[torch.Tensor] = None,
                static_h: Optional[torch.Tensor] = None, fuse_swiglu: bool = True,
                fuse_quant_sort: bool = True) -> torch.Tensor:
    """One forward pass of the expert FFN; returns buf.y (bf16 [T, D]).

    Steps 1 and 2 run as one call (moe_quantize_sort; buf.x_q / buf.x_s are
    then not written), and where the scale modes allow it steps 3 and 4 run as
    one fused kernel (gmm_fp8_swiglu, bit-identical to gmm_fp8 +
    moe_swiglu_quant); buf.a then holds a only when the buffers were made for
    a backward pass.  Buffers made for another shape or scale mode are refused."""
    E = W.w_in.shape[0]
    T, k = _arg("ffn_forward topk_ids", topk_ids, torch.int32, 2).shape
    if x.dtype is not torch.bfloat16 or x.shape != (T, buf.D):
        raise MoEError(f"ffn_forward x: expected {torch.bfloat16} {[T, buf.D]}, got {x.dtype} {list(x.shape)}")
    buf.check("ffn_forward", W, topk_w, T, k)
    if act_mode != buf.act_mode and (act_mode != PER_TENSOR or buf.act_mode == MX4):
        raise MoEError(f"ffn_forward: the buffers were made for scale mode {buf.act_mode}, got {act_mode}")
    if act_mode == MX32:
        if W.in_mode != MX32:
            raise MoEError("the MXFP8 forward needs MXFP8 weights")
        s = quantize_sort_mx(x, topk_ids, E, out=buf.sort)
        if fuse_swiglu and buf.F % 128 == 0:
            gmm_mx_swiglu(s["xs_q"], s["xs_scale"], W.w_in, W.s_in, s["group_sizes"],
                          a_out=buf.a if buf.keep_a else None, h_q=buf.h_q, h_sf=buf.h_s)
        else:
            gmm_mx(s["xs_q"], s["xs_scale"], W.w_in, W.s_in, s["group_sizes"], out=buf.a)
            swiglu_quant_mx(buf.a, h_q=buf.h_q, h_sf=buf.h_s)
        gmm_mx(buf.h_q, buf.h_s, W.w_out, W.s_out, s["group_sizes"], out=buf.o)
        ragged_gather_reduce(buf.o, s["pos"], topk_w, k, out=buf.y)
        return buf.y
    if act_mode == MX4:
        if W.in_mode != MX4:
            raise MoEError("the MXFP4 forward needs MXFP4 weights")
        s = quantize_sort_mx4(x, topk_ids, E, out=buf.sort)
        gmm_mx4(s["xs_q"], s["xs_scale"], W.w_in, W.s_in, s["group_sizes"], out=buf.a)
        swiglu_quant_mx4(buf.a, h_q=buf.h_q, h_sf=buf.h_s)
        gmm_mx4(buf.h_q, buf.h_s, W.w_out, W.s_out, s["group_sizes"], out=buf.o)
        ragged_gather_reduce(buf.o, s["pos"], topk_w, k, out=buf.y)
        return buf.y
    if W.in_mode == PER_BLOCK128:
        if act_mode != PER_ROW_BLOCK128:
            raise MoEError("PER_BLOCK128 weights take PER_ROW_BLOCK128 activations")
        s = quantize_sort(x, topk_ids, E, act_mode, out=buf.sort)
        gmm_block(s["xs_q"], s["xs_scale"], W.w_in, W.s_in, s["group_sizes"], out=buf.a)
        swiglu_quant(buf.a, act_mode, h_q=buf.h_q, h_scale=buf.h_s)
        gmm_block(buf.h_q, buf.h_s, W.w_out, W.s_out, s["group_sizes"], out=buf.o)
        ragged_gather_reduce(buf.o, s["pos"], topk_w, k, out=buf.y)
        return buf.y
    if W.in_mode == MX4:
        raise MoEError("MXFP4 weights take MXFP4 activations (act_mode MX4)")
    w8 = W.w_in.dtype == torch.int8
    if w8 and act_mode not in (PER_ROW, PER_TENSOR):
        raise MoEError("int8 weights take per-token or static activation scales")
    if fuse_quant_sort:
        s = quantize_sort(x, topk_ids, E, act_mode, static_x, out=buf.sort)
    else:
        quantize_rows(x, act_mode, static_x, q=buf.x_q, scale=buf.x_s)
        s = ragged_sort(topk_ids, E, buf.x_q, buf.x_s if act_mode != PER_TENSOR else static_x, act_mode,
                        out=buf.sort)
    xs_s = s["xs_scale"] if act_mode != PER_TENSOR else static_x
    if w8:
        ws = buf.w8_workspace()
        gmm_w8(s["xs_q"], xs_s, act_mode, W.w_in, W.s_in, W.in_mode, s["group_sizes"], out=buf.a, workspace=ws)
        swiglu_quant(buf.a, act_mode, static_h, h_q=buf.h_q, h_scale=buf.h_s)
    elif fuse_swiglu and swiglu_fuse_pays(act_mode, W.in_mode, buf.F):
        gmm_swiglu(s["xs_q"], xs_s, act_mode, W.w_in, W.s_in, W.in_mode, s["group_sizes"], act_mode, static_h,
                   a_out=buf.a if buf.keep_a else None, h=buf.h, h_q=buf.h_q, h_scale=buf.h_s)
    else:
        gmm(s["xs_q"], xs_s, act_mode, W.w_in, W.s_in, W.in_mode, s["group_sizes"], out=buf.a)
        swiglu_quant(buf.a, act_mode, static_h, h_q=buf.h_q, h_scale=buf.h_s)
    h_s = buf.h_s if act_mode != PER_TENSOR else static_h
    if w8:
        gmm_w8(buf.h_q, h_s, act_mode, W.w_out, W.s_out, W.out_mode, s["group_sizes"], out=buf.o, workspace=ws)
    else:
        gmm(buf.h_q, h_s, act_mode, W.w_out, W.s_out, W.out_mode, s["group_sizes"], out=buf.o)
    ragged_gather_reduce(buf.o, s["pos"], topk_w, k, out=buf.y)
    return buf.y


class DecodeBuffers:
    """The output and the workspace of ffn_decode for up to T tokens, allocated once.

    They may be used on any stream at once: the constructor waits until the
    workspace is zero (not while the current stream is captured, and not with
    `settle` false; it is then zero in the current stream's order).
    After a step that timed out (device_error() & 0x4) the workspace holds what
    that step left, and every step on it reports the error until reset()."""

    def __init__(self, T, D, E, k, F, device, settle: bool = True):
        self.T, self.D, self.E, self.k, self.F = T, D, E, k, F
        n = int(lib().moe_ffn_decode_workspace_bytes(T, k, D, F))
        if not n:
            raise MoEError(f"ffn_decode does not take T = {T}, k = {k}, D = {D}, F = {F}")
        self.y = torch.empty(T, D, dtype=torch.bfloat16, device=device)
        self.ws = torch.zeros(n, dtype=torch.uint8, device=device)  # (its counters have to start at zero)
        self.ws_bytes = n
        if settle and self.ws.is_cuda:
            with torch.cuda.device(self.ws.device):
                if not torch.cuda.is_current_stream_capturing():
                    torch.cuda.current_stream().synchronize()

    def reset(self):
        """Zero the workspace, in the current stream's order, after a step that timed out."""
        self.ws.zero_()


def ffn_decode(x: torch.Tensor, topk_ids: torch.Tensor, topk_w: Optional[torch.Tensor], W: ExpertWeights,
               buf: Optional[DecodeBuffers] = None, E: Optional[int] = None, group_offset: int = 0) -> torch.Tensor:
    """The expert FFN of a decoding step, T <= 64 tokens, in one kernel; bf16 [T, D].

    x bf16 [T, D] and h are not quantised (with a few tokens the weights' bytes
    are the cost); W as prepare_weights or prepare_weights_w8 made it, in every
    type.  topk_ids int32 [T, k], topk_w fp32
    [T, k] or None (ones).  W may hold the experts [group_offset, group_offset
    + W.w_in.shape[0]) of E; the others add nothing.  With `buf` (made for T
    tokens or more) the result is a part of buf.y, which may also hold x, and
    nothing is allocated; calls that may overlap on the GPU need buffers of their own.  Without, buffers are
    made and zeroed in the current stream's order for the one call."""
    T, k = _arg("ffn_decode topk_ids", topk_ids, torch.int32, 2).shape
    D = _arg("ffn_decode x", x, torch.bfloat16, 2).shape[1]
    El, F2 = W.w_in.shape[:2]
    F = F2 // 2
    E = group_offset + El if E is None else E
    in_mode, out_mode, dev = W.in_mode, W.out_mode, _dev("ffn_decode", x)
    if in_mode in (MX32, MX4) or out_mode in (MX32, MX4):
        kind, code, half = 2 + (in_mode == MX4), torch.uint8, 1 + (in_mode == MX4)
        if in_mode != out_mode:
            raise MoEError("ffn_decode: w_in and w_out hold different weight types")
        s_type, s_in, s_out, m_in, m_out = torch.uint8, (D // 128, El * 2 * F, 4), (F // 128, El * D, 4), 0, 0
    else:
        kind, code, half = (1, torch.int8, 1) if W.w_in.dtype is torch.int8 else (0, torch.uint8, 1)
        s_type, s_in, s_out = torch.float32, _decode_scale(in_mode, El, 2 * F, D), _decode_scale(out_mode, El, D, F)
        m_in, m_out = in_mode, out_mode
    px = _ptr("ffn_decode x", x, torch.bfloat16, (T, D), dev)
    pi = _ptr("ffn_decode topk_ids", topk_ids, torch.int32, (T, k), dev)
    pw = None if topk_w is None else _ptr("ffn_decode topk_w", topk_w, torch.float32, (T, k), dev)
    p_in = _ptr("ffn_decode w_in", W.w_in, code, (El, 2 * F, D // half), dev)
    p_out = _ptr("ffn_decode w_out", W.w_out, code, (El, D, F // half), dev)
    ps_in = _ptr("ffn_decode s_in", W.s_in, s_type, s_in, dev)
    ps_out = _ptr("ffn_decode s_out", W.s_out, s_type, s_out, dev)
    if buf is None:
        buf = DecodeBuffers(max(T, 1), D, E, k, F, x.device, settle=False)
    elif buf.T < T or buf.k != k or buf.D != D or buf.F != F or buf.y.get_device() != dev:
        raise MoEError("ffn_decode: the buffers were made for another shape or device")
    y = buf.y if T == buf.T else buf.y[:T]
    if T:
        check(lib().moe_ffn_decode(px, pi, pw, T, k, E, group_offset, El, D, F, kind, p_in, ps_in, m_in, p_out, ps_out,
                                   m_out, y.data_ptr(), buf.ws.data_ptr(), buf.ws_bytes, _s()), "moe_ffn_decode")
    return y


def _decode_scale(mode: int, El: int, N: int, K: int) -> tuple:
    """Shape of the fp32 scales of weights [El, N, K]."""
    if mode == PER_ROW:
        return (El, N)
    if mode == PER_ROW_BLOCK128:
        return (El, _nb(K), N)
    if mode == PER_TENSOR:
        return (1,)
    raise MoEError(f"ffn_decode: scale mode {mode}" + (" (decode_weights gives what it takes)" if mode == PER_BLOCK128 else ""))


def ffn_backward(dY: torch.Tensor, topk_w: torch.Tensor, W: ExpertWeights, buf: FFNBuffers,
                 static_x: Optional[torch.Tensor] = None, static_h: Optional[torch.Tensor] = None,
                 keep: Optional[dict] = None, x: Optional[torch.Tensor] = None):
    """Backward pass after ffn_forward on `buf`: of the static scheme (static_x and static_h
    as the forward had them), or of PER_BLOCK128 weights (x as the forward had it).

    Returns (dX bf16 [T, D], dW_in fp32 [E, D, 2F], dW_out fp32 [E, F, D]):
    dW_in holds grad_wi_0 | grad_wi_1 and dW_out grad_wo, in the pages'
    [E, in, out] layouts.  With `keep` (a dict), the intermediate gradients
    (dO, dO_q, dO_s, dA, dA_q, dA_s, dAg_s, dOg_s; with PER_BLOCK128 weights h in place
    of the last two) are stored in it."""
    s = buf.sort
    k = buf.k
    if dY.dtype is not torch.bfloat16 or dY.shape != (buf.T, buf.D):
        raise MoEError(f"ffn_backward dY: expected {torch.bfloat16} {[buf.T, buf.D]}, got {dY.dtype} {list(dY.shape)}")
    buf.check("ffn_backward", W, topk_w, buf.T, k)
    if W.in_mode == PER_BLOCK128:
        if W.w_in_t is None or x is None:
            raise MoEError("ffn_backward: PER_BLOCK128 weights made with for_backward, and x, are needed")
        if x.shape != dY.shape:
            raise MoEError(f"ffn_backward x: expected {list(dY.shape)}, got {list(x.shape)}")
    elif static_x is None or static_h is None:
        raise MoEError("ffn_backward: the static scheme needs static_x and static_h")
    if not buf.keep_a:
        raise MoEError("ffn_backward: buffers made with backward=True are needed")
    if not s or s["group_sizes"].shape[0] != W.w_in.shape[0]:
        raise MoEError("ffn_backward: ffn_forward has to run on these buffers first, on the same weights")
    if W.in_mode == PER_BLOCK128:
        sizes, ws = s["group_sizes"], buf.tgmm_workspace(W.w_in.shape[0])
        dO, dO_q, dO_s = gather_scale_quant_block(dY, topk_w, s["sorted_src"], k)
        gmm_block(dO_q, dO_s, W.w_out_t, W.s_out_t, sizes, out=buf.dH)
        dA, dA_q, dA_s, h = swiglu_bwd_quant_block(buf.dH, buf.a)
        gmm_block(dA_q, dA_s, W.w_in_t, W.s_in_t, sizes, out=buf.dXs)
        ragged_gather_reduce(buf.dXs, s["pos"], None, k, out=buf.dX)
        # both operands of a weight gradient are rounded along the rows that it contracts
        dW_in = tgmm_mx(x, dA, sizes, lhs_rows=s["sorted_src"], k=k, workspace=ws)
        dW_out = tgmm_mx(h, dO, sizes, workspace=ws)
        if keep is not None:
            keep.update(dO=dO, dO_q=dO_q, dO_s=dO_s, dA=dA, dA_q=dA_q, dA_s=dA_s, h=h)
        return buf.dX, dW_in, dW_out
    dO, dO_q, dO_s = gather_scale_quant(dY, topk_w, s["sorted_src"], k)
    gmm(dO_q, dO_s, PER_ROW, W.w_out_t, W.s_out, PER_TENSOR, s["group_sizes"], out=buf.dH)
    dA, dA_q, dA_s = swiglu_bwd_quant(buf.dH, buf.a)
    # dXs = dA0 W0^T + dA1 W1^T: one contraction over [dA0 | dA1], one static scale per K half
    gmm_ksplit(dA_q, dA_s, PER_ROW, W.w_in_t, W.s_in_split, buf.F, s["group_sizes"], out=buf.dXs)
    ragged_gather_reduce(buf.dXs, s["pos"], None, k, out=buf.dX)
    # per-(expert, column) gradient scales; their codes are made inside the weight-gradient contractions
    _, dAg_s = quantize_group_cols(dA, s["group_sizes"], scales_only=True)
    _, dOg_s = quantize_group_cols(dO, s["group_sizes"], scales_only=True)
    dW_in = tgmm_gcq(s["xs_q"], static_x, PER_TENSOR, dA, dAg_s, s["group_sizes"])
    dW_out = tgmm_gcq(buf.h_q, static_h, PER_TENSOR, dO, dOg_s, s["group_sizes"])
    if keep is not None:
        keep.update(dO=dO, dO_q=dO_q, dO_s=dO_s, dA=dA, dA_q=dA_q, dA_s=dA_s, dAg_s=dAg_s, dOg_s=dOg_s)
    return buf.dX, dW_in, dW_out

"""The operators of 4-bit expert weights and of single decoding steps, as cases to be measured.

Three operators of the expert FFN:

quantise  MXFP4 quantisation and reading back: bf16 rows (or expert weights, or the
          tokens of a chunk sorted by expert) to packed e2m1 codes with one
          power-of-two scale per 32 values, and from there to the values they stand for.
gmm       grouped matmul of MXFP4 activations with MXFP4 expert weights, bf16 out.
decode    the whole expert FFN (wi, SwiGLU, wo, weighted sum over the chosen experts)
          for a few tokens, on bf16 activations and quantised expert weights of every
          type that the framework has.

Each case is a dict of plain values.  `run` computes the plain form with elementary
torch operations in 32 bits, or, where `own` is true, calls the framework.
"""

import math

import torch

own = False


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # expert weights [E, N, K] of one layer as rows of K (E = 32 experts of a 4096-wide, 1408-deep layer), read back as a check of the layer would
        {"name": "quantise weights 90112x4096", "op": "quantise", "rows": 90112, "cols": 4096},
        # the tokens of a prompt's chunk: quantised once, copied to their eight experts' rows
        {"name": "quantise-sort 2048 tokens", "op": "quantise_sort", "T": 2048, "k": 8, "E": 128, "cols": 2048},
        # a short prompt: a few ragged groups, a row count that fills no tile, N with a tail of 16
        {"name": "gmm 129 rows, 4 experts", "op": "gmm", "M": 129, "K": 1024, "N": 1296, "E": 4, "g0": 0, "El": 4},
        # the wi product of a 2048-token chunk over 128 small experts
        {"name": "gmm 16384 rows, 128 experts", "op": "gmm", "M": 16384, "K": 2048, "N": 1536, "E": 128, "g0": 0, "El": 128},
        # the wi product of 8 large experts
        {"name": "gmm 16384 rows, 8 experts", "op": "gmm", "M": 16384, "K": 4096, "N": 28672, "E": 8, "g0": 0, "El": 8},
        # one expert-parallel shard: 32 of 64 experts are local, the other rows are zero
        {"name": "gmm shard 32 of 64 experts", "op": "gmm", "M": 12000, "K": 7168, "N": 4096, "E": 64, "g0": 16, "El": 32},
        # one token of a small layer: latency
        {"name": "decode 1 token, small, block", "op": "decode", "T": 1, "k": 8, "E": 128, "D": 2048, "F": 768, "w": "e4m3", "mode": "block"},
        # one token of a large layer with two of eight experts
        {"name": "decode 1 token, e4m3", "op": "decode", "T": 1, "k": 2, "E": 8, "D": 4096, "F": 14336, "w": "e4m3", "mode": "channel"},
        # an ordinary serving batch on int8 weights
        {"name": "decode 7 tokens, int8", "op": "decode", "T": 7, "k": 2, "E": 8, "D": 4096, "F": 14336, "w": "int8", "mode": "channel"},
        # MXFP8 weights, a few tokens over many experts
        {"name": "decode 5 tokens, MXFP8", "op": "decode", "T": 5, "k": 8, "E": 128, "D": 2048, "F": 768, "w": "mx8", "mode": "mx"},
        # MXFP4 weights, most experts hold one token or none
        {"name": "decode 16 tokens, MXFP4", "op": "decode", "T": 16, "k": 8, "E": 256, "D": 7168, "F": 2048, "w": "mx4", "mode": "mx"},
        # the largest batch: nearly every expert is read
        {"name": "decode 64 tokens, block", "op": "decode", "T": 64, "k": 8, "E": 256, "D": 7168, "F": 2048, "w": "e4m3", "mode": "block"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "quantise_sort", "gmm", "gmm", "decode", "decode", "decode"])
    if op == "quantise":
        cols = 128 * _log(rng, 1, 112)
        return {"op": op, "rows": _log(rng, 1, min(1 << 20, 90112 * 4096 // cols)), "cols": cols}
    if op == "quantise_sort":
        E = _log(rng, 2, 256)
        return {"op": op, "T": _log(rng, 1, 8192), "k": rng.randint(1, min(8, E)), "E": E, "cols": 128 * _log(rng, 1, 56)}
    if op == "gmm":
        E = _log(rng, 1, 128)
        El = rng.randint(max(1, E // 4), E)
        K, N = 128 * _log(rng, 1, 56), 16 * _log(rng, 1, 512)
        M = _log(rng, 1, 16384)
        return {"op": op, "M": M, "K": K, "N": N, "E": E, "g0": rng.randint(0, E - El), "El": El}
    w, mode = rng.choice([("e4m3", "channel"), ("e4m3", "block"), ("e4m3", "static"), ("int8", "channel"), ("int8", "block"), ("mx8", "mx"), ("mx4", "mx")])
    step = 16 if mode in ("channel", "static") else 128
    D, F = step * _log(rng, 256 // step, 7168 // step), step * _log(rng, 256 // step, 14336 // step)
    E = max(2, min(_log(rng, 2, 256), 256 * 7168 * 2048 // (D * F)))
    return {"op": op, "T": _log(rng, 1, 64), "k": rng.randint(1, min(8, E)), "E": E, "D": D, "F": F, "w": w, "mode": mode}


# ------------------------------------------------------------------ inputs

def _mx_scale_exp(x, emax):
    """Shared exponent of each 32-wide block of fp32 x [..., cols]: floor(log2(amax)) - emax, at least -127."""
    amax = x.unflatten(-1, (-1, 32)).abs().amax(-1)
    e = torch.frexp(amax)[1] - 1 - emax
    return torch.where(amax > 0, e, -127).clamp(-127, 127)


def _e2m1(v):
    """|v| rounded to the e2m1 grid (ties to even, at most 6), with the sign of v."""
    a = v.abs()
    a = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2)).clamp(max=6)
    return torch.copysign(a, v)


def _e2m1_code(v):
    a = v.abs()
    m = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    return m | (torch.signbit(v).to(torch.uint8) << 3)


def _mx4(x):
    """fp32 rows [R, cols] -> (packed codes [R, cols/2], scale codes [cols/128, R, 4])."""
    e = _mx_scale_exp(x, 2)
    c = _e2m1_code(_e2m1(torch.ldexp(x.unflatten(-1, (-1, 32)), -e.unsqueeze(-1)).flatten(-2)))
    sf = (e + 127).to(torch.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4), sf.unflatten(-1, (-1, 4)).transpose(0, 1).contiguous()


def _mx8(x):
    """fp32 rows [R, cols] -> (e4m3 codes [R, cols], scale codes [cols/128, R, 4])."""
    e = _mx_scale_exp(x, 8)
    v = torch.ldexp(x.unflatten(-1, (-1, 32)), -e.unsqueeze(-1)).flatten(-2).clamp(-448, 448)
    sf = (e + 127).to(torch.uint8)
    return v.to(torch.float8_e4m3fn).view(torch.uint8), sf.unflatten(-1, (-1, 4)).transpose(0, 1).contiguous()


def _routing(T, k, E, gen):
    """Distinct experts for each token, the most probable ones first, and their probabilities."""
    p = torch.softmax(torch.randn(T, E, generator=gen, device="cuda"), -1)
    w, ids = torch.topk(p, k, dim=-1)
    return ids.to(torch.int32).contiguous(), w.contiguous()


def _mx_rows(rows, cols, std, quantise, gen, part=1 << 26):
    """Quantised N(0, std) rows, made in parts: codes [rows, ...], scale codes [cols/128, rows, 4]."""
    step = max(1, part // cols)
    got = [quantise(torch.randn(min(step, rows - r), cols, generator=gen, device="cuda").mul_(std).bfloat16().float()) for r in range(0, rows, step)]
    return torch.cat([q for q, _ in got]), torch.cat([s for _, s in got], 1)


def _weights(E, N, K, w, mode, gen):
    """Codes [E, N, K] (mx4: [E, N, K/2]) and scales of weights N(0, 0.02)."""
    if w in ("mx8", "mx4"):
        q, sf = _mx_rows(E * N, K, 0.02, _mx8 if w == "mx8" else _mx4, gen)
        return q.view(E, N, -1), sf
    top = 448.0 if w == "e4m3" else 127.0
    s = 0.08 / top
    q = torch.empty(E, N, K, dtype=torch.uint8 if w == "e4m3" else torch.int8, device="cuda")
    for e in range(E):
        v = torch.randn(N, K, generator=gen, device="cuda").mul_(top / 4).clamp_(-top, top)
        q[e] = v.to(torch.float8_e4m3fn).view(torch.uint8) if w == "e4m3" else v.round_().to(torch.int8)
    shape = {"channel": (E, N), "block": (E, K // 128, N), "static": (1,)}[mode]
    return q, s * (0.75 + 0.5 * torch.rand(*shape, generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case)
    if case["op"] == "quantise":
        x = torch.randn(case["rows"], case["cols"], generator=gen, device="cuda")
        st["x"] = x.mul_(0.02 * torch.exp(torch.randn(case["rows"], 1, generator=gen, device="cuda"))).bfloat16()
    elif case["op"] == "quantise_sort":
        st["x"] = torch.randn(case["T"], case["cols"], generator=gen, device="cuda").bfloat16()
        st["ids"], _ = _routing(case["T"], case["k"], case["E"], gen)
    elif case["op"] == "gmm":
        M, K, N, E = (case[v] for v in ("M", "K", "N", "E"))
        # experts of unequal popularity, some without rows
        p = torch.softmax(torch.randn(E, generator=gen, device="cuda") * 0.7, 0)
        p = torch.where(torch.rand(E, generator=gen, device="cuda") < 0.06, torch.zeros_like(p), p) + 1e-9
        expert = torch.multinomial(p, M, replacement=True, generator=gen)
        st["group_sizes"] = torch.bincount(expert, minlength=E).to(torch.int32)
        st["most"] = int(st["group_sizes"].max())
        st["lhs_q"], st["lhs_sf"] = _mx_rows(M, K, 1.0, _mx4, gen)
        q, st["rhs_sf"] = _mx_rows(case["El"] * N, K, 0.02, _mx4, gen)
        st["rhs_q"] = q.view(case["El"], N, K // 2)
    else:
        T, k, E, D, F, w, mode = (case[v] for v in ("T", "k", "E", "D", "F", "w", "mode"))
        st["x"] = torch.randn(T, D, generator=gen, device="cuda").bfloat16()
        st["ids"], st["topk_w"] = _routing(T, k, E, gen)
        st["w_in"], st["s_in"] = _weights(E, 2 * F, D, w, "channel" if mode == "static" else mode, gen)
        st["w_out"], st["s_out"] = _weights(E, D, F, w, mode, gen)
    return st


# -------------------------------------------------------------------- plain forms

def _pow2(code):
    """2^(code - 127) in fp32."""
    return torch.ldexp(torch.ones((), device=code.device), code.to(torch.int32) - 127)


def _mx4_values(q, sf_rows):
    """Packed codes [..., cols/2], scale codes [..., cols/32] -> fp32 values [..., cols]."""
    m = torch.stack([q & 15, q >> 4], -1).flatten(-2)
    a = (m & 7).half()  # small numbers, exact here
    v = torch.where(a < 4, a / 2, torch.where(a < 6, a - 2, 2 * a - 8))
    v = torch.where(m > 7, -v, v)
    return v.float().unflatten(-1, (-1, 32)).mul_(_pow2(sf_rows).unsqueeze(-1)).flatten(-2)


def _sf_rows(sf, shape):
    """Scale codes [cols/128, rows, 4] -> [*shape, cols/32]."""
    return sf.transpose(0, 1).reshape(*shape, 4 * sf.shape[0])


def _quantise_plain(x):
    v = x.float()
    e = _mx_scale_exp(v, 2).unsqueeze(-1)
    return torch.ldexp(_e2m1(torch.ldexp(v.unflatten(-1, (-1, 32)), -e)), e).flatten(-2).bfloat16()


def _sort_plain(st):
    ids, k, E = st["ids"].flatten().long(), st["k"], st["E"]
    src = torch.argsort(ids, stable=True)
    sizes = torch.zeros(E, dtype=torch.int32, device=ids.device).index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    offsets = torch.nn.functional.pad(torch.cumsum(sizes, 0), (1, 0)).to(torch.int32)
    pos = torch.empty_like(src).index_copy_(0, src, torch.arange(src.numel(), device=src.device))
    return {"src": src.to(torch.int32), "pos": pos.to(torch.int32), "sizes": sizes, "offsets": offsets, "values": _quantise_plain(st["x"])[src // k]}


def _gmm_plain(st):
    sizes, M, N, g0, El = st["group_sizes"].long(), st["M"], st["N"], st["g0"], st["El"]
    start = torch.cumsum(sizes, 0) - sizes
    place = torch.arange(st["most"], device="cuda")
    rows = (start[g0:g0 + El, None] + place).clamp(max=M)  # the last row stands for the places that a group does not fill
    rows = torch.where(place < sizes[g0:g0 + El, None], rows, M)
    x = _mx4_values(st["lhs_q"], _sf_rows(st["lhs_sf"], (M,)))
    w = _mx4_values(st["rhs_q"], _sf_rows(st["rhs_sf"], (El, N)))
    x = torch.nn.functional.pad(x, (0, 0, 0, 1))[rows]
    out = torch.zeros(M + 1, N, dtype=torch.bfloat16, device="cuda")
    out[rows.flatten()] = torch.bmm(x, w.transpose(1, 2)).flatten(0, 1).bfloat16()
    return out[:M]


def _weight_values(q, s, w, mode, sel):
    """fp32 weights [E or len(sel), N, K]; `sel`: the experts wanted, or None for all."""
    E, N = q.shape[:2]
    if w in ("mx8", "mx4"):
        s = _sf_rows(s, (E, N))
    if sel is not None:
        q = q[sel]
        s = s if mode == "static" else s[sel]
    if w == "mx4":
        return _mx4_values(q, s)
    v = (q.view(torch.float8_e4m3fn) if q.dtype == torch.uint8 else q).float()
    if w == "mx8":
        return v.unflatten(-1, (-1, 32)).mul_(_pow2(s).unsqueeze(-1)).flatten(-2)
    if mode == "channel":
        return v.mul_(s.unsqueeze(-1))
    if mode == "block":
        return v.unflatten(-1, (-1, 128)).mul_(s.transpose(-1, -2).unsqueeze(-1)).flatten(-2)
    return v.mul_(s)


def _decode_plain(st):
    T, k, E, F, w, mode = (st[v] for v in ("T", "k", "E", "F", "w", "mode"))
    x, ids = st["x"].float(), st["ids"].long()
    in_mode = "channel" if mode == "static" else mode
    if T * k <= E:  # the chosen experts' weights, pair by pair
        flat = ids.flatten()
        a = torch.bmm(_weight_values(st["w_in"], st["s_in"], w, in_mode, flat), x.repeat_interleave(k, 0).unsqueeze(-1)).squeeze(-1)
        h = a[:, :F] / (1 + torch.exp(-a[:, :F])) * a[:, F:]
        o = torch.bmm(_weight_values(st["w_out"], st["s_out"], w, mode, flat), h.unsqueeze(-1)).squeeze(-1)
        return (o.view(T, k, -1) * st["topk_w"].unsqueeze(-1)).sum(1).bfloat16()
    # every expert on every token, weighted by its probability or by zero
    share = torch.zeros(T, E, device="cuda").scatter_add_(1, ids, st["topk_w"])
    a = torch.matmul(x, _weight_values(st["w_in"], st["s_in"], w, in_mode, None).transpose(1, 2))  # [E, T, 2F]
    h = a[..., :F] / (1 + torch.exp(-a[..., :F])) * a[..., F:] * share.t().unsqueeze(-1)
    return torch.bmm(h, _weight_values(st["w_out"], st["s_out"], w, mode, None).transpose(1, 2)).sum(0).bfloat16()


# ------------------------------------------------------------------------- a pass

def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "quantise":
        return _quantise_plain(state["x"])
    if op == "quantise_sort":
        return _sort_plain(state)
    if op == "gmm":
        return _gmm_plain(state)
    return _decode_plain(state)


def _run_own(st):
    import fp8_quantized_moe_gb300 as moe

    op = st["op"]
    if op == "quantise":
        return moe.dequantize_rows_mx4(*moe.quantize_rows_mx4(st["x"]))
    if op == "quantise_sort":
        o = moe.quantize_sort_mx4(st["x"], st["ids"], st["E"])
        return {"src": o["sorted_src"], "pos": o["pos"], "sizes": o["group_sizes"], "offsets": o["group_offsets"], "values": moe.dequantize_rows_mx4(o["xs_q"], o["xs_scale"])}
    if op == "gmm":
        return moe.gmm_mx4(st["lhs_q"], st["lhs_sf"], st["rhs_q"], st["rhs_sf"], st["group_sizes"], group_offset=st["g0"], E_local=st["El"])
    if "layer" not in st:  # what a server holds for a layer: its weights' handle and the step's buffers
        mode = {"channel": moe.PER_ROW, "block": moe.PER_ROW_BLOCK128, "static": moe.PER_TENSOR, "mx": moe.MX4 if st["w"] == "mx4" else moe.MX32}
        st["layer"] = moe.ExpertWeights(st["w_in"], st["s_in"], mode["channel" if st["mode"] == "static" else st["mode"]], st["w_out"], st["s_out"], mode[st["mode"]])
        st["buf"] = moe.DecodeBuffers(st["T"], st["D"], st["E"], st["k"], st["F"], "cuda")
    return moe.ffn_decode(st["x"], st["ids"], st["topk_w"], st["layer"], st["buf"])


# ------------------------------------------------------------------- exact, work

def _grid_round(v):
    """v (64 bits) to the nearest of the e2m1 values, ties to the one with the even code, at most 6."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=v.device)
    half = (grid[1:] + grid[:-1]) / 2
    a = v.abs()
    low = torch.bucketize(a, half, right=False)  # midpoints strictly below a
    tie = (a == half[low.clamp(max=6)]) & (low < 7)
    return torch.sign(v) * grid[low + (tie & (low % 2 == 1)).long()]


def _exact_quantise(x):
    b = x.double().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -200))) - 2), 2.0 ** -127).clamp(min=2.0 ** -127)
    return (_grid_round(b / scale) * scale).flatten(-2)


def _exact_codes(q, sf, row0, rows):
    """64-bit values of packed MXFP4 rows row0 .. row0 + rows of a [R, cols/2] code matrix."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    c = q[row0:row0 + rows].long()
    v = torch.stack([table[c % 16], table[c // 16]], -1).flatten(1)
    s = torch.exp2(sf[:, row0:row0 + rows].double() - 127).transpose(0, 1).flatten(1)
    return v * s.repeat_interleave(32, 1)


def _exact_weight(st, which, e):
    """64-bit weights [N, K] of expert e."""
    q, s, w, mode = st["w_" + which], st["s_" + which], st["w"], st["mode"]
    N = q.shape[1]
    if w == "mx4":
        return _exact_codes(q.flatten(0, 1), s, e * N, N)
    v = (q[e].view(torch.float8_e4m3fn) if q.dtype == torch.uint8 else q[e]).double()
    if w == "mx8":
        return v * torch.exp2(s[:, e * N:(e + 1) * N].double() - 127).transpose(0, 1).flatten(1).repeat_interleave(32, 1)
    if mode == "block":
        return v * s[e].double().t().repeat_interleave(128, 1)
    if mode == "static" and which == "out":
        return v * s.double()
    return v * s[e].double().unsqueeze(1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        return torch.cat([_exact_quantise(p) for p in st["x"].split(8192)])
    if op == "quantise_sort":
        flat = st["ids"].flatten().tolist()
        order = sorted(range(len(flat)), key=lambda i: (flat[i], i))
        place = [0] * len(flat)
        for r, i in enumerate(order):
            place[i] = r
        sizes = [0] * case["E"]
        for e in flat:
            sizes[e] += 1
        offsets = [sum(sizes[:e]) for e in range(case["E"] + 1)]
        as_int = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
        token = torch.tensor([i // case["k"] for i in order], device="cuda")
        return {"src": as_int(order), "pos": as_int(place), "sizes": as_int(sizes), "offsets": as_int(offsets), "values": _exact_quantise(st["x"])[token]}
    if op == "gmm":
        out = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
        row, N = 0, case["N"]
        for g, n in enumerate(st["group_sizes"].tolist()):
            if n and 0 <= g - case["g0"] < case["El"]:
                w = _exact_codes(st["rhs_q"].flatten(0, 1), st["rhs_sf"], (g - case["g0"]) * N, N)
                out[row:row + n] = _exact_codes(st["lhs_q"], st["lhs_sf"], row, n) @ w.t()
            row += n
        return out
    y = torch.zeros(case["T"], case["D"], dtype=torch.float64, device="cuda")
    F, x = case["F"], st["x"].double()
    for e in sorted(set(st["ids"].flatten().tolist())):
        token, j = torch.nonzero(st["ids"] == e, as_tuple=True)
        a = x[token] @ _exact_weight(st, "in", e).t()
        h = a[:, :F] * torch.sigmoid(a[:, :F]) * a[:, F:]
        y.index_add_(0, token, (h @ _exact_weight(st, "out", e).t()) * st["topk_w"][token, j].double().unsqueeze(1))
    return y


def work(case):
    op = case["op"]
    mx4 = 0.5 + 1 / 32  # bytes of an MXFP4 value with its share of the scale
    if op == "quantise":  # read, codes written and read back, values written
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 + 2 * mx4 + 2), "flops": 2 * n}
    if op == "quantise_sort":
        n, R = case["T"] * case["cols"], case["T"] * case["k"]
        return {"bytes": 2 * n + R * case["cols"] * (2 * mx4 + 2) + 12 * R + 8 * case["E"], "flops": 2 * n}
    if op == "gmm":  # the local share of the rows, the experts that M rows reach; zeros are written for the other rows
        M, El = case["M"] * case["El"] / case["E"], case["El"] * (1 - (1 - 1 / case["E"]) ** case["M"])
        return {"bytes": mx4 * (M * case["K"] + El * case["N"] * case["K"]) + 2 * case["M"] * case["N"] + 4 * case["E"], "flops": 2 * M * case["K"] * case["N"]}
    T, k, E, D, F = (case[v] for v in ("T", "k", "E", "D", "F"))
    experts = E * (1 - (1 - k / E) ** T)  # as many as T tokens choose, on average
    each = {"channel": 1 + 4 / D, "static": 1 + 4 / D, "block": 1 + 4 / 128, "mx": 1 + 1 / 32}[case["mode"]] if case["w"] != "mx4" else mx4
    return {"bytes": experts * 3 * D * F * each + T * (4 * D + 8 * k), "flops": 2 * T * k * 3 * D * F}

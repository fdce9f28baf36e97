"""The operators of training with block-scaled 8-bit experts, as cases to be measured.

Three operators:

gmm      grouped matmul of e4m3 activations that carry one fp32 scale per row and 128
         columns with e4m3 expert weights that carry one for each 128 x 128 block, bf16
         out: the forward product and, on the transposed weights, the input gradient.
         With one group it is a dense layer's product.
tgmm     the weight gradient: lhs^T rhs over each expert's rows, from the bf16 operands,
         which the operator rounds to e4m3 with a power-of-two scale for every 32 rows
         of an expert and column; fp32 out.  The lhs rows may be picked by an index
         (tokens by their sorted pairs).
balance  the router's balance loss with per-expert counts, and its gradient.

Each case is a dict of plain values.  `run` computes the plain form with elementary
torch operations in 32 bits, or, where `own` is true, calls the framework.
"""

import math

import torch

own = False


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one token through a small dense layer: latency
        {"name": "gmm 1 row, dense", "op": "gmm", "M": 1, "K": 2048, "N": 1536, "E": 1, "g0": 0, "El": 1, "dense": True},
        # a short prompt: a few ragged groups, rows that fill no tile, N with a tail of 16
        {"name": "gmm 129 rows, 4 experts", "op": "gmm", "M": 129, "K": 1024, "N": 1296, "E": 4, "g0": 0, "El": 4, "dense": False},
        # the wi product of a 2048-token chunk over 128 small experts
        {"name": "gmm 16384 rows, 128 experts", "op": "gmm", "M": 16384, "K": 2048, "N": 1536, "E": 128, "g0": 0, "El": 128, "dense": False},
        # the wi product of an expert-parallel shard's training step: 64 of 96 experts are local, the other rows are zero
        {"name": "gmm shard 64 of 96 experts", "op": "gmm", "M": 49152, "K": 7168, "N": 4096, "E": 96, "g0": 16, "El": 64, "dense": False},
        # the input gradient of 8 large experts: a contraction over both halves of wi
        {"name": "gmm input gradient, 8 experts", "op": "gmm", "M": 16384, "K": 28672, "N": 4096, "E": 8, "g0": 0, "El": 8, "dense": False},
        # a few tokens of a short step: ragged groups, one of them empty
        {"name": "tgmm 77 rows, 3 experts", "op": "tgmm", "M": 77, "T": 77, "k": 1, "K": 256, "N": 400, "E": 3, "g0": 0, "El": 3},
        # wi's gradient of 128 small experts from a 2048-token chunk: the gradients' bytes are the cost
        {"name": "tgmm 16384 rows, 128 experts", "op": "tgmm", "M": 16384, "T": 2048, "k": 8, "K": 2048, "N": 1536, "E": 128, "g0": 0, "El": 128},
        # wi's gradient of 64 experts, tokens picked by their sorted pairs
        {"name": "tgmm 49152 rows, 64 experts", "op": "tgmm", "M": 49152, "T": 8192, "k": 6, "K": 4096, "N": 2816, "E": 64, "g0": 0, "El": 64},
        # wi's gradient of 8 large experts
        {"name": "tgmm 16384 rows, 8 experts", "op": "tgmm", "M": 16384, "T": 8192, "k": 2, "K": 4096, "N": 28672, "E": 8, "g0": 0, "El": 8},
        # a few tokens of a small layer: latency
        {"name": "balance 24 tokens, 128 experts", "op": "balance", "S": 1, "L": 24, "E": 128, "k": 8, "padded": False, "closed": False},
        # four padded sequences of a large layer, a few experts closed by a logit of minus infinity
        {"name": "balance 4 x 4096 tokens, 256 experts", "op": "balance", "S": 4, "L": 4096, "E": 256, "k": 8, "padded": True, "closed": True},
        # a long accumulated batch over few experts
        {"name": "balance 262144 tokens, 64 experts", "op": "balance", "S": 32, "L": 8192, "E": 64, "k": 6, "padded": False, "closed": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gmm", "gmm", "tgmm", "tgmm", "balance"])
    if op == "gmm":
        E = _log(rng, 1, 128)
        El = rng.randint(max(1, E // 4), E)
        K, N = 128 * _log(rng, 1, 112), 16 * _log(rng, 1, 512)
        El = max(1, min(El, 64 * 4096 * 7168 // (K * N)))
        M = min(_log(rng, 1, 32768), 16384 * 28672 * 4096 // (K * N))
        return {"op": op, "M": max(1, M), "K": K, "N": N, "E": E, "g0": rng.randint(0, E - El), "El": El, "dense": E == 1 and rng.random() < 0.5}
    if op == "tgmm":
        E = _log(rng, 1, 128)
        El = rng.randint(max(1, E // 2), E)
        k = rng.randint(1, min(8, E))
        K, N = 16 * _log(rng, 1, 448), 16 * _log(rng, 1, 448)
        El = max(1, min(El, 8 * 4096 * 28672 // (K * N)))
        T = _log(rng, 1, 4096)
        return {"op": op, "M": T * k, "T": T, "k": k, "K": K, "N": N, "E": E, "g0": rng.randint(0, E - El), "El": El}
    E = _log(rng, 2, 512)
    S = _log(rng, 1, 64)
    L = _log(rng, 1, max(1, (1 << 24) // (E * S)))
    return {"op": op, "S": S, "L": L, "E": E, "k": rng.randint(1, min(8, E)), "padded": rng.random() < 0.5, "closed": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs

def _e4m3(v):
    return v.clamp(-448, 448).to(torch.float8_e4m3fn)


def _rows_q(rows, K, gen, part=1 << 26):
    """Activations with rows of unequal size: codes [rows, K], scales [rows, K/128]."""
    q = torch.empty(rows, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(rows, K // 128, device="cuda")
    step = max(1, part // K)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        x = torch.randn(n, K, generator=gen, device="cuda").mul_(torch.exp(0.5 * torch.randn(n, 1, generator=gen, device="cuda")))
        b = x.unflatten(1, (-1, 128))
        sc = b.abs().amax(-1) / 448
        s[r:r + n] = sc
        q[r:r + n] = _e4m3(b / sc.unsqueeze(-1)).view(torch.uint8).flatten(1)
    return q, s


def _weights_q(E, N, K, gen):
    """Expert weights N(0, 0.02): codes [E, N, K], scales [E, ceil(N/128), K/128]."""
    nb = (N + 127) // 128
    q = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, nb, K // 128, device="cuda")
    for e in range(E):
        w = torch.randn(N, K, generator=gen, device="cuda").mul_(0.02)
        b = torch.nn.functional.pad(w, (0, 0, 0, nb * 128 - N)).view(nb, 128, K // 128, 128)
        s[e] = b.abs().amax((1, 3)) / 448
        q[e] = _e4m3(b / s[e][:, None, :, None]).view(torch.uint8).reshape(nb * 128, K)[:N]
    return q, s


def _popularity(E, gen):
    """Experts of unequal popularity, some without rows."""
    p = torch.softmax(torch.randn(E, generator=gen, device="cuda") * 0.7, 0)
    return torch.where(torch.rand(E, generator=gen, device="cuda") < 0.06, torch.zeros_like(p), p) + 1e-9


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case)
    if case["op"] == "gmm":
        expert = torch.multinomial(_popularity(case["E"], gen), case["M"], replacement=True, generator=gen)
        st["group_sizes"] = torch.bincount(expert, minlength=case["E"]).to(torch.int32)
        st["most"] = int(st["group_sizes"].max())
        st["lhs_q"], st["lhs_s"] = _rows_q(case["M"], case["K"], gen)
        st["rhs_q"], st["rhs_s"] = _weights_q(case["El"], case["N"], case["K"], gen)
    elif case["op"] == "tgmm":
        T, k, K, N, E = (case[v] for v in ("T", "k", "K", "N", "E"))
        score = torch.log(_popularity(E, gen)) - torch.log(-torch.log(torch.rand(T, E, generator=gen, device="cuda").clamp(1e-7, 1 - 1e-7)))
        ids = torch.topk(score, k, dim=-1)[1].flatten()
        st["group_sizes"] = torch.bincount(ids, minlength=E).to(torch.int32)
        st["most"] = int(st["group_sizes"].max())
        st["sorted_src"] = torch.argsort(ids, stable=True).to(torch.int32)
        st["x"] = torch.randn(T, K, generator=gen, device="cuda").bfloat16()
        d = torch.empty(T * k, N, dtype=torch.bfloat16, device="cuda")
        for part in d.split(4096):  # gradients: rows of very unequal size
            part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * torch.exp(torch.randn(part.shape[0], 1, generator=gen, device="cuda") - 7))
        st["d"] = d
    else:
        T, E, k = case["S"] * case["L"], case["E"], case["k"]
        p = _popularity(E, gen)
        st["logits"] = 1.5 * torch.randn(T, E, generator=gen, device="cuda") + torch.log(p).clamp(min=-9)
        if case["closed"]:
            st["logits"][:, 1:].masked_fill_(p[1:] < 1e-8, -math.inf)
        st["ids"] = torch.topk(st["logits"], k, dim=-1)[1].to(torch.int32).contiguous()
        st["coef"], st["valid"] = 0.01, None
        st["grad"] = 2.0 ** 10 * (0.5 + torch.rand(1, generator=gen, device="cuda"))  # the loss scale
        if case["padded"]:  # sequences of unequal lengths
            length = (torch.rand(case["S"], 1, generator=gen, device="cuda") * (case["L"] + 1)).long()
            st["valid"] = (torch.arange(case["L"], device="cuda") < length).flatten()
    return st


# -------------------------------------------------------------------- plain forms

def _groups(st, M):
    """The rows of each local group, [El, most]; M stands for the places that a group does not fill."""
    sizes, g0, El = st["group_sizes"].long(), st["g0"], st["El"]
    start = torch.cumsum(sizes, 0) - sizes
    place = torch.arange(st["most"], device="cuda")
    rows = start[g0:g0 + El, None] + place
    return torch.where(place < sizes[g0:g0 + El, None], rows, M)


def _rows_plain(q, s):
    return q.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 128)).mul_(s.unsqueeze(-1)).flatten(-2)


def _gmm_plain(st):
    M, N, El = st["M"], st["N"], st["El"]
    x = _rows_plain(st["lhs_q"], st["lhs_s"])
    w = _rows_plain(st["rhs_q"], st["rhs_s"].repeat_interleave(128, 1)[:, :N])
    if st["dense"]:
        return torch.matmul(x, w[0].t()).bfloat16()
    rows = _groups(st, M)
    x = torch.nn.functional.pad(x, (0, 0, 0, 1))[rows]
    out = torch.zeros(M + 1, N, dtype=torch.bfloat16, device="cuda")
    out[rows.flatten()] = torch.bmm(x, w.transpose(1, 2)).flatten(0, 1).bfloat16()
    return out[:M]


def _round_rows(v):
    """fp32 [El, rows, cols] -> e4m3 values times 2^X for every 32 rows and column, 2^X the
    smallest power of two (2^-127 at least) that brings the largest one to 448 or below."""
    El, R, C = v.shape
    b = torch.nn.functional.pad(v, (0, 0, 0, -R % 32)).view(El, -1, 32, C)
    m, e = torch.frexp(b.abs().amax(2, keepdim=True))  # amax = m 2^e, m in [1/2, 1)
    X = torch.where(m > 0, e - 9 + (m > 0.875), -127).clamp(-127, 127)
    return torch.ldexp(_e4m3(torch.ldexp(b, -X)).float(), X).flatten(1, 2)


def _tgmm_plain(st):
    M = st["M"]
    rows = _groups(st, M)
    pad = lambda t: torch.cat([t, torch.zeros_like(t[:1])])  # noqa: E731
    src = pad(st["sorted_src"].long() // st["k"])
    src[M] = st["T"]  # a row of zeros
    lhs = _round_rows(pad(st["x"])[src[rows]].float())
    return torch.bmm(lhs.transpose(1, 2), _round_rows(pad(st["d"])[rows].float()))


def _balance_plain(st):
    S, L, E, k = st["S"], st["L"], st["E"], st["k"]
    x, ids = st["logits"], st["ids"].long()
    v = torch.ones(S * L, dtype=torch.bool, device="cuda") if st["valid"] is None else st["valid"]
    n = v.view(S, L).sum(1)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    p = torch.where(v.unsqueeze(-1), e / e.sum(-1, keepdim=True), 0)
    seq = torch.arange(S * L, device="cuda") // L
    counts = torch.zeros(S * E, dtype=torch.int32, device="cuda")
    counts.index_add_(0, (seq.unsqueeze(-1) * E + ids).flatten(), v.int().repeat_interleave(k))
    counts = counts.view(S, E)
    mean = p.view(S, L, E).sum(1) / n.clamp(min=1).unsqueeze(-1)
    f = counts * (E / (k * n.clamp(min=1).float())).unsqueeze(-1)
    loss = (f * mean).sum().reshape(1) * (st["coef"] / S)
    # counts relative to the most probable expert's: where its p is near 1, the difference below loses nothing
    c = counts.repeat_interleave(L, 0)
    c = (c - c.gather(1, x.argmax(-1, keepdim=True))).float()
    factor = (st["grad"] * st["coef"] / S * E / k) / n.clamp(min=1).float() ** 2
    d = p * (c - (p * c).sum(-1, keepdim=True)) * factor.repeat_interleave(L).unsqueeze(-1)
    return {"loss": loss, "counts": counts, "mean": mean, "dlogits": d}


# ------------------------------------------------------------------------- a pass

def run(state):
    if own:
        return _run_own(state)
    return {"gmm": _gmm_plain, "tgmm": _tgmm_plain, "balance": _balance_plain}[state["op"]](state)


def _run_own(st):
    import fp8_quantized_moe_gb300 as moe

    if st["op"] == "gmm":
        sizes = None if st["dense"] else st["group_sizes"]
        return moe.gmm_block(st["lhs_q"], st["lhs_s"], st["rhs_q"], st["rhs_s"], sizes, group_offset=st["g0"])
    if st["op"] == "tgmm":
        if "ws" not in st:  # what a trainer holds for a layer
            n = moe.tgmm_mx_workspace_bytes(st["M"], st["K"], st["N"], st["El"])
            st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return moe.tgmm_mx(st["x"], st["d"], st["group_sizes"], group_offset=st["g0"], E_local=st["El"], lhs_rows=st["sorted_src"], k=st["k"], workspace=st["ws"])
    b = moe.router_balance_loss(st["logits"], st["ids"], st["coef"], seqs=st["S"], valid=st["valid"])
    d = moe.router_balance_loss_backward(st["logits"], b, st["grad"])
    return {"loss": b.loss, "counts": b.counts, "mean": b.mean, "dlogits": d}


# ------------------------------------------------------------------- exact, work

def _exact_round_rows(v):
    """As defined: every 32 rows of a column share 2^X, X the least integer with amax <= 448 * 2^X."""
    out = torch.zeros_like(v)
    for r in range(0, v.shape[0], 32):
        b = v[r:r + 32]
        top = b.abs().amax(0)
        X = torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -200)))
        X = torch.where(top > 448 * torch.exp2(X), X + 1, torch.where(top <= 224 * torch.exp2(X), X - 1, X)).clamp(min=-127)
        a = b / torch.exp2(X)
        ulp = torch.exp2(torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -6))) - 3)
        out[r:r + 32] = torch.round(a / ulp) * ulp * torch.exp2(X)  # (torch.round: ties to even)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "gmm":
        out = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
        row = 0
        for g, n in enumerate(st["group_sizes"].tolist()):
            e = g - case["g0"]
            if n and 0 <= e < case["El"]:
                w = st["rhs_q"][e].view(torch.float8_e4m3fn).double()
                for j in range(st["rhs_s"].shape[1]):
                    w[128 * j:128 * j + 128] *= st["rhs_s"][e, j].double().repeat_interleave(128)
                x = st["lhs_q"][row:row + n].view(torch.float8_e4m3fn).double()
                out[row:row + n] = (x * st["lhs_s"][row:row + n].double().repeat_interleave(128, 1)) @ w.t()
            row += n
        return out
    if op == "tgmm":
        out = torch.zeros(case["El"], case["K"], case["N"], dtype=torch.float64, device="cuda")
        row, token = 0, st["sorted_src"].long() // case["k"]
        for g, n in enumerate(st["group_sizes"].tolist()):
            e = g - case["g0"]
            if n and 0 <= e < case["El"]:
                out[e] = _exact_round_rows(st["x"][token[row:row + n]].double()).t() @ _exact_round_rows(st["d"][row:row + n].double())
            row += n
        return out
    S, L, E, k = (case[v] for v in ("S", "L", "E", "k"))
    counts = torch.zeros(S, E, dtype=torch.int32, device="cuda")
    mean = torch.zeros(S, E, dtype=torch.float64, device="cuda")
    d = torch.zeros(S * L, E, dtype=torch.float64, device="cuda")
    loss = 0.0
    for s in range(S):
        rows = torch.arange(s * L, s * L + L, device="cuda")
        if st["valid"] is not None:
            rows = rows[st["valid"][s * L:s * L + L]]
        n = rows.numel()
        if not n:
            continue
        p = torch.softmax(st["logits"][rows].double(), -1)
        counts[s] = torch.bincount(st["ids"][rows].flatten().long(), minlength=E).int()
        mean[s] = p.mean(0)
        f = counts[s].double() * E / (k * n)
        loss += st["coef"] / S * float((f * mean[s]).sum())
        c = float(st["grad"]) * st["coef"] / (S * n) * f
        d[rows] = p * (c - (p @ c).unsqueeze(-1))
    return {"loss": torch.tensor([loss], dtype=torch.float64), "counts": counts, "mean": mean, "dlogits": d}


def work(case):
    op = case["op"]
    if op == "balance":  # logits read and their gradient written; ids, means and counts
        T, E = case["S"] * case["L"], case["E"]
        return {"bytes": T * (8 * E + 4 * case["k"]) + 8 * case["S"] * E + (T if case["padded"] else 0), "flops": 8 * T * E}
    M, K, N, E, El = (case[v] for v in ("M", "K", "N", "E", "El"))
    Ml = M * El / E  # the local share of the rows
    if op == "gmm":  # the experts that M rows reach; zeros are written for the other rows
        reached = El * (1 - (1 - 1 / E) ** M)
        return {"bytes": (1 + 4 / 128) * Ml * K + reached * N * K * (1 + 4 / 128 ** 2) + 2 * M * N + 4 * E, "flops": 2 * Ml * K * N}
    T = min(Ml, case["T"])  # each token is read once
    return {"bytes": 2 * T * K + 2 * Ml * N + 4 * M + 4 * El * K * N + 4 * E, "flops": 2 * Ml * K * N}

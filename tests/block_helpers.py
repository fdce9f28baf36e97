"""Plain 64-bit forms of the operators on block-scaled 8-bit experts, for their tests."""

import torch

F64 = torch.float64


def e4m3(codes: torch.Tensor) -> torch.Tensor:
    """The values of e4m3 codes, 64 bits."""
    return codes.view(torch.float8_e4m3fn).to(F64)


def round_e4m3(v: torch.Tensor) -> torch.Tensor:
    """v (64 bits, |v| <= 464) to the nearest e4m3 value, ties to even, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def rows_value(q, s):
    """Codes [M, K] and scales [M, K/128] -> 64-bit values."""
    return e4m3(q) * s.to(F64).repeat_interleave(128, 1)


def weight_value(q, s):
    """Codes [E, N, K] and scales [E, ceil(N/128), K/128] -> 64-bit values."""
    N = q.shape[1]
    return e4m3(q) * s.to(F64).repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)


def block_scale(amax):
    """fp32(amax / 448), 1 for zero, as a 64-bit value (amax: fp32 values; rounding the 64-bit quotient is the
    fp32 division's own rounding)."""
    s = (amax.to(F64) / 448).float().to(F64)
    return torch.where(amax > 0, s, torch.ones_like(s))


def quantise_blocks(w):
    """bf16 [E, N, K] -> (64-bit values of the codes [E, N, K], scales [E, ceil(N/128), K/128])."""
    E, N, K = w.shape
    nb = -(-N // 128)
    v = torch.zeros(E, nb * 128, K, dtype=F64, device=w.device)
    v[:, :N] = w.to(F64)
    b = v.view(E, nb, 128, K // 128, 128)
    s = block_scale(b.abs().amax((2, 4)))
    # the quotient is an fp32 value (rounding it from 64 bits is the division's own rounding)
    q = round_e4m3((b / s[:, :, None, :, None]).float().to(F64))
    return q.reshape(E, nb * 128, K)[:, :N], s


def quantise_rows128(x):
    """bf16 [R, C] -> (64-bit values of the codes, scales [R, C/128])."""
    b = x.to(F64).unflatten(1, (-1, 128))
    s = block_scale(b.abs().amax(2))
    return round_e4m3((b / s.unsqueeze(2)).float().to(F64)).flatten(1), s


def round_rows(x):
    """A group's rows [R, C] rounded to e4m3 times 2^X, X the least integer >= -127 with
    amax <= 448 * 2^X over every 32 rows of a column (64 bits)."""
    out = torch.zeros(x.shape, dtype=F64, device=x.device)
    for r in range(0, x.shape[0], 32):
        b = x[r:r + 32].to(F64)
        m, e = torch.frexp(b.abs().amax(0))
        X = torch.where(m > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -127)).clamp(min=-127).to(F64)
        out[r:r + 32] = round_e4m3(b / torch.exp2(X)) * torch.exp2(X)
    return out


def groups(sizes, g0, El):
    """(local expert, first row, rows) of the local groups."""
    row = 0
    for g, n in enumerate(sizes):
        if g0 <= g < g0 + El:
            yield g - g0, row, n
        row += n


def gmm(lhs_q, lhs_s, rhs_q, rhs_s, sizes, g0=0):
    """(out, sum of the products' magnitudes), 64 bits."""
    El, N, _ = rhs_q.shape
    x, w = rows_value(lhs_q, lhs_s), weight_value(rhs_q, rhs_s)
    out = torch.zeros(x.shape[0], N, dtype=F64, device=x.device)
    mag = torch.zeros_like(out)
    for e, r, n in groups(sizes, g0, El):
        out[r:r + n] = x[r:r + n] @ w[e].t()
        mag[r:r + n] = x[r:r + n].abs() @ w[e].abs().t()
    return out, mag


def tgmm(lhs, rhs, sizes, g0, El):
    """(out, sum of the products' magnitudes), 64 bits; lhs: the picked rows."""
    out = torch.zeros(El, lhs.shape[1], rhs.shape[1], dtype=F64, device=lhs.device)
    mag = torch.zeros_like(out)
    for e, r, n in groups(sizes, g0, El):
        if n:
            a, b = round_rows(lhs[r:r + n]), round_rows(rhs[r:r + n])
            out[e] = a.t() @ b
            mag[e] = a.abs().t() @ b.abs()
    return out, mag


def balance(logits, ids, coef, seqs, valid, grad=1.0):
    """(loss, counts, mean, tokens, dlogits), 64 bits."""
    T, E = logits.shape
    L, k = T // seqs, ids.shape[1]
    counts = torch.zeros(seqs, E, dtype=torch.int64)
    mean = torch.zeros(seqs, E, dtype=F64)
    tokens = torch.zeros(seqs, dtype=torch.int64)
    d = torch.zeros(T, E, dtype=F64)
    loss = 0.0
    for s in range(seqs):
        rows = torch.arange(s * L, s * L + L)
        if valid is not None:
            rows = rows[valid[rows]]
        n = tokens[s] = len(rows)
        if not n:
            continue
        x = logits[rows].to(F64)
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(top == -torch.inf, 0.0, top))
        z = e.sum(1, keepdim=True)
        p = torch.where(z == 0, 0.0, e / z)
        flat = ids[rows].flatten().long()
        counts[s] = torch.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
        mean[s] = p.mean(0)
        f = counts[s].to(F64) * E / (k * int(n))
        loss += coef / seqs * float((f * mean[s]).sum())
        c = grad * coef / (seqs * int(n)) * f
        d[rows] = p * (c - (p @ c).unsqueeze(1))
    return loss, counts, mean, tokens, d

"""Layout moves between the oracle's row-major MXFP4 arrays and the library's
packed, K-block-major ones (pure data movement), and rows whose blocks go
through the format's special cases."""

import numpy as np
import torch


def bf16(a) -> np.ndarray:
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def pack(q):
    """Codes [..., cols] one a byte -> [..., cols/2], the even column in the low half."""
    return (q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8)


def unpack(p):
    return np.stack([p & 15, p >> 4], -1).reshape(*p.shape[:-1], 2 * p.shape[-1])


def sf_kmajor(sf):
    """Row-major scale codes [rows, cols/32] -> [cols/128, rows, 4]."""
    rows, nb = sf.shape
    return np.ascontiguousarray(sf.reshape(rows, nb // 4, 4).transpose(1, 0, 2))


def sf_rows(sf):
    """[cols/128, rows, 4] -> [rows, cols/32]."""
    kb, rows, _ = sf.shape
    return np.ascontiguousarray(sf.transpose(1, 0, 2).reshape(rows, 4 * kb))


def special_rows(rng, rows, cols):
    """bf16 bits [rows, cols] whose blocks span many binades, with zero blocks,
    saturating ones, ties of e2m1 rounding, subnormal amax, values next to
    the largest bf16 and negative zeros."""
    x = rng.standard_normal((rows, cols)).astype(np.float32)
    x *= np.repeat(np.ldexp(1.0, rng.integers(-40, 40, (rows, cols // 32))), 32, axis=1).astype(np.float32)
    for r in range(rows):
        b = int(rng.integers(0, cols // 32))
        blk = x[r, 32 * b:32 * b + 32]
        kind = r % 7
        if kind == 0:
            blk[:] = 0.0
        elif kind == 1:  # 7.75 at scale 1: above 6, saturates
            blk[:] = [7.75, -6.5, 5.0, -5.0] * 8
        elif kind == 2:  # every midpoint of the e2m1 grid at scale 1
            blk[:] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] * 4
        elif kind == 3:
            blk[:] = [-4.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0] * 4
        elif kind == 4:  # a subnormal amax: X clamps to -127
            blk[:] = np.ldexp(1.0, -130)
        elif kind == 5:
            blk[:] = np.float32(3.3895e38)
        else:
            blk[:] = -0.0
    return bf16(x)

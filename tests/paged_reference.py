"""Plain 64-bit definitions of the chunk-paged serving calls, written value by
value on the host: the rotation, the 4-bit rows and their layout, the placing
of a ragged batch."""
import numpy as np

C = 64
GROUP = 32


def places(seqlens, cu):
    """[(token, sequence, position)] of a ragged batch."""
    out = []
    for b, n in enumerate(seqlens):
        first = n - (cu[b + 1] - cu[b])
        out += [(t, b, first + t - cu[b]) for t in range(cu[b], cu[b + 1])]
    return out


def rotate(x, table, pos, interleaved):
    """x [T, H, d] rotated by the table rows of pos [T]; also the magnitude
    sum |x c| + |y s| that bounds the rounding of each result."""
    x = np.asarray(x, np.float64)
    if table is None:
        return x, np.zeros_like(x)
    r = table.shape[1]
    y, mag = x.copy(), np.zeros_like(x)
    for i in range(r // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        c = table[pos, i].astype(np.float64)[:, None]
        s = table[pos, r // 2 + i].astype(np.float64)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = abs(x[..., a] * c) + abs(x[..., b] * s)
        mag[..., b] = abs(x[..., b] * c) + abs(x[..., a] * s)
    return y, mag


def unit_and_nibble(dim, d):
    """Where dim's code lives in a row of codes: (byte, shift)."""
    g, e, i = dim // GROUP, dim % GROUP // 4, dim % 4
    return 2 * (e * (d // GROUP) + g) + i // 2, 4 * (i % 2)


def unpack(pages, d):
    """(codes [n, H, 64, d] int, step and least value [n, H, 64, d/32] double) of 4-bit pages [n, H, bytes]."""
    n, H, _ = pages.shape
    rows = pages[:, :, : C * d // 2].reshape(n, H, C, d // 2)
    par = np.ascontiguousarray(pages[:, :, C * d // 2:]).view(np.float16).reshape(n, H, C, d // GROUP, 2)
    codes = np.empty((n, H, C, d), np.int64)
    for dim in range(d):
        byte, shift = unit_and_nibble(dim, d)
        codes[..., dim] = (rows[..., byte] >> shift) & 15
    return codes, par[..., 0].astype(np.float64), par[..., 1].astype(np.float64)


def values(pages, d):
    """What 4-bit pages stand for [n, H, 64, d], rounded once to fp32 (a step times a code plus a least value is exact
    in 64 bits)."""
    codes, step, least = unpack(pages, d)
    with np.errstate(invalid="ignore"):
        v = np.repeat(least, GROUP, -1) + np.repeat(step, GROUP, -1) * codes
    return v.astype(np.float32)


def quantise(x):
    """(quotients before rounding, codes, step, least) of x [..., d] in 64 bits."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, GROUP)
    lo, hi = g.min(-1), g.max(-1)
    least = lo.astype(np.float16).astype(np.float64)
    step = ((hi - lo) / 15).astype(np.float16).astype(np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        ratio = np.where(step[..., None] > 0, (g - least[..., None]) / step[..., None], 0.0)
    codes = np.clip(np.rint(ratio), 0, 15).astype(np.int64)
    return ratio.reshape(x.shape), codes.reshape(x.shape), step, least


def pack(x):
    """4-bit blocks [n, H, bytes] of rows x [n, H, 64, d]."""
    n, H, _, d = x.shape
    _, codes, step, least = quantise(x)
    rows = np.zeros((n, H, C, d // 2), np.uint8)
    for dim in range(d):
        byte, shift = unit_and_nibble(dim, d)
        rows[..., byte] |= (codes[..., dim] << shift).astype(np.uint8)
    par = np.stack([step, least], -1).astype(np.float16).view(np.uint8).reshape(n, H, -1)
    return np.concatenate([rows.reshape(n, H, -1), par], -1)

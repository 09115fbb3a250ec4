"""Plain 64-bit forms of the 4-bit quantisation and its layout, on the host
(numpy, no library code)."""
import math

import numpy as np
import torch

NV, MX = 0, 1
LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([k * 2.0 ** -9 for k in range(8)]
                + [(8 + k) * 2.0 ** (e - 3) for e in range(-6, 9) for k in range(8)][:-1])
E8M0 = np.array([2.0 ** e for e in range(-127, 128)])


def block_of(fmt):
    return 32 if fmt == MX else 16


def philox(seed, side, rows, cols):
    """The 16 random bits of each element (Philox4x32-10), in Python integers."""
    per = -(-cols // 8)
    out = np.zeros((rows, per * 8), np.int64)
    for n in range(rows * per):
        c = [n & 0xFFFFFFFF, n >> 32, side, 0]
        k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
        for _ in range(10):
            a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
            c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
            k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
        r, g = divmod(n, per)
        for j, w in enumerate(c):
            out[r, g * 8 + 2 * j], out[r, g * 8 + 2 * j + 1] = w & 0xFFFF, w >> 16
    return out[:, :cols]


def exponent(x, fmt):
    """e of a matrix's power of two (0 for E8M0 scales)."""
    if fmt == MX:
        return 0
    a = np.abs(x[np.isfinite(x)])
    top = float(a.max()) if a.size else 0.0
    if top == 0.0:
        return -126
    e = math.frexp(top / 2688)[1] - 2
    while top > 2688 * 2.0 ** e:
        e += 1
    return max(e, -126)


def quantized(x, fmt, seed=None, side=0):
    """(codes, scale bytes, values) of a float64 matrix, by search through the
    scale's and the element's values."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    b = block_of(fmt)
    blocks = -(-cols // b)
    unit = 2.0 ** exponent(x, fmt)
    table = E8M0 if fmt == MX else E4M3
    codes = np.zeros((rows, cols), np.int64)
    scales = np.zeros((rows, blocks), np.int64)
    values = np.zeros((rows, cols))
    u = None if seed is None else philox(seed, side, rows, cols)
    for j in range(blocks):
        at = slice(j * b, min(cols, (j + 1) * b))
        v = np.abs(x[:, at])
        bad = ~np.isfinite(v).all(1)
        v = np.where(bad[:, None], 0.0, v)
        byte = np.searchsorted(6 * table, v.max(1) / unit)
        s = (table[byte] * unit)[:, None]
        y = v / np.where(s > 0, s, 1.0)
        i = np.clip(np.searchsorted(LEVELS, y, side="right") - 1, 0, 7)
        lo, hi = LEVELS[i], LEVELS[np.minimum(i + 1, 7)]
        if u is None:
            up = (y > (lo + hi) / 2) | ((y == (lo + hi) / 2) & (i % 2 == 1))
        else:
            up = v - lo * s > (2 * u[:, at] + 1) * 2.0 ** -17 * (hi - lo) * s
        up &= i < 7
        c = i + up
        sign = np.signbit(x[:, at])
        codes[:, at] = np.where(bad[:, None], 0, c + 8 * sign)
        values[:, at] = np.where(bad[:, None], np.nan, np.where(sign, -1.0, 1.0) * LEVELS[c] * s)
        scales[:, j] = np.where(bad, 0xFF if fmt == MX else 0x7F, byte)
    return codes, scales, values


def unpacked(codes, scales, rows, cols, fmt):
    """(codes, scale bytes, codes behind the last column, scales behind the last
    row and block) of the stored bytes, as the layout is documented."""
    pitch = -(-cols // 32) * 16
    c = np.asarray(codes).reshape(rows, pitch)
    c = np.stack([c & 15, c >> 4], 2).reshape(rows, pitch * 2)
    blocks = -(-cols // block_of(fmt))
    tiles = -(-blocks // 4)
    s = np.asarray(scales).reshape(-(-rows // 128), tiles, 32, 4, 4)
    s = s.transpose(0, 3, 2, 1, 4).reshape(-1, tiles * 4)
    return (c[:, :cols].astype(np.int64), s[:rows, :blocks].astype(np.int64), c[:, cols:],
            np.concatenate([s[rows:].ravel(), s[:rows, blocks:].ravel()]))


def values_of(q):
    """Values of a library matrix from its stored bytes, in float64."""
    c, s, _, _ = unpacked(q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.rows, q.cols, q.format)
    scale = np.append(E8M0, np.nan)[s] if q.format == MX else np.append(E4M3, np.nan)[np.minimum(s, 0x7F)]
    unit = 1.0
    if q.format == NV:
        unit = 2.0 ** exponent(q.amax[:1].cpu().double().numpy().reshape(1, 1), NV)
    v = np.where(c & 8, -1.0, 1.0) * LEVELS[c & 7]
    return v * np.repeat(scale, block_of(q.format), 1)[:, :q.cols] * unit


def spread(rows, cols, seed, dtype, scale=1e-3):
    """Values whose rows and columns differ in size."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))
    x = x * torch.exp(0.5 * torch.randn(1, cols, generator=g))
    return (scale * x).to(dtype)


def product_bound(a, b, out_dtype, c):
    """Largest allowed |error| of each element of a b^T (float64 values).  A
    product step adds 64 terms to an fp32 sum and may cut what lies below the
    last place of the largest, up to 8 parts of a sum are added and one addition
    to C may follow, each with one more rounding: 2^-23 of the sum of magnitudes
    for each, twice that for what a step cuts of its own terms.  Then half a
    step of the result's type."""
    k = a.shape[1]
    steps = 2 * (-(-k // 64) + 10)
    eps = torch.finfo(out_dtype).eps / 2
    return steps * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T) + eps * np.abs(c) + 1e-37

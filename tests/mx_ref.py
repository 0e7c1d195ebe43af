"""Plain 64-bit implementations of the microscaled operators on the CPU, from
the formats' definition (32 elements per power-of-two scale).  Shares no code
with the library."""
import math

import numpy as np
import torch

FP8, FP4 = 1, 2
EMAX = {FP8: 8, FP4: 2}
BLOCK_BYTES = {FP8: 32, FP4: 16}


def code_values(fmt):
    """Value of every code (numpy float64 [256] or [16])."""
    if fmt == FP4:
        pos = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    else:
        pos = [math.ldexp(c % 8, -9) if c < 8 else math.ldexp(8 + c % 8, c // 8 - 10) for c in range(127)]
        pos.append(math.nan)
    return np.array(pos + [-v for v in pos])


def quantise(x, fmt):
    """(codes uint8 [M, nb * 32] one per element, scales uint8 [M, nb]) of a
    float64 array."""
    x = np.asarray(x, np.float64)
    M, k = x.shape
    nb = -(-k // 32)
    v = np.zeros((M, nb * 32))
    v[:, :k] = x
    v = v.reshape(M, nb, 32)
    bad = ~np.isfinite(v).all(-1)
    top = np.abs(np.where(bad[..., None], 0, v)).max(-1)
    e = np.where(top > 0, np.frexp(np.where(top > 0, top, 1))[1] - 1 - EMAX[fmt], -127)
    e = np.maximum(e, -127)
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    u = np.ldexp(np.where(bad[..., None], 0, v), -e[..., None])
    vals = code_values(fmt)
    n = 127 if fmt == FP8 else 8
    table = vals[:n]
    mid = (table[1:] + table[:-1]) / 2
    a = np.abs(u)
    lo = np.searchsorted(mid, a)  # midpoints below a
    tie = (lo < n - 1) & (a == mid[np.minimum(lo, n - 2)]) & (lo % 2 == 1)
    code = (lo + tie).astype(np.uint8) | (np.signbit(u).astype(np.uint8) << (7 if fmt == FP8 else 3))
    code[bad] = 0
    return code.reshape(M, nb * 32), s


def pack(codes, fmt):
    return codes if fmt == FP8 else (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(q, fmt, nb):
    q = np.asarray(q)[:, :nb * BLOCK_BYTES[fmt]]
    if fmt == FP8:
        return q
    out = np.empty((q.shape[0], 2 * q.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def dequantise(codes, scales, fmt, k):
    """float64 [M, k] of one code per element and scale bytes."""
    M, n = codes.shape
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (code_values(fmt)[codes].reshape(M, n // 32, 32) * s[:, :n // 32, None]).reshape(M, n)[:, :k]


def quantised_values(x, fmt):
    c, s = quantise(x, fmt)
    return dequantise(c, s, fmt, x.shape[1])


def rmsnorm(x, weight, eps, residual=None):
    """(h, y) in float64."""
    h = np.asarray(x, np.float64) if residual is None else np.asarray(x, np.float64) + np.asarray(residual, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        return h, h / np.sqrt((h * h).mean(-1, keepdims=True) + float(np.float32(eps))) * np.asarray(weight, np.float64)


def f64(t):
    return t.detach().double().cpu().numpy()


def half_step(dtype):
    """Largest relative error of one rounding to nearest."""
    return torch.finfo(dtype).eps / 2


# (M, k, d) for each of the product's tile shapes in turn, by the format of x:
# k goes nearly twice round the longest ring of LDS tiles or scales and ends
# inside a block; d (and M but for the smallest tiles) is whole tiles and a part.
LONG = {
    FP8: [
        (1, 8204, 19), (18, 4421, 2074), (2103, 4135, 71), (34, 4418, 6539), (49, 3132, 9651), (4225, 3391, 68),
        (102, 3042, 5705), (67, 3089, 8216), (3273, 2195, 285), (129, 2260, 8223), (539, 4043, 7444),
        (4127, 4067, 686), (5480, 4059, 666), (1561, 2055, 3801), (775, 2321, 8363), (1036, 2072, 8909),
        (1381, 2114, 8196)],
    FP4: [
        (1, 8016, 19), (33, 4241, 4174), (33, 4083, 1466), (2823, 4021, 73), (34, 4559, 6198), (5486, 3133, 66),
        (69, 3150, 6418), (71, 2719, 8367), (3351, 3151, 263), (142, 3185, 8253), (270, 2114, 9552),
        (5709, 4231, 264), (5545, 4003, 457), (1025, 2098, 5542), (517, 2319, 9825), (1410, 2090, 5448),
        (1092, 2082, 8278), (1113, 2125, 9838)],
}

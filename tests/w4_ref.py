"""Plain 64-bit implementations, on the CPU, of the operators over a 4-bit
weight with group scales and zero points and of the norm and rotation of heads.
Shares no code with the library."""
import numpy as np
import torch


def weight(seed, d, k, group, zeros=True, dtype=torch.bfloat16, exact=False):
    """Codes [d, k], scales [d, groups] (torch, dtype), zero points [d, groups]
    uint8 or None.  exact: scales are 0.5, 1 or 2."""
    rng = np.random.default_rng(seed)
    ng = -(-k // group)
    q = rng.integers(0, 16, (d, k)).astype(np.uint8)
    if exact:
        s = torch.from_numpy(rng.choice([0.5, 1.0, 2.0], (d, ng))).to(dtype)
    else:
        s = torch.from_numpy(np.exp(rng.normal(0, 0.5, (d, ng))) * rng.choice([1, 1, 1, -1], (d, ng)) / 5).to(dtype)
    z = rng.integers(0, 16, (d, ng)).astype(np.uint8) if zeros else None
    return q, s, z


def pack(q):
    """Two codes a byte, the even column low; a missing last one is 15."""
    d, k = q.shape
    full = np.full((d, (k + 1) // 2 * 2), 15, np.uint8)
    full[:, :k] = q
    return (full[:, 0::2] | (full[:, 1::2] << 4)).astype(np.uint8)


def dequant(q, s, z, group):
    k = q.shape[1]
    zz = np.full(s.shape, 8.0) if z is None else z.astype(np.float64) % 32
    rep = lambda a: np.repeat(a, group, 1)[:, :k]
    return rep(s.double().numpy()) * (q.astype(np.float64) - rep(zz))


def kept(s):
    """Scales with 19 significant bits, to nearest, ties to even."""
    m, e = np.frexp(s.double().numpy())
    return torch.from_numpy(np.ldexp(np.round(m * 2.0 ** 19), e - 19))


def sum_bound(x, s, z, group):
    """Bound of the fp32 part of a product's error: a group of at most 128
    columns is a sum of products with codes (at most 15) and one of x times a
    zero point (at most 31); 2^-23 of the magnitudes for each of 128 additions,
    and as much again for the groups' sums (fewer than 128 of them)."""
    k = x.shape[1]
    rep = np.repeat(np.abs(s.double().numpy()), group, 1)[:, :k]
    return 2 * 128 * 2.0 ** -23 * (15 + 31) * (np.abs(x) @ rep.T)


def heads(x, w, eps, cos, sin, rot, interleaved):
    """x [M, H, D] float64; cos, sin [M, rot / 2] or None.  (result, magnitude
    of what is added up for it)."""
    u = x.copy()
    if w is not None:
        u = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps) * w
    if cos is None:
        return u, np.abs(u)
    first = np.arange(rot // 2) * (2 if interleaved else 1)
    second = first + (1 if interleaved else rot // 2)
    out, mag = u.copy(), np.abs(u)
    a, b, c, s = u[..., first], u[..., second], cos[:, None], sin[:, None]
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    m = np.abs(a) + np.abs(b)
    mag[..., first] = mag[..., second] = m
    return out, mag

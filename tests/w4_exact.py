"""Layers over a 4-bit weight whose every sum is exact in fp32, in any order, for
the GPU tests that compare bit for bit.  Shares no code with the library.

x holds whole numbers of -4 .. 4, codes less zero points lie in -15 .. 15, the
weight's scales are 0.5, 1 or 2, A holds -1 .. 1, B -2 .. 2, the adapters' scales
are powers of two of 0.5 .. 4: every value is a multiple of 0.5.  A base sum's
terms are at most 120, so any part of it stays below 2^21 for k <= 2^14.  t is
asserted below 2^15, which two bf16 of 8 bits hold exactly (what the first leaves
of a multiple of 0.5 below 2^15 has at most 8 bits), and 2 sum |t|, the bound of
any part of t B^T, below 2^22.  All sums are then below 2^23, and fp32 holds
multiples of 0.5 up to there.
"""
import numpy as np
import torch

BF = torch.bfloat16


class Weight:
    """A random such weight, made on the device: q uint8 [d, k], scales, zeros."""

    def __init__(self, seed, d, k, group, zeros=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        ng = -(-k // group)
        self.d, self.k, self.group = d, k, group
        self.q = torch.randint(0, 16, (d, k + k % 2), generator=g, device="cuda", dtype=torch.uint8)
        self.s = torch.tensor([0.5, 1.0, 2.0], device="cuda")[
            torch.randint(0, 3, (d, ng), generator=g, device="cuda")].to(BF)
        self.z = torch.randint(0, 16, (d, ng), generator=g, device="cuda", dtype=torch.uint8) if zeros else None

    def packed(self):
        return (self.q[:, 0::2] | (self.q[:, 1::2] << 4)).contiguous()

    def dense(self):
        """float64 [d, k]."""
        rep = lambda a: a.double().repeat_interleave(self.group, 1)[:, :self.k]
        z = torch.full_like(self.s, 8.0) if self.z is None else self.z
        return rep(self.s) * (self.q[:, :self.k].double() - rep(z))


def rows(seed, M, k):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-4, 5, (M, k), generator=g, device="cuda").to(BF)


def adapters(seed, S, R, k, d, ranks):
    """A [S, R, k], B [S, d, R], NaN past each rank."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    A = torch.randint(-1, 2, (S, R, k), generator=g, device="cuda").to(BF)
    B = torch.randint(-2, 3, (S, d, R), generator=g, device="cuda").to(BF)
    for i, r in enumerate(ranks):
        A[i, r:] = float("nan")
        B[i, :, r:] = float("nan")
    return A, B


def layer(x, dense, ds, sets, ranks, scales, ids, twice):
    """(y in bf16, the same without adapters): y rounded once or, where `twice`,
    the base first."""
    base = x.double() @ dense.T
    add = torch.zeros_like(base)
    ids = torch.as_tensor(np.asarray(ids))
    for i, r in enumerate(ranks):
        mine = (ids == i).nonzero().flatten().cuda()
        if r <= 0 or len(mine) == 0:
            continue
        c0 = 0
        for (A, B), d in zip(sets, ds):
            t = x[mine].double() @ A[i, :r].double().T * float(scales[i])
            assert float(t.abs().max()) < 2 ** 15 and float(t.abs().sum(1).max()) < 2 ** 21
            add[mine, c0:c0 + d] += t @ B[i, :, :r].double().T
            c0 += d
    assert x.shape[1] <= 2 ** 14
    plain = base.float().to(BF)
    return ((plain.double() if twice else base) + add).float().to(BF), plain

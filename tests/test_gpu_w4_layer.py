"""The adapters' part of the 4-bit layer, where it must show: bit for bit over
whole numbers through every kernel that the layer takes, and element by element
over values as a model has them, with adapters as large as the base.

Where the layer's sums are exact (w4_exact) the result is one value: the sum
rounded once up to 32 rows, else the base product rounded to bf16 and the sum
rounded again.  `real_tolerance` derives the other bound.
"""
import numpy as np
import pytest
import torch

import lora_row_adapter_amd as lr
import test_gpu_w4 as T
import test_gpu_w4_heads as H
import w4_exact as E
from gpu_helpers import say
from test_w4_shapes_host import layer_sizes

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the gpu tests need an MI355X")
    torch.cuda.set_device(0)
    lr.load_library()
    yield
    torch.cuda.synchronize()


def device_slices(sets, ranks, scales, ds, k, R, pools, page=4096):
    cpu = [(A.cpu(), B.cpu()) for A, B in sets] if pools else sets
    rk = torch.tensor(ranks, dtype=torch.int32).cuda()
    sc = torch.tensor(scales, dtype=F32).cuda()
    out = []
    for n, ((A, B), d) in enumerate(zip(cpu, ds)):
        if pools:
            pool, table = T.paged((A, B), ranks, k, d, page=page, seed=n)
            ad = lr.Adapters.paged(pool, table, rk, page, R)
        else:
            ad = lr.Adapters.slots(A, B, rk)
        out.append(lr.Slice(d, ad, sc))
    return out


class Exact:
    """A layer over whole numbers."""

    def __init__(self, seed, M, k, ds, group, R, ranks, pools):
        self.M, self.k, self.ds, self.ranks = M, k, ds, ranks
        S = len(ranks)
        w = E.Weight(seed, sum(ds), k, group, zeros=seed % 3 > 0)
        self.W, self.dense = lr.lora_w4_pack(w.packed(), w.s, k, group, zeros=w.z), w.dense()
        self.x = E.rows(seed + 1, M, k)
        self.sets = [E.adapters(seed + 2 + i, S, R, k, d, ranks) for i, d in enumerate(ds)]
        self.scales = np.random.default_rng(seed).choice([0.5, 1.0, 2.0, 4.0], S)
        self.slices = device_slices(self.sets, ranks, self.scales, ds, k, R, pools)

    def run(self, ids, **kw):
        return lr.lora_linear_sliced_w4(self.x, self.W, self.slices, torch.from_numpy(ids.astype(np.int32)).cuda(), **kw)

    def workspace(self):
        return torch.zeros(lr.workspace_bytes_sliced_w4(self.M, self.k, self.slices), dtype=torch.uint8, device="cuda")

    def want(self, ids, twice=None):
        y, plain = E.layer(self.x, self.dense, self.ds, self.sets, self.ranks, self.scales, ids,
                           self.M > 32 if twice is None else twice)
        # adapters left out would show in every row that has one
        has = torch.tensor([0 <= i < len(self.ranks) and self.ranks[i] > 0 for i in ids]).cuda()
        assert bool((y != plain).any(1)[has].all())
        return y, plain


@pytest.mark.parametrize("pools", [False, True])
@pytest.mark.parametrize("shape,group", sorted((i, g) for i in range(21) for g in (32, 64, 128)))
def test_every_product_of_the_layer_exactly(shape, group, pools):
    """Each shape that the layer's product takes, with each size of group; the
    plan in its launch or ahead, then reused; a plan's counts."""
    M, k, d = layer_sizes()[shape, group]
    say("w4 layer shape %d: %dx%dx%d g%d pools=%d" % (shape, M, d, k, group, pools))
    assert lr.test_linear_w4_shape(M, k, d, group)[0] == shape
    ranks = [16, 5, 0, 9, 8]
    t = Exact(shape * 7 + group, M, k, (d - d // 3, d // 3), group, 16, ranks, pools)
    ids = np.random.default_rng(shape).integers(-1, 5, M)
    ids[[0, M // 2, M - 1]] = [0, 7, 1]  # 7: no adapter there is
    want, plain = t.want(ids)
    ws = t.workspace()
    assert torch.equal(t.run(ids, workspace=ws), want)
    counts = lr.lora_check(ws)
    assert (counts["n_bad_ids"], counts["n_bad_ranks"], counts["n_bad_pages"]) == (1, 0, 0)
    assert torch.equal(t.run(ids, workspace=ws, flags=lr.FLAG_REUSE_PLAN), want)
    assert torch.equal(lr.lora_gemm_w4(t.x, t.W), plain)


def id_sets(M, S, seed):
    rng = np.random.default_rng(seed)
    some = rng.integers(-1, S, M)
    some[0] = 0
    return [some, np.arange(M) % S, np.sort(rng.integers(0, S, M)), np.where(np.arange(M) == M // 2, 0, -1)]


CASES = (T.LAYERS + T.FEW +
         [(M, H.K, H.DS, 64, 16, H.RANKS) for M in (1, 7, 32, 40, 300)] +
         [(20, 904, (40, 37), 128, 8, [8, 3]), (32, 4104, (300,), 32, 256, [256, 100, 33, 200]), (3, 12680, (64,), 128, 64, [64, 63])])


@pytest.mark.parametrize("pools", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "%dx%s-%d" % (c[0], "+".join(map(str, c[2])), len(c[5])))
def test_layers_exactly(case, pools):
    M, k, ds, group, R, ranks = case
    say("w4 layer exactly %s pools=%d" % (case, pools))
    t = Exact(M + k, M, k, ds, group, R, ranks, pools)
    for n, ids in enumerate(id_sets(M, len(ranks), M)):
        assert torch.equal(t.run(ids), t.want(ids)[0])
        if n == 0:
            assert torch.equal(t.run(ids, path=lr.PATH_GATHER), t.want(ids, twice=True)[0])


@pytest.mark.parametrize("pools", [False, True])
@pytest.mark.parametrize("M", [6, 32, 100])
def test_rows_of_bad_ids_ranks_and_pages_exactly(M, pools):
    """Rows whose adapter cannot be had get the base; those beside them all of
    theirs."""
    k, ds, R = 264, (48, 30), 8
    ranks = [4, 8, 5, 8]
    t = Exact(M, M, k, ds, 64, R, ranks, pools)
    ids = np.arange(M) % 6 - 1  # -1: none; 4: no adapter there is
    t.slices = device_slices(t.sets, ranks, t.scales, ds, k, R, pools, page=1024)
    t.slices[1].adapters.ranks[1] = 99
    t.slices[0].adapters.ranks[1] = 99
    if pools:
        t.slices[1].adapters.page_table[3, 1] = 1 << 20
    ws = t.workspace()
    y = t.run(ids, workspace=ws)
    c = lr.lora_check(ws)
    n = [int((ids == i).sum()) for i in range(5)]
    assert (c["n_bad_ids"], c["n_bad_ranks"], c["n_bad_pages"]) == (n[4], n[1], n[3] if pools else 0)
    good = np.where((ids == 0) | (ids == 2) | ((ids == 3) & (not pools)), ids, -1)
    assert torch.equal(y, t.want(good)[0])


def real_tolerance(x, s, group, Wd, want, base, parts, M, k, rounds):
    """What a layer's value may be off by, per element.

    y is rounded to bf16 once, and past 32 rows the base before that (2^-8 of
    each).  The base's fp32 sums: a chain of at most 128 additions in a group,
    two for its scale and zero point, a record's groups (4 nb at most, over
    the waves or not) and 16 waves' sums, each off by 2^-23 of the magnitudes
    (code and zero point: at most 15 + 15 times |x| |s|); where the weights are
    rounded, 2^-8 of |x| |W|.  The adapters': t is a sum over chains of at most
    k / 32 + 64 additions of |x| |A|, held to 2^-16 of itself, its products with B
    are summed over at most 2 R + 16."""
    eps, nb = 2.0 ** -23, -(-k // 128)
    rep = s.double().abs().repeat_interleave(group, 1)[:, :k]
    tol = 2.0 ** -8 * want.abs() + (128 + 2 + 4 * nb + 16) * eps * 30 * (x.abs() @ rep.T)
    if M > 32:
        tol += 2.0 ** -8 * base.abs()
    if rounds:
        tol += 2.0 ** -8 * (x.abs() @ Wd.abs().T)
    for mine, c0, c1, tmag, tabs, Bm, R in parts:
        tol[mine, c0:c1] += ((k / 32 + 64) * eps * tmag + (2.0 ** -16 + (2 * R + 16) * eps) * tabs) @ Bm.abs().T
    return tol


REAL = [  # M, k, ds, group, max_rank, ranks
    (1, 8192, (300, 77), 128, 64, [64]), (5, 1032, (130, 34), 64, 64, [4, 64, 16, 0]), (16, 4104, (1000,), 32, 16, [16, 8, 12, 5]),
    (19, 1288, (33,), 128, 12, [12, 7, 1]), (30, 2056, (12555,), 64, 8, [8, 3]), (32, 520, (5, 7, 3, 40), 32, 256, [200]),
    (33, 1288, (33, 70), 128, 12, [12, 7, 1]), (64, 904, (128, 40), 32, 64, [4, 16, 64, 8]),
    (300, 1024, (288,), 128, 64, [4, 16, 64, 8]), (700, 2056, (544, 20), 64, 32, [32, 1, 8]),
    (1500, 1032, (657,), 32, 16, [16, 9, 4]), (100, 520, (64,), 64, 128, [128, 100]),
]


@pytest.mark.parametrize("pools", [False, True])
@pytest.mark.parametrize("case", REAL, ids=lambda c: "%dx%s" % (c[0], "+".join(map(str, c[2]))))
def test_real_values_element_by_element(case, pools):
    M, k, ds, group, R, ranks = case
    say("w4 layer, real values %s pools=%d" % (case, pools))
    S = len(ranks)
    g = torch.Generator(device="cuda").manual_seed(M + k)
    w = E.Weight(M, sum(ds), k, group)
    w.s = ((0.05 + torch.rand(w.s.shape, generator=g, device="cuda")) * 0.1).to(BF)
    W, Wd = lr.lora_w4_pack(w.packed(), w.s, k, group, zeros=w.z), w.dense()
    x = (torch.randn(M, k, generator=g, device="cuda") * torch.exp(torch.randn(k, generator=g, device="cuda"))).to(BF)
    xd = x.double()
    base = xd @ Wd.T
    size = float(base.pow(2).mean().sqrt())
    scales = np.random.default_rng(k).uniform(0.25, 4, S).astype(np.float32)
    sets, ids = [], np.random.default_rng(M).integers(-1, S, M)
    ids[0] = 0
    for n, d in enumerate(ds):
        A = (torch.randn(S, R, k, generator=g, device="cuda") * k ** -0.5).to(BF)
        B = torch.randn(S, d, R, generator=g, device="cuda")
        for i, r in enumerate(ranks):  # the adapter's part as large as the base
            t = xd @ A[i, :r].double().T * float(scales[i])
            B[i, :, :r] *= size / float(t.pow(2).sum(1).mean().sqrt() if r else 1)
        B = B.to(BF)
        for i, r in enumerate(ranks):
            A[i, r:], B[i, :, r:] = float("nan"), float("nan")
        sets.append((A, B))
    want, half, parts = base.clone(), base.clone(), []
    it = torch.from_numpy(ids)
    for i, r in enumerate(ranks):
        mine = (it == i).nonzero().flatten().cuda()
        c0 = 0
        for (A, B), d in zip(sets, ds):
            if r and len(mine):
                Ad, Bd, sc = A[i, :r].double(), B[i, :, :r].double(), float(scales[i])
                t = xd[mine] @ Ad.T * sc
                want[mine, c0:c0 + d] += t @ Bd.T
                half[mine, c0:c0 + d] += t[:, :r // 2] @ Bd[:, :r // 2].T
                parts.append((mine, c0, c0 + d, xd[mine].abs() @ Ad.abs().T * sc, t.abs(), Bd, r))
            c0 += d
    rounds = M > 32 and lr.test_gemm_w4_shape(M, k, sum(ds), group)[3]
    tol = real_tolerance(xd, w.s, group, Wd, want, base, parts, M, k, rounds)
    # the bound tells a layer without its adapters, or with half their ranks, from this one
    has = torch.tensor([i >= 0 and ranks[i] > 0 for i in ids]).cuda()
    for wrong in (base, half):
        assert bool(((wrong - want).abs() > tol).any(1)[has].all())
    slices = device_slices(sets, ranks, scales, ds, k, R, pools)
    y = lr.lora_linear_sliced_w4(x, W, slices, it.to(torch.int32).cuda()).double()
    say("  at most %.2f of the bound" % float(((y - want).abs() / tol).max()))
    assert bool(((y - want).abs() <= tol).all())

"""The 4-bit base weight with group scales and zero points on the GPU against
plain 64-bit implementations.

Tolerances.  One rounding to bf16 is off by at most 2^-8 of the value.  A
product rounds its fp32 sum once; w4_ref.sum_bound bounds that sum's error.
Where x holds small whole numbers and scales are powers of two every sum is
exact in fp32, in any order (|x| <= 4, 2 * 31 * 4 * k < 2^24), and so is every
weight in bf16: the result is then the exact one rounded once, bit for bit.
"""
import numpy as np
import pytest
import torch

import lora_row_adapter_amd as lr
from lora_row_adapter_amd import workloads as wl
import w4_ref as R
from gpu_helpers import normwise, say

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


def device_weight(q, s, z, group):
    return lr.lora_w4_pack(torch.from_numpy(R.pack(q)).cuda(), s.cuda(), q.shape[1], group,
                           zeros=None if z is None else torch.from_numpy(z).cuda())


def whole(seed, M, k, most=4):
    return torch.from_numpy(np.random.default_rng(seed).integers(-most, most + 1, (M, k)).astype(np.float32)).to(BF)


def loud(seed, M, k):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, k, generator=g) * torch.exp(1.2 * torch.randn(k, generator=g))).to(BF)


# ------------------------------------------------------------ layout, reading back
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("d,k,group", [(1, 1, 32), (1, 128, 128), (16, 128, 64), (17, 129, 32), (5, 1000, 128),
                                       (33, 500, 64), (100, 257, 256), (48, 4096, 384), (31, 320, 1024)])
def test_read_back_exactly(d, k, group, zeros):
    say("w4 read back %dx%d g%d" % (d, k, group))
    for dtype in (BF, F32):
        q, s, z = R.weight(d + k, d, k, group, zeros, dtype)
        W = device_weight(q, s, z, group)
        want = torch.from_numpy(R.dequant(q, R.kept(s), z, group))
        assert torch.equal(lr.lora_w4_dequantize(W, F32).cpu().double(), want)
        # one rounding: the exact products have at most 24 bits
        assert torch.equal(lr.lora_w4_dequantize(W, BF).cpu(), want.float().to(BF))


def test_every_code_and_zero_point():
    k = 32 * 16
    q = np.tile(np.arange(16, dtype=np.uint8), (40, 32))
    z = (np.arange(40)[:, None] + np.arange(16)[None] * 7).astype(np.uint8)  # past 31 too: modulo 32
    s = torch.ones(40, 16, dtype=F32)
    W = device_weight(q, s, z, 32)
    assert torch.equal(lr.lora_w4_dequantize(W, F32).cpu().double(), torch.from_numpy(R.dequant(q, s, z, 32)))
    x = torch.eye(k, dtype=BF)[:64].cuda()
    y = lr.lora_gemm_w4(x, W)
    assert torch.equal(y.cpu().double(), torch.from_numpy(R.dequant(q, s, z, 32)[:, :64].T))


def test_fp32_scales_are_rounded_to_19_bits():
    s = torch.randn(64, 4, generator=torch.Generator().manual_seed(1))
    s[0, 0], s[0, 1], s[1, 0], s[2, 0] = float("inf"), float("nan"), 0.0, -0.0
    s[3, 0] = 1 + 2.0 ** -19  # a tie
    s[3, 1] = 1 + 3 * 2.0 ** -19
    q = np.full((64, 128), 9, np.uint8)
    z = np.full((64, 4), 8, np.uint8)
    got = lr.lora_w4_dequantize(device_weight(q, s, z, 32), F32).cpu()[:, ::32].double()
    want = R.kept(s)
    want[0, 0], want[0, 1] = float("inf"), float("nan")
    assert torch.equal(torch.nan_to_num(got, nan=7.5), torch.nan_to_num(want, nan=7.5))


def test_pack_reads_strided_inputs_and_writes_out_only():
    d, k, group = 21, 200, 64
    q, s, z = R.weight(3, d, k, group)
    wide_q = torch.full((d, 133), 0xAB, dtype=torch.uint8).cuda()
    wide_q[:, 3:103] = torch.from_numpy(R.pack(q)).cuda()
    wide_s = torch.full((d, 9), float("nan"), dtype=BF).cuda()
    wide_s[:, 2:6] = s.cuda()
    wide_z = torch.full((d, 7), 255, dtype=torch.uint8).cuda()
    wide_z[:, 1:5] = torch.from_numpy(z).cuda()
    n = lr.W4.bytes(d, k, group)
    buf = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    W = lr.lora_w4_pack(wide_q[:, 3:103], wide_s[:, 2:6], k, group, zeros=wide_z[:, 1:5], out=buf[256:256 + n])
    assert torch.equal(lr.lora_w4_dequantize(W, F32).cpu().double(), torch.from_numpy(R.dequant(q, s, z, group)))
    assert bool((buf[:256] == 0x5A).all()) and bool((buf[256 + n:] == 0x5A).all())
    y = torch.full((d, k + 5), 3.0, dtype=BF, device="cuda")
    lr.lora_w4_dequantize(W, BF, out=y[:, 1:k + 1])
    assert torch.equal(y[:, 1:k + 1].cpu(), torch.from_numpy(R.dequant(q, s, z, group)).float().to(BF))
    assert bool((y[:, 0] == 3).all()) and bool((y[:, k + 1:] == 3).all())


# ------------------------------------------------------------ product
SIZES = [  # M, k, d, group
    (1, 8, 1, 32), (1, 128, 16, 128), (1, 136, 17, 64), (1, 5000, 65, 32), (1, 8192, 300, 128), (2, 1024, 64, 32),
    (3, 264, 33, 128), (4, 4096, 48, 256), (5, 1000, 100, 64), (7, 2056, 31, 32), (8, 384, 256, 128),
    (15, 640, 40, 64), (16, 4096, 130, 128), (17, 512, 80, 32), (31, 904, 60, 128), (32, 1024, 257, 64),
    (33, 136, 128, 128), (48, 2000, 50, 32), (63, 768, 96, 128), (64, 4096, 64, 64), (65, 320, 200, 32),
    (100, 1032, 144, 128), (127, 256, 129, 64), (128, 640, 128, 128), (129, 2048, 63, 32), (200, 520, 320, 512),
    (255, 128, 511, 128), (256, 1024, 256, 64), (300, 904, 250, 32), (511, 384, 130, 128), (513, 264, 385, 64),
    (1000, 512, 200, 128), (1030, 136, 96, 32), (2048, 1024, 512, 128), (4097, 264, 130, 64),
]


@pytest.mark.parametrize("M,k,d,group", SIZES)
def test_product_of_whole_numbers_exactly(M, k, d, group):
    say("w4 product %dx%dx%d g%d, whole numbers" % (M, d, k, group))
    q, s, z = R.weight(M + k + d, d, k, group, zeros=d % 2 == 0, exact=True)
    x = whole(M, M, k)
    y = lr.lora_gemm_w4(x.cuda(), device_weight(q, s, z, group))
    want = torch.from_numpy(x.double().numpy() @ R.dequant(q, s, z, group).T).float().to(BF)
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("M,k,d,group", SIZES)
def test_product(M, k, d, group):
    say("w4 product %dx%dx%d g%d" % (M, d, k, group))
    q, s, z = R.weight(M * 3 + k + d, d, k, group, zeros=d % 2 == 1)
    x = loud(k, M, k)
    y = lr.lora_gemm_w4(x.cuda(), device_weight(q, s, z, group)).cpu().double().numpy()
    xd, Wd = x.double().numpy(), R.dequant(q, s, z, group)
    want = xd @ Wd.T
    tol = 2.0 ** -8 * np.abs(want) + R.sum_bound(xd, s, z, group)
    if lr.test_gemm_w4_shape(M, k, d, group)[3]:  # each weight rounded once to bf16
        tol += 2.0 ** -8 * (np.abs(xd) @ np.abs(Wd).T)
    assert (np.abs(y - want) <= tol).all()


# a size for every tile shape, its sizes odd and k past every ring of stages
def one_for_each_shape():
    found = {}
    for M in (1, 3, 16, 30, 60, 100, 200, 300, 500, 800, 1100, 1500, 2100, 3000):
        for d in (33, 300, 1000, 2050, 4100):
            for k in (1032, 2056):
                for group in (32, 64, 128):
                    shape = lr.test_gemm_w4_shape(M, k, d, group)
                    found.setdefault((shape[0], min(group, 128)), (M, k, d, group))
    return found


def test_every_tile_shape_exactly():
    found = one_for_each_shape()
    assert len({i for i, _ in found}) >= 12
    for (i, _), (M, k, d, group) in sorted(found.items()):
        say("w4 shape %d: %dx%dx%d g%d" % (i, M, d, k, group))
        q, s, z = R.weight(M + d, d, k, group, exact=True)
        x = whole(M, M, k)
        y = lr.lora_gemm_w4(x.cuda(), device_weight(q, s, z, group))
        want = (x.cuda().double() @ torch.from_numpy(R.dequant(q, s, z, group)).cuda().T).float().to(BF)
        assert torch.equal(y, want)


@pytest.mark.parametrize("M", [1, 4, 16, 40, 130, 700])
def test_product_of_strided_views(M):
    """x and y are columns of wide buffers; nothing past a row is written, and
    what lies past a row of x is not read into the sums."""
    k, d, group = 904, 77, 128
    say("w4 product of views, %d rows" % M)
    q, s, z = R.weight(M, d, k, group, exact=True)
    W = device_weight(q, s, z, group)
    x = whole(M, M, k)
    wide = torch.full((M, k + 40), float("nan"), dtype=BF, device="cuda")
    wide[:, 16:16 + k] = x.cuda()
    out = torch.full((M, d + 9), 5.0, dtype=BF, device="cuda")
    lr.lora_gemm_w4(wide[:, 16:16 + k], W, y=out[:, 3:3 + d])
    want = torch.from_numpy(x.double().numpy() @ R.dequant(q, s, z, group).T).float().to(BF)
    assert torch.equal(out[:, 3:3 + d].cpu(), want)
    assert bool((out[:, :3] == 5).all()) and bool((out[:, 3 + d:] == 5).all())


def test_product_of_far_rows():
    """Rows of x more than 2^32 bytes apart (the last tokens of long sequences)."""
    k, d = 256, 40
    q, s, z = R.weight(9, d, k, 64, exact=True)
    W = device_weight(q, s, z, 64)
    x = whole(5, 3, k)
    far = torch.empty(2 * (1 << 31) + 4096, dtype=BF, device="cuda")
    view = far.as_strided((3, k), (1 << 31, 1))
    view.copy_(x.cuda())
    y = lr.lora_gemm_w4(view, W)
    want = torch.from_numpy(x.double().numpy() @ R.dequant(q, s, z, 64).T).float().to(BF)
    assert torch.equal(y.cpu(), want)
    # and many rows of a stride just past a tile's 32-bit offsets
    x = whole(6, 100, k)
    view = far.as_strided((100, k), (1 << 23, 1))
    view.copy_(x.cuda())
    y = lr.lora_gemm_w4(view, W)
    want = torch.from_numpy(x.double().numpy() @ R.dequant(q, s, z, 64).T).float().to(BF)
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("M,d", [((1 << 18) + 70, 24), (3, (1 << 20) + 40), (70, (1 << 20) + 17)])
def test_product_past_a_slab(M, d):
    """More rows, or columns, than one launch takes."""
    k = 64
    q, s, z = R.weight(1, d, k, 32, exact=True)
    x = whole(2, M, k)
    y = lr.lora_gemm_w4(x.cuda(), device_weight(q, s, z, 32))
    want = (x.cuda().float() @ torch.from_numpy(R.dequant(q, s, z, 32)).float().cuda().T).to(BF)  # exact in fp32
    assert torch.equal(y, want)


def test_empty_batch():
    q, s, z = R.weight(2, 20, 256, 128)
    W = device_weight(q, s, z, 128)
    assert lr.lora_gemm_w4(torch.empty(0, 256, dtype=BF, device="cuda"), W).shape == (0, 20)


@pytest.mark.parametrize("M", [1, 16, 50, 600])
def test_nan_and_infinity_stay_in_their_row(M):
    q, s, z = R.weight(4, 70, 512, 64)
    W = device_weight(q, s, z, 64)
    x = loud(3, M, 512).cuda()
    clean = lr.lora_gemm_w4(x, W)
    bad = x.clone()
    bad[M // 2, 77] = float("nan")
    bad[M - 1, 500] = float("inf")
    y = lr.lora_gemm_w4(bad, W)
    assert bool(torch.isnan(y[M // 2]).all())
    assert not bool(torch.isfinite(y[M - 1]).any())
    rest = [m for m in range(M) if m not in (M // 2, M - 1)]
    assert torch.equal(y[rest], clean[rest])


@pytest.mark.parametrize("M", [1, 16, 64, 300])
def test_product_runs_alike_each_time(M):
    q, s, z = R.weight(6, 513, 2056, 32)
    W = device_weight(q, s, z, 32)
    x = loud(8, M, 2056).cuda()
    first = lr.lora_gemm_w4(x, W)
    for _ in range(5):
        assert torch.equal(lr.lora_gemm_w4(x, W), first)


# ------------------------------------------------------------ layer
def adapter_set(seed, S, R_, k, d, ranks, exact=False, pad=0.0):
    """Slot tensors whose padding holds `pad`, and float64 A, B lists."""
    g = torch.Generator().manual_seed(seed)
    A = torch.full((S, R_, k), pad).to(BF)
    B = torch.full((S, d, R_), pad).to(BF)
    for i, r in enumerate(ranks):
        if exact:
            A[i, :r] = torch.randint(-1, 2, (r, k), generator=g).to(BF)
            B[i, :, :r] = torch.randint(-2, 3, (d, r), generator=g).to(BF)
        else:
            A[i, :r] = (torch.randn(r, k, generator=g) * k ** -0.5).to(BF)
            B[i, :, :r] = (torch.randn(d, r, generator=g) * 0.2).to(BF)
    return A, B


def layer_ref(x, Wd, ds, sets, ranks, scales, ids):
    """float64 layer; sets: (A, B) per slice."""
    xd = x.double().numpy()
    y = xd @ Wd.T
    for m, i in enumerate(ids):
        if i < 0:
            continue
        c0 = 0
        for (A, B), d in zip(sets, ds):
            r = int(ranks[i])
            t = xd[m] @ A[i, :r].double().numpy().T
            y[m, c0:c0 + d] += scales[i] * (B[i, :, :r].double().numpy() @ t)
            c0 += d
    return y


def paged(sets_i, ranks, k, d, page=4096, seed=0):
    """The same adapters in a pool of pages handed out in a shuffled order."""
    A, B = sets_i
    rng = np.random.default_rng(seed)
    spaces = []
    for i, r in enumerate(ranks):
        raw = torch.cat([A[i, :r].reshape(-1), B[i, :, :r].reshape(-1)]).view(torch.uint8).numpy()
        spaces.append(np.pad(raw, (0, -len(raw) % page)))
    n = sum(len(s) // page for s in spaces)
    order = rng.permutation(n + 3)
    width = max(1, max(len(s) // page for s in spaces))
    pool = np.full((n + 3, page), 0xFF, np.uint8)
    table = np.full((len(ranks), width), -1, np.int32)
    at = 0
    for i, s in enumerate(spaces):
        for j in range(len(s) // page):
            pool[order[at]] = s[j * page:(j + 1) * page]
            table[i, j] = order[at]
            at += 1
    return torch.from_numpy(pool.reshape(-1)).cuda(), torch.from_numpy(table).cuda()


def device_slices(sets, ranks, scales, ds, k, R_, pools=False):
    rk = torch.tensor(ranks, dtype=torch.int32).cuda()
    sc = torch.tensor(scales, dtype=F32).cuda()
    out = []
    for n, ((A, B), d) in enumerate(zip(sets, ds)):
        if pools:
            pool, table = paged((A, B), ranks, k, d, seed=n)
            ad = lr.Adapters.paged(pool, table, rk, 4096, R_)
        else:
            ad = lr.Adapters.slots(A.cuda(), B.cuda(), rk)
        out.append(lr.Slice(d, ad, sc))
    return out


LAYERS = [  # M, k, ds, group, max_rank, ranks
    (1, 256, (64,), 128, 16, [16]),
    (1, 1000, (130, 34), 64, 64, [4, 64, 16, 0]),
    (2, 136, (18,), 32, 8, [8, 3]),
    (5, 2048, (256, 32, 32), 128, 32, [32, 8, 4, 16, 1]),
    (8, 512, (50, 50), 32, 128, [100, 128, 7]),
    (16, 1032, (300,), 128, 64, [64, 32, 16, 8, 4, 64, 64]),
    (17, 512, (96, 30), 64, 16, [16, 9]),
    (64, 904, (128, 40), 32, 64, [4, 16, 64, 8]),
    (300, 1024, (288,), 128, 64, [4, 16, 64, 8]),
    (700, 264, (144, 20), 64, 32, [32, 1, 8]),
]


@pytest.mark.parametrize("pools", [False, True])
@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "%dx%s" % (c[0], "+".join(map(str, c[2]))))
def test_layer(case, pools):
    M, k, ds, group, R_, ranks = case
    say("w4 layer %s pools=%d" % (case, pools))
    S = len(ranks)
    rng = np.random.default_rng(M)
    ids = rng.integers(-1, S, M).astype(np.int32)
    ids[0] = 0
    scales = rng.uniform(0.25, 4, S).astype(np.float32)
    q, s, z = R.weight(M, sum(ds), k, group)
    W = device_weight(q, s, z, group)
    sets = [adapter_set(7 + i, S, R_, k, d, ranks, pad=float("nan")) for i, d in enumerate(ds)]
    x = loud(M, M, k)
    slices = device_slices(sets, ranks, scales, ds, k, R_, pools)
    ids_d = torch.from_numpy(ids).cuda()
    ws = torch.zeros(lr.workspace_bytes_sliced_w4(M, k, slices), dtype=torch.uint8, device="cuda")
    want = layer_ref(x, R.dequant(q, s, z, group), ds, sets, ranks, scales.astype(np.float64), ids)
    base = lr.lora_gemm_w4(x.cuda(), W)
    none = torch.from_numpy(np.flatnonzero(ids < 0)).cuda()
    for path in (lr.PATH_AUTO, lr.PATH_GATHER):
        y = lr.lora_linear_sliced_w4(x.cuda(), W, slices, ids_d, workspace=ws, path=path)
        err = normwise(y.double().cpu().numpy(), want)
        say("  path %d normwise %.3g" % (path, err))
        assert err <= 2e-2
        assert torch.equal(y[none], base[none])
        chk = lr.lora_check(ws)
        assert chk["n_bad_ids"] == chk["n_bad_ranks"] == chk["n_bad_pages"] == chk["n_sync_expired"] == 0


FEW = [  # M, k, ds, group, max_rank, ranks: at and around 32 and 64 rows
    (32, 520, (5, 7, 3, 40), 32, 256, [200]),
    (32, 264, (48, 17), 64, 64, list(range(1, 33))),
    (19, 1288, (33,), 128, 12, [12, 7, 1]),
    (9, 4104, (16, 300), 128, 96, [96, 8, 64, 72, 0]),
    (16, 136, (300, 4500), 128, 20, [20, 16, 3]),
    (30, 1032, (8200,), 64, 8, [8, 3]),
    (33, 264, (48, 17), 64, 64, list(range(1, 34))),
    (64, 520, (5, 7, 3, 40), 32, 256, [200]),             # one adapter's rows; slices inside 16 columns
    (64, 264, (48, 17), 64, 64, list(range(1, 65))),      # an adapter for every row
    (33, 1288, (33,), 128, 12, [12, 7, 1]),               # B's rows no whole vectors
    (48, 4104, (16, 300), 128, 96, [96, 8, 64, 72, 0]),   # more than 64 ranks, k past what a workgroup takes
    (65, 264, (48, 17), 64, 64, list(range(1, 65))),
]


@pytest.mark.parametrize("pools", [False, True])
@pytest.mark.parametrize("case", FEW, ids=lambda c: "%dx%s" % (c[0], "+".join(map(str, c[2]))))
def test_layer_of_few_rows(case, pools):
    M, k, ds, group, R_, ranks = case
    say("w4 layer of few rows %s pools=%d" % (case, pools))
    S = len(ranks)
    rng = np.random.default_rng(M + S)
    scales = rng.uniform(0.25, 4, S).astype(np.float32)
    q, s, z = R.weight(M, sum(ds), k, group)
    W = device_weight(q, s, z, group)
    sets = [adapter_set(17 + i, S, R_, k, d, ranks, pad=float("nan")) for i, d in enumerate(ds)]
    x = loud(M, M, k)
    slices = device_slices(sets, ranks, scales, ds, k, R_, pools)
    base = lr.lora_gemm_w4(x.cuda(), W)
    for ids in (np.arange(M) % S, np.sort(rng.integers(0, S, M)), np.where(np.arange(M) == M // 2, S - 1, -1)):
        ids = ids.astype(np.int32)
        y = lr.lora_linear_sliced_w4(x.cuda(), W, slices, torch.from_numpy(ids).cuda())
        want = layer_ref(x, R.dequant(q, s, z, group), ds, sets, ranks, scales.astype(np.float64), ids)
        err = normwise(y.double().cpu().numpy(), want)
        say("  normwise %.3g" % err)
        assert err <= 2e-2
        none = np.flatnonzero(ids < 0)
        assert torch.equal(y[none], base[none])


@pytest.mark.parametrize("M", [20, 64])
def test_layer_keeps_an_adapters_nan_to_its_rows(M):
    k, ds, ranks = 264, (40, 9), [8, 16, 5]
    q, s, z = R.weight(2, sum(ds), k, 64)
    W = device_weight(q, s, z, 64)
    sets = [adapter_set(5 + i, 3, 16, k, d, ranks) for i, d in enumerate(ds)]
    ids = torch.arange(M, dtype=torch.int32).cuda() % 3
    x = loud(2, M, k).cuda()
    run = lambda: lr.lora_linear_sliced_w4(x, W, device_slices(sets, ranks, [1.0] * 3, ds, k, 16), ids)
    clean = run()
    for A, B in sets:
        A[1] = float("nan")
        B[1, ::2] = float("inf")
    y = run()
    other = ids.cpu() != 1
    assert torch.equal(y[other], clean[other])
    assert y[~other].isnan().all()
    for A, B in sets:  # an infinite t times finite B
        A[1] = 3e38
        B[1] = 1.0
    y = run()
    assert torch.equal(y[other], clean[other])
    assert not torch.isfinite(y[~other].float()).any()


@pytest.mark.parametrize("d", [64, 16 * 512, 16 * 768])  # tiles that leave room beside them, and do not
@pytest.mark.parametrize("M", [1, 16, 40, 64, 150])
def test_plan_is_left_and_reused(M, d):
    """The plan a call makes serves a dense layer of the same rows, and the
    other way about; a call that reuses one leaves it as it is."""
    k, ranks = 128, [4, 16, 9, 0, 7]
    say("w4 plan %d %d" % (M, d))
    q, s, z = R.weight(3, d, k, 64)
    W = device_weight(q, s, z, 64)
    Wd = lr.lora_w4_dequantize(W)
    slices = device_slices([adapter_set(1, 5, 16, k, d, ranks)], ranks, [1.0, 2.0, 0.5, 1.0, 3.0], (d,), k, 16)
    ids = torch.from_numpy(np.random.default_rng(M).integers(-2, 7, M).astype(np.int32)).cuda()
    x = loud(4, M, k).cuda()
    n = max(lr.workspace_bytes_sliced_w4(M, k, slices), lr.workspace_bytes_sliced(M, k, BF, slices))
    new = lambda: torch.zeros(n, dtype=torch.uint8, device="cuda")
    four = lambda ws, flags=0: lr.lora_linear_sliced_w4(x, W, slices, ids, workspace=ws, flags=flags)
    dense = lambda ws, flags=0: lr.lora_linear_sliced(x, Wd, slices, ids, workspace=ws, flags=flags)
    ws, other = new(), new()
    y = four(ws)
    counts = lr.lora_check(ws)
    assert torch.equal(dense(ws, lr.FLAG_REUSE_PLAN), dense(other))
    assert {n: v for n, v in lr.lora_check(other).items()} == counts
    assert torch.equal(four(other, lr.FLAG_REUSE_PLAN), y)
    assert torch.equal(dense(other, lr.FLAG_REUSE_PLAN), dense(new()))
    assert torch.equal(four(ws, lr.FLAG_REUSE_PLAN), y)


@pytest.mark.parametrize("pools", [False, True])
@pytest.mark.parametrize("M", [1, 3, 16, 33, 200])
def test_layer_of_whole_numbers_exactly(M, pools):
    """Every sum exact in fp32 (t within 16 bits): the layer's value rounded
    once where it is rounded once, and at most twice."""
    k, ds, group, R_, ranks = 136, (48, 30), 32, 16, [16, 5, 0, 9]
    say("w4 layer whole numbers %d pools=%d" % (M, pools))
    rng = np.random.default_rng(M)
    ids = rng.integers(-1, 4, M).astype(np.int32)
    scales = np.array([1, 2, 0.5, 4], np.float32)
    q, s, z = R.weight(M, sum(ds), k, group, exact=True)
    W = device_weight(q, s, z, group)
    sets = [adapter_set(70 + i, 4, R_, k, d, ranks, exact=True) for i, d in enumerate(ds)]
    x = whole(M, M, k)
    slices = device_slices(sets, ranks, scales, ds, k, R_, pools)
    y = lr.lora_linear_sliced_w4(x.cuda(), W, slices, torch.from_numpy(ids).cuda()).cpu().double().numpy()
    Wd = R.dequant(q, s, z, group)
    want = layer_ref(x, Wd, ds, sets, ranks, scales.astype(np.float64), ids)
    base = x.double().numpy() @ Wd.T
    assert (np.abs(y - want) <= 2.0 ** -8 * (np.abs(want) + np.abs(base))).all()


def check_whole_layer(x, Wq, ds, sets, ranks, scales, ids, group, y):
    """As in test_layer_of_whole_numbers_exactly."""
    Wd = R.dequant(*Wq, group)
    want = layer_ref(x, Wd, ds, sets, ranks, scales, ids)
    base = x.double().numpy() @ Wd.T
    got = y.cpu().double().numpy()
    assert (np.abs(got - want) <= 2.0 ** -8 * (np.abs(want) + np.abs(base))).all()


@pytest.mark.parametrize("pools", [False, True])
@pytest.mark.parametrize("M", [1, 5, 20, 100])
def test_layer_of_views(M, pools):
    """x and y are columns of wide buffers, y's at an odd place; nothing past
    a row is written or read into the sums."""
    k, ds, group, ranks = 904, (40, 37), 128, [8, 3]
    q = R.weight(M, sum(ds), k, group, exact=True)
    sets = [adapter_set(30 + i, 2, 8, k, d, ranks, exact=True) for i, d in enumerate(ds)]
    ids = (np.arange(M) % 3 - 1).astype(np.int32)
    x = whole(M, M, k)
    wide = torch.full((M, k + 40), float("nan"), dtype=BF, device="cuda")
    wide[:, 16:16 + k] = x.cuda()
    out = torch.full((M, sum(ds) + 9), 5.0, dtype=BF, device="cuda")
    lr.lora_linear_sliced_w4(wide[:, 16:16 + k], device_weight(*q, group),
                             device_slices(sets, ranks, [1.0, 2.0], ds, k, 8, pools), torch.from_numpy(ids).cuda(),
                             y=out[:, 3:3 + sum(ds)])
    check_whole_layer(x, q, ds, sets, ranks, [1.0, 2.0], ids, group, out[:, 3:3 + sum(ds)])
    assert bool((out[:, :3] == 5).all()) and bool((out[:, 3 + sum(ds):] == 5).all())


@pytest.mark.parametrize("M,far", [(3, 1 << 31), (30, 1 << 24), (100, 1 << 23)])
def test_layer_of_far_rows(M, far):
    k, d, ranks = 256, 40, [8, 3]
    q = R.weight(9, d, k, 64, exact=True)
    sets = [adapter_set(30, 2, 8, k, d, ranks, exact=True)]
    ids = (np.arange(M) % 3 - 1).astype(np.int32)
    x = whole(5, M, k)
    view = torch.empty((M - 1) * far + k, dtype=BF, device="cuda").as_strided((M, k), (far, 1))
    view.copy_(x.cuda())
    y = lr.lora_linear_sliced_w4(view, device_weight(*q, 64), device_slices(sets, ranks, [1.0, 2.0], (d,), k, 8),
                                 torch.from_numpy(ids).cuda())
    check_whole_layer(x, q, (d,), sets, ranks, [1.0, 2.0], ids, 64, y)


@pytest.mark.parametrize("M", [2, 40])
def test_layer_past_a_slab(M):
    """More columns than one launch of the product takes."""
    k, d, ranks = 64, (1 << 20) + 40, [4, 2]
    q = R.weight(1, d, k, 64, exact=True)
    sets = [adapter_set(3, 2, 8, k, d, ranks, exact=True)]
    ids = (np.arange(M) % 3 - 1).astype(np.int32)
    x = whole(3, M, k)
    y = lr.lora_linear_sliced_w4(x.cuda(), device_weight(*q, 64), device_slices(sets, ranks, [1.0, 2.0], (d,), k, 8),
                                 torch.from_numpy(ids).cuda())
    check_whole_layer(x, q, (d,), sets, ranks, [1.0, 2.0], ids, 64, y)


@pytest.mark.parametrize("M", [6, 100])
def test_layer_counts_bad_rows_and_serves_them_the_base(M):
    k, d, ranks = 256, 64, [4, 99, -2, 8]
    q, s, z = R.weight(1, d, k, 128)
    W = device_weight(q, s, z, 128)
    A, B = adapter_set(3, 4, 8, k, d, [4, 8, 8, 8])
    slices = [lr.Slice(d, lr.Adapters.slots(A.cuda(), B.cuda(), torch.tensor(ranks, dtype=torch.int32).cuda()),
                       torch.ones(4, device="cuda"))]
    ids = np.full(M, -1, np.int32)
    ids[:6] = [0, 1, 2, 3, 4, -7]
    x = loud(2, M, k)
    ws = torch.zeros(lr.workspace_bytes_sliced_w4(M, k, slices), dtype=torch.uint8, device="cuda")
    y = lr.lora_linear_sliced_w4(x.cuda(), W, slices, torch.from_numpy(ids).cuda(), workspace=ws)
    chk = lr.lora_check(ws)
    assert (chk["n_bad_ids"], chk["n_bad_ranks"], chk["n_bad_pages"]) == (2, 2, 0)
    base = lr.lora_gemm_w4(x.cuda(), W)
    plain = [m for m in range(M) if m not in (0, 3)]
    assert torch.equal(y[plain], base[plain])
    good = np.where((ids == 0) | (ids == 3), ids, -1)
    want = layer_ref(x, R.dequant(q, s, z, 128), (d,), [(A, B)], [4, 0, 0, 8], np.ones(4), good)
    assert normwise(y.double().cpu().numpy(), want) <= 2e-2


@pytest.mark.parametrize("M", [4, 60])
def test_layer_counts_bad_pages(M):
    """An adapter with a page outside the pool serves its rows the base."""
    k, d, ranks = 256, 64, [4, 8]
    q, s, z = R.weight(1, d, k, 128)
    W = device_weight(q, s, z, 128)
    sets = adapter_set(3, 2, 8, k, d, ranks)
    pool, table = paged(sets, ranks, k, d, page=1024)
    rk = torch.tensor(ranks, dtype=torch.int32).cuda()
    bad = table.clone()
    bad[1, 2] = 1 << 20
    ids = torch.tensor([0, 1] * (M // 2), dtype=torch.int32).cuda()
    x = loud(2, M, k).cuda()
    sl = [lr.Slice(d, lr.Adapters.paged(pool, bad, rk, 1024, 8), torch.ones(2, device="cuda"))]
    ws = torch.zeros(lr.workspace_bytes_sliced_w4(M, k, sl), dtype=torch.uint8, device="cuda")
    y = lr.lora_linear_sliced_w4(x, W, sl, ids, workspace=ws)
    chk = lr.lora_check(ws)
    assert (chk["n_bad_ids"], chk["n_bad_ranks"], chk["n_bad_pages"]) == (0, 0, M // 2)
    assert torch.equal(y[1::2], lr.lora_gemm_w4(x, W)[1::2])


def test_layer_past_the_plan_limit():
    """More rows than one plan holds."""
    M, k, d = 8192 + 100, 128, 32
    q, s, z = R.weight(1, d, k, 128, exact=True)
    W = device_weight(q, s, z, 128)
    A, B = adapter_set(3, 2, 8, k, d, [8, 4], exact=True)
    slices = device_slices([(A, B)], [8, 4], [1.0, 2.0], (d,), k, 8)
    ids = (np.arange(M) % 3 - 1).astype(np.int32)
    x = whole(3, M, k)
    y = lr.lora_linear_sliced_w4(x.cuda(), W, slices, torch.from_numpy(ids).cuda()).cpu().double().numpy()
    Wd = R.dequant(q, s, z, 128)
    want = layer_ref(x, Wd, (d,), [(A, B)], [8, 4], [1.0, 2.0], ids)
    assert (np.abs(y - want) <= 2.0 ** -8 * (np.abs(want) + np.abs(x.double().numpy() @ Wd.T))).all()


@pytest.mark.parametrize("M", [1, 16, 200])
def test_captured_layer_replays(M):
    """A captured product and layer, replayed with eager work between, on other
    inputs and ids each time."""
    k, ds, ranks = 512, (96, 32), [16, 4, 8]
    q, s, z = R.weight(1, sum(ds), k, 64)
    W = device_weight(q, s, z, 64)
    sets = [adapter_set(3 + i, 3, 16, k, d, ranks) for i, d in enumerate(ds)]
    slices = device_slices(sets, ranks, [1.0, 2.0, 0.5], ds, k, 16)
    x, ids = loud(1, M, k).cuda(), torch.zeros(M, dtype=torch.int32, device="cuda")
    y, y0 = (torch.empty(M, sum(ds), dtype=BF, device="cuda") for _ in range(2))
    ws = torch.zeros(lr.workspace_bytes_sliced_w4(M, k, slices), dtype=torch.uint8, device="cuda")

    def go():
        lr.lora_gemm_w4(x, W, y=y0)
        lr.lora_linear_sliced_w4(x, W, slices, ids, y=y, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for n in range(4):
        x.copy_(loud(10 + n, M, k))
        ids.copy_(torch.from_numpy(np.random.default_rng(n).integers(-1, 3, M).astype(np.int32)))
        g.replay()
        a, b = y.clone(), y0.clone()
        go()
        torch.cuda.synchronize()
        assert torch.equal(a, y) and torch.equal(b, y0)


@pytest.mark.parametrize("M", [3, 150])
def test_two_streams(M):
    """Layers on two streams with a workspace each, and made under their stream."""
    k, d, ranks = 1024, 128, [16, 4]
    q, s, z = R.weight(1, d, k, 128)
    W = device_weight(q, s, z, 128)
    sets = [adapter_set(3, 2, 16, k, d, ranks)]
    slices = device_slices(sets, ranks, [1.0, 2.0], (d,), k, 16)
    xs = [loud(i, M, k).cuda() for i in range(2)]
    ids = torch.from_numpy((np.arange(M) % 3 - 1).astype(np.int32)).cuda()
    want = [lr.lora_linear_sliced_w4(x, W, slices, ids) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [lr.lora_linear_sliced_w4(x, W, slices, ids, stream=st) for x, st in zip(xs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------ the binding's refusals
def test_binding_refuses():
    q, s, z = R.weight(1, 32, 256, 128)
    qd, sd, zd = torch.from_numpy(R.pack(q)).cuda(), s.cuda(), torch.from_numpy(z).cuda()
    for bad in [dict(q=qd.float()), dict(q=qd.cpu()), dict(q=qd[:, :100]), dict(q=qd.t()), dict(scales=sd.half()),
                dict(scales=sd[:, :1]), dict(scales=sd.cpu()), dict(zeros=zd.int()), dict(zeros=zd[:5]),
                dict(group=48), dict(k=0), dict(out=torch.empty(8, dtype=torch.uint8, device="cuda")),
                dict(out=torch.empty(1 << 16, dtype=torch.uint8, device="cuda")[1:])]:
        kw = dict(dict(q=qd, scales=sd, k=256, group=128, zeros=zd), **bad)
        with pytest.raises((TypeError, ValueError, lr.LoraError)):
            lr.lora_w4_pack(kw.pop("q"), kw.pop("scales"), **kw)
    W = device_weight(q, s, z, 128)
    x = torch.zeros(4, 256, dtype=BF, device="cuda")
    for args, kw in [((x.float(), W), {}), ((x[:, :128], W), {}), ((x.cpu(), W), {}),
                     ((x, W), dict(y=torch.empty(4, 31, dtype=BF, device="cuda"))),
                     ((x, W), dict(y=torch.empty(4, 32, device="cuda")))]:
        with pytest.raises((TypeError, ValueError, lr.LoraError)):
            lr.lora_gemm_w4(*args, **kw)
    A, B = adapter_set(1, 2, 8, 256, 32, [8, 8])
    rk, ones = torch.tensor([8, 8], dtype=torch.int32).cuda(), torch.ones(2, device="cuda")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    good = [lr.Slice(32, lr.Adapters.slots(A.cuda(), B.cuda(), rk), ones)]
    lr.lora_linear_sliced_w4(x, W, good, ids)
    for sl, i in [([lr.Slice(31, good[0].adapters, ones)], ids), (good, ids[:3]), (good, ids.long()), (good, ids.cpu()),
                  ([lr.Slice(32, good[0].adapters, ones[:1])], ids),
                  ([lr.Slice(32, lr.Adapters.slots(A.cuda()[:, :, :128].contiguous(), B.cuda(), rk), ones)], ids),
                  ([lr.Slice(32, lr.Adapters.slots(A.cuda().float(), B.cuda().float(), rk), ones)], ids)]:
        with pytest.raises((TypeError, ValueError, lr.LoraError)):
            lr.lora_linear_sliced_w4(x, W, sl, i)

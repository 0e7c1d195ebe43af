"""Microscaled operators on the GPU against plain 64-bit implementations.

Tolerances.  One rounding to a type is off by at most half a step, eps / 2 of
the type relative to the value.  Quantising and reading back are exact: codes,
scales and values are compared for equality.  The norm computes in 64 bits and
rounds each output once.  A product rounds its fp32 sum once to bf16; where
every partial sum is a small whole number it is exact before that rounding,
elsewhere the sum itself is off by at most 2^-12 of the sum of the magnitudes
(the instruction adds 128 products at a time in a format of at least fp32's
fraction: 2^-23 for each of the k additions, k <= 2^11 here).
"""
import numpy as np
import pytest
import torch

import lora_row_adapter_amd as lr
from lora_row_adapter_amd import workloads as wl
import mx_ref as R
from gpu_helpers import DevWorkload, normwise, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
FORMATS = [lr.MX_FP8, lr.MX_FP4]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the gpu tests need an MI355X")
    torch.cuda.set_device(0)
    lr.load_library()
    yield
    torch.cuda.synchronize()


def rand(seed, M, k, dtype, loud=1.2):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, k, generator=g) * torch.exp(loud * torch.randn(k, generator=g))
    return x.to(dtype)


def codes_of(m):
    """One code per element and the scale bytes of a device MX."""
    nb = (m.k + 31) // 32
    return R.unpack(m.q.cpu().numpy(), m.fmt, nb), m.scales.cpu().numpy()[:, :nb]


def to_device(codes, scales, fmt, k, pad_q=0, pad_s=None, fill=0xFF):
    """A device MX of one code per element; wider rows hold `fill` past the end."""
    q = R.pack(codes, fmt)
    M, nb = scales.shape
    pad_s = -nb % 4 if pad_s is None else pad_s
    Q = np.full((M, q.shape[1] + pad_q), fill, np.uint8)
    S = np.full((M, nb + pad_s), fill, np.uint8)
    Q[:, :q.shape[1]], S[:, :nb] = q, scales
    return lr.MX(fmt, torch.from_numpy(Q).cuda(), torch.from_numpy(S).cuda(), k)


def same_bits(a, b):
    a, b = a.contiguous(), b.contiguous()
    t = torch.int16 if a.dtype == BF else torch.int32
    nan = torch.isnan(a) & torch.isnan(b)
    return bool(((a.view(t) == b.view(t)) | nan).all())


# ------------------------------------------------------------ quantise, read back
SIZES = [(1, 1), (1, 32), (3, 31), (2, 33), (5, 100), (64, 128), (7, 1000), (300, 96), (33, 4999), (2, 8192),
         (1, 70001), (513, 40)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,k", SIZES)
def test_quantise_and_read_back_exactly(M, k, dtype, fmt):
    say("quantise %dx%d %s fmt %d" % (M, k, dtype, fmt))
    x = rand(M * 7 + k, M, k, dtype)
    m = lr.lora_mx_quantize(x.cuda(), fmt)
    want_c, want_s = R.quantise(R.f64(x), fmt)
    c, s = codes_of(m)
    assert np.array_equal(s, want_s)
    assert np.array_equal(c, want_c)
    want = torch.from_numpy(R.dequantise(want_c, want_s, fmt, k))
    for t in (F32, BF):
        assert same_bits(lr.lora_mx_dequantize(m, t).cpu(), want.float().to(t))


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantise_every_bf16_value(fmt):
    """Each bf16 pattern, alone in its block and beside the format's ties."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF)
    blk = torch.zeros(65536, 32, dtype=BF)
    blk[:, 7] = x
    blk[32768:, 9] = 1.0
    m = lr.lora_mx_quantize(blk.cuda(), fmt)
    c, s = codes_of(m)
    want_c, want_s = R.quantise(R.f64(blk), fmt)
    assert np.array_equal(s, want_s)
    assert np.array_equal(c, want_c)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantise_special_values(fmt):
    """Zeros of both signs, subnormals, the largest fp32, infinities and NaNs
    (their whole block reads back as NaN, its neighbours do not)."""
    big = torch.finfo(F32).max
    x = torch.randn(6, 160, generator=torch.Generator().manual_seed(3))
    x[0, :32], x[0, 3] = 0.0, -0.0
    x[1, 32:64] = 1e-45
    x[1, 64:96] = torch.randn(32, generator=torch.Generator().manual_seed(4)) * 2.0 ** -126
    x[2, 0], x[3, 40], x[3, 41], x[4, 159] = float("inf"), float("nan"), 1.0, float("-inf")
    x[5, :32], x[5, 1] = big, -big
    m = lr.lora_mx_quantize(x.cuda(), fmt)
    c, s = codes_of(m)
    want_c, want_s = R.quantise(R.f64(x), fmt)
    assert np.array_equal(s, want_s) and np.array_equal(c, want_c)
    y = lr.lora_mx_dequantize(m, F32).cpu()
    assert torch.isnan(y[2, :32]).all() and not torch.isnan(y[2, 32:]).any()
    assert torch.isnan(y[3, 32:64]).all() and not torch.isnan(y[3, :32]).any()
    want = torch.from_numpy(R.dequantise(want_c, want_s, fmt, 160))
    assert same_bits(y, want.float())
    assert same_bits(lr.lora_mx_dequantize(m, BF).cpu(), want.float().to(BF))


@pytest.mark.parametrize("fmt", FORMATS)
def test_read_back_every_code_and_scale(fmt):
    """All codes under all 256 scale bytes: 0 is 2^-127, 255 is NaN, values
    past fp32's range are infinite, bf16 rounds to nearest even."""
    n = 256 if fmt == lr.MX_FP8 else 32
    codes = np.tile((np.arange(n) % (256 if fmt == lr.MX_FP8 else 16)).astype(np.uint8), (256, 1))
    scales = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, n // 32))
    m = to_device(codes, scales, fmt, n)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(R.dequantise(codes, scales, fmt, n)).float()
    assert same_bits(lr.lora_mx_dequantize(m, F32).cpu(), want)
    assert same_bits(lr.lora_mx_dequantize(m, BF).cpu(), want.to(BF))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantise_strided_rows(dtype, fmt):
    """Columns of a wider tensor at an odd offset, rows of codes and scales
    inside wider storage: neighbours keep their bytes."""
    wide = rand(5, 37, 401, dtype).cuda()
    x = wide[:, 3:3 + 197]
    nb = 7
    q = torch.full((37, nb * R.BLOCK_BYTES[fmt] + 32), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((37, 16), 0x5A, dtype=torch.uint8, device="cuda")
    m = lr.MX(fmt, q, s, 197)
    lr.lora_mx_quantize(x, fmt, out=m)
    want_c, want_s = R.quantise(R.f64(x), fmt)
    c, sc = codes_of(m)
    assert np.array_equal(c, want_c) and np.array_equal(sc, want_s)
    assert (q[:, nb * R.BLOCK_BYTES[fmt]:] == 0xA5).all() and (s[:, nb:] == 0x5A).all()
    out = torch.full((37, 300), 7.0, dtype=dtype, device="cuda")
    lr.lora_mx_dequantize(m, dtype, out=out[:, 1:198])
    want = torch.from_numpy(R.dequantise(want_c, want_s, fmt, 197)).float().to(dtype)
    assert same_bits(out[:, 1:198].cpu(), want)
    assert (out[:, 0] == 7).all() and (out[:, 198:] == 7).all()


def test_quantise_past_32_bit_offsets():
    """More than 2^31 bytes of codes: the last rows as if alone."""
    M, k = 270_000, 8192
    x = torch.zeros(M, k, dtype=BF, device="cuda")
    tail = rand(9, 5, k, BF).cuda()
    x[-5:] = tail
    m = lr.lora_mx_quantize(x, lr.MX_FP8)
    alone = lr.lora_mx_quantize(tail, lr.MX_FP8)
    assert torch.equal(m.q[-5:], alone.q) and torch.equal(m.scales[-5:], alone.scales)
    y = lr.lora_mx_dequantize(m, BF, out=x)
    assert torch.equal(y[-5:], lr.lora_mx_dequantize(alone, BF))
    W = lr.lora_mx_quantize(rand(10, 48, k, BF, loud=0).cuda(), lr.MX_FP4)
    assert torch.equal(lr.lora_gemm_mx(m, W)[-5:], lr.lora_gemm_mx(lr.MX(lr.MX_FP8, m.q[-256:], m.scales[-256:], k), W)[-5:])


# ------------------------------------------------------------ norm
NORM_SIZES = [(1, 1), (2, 31), (5, 100), (9, 256), (3, 1000), (17, 2050), (2, 4096), (4, 5003), (1, 8192), (3, 20000),
              (2, 40001)]


def check_norm(x, w, eps, res, h, y, m, fmt):
    with np.errstate(invalid="ignore"):
        H, Y = R.rmsnorm(R.f64(x), R.f64(w), eps, None if res is None else R.f64(res))
    tiny = 2.0 ** -133 if x.dtype == BF else 2.0 ** -149
    for got, want in ((h, H), (y, Y)):
        if got is None:
            continue
        err = np.abs(R.f64(got) - want)
        assert (err <= R.half_step(x.dtype) * np.abs(want) * (1 + 1e-12) + tiny).all()
    if m is not None:
        c, s = codes_of(m)
        want_c, want_s = R.quantise(Y, fmt)
        assert np.array_equal(s, want_s)
        assert np.array_equal(c, want_c)


@pytest.mark.parametrize("fmt", [None] + FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,k", NORM_SIZES)
def test_rmsnorm(M, k, dtype, fmt):
    say("rmsnorm %dx%d %s fmt %s" % (M, k, dtype, fmt))
    x, r = rand(M + k, M, k, dtype).cuda(), rand(M + k + 1, M, k, dtype).cuda()
    w = (1 + 0.3 * torch.randn(k, generator=torch.Generator().manual_seed(k))).to(dtype).cuda()
    for res in (None, r):
        h = None if res is None else torch.empty_like(x)
        m = None if fmt is None else lr.MX.empty(M, k, fmt)
        y = torch.empty_like(x)
        lr.lora_rmsnorm(x, lr.Norm(w, 1e-5, residual=res, residual_out=h), y=y, yq=m)
        check_norm(x, w, 1e-5, res, h, y, m, fmt)
        if m is not None:  # the codes alone are the same
            m2 = lr.MX.empty(M, k, fmt)
            assert lr.lora_rmsnorm(x, lr.Norm(w, 1e-5, residual=res), yq=m2) is None
            assert torch.equal(m.q, m2.q) and torch.equal(m.scales[:, :(k + 31) // 32], m2.scales[:, :(k + 31) // 32])


@pytest.mark.parametrize("k", [96, 40001])
def test_rmsnorm_in_place_and_strided(k):
    """The sum in place of the residual, the normed rows in place of x, every
    tensor a column range of a wider one."""
    M, pad = 6, 5
    def wide(seed):  # noqa: E306
        t = torch.full((M, k + 2 * pad), 3.0, dtype=BF, device="cuda")
        t[:, pad:pad + k] = rand(seed, M, k, BF).cuda()
        return t
    X, Rs = wide(1), wide(2)
    x, r = X[:, pad:pad + k], Rs[:, pad:pad + k]
    x0, r0 = x.clone(), r.clone()
    w = torch.ones(k, dtype=BF, device="cuda")
    out = lr.lora_rmsnorm(x, lr.Norm(w, 1e-6, residual=r, residual_out=r), y=x)
    assert out is x
    check_norm(x0, w, 1e-6, r0, r, x, None, None)
    for t in (X, Rs):
        assert (t[:, :pad] == 3).all() and (t[:, pad + k:] == 3).all()
    # the other way round: the sum in place of x, the normed rows in place of the residual
    x.copy_(x0), r.copy_(r0)
    lr.lora_rmsnorm(x, lr.Norm(w, 1e-6, residual=r, residual_out=x), y=r)
    check_norm(x0, w, 1e-6, r0, x, r, None, None)


def test_rmsnorm_zero_and_non_finite_rows():
    x = rand(4, 5, 192, F32)
    x[0] = 0
    x[1, 5], x[2, 7] = float("inf"), float("nan")
    x[3] = 1e30   # squares past fp32's range
    x[4] = 1e-30
    w = torch.ones(192)
    m = lr.MX.empty(5, 192, lr.MX_FP8)
    y = torch.empty(5, 192, device="cuda")
    lr.lora_rmsnorm(x.cuda(), lr.Norm(w.cuda(), 0.0), y=y, yq=m)
    y = y.cpu()
    assert torch.isnan(y[0]).all()              # 0 / sqrt(0)
    assert torch.isnan(y[1, 5]) and (y[1, :5] == 0).all()
    assert torch.isnan(y[2]).all()
    assert torch.allclose(y[3:], torch.ones(2, 192), rtol=1e-6, atol=0)
    _, s = codes_of(m)
    assert (s[0] == 255).all() and s[1, 0] == 255 and (s[1, 1:] == 0).all() and (s[2] == 255).all()
    y = lr.lora_rmsnorm(x.cuda(), lr.Norm(w.cuda(), 1e-6)).cpu()
    assert (y[0] == 0).all()


def test_rmsnorm_codes_do_not_depend_on_the_batch():
    """A row's outputs alone and in a large batch, and with its values at
    another alignment."""
    k = 5120
    x = rand(8, 700, k, BF).cuda()
    w = torch.ones(k, dtype=BF, device="cuda")
    m = lr.MX.empty(700, k, lr.MX_FP8)
    lr.lora_rmsnorm(x, lr.Norm(w), yq=m)
    one = lr.MX.empty(1, k, lr.MX_FP8)
    wide = torch.zeros(1, k + 1, dtype=BF, device="cuda")
    wide[:, 1:] = x[333]
    lr.lora_rmsnorm(wide[:, 1:], lr.Norm(w), yq=one)
    assert torch.equal(one.q[0], m.q[333]) and torch.equal(one.scales[0], m.scales[333])


# ------------------------------------------------------------ product
def random_mx(seed, rows, k, fmt, **kw):
    x = rand(seed, rows, k, F32, loud=0.5)
    c, s = R.quantise(R.f64(x), fmt)
    return to_device(c, s, fmt, k, **kw), R.dequantise(c, s, fmt, k)


def whole_mx(seed, rows, k, fmt, **kw):
    """Whole numbers up to 4 under scales of 1 or 2: every sum is exact."""
    g = np.random.default_rng(seed)
    vals = R.code_values(fmt)
    ok = np.flatnonzero(np.isfinite(vals) & (vals == np.round(vals)) & (np.abs(vals) <= 4)).astype(np.uint8)
    nb = -(-k // 32)
    c = ok[g.integers(0, ok.size, (rows, nb * 32))]
    c[:, k:] = 0
    s = g.integers(127, 129, (rows, nb)).astype(np.uint8)
    return to_device(c, s, fmt, k, **kw), R.dequantise(c, s, fmt, k)


# M (rows of x), k, d: odd and ragged sizes, one row and one column, lengths
# next to the steps of 128, 256 and 512 elements
PRODUCTS = [(1, 32, 1), (1, 1, 16), (1, 512, 48), (3, 100, 17), (16, 544, 33), (17, 480, 64), (31, 1000, 100),
            (33, 2048, 130), (48, 160, 257), (64, 640, 96), (65, 1056, 65), (100, 2000, 300), (128, 256, 144),
            (200, 384, 520), (256, 512, 288), (300, 896, 700), (513, 288, 1000), (1024, 512, 1024),
            (1500, 128, 2100), (2048, 320, 2304)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,k,d", PRODUCTS)
def test_product_exact_on_whole_numbers(M, k, d, fmt):
    """Exact sums: y is their one rounding to bf16.  Wider rows of codes and
    scales hold 0xFF (NaN) past the end."""
    say("product exact %dx%dx%d fmt %d" % (M, k, d, fmt))
    x, X = whole_mx(M + k, M, k, fmt, pad_q=16)
    W, Wv = whole_mx(d + k + 1, d, k, lr.MX_FP4, pad_q=32)
    y = lr.lora_gemm_mx(x, W)
    assert same_bits(y.cpu(), torch.from_numpy(X @ Wv.T).float().to(BF))


# a size for each tile shape that the ones above do not take
TILES8 = [(5057, 1343, 8), (4317, 653, 8), (64, 3000, 9000), (4113, 1169, 65), (4439, 730, 67), (5617, 1880, 144),
          (130, 757, 5733), (5443, 705, 194), (788, 645, 5030), (1857, 1322, 1677), (1184, 1040, 3402),
          (1604, 635, 3774), (2062, 641, 3904), (2466, 636, 4038), (2343, 633, 4956)]
TILES4 = [(5146, 915, 34), (5001, 686, 33), (5572, 1503, 71), (5560, 694, 66), (423, 770, 5094), (130, 757, 5733),
          (258, 857, 5057), (779, 641, 4812), (521, 638, 3703), (2216, 631, 1801), (1604, 635, 3774),
          (1685, 800, 3564), (2216, 649, 3599), (3076, 670, 3124), (2507, 631, 4844)]


@pytest.mark.parametrize("M,k,d,fmt", [t + (lr.MX_FP8,) for t in TILES8] + [t + (lr.MX_FP4,) for t in TILES4])
def test_product_exact_on_every_tile_shape(M, k, d, fmt):
    test_product_exact_on_whole_numbers(M, k, d, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,k,d", PRODUCTS)
def test_product(M, k, d, fmt):
    say("product %dx%dx%d fmt %d" % (M, k, d, fmt))
    x, X = random_mx(M + k, M, k, fmt)
    W, Wv = random_mx(d + k + 1, d, k, lr.MX_FP4)
    y = R.f64(lr.lora_gemm_mx(x, W))
    want, mag = X @ Wv.T, np.abs(X) @ np.abs(Wv).T
    assert (np.abs(y - want) <= R.half_step(BF) * np.abs(want) + 2.0 ** -12 * mag).all()
    assert np.linalg.norm(y - want) <= R.half_step(BF) * np.linalg.norm(want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_product_into_a_wider_tensor(fmt):
    x, X = whole_mx(1, 70, 96, fmt)
    W, Wv = whole_mx(2, 45, 96, lr.MX_FP4)
    for off, width in ((0, 45), (1, 64), (3, 51), (8, 64)):
        out = torch.full((70, width + 8), 9.0, dtype=BF, device="cuda")
        lr.lora_gemm_mx(x, W, y=out[:, off:off + 45])
        assert same_bits(out[:, off:off + 45].cpu(), torch.from_numpy(X @ Wv.T).float().to(BF))
        assert (out[:, :off] == 9).all() and (out[:, off + 45:] == 9).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,k,d", [(5, 96, 70), (40, 1056, 130), (300, 2080, 260)])
def test_product_of_strided_operands_that_end_with_their_storage(M, k, d, fmt):
    """Rows far apart, the last one's codes and scales the last bytes there
    are; between the rows codes and scales that mean NaN."""
    def far_apart(m):
        nb = (k + 31) // 32
        width, read = m.q.shape[1], (nb + 3) // 4 * 4
        out = []
        for t, used, pad in ((m.q, width, 48), (m.scales, read, 36)):
            wide = torch.full(((m.rows - 1) * (used + pad) + used,), 0xFF, dtype=torch.uint8, device="cuda")
            v = wide.as_strided((m.rows, used), (used + pad, 1))
            v[:, :t.shape[1]] = t
            v[:, nb if t is m.scales else used:] = 0xFF
            out.append(v)
        return lr.MX(m.fmt, out[0], out[1], k)
    x, _ = random_mx(M, M, k, fmt)
    W, _ = random_mx(d, d, k, lr.MX_FP4)
    assert torch.equal(lr.lora_gemm_mx(far_apart(x), far_apart(W)), lr.lora_gemm_mx(x, W))


@pytest.mark.parametrize("M", [1, 20, 70, 300])
def test_product_keeps_nan_blocks_to_their_rows(M):
    """A NaN block of x makes its row NaN, one of W its column; nothing else."""
    g = np.random.default_rng(M)
    for fmt in FORMATS:
        c, s = R.quantise(g.standard_normal((M, 200)), fmt)
        s[M // 2, 3] = 255
        cw, sw = R.quantise(g.standard_normal((90, 200)), lr.MX_FP4)
        sw[41, 6] = 255
        y = lr.lora_gemm_mx(to_device(c, s, fmt, 200), to_device(cw, sw, lr.MX_FP4, 200)).cpu()
        want = torch.zeros(M, 90, dtype=torch.bool)
        want[M // 2] = True
        want[:, 41] = True
        assert torch.equal(torch.isnan(y), want)


def test_product_rows_do_not_depend_on_their_neighbours():
    """The same inputs twice are the same bits; rows of a batch of one tile
    shape keep their bits when the other rows change."""
    x, _ = random_mx(1, 130, 700, lr.MX_FP8)
    W, _ = random_mx(2, 200, 700, lr.MX_FP4)
    a = lr.lora_gemm_mx(x, W)
    assert torch.equal(a, lr.lora_gemm_mx(x, W))
    x.q[1:] = 0
    assert torch.equal(a[0], lr.lora_gemm_mx(x, W)[0])


# ------------------------------------------------------------ layer
def layer_inputs(w, names=("out",), W_seed=5):
    dev = torch.device("cuda")
    slices, ranks = [], torch.from_numpy(w.ranks).to(dev)
    for n in names:
        p = w.proj(n)
        A, Bm = wl.slots(w, p, pad_value=float("nan"))
        slices.append(lr.Slice(p.d, lr.Adapters.slots(A.to(dev), Bm.to(dev), ranks),
                               torch.from_numpy(w.scales).to(dev)))
    Wd = torch.cat([w.proj(n).W for n in names])
    c, s = R.quantise(R.f64(Wd), R.FP4)
    return slices, to_device(c, s, R.FP4, w.k), R.dequantise(c, s, R.FP4, w.k)


def oracle_layer(oracle_mod, w, names, X, XQ, Wv):
    """Per slice: the layer over the quantised base plus the adapters on X."""
    outs, d0 = [], 0
    for n in names:
        p = w.proj(n)
        zero = np.zeros((p.d, w.k))
        delta = oracle_mod.lora_linear(X, zero, p.A, p.B, w.scales.astype(np.float64), w.ids, max_rank=w.max_rank)
        outs.append(XQ @ Wv[d0:d0 + p.d].T + delta)
        d0 += p.d
    return np.concatenate(outs, 1)


# Each of the layer's four roundings to bf16 (the normed rows, t, the base
# term, y) is off by at most 2^-8 of a term that is at most about the largest
# |y|: 4 x 2^-8 < 2e-2 normwise, the bound of every bf16 output of the layer.
TOL = 2e-2


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("with_norm", [False, True])
@pytest.mark.parametrize("M,k,d", [(1, 256, 96), (37, 264, 200), (300, 1024, 288), (530, 512, 1000)])
def test_layer(oracle_mod, M, k, d, with_norm, fmt):
    say("layer %dx%dx%d norm %s fmt %d" % (M, k, d, with_norm, fmt))
    w = wl.custom(seed=M, M=M, k=k, d=d, ranks=[4, 16, 64, 8], max_rank=64, none_frac=0.2)
    slices, W, Wv = layer_inputs(w)
    x, ids = w.x.cuda(), torch.from_numpy(w.ids).cuda()
    X, norm, h = R.f64(w.x), None, None
    if with_norm:
        res = rand(3, M, k, BF)
        g = (1 + 0.2 * torch.randn(k, generator=torch.Generator().manual_seed(1))).to(BF)
        h = torch.empty_like(x)
        norm = lr.Norm(g.cuda(), 1e-5, residual=res.cuda(), residual_out=h)
        H, X = R.rmsnorm(X, R.f64(g), 1e-5, R.f64(res))
    want = oracle_layer(oracle_mod, w, ["out"], torch.from_numpy(X).float(), R.quantised_values(X, fmt), Wv)
    none = torch.from_numpy(np.flatnonzero(w.ids < 0)).cuda()
    if norm is None:
        q = lr.lora_mx_quantize(x, fmt)
    else:
        q = lr.MX.empty(M, k, fmt)
        lr.lora_rmsnorm(x, norm, yq=q)
    base = lr.lora_gemm_mx(q, W)
    for path in (lr.PATH_AUTO, lr.PATH_GATHER, lr.PATH_SGMV):
        if h is not None:
            h.zero_()
        y = lr.lora_linear_sliced_mx(x, W, slices, ids, x_format=fmt, norm=norm, path=path)
        err = normwise(R.f64(y), want)
        say("  path %d: normwise error %.3g" % (path, err))
        assert err <= TOL
        assert torch.equal(y[none], base[none])
        if h is not None:
            assert (np.abs(R.f64(h) - H) <= R.half_step(BF) * np.abs(H) * (1 + 1e-12)).all()


def test_layer_two_slices_reused_plan_and_workspace_report(oracle_mod):
    w = wl._build("two", 77, BF, 200, 512, {"q": 320, "v": 96}, [4, 16, 64], [8.0, 32.0, 128.0], 64,
                  wl._uniform_ids(200, 3))
    slices, W, Wv = layer_inputs(w, ("q", "v"))
    x = w.x.cuda()
    ids = w.ids.copy()
    ids[[3, 50]] = (99, -7)  # counted, served without an adapter
    ids_d = torch.from_numpy(ids).cuda()
    w.ids = np.where((ids < 0) | (ids > 2), -1, ids).astype(np.int32)
    n = lr.workspace_bytes_sliced_mx(200, 512, lr.MX_FP8, slices)
    guard = torch.zeros(n + 4096, dtype=torch.uint8, device="cuda")
    guard[n:] = 0xC3
    ws = guard[:n]
    X = R.f64(w.x)
    want = oracle_layer(oracle_mod, w, ["q", "v"], w.x, R.quantised_values(X, R.FP8), Wv)
    y = lr.lora_linear_sliced_mx(x, W, slices, ids_d, workspace=ws)
    assert normwise(R.f64(y), want) <= TOL
    assert lr.lora_check(ws)["n_bad_ids"] == 2
    again = lr.lora_linear_sliced_mx(x, W, slices, ids_d, workspace=ws, flags=lr.FLAG_REUSE_PLAN)
    assert torch.equal(y, again)
    assert (guard[n:] == 0xC3).all()


def test_layer_past_the_plan_rows():
    """More rows than one plan holds: as the two halves alone."""
    w = wl.custom(seed=9, M=8200, k=64, d=48, ranks=[8, 16], max_rank=16, none_frac=0.3)
    slices, W, _ = layer_inputs(w)
    x, ids = w.x.cuda(), torch.from_numpy(w.ids).cuda()
    res = rand(1, 8200, 64, BF).cuda()
    g = torch.ones(64, dtype=BF, device="cuda")
    h = torch.empty_like(x)
    y = lr.lora_linear_sliced_mx(x, W, slices, ids, norm=lr.Norm(g, 1e-5, res, h))
    for a, b in ((0, 8192), (8192, 8200)):
        h2 = torch.empty_like(x[a:b])
        part = lr.lora_linear_sliced_mx(x[a:b], W, slices, ids[a:b].contiguous(),
                                        norm=lr.Norm(g, 1e-5, res[a:b], h2))
        assert torch.equal(h[a:b], h2)
        assert normwise(R.f64(y[a:b]), R.f64(part)) <= 2.0 ** -7  # another tile shape sums in another order


def test_layer_all_rows_without_adapter_and_in_place_residual():
    w = wl.custom(seed=4, M=50, k=128, d=64, ranks=[8], max_rank=8)
    slices, W, _ = layer_inputs(w)
    x = w.x.cuda()
    ids = torch.full((50,), -1, dtype=torch.int32, device="cuda")
    res = rand(1, 50, 128, BF).cuda()
    r0 = res.clone()
    g = torch.ones(128, dtype=BF, device="cuda")
    y = lr.lora_linear_sliced_mx(x, W, slices, ids, norm=lr.Norm(g, 1e-5, res, res), x_format=lr.MX_FP4)
    h = torch.empty_like(x)
    q = lr.MX.empty(50, 128, lr.MX_FP4)
    lr.lora_rmsnorm(x, lr.Norm(g, 1e-5, r0, h), yq=q)
    assert torch.equal(h, res) and torch.equal(y, lr.lora_gemm_mx(q, W))


# ------------------------------------------------------------ streams, graphs
def chain(x, r, w, W, m, h, stream=None):
    lr.lora_rmsnorm(x, lr.Norm(w, 1e-5, r, h), yq=m, stream=stream)
    return lr.lora_gemm_mx(m, W, stream=stream)


def test_chain_on_another_stream_and_captured():
    """Norm, then product, as a server runs them: on a side stream, and as two
    captured graphs replayed in turn with new inputs, against eager calls."""
    M, k, d = 40, 1024, 520
    w = torch.ones(k, dtype=BF, device="cuda")
    W, _ = random_mx(3, d, k, lr.MX_FP4)
    bufs = []
    for i in range(2):
        bufs.append((rand(i, M, k, BF).cuda(), rand(i + 9, M, k, BF).cuda(), lr.MX.empty(M, k, lr.MX_FP8),
                     torch.empty(M, k, dtype=BF, device="cuda")))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y_side = chain(bufs[0][0], bufs[0][1], w, W, bufs[0][2], bufs[0][3])
    side.synchronize()
    eager = [chain(x, r, w, W, m, h) for x, r, m, h in bufs]
    assert torch.equal(y_side, eager[0])
    graphs, outs = [], []
    for x, r, m, h in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(chain(x, r, w, W, m, h))
        graphs.append(g)
    for rep in range(4):
        for i in (0, 1):
            bufs[i][0].copy_(rand(100 + 2 * rep + i, M, k, BF))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for i in (0, 1):
            x, r, m, h = bufs[i]
            m2, h2 = lr.MX.empty(M, k, lr.MX_FP8), torch.empty_like(h)
            assert torch.equal(got[i], chain(x, r, w, W, m2, h2))


def test_layer_captured():
    w = wl.custom(seed=12, M=64, k=512, d=320, ranks=[8, 32], max_rank=32, none_frac=0.2)
    slices, W, _ = layer_inputs(w)
    x, ids = w.x.cuda(), torch.from_numpy(w.ids).cuda()
    ws = torch.zeros(lr.workspace_bytes_sliced_mx(64, 512, lr.MX_FP8, slices), dtype=torch.uint8, device="cuda")
    g = torch.ones(512, dtype=BF, device="cuda")
    r, h = rand(2, 64, 512, BF).cuda(), torch.empty_like(x)
    norm = lr.Norm(g, 1e-5, r, h)
    y = torch.empty(64, 320, dtype=BF, device="cuda")
    lr.lora_linear_sliced_mx(x, W, slices, ids, norm=norm, y=y, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lr.lora_linear_sliced_mx(x, W, slices, ids, norm=norm, y=y, workspace=ws)
    for rep in range(3):
        x.copy_(rand(50 + rep, 64, 512, BF))
        ids.copy_(torch.randint(-1, 2, (64,), dtype=torch.int32))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got, got_h = y.clone(), h.clone()
        want = lr.lora_linear_sliced_mx(x, W, slices, ids, norm=norm)
        assert torch.equal(got, want) and torch.equal(got_h, h)


# ------------------------------------------------------------ the plan beside the norm or the quantising
def more_slots(slices, S):
    """The same adapters with unused ones behind them, S in all."""
    out = []
    for sl in slices:
        ad = sl.adapters
        n = S - ad.n_adapters
        A = torch.cat([ad.A, torch.zeros((n,) + ad.A.shape[1:], dtype=BF, device="cuda")])
        B = torch.cat([ad.B, torch.zeros((n,) + ad.B.shape[1:], dtype=BF, device="cuda")])
        ranks = torch.cat([ad.ranks, torch.zeros(n, dtype=ad.ranks.dtype, device="cuda")])
        out.append(lr.Slice(sl.d, lr.Adapters.slots(A, B, ranks), torch.cat([sl.scales, sl.scales.new_ones(n)])))
    return out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("with_norm", [False, True])
@pytest.mark.parametrize("M,k", [(1, 32), (3, 256), (257, 8000), (1024, 64), (1025, 64), (4100, 2048), (70, 16384),
                                 (70, 16392)])
def test_layer_plan_beside_equals_a_plan_of_its_own(M, k, with_norm, fmt):
    """Up to 64 adapters the plan is made beside the first launch: it equals
    the one that lora_plan makes, and so do the layer's bits on that one."""
    say("layer plan %dx%d norm %s fmt %d" % (M, k, with_norm, fmt))
    w = wl.custom(seed=M + k, M=M, k=k, d=80, ranks=[4, 16, 64, 8], max_rank=64, none_frac=0.2)
    slices, W, _ = layer_inputs(w)
    x = w.x.cuda()
    ids = w.ids.copy()
    ids[0] = -5                      # counted, served without an adapter
    ids = torch.from_numpy(ids).cuda()
    norm = lr.Norm(rand(1, 1, k, BF)[0].cuda(), 1e-5, rand(2, M, k, BF).cuda()) if with_norm else None
    for sl in (slices, more_slots(slices, 64), more_slots(slices, 65)):
        n = lr.workspace_bytes_sliced_mx(M, k, fmt, sl)
        ws, ws2 = (torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda") for _ in range(2))
        y = lr.lora_linear_sliced_mx(x, W, sl, ids, x_format=fmt, norm=norm, workspace=ws)
        report = lr.lora_check(ws)  # n_sync_expired belongs to zero-filled workspaces alone
        assert (report["n_bad_ids"], report["n_bad_ranks"], report["n_bad_pages"]) == (1, 0, 0)
        assert not torch.isnan(y).any()
        lr.lora_plan(ids, sl[0].adapters, k, 80, BF, ws2)
        for other in (ws, ws2):
            again = lr.lora_linear_sliced_mx(x, W, sl, ids, x_format=fmt, norm=norm, workspace=other,
                                             flags=lr.FLAG_REUSE_PLAN)
            assert torch.equal(y, again)
        one, two = (lr.lora_plan_view(t, M, sl[0].adapters) for t in (ws, ws2))
        assert one.keys() == two.keys()
        for name in one:
            assert np.array_equal(one[name], two[name]), name


@pytest.mark.parametrize("with_norm", [False, True])
def test_layer_paged_adapters(with_norm):
    """Adapters in a paged pool give the bits of the same adapters in slots."""
    w = wl.custom(seed=21, M=90, k=512, d=320, ranks=[4, 16, 64, 8], max_rank=64, none_frac=0.2)
    slices, W, _ = layer_inputs(w)
    dev = DevWorkload(w, w.proj("out"), pooled=True)
    paged = [lr.Slice(320, dev.ad, slices[0].scales)]
    x, ids = w.x.cuda(), torch.from_numpy(w.ids).cuda()
    norm = lr.Norm(torch.ones(512, dtype=BF, device="cuda"), 1e-5) if with_norm else None
    ws = torch.empty(lr.workspace_bytes_sliced_mx(90, 512, lr.MX_FP8, paged), dtype=torch.uint8, device="cuda")
    y = lr.lora_linear_sliced_mx(x, W, paged, ids, norm=norm, workspace=ws)
    assert lr.lora_check(ws)["n_bad_pages"] == 0
    assert torch.equal(y, lr.lora_linear_sliced_mx(x, W, slices, ids, norm=norm))


def test_layers_on_two_streams_at_once():
    """Two layers in flight together, a workspace each, against one after the
    other; a captured one replayed beside an eager one."""
    w = wl.custom(seed=31, M=200, k=1024, d=640, ranks=[8, 32, 64], max_rank=64, none_frac=0.1)
    slices, W, _ = layer_inputs(w)
    ids = torch.from_numpy(w.ids).cuda()
    n = lr.workspace_bytes_sliced_mx(200, 1024, lr.MX_FP8, slices)
    g = torch.ones(1024, dtype=BF, device="cuda")
    sets = [(rand(i, 200, 1024, BF).cuda(), lr.Norm(g, 1e-5, rand(i + 5, 200, 1024, BF).cuda()),
             torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty(200, 640, dtype=BF, device="cuda"))
            for i in range(2)]

    def call(i):
        x, norm, ws, y = sets[i]
        return lr.lora_linear_sliced_mx(x, W, slices, ids, norm=norm, workspace=ws, y=y)

    want = [call(i).clone() for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for rep in range(3):
        for i in (0, 1):
            sets[i][3].zero_()
        torch.cuda.synchronize()
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                call(i)
        torch.cuda.synchronize()
        for i in (0, 1):
            assert torch.equal(sets[i][3], want[i])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0)
    for rep in range(3):
        for i in (0, 1):
            sets[i][3].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            graph.replay()
        with torch.cuda.stream(streams[1]):
            call(1)
        torch.cuda.synchronize()
        for i in (0, 1):
            assert torch.equal(sets[i][3], want[i])


def test_empty_batches():
    """No rows: nothing is read, written or launched."""
    w = wl.custom(seed=5, M=4, k=64, d=48, ranks=[8, 16], max_rank=16)
    slices, W, _ = layer_inputs(w)
    x, ids = w.x.cuda()[:0], torch.empty(0, dtype=torch.int32, device="cuda")
    g = torch.ones(64, dtype=BF, device="cuda")
    h = torch.empty_like(x)
    m = lr.MX.empty(0, 64, lr.MX_FP8)
    assert lr.lora_rmsnorm(x, lr.Norm(g, 1e-5, x, h), yq=m) is None
    assert lr.lora_mx_dequantize(m).shape == (0, 64)
    for norm in (None, lr.Norm(g, 1e-5, x, h)):
        ws = torch.full((lr.workspace_bytes_sliced_mx(4, 64, lr.MX_FP8, slices),), 7, dtype=torch.uint8, device="cuda")
        assert lr.lora_linear_sliced_mx(x, W, slices, ids, norm=norm, workspace=ws).shape == (0, 48)
        assert (ws == 7).all()


# ------------------------------------------------------------ norm: roundings at their edges
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rmsnorm_values_on_midpoints(dtype, fmt):
    """Rows of +-1 with eps = 0 leave the weights themselves: midpoints and
    neighbours of codes (and of bf16 values, in the sum), at every scale."""
    k = 512
    g = torch.Generator().manual_seed(3)
    sign = torch.randint(0, 2, (40, k), generator=g) * 2 - 1
    x = (sign * torch.exp2(torch.arange(40) - 20.0)[:, None]).to(dtype)
    codes = R.code_values(fmt)[:127 if fmt == R.FP8 else 8]
    mid = torch.from_numpy(np.concatenate([codes, (codes[:-1] + codes[1:]) / 2, codes * (1 + 2.0 ** -7)])).float()
    w = mid[torch.randint(0, len(mid), (k,), generator=g)]
    w = (w * torch.exp2(torch.arange(k) // 32 - 8.0)).to(dtype)
    m = lr.MX.empty(40, k, fmt)
    y = torch.empty(40, k, dtype=dtype, device="cuda")
    lr.lora_rmsnorm(x.cuda(), lr.Norm(w.cuda(), 0.0), y=y, yq=m)
    assert torch.equal(y.cpu(), (sign * w.float()).to(dtype))
    check_norm(x, w, 0.0, None, None, y, m, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size,weight", [(1e37, 1.0), (1e-38, 1.0), (1e-33, 1e33), (1e30, 1e-36), (1.0, 1e-38),
                                         (1e-39, 1e-20)])
def test_rmsnorm_far_from_one(size, weight, dtype, fmt):
    """Magnitudes whose norm's factor, or whose product with it or with the
    weight, leaves fp32's normal range on the way."""
    M, k = 6, 200
    x = (rand(5, M, k, F32, loud=0.3) * size).to(dtype)
    r = (rand(6, M, k, F32, loud=0.3) * (size * 0.3)).to(dtype)
    w = (rand(7, 1, k, F32, loud=0.3)[0] * weight).to(dtype)
    h, y, m = torch.empty(M, k, dtype=dtype, device="cuda"), torch.empty(M, k, dtype=dtype, device="cuda"), \
        lr.MX.empty(M, k, fmt)
    lr.lora_rmsnorm(x.cuda(), lr.Norm(w.cuda(), 0.0, r.cuda(), h), y=y, yq=m)
    check_norm(x, w, 0.0, r, h, y, m, fmt)


def test_rmsnorm_sum_of_far_exponents():
    """x + residual at every distance of exponents: the sum is bf16's rounding
    of the exact one."""
    e = torch.arange(-40, 41, dtype=torch.float64)
    a = torch.arange(128, 256, dtype=torch.float64) / 128
    x = (a[:, None] * torch.ones(81, dtype=torch.float64)).to(BF)
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        b = a[torch.randint(0, 128, (128, 81), generator=g)] * (torch.randint(0, 2, (128, 81), generator=g) * 2 - 1)
        r = (b * torch.exp2(e)).to(BF)
        h = torch.empty(128, 81, dtype=BF, device="cuda")
        lr.lora_rmsnorm(x.cuda(), lr.Norm(torch.ones(81, dtype=BF, device="cuda"), 1e-5, r.cuda(), h))
        # 8 bits each, 40 places apart at most: exact in 64 bits
        want = torch.from_numpy(R.f64(x) + R.f64(r))
        err = (torch.from_numpy(R.f64(h)) - want).abs()
        up = torch.nextafter(h.cpu(), torch.full_like(h.cpu(), float("inf"))).double()
        dn = torch.nextafter(h.cpu(), torch.full_like(h.cpu(), float("-inf"))).double()
        assert ((err <= (up - want).abs()) & (err <= (dn - want).abs())).all()


# ------------------------------------------------------------ refusals of the binding
def test_binding_refuses_device_tensors_that_do_not_fit():
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    x = rand(1, 4, 64, BF).cuda()
    q = lr.lora_mx_quantize(x)
    for bad in (lambda: lr.MX(lr.MX_FP8, u(4, 32), u(4, 4), 64),            # too few codes
                lambda: lr.MX(lr.MX_FP8, u(4, 64), u(3, 4), 64),            # rows differ
                lambda: lr.MX(lr.MX_FP8, u(4, 64), u(4, 1), 64),            # too few scales
                lambda: lr.MX(lr.MX_FP8, u(4, 64), u(4 * 4 - 1)[:14].as_strided((4, 2), (4, 1)), 64),
                lambda: lr.MX(lr.MX_FP8, u(64, 4).t(), u(4, 4), 64),        # no unit stride
                lambda: lr.MX(lr.MX_FP8, u(4, 64), u(4, 4).cpu(), 64),
                lambda: lr.MX(lr.MX_FP8, u(256), u(4, 4), 64),
                lambda: lr.lora_mx_quantize(x.t()),
                lambda: lr.lora_mx_quantize(x[0]),
                lambda: lr.lora_mx_quantize(x, lr.MX_FP4, out=q),           # another format
                lambda: lr.lora_mx_quantize(x[:3], lr.MX_FP8, out=q),       # another size
                lambda: lr.lora_mx_dequantize(q, out=torch.empty(4, 65, dtype=BF, device="cuda")),
                lambda: lr.lora_mx_dequantize(q, out=torch.empty(4, 64, dtype=BF)),
                lambda: lr.lora_rmsnorm(x, lr.Norm(torch.ones(63, dtype=BF, device="cuda"))),
                lambda: lr.lora_rmsnorm(x, lr.Norm(torch.ones(64, dtype=BF))),
                lambda: lr.lora_rmsnorm(x, lr.Norm(torch.ones(64, dtype=BF, device="cuda"), 1e-5, x[:3])),
                lambda: lr.lora_gemm_mx(q, lr.MX.empty(8, 96, lr.MX_FP4))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lr.lora_mx_quantize(x.half()), lambda: lr.lora_mx_dequantize(q, torch.float16),
                lambda: lr.lora_mx_dequantize(q, F32, out=torch.empty(4, 64, dtype=BF, device="cuda")),
                lambda: lr.lora_rmsnorm(x, lr.Norm(torch.ones(64, device="cuda"))),
                lambda: lr.MX(lr.MX_FP8, u(4, 64).char(), u(4, 4), 64)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: lr.MX(lr.MX_FP8, u(4 * 64 + 8)[8:].view(4, 64), u(4, 4), 64),  # misaligned codes
                lambda: lr.MX(lr.MX_FP8, u(4, 72), u(4, 4), 64)):                      # rows of 72 bytes
        with pytest.raises(lr.LoraError):
            lr.lora_mx_quantize(x, out=bad())
    with pytest.raises(lr.LoraError):  # the weight must be fp4
        lr.lora_gemm_mx(q, q)
    with pytest.raises(lr.LoraError):  # the sum and the normed rows in one place
        lr.lora_rmsnorm(x, lr.Norm(torch.ones(64, dtype=BF, device="cuda"), 1e-5, x, x), y=x)
    assert lr.lora_mx_quantize(x[:0]).rows == 0
    assert lr.lora_gemm_mx(lr.lora_mx_quantize(x[:0]), lr.lora_mx_quantize(x, lr.MX_FP4)).shape == (0, 4)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("k", [1023, 1024, 40001])
def test_rmsnorm_values_past_fp32(k, dtype, fmt):
    """A row with one element other than 0 leaves sqrt(k) times its weight:
    values next to and past fp32's largest.  What rounds to an infinity there
    is one for the codes as for y, and its neighbours keep theirs."""
    M = 9
    at = np.arange(M) * 40 % k                     # one block or two apart
    x = torch.zeros(M, k, dtype=dtype)
    w = torch.ones(k, dtype=dtype)
    root = 2.0 ** np.floor(np.log2(np.sqrt(k)))
    for m in range(M):
        x[m, at[m]] = -3.0 if m % 2 else 3.0
        # (for k = 1024, row 3: the largest bf16; row 6: 2^128)
        w[at[m]] = [2.0 ** 120, 2.0 ** 127, 2.0 ** 127 * (1 + 126 / 128), 2.0 ** 127 * (1 + 127 / 128), 2.0 ** 126,
                    2.0 ** 124 * 1.5, 2.0 ** 128, 2.0 ** 129, 2.0 ** 130][m] / root
    y, m = torch.empty(M, k, dtype=dtype, device="cuda"), lr.MX.empty(M, k, fmt)
    lr.lora_rmsnorm(x.cuda(), lr.Norm(w.cuda(), 0.0), y=y, yq=m)
    _, Y = R.rmsnorm(R.f64(x), R.f64(w), 0.0)
    edge = 2.0 ** 128 - 2.0 ** 103                 # halfway from the largest fp32 to 2^128
    assert (np.abs(Y).max(1) >= edge).any() and (np.abs(np.abs(Y) / edge - 1) > 1e-12).all()
    c, s = codes_of(m)
    want_c, want_s = R.quantise(np.where(np.abs(Y) < edge, Y, np.copysign(np.inf, Y)), fmt)
    assert np.array_equal(s, want_s) and np.array_equal(c, want_c)
    half = 2.0 ** 128 - (2.0 ** 119 if dtype is BF else 2.0 ** 103)
    assert np.array_equal(np.isinf(R.f64(y)), np.abs(Y) >= half)
    m2 = lr.MX.empty(M, k, fmt)                    # and with a residual
    lr.lora_rmsnorm(x.cuda(), lr.Norm(w.cuda(), 0.0, torch.zeros_like(x).cuda()), yq=m2)
    c2, s2 = codes_of(m2)
    assert np.array_equal(s2, want_s) and np.array_equal(c2, want_c)


def test_profiler_times_the_product_and_the_layer():
    """One launch of the base product's class each; the row operators called by
    themselves have no class."""
    w = wl.custom(seed=6, M=20, k=256, d=96, ranks=[8], max_rank=8)
    slices, W, _ = layer_inputs(w)
    x, ids = w.x.cuda(), torch.from_numpy(w.ids).cuda()
    with lr.Profiler():
        m = lr.lora_mx_quantize(x)
        lr.lora_rmsnorm(x, lr.Norm(torch.ones(256, dtype=BF, device="cuda")), yq=m)
        lr.lora_mx_dequantize(m)
        assert all(lr.Profiler.read()[c]["launches"] == 0 for c in lr.KERNEL_CLASSES)
        lr.lora_gemm_mx(m, W)
        one = lr.Profiler.read()
        lr.lora_linear_sliced_mx(x, W, slices, ids)
        two = lr.Profiler.read(reset=True)
    assert one["gemm"]["launches"] == 1 and one["gemm"]["ms"] > 0
    assert two["gemm"]["launches"] == 2 and two["sgmv_shrink"]["launches"] == 1 == two["sgmv_expand"]["launches"]


@pytest.mark.parametrize("M,k,d,fmt", [t + (f,) for f in FORMATS for t in R.LONG[f]])
def test_product_exact_past_the_rings_of_every_tile_shape(M, k, d, fmt):
    """k long enough that every LDS stage and scale slot is read, freed and
    filled again (sums up to 64 k < 2^24: exact)."""
    assert lr.test_gemm_mx_shape(M, k, d, fmt)[0] == R.LONG[fmt].index((M, k, d))
    test_product_exact_on_whole_numbers(M, k, d, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("with_norm", [False, True])
@pytest.mark.parametrize("M,k,d,scale", [(1, 256, 96, 1.0), (37, 264, 200, 1.0), (300, 1024, 288, 0.03),
                                         (530, 512, 1000, 30.0), (700, 2048, 264, 1.0)])
def test_layer_roundings(M, k, d, scale, with_norm, fmt):
    """Every element within its two roundings: h = 2^-8 of the base term (in
    bf16 on its way through y) and h of the sum, with the sums' own error E on
    top.  E: fp32 sums over k <= 2^11 of the base and of x A^T (2^-23 an
    addition, 2^-12 of the magnitudes' sum), the two bf16 parts of x A^T (2^-16)
    and the sum over the rank (64 x 2^-23): 2^-11 of the magnitudes' sums at
    most.  Rows without an adapter are rounded once."""
    w = wl.custom(seed=M + 1, M=M, k=k, d=d, ranks=[4, 16, 64, 8], max_rank=64, none_frac=0.2)
    w.scales = (w.scales * scale).astype(np.float32)
    slices, W, Wv = layer_inputs(w)
    x, ids = w.x.cuda(), torch.from_numpy(w.ids).cuda()
    norm, X, xn = None, R.f64(w.x), R.f64(w.x)
    if with_norm:
        g = (1 + 0.2 * torch.randn(k, generator=torch.Generator().manual_seed(1))).to(BF)
        norm = lr.Norm(g.cuda(), 1e-5)
        X = R.rmsnorm(X, R.f64(g), 1e-5)[1]
        xn = R.f64(lr.lora_rmsnorm(x, norm))  # its own test compares it with X
    XQ, p = R.quantised_values(X, fmt), w.proj("out")
    base, mag = XQ @ Wv.T, np.abs(XQ) @ np.abs(Wv).T
    delta, dmag = np.zeros((M, d)), np.zeros((M, d))
    for s in range(w.S):
        m, A, Bm, sc = w.ids == s, R.f64(p.A[s]), R.f64(p.B[s]), float(w.scales[s])
        delta[m] = sc * (xn[m] @ A.T @ Bm.T)
        dmag[m] = abs(sc) * (np.abs(xn[m]) @ np.abs(A).T @ np.abs(Bm).T)
    h, want, E = R.half_step(BF), base + delta, 2.0 ** -12 * mag + 2.0 ** -11 * dmag
    once = h * (np.abs(base) + E)
    limit = np.where((w.ids >= 0)[:, None], once + h * (np.abs(want) + E + once), once) + E
    for path in (lr.PATH_AUTO, lr.PATH_GATHER, lr.PATH_SGMV):
        err = np.abs(R.f64(lr.lora_linear_sliced_mx(x, W, slices, ids, x_format=fmt, norm=norm, path=path)) - want)
        say("layer %dx%dx%d norm %s fmt %d path %d: %.3f of the limit" % (M, k, d, with_norm, fmt, path,
                                                                         (err / limit).max()))
        assert (err <= limit).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,k,d", [(3, 256, 40), (300, 2080, 520)])
def test_product_at_far_scales(M, k, d, fmt):
    """Scales at both ends whose products are ordinary, subnormal or nothing,
    and the largest two over zero codes: whole numbers times one power of two,
    so exact but for the last rounding."""
    g = np.random.default_rng(k)
    vals = R.code_values(fmt)
    cx = np.flatnonzero(np.isfinite(vals) & (np.abs(vals) <= 4) & (vals == np.round(vals))).astype(np.uint8)
    cw = np.array([2, 4, 5, 6, 10, 12, 13, 14], np.uint8)  # 1, 2, 3, 4 and their negatives
    nb = -(-k // 32)
    for sx, sw in ((254, 0), (0, 254), (127, 0), (0, 127), (60, 60), (100, 20), (40, 70), (0, 0), (254, 254)):
        x, w = cx[g.integers(0, cx.size, (M, nb * 32))], cw[g.integers(0, cw.size, (d, nb * 32))]
        SX, SW = np.full((M, nb), sx, np.uint8), np.full((d, nb), sw, np.uint8)
        if sx + sw == 508:  # only the first block counts
            x[:, 32:], SX[:, 0], SW[:, 0] = 0, 127, 127
        y = lr.lora_gemm_mx(to_device(x, SX, fmt, k), to_device(w, SW, R.FP4, k)).cpu()
        want = R.dequantise(x, SX, fmt, k) @ R.dequantise(w, SW, R.FP4, k).T
        assert torch.equal(y, torch.from_numpy(want).float().to(BF)), (sx, sw)


# ------------------------------------------------------------ calls that the documents allow
@pytest.mark.parametrize("fmt", FORMATS)
def test_product_of_more_columns_than_a_slab(fmt):
    """More than 2^18 rows of W: launches of their own for those past them."""
    d = (1 << 18) + 700
    x, X = whole_mx(1, 3, 96, fmt)
    W, Wv = whole_mx(2, d, 96, lr.MX_FP4)
    assert same_bits(lr.lora_gemm_mx(x, W).cpu(), torch.from_numpy(X @ Wv.T).float().to(BF))


def rows_in_wide(t, before, after, fill=5.0):
    """The same rows as columns of a wider tensor."""
    wide = torch.full((t.shape[0], before + t.shape[1] + after), fill, dtype=t.dtype, device="cuda")
    v = wide[:, before:before + t.shape[1]]
    v.copy_(t)
    return wide, v


@pytest.mark.parametrize("path", [lr.PATH_AUTO, lr.PATH_GATHER, lr.PATH_SGMV])
@pytest.mark.parametrize("with_norm", [False, True])
@pytest.mark.parametrize("M,k,d", [(1, 64, 33), (130, 264, 201), (700, 512, 1)])
def test_layer_of_odd_widths_in_wider_tensors(M, k, d, with_norm, path):
    """Every tensor a column range of a wider one, y and the norm's at odd
    offsets: the bits of the same rows alone, and nothing beside them."""
    w = wl.custom(seed=d, M=M, k=k, d=d, ranks=[4, 16, 64, 8], max_rank=64, none_frac=0.2)
    slices, W, _ = layer_inputs(w)
    x, ids = w.x.cuda(), torch.from_numpy(w.ids).cuda()
    res, g = rand(3, M, k, BF).cuda(), torch.ones(k, dtype=BF, device="cuda")
    h = torch.empty_like(x) if with_norm else None
    want = lr.lora_linear_sliced_mx(x, W, slices, ids, path=path, norm=lr.Norm(g, 1e-5, res, h) if with_norm else None)
    Xw, xs = rows_in_wide(x, 8, 16)
    Rw, rs = rows_in_wide(res, 3, 2)
    Hw, hs = rows_in_wide(torch.zeros_like(res), 1, 4)
    Yw, ys = rows_in_wide(torch.zeros(M, d, dtype=BF, device="cuda"), 3, 7)
    norm = lr.Norm(g, 1e-5, rs, hs) if with_norm else None
    lr.lora_linear_sliced_mx(xs, W, slices, ids, path=path, norm=norm, y=ys)
    assert torch.equal(ys, want)
    assert (Yw[:, :3] == 5).all() and (Yw[:, 3 + d:] == 5).all()
    assert (Xw[:, :8] == 5).all() and (Xw[:, 8 + k:] == 5).all() and torch.equal(xs, x)
    if with_norm:
        assert torch.equal(hs, h) and (Hw[:, :1] == 5).all() and (Hw[:, 1 + k:] == 5).all()


def test_layer_of_ranks_past_the_matrix_paths(oracle_mod):
    """Ranks up to 128 take the gather path; SGMV refuses them."""
    w = wl.custom(seed=2, M=90, k=256, d=136, ranks=[128, 8, 100], max_rank=128, none_frac=0.1)
    slices, W, Wv = layer_inputs(w)
    x, ids = w.x.cuda(), torch.from_numpy(w.ids).cuda()
    want = oracle_layer(oracle_mod, w, ["out"], w.x, R.quantised_values(R.f64(w.x), R.FP8), Wv)
    assert normwise(R.f64(lr.lora_linear_sliced_mx(x, W, slices, ids)), want) <= TOL
    with pytest.raises(lr.LoraError):
        lr.lora_linear_sliced_mx(x, W, slices, ids, path=lr.PATH_SGMV)


def test_layer_captured_with_a_plan_of_its_own():
    """More than 64 adapters: the plan runs on a stream beside, in a graph as
    outside; two captured layers replayed in turn with eager ones between."""
    w = wl.custom(seed=13, M=64, k=512, d=320, ranks=[8, 32], max_rank=32, none_frac=0.2)
    slices, W, _ = layer_inputs(w)
    slices = more_slots(slices, 80)
    g = torch.ones(512, dtype=BF, device="cuda")
    n = lr.workspace_bytes_sliced_mx(64, 512, lr.MX_FP8, slices)
    sets = [(rand(i, 64, 512, BF).cuda(), torch.from_numpy(np.roll(w.ids, i)).cuda(),
             torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty(64, 320, dtype=BF, device="cuda"))
            for i in range(2)]

    def call(i):
        x, ids, ws, y = sets[i]
        return lr.lora_linear_sliced_mx(x, W, slices, ids, norm=lr.Norm(g), y=y, workspace=ws)

    for i in (0, 1):
        call(i)
    torch.cuda.synchronize()
    graphs = []
    for i in (0, 1):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            call(i)
    for rep in range(4):
        for i in (0, 1):
            sets[i][0].copy_(rand(60 + 2 * rep + i, 64, 512, BF))
            sets[i][3].zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            got = sets[i][3].clone()
            want = lr.lora_linear_sliced_mx(sets[i][0], W, slices, sets[i][1], norm=lr.Norm(g))
            assert torch.equal(got, want)

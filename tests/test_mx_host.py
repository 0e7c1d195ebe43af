"""Microscaled operators without a GPU: every refusal of the C entry points is
decided on the host before anything is launched, the plain reference agrees
with the formats' definition, and the binding checks its tensors."""
import ctypes

import numpy as np
import pytest
import torch

import lora_row_adapter_amd as lr
from lora_row_adapter_amd import _binding as B
import mx_ref as R

ARG, SHAPE, DTYPE, WORKSPACE, UNSUPPORTED = 1, 2, 3, 5, 8


def mx(fmt=1, q=1 << 20, ldq=64, scales=1 << 24, lds=4):
    c = B._CMx()
    c.format, c.q, c.ldq, c.scales, c.lds = fmt, q, ldq, scales, lds
    return c


def norm(weight=1 << 28, eps=1e-5, residual=0, ldr=0, out=0, ldro=0):
    c = B._CNorm()
    c.weight, c.eps, c.residual, c.ldr, c.residual_out, c.ldro = weight, eps, residual, ldr, out, ldro
    return c


def ref(c):
    return None if c is None else ctypes.byref(c)


def quantize(m, dtype=1, M=4, k=64, x=1 << 16, ldx=64, fn="lora_mx_quantize"):
    lib = lr.load_library()
    if fn == "lora_mx_quantize":
        return lib.lora_mx_quantize(dtype, M, k, x, ldx, ref(m), None)
    return lib.lora_mx_dequantize(dtype, M, k, ref(m), x, ldx, None)


@pytest.mark.parametrize("fn", ["lora_mx_quantize", "lora_mx_dequantize"])
@pytest.mark.parametrize("want,kw,m", [
    (ARG, {}, None),
    (ARG, {"x": 0}, mx()),
    (ARG, {}, mx(q=0)),
    (ARG, {}, mx(scales=0)),
    (DTYPE, {"dtype": 2}, mx()),
    (DTYPE, {}, mx(fmt=0)),
    (DTYPE, {}, mx(fmt=3)),
    (SHAPE, {"M": -1}, mx()),
    (SHAPE, {"k": 0}, mx()),
    (SHAPE, {"k": 1 << 31, "ldx": 1 << 31}, mx(ldq=1 << 32, lds=1 << 27)),
    (SHAPE, {"ldx": 63}, mx()),
    (SHAPE, {"x": (1 << 16) + 1}, mx()),         # element alignment
    (SHAPE, {}, mx(q=(1 << 20) + 8)),            # codes not 16-byte aligned
    (SHAPE, {}, mx(ldq=72)),                     # ldq not a multiple of 16
    (SHAPE, {}, mx(ldq=48)),                     # ldq below a row's codes
    (SHAPE, {}, mx(scales=(1 << 24) + 2)),
    (SHAPE, {}, mx(lds=6)),
    (SHAPE, {"k": 129, "ldx": 129}, mx(ldq=160)),  # five blocks, four scales
    (ARG, {"x": 1 << 20}, mx()),                 # x over the codes
    (ARG, {"x": (1 << 24) + 8}, mx()),           # x over the scales
    (ARG, {}, mx(scales=(1 << 20) + 64)),        # scales over the codes
])
def test_quantize_and_dequantize_refuse(fn, want, kw, m):
    assert quantize(m, fn=fn, **kw) == want


def test_empty_matrices_are_no_ops():
    lib = lr.load_library()
    m = mx(q=0, scales=0)
    assert quantize(m, M=0, x=0) == 0
    assert quantize(m, M=0, x=0, fn="lora_mx_dequantize") == 0
    assert lib.lora_rmsnorm(1, 0, 64, None, 0, ref(norm(weight=0)), 1 << 16, 64, None, None) == 0
    W = mx(fmt=2, ldq=32)
    assert lib.lora_gemm_mx(0, 64, 8, ref(m), ref(W), None, 8, None) == 0


def rms(n, dtype=1, M=4, k=64, x=1 << 16, ldx=64, y=1 << 17, ldy=64, yq=None):
    return lr.load_library().lora_rmsnorm(dtype, M, k, x, ldx, ref(n), y, ldy, ref(yq), None)


@pytest.mark.parametrize("want,kw,n", [
    (ARG, {}, None),
    (ARG, {}, norm(weight=0)),
    (ARG, {}, norm(eps=-1.0)),
    (ARG, {}, norm(eps=float("nan"))),
    (ARG, {}, norm(eps=float("inf"))),
    (ARG, {"x": 0}, norm()),
    (ARG, {"y": None}, norm()),                              # nothing asked for
    (DTYPE, {"dtype": 9}, norm()),
    (DTYPE, {"yq": mx(fmt=7)}, norm()),
    (SHAPE, {"ldx": 60}, norm()),
    (SHAPE, {"ldy": 60}, norm()),
    (SHAPE, {}, norm(residual=1 << 18, ldr=60)),
    (SHAPE, {}, norm(out=1 << 18, ldro=60)),
    (SHAPE, {}, norm(weight=(1 << 28) + 1)),
    (SHAPE, {"yq": mx(ldq=32)}, norm()),
    (ARG, {"y": (1 << 16) + 128 * 2}, norm()),               # y over x, two rows further
    (ARG, {"y": 1 << 16, "ldy": 128}, norm()),               # y over x with another stride
    (ARG, {}, norm(out=1 << 17, ldro=64)),                   # both outputs in one place
    (ARG, {"y": 1 << 16}, norm(out=1 << 16, ldro=64)),       # both in place of x
    (ARG, {"y": 1 << 28}, norm()),                           # y over the weight
    (ARG, {"yq": mx(q=1 << 16)}, norm()),                    # codes over x
    (ARG, {"yq": mx(q=1 << 17)}, norm()),                    # codes over y
    (ARG, {"yq": mx(scales=1 << 18)}, norm(residual=1 << 18, ldr=64)),
])
def test_rmsnorm_refuses(want, kw, n):
    assert rms(n, **kw) == want


def gemm(x, W, M=4, k=64, d=8, y=1 << 26, ldy=8):
    return lr.load_library().lora_gemm_mx(M, k, d, ref(x), ref(W), y, ldy, None)


@pytest.mark.parametrize("want,kw,x,W", [
    (ARG, {}, None, mx(fmt=2)),
    (ARG, {}, mx(), None),
    (ARG, {"y": None}, mx(), mx(fmt=2)),
    (DTYPE, {}, mx(fmt=5), mx(fmt=2)),
    (UNSUPPORTED, {}, mx(), mx(fmt=1)),          # an 8-bit base weight
    (SHAPE, {"M": -1}, mx(), mx(fmt=2)),
    (SHAPE, {"d": 0}, mx(), mx(fmt=2)),
    (SHAPE, {"ldy": 7}, mx(), mx(fmt=2)),
    (SHAPE, {"y": (1 << 26) + 1}, mx(), mx(fmt=2)),
    (SHAPE, {}, mx(ldq=1 << 24), mx(fmt=2)),     # rows past the 32-bit offsets of a tile
    (SHAPE, {}, mx(), mx(fmt=2, ldq=1 << 24)),
])
def test_gemm_refuses(want, kw, x, W):
    assert gemm(x, W, **kw) == want


def slices(d=8, S=4, Rk=16):
    a = (B._CSlice * 1)()
    a[0].d, a[0].scales = d, 1 << 12
    c = a[0].adapters
    c.n_adapters, c.max_rank, c.ranks, c.A, c.B = S, Rk, 1 << 12, 1 << 12, 1 << 12
    return a


def layer(M=4, k=64, x=1 << 16, ldx=64, n=None, fmt=1, W="w", sl=None, ids=1 << 14, y=1 << 26, ldy=8,
          ws=1 << 30, ws_bytes=1 << 28, path=0, flags=0):
    W = mx(fmt=2, ldq=32) if W == "w" else W
    return lr.load_library().lora_linear_sliced_mx(M, k, x, ldx, ref(n), fmt, ref(W), 1, sl or slices(), ids, y,
                                                   ldy, ws, ws_bytes, path, flags, None)


@pytest.mark.parametrize("want,kw", [
    (DTYPE, {"fmt": 0}),
    (ARG, {"W": None}),
    (UNSUPPORTED, {"W": mx(fmt=1)}),
    (ARG, {"x": None}),
    (ARG, {"ids": None}),
    (ARG, {"ws": None}),
    (SHAPE, {"k": 60, "ldx": 64}),               # k not a multiple of 8
    (SHAPE, {"x": (1 << 16) + 2}),
    (SHAPE, {"ldy": 7}),
    (WORKSPACE, {"ws": (1 << 30) + 16}),
    (WORKSPACE, {"ws_bytes": 4096}),
    (ARG, {"path": 7}),
    (ARG, {"flags": 8}),
    (ARG, {"n": norm(weight=0)}),
    (ARG, {"n": norm(eps=-1.0)}),
    (ARG, {"n": norm(out=1 << 26, ldro=64)}),    # the residual's sum over y
    (SHAPE, {"n": norm(residual=1 << 18, ldr=8)}),
])
def test_layer_refuses(want, kw):
    assert layer(**kw) == want


def test_layer_workspace_bytes():
    lib = lr.load_library()
    sl = slices()
    plan = lib.lora_workspace_bytes_sliced(100, 96, 1, 1, sl)
    # behind the plan: codes, scales (rows of 3 blocks: 4 bytes), normed bf16 rows, each up to 256
    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    assert lib.lora_workspace_bytes_sliced_mx(100, 96, 1, 1, sl) == plan + up(9600) + up(400) + up(19200)
    assert lib.lora_workspace_bytes_sliced_mx(100, 96, 2, 1, sl) == plan + up(4800) + up(400) + up(19200)
    # batches past the plan's rows run in chunks
    assert lib.lora_workspace_bytes_sliced_mx(8192, 96, 1, 1, sl) == lib.lora_workspace_bytes_sliced_mx(90000, 96, 1, 1, sl)
    for bad in ((100, 96, 0, 1, sl), (-1, 96, 1, 1, sl), (100, 0, 1, 1, sl), (100, 96, 1, 0, sl), (100, 96, 1, 1, None)):
        assert lib.lora_workspace_bytes_sliced_mx(*bad) == 0
    # a workspace one byte short is refused
    n = lib.lora_workspace_bytes_sliced_mx(4, 64, 1, 1, sl)
    assert layer(ws_bytes=n - 1 - 256) == WORKSPACE


def test_binding_refuses_host_tensors_and_wrong_types():
    u = torch.zeros(4, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        lr.MX(lr.MX_FP8, u, torch.zeros(4, 4, dtype=torch.uint8), 64)
    with pytest.raises(ValueError):
        lr.MX(9, u, u, 64)
    with pytest.raises(TypeError):
        lr.MX(lr.MX_FP8, u.float(), u, 64)
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        lr.lora_mx_quantize(x)
    with pytest.raises(TypeError):
        lr.lora_mx_quantize(x.half())
    with pytest.raises(ValueError):
        lr.lora_rmsnorm(x, lr.Norm(torch.ones(64)))
    with pytest.raises(TypeError):
        lr.lora_linear_sliced_mx(x, None, [], torch.zeros(4))


def test_reference_quantiser_on_known_values():
    # e2m1 with amax 6 -> scale 1: ties go to the even code, the sign is kept
    x = np.zeros((1, 32))
    x[0, :12] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -5.1, 7.9, -0.0]
    c, s = R.quantise(x, R.FP4)
    assert s[0, 0] == 127
    vals = R.code_values(R.FP4)[c[0, :12]]
    assert vals.tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -6, 6, 0]
    assert c[0, 8] == 8 and c[0, 11] == 8      # -0
    # e4m3: 448 is the largest code, the smallest is 2^-9
    x[0, :5] = [500, 256, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10]
    c, s = R.quantise(x[:, :], R.FP8)
    assert s[0, 0] == 127
    assert R.code_values(R.FP8)[c[0, :5]].tolist() == [448, 256, 2.0 ** -9, 0, 2.0 ** -8]
    # zero blocks, subnormal blocks, blocks with an infinity or NaN
    x = np.zeros((4, 32))
    x[1, 3], x[2, 0], x[3, 31] = 2.0 ** -149, np.inf, np.nan
    c, s = R.quantise(x, R.FP8)
    assert s[:, 0].tolist() == [0, 0, 255, 255]
    assert not c.any()
    # a short last block is filled with zeros
    c, s = R.quantise(np.ones((2, 33)), R.FP4)
    assert c.shape == (2, 64) and s.shape == (2, 2) and not c[:, 33:].any()
    assert (R.dequantise(c, s, R.FP4, 33) == 1).all()


@pytest.mark.parametrize("kw,x,W", [
    ({"y": 1 << 20}, mx(), mx(fmt=2, q=1 << 21, scales=1 << 25)),                  # over x's codes
    ({"y": (1 << 24) + 12}, mx(), mx(fmt=2, q=1 << 21, scales=1 << 25)),           # over x's last scales
    ({"y": (1 << 21) - 62}, mx(), mx(fmt=2, q=1 << 21, scales=1 << 25)),           # into W's codes
    ({"y": 1 << 25}, mx(), mx(fmt=2, q=1 << 21, scales=1 << 25)),
    ({"M": 1 << 30, "y": 1 << 30, "ldy": 1 << 39}, mx(q=1 << 40), mx(fmt=2, q=1 << 21)),  # ranges past 64 bits
])
def test_gemm_refuses_an_output_over_an_operand(kw, x, W):
    assert gemm(x, W, **kw) == ARG


@pytest.mark.parametrize("kw", [
    {"y": 1 << 16},                                                # y over x
    {"y": (1 << 16) + 4 * 128 - 2},                                # the last element of x
    {"y": 1 << 18, "n": norm(residual=1 << 18, ldr=64)},           # over the residual
    {"y": 1 << 16, "n": norm()},
    {"y": 1 << 30},                                                # in the workspace
    {"x": 1 << 30},
    {"n": norm(out=(1 << 30) + (1 << 20), ldro=64)},
    {"n": norm(residual=(1 << 30) + (1 << 20), ldr=64)},
])
def test_layer_refuses_overlaps(kw):
    assert layer(**kw) == ARG


@pytest.mark.parametrize("kw", [{"ldy": 1 << 60}, {"ldx": 1 << 60}])
def test_layer_refuses_strides_past_any_memory(kw):
    assert layer(**kw) == SHAPE


APART = mx(fmt=2, q=1 << 40, ldq=32, scales=1 << 41)


@pytest.mark.parametrize("kw", [
    {"y": 1 << 40},                                                # y over W's codes
    {"y": (1 << 40) + 8 * 32 - 2},                                 # their last bytes
    {"y": (1 << 40) - 4 * 16 + 2},                                 # y's last element over their first byte
    {"y": 1 << 41},                                                # over W's scales
    {"y": (1 << 41) + 7 * 4},                                      # the last row's
    {"ws": 1 << 40},
    {"ws": (1 << 41) - (1 << 28) + 256},
    {"n": norm(out=1 << 40, ldro=64)},                             # the residual's sum over W
    {"n": norm(out=(1 << 41) + 16, ldro=64)},
    {"y": 1 << 28, "n": norm()},                                   # y over the norm's weight
    {"y": (1 << 28) + 126, "n": norm()},
    {"ws": 1 << 28, "ws_bytes": 1 << 20, "n": norm()},
    {"n": norm(out=1 << 28, ldro=64)},
])
def test_layer_refuses_outputs_over_its_weights(kw):
    kw = dict({"ws": 1 << 45}, **kw)
    assert layer(W=APART, **kw) == ARG


@pytest.mark.parametrize("M,k,d", [(4, 64, 8), (512, 8192, 9216), (256, 4096, 1024), (8192, 4096, 4096), (1, 8192, 9216)])
def test_layer_workspace_is_what_the_layer_checks_for(M, k, d):
    """Not a byte more: one less is refused, also at sizes where the dense
    layer's workspace has a region for its base product."""
    lib = lr.load_library()
    sl = slices(d=d)
    for fmt in (1, 2):
        n = lib.lora_workspace_bytes_sliced_mx(M, k, fmt, 1, sl)
        own = sum((v + 255) // 256 * 256 for v in (M * k // fmt, M * k // 32, 2 * M * k))
        assert n == lib.lora_workspace_bytes_sliced(M, k, 0, 1, sl) + own  # fp32: the plan's regions
        short = dict(M=M, k=k, ldx=k, fmt=fmt, W=mx(fmt=2, ldq=k // 2, lds=max(k // 32, 4), q=1 << 40, scales=1 << 41),
                     sl=sl, ldy=d, x=1 << 33, y=1 << 34, ws=1 << 45)
        assert layer(ws_bytes=n - 1, **short) == WORKSPACE


@pytest.mark.parametrize("fmt", [R.FP8, R.FP4])
def test_long_sizes_reach_every_tile_shape(fmt):
    """The sizes of the products with long k take each tile shape once, go
    round its rings and leave a part of a tile."""
    for i, (M, k, d) in enumerate(R.LONG[fmt]):
        at, rows, cols, ring = lr.test_gemm_mx_shape(M, k, d, fmt)
        assert at == i
        assert k > 1.9 * ring and k % 32 and d > cols and d % cols and M % rows
    seen = {lr.test_gemm_mx_shape(int(2 ** m), int(2 ** k), int(2 ** d), fmt)[0]
            for m in np.arange(0, 13.1, 0.25) for k in np.arange(5, 14, 0.5) for d in np.arange(0, 14.1, 0.25)}
    assert seen <= set(range(len(R.LONG[fmt])))


def test_shape_hook_refuses():
    lib = lr.load_library()
    out = (ctypes.c_int32 * 3)()
    for bad in ((0, 64, 8, 1, out), (4, 0, 8, 1, out), (4, 64, 0, 1, out), (4, 64, 8, 3, out), (4, 64, 8, 1, None),
                (4, 1 << 31, 8, 1, out)):
        assert lib.lora_test_gemm_mx_shape(*bad) == -1
    with pytest.raises(lr.LoraError):
        lr.test_gemm_mx_shape(4, 64, 8, 0)

"""The operators over a 4-bit weight and the norm and rotation of heads without
a GPU: every refusal of the C entry points is decided on the host before
anything is launched, and the plain references agree with the definitions."""
import ctypes

import numpy as np
import pytest
import torch

import lora_row_adapter_amd as lr
from lora_row_adapter_amd import _binding as B
import w4_ref as R

ARG, SHAPE, DTYPE, RANK, WORKSPACE, UNSUPPORTED = 1, 2, 3, 4, 5, 8


def ref(c):
    return None if c is None else ctypes.byref(c)


# ------------------------------------------------------------ weight
@pytest.mark.parametrize("d,k,group,want", [
    (1, 1, 32, 1024 + 256), (16, 128, 64, 1024 + 128), (16, 128, 128, 1024 + 64), (17, 129, 128, 4 * 1088),
    (9216, 8192, 128, 576 * 64 * 1088), (16, 128, 1024, 1088),
    (0, 128, 128, 0), (16, 0, 128, 0), (16, 128, 0, 0), (16, 128, -32, 0), (16, 128, 16, 0), (16, 128, 96, 0),
    (16, 128, 192, 0), (16, 1 << 25, 128, 0), (1 << 31, 128, 128, 0), ((1 << 31) - 1, 1 << 24, 128, 0),
])
def test_bytes(d, k, group, want):
    assert lr.load_library().lora_w4_bytes(d, k, group) == want


def pack(d=16, k=256, group=128, q=1 << 16, ldq=128, dt=1, s=1 << 20, lds=2, z=1 << 22, ldz=2, out=1 << 24):
    return lr.load_library().lora_w4_pack(d, k, group, q, ldq, dt, s, lds, z, ldz, out, None)


@pytest.mark.parametrize("want,kw", [
    (DTYPE, {"dt": 2}), (DTYPE, {"dt": -1}), (SHAPE, {"d": 0}), (SHAPE, {"k": 0}), (SHAPE, {"group": 100}),
    (ARG, {"q": 0}), (ARG, {"s": 0}), (ARG, {"out": 0}),
    (SHAPE, {"ldq": 127}), (SHAPE, {"lds": 1}), (SHAPE, {"ldz": 1}), (SHAPE, {"ldq": 1 << 41}),
    (SHAPE, {"s": (1 << 20) + 1}), (SHAPE, {"s": (1 << 20) + 2, "dt": 0}), (SHAPE, {"out": (1 << 24) + 128}),
    (ARG, {"out": 1 << 16}), (ARG, {"out": (1 << 20) - 256}), (ARG, {"out": 1 << 22}),
])
def test_pack_refuses(want, kw):
    assert pack(**kw) == want


def w4(data=1 << 24, group=128):
    return B._CW4(group, data)


def dequant(W, dt=1, d=16, k=256, y=1 << 28, ldy=256):
    return lr.load_library().lora_w4_dequantize(dt, d, k, ref(W), y, ldy, None)


@pytest.mark.parametrize("want,kw,W", [
    (ARG, {}, None), (ARG, {}, w4(data=0)), (SHAPE, {}, w4(data=(1 << 24) + 16)), (SHAPE, {}, w4(group=33)),
    (DTYPE, {"dt": 5}, w4()), (ARG, {"y": 0}, w4()), (SHAPE, {"ldy": 255}, w4()), (SHAPE, {"y": (1 << 28) + 1}, w4()),
    (SHAPE, {"d": 0}, w4()), (SHAPE, {"k": 0}, w4()), (ARG, {"y": (1 << 24) + 16}, w4()),
])
def test_dequantize_refuses(want, kw, W):
    assert dequant(W, **kw) == want


def gemm(W, M=4, k=256, d=16, x=1 << 26, ldx=256, y=1 << 28, ldy=16):
    return lr.load_library().lora_gemm_w4(M, k, d, x, ldx, ref(W), y, ldy, None)


@pytest.mark.parametrize("want,kw,W", [
    (ARG, {}, None), (ARG, {}, w4(data=0)), (SHAPE, {}, w4(group=1)), (SHAPE, {"M": -1}, w4()), (SHAPE, {"d": 0}, w4()),
    (SHAPE, {"M": 1 << 31}, w4()), (SHAPE, {"k": 0}, w4()), (SHAPE, {"k": (1 << 24) + 8, "ldx": 1 << 25}, w4()),
    (ARG, {"x": 0}, w4()), (ARG, {"y": 0}, w4()), (SHAPE, {"ldx": 248}, w4()), (SHAPE, {"ldx": 257}, w4()),
    (SHAPE, {"x": (1 << 26) + 8}, w4()), (SHAPE, {"k": 252}, w4()), (SHAPE, {"ldy": 15}, w4()),
    (SHAPE, {"y": (1 << 28) + 1}, w4()), (SHAPE, {"ldy": 1 << 40}, w4()),
    (ARG, {"y": (1 << 26) + 512}, w4()), (ARG, {"y": 1 << 24}, w4()),
    (0, {"M": 0, "x": 0, "y": 0}, w4()),
])
def test_gemm_refuses(want, kw, W):
    assert gemm(W, **kw) == want


def slices(d=16, S=4, Rk=16, scales=1 << 12):
    a = (B._CSlice * 1)()
    a[0].d, a[0].scales = d, scales
    c = a[0].adapters
    c.n_adapters, c.max_rank, c.ranks, c.A, c.B = S, Rk, 1 << 12, 1 << 12, 1 << 12
    return a


def layer(W="w", M=4, k=256, x=1 << 26, ldx=256, sl=None, n=1, ids=1 << 14, y=1 << 28, ldy=16, ws=1 << 32, wsn=1 << 28,
          path=0, flags=0):
    W = w4() if W == "w" else W
    return lr.load_library().lora_linear_sliced_w4(M, k, x, ldx, ref(W), n, slices() if sl is None else sl, ids, y, ldy,
                                                   ws, wsn, path, flags, None)


@pytest.mark.parametrize("want,kw", [
    (ARG, {"W": None}), (ARG, {"x": 0}), (ARG, {"y": 0}), (ARG, {"ids": 0}), (ARG, {"ws": 0}), (ARG, {"n": 0}),
    (ARG, {"n": 5}), (ARG, {"path": 3}), (ARG, {"flags": 8}), (WORKSPACE, {"wsn": 256}), (WORKSPACE, {"ws": (1 << 32) + 64}),
    (ARG, {"sl": slices(scales=0)}), (RANK, {"sl": slices(Rk=300)}), (SHAPE, {"sl": slices(d=17)}),
    (ARG, {"sl": slices(S=0)}), (UNSUPPORTED, {"sl": slices(Rk=128), "path": 2}),
    (ARG, {"y": 1 << 32}), (ARG, {"y": 1 << 26}), (ARG, {"y": 1 << 24}), (ARG, {"x": 1 << 32}), (ARG, {"M": 9000, "flags": 1}),
    (SHAPE, {"k": 100}), (0, {"M": 0}),
])
def test_layer_refuses(want, kw):
    assert layer(**kw) == want


def test_shape_hook():
    lib = lr.load_library()
    out = (ctypes.c_int32 * 3)()
    assert lib.lora_test_gemm_w4_shape(1, 8192, 9216, 128, out) >= 0 and out[0] == 16 and out[2] == 0
    assert lib.lora_test_gemm_w4_shape(8192, 4096, 4096, 64, out) >= 0 and out[0] >= 128 and out[2] == 1
    for M, k, d, group, o in [(0, 64, 64, 32, out), (1, 0, 64, 32, out), (1, 64, 0, 32, out), (1, 64, 64, 31, out),
                              (1, 64, 64, 32, None)]:
        assert lib.lora_test_gemm_w4_shape(M, k, d, group, o) == -1


def test_workspace_sizes():
    lib = lr.load_library()
    sl = slices()
    n = lib.lora_workspace_bytes_sliced_w4(64, 256, 1, sl)
    assert 0 < n <= lib.lora_workspace_bytes_sliced_w4(4096, 256, 1, sl)
    assert lib.lora_workspace_bytes_sliced_w4(-1, 256, 1, sl) == 0
    assert lib.lora_workspace_bytes_sliced_w4(64, 0, 1, sl) == 0
    assert lib.lora_workspace_bytes_sliced_w4(64, 1 << 25, 1, sl) == 0
    assert lib.lora_workspace_bytes_sliced_w4(64, 256, 5, sl) == 0
    assert lib.lora_workspace_bytes_sliced_w4(64, 256, 1, None) == 0


# ------------------------------------------------------------ heads
def heads(x=1 << 20, lr_=256, lh=64, n=4, w=1 << 18, out=1 << 24, lor=256, loh=64):
    return B._CHeads(n, x, lr_, lh, w, out, lor, loh)


def rope(pos=1 << 16, inv=1 << 17, rot=64, inter=0, scale=1.0):
    return B._CRope(pos, inv, rot, inter, scale)


def norm_rope(q="q", k=None, r="r", dt=1, M=3, D=64, eps=1e-6):
    q = heads() if q == "q" else q
    r = rope() if r == "r" else r
    return lr.load_library().lora_qk_norm_rope(dt, M, D, eps, ref(q), ref(k), ref(r), None)


@pytest.mark.parametrize("want,kw", [
    (ARG, {"q": None}), (DTYPE, {"dt": 2}), (SHAPE, {"M": -1}), (SHAPE, {"M": 1 << 31}), (SHAPE, {"D": 0}),
    (SHAPE, {"D": 1025}), (ARG, {"eps": -1e-6}), (ARG, {"eps": float("nan")}), (ARG, {"eps": float("inf")}),
    (ARG, {"q": heads(x=0)}), (ARG, {"q": heads(out=0)}), (SHAPE, {"q": heads(n=0)}), (SHAPE, {"q": heads(n=65536)}),
    (SHAPE, {"q": heads(x=(1 << 20) + 1)}), (SHAPE, {"q": heads(out=(1 << 24) + 1)}), (SHAPE, {"q": heads(w=(1 << 18) + 1)}),
    (SHAPE, {"q": heads(lh=63)}), (SHAPE, {"q": heads(lr_=200)}), (SHAPE, {"q": heads(lor=32)}), (SHAPE, {"q": heads(loh=0)}),
    (SHAPE, {"q": heads(lr_=1 << 41)}), (SHAPE, {"q": heads(lr_=64, lh=128)}),
    (SHAPE, {"r": rope(rot=0)}), (SHAPE, {"r": rope(rot=63)}), (SHAPE, {"r": rope(rot=66)}), (ARG, {"r": rope(inter=2)}),
    (ARG, {"r": rope(scale=float("inf"))}), (ARG, {"r": rope(scale=float("nan"))}), (ARG, {"r": rope(pos=0)}),
    (ARG, {"r": rope(inv=0)}), (SHAPE, {"r": rope(pos=(1 << 16) + 4)}), (SHAPE, {"r": rope(inv=(1 << 17) + 2)}),
    # outputs over inputs
    (ARG, {"q": heads(out=(1 << 20) + 2)}),                       # a shifted copy of itself
    (ARG, {"q": heads(out=1 << 20, loh=64, lor=512)}),            # its own place with another stride
    (ARG, {"k": heads(x=1 << 24, out=1 << 26)}),                  # q's output over k
    (ARG, {"k": heads(x=1 << 22, out=1 << 24)}),                  # both outputs in one place
    (ARG, {"q": heads(out=1 << 18)}), (ARG, {"q": heads(out=1 << 16)}), (ARG, {"q": heads(out=1 << 17)}),
    # heads of q and k in one buffer, one of them shared
    (ARG, {"q": heads(out=1 << 20, lr_=512, lor=512), "k": heads(x=(1 << 20) + 384, lr_=512, out=1 << 26)}),
    (ARG, {"q": heads(n=4, lr_=768, lor=768, lh=192, loh=192, out=1 << 20),
           "k": heads(x=(1 << 20) + 64, lr_=768, lh=192, out=(1 << 20) + 64, lor=768, loh=192)}),
    (0, {"M": 0, "q": heads(x=0, out=0)}),
])
def test_norm_rope_refuses(want, kw):
    assert norm_rope(**kw) == want


def test_reference_packing_and_rotation():
    q, s, z = R.weight(1, 3, 5, 32)
    p = R.pack(q)
    assert p.shape == (3, 3) and (p[:, 0] & 15 == q[:, 0]).all() and (p[:, 1] >> 4 == q[:, 3]).all()
    W = R.dequant(q, s, z, 32)
    assert W[1, 2] == float(s[1, 0]) * (int(q[1, 2]) - int(z[1, 0]))
    # a rotation by a right angle, by hand, in both pairings
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    c, sn = np.zeros((1, 2)), np.ones((1, 2))
    assert R.heads(x, None, 0, c, sn, 4, False)[0].ravel().tolist() == [-3, -4, 1, 2]
    assert R.heads(x, None, 0, c, sn, 4, True)[0].ravel().tolist() == [-2, 1, -4, 3]
    # and a norm: mean square 7.5
    assert np.allclose(R.heads(x, np.ones(4), 0, None, None, 0, False)[0], x / np.sqrt(7.5))

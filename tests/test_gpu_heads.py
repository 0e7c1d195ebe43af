"""Norm and rotation of query and key heads on the GPU against a plain 64-bit
implementation.

Tolerance.  In fp32 a normed value takes two roundings (2^-24 each), cos and
sin are off by at most 2^-22 (their argument's rounding, 2 pi 2^-25, and the
function's error of a few units in the last place), a rotated value two
products and a sum: in all below 2^-21 of the two values' magnitudes.  The
output's rounding adds 2^-24 (fp32) or 2^-8 (bf16) of the value.
"""
import math

import numpy as np
import pytest
import torch

import lora_row_adapter_amd as lr
import w4_ref as R
from gpu_helpers import say

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


def f64(t):
    return t.detach().cpu().double().numpy()


def rand(seed, *shape, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * torch.exp(torch.randn(shape[-1], generator=g))).to(dtype)


def freqs(rot, base=10000.0):
    return torch.tensor([base ** (-2 * i / rot) for i in range(rot // 2)], dtype=F32)


def turns(pos, inv, scale=1.0):
    angle = pos.astype(np.float64)[:, None] * f64(inv)[None]
    return np.cos(angle) * scale, np.sin(angle) * scale


def check(got, x, w, eps, cs, rot, interleaved, rows=None):
    want, mag = R.heads(f64(x), None if w is None else f64(w), eps, *(cs or (None, None)), rot, interleaved)
    g = f64(got)
    tol = 2.0 ** -21 * mag + (2.0 ** -8 if got.dtype == BF else 2.0 ** -24) * np.abs(want)
    ok = np.abs(g - want) <= tol
    assert ok[slice(None) if rows is None else rows].all()


CASES = [  # M, hq, hk, D, rot, interleaved
    (1, 1, 1, 2, 2, False), (1, 64, 8, 128, 128, False), (3, 5, 2, 64, 64, True), (7, 4, 4, 80, 40, False),
    (7, 4, 4, 80, 40, True), (2, 3, 1, 96, 96, False), (33, 12, 3, 128, 64, True), (5, 2, 2, 256, 256, False),
    (4, 1, 1, 1024, 1024, False), (4, 1, 1, 1024, 6, True), (6, 3, 2, 33, 32, False), (6, 3, 2, 17, 2, True),
    (130, 7, 1, 68, 34, False), (9, 2, 1, 576, 64, False), (257, 2, 2, 16, 16, True), (1000, 3, 1, 40, 40, False),
    (5, 130, 9, 128, 128, False), (11, 9, 9, 72, 72, True), (3, 1, 1, 1, 0, False), (12, 10, 2, 192, 128, True),
]


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_heads(case, dtype, norm):
    M, hq, hk, D, rot, inter = case
    say("heads %s %s norm=%d" % (case, dtype, norm))
    q, k = rand(M, M, hq, D, dtype=dtype), rand(M + 1, M, hk, D, dtype=dtype)
    wq, wk = (1 + 0.3 * rand(3, D).to(dtype), 1 + 0.3 * rand(4, D).to(dtype)) if norm else (None, None)
    pos = np.random.default_rng(M).integers(0, 200000, M)
    rope = cs = None
    if rot:
        inv = freqs(rot)
        rope, cs = lr.Rope(inv.cuda(), interleaved=inter, scale=1.25), turns(pos, inv, 1.25)
    dev = lambda t: None if t is None else t.cuda()
    a, b = lr.lora_qk_norm_rope(q.cuda(), k.cuda(), torch.from_numpy(pos).cuda(), rope, dev(wq), dev(wk), eps=1e-5)
    check(a, q, wq, 1e-5, cs, rot, inter)
    check(b, k, wk, 1e-5, cs, rot, inter)


LAYOUTS = ["rows", "heads_first", "fused", "interleaved", "padded", "odd"]


def lay(t, layout, fill=0.0):
    """A device view of t [M, H, D] in that layout, and the buffer under it."""
    M, H, D = t.shape
    if layout == "heads_first":
        buf = torch.full((H, M, D), fill, dtype=t.dtype, device="cuda")
        view = buf.permute(1, 0, 2)
    elif layout == "padded":
        buf = torch.full((M, H + 1, D + 8), fill, dtype=t.dtype, device="cuda")
        view = buf[:, :H, :D]
    elif layout == "odd":  # neither 16-byte rows nor heads
        buf = torch.full((M * H * (D + 3) + 1,), fill, dtype=t.dtype, device="cuda")
        view = buf[1:].view(M, H, D + 3)[:, :, :D]
    else:
        buf = torch.full((M, H, D), fill, dtype=t.dtype, device="cuda")
        view = buf
    view.copy_(t)
    return view, buf


@pytest.mark.parametrize("place", ["in", "out"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_layouts(layout, place, dtype):
    """Views of every kind, in place and out of place; nothing beside a head is
    written."""
    M, hq, hk, D, rot = 19, 4, 4, 64, 48
    say("heads layout %s %s %s" % (layout, place, dtype))
    q, k = rand(1, M, hq, D, dtype=dtype), rand(2, M, hk, D, dtype=dtype)
    w = (1 + 0.3 * rand(3, D)).to(dtype)
    inv, pos = freqs(rot), np.arange(M) * 31
    bufs = []
    if layout in ("fused", "interleaved"):
        shape = (M, 3 * hq, D)
        buf = torch.full(shape, 7.0, dtype=dtype, device="cuda")
        if layout == "fused":
            qv, kv, rest = buf[:, :hq], buf[:, hq:2 * hq], buf[:, 2 * hq:]
        else:
            qv, kv, rest = buf[:, 0::3], buf[:, 1::3], buf[:, 2::3]
        qv.copy_(q)
        kv.copy_(k)
    else:
        (qv, b1), (kv, b2) = lay(q, layout, 7.0), lay(k, layout, 7.0)
        bufs = [b1, b2]
        rest = None
    cs = turns(pos, inv)
    kw = {}
    if place == "in":
        kw = dict(q_out=qv, k_out=kv)
    elif bufs:
        qo, ko = lay(torch.zeros_like(q), layout, 7.0), lay(torch.zeros_like(k), layout, 7.0)
        bufs = [qo[1], ko[1]]
        kw = dict(q_out=qo[0], k_out=ko[0])
    a, b = lr.lora_qk_norm_rope(qv, kv, torch.from_numpy(pos).cuda(), lr.Rope(inv.cuda()), w.cuda(), w.cuda(), **kw)
    check(a, q, w, 1e-6, cs, rot, False)
    check(b, k, w, 1e-6, cs, rot, False)
    if rest is not None:
        assert bool((rest == 7).all())
    for buf, view in zip(bufs, (a, b)):
        view.fill_(7.0)
        assert bool((buf == 7).all())


def test_queries_alone_and_norm_alone():
    q = rand(1, 6, 3, 48)
    w = (1 + 0.2 * rand(2, 48))
    a, b = lr.lora_qk_norm_rope(q.cuda(), q_weight=w.cuda())
    assert b is None
    check(a, q, w, 1e-6, None, 0, False)
    # neither norm nor rotation: a copy
    a, _ = lr.lora_qk_norm_rope(q.cuda())
    assert torch.equal(a.cpu(), q)
    # no rotation: positions are not looked at
    a, _ = lr.lora_qk_norm_rope(q.cuda(), None, torch.full((6,), -1).cuda(), None)
    assert torch.equal(a.cpu(), q)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_padding_rows_are_left(dtype):
    M = 40
    q, k = rand(1, M, 4, 64, dtype=dtype), rand(2, M, 2, 64, dtype=dtype)
    w = torch.ones(64, dtype=dtype)
    pos = np.arange(M)
    pos[[0, 3, 38, 39]] = [-1, -(1 << 62), -5, -1]
    inv = freqs(64)
    qo = torch.full((M, 4, 64), 9.0, dtype=dtype, device="cuda")
    ko = torch.full((M, 2, 64), 9.0, dtype=dtype, device="cuda")
    lr.lora_qk_norm_rope(q.cuda(), k.cuda(), torch.from_numpy(pos).cuda(), lr.Rope(inv.cuda()), w.cuda(), w.cuda(),
                         q_out=qo, k_out=ko)
    live = pos >= 0
    assert bool((qo[~live] == 9).all()) and bool((ko[~live] == 9).all())
    cs = turns(np.maximum(pos, 0), inv)
    check(qo, q, w, 1e-6, cs, 64, False, rows=live)
    check(ko, k, w, 1e-6, cs, 64, False, rows=live)


def test_far_positions():
    """Angles of positions to 2^26 keep fp32's last bits."""
    pos = np.array([0, 1, 4095, 131071, 1 << 20, (1 << 24) + 1, (1 << 26) - 1])
    M = len(pos)
    q = rand(5, M, 2, 128, dtype=F32)
    inv = freqs(128, 500000.0)
    a, _ = lr.lora_qk_norm_rope(q.cuda(), None, torch.from_numpy(pos).cuda(), lr.Rope(inv.cuda()))
    check(a, q, None, 1e-6, turns(pos, inv), 128, False)


def test_values_at_both_ends():
    """Squares past fp32's range, zeros, subnormals, and a NaN or an infinity,
    which stays in its head."""
    for dtype in (BF, F32):
        x = rand(1, 8, 2, 64, dtype=F32)
        x[0, 0] *= 1e30
        x[1, 0] *= 1e-30
        x[2, 0] = 0
        x[3, 0, 5] = float("nan")
        x[4, 0, 7] = float("inf")
        x[5, 0] = x[5, 0].sign() * 3e38
        x[6, 0] *= 1e-38
        x = x.to(dtype)
        w = (1 + 0.2 * rand(2, 64)).to(dtype)
        a, _ = lr.lora_qk_norm_rope(x.cuda(), q_weight=w.cuda(), eps=0.0)
        rows = [0, 1, 5, 7]
        check(a, x, w, 0.0, None, 0, False, rows=rows)
        with np.errstate(all="ignore"):
            want, _ = R.heads(f64(x), f64(w), 0.0, None, None, 0, False)
        assert (np.abs(f64(a)[:, 1] - want[:, 1]) <= 2.0 ** -7 * np.abs(want[:, 1])).all()
        assert bool(torch.isnan(a[3, 0]).all())
        assert not bool(torch.isfinite(a[4, 0, 7]))
        b, _ = lr.lora_qk_norm_rope(x[2:3].cuda(), q_weight=w.cuda(), eps=1e-6)
        assert bool((b[0, 0] == 0).all())


def test_empty_batch_graph_and_stream():
    D = 64
    w, inv = torch.ones(D, dtype=BF).cuda(), freqs(D).cuda()
    rope = lr.Rope(inv)
    e = torch.empty(0, 3, D, dtype=BF, device="cuda")
    a, _ = lr.lora_qk_norm_rope(e, None, torch.empty(0, dtype=torch.int64, device="cuda"), rope, w)
    assert a.shape == (0, 3, D)
    M = 50
    q, k = rand(1, M, 6, D).cuda(), rand(2, M, 2, D).cuda()
    pos = torch.arange(M).cuda()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    go = lambda: lr.lora_qk_norm_rope(q, k, pos, rope, w, w, q_out=qo, k_out=ko)
    go()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for n in range(4):
        q.copy_(rand(10 + n, M, 6, D))
        k.copy_(rand(20 + n, M, 2, D))
        pos.copy_(torch.arange(M) * (n + 1))
        g.replay()
        got = qo.clone(), ko.clone()
        want = lr.lora_qk_norm_rope(q, k, pos, rope, w, w)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = lr.lora_qk_norm_rope(q, k, pos, rope, w, w, stream=st)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_binding_refuses():
    q, k = rand(1, 4, 3, 64).cuda(), rand(2, 4, 2, 64).cuda()
    pos, rope, w = torch.arange(4).cuda(), lr.Rope(freqs(64).cuda()), torch.ones(64, dtype=BF).cuda()
    good = dict(q=q, k=k, positions=pos, rope=rope, q_weight=w, k_weight=w)
    lr.lora_qk_norm_rope(**good)
    for bad in [dict(q=q[0]), dict(q=q.half()), dict(k=k[:3]), dict(k=k[:, :, :32]), dict(k=k.float()),
                dict(positions=None), dict(positions=pos.int()), dict(positions=pos[:3]), dict(positions=pos.cpu()),
                dict(q_weight=w[:32]), dict(q_weight=w.float()), dict(k_weight=w.cpu()), dict(q=q.cpu()),
                dict(q_out=k), dict(q_out=torch.empty(4, 3, 64, device="cuda")),
                dict(q_out=q, k_out=q[:, :2]), dict(q_out=torch.empty(4, 64, 3, dtype=BF, device="cuda").permute(0, 2, 1)),
                dict(rope=lr.Rope(freqs(66).cuda())), dict(eps=-1.0), dict(eps=float("nan")),
                dict(q_out=q.as_strided(q.shape, (3 * 64, 32, 1))), dict(k_out=q[:, 1:])]:
        with pytest.raises((TypeError, ValueError, lr.LoraError)):
            lr.lora_qk_norm_rope(**dict(good, **bad))
    for bad in [freqs(64), freqs(64).cuda().double(), freqs(64).cuda().view(2, 16)]:
        with pytest.raises((TypeError, ValueError)):
            lr.Rope(bad)

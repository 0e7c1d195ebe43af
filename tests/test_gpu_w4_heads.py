"""The 4-bit adapted projections of query, key and value, and the norm and
rotation of the heads in their output, as one step of a model.

Tolerances.  The layer's as in its own tests (normwise 2e-2 against 64 bits);
the heads' against the 64-bit formula on the bits that the layer wrote: 2^-21
of the two values' magnitudes and one rounding to bf16, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import lora_row_adapter_amd as lr
import w4_ref as R
from gpu_helpers import normwise, say
from test_gpu_w4 import adapter_set, device_slices, device_weight, layer_ref, loud

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
HQ, HK, D, K = 6, 2, 64, 384
DS = (HQ * D, HK * D, HK * D)
RANKS = [16, 8, 4]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the gpu tests need an MI355X")
    torch.cuda.set_device(0)
    lr.load_library()
    yield
    torch.cuda.synchronize()


class Step:
    def __init__(self, M, pools=False, rot=D):
        self.M, self.rot = M, rot
        self.q4 = R.weight(M, sum(DS), K, 64)
        self.W = device_weight(*self.q4, 64)
        self.sets = [adapter_set(i, len(RANKS), 16, K, d, RANKS) for i, d in enumerate(DS)]
        self.scales = np.array([1.0, 0.5, 2.0])
        self.slices = device_slices(self.sets, RANKS, self.scales, DS, K, 16, pools)
        g = torch.Generator().manual_seed(M)
        self.wq, self.wk = (torch.randn(D, generator=g).to(BF).cuda() for _ in range(2))
        inv = torch.tensor([1e4 ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float32)
        self.rope = lr.Rope(inv.cuda(), interleaved=False)
        self.x = torch.empty(M, K, dtype=BF, device="cuda")
        self.ids = torch.empty(M, dtype=torch.int32, device="cuda")
        self.pos = torch.empty(M, dtype=torch.int64, device="cuda")
        self.y = torch.empty(M, sum(DS), dtype=BF, device="cuda")
        self.ws = torch.zeros(lr.workspace_bytes_sliced_w4(M, K, self.slices), dtype=torch.uint8, device="cuda")

    def inputs(self, seed):
        """A padded batch: some rows past the last sequence, some of no adapter."""
        rng = np.random.default_rng(seed)
        ids, pos = rng.integers(-1, len(RANKS), self.M), rng.integers(0, 100000, self.M)
        pad = rng.random(self.M) < 0.2
        pad[0] = False
        ids[pad], pos[pad] = -1, -1
        self.x.copy_(loud(seed, self.M, K))
        self.ids.copy_(torch.from_numpy(ids.astype(np.int32)))
        self.pos.copy_(torch.from_numpy(pos))
        return ids, pos

    def project(self, y=None, stream=None):
        return lr.lora_linear_sliced_w4(self.x, self.W, self.slices, self.ids, y=self.y if y is None else y,
                                        workspace=self.ws, stream=stream)

    def heads(self, y):
        q, k, v = y.split(DS, dim=1)
        return q.view(-1, HQ, D), k.view(-1, HK, D), v

    def run(self, stream=None):
        self.project(stream=stream)
        q, k, _ = self.heads(self.y)
        lr.lora_qk_norm_rope(q, k, positions=self.pos, rope=self.rope, q_weight=self.wq, k_weight=self.wk, eps=1e-6,
                             q_out=q, k_out=k, stream=stream)
        return self.y

    def check(self, y, projected, pos):
        angle = pos.astype(np.float64)[:, None] * self.rope.inv_freq.cpu().double().numpy()
        for got, was, w in zip(self.heads(y)[:2], self.heads(projected)[:2], (self.wq, self.wk)):
            got, was = got.cpu().double().numpy(), was.cpu().double().numpy()
            want, mag = R.heads(was, w.cpu().double().numpy(), 1e-6, np.cos(angle), np.sin(angle), self.rot, False)
            live = pos >= 0
            assert (np.abs(got - want) <= 2.0 ** -21 * mag + 2.0 ** -8 * np.abs(want))[live].all()
            assert (got == was)[~live].all()
        assert torch.equal(self.heads(y)[2], self.heads(projected)[2])


@pytest.mark.parametrize("pools", [False, True])
@pytest.mark.parametrize("M,rot", [(1, 64), (7, 64), (32, 32), (40, 64), (300, 64)])
def test_step(M, rot, pools):
    say("w4 projections and heads M=%d rot=%d pools=%d" % (M, rot, pools))
    st = Step(M, pools, rot)
    ids, pos = st.inputs(5)
    projected = st.project().clone()
    want = layer_ref(st.x.cpu(), R.dequant(*st.q4, 64), DS, st.sets, RANKS, st.scales, ids)
    assert normwise(projected.cpu().double().numpy(), want) <= 2e-2
    st.check(st.run(), projected, pos)


@pytest.mark.parametrize("M", [1, 20, 130])
def test_step_captured(M):
    st = Step(M)
    st.inputs(0)
    st.run()  # the first call on a device is made outside a capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.run()
    for n in range(5):
        _, pos = st.inputs(20 + n)
        g.replay()
        got = st.y.clone()
        projected = st.project(y=torch.empty_like(st.y))
        st.check(got, projected, pos)
        torch.cuda.synchronize()
        assert torch.equal(st.run(), got)


def test_two_steps_at_once():
    """Two batches on two streams, each with a workspace of its own."""
    steps = [Step(17), Step(90)]
    for n, st in enumerate(steps):
        st.inputs(n)
    want = [st.run().clone() for st in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(20):
        for st, s in zip(steps, streams):
            st.run(stream=s)
    torch.cuda.synchronize()
    for st, w in zip(steps, want):
        assert torch.equal(st.y, w)

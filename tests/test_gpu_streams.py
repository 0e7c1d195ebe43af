"""Calls that are given a stream while the current one is busy: what they make
belongs to that stream, and their results are those of the current stream."""
import pytest
import torch

import lora_row_adapter_amd as lr
from lora_row_adapter_amd import workloads as wl
from gpu_helpers import say

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the gpu tests need an MI355X")
    torch.cuda.set_device(0)
    lr.load_library()
    yield
    torch.cuda.synchronize()


def pool_stream(t):
    """The stream in whose pool a tensor's memory is."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment holds the tensor")


def check_beside_busy(calls):
    """Each call on the current stream, then on another one while the current
    one is busy and keeps writing what it frees."""
    want = [c(None) for c in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for c, w in zip(calls, want):
        a = torch.ones(4096, 4096, device="cuda")
        for _ in range(8):
            a = a @ a * 2.0 ** -12
        got = c(side)
        for _ in range(4):  # where a dropped workspace's memory would come back
            torch.full((1 << 22,), 0xA5, dtype=torch.uint8, device="cuda")
        side.synchronize()
        for g, e in zip(got, w):
            assert torch.equal(g, e)
            assert pool_stream(g) == side.cuda_stream
        torch.cuda.synchronize()


def test_microscaled_calls_beside_a_busy_stream():
    g = torch.Generator().manual_seed(1)
    w = wl.custom(seed=3, M=200, k=1024, d=640, ranks=[8, 32, 64], max_rank=64, none_frac=0.1)
    p = w.proj("out")
    A, Bm = wl.slots(w, p)
    ad = lr.Adapters.slots(A.cuda(), Bm.cuda(), torch.from_numpy(w.ranks).cuda())
    slices = [lr.Slice(640, ad, torch.from_numpy(w.scales).cuda())]
    x, ids = w.x.cuda(), torch.from_numpy(w.ids).cuda()
    W = lr.lora_mx_quantize(p.W.cuda(), lr.MX_FP4)
    q = lr.lora_mx_quantize(x)
    norm = lr.Norm((1 + 0.1 * torch.randn(1024, generator=g)).to(BF).cuda(), 1e-5)
    nb = 1024 // 32

    def quantize(s):
        m = lr.lora_mx_quantize(x, stream=s)
        return m.q, m.scales[:, :nb]

    say("microscaled calls beside a busy stream")
    check_beside_busy([
        quantize,
        lambda s: [lr.lora_mx_dequantize(q, stream=s)],
        lambda s: [lr.lora_rmsnorm(x, norm, stream=s)],
        lambda s: [lr.lora_gemm_mx(q, W, stream=s)],
        lambda s: [lr.lora_linear_sliced_mx(x, W, slices, ids, norm=norm, stream=s)],
        lambda s: [lr.lora_linear_sliced_mx(x, W, slices, ids, x_format=lr.MX_FP4, stream=s)],
    ])


def test_dense_and_quantised_calls_beside_a_busy_stream():
    w = wl.custom(seed=4, M=200, k=1024, d=640, ranks=[8, 32, 64], max_rank=64, none_frac=0.1)
    p = w.proj("out")
    A, Bm = wl.slots(w, p)
    ad = lr.Adapters.slots(A.cuda(), Bm.cuda(), torch.from_numpy(w.ranks).cuda())
    scales = torch.from_numpy(w.scales).cuda()
    slices = [lr.Slice(640, ad, scales)]
    x, ids, W = w.x.cuda(), torch.from_numpy(w.ids).cuda(), p.W.cuda()
    g = torch.Generator().manual_seed(5)
    Q = lr.QWeight(lr.W_INT8, torch.randint(-127, 128, (640, 1024), generator=g, dtype=torch.int8).cuda(),
                   torch.full((640,), 0.01, device="cuda"), 1024)
    say("dense and quantised calls beside a busy stream")
    check_beside_busy([
        lambda s: [lr.lora_gemm(x, W, stream=s)],
        lambda s: [lr.lora_linear(x, W, ad, ids, scales, stream=s)],
        lambda s: [lr.lora_linear_sliced(x, W, slices, ids, stream=s)],
        lambda s: [lr.lora_gemm_q(x, Q, stream=s)],
        lambda s: [lr.lora_linear_sliced_q(x, Q, slices, ids, stream=s)],
        lambda s: [lr.lora_merge(W, ad, 1, scales, stream=s)],
    ])

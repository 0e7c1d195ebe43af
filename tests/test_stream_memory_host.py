"""What a call makes when it is given a stream is made under that stream, on a
recorded allocator and a library that does nothing (no GPU)."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import lora_row_adapter_amd as lr
from lora_row_adapter_amd import _binding as B

BF = torch.bfloat16
DEV = torch.device("cuda", 0)


class Tensor:
    """As much of a device tensor as the binding looks at."""

    is_cuda, device = True, DEV

    def __init__(self, shape, dtype=BF):
        self.shape, self.dtype = torch.Size((shape,) if isinstance(shape, int) else shape), dtype

    def stride(self, i=None):
        st = tuple(self.shape[j + 1:].numel() for j in range(len(self.shape)))
        return st if i is None else st[i]

    def data_ptr(self):
        return 4096

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True


class Library:
    """Every entry point succeeds; the workspace sizes are 512."""

    def __getattr__(self, name):
        return lambda *a: 512 if "workspace_bytes" in name else 0


@pytest.fixture
def made(monkeypatch):
    """(function, stream) of each tensor that is made, the stream that is
    current at the time."""
    out, current = [], ["current"]

    @contextlib.contextmanager
    def under(stream):
        current.append(stream.name)
        yield
        current.pop()

    def maker(name):
        def make(shape, dtype=torch.float32, device=None):
            out.append((name, current[-1]))
            return Tensor(shape, dtype)
        return make

    monkeypatch.setattr(B, "_lib", Library())
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(B, "_slice_array", lambda slices: None)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: SimpleNamespace(cuda_stream=0))
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, maker(name))
    return out


SIDE = SimpleNamespace(name="side", cuda_stream=7)
SLICES = [SimpleNamespace(d=8, adapters=SimpleNamespace(kind=B.KIND_POOL))]


def mx(rows, fmt):
    m = B.MX.__new__(B.MX)
    m._set(fmt, 64, rows, DEV, 4096, 64, 4096, 4)
    return m


# calls and how many tensors each one makes
MX_CALLS = {
    "quantize": (1, lambda s: lr.lora_mx_quantize(Tensor((4, 64)), stream=s)),
    "dequantize": (1, lambda s: lr.lora_mx_dequantize(mx(4, lr.MX_FP8), stream=s)),
    "rmsnorm": (1, lambda s: lr.lora_rmsnorm(Tensor((4, 64)), lr.Norm(Tensor(64)), stream=s)),
    "gemm": (1, lambda s: lr.lora_gemm_mx(mx(4, lr.MX_FP8), mx(8, lr.MX_FP4), stream=s)),
    "layer": (2, lambda s: lr.lora_linear_sliced_mx(Tensor((4, 64)), mx(8, lr.MX_FP4), SLICES,
                                                    Tensor(4, torch.int32), stream=s)),
}


@pytest.mark.parametrize("name", MX_CALLS)
def test_microscaled_calls_make_their_tensors_under_their_stream(name, made):
    n, call = MX_CALLS[name]
    call(SIDE)
    assert [s for _, s in made] == ["side"] * n
    made.clear()
    call(None)
    assert [s for _, s in made] == ["current"] * n


def test_microscaled_layer_fills_no_workspace(made):
    MX_CALLS["layer"][1](None)
    assert [f for f, _ in made] == ["empty", "empty"]


def adapters():
    return SimpleNamespace(kind=B.KIND_POOL, ref=lambda: None)


def qweight():
    return SimpleNamespace(d=8, ref=lambda: None)


def x():
    return Tensor((4, 64))


def ids():
    return Tensor(4, torch.int32)


CALLS = {
    "gemm": (2, lambda s: lr.lora_gemm(x(), Tensor((8, 64)), stream=s)),
    "linear": (2, lambda s: lr.lora_linear(x(), Tensor((8, 64)), adapters(), ids(), Tensor(4, torch.float32), stream=s)),
    "sliced": (2, lambda s: lr.lora_linear_sliced(x(), Tensor((8, 64)), SLICES, ids(), stream=s)),
    "gemm_q": (1, lambda s: lr.lora_gemm_q(x(), qweight(), stream=s)),
    "sliced_q": (2, lambda s: lr.lora_linear_sliced_q(x(), qweight(), SLICES, ids(), stream=s)),
    "merge": (1, lambda s: lr.lora_merge(Tensor((8, 64)), adapters(), 0, Tensor(4, torch.float32), stream=s)),
    "translate": (1, lambda s: lr.lora_translate(adapters(), ids(), Tensor(4, torch.int64), stream=s)),
}


@pytest.mark.parametrize("name", CALLS)
def test_calls_make_their_tensors_under_their_stream(name, made):
    n, call = CALLS[name]
    call(SIDE)
    assert [s for _, s in made] == ["side"] * n
    made.clear()
    call(None)
    assert [s for _, s in made] == ["current"] * n


@pytest.mark.parametrize("name", ["gemm", "linear", "sliced", "sliced_q"])
def test_dense_workspaces_are_zero_filled(name, made):
    """The split-K base product counts expired waits from 0 on."""
    CALLS[name][1](None)
    assert [f for f, _ in made] == ["empty", "zeros"]


def test_a_pool_is_made_under_its_stream(made, monkeypatch):
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: Tensor(
        shape, dtype) if shape == () else real(shape, dtype=dtype, device=device))
    monkeypatch.setattr(Tensor, "element_size", lambda self: 2, raising=False)
    lr.AdapterPool(4, 1024, 2, 2, 8, 64, 64, device=DEV, stream=SIDE)
    assert [s for _, s in made] == ["side"] * 3

"""Which kernels the sizes of a 4-bit product take, as the library's host hooks
name them; no GPU."""
import ctypes

import pytest

import lora_row_adapter_amd as lr

WEIGHTS = [  # d, k
    (9216, 8192), (4096, 4096), (5120, 5120), (1024, 4096), (1024, 1024), (1024, 8192), (512, 2048), (4096, 512),
    (8192, 1024), (28672, 8192), (14336, 4096), (8192, 28672), (4096, 14336), (10240, 8192), (300, 1000), (33, 1032),
    (2050, 2056), (65536, 4096), (1 << 21, 128),
]


def shape(M, k, d, group):
    out = (ctypes.c_int32 * 3)()
    i = lr.load_library().lora_test_gemm_w4_shape(M, k, d, group, out)
    assert i >= 0
    return (i,) + tuple(out)


@pytest.mark.parametrize("group", [32, 64, 128, 512])
@pytest.mark.parametrize("d,k", WEIGHTS)
def test_weights_are_rounded_from_one_number_of_rows_on(d, k, group):
    """A row's sums do not go back and forth between exact and rounded weights
    as more rows join its batch."""
    rounds = [shape(M, k, d, group)[3] for M in list(range(1, 1400)) + list(range(1400, 20000, 37)) + [1 << 18, 1 << 30]]
    assert rounds[:32] == [0] * 32
    assert rounds == sorted(rounds)


def product(M, k, d, group):
    out = (ctypes.c_int32 * 3)()
    i = lr.load_library().lora_test_linear_w4_shape(M, k, d, group, out)
    assert i >= 0
    return (i,) + tuple(out)


def test_layer_hook():
    """It names lora_gemm_w4's shapes from 33 rows on, and refuses what is no layer."""
    for M, k, d, group in [(33, 1024, 300, 32), (512, 8192, 9216, 128), (8192, 4096, 4096, 64), (20, 128, 1 << 21, 32)]:
        few = 7  # shapes that add the adapters' part
        assert product(M, k, d, group)[0] == few + shape(M, k, d, group)[0]
        assert product(M, k, d, group)[1:3] == shape(M, k, d, group)[1:3]
    assert product(32, 1024, 300, 32)[0] < 7 and product(1, 8192, 9216, 128)[3] == 1
    out = (ctypes.c_int32 * 3)()
    f = lr.load_library().lora_test_linear_w4_shape
    for M, k, d, group, o in [(0, 64, 64, 32, out), (8193, 64, 64, 32, out), (1, 0, 64, 32, out), (1, 60, 64, 32, out),
                              (1, 64, 0, 32, out), (1, 64, 64, 31, out), (1, 64, 64, 32, None)]:
        assert f(M, k, d, group, o) == -1
    with pytest.raises(lr.LoraError):
        lr.test_linear_w4_shape(8193, 64, 64, 32)


def test_every_shape_is_taken_with_every_group():
    """Of the layer's products for few rows and of lora_gemm_w4's: none stands in
    its table for nothing, and the GPU tests' sizes reach them all."""
    found = layer_sizes()
    assert sorted({(i, g) for i, g in found}) == [(i, g) for i in range(7 + 14) for g in (32, 64, 128)]


_SIZES = {}


def layer_sizes():
    """(shape, group) -> the cheapest (M, k, d) of a list that takes it, k past
    every ring of stages, the plan in its launch and more than one tile of columns
    where that can be."""
    if not _SIZES:
        ds = [16, 33, 300, 305, 353, 424, 490, 547, 657, 760, 788, 911, 1000, 1134, 1176, 1959, 3914, 5432, 7820, 8411, 12555]
        cost = {}
        for M in (9, 30, 40, 200, 300, 700, 1000, 1500, 2100, 4097):
            for k in (136, 264, 1032, 2056, 4104, 8200, 12680):
                for d in ds:
                    if M * d > 3e7 or d * k > 1e8:
                        continue
                    for group in (32, 64, 128):
                        i, _, _, beside = product(M, k, d, group)
                        c = (k < (2056 if M <= 32 else 1032), not beside, d < 300, d * k + M * (4 * d + k))
                        if (i, group) not in cost or c < cost[i, group]:
                            cost[i, group] = c
                            _SIZES[i, group] = (M, k, d)
    return _SIZES

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

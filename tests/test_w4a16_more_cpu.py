"""Limits of the W4A16 linear layer, on the CPU: refused before any CUDA work, so the addresses are made up and never
followed."""
import ctypes

import pytest

import w4a16_mixture_experts_gb300 as moe
from w4a16_mixture_experts_gb300 import _build

UNSUPPORTED = 2
A = 0x10000   # a 16-byte aligned address


@pytest.fixture(scope="module")
def L():
    _build.build()
    return moe.lib()


@pytest.mark.parametrize("N", [2 ** 31 - 1, 2 ** 31 - 15, 2 ** 31 - 16, 2 ** 31 - 17, 2 ** 31 - 255])
def test_rows_whose_indexes_pass_32_bits_are_refused(L, N):
    # a CTA takes 128 rows: rows up to the next multiple of 128 are counted in 32 bits
    n = ctypes.c_size_t(0)
    assert L.moe_w4a16_workspace_size(1, N, 128, ctypes.byref(n)) == UNSUPPORTED
    for T in (0, 1):
        assert L.moe_w4a16_linear(A, A, A, A, T, N, 128, A, 1 << 40, None) == UNSUPPORTED


def test_the_largest_number_of_rows(L):
    N = 2 ** 31 - 256
    assert moe.moe_w4a16_workspace_size(1, N, 128) >= 256
    # the kernel's indexes at that size: 16 rows a warp, 8 warps a CTA, row and row + 8 a lane
    blocks = (N + 15) // 16
    last = (blocks + 7) // 8 * 8 - 1
    assert N + 15 < 2 ** 31 and last * 16 + 7 + 8 < 2 ** 31


def test_a_workspace_for_the_largest_batch_does_for_smaller_ones(L):
    for N, K in [(5120, 2560), (320, 10240), (2560, 640), (17, 65536)]:
        sizes = [moe.moe_w4a16_workspace_size(T, N, K) for T in (0, 1, 2, 4, 8, 9, 16, 40, 64, 100, 128, 129, 500, 4096, 1 << 20)]
        assert sizes == sorted(sizes)

"""Refusals of the W4A16 linear layer, on the CPU: every one is answered before any CUDA work, so the addresses
are made up and never followed."""
import ctypes

import pytest
import torch

import w4a16_mixture_experts_gb300 as moe
from w4a16_mixture_experts_gb300 import _build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = 0x10000   # a 16-byte aligned address
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    _build.build()
    return moe.lib()


def _linear(L, **over):
    v = dict(x=A, w=A, s=A, y=A, T=0, N=64, K=256, ws=A, n=BIG, stream=None)
    v.update(over)
    return L.moe_w4a16_linear(*v.values())


@pytest.mark.parametrize("over,status", [
    (dict(), OK), (dict(x=None, y=None), OK), (dict(T=4, N=0), OK), (dict(T=4, N=0, w=None, s=None, y=None), OK),
    (dict(T=-1), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID), (dict(K=-128), INVALID),
    (dict(K=64), UNSUPPORTED), (dict(K=192), UNSUPPORTED), (dict(K=65536 + 128), UNSUPPORTED), (dict(T=(1 << 20) + 1), UNSUPPORTED),
    (dict(T=1, x=None), INVALID), (dict(T=1, w=None), INVALID), (dict(T=1, s=None), INVALID), (dict(T=1, y=None), INVALID),
    (dict(T=1, x=A + 2), INVALID), (dict(T=1, w=A + 4), INVALID), (dict(T=1, s=A + 2), INVALID), (dict(T=1, y=A + 8), INVALID),
    (dict(ws=None), INVALID), (dict(ws=A + 8), INVALID), (dict(n=255), WORKSPACE), (dict(T=1, n=0), WORKSPACE),
])
def test_linear_refusals(L, over, status):
    assert _linear(L, **over) == status


def test_workspace_size(L):
    assert moe.moe_w4a16_workspace_size(0, 64, 128) == 256
    for T, N, K in [(1, 1, 128), (8, 248320, 2560), (9, 17, 65536), (1 << 20, 100, 128)]:
        assert moe.moe_w4a16_workspace_size(T, N, K) >= 256
    n = ctypes.c_size_t(0)
    assert L.moe_w4a16_workspace_size(1, 64, 128, None) == INVALID
    for T, N, K, status in [(-1, 64, 128, INVALID), (1, -1, 128, INVALID), (1, 64, 0, INVALID), (1, 64, 100, UNSUPPORTED),
                            (1, 64, 1 << 17, UNSUPPORTED), (1 << 21, 64, 128, UNSUPPORTED)]:
        assert L.moe_w4a16_workspace_size(T, N, K, ctypes.byref(n)) == status


def test_the_workspace_size_grows_with_the_batch_only_where_results_are_joined(L):
    # a workspace for the largest batch of a server must do for its smaller ones
    for N, K in [(5120, 2560), (320, 10240), (2560, 640), (17, 65536)]:
        sizes = [moe.moe_w4a16_workspace_size(T, N, K) for T in (1, 2, 4, 8, 9, 16, 40, 64, 100, 128, 129, 500, 4096)]
        assert all(b < 1 << 30 for b in sizes)


def test_the_binding_checks_its_tensors(L):
    x, w, s = torch.zeros(2, 256, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.int32), torch.zeros(8, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be"):      # not on a GPU
        moe.moe_w4a16_linear(x, w, s)
    with pytest.raises(TypeError, match="x must be"):
        moe.moe_w4a16_linear([1], w, s)

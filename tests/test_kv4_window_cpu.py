"""Refusals of attention with a window, on the CPU: every one is answered before any CUDA work, so the addresses are
made up and never followed."""
import pytest
import torch

import w4a16_mixture_experts_gb300 as moe
from w4a16_mixture_experts_gb300 import _build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = 0x10000   # a 16-byte aligned address


@pytest.fixture(scope="module")
def L():
    _build.build()
    return moe.lib()


def _cache(**over):
    v = dict(k_codes=A, k_scales=A, v_codes=A, v_scales=A, n_pages=8, Hkv=2, page_size=16, D=128)
    v.update(over)
    return moe.moe_kv4_cache(*v.values())


def _attend(L, **over):
    rows = moe.moe_strides(4 * 128, 128)
    v = dict(q=A, qs=rows, c=_cache(), table=A, max_pages=4, lens=A, cu=A, B=2, T=0, Hq=4, max_q=2, scale=0.1, window=10, sinks=2, out=A,
             os=rows, lse=None, ws=A, n=1 << 30, stream=None)
    v.update(over)
    return L.moe_kv4_attention_window(*v.values())


@pytest.mark.parametrize("over,status", [
    (dict(), OK), (dict(window=1, sinks=0), OK), (dict(window=2 ** 31 - 1, sinks=2 ** 31 - 1), OK),
    (dict(window=0), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(window=-2 ** 31), INVALID),
    (dict(T=4, q=None), INVALID), (dict(T=4, out=A + 8), INVALID), (dict(T=4, lens=None), INVALID), (dict(T=4, table=None), INVALID),
    (dict(T=4, cu=None), INVALID), (dict(T=4, lse=A + 2), INVALID), (dict(T=-1), INVALID), (dict(B=4097), UNSUPPORTED), (dict(Hq=5), INVALID),
    (dict(Hq=66), UNSUPPORTED), (dict(max_pages=1 << 27), UNSUPPORTED), (dict(scale=float("nan")), INVALID), (dict(ws=None), INVALID),
    (dict(n=255), WORKSPACE), (dict(c=_cache(D=96)), UNSUPPORTED), (dict(c=_cache(page_size=24)), UNSUPPORTED),
])
def test_window_refusals(L, over, status):
    assert _attend(L, **over) == status


def test_the_binding_checks_its_tensors(L):
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):   # not on a GPU
        moe.moe_kv4_attention_window(x, moe.kv4_cache(2, 2, 16, 128, device="cpu"), torch.zeros(4, 1, dtype=torch.int32),
                                     torch.ones(4, dtype=torch.int32), 10)

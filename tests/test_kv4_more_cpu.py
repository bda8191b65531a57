"""The attention block's calls where there is nothing to do, and what the binding checks before them: on the CPU."""
import pytest

import w4a16_mixture_experts_gb300 as moe
from w4a16_mixture_experts_gb300 import _build
from test_kv4_cpu import OK, WORKSPACE, _attend


@pytest.fixture(scope="module")
def L():
    _build.build()
    return moe.lib()


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (32, 8, 64)])
def test_a_batch_of_no_tokens_needs_what_its_size_says(L, Hq, Hkv, D):
    n = moe.moe_kv4_workspace_size(0, Hq, Hkv, D)
    c = moe.moe_kv4_cache(0x10000, 0x10000, 0x10000, 0x10000, 8, Hkv, 16, D)
    for b, cu in ((0, None), (3, 0x10000)):
        assert _attend(L, c=c, Hq=Hq, T=0, B=b, cu=cu, q=None, out=None, n=n) == OK
        assert _attend(L, c=c, Hq=Hq, T=0, B=b, cu=cu, q=None, out=None, n=n - 1) == WORKSPACE
    # what the binding makes for such a batch
    assert moe.kv4_workspace(0, Hq, Hkv, D, device="cpu").numel() == n == 256

"""Refusals of the verification of drafts, on the CPU: every one is answered before any CUDA work, so the addresses
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


def _verify(L, **over):
    v = dict(logits=A, ls=512, draft=A, ds=512, drafts=A, cu=A, temperature=A, uniform=A, noise=A, ns=512, B=0, T=6, V=500, tokens=A, accepted=A,
             ws=A, n=BIG, stream=None)
    v.update(over)
    return L.moe_verify_drafts(*v.values())


@pytest.mark.parametrize("over,status", [
    (dict(), OK), (dict(T=0, logits=None, draft=None, drafts=None, uniform=None, tokens=None, noise=None, cu=None, accepted=None), OK),
    (dict(draft=None, ds=3), OK), (dict(temperature=None), OK), (dict(ls=504), OK), (dict(T=1, ls=0, ds=0), OK),
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(V=0), INVALID), (dict(V=-5), INVALID),
    (dict(V=(1 << 20) + 1), UNSUPPORTED), (dict(T=65537), UNSUPPORTED), (dict(B=4097), UNSUPPORTED),
    (dict(ls=500), INVALID), (dict(ls=496), INVALID), (dict(ds=508), INVALID), (dict(ds=-512), INVALID), (dict(ls=0), INVALID),
    (dict(B=2, ns=502), INVALID), (dict(B=2, ns=496), INVALID), (dict(ns=-4), INVALID),
    (dict(logits=None), INVALID), (dict(logits=A + 8), INVALID), (dict(draft=A + 2), INVALID), (dict(B=2, noise=None), INVALID),
    (dict(B=2, noise=A + 4), INVALID), (dict(drafts=None), INVALID), (dict(drafts=A + 1), INVALID), (dict(uniform=A + 2), INVALID),
    (dict(uniform=None), INVALID), (dict(tokens=None), INVALID), (dict(tokens=A + 2), INVALID), (dict(B=2, cu=None), INVALID),
    (dict(B=2, accepted=None), INVALID), (dict(B=2, cu=A + 2), INVALID), (dict(temperature=A + 2), INVALID),
    (dict(ws=None), INVALID), (dict(ws=A + 8), INVALID), (dict(n=256), WORKSPACE),
])
def test_verify_refusals(L, over, status):
    assert _verify(L, **over) == status


def test_workspace_size(L):
    n = ctypes.c_size_t(0)
    assert L.moe_verify_workspace_size(1, 1, 1, None) == INVALID
    for B, T, V, status in [(0, 0, 1, OK), (4096, 65536, 1 << 20, OK), (-1, 1, 1, INVALID), (1, -1, 1, INVALID), (1, 1, 0, INVALID),
                            (4097, 1, 1, UNSUPPORTED), (1, 65537, 1, UNSUPPORTED), (1, 1, (1 << 20) + 1, UNSUPPORTED)]:
        assert L.moe_verify_workspace_size(B, T, V, ctypes.byref(n)) == status
    sizes = [moe.moe_verify_workspace_size(*d) for d in [(1, 4, 1000), (8, 40, 1000), (8, 40, 250000), (64, 500, 250000)]]
    assert sizes == sorted(sizes)


def test_the_binding_checks_its_tensors(L):
    l, i, f = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    with pytest.raises(ValueError, match="logits must be"):   # not on a GPU
        moe.moe_verify_drafts(l, i, i, f, torch.zeros(3, 64))
    with pytest.raises(TypeError, match="logits must be"):
        moe.moe_verify_drafts(None, i, i, f, torch.zeros(3, 64))

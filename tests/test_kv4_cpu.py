"""Refusals of the attention block's calls, on the CPU: every one is answered before any CUDA work, so the
addresses are made up and never followed."""
import ctypes

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


def _rows(T=4, heads=2, D=128):
    return moe.moe_strides(heads * D, D)


def _cache(**over):
    v = dict(k_codes=A, k_scales=A, v_codes=A, v_scales=A, n_pages=8, Hkv=2, page_size=16, D=128)
    v.update(over)
    return moe.moe_kv4_cache(*v.values())


def _rope(L, **over):
    v = dict(q=A, qs=_rows(heads=4), k=A, ks=_rows(), qw=None, kw=None, pos=A, freq=A, rot=128, inter=0, eps=1e-6, qo=A,
             qos=_rows(heads=4), ko=A, kos=_rows(), T=4, Hq=4, Hkv=2, D=128, stream=None)
    v.update(over)
    return L.moe_qk_norm_rope(*v.values())


@pytest.mark.parametrize("over,status", [
    (dict(T=0), OK), (dict(T=0, q=None, k=None, qo=None, ko=None), OK), (dict(Hq=0, Hkv=0), OK),
    (dict(T=-1), INVALID), (dict(q=None), INVALID), (dict(ko=None), INVALID), (dict(q=A + 2), INVALID),
    (dict(qs=moe.moe_strides(511, 128)), INVALID), (dict(ks=moe.moe_strides(-256, 128)), INVALID),
    (dict(qos=moe.moe_strides(0, 128)), INVALID), (dict(kos=moe.moe_strides(256, 0)), INVALID),
    (dict(qos=moe.moe_strides(256, 128)), INVALID),
    (dict(rot=130), INVALID), (dict(rot=-16), INVALID), (dict(rot=24), UNSUPPORTED), (dict(pos=None), INVALID),
    (dict(freq=A + 2), INVALID), (dict(inter=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(D=96), INVALID), (dict(D=96, rot=96), UNSUPPORTED), (dict(D=512), UNSUPPORTED), (dict(qw=A + 8), INVALID),
    (dict(T=(1 << 20) + 1), UNSUPPORTED), (dict(Hq=-1), INVALID), (dict(Hkv=1025), UNSUPPORTED),
])
def test_norm_rope_refusals(L, over, status):
    assert _rope(L, **over) == status


def _append(L, c=None, **over):
    v = dict(k=A, ks=_rows(), v=A, vs=_rows(), slots=A, T=4, c=c or _cache(), ws=A, n=256, stream=None)
    v.update(over)
    return L.moe_kv4_append(*v.values())


CACHES = [(dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
          (dict(page_size=2048), UNSUPPORTED), (dict(n_pages=0), INVALID), (dict(Hkv=0), INVALID), (dict(k_codes=None), INVALID),
          (dict(v_scales=A + 2), INVALID), (dict(n_pages=1 << 27), UNSUPPORTED), (dict(Hkv=2000), UNSUPPORTED),
          (dict(n_pages=1 << 20, page_size=1024, Hkv=4), UNSUPPORTED)]


@pytest.mark.parametrize("over,status", CACHES)
def test_cache_refusals(L, over, status):
    assert _append(L, c=_cache(**over)) == status
    assert L.moe_kv4_read(A, 4, _cache(**over), A, A, A, 256, None) == status
    assert _attend(L, c=_cache(**over)) == status


@pytest.mark.parametrize("over,status", [
    (dict(T=0), OK), (dict(T=0, k=None, v=None, slots=None), OK), (dict(T=-1), INVALID), (dict(k=None), INVALID), (dict(v=A + 4), INVALID),
    (dict(slots=None), INVALID), (dict(slots=A + 1), INVALID), (dict(ws=None), INVALID), (dict(n=255), WORKSPACE),
    (dict(ks=moe.moe_strides(256, 127)), INVALID), (dict(T=(1 << 20) + 1), UNSUPPORTED),
])
def test_append_refusals(L, over, status):
    assert _append(L, **over) == status


@pytest.mark.parametrize("args,status", [
    ((None, 0, A, A, A, 256), OK), ((A, -1, A, A, A, 256), INVALID), ((None, 4, A, A, A, 256), INVALID), ((A, 4, None, A, A, 256), INVALID),
    ((A, 4, A, A + 8, A, 256), INVALID), ((A, 4, A, A, None, 256), INVALID), ((A, 4, A, A, A, 0), WORKSPACE),
])
def test_read_refusals(L, args, status):
    assert L.moe_kv4_read(args[0], args[1], _cache(), args[2], args[3], args[4], args[5], None) == status


def _attend(L, **over):
    v = dict(q=A, qs=_rows(heads=4), c=_cache(), table=A, max_pages=4, lens=A, cu=A, B=2, T=4, Hq=4, max_q=2, scale=0.1, out=A,
             os=_rows(heads=4), lse=None, ws=A, n=1 << 30, stream=None)
    v.update(over)
    return L.moe_kv4_attention(*v.values())


@pytest.mark.parametrize("over,status", [
    (dict(T=0), OK), (dict(T=0, B=0, q=None, out=None, lens=None, cu=None, table=None), OK), (dict(T=-1), INVALID),
    (dict(B=-1), INVALID), (dict(B=0), INVALID), (dict(cu=None), INVALID), (dict(B=4097), UNSUPPORTED), (dict(Hq=5), INVALID),
    (dict(Hq=66), UNSUPPORTED), (dict(Hq=0), INVALID), (dict(max_pages=-1), INVALID), (dict(max_pages=1 << 27), UNSUPPORTED),
    (dict(max_q=-1), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID), (dict(q=None), INVALID),
    (dict(out=A + 8), INVALID), (dict(os=moe.moe_strides(0, 128)), INVALID), (dict(qs=moe.moe_strides(4, 128)), INVALID),
    (dict(lens=None), INVALID), (dict(table=None), INVALID), (dict(lse=A + 2), INVALID), (dict(ws=None), INVALID), (dict(ws=A + 8), INVALID),
    (dict(n=255), WORKSPACE),
])
def test_attention_refusals(L, over, status):
    assert _attend(L, **over) == status


def test_workspace_size():
    n = moe.moe_kv4_workspace_size(1, 32, 4, 128)
    assert n >= 256 and n % 256 == 0
    assert moe.moe_kv4_workspace_size(4096, 32, 4, 128) >= n
    for dims, status in (((-1, 4, 2, 128), INVALID), ((1, 5, 2, 128), INVALID), ((1, 4, 0, 128), INVALID), ((1, 4, 2, 96), UNSUPPORTED),
                         ((1, 66, 2, 128), UNSUPPORTED), (((1 << 20) + 1, 4, 2, 128), UNSUPPORTED)):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_kv4_workspace_size(*dims)
        assert e.value.status == status
    assert moe.lib().moe_kv4_workspace_size(1, 4, 2, 128, ctypes.POINTER(ctypes.c_size_t)()) == INVALID


def test_binding_refuses_other_types_and_shapes():
    """The binding's checks come before the library's."""
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        moe.moe_qk_norm_rope(None, x, None, None)
    with pytest.raises(ValueError):
        moe.moe_qk_norm_rope(x.float(), x, None, None)
    with pytest.raises(ValueError):
        moe.moe_qk_norm_rope(x, x, None, None)                       # not on the GPU
    with pytest.raises(ValueError):
        moe.moe_qk_norm_rope(x[..., ::2], x, None, None)
    cache = moe.kv4_cache(2, 2, 16, 128, device="cpu")
    assert cache.k_codes.shape == (2, 2, 16, 16) and cache.v_scales.shape == (2, 2, 16)
    assert (((cache.k_codes >> 12) & 15) == 8).all() and (cache.k_scales == 0).all()
    with pytest.raises(ValueError):
        moe.moe_kv4_append(x, x, torch.zeros(4, dtype=torch.int32), cache)
    with pytest.raises(ValueError):
        moe.moe_kv4_read(torch.zeros(4, dtype=torch.int32), cache)
    with pytest.raises(ValueError):
        moe.moe_kv4_attention(x, cache, torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, dtype=torch.int32))

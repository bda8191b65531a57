"""The attention block's calls where there is nothing to do, and what the binding checks before them: on the CPU."""
import pytest
import torch

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


class _OnGpu(torch.Tensor):
    """A tensor that says it is on the GPU: for checks that come before anything is launched."""
    is_cuda = property(lambda self: True)


def _fake_cache(n=4, h=2, p=16, w=16):
    on = lambda *s, dtype: torch.zeros(*s, dtype=dtype).as_subclass(_OnGpu)  # noqa: E731
    return moe.Kv4Cache(on(n, h, p, w, dtype=torch.int32), on(n, h, p, dtype=torch.bfloat16),
                        on(n, h, p, w, dtype=torch.int32), on(n, h, p, dtype=torch.bfloat16))


def test_a_cache_is_checked_at_every_call():
    """A tensor at the same address with another shape, stride or type is another tensor."""
    cache = _fake_cache()
    c, h, d = cache.c()
    assert (c.n_pages, c.Hkv, c.page_size, c.D, h, d) == (4, 2, 16, 128, 2, 128) and c.v_codes == cache.v_codes.data_ptr()
    for name, others in (("k_scales", (lambda t: t[:2], lambda t: t.transpose(0, 1), lambda t: t.view(torch.int16), lambda t: t.view(-1))),
                         ("v_scales", (lambda t: t[:3], lambda t: t[..., ::2], lambda t: t.view(torch.float16))),
                         ("v_codes", (lambda t: t[:1], lambda t: t.view(4, 2, 32, 8), lambda t: t.view(torch.float32), lambda t: t[..., :8])),
                         ("k_codes", (lambda t: t[:3], lambda t: t.view(torch.float32), lambda t: t.transpose(1, 2), lambda t: t.view(4, -1)))):
        kept = getattr(cache, name)
        for other in others:
            view = other(kept)
            assert view.data_ptr() == kept.data_ptr()
            setattr(cache, name, view)
            with pytest.raises(ValueError):
                cache.c()
        setattr(cache, name, kept)
        cache.c()
    cache.v_scales = None
    with pytest.raises(TypeError):
        cache.c()
    # resized in place: the address stays
    cache = _fake_cache()
    cache.c()
    cache.k_scales.resize_(1, 2, 16)
    with pytest.raises(ValueError):
        cache.c()


class _Calls:
    """Stands for the library: notes a call's arguments and answers OK."""

    def __init__(self):
        self.args = {}

    def __getattr__(self, name):
        def call(*args):
            self.args[name] = args
            return OK
        return call


@pytest.fixture
def calls(monkeypatch):
    c = _Calls()
    monkeypatch.setattr(moe, "lib", lambda: c)
    monkeypatch.setattr(moe, "_stream", lambda s: 0)
    return c.args


def _on(*shape, dtype):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_OnGpu)


@pytest.mark.parametrize("T,B,cu,given,chosen", [(6, 6, False, None, 1), (6, 6, False, 3, 3), (500, 1, True, None, 500),
                                                 (24, 6, True, None, 4), (25, 6, True, None, 5), (6, 6, True, None, 1),
                                                 (500, 1, True, 1, 1), (0, 0, True, None, 0), (0, 2, True, None, 0)])
def test_max_q_left_out(calls, T, B, cu, given, chosen):
    """A prompt whose caller leaves max_q out does not go to the kernel for single tokens."""
    q = _on(T, 4, 128, dtype=torch.bfloat16)
    kw = {} if given is None else dict(max_q=given)
    moe.moe_kv4_attention(q, _fake_cache(), _on(B, 3, dtype=torch.int32), _on(B, dtype=torch.int32),
                          cu_q=_on(B + 1, dtype=torch.int32) if cu else None, out=_on(T, 4, 128, dtype=torch.bfloat16),
                          ws=_on(1 << 10, dtype=torch.uint8), **kw)
    args = calls["moe_kv4_attention"]
    assert args[7:11] == (B, T, 4, chosen)


def _block_calls(ws):
    cache, x, q = _fake_cache(), _on(3, 2, 128, dtype=torch.bfloat16), _on(3, 4, 128, dtype=torch.bfloat16)
    slots = _on(3, dtype=torch.int32)
    return (lambda: moe.moe_kv4_append(x, x, slots, cache, ws=ws),
            lambda: moe.moe_kv4_read(slots, cache, x, x, ws=ws),
            lambda: moe.moe_kv4_attention(q, cache, _on(3, 2, dtype=torch.int32), slots, out=q, ws=ws))


def test_a_workspace_that_the_gpu_cannot_use_is_refused(calls):
    """One in the host's memory, or strided, never reaches a kernel."""
    for ws, error in ((torch.zeros(1 << 10, dtype=torch.uint8), ValueError), (_on(1 << 10, 2, dtype=torch.uint8)[:, 0], ValueError),
                      (1 << 20, TypeError)):
        for call in _block_calls(ws):
            with pytest.raises(error):
                call()
    assert not calls
    # its size is in bytes, whatever its type
    ws = _on(1 << 10, dtype=torch.float32)
    for call in _block_calls(ws):
        call()
    assert calls["moe_kv4_append"][7:9] == calls["moe_kv4_read"][5:7] == calls["moe_kv4_attention"][15:17] == (ws.data_ptr(), 1 << 12)

"""The decoder layer example: a step replayed as a graph gives the bits of the same calls made one by one."""
import importlib.util
import os

import pytest
import torch

import w4a16_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "decoder_layer.py")


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("decoder_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 128, 16), (12, 3, 64, 32)])
def test_graph_steps_equal_the_calls(ex, Hq, Hkv, D, page):
    layer = ex.Layer(H=512, Hq=Hq, Hkv=Hkv, D=D, E=8, k=2, I=128, pages=64, page=page, max_tokens=512)
    prompts, steps = [37, 1, 150], 20
    g = torch.Generator(device="cuda").manual_seed(D)
    table = torch.randperm(48, generator=g, device="cuda").to(torch.int32).view(3, 16)
    x = torch.randn(sum(prompts), layer.H, generator=g, device="cuda").bfloat16()
    ex.prefill(layer, x, prompts, table)
    mine, cache = layer.cache, moe.Kv4Cache(*(t.clone() for t in layer.cache))
    decode = ex.Decode(layer, prompts, table)
    lens, rows = torch.tensor(prompts, dtype=torch.int32, device="cuda"), torch.arange(3, device="cuda")
    for _ in range(steps):
        x = torch.randn(3, layer.H, generator=g, device="cuda").bfloat16()
        decode.x.copy_(x)
        got = decode.step()
        layer.cache = cache
        want = layer(x, lens, ex.slots_of(table, lens, rows, page), table, lens + 1)
        layer.cache = mine
        lens = lens + 1
        assert torch.isfinite(got).all() and torch.equal(got, want)
    assert all(torch.equal(a, b) for a, b in zip(mine, cache))
    assert moe.moe_check_device_error(layer.ws) == 0


def test_run(ex):
    layer = ex.Layer(H=512, Hq=8, Hkv=2, D=64, E=4, k=2, I=128, pages=64, page=16, max_tokens=512)
    y, want, us = ex.run(layer, [37, 1, 150], 3)
    assert y.shape == want.shape == (3, 512) and torch.isfinite(y).all() and torch.isfinite(want).all() and us > 0
    with pytest.raises(ValueError):
        ex.run(layer, [1000], 1)

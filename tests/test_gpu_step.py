"""A step with drafted tokens, its calls in the order of their use: projections in 4 bits, norms and turn, rows into
the cache, attention over a window, the head, the verification."""
import pytest
import torch

import w4a16_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu


def test_a_step_with_drafts():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    g = torch.Generator(device="cuda").manual_seed(0)
    H, Hq, Hkv, D, V, S, n = 512, 8, 2, 64, 1000, 16, 40
    quant = lambda rows, cols: moe.moe_quantize_int4((torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5).bfloat16())  # noqa: E731
    qkv, o, head = quant((Hq + 2 * Hkv) * D, H), quant(H, Hq * D), quant(V, H)
    cache = moe.kv4_cache(8, Hkv, S, D)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
    freq = (1e4 ** (-torch.arange(0, D, 2, device="cuda").double() / D)).float()
    T = n + 4   # a prompt and its last token's three drafts behind it, in one pass
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pos = torch.arange(T, dtype=torch.int32, device="cuda")

    def layer(x, pos, length):
        q, k, v = moe.moe_w4a16_linear(x, *qkv).view(len(x), -1, D).split([Hq, Hkv, Hkv], 1)
        moe.moe_qk_norm_rope(q, k, pos, freq, q_out=q, k_out=k)
        moe.moe_kv4_append(k, v, pos, cache)
        a = moe.moe_kv4_attention_window(q, cache, table, i32(length), 20, 2, cu_q=i32(0, len(x)), max_q=len(x))
        return moe.moe_w4a16_linear(moe.moe_w4a16_linear(a.view(len(x), -1), *o), *head)

    whole = layer(x, pos, T)[n:]
    step = layer(x[n:].contiguous(), pos[n:].contiguous(), T)
    # the step's rows are the whole pass's but for the roundings of its kernels
    assert float((whole.double() - step.double()).norm() / whole.double().norm()) < 0.03
    best = step.float().argmax(1).to(torch.int32)
    drafts = best.clone()
    drafts[2] = (best[2] + 1) % V
    args = (drafts, i32(0, 4), torch.rand(4, generator=g, device="cuda"), torch.ones(1, V, device="cuda"))
    tokens, accepted = moe.moe_verify_drafts(step, *args, temperature=torch.zeros(1, device="cuda"))
    assert accepted.tolist() == [2] and tokens.tolist() == best[:3].tolist() + [-1]

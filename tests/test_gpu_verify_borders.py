"""The verification of drafted tokens where a decision is near: large noise, draws at the border of an acceptance,
residuals that nearly vanish, vocabularies at the borders of the kernels' chunks. Expected tokens follow from the
definition in 64 bits or from arithmetic stated beside the case."""
import pytest
import torch

import w4a16_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.lib()


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _f32(*v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


@pytest.mark.parametrize("e", [2.0 ** 126, 1e38, 3.4e38])
def test_noise_of_the_largest_size(e):
    # token 11: score about 1 / e >= 2.9e-39; token 500: e^-70 / 1e10 < 4e-41; the others have no weight
    V = 600
    for winner, other in ((11, 500), (500, 11)):
        l = torch.full((1, V), -torch.inf, dtype=torch.bfloat16, device="cuda")
        noise = torch.ones(1, V, device="cuda")
        l[0, winner], noise[0, winner] = 0, e
        l[0, other], noise[0, other] = -70, 1e10
        t, a = moe.moe_verify_drafts(l, _i32(0), _i32(0, 1), _f32(0.5), noise)
        assert t.tolist() == [winner] and a.tolist() == [0]


def test_noise_that_is_infinite_loses_to_any_weight():
    V = 600
    l = torch.full((1, V), -torch.inf, dtype=torch.bfloat16, device="cuda")
    noise = torch.full((1, V), 3e38, device="cuda")
    l[0, 11], noise[0, 11] = 0, torch.inf
    l[0, 500] = -70
    t, _ = moe.moe_verify_drafts(l, _i32(0), _i32(0, 1), _f32(0.5), noise)
    assert t.tolist() == [500]   # e^-70 / 3e38 > 0 = 1 / inf


def _softmax(l, t):
    return torch.softmax(l.double() / t, -1)


def _row(g, V, spread=2.0):
    l = torch.randn(1, -(-V // 8) * 8, generator=g, device="cuda") * spread
    l[0, :V].scatter_add_(0, torch.randint(0, V, (24,), generator=g, device="cuda"), 4 + 9 * torch.rand(24, generator=g, device="cuda"))
    return l


@pytest.mark.parametrize("V", [8, 333, 50257, 248320])
def test_a_token_of_probability_one_is_accepted_whatever_is_drawn(V):
    # all the others at -inf: p = 1 > u
    pitch = -(-V // 8) * 8
    n = 60
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randint(0, V, (2 * n,), generator=g, device="cuda").to(torch.int32)
    l = torch.full((2 * n, pitch), -torch.inf, dtype=torch.bfloat16, device="cuda")
    l[torch.arange(2 * n, device="cuda"), x.long()] = (20 * torch.randn(2 * n, generator=g, device="cuda")).bfloat16()
    t = 0.1 + 2 * torch.rand(n, generator=g, device="cuda")
    noise = torch.ones(n, pitch, device="cuda")[:, :V]
    u = torch.full((2 * n,), 1 - 2.0 ** -24, device="cuda")
    tokens, a = moe.moe_verify_drafts(l[:, :V], x, torch.arange(0, 2 * n + 1, 2, dtype=torch.int32, device="cuda"), u, noise, temperature=t)
    assert a.tolist() == [1] * n and torch.equal(tokens, x)


@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("V", [40, 5001, 50257, 248320])
def test_draws_next_to_the_border(V, with_q):
    """u just below p(x) / q(x) accepts, just above refuses: the two numbers of fp32 around the quotient, which are
    2^-26 of it away from it at least (others are not tried), where 64-bit sums are off by V 2^-53 at most."""
    tried = 0
    for seed in range(40):
        g = torch.Generator(device="cuda").manual_seed(seed)
        l = _row(g, V)
        d = l + 0.6 * torch.randn(l.shape, generator=g, device="cuda")
        l, d = l.bfloat16().repeat(2, 1)[:, :V], d.bfloat16().repeat(2, 1)[:, :V]   # (rows of a multiple of 16 bytes)
        t = 0.5 + seed / 40
        p, q = _softmax(l[0], _f32(t).double()), _softmax(d[0], _f32(t).double())
        x = int((p * (p < q) if with_q else p).argmax())
        border = float(p[x] / q[x]) if with_q else float(p[x])
        near = torch.tensor(border, dtype=torch.float64).float()
        around = [near, torch.nextafter(near, torch.tensor(0.0)), torch.nextafter(near, torch.tensor(2.0))]
        for u in {float(v) for v in around}:
            if abs(u - border) < 2.0 ** -26 * border or u >= 1:
                continue
            tried += 1
            _, a = moe.moe_verify_drafts(l, _i32(x, 0), _i32(0, 2), _f32(u, 0.5), torch.ones(1, -(-V // 4) * 4, device="cuda")[:, :V],
                                         draft_logits=d if with_q else None, temperature=_f32(t))
            assert a.tolist() == [int(u < border)], (seed, u, border)
    assert tried > 40


@pytest.mark.parametrize("V", [40, 5001, 50257])
def test_races_that_are_nearly_even(V):
    """Two tokens of the residual whose scores differ by 2^-21 of themselves; the others have lost by far. (u = 1 refuses
    any draft with p < q; a difference of 64-bit numbers below 2^-20 of them is not told to 2^-21 of itself well enough.)"""
    tried = 0
    for seed in range(40):
        g = torch.Generator(device="cuda").manual_seed(seed)
        l = _row(g, V)
        d = l + 0.6 * torch.randn(l.shape, generator=g, device="cuda")
        l, d = l.bfloat16().repeat(2, 1)[:, :V], d.bfloat16().repeat(2, 1)[:, :V]   # (rows of a multiple of 16 bytes)
        t = 0.5 + seed / 40
        p, q = _softmax(l[0], _f32(t).double()), _softmax(d[0], _f32(t).double())
        w = (p - q).clip(min=0)
        pair = w.topk(2).indices
        x = int((q - p).argmax())
        if (w[pair] < 2.0 ** -20 * (p + q)[pair]).any():
            continue
        tried += 1
        for first in (0, 1):
            noise = torch.full((1, -(-V // 4) * 4), 1e6, device="cuda")[:, :V]
            a, b = int(pair[first]), int(pair[1 - first])
            noise[0, a] = 1.0
            noise[0, b] = float(w[b] / w[a]) * (1 + 2.0 ** -21)   # (rounded by 2^-24 of itself)
            tokens, acc = moe.moe_verify_drafts(l, _i32(x, 0), _i32(0, 2), _f32(1.0, 0.5), noise,
                                                draft_logits=d, temperature=_f32(t))
            assert acc.tolist() == [0] and tokens.tolist() == [a, -1], (seed, first)
    assert tried > 25


@pytest.mark.parametrize("with_q", [True, False])
def test_temperatures_as_small_as_the_logits_differences(with_q):
    V = 3000
    for t, size in ((1e-42, 1e-38), (1e-40, 1e-35), (1e-31, 4e-30), (1e-36, 1e-30)):
        # the largest logit ahead of the next by size, 100 t or more in the first two and the last: p = 1 there
        l = torch.zeros(2, V, dtype=torch.bfloat16, device="cuda")
        l[:, 77], l[:, 1500], l[:, 9] = size, 2 * size, -size
        d = torch.zeros_like(l)
        noise = torch.ones(1, V, device="cuda")
        noise[0, 1500] = 2.0
        p, q = _softmax(l[0], _f32(t).double()), _softmax(d[0], _f32(t).double())
        for x, u in ((1500, 0.9), (77, 0.9), (77, 1e-30), (5, 0.5)):
            keep = u * (float(q[x]) if with_q else 1.0) < float(p[x])
            r = (p - (q if with_q else torch.nn.functional.one_hot(torch.tensor(x), V).cuda())).clip(min=0)
            want = [x, int((p / noise[0]).argmax())] if keep else [int(((r if r.sum() > 0 else p) / noise[0]).argmax()), -1]
            tokens, a = moe.moe_verify_drafts(l, _i32(x, 0), _i32(0, 2), _f32(u, 0.5), noise, draft_logits=d if with_q else None, temperature=_f32(t))
            assert tokens.tolist() == want and a.tolist() == [int(keep)], (t, x, u)


@pytest.mark.parametrize("t,size", [(3e38, 3e38), (1e38, 3e38), (2e37, 2e37)])
def test_temperatures_as_large_as_the_logits(t, size):
    # differences of logits pass fp32's range: p(7) = 1 / (1 + 999 e^(-2 size / t)), the others e^(-2 size / t) of it
    V = 1000
    l = torch.full((2, V), -size, dtype=torch.bfloat16, device="cuda")
    l[:, 7] = size
    p = _softmax(l[0], _f32(t).double())
    for x, u in ((7, float(p[7]) * 0.9), (7, float(p[7]) * 1.1), (5, float(p[5]) * 0.9), (5, float(p[5]) * 1.1)):
        keep = u < float(p[x])
        for fast in (7, 6):
            noise = torch.ones(1, V, device="cuda")
            noise[0, fast] = 1e-4
            r = p.clone() if keep else torch.where(torch.arange(V, device="cuda") == x, 0, p)
            want = int((r / noise[0]).argmax())
            tokens, a = moe.moe_verify_drafts(l, _i32(x, 0), _i32(0, 2), _f32(u, 0.5), noise, temperature=_f32(t))
            assert tokens.tolist() == ([x, want] if keep else [want, -1]) and a.tolist() == [int(keep)], (x, u, fast)


@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("rows,V", [([3, 4], 16383), ([3, 4], 16384), ([3, 4], 16385), ([3], 32767), ([3], 32768), ([3], 32769), ([2], 2 ** 20 - 1), ([3], 2 ** 20)])
def test_vocabularies_at_the_borders_of_chunks(rows, V, with_q):
    from test_gpu_verify import _compare, _inputs
    done = 0
    for seed in range(12):   # until three draws are clear
        done += _compare(_inputs(rows, V, with_q, (0, 0.4, 1)[seed % 3], V + seed, spread=(2.0, 0.3, 6.0)[seed % 3]), rows)
        if done == 3:
            break
    assert done == 3


def test_ties_at_the_borders_of_chunks():
    V = 2 ** 20
    for t in (0.0, 1.0):
        l = torch.full((1, V), -1.0, dtype=torch.bfloat16, device="cuda")
        e = torch.ones(1, V, device="cuda")
        for at in (16383, 16384, 32767, 32768, V - 1):
            l[0, :at] = -1
            l[0, at:] = 1
            tok, a = moe.moe_verify_drafts(l, _i32(0), _i32(0, 1), _f32(0.0), e, temperature=_f32(t))
            assert tok.tolist() == [at] and a.tolist() == [0]

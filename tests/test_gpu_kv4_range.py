"""Attention over the 4-bit cache where values lie far apart: scores far below zero.

Tolerances are those that test_gpu_kv4.py derives.
"""
import math

import pytest
import torch

import w4a16_mixture_experts_gb300 as moe
from test_gpu_kv4 import _check, _filled, _gen, _randn, _tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.lib()


def _words(n):
    """Packed words of codes n (whole numbers in [-8, 7], [..., D])."""
    n = (n.to(torch.int32) + 8).unflatten(-1, (-1, 8))
    out = torch.zeros(n.shape[:-1], dtype=torch.int32, device=n.device)
    for i in range(8):
        out |= n[..., i] << (4 * i)
    return out


def _one_sequence(g, n, S, D, Hkv=1):
    """A cache with one sequence of n keys in it, its table, and (page, place) of each key."""
    pages = -(-n // S) + 2
    cache = _filled(g, pages, Hkv, S, D)
    table = _tables(g, [n], S, pages)
    j = torch.arange(n, device="cuda")
    return cache, table, table[0].long()[j // S], j % S


# ---- scores far below zero -----------------------------------------------------------------------------------

@pytest.mark.parametrize("nats", [-100])
@pytest.mark.parametrize("n", [1, 128, 3000])
@pytest.mark.parametrize("nq,D", [(1, 128), (1, 64), (6, 128), (140, 64)])
def test_scores_that_all_lie_far_below_zero(nats, n, nq, D):
    """A softmax does not care where its scores lie."""
    g = _gen(n + nq)
    S, G = 16, 4
    n += nq - 1
    cache, table, page, at = _one_sequence(g, n, S, D)
    codes = (_randn(g, n, D) * 1.2).round().clamp(-8, 7)
    codes[:, 0] = 7                                     # one value carries the offset: q[0] * 3.5
    cache.k_codes[page, 0, at] = _words(codes)
    cache.k_scales.fill_(0.5)
    q = _randn(g, nq, G, D).bfloat16()
    q[..., 0] = nats / 3.5 * D ** 0.5
    for max_q in (nq, 1, 4096):
        _check(q, cache, table, [n], [nq], max_q=max_q)


@pytest.mark.parametrize("nq", [1, 6, 140])
def test_keys_far_below_zero_beside_others(nq):
    """Whole shares of a row far below the rest, before and after them."""
    g = _gen(nq)
    n, S, G, D = 5000, 32, 8, 128
    cache, table, page, at = _one_sequence(g, n, S, D)
    codes = (_randn(g, n, D) * 1.2).round().clamp(-8, 7)
    codes[:, 0] = 0
    codes[:700, 0] = codes[3000:4100, 0] = 7
    cache.k_codes[page, 0, at] = _words(codes)
    cache.k_scales.fill_(0.5)
    q = _randn(g, nq, G, D).bfloat16()
    q[..., 0] = -150 / 3.5 * D ** 0.5
    for max_q in (nq, 1, 4096):
        _check(q, cache, table, [n], [nq], max_q=max_q)


# ---- queries that are not finite, and no key --------------------------------------------------------------------

@pytest.mark.parametrize("nq", [6, 140])
def test_queries_that_are_not_finite_and_see_nothing(nq):
    g = _gen(nq)
    n, G = 3, 4
    cache, table, _, _ = _one_sequence(g, n, 16, 128, Hkv=2)
    q = _randn(g, nq, 2 * G, 128).bfloat16()
    q[0, 1, 5], q[1, 7, 0], q[nq - n - 1, 2, 127] = float("nan"), float("inf"), -float("inf")
    q[nq - 1, 3, 9] = float("nan")                       # this one sees keys
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for max_q in (1, nq, 4096):
        out, lse = moe.moe_kv4_attention(q, cache, table, i32(n), cu_q=i32(0, nq), max_q=max_q, lse=True)
        assert (out[:nq - n] == 0).all() and (lse[:nq - n] == -math.inf).all()
        assert out[nq - 1, 3].isnan().all() and lse[nq - 1, 3].isnan()
        assert out[nq - 1, [0, 1, 2, 4, 5, 6, 7]].isfinite().all()

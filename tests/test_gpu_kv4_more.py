"""The 4-bit cache's attention and appends where the sizes and values are unusual: more sequences than a block has
threads, row tiles that end anywhere, several items a block, queries that are not finite, scales beside the smallest.
The tolerances are those that test_gpu_kv4.py derives."""
import pytest
import torch

import w4a16_mixture_experts_gb300 as moe
from test_gpu_kv4 import _check, _filled, _gen, _quantised, _randn, _reference, _rows, _tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.lib()


@pytest.mark.parametrize("Hkv,G,D,S,B", [(1, 8, 128, 16, 700), (2, 2, 64, 32, 1500)])
def test_more_sequences_than_threads(Hkv, G, D, S, B):
    """Prompts of a few tokens, one long enough that the kernel for many rows takes them all; some without any."""
    g = _gen(B)
    nqs = [(i * 7) % 4 for i in range(B)]
    nqs[B // 2], nqs[-1] = 65, 0
    lens = [n + (i * 5) % 3 * (n > 0) for i, n in enumerate(nqs)]
    pages = sum(-(-n // S) for n in lens)
    cache = _filled(g, pages, Hkv, S, D)
    q = _randn(g, sum(nqs), Hkv * G, D).bfloat16()
    _check(q, cache, _tables(g, lens, S, pages), lens, nqs)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,nqs", [(1, [127, 128, 129]), (3, [85, 86, 43]), (8, [16, 17, 33]), (5, [1, 200, 3]), (32, [3, 4, 9])])
def test_row_tiles_that_end_anywhere(D, G, nqs):
    """128 and 256 rows and their neighbours, with keys before them that end inside a page and a stage."""
    g = _gen(D + G)
    lens = [n + x for n, x in zip(nqs, (0, 301, 127))]
    S = 16
    pages = sum(-(-n // S) for n in lens)
    cache = _filled(g, pages, 2, S, D)
    q = _randn(g, sum(nqs), 2 * G, D).bfloat16()
    _check(q, cache, _tables(g, lens, S, pages), lens, nqs, max_q=max(max(nqs), 33))


@pytest.mark.parametrize("nq", [1, 3, 70])
def test_queries_that_are_not_finite(nq):
    """Such a query's row is NaN, and the others are what they would be."""
    g = _gen(nq)
    lens, nqs = [300, nq, 129], [nq] * 3
    cache = _filled(g, 64, 2, 16, 128)
    table = _tables(g, lens, 16, 64)
    q = _randn(g, 3 * nq, 8, 128).bfloat16()
    want, z, tol, ltol = _reference(q, cache, table, lens, nqs, 128 ** -0.5)
    bad = torch.zeros(3 * nq, 8, dtype=torch.bool, device="cuda")
    for t, h, d, x in ((0, 0, 3, "nan"), (nq - 1, 5, 127, "inf"), (2 * nq, 7, 0, "-inf")):
        q[t, h, d] = float(x)
        bad[t, h] = True
    cu = torch.arange(0, 3 * nq + 1, nq, dtype=torch.int32, device="cuda")
    out, lse = moe.moe_kv4_attention(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), cu_q=cu, max_q=nq, lse=True)
    assert out[bad].isnan().all()
    assert ((out.double() - want).abs() <= tol)[~bad].all() and ((lse.double() - z).abs() <= ltol)[~bad].all()


@pytest.mark.parametrize("top", [2.0 ** -126, 2.0 ** -124, 3e-37, 7e-37, 1e-36])
def test_appends_beside_the_smallest_scales(top):
    g = _gen(3)
    x = (torch.rand(40, 2, 128, generator=g, device="cuda") * 2 - 1).double()
    x = (x / x.abs().amax(-1, keepdim=True) * top).bfloat16()
    cache = moe.kv4_cache(3, 2, 16, 128)
    slots = torch.arange(40, dtype=torch.int32, device="cuda")
    moe.moe_kv4_append(x, x, slots, cache)
    # the formula's own fp32 quotient, on the host, where subnormals are kept
    q, s = _quantised(x.cpu())
    at = slots.long().cpu()
    codes, scales = cache.k_codes.cpu()[at // 16, :, at % 16], cache.k_scales.cpu()[at // 16, :, at % 16]
    assert torch.equal(scales, s) and torch.equal(_rows(codes).float(), q)

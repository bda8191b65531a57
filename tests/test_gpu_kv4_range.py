"""Attention over the 4-bit cache where values lie far apart: scores far below zero, queries, keys and values of very
different sizes in one sequence, long tails of small probabilities.

Tolerances are those that test_gpu_kv4.py derives, key by key, with tighter terms where the kernels promise more. With
p_j the probabilities, v_j = s_j n_j a row of V (scale, codes), C = max_j p_j s_j the weight of the row's largest key:
 - a score's error goes with its own key's products, so a probability's does: a huge key that has no probability adds
   nothing to the others' bound;
 - a query value keeps 2^-33 of the row's largest at least (half a step of fp16's smallest, against a largest of 2^8);
 - p_j s_j enters the tensor core as fp16 against the row's own largest: off by `floor` * C at most where it is small.
   2^-31: half of fp16's smallest step, against 2^6 at least; a kernel that scales V by a common power of two takes off
   p_j alone, at 2^-32 of the largest p, and may do so where the scales seen so far lie within 2^11 of each other,
   which is 2^-21 of C.
 - a CTA adds at most its share of the keys, 16 at a time, and the shares' sums are joined.
"""
import math

import pytest
import torch

import w4a16_mixture_experts_gb300 as moe
from test_gpu_kv4 import U16, U32, UB, _check, _filled, _gen, _randn, _tables, _unpack

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


def _near(q, cache, table, n, max_q, scale=None, floor=2.0 ** -21, rows=None, copies=1):
    """Attention of the last queries of one sequence of n keys against 64 bits; rows: of the queries, which to compare.
    copies: sequences that are all this one (on the same pages), so that a block has whole sequences and not a few keys."""
    nq, Hq, D = q.shape
    Hkv, S = cache.k_scales.shape[1:]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = moe.kv4_workspace(copies * nq, Hq, Hkv, D)
    cu = torch.arange(0, copies * nq + 1, nq, dtype=torch.int32, device="cuda")
    out, lse = moe.moe_kv4_attention(q.repeat(copies, 1, 1), cache, table.repeat(copies, 1), i32(*[n] * copies), cu_q=cu, max_q=max_q,
                                     scale=scale, lse=True, ws=ws)
    assert moe.moe_check_device_error(ws) == 0
    out, lse = out.view(copies, nq, Hq, D), lse.view(copies, nq, Hq)
    shares = torch.cuda.get_device_properties(0).multi_processor_count if copies == 1 else 1   # that the keys are cut into, at least
    adds = n / (16 * shares) + 4 * 128 / 16 + 640
    pages = table[0, :-(-n // S)].long()
    for h in range(Hkv):
        vs = cache.v_scales[pages, h].reshape(-1)[:n].double()
        codes = _unpack(cache.v_codes[pages, h], torch.ones_like(cache.v_scales[pages, h])).reshape(-1, D)[:n]
        k = _unpack(cache.k_codes[pages, h], cache.k_scales[pages, h]).reshape(-1, D)[:n]
        for i in range(nq) if rows is None else rows:
            seen = n - nq + i + 1
            assert seen > 0
            x = q[i, h * G:(h + 1) * G].double()
            s = scale * (x @ k[:seen].T)
            z = torch.logsumexp(s, -1, keepdim=True)
            p, ka = (s - z).exp(), k[:seen].abs()
            ds = 2 * U32 * (D + 4) * abs(scale) * (x.abs() @ ka.T) + abs(scale) * 2.0 ** -33 * x.abs().amax(-1, keepdim=True) * ka.sum(-1)
            ds = torch.expm1(2 * ds).clamp(max=1e30)   # (a finite bound, so that no probability times it is none)
            want = (p * vs[:seen]) @ codes[:seen]
            absolute = codes[:seen].abs()
            mass = (p * vs[:seen]) @ absolute
            C = (p * vs[:seen]).amax(-1, keepdim=True)
            dl = (p * ds).sum(-1, keepdim=True)
            tol = UB * want.abs() + (U16 + dl + 2 * U32 * adds) * mass + (p * vs[:seen] * ds) @ absolute + floor * C * absolute.sum(0)
            off = (out[:, i, h * G:(h + 1) * G].double() - want).abs()
            assert (off <= tol).all(), (i, h, float((off - tol).max()), float((off / tol.clamp(min=1e-300)).max()))
            off = (lse[:, i, h * G:(h + 1) * G].double() - z.squeeze(-1)).abs()
            ltol = dl.squeeze(-1) + 2 * U32 * adds + 2 * U32 * z.squeeze(-1).abs()
            assert (off <= ltol).all(), (i, h, float((off - ltol).max()))


# ---- scores far below zero -----------------------------------------------------------------------------------

@pytest.mark.parametrize("nats", [-100, -1000, -30000])
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


# ---- queries with one value far above the rest -------------------------------------------------------------------

@pytest.mark.parametrize("nq,max_q", [(1, 1), (1, 4096), (5, 1), (5, 5), (70, 1), (70, 70)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("above", [9, 11, 13, 17, 20])
def test_queries_with_a_value_far_above_the_rest(nq, max_q, D, above):
    """Where K holds zeros beside it, the rest alone decides."""
    g = _gen(above + D)
    n, S, G = 700, 16, 4
    cache, table, page, at = _one_sequence(g, n, S, D)
    for d in (4, 37):
        codes = _unpack(cache.k_codes[page, 0, at], torch.ones(n, device="cuda"))
        codes[:, d] = 0
        cache.k_codes[page, 0, at] = _words(codes)
    q = (1.6 * _randn(g, nq, G, D)).bfloat16()
    q[..., 4], q[..., 37] = 2.0 ** above, -1.7 * 2.0 ** above
    _near(q, cache, table, n, max_q)


# ---- scales far apart in one sequence ------------------------------------------------------------------------------

@pytest.mark.parametrize("copies", [1, 700])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("by", [2.0 ** 18, 2.0 ** 26, 2.0 ** 60])
@pytest.mark.parametrize("nq,max_q", [(6, 1), (6, 6), (6, 4096), (140, 140), (140, 1)])
def test_one_key_with_a_huge_scale(which, by, nq, max_q, copies):
    """The last key's scale is far above the others', and only the last query sees it."""
    g = _gen(nq)
    n, S, G, D = 500, 16, 4, 128
    cache, table, page, at = _one_sequence(g, n, S, D)
    scales = cache.k_scales if which == "k" else cache.v_scales
    scales[page[-1], 0, at[-1]] *= by
    q = (1.6 * _randn(g, nq, G, D)).bfloat16()
    rows = sorted(set(range(0, nq, 17)) | {nq - 2, nq - 1})
    _near(q, cache, table, n, max_q, rows=rows, copies=copies)


@pytest.mark.parametrize("copies", [1, 700])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nq,max_q", [(1, 1), (1, 4096), (6, 1), (6, 6), (140, 140), (140, 1)])
def test_scales_spread_over_thirty_octaves(nq, max_q, D, first, copies):
    """K's and V's scales from 2^-30 to 1, the largest on keys that most rows do not see, or on the first."""
    g = _gen(nq + D)
    n, S, G = 1100, 16, 5
    cache, table, page, at = _one_sequence(g, n, S, D)
    for scales in (cache.k_scales, cache.v_scales):
        e = -30 * torch.rand(n, generator=g, device="cuda")
        if first:
            e[:3] = 0
        else:
            e -= 12                                      # and then far above
            e[-2:] = 0
        scales[page, 0, at] = torch.exp2(e).bfloat16()
    q = (40 * _randn(g, nq, G, D)).bfloat16()
    rows = sorted(set(range(0, nq, 17)) | {max(nq - 3, 0), nq - 1})
    _near(q, cache, table, n, max_q, rows=rows, copies=copies)


@pytest.mark.parametrize("copies", [1, 700])
@pytest.mark.parametrize("order", ["up", "down"])
@pytest.mark.parametrize("nq,max_q", [(1, 1), (1, 4096), (6, 6), (140, 140)])
def test_scales_that_change_along_the_sequence(nq, max_q, order, copies):
    """V's scales fall or rise by 2^40 from the first key to the last, while the scores favour the small ones."""
    g = _gen(nq)
    n, S, G, D = 2000, 32, 2, 64
    cache, table, page, at = _one_sequence(g, n, S, D)
    e = -40 * torch.arange(n, device="cuda") / n
    e = e if order == "down" else e.flip(0)
    cache.v_scales[page, 0, at] = torch.exp2(e).bfloat16()
    codes = (_randn(g, n, D) * 1.2).round().clamp(-8, 7)
    # the score makes up for the scale: exp(score) * scale is about 1 everywhere
    codes[:, 0] = (-e / 40 * 15 - 8).round().clamp(-8, 7)
    cache.k_codes[page, 0, at] = _words(codes)
    cache.k_scales.fill_(0.5)
    q = (0.3 * _randn(g, nq, G, D)).bfloat16()
    q[..., 0] = 40 * math.log(2) / 15 / 0.5 * D ** 0.5
    rows = sorted(set(range(0, nq, 17)) | {nq - 1})
    _near(q, cache, table, n, max_q, rows=rows, copies=copies)


# ---- long tails ---------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("nq,max_q,copies", [(1, 1, 1), (1, 1, 1300), (4, 4, 1300), (10, 10, 1000), (40, 40, 1), (40, 40, 310)])
@pytest.mark.parametrize("D", [64, 128])
def test_a_peak_and_a_long_flat_tail(nq, max_q, copies, D):
    """One key 18 nats above 2^17 others: the others' mass is small, and all of V that the row has."""
    g = _gen(D)
    n, S, G = (1 << 17) + 77, 64, 2
    cache, table, page, at = _one_sequence(g, n, S, D)
    codes = torch.zeros(n, D, device="cuda")
    codes[333] = 7
    cache.k_codes[page, 0, at] = _words(codes)
    cache.k_scales.fill_(0.5)
    values = 5 + (torch.rand(n, D, generator=g, device="cuda") * 2).floor()
    values[333] = 0
    cache.v_codes[page, 0, at] = _words(values)
    cache.v_scales.fill_(0.5)
    q = torch.full((nq, G, D), 18 / 3.5 / D ** 0.5, device="cuda").bfloat16()
    _near(q, cache, table, n, max_q, floor=2.0 ** -31, rows=[0, nq - 1], copies=copies)


# ---- zeros ----------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("then", [1.0, 2.0 ** -60, 2.0 ** 60])
@pytest.mark.parametrize("nq,max_q", [(1, 1), (6, 6), (140, 140)])
def test_zero_scales_before_others(nq, max_q, then):
    """The first keys' rows are zeros, so that their scales give no exponent, then come others, some of them far apart."""
    g = _gen(nq)
    n, S, G, D = 1000, 16, 4, 64
    cache, table, page, at = _one_sequence(g, n, S, D)
    cache.k_scales[page[:300], 0, at[:300]] = 0
    cache.v_scales[page[:300], 0, at[:300]] = 0
    cache.v_scales[page[300:], 0, at[300:]] *= then
    cache.v_scales[page[700:], 0, at[700:]] *= 2.0 ** -20
    q = (1.6 * _randn(g, nq, G, D)).bfloat16()
    _near(q, cache, table, n, max_q, rows=sorted({0, nq // 2, nq - 1}), copies=700)


@pytest.mark.parametrize("where", [0, 200, 900])
@pytest.mark.parametrize("nq,max_q", [(1, 1), (6, 6), (140, 140)])
def test_a_zero_row_that_has_all_the_probability(nq, max_q, where):
    """A key 40 nats above the others holds zeros: what the others add, 2^-58 of their values, is all that there is."""
    g = _gen(nq)
    n, S, G, D = 1200, 16, 4, 128
    cache, table, page, at = _one_sequence(g, n, S, D)
    codes = (_randn(g, n, D) * 1.2).round().clamp(-8, 7)
    codes[:, 0] = 0
    codes[where, 0] = 7
    cache.k_codes[page, 0, at] = _words(codes)
    cache.k_scales.fill_(0.5)
    cache.v_scales[page[where], 0, at[where]] = 0
    if where == 200:                                     # and nothing but zeros before it
        cache.v_scales[page[:200], 0, at[:200]] = 0
    q = _randn(g, nq, G, D).bfloat16()
    q[..., 0] = 40 / 3.5 * D ** 0.5
    _near(q, cache, table, n, max_q, rows=sorted({0, nq // 2, nq - 1}), copies=700)

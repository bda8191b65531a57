"""Attention over the 4-bit cache with a sliding window and first keys that stay visible, against its formula in 64
bits. Every case runs through both kernels. Pages that no query sees are gone (their table entries are -1), and keys
that no query sees hold NaN. The tolerances are those that test_gpu_kv4.py derives, over the keys that a row sees, and
one term that test_gpu_kv4_range.py derives: a probability may enter the tensor core as its product with its key's V
scale, rounded at 2^-31 of the row's largest such product C (half of fp16's smallest step, 2^-25, against 2^6 at least),
so an output may be off by 2^-31 C sum_j |code_j|. (It matters where the key that C comes from has zeros: there the
output is made of the other keys alone, and the other terms follow those.)"""
import math

import pytest
import torch

import w4a16_mixture_experts_gb300 as moe
from test_gpu_kv4 import U16, U32, UB, _filled, _gen, _randn, _tables, _unpack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.lib()


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _seen(n, nq, window, sinks):
    """[nq, n]: which keys each query sees."""
    pos = torch.arange(n - nq, n, device="cuda").unsqueeze(1)
    j = torch.arange(n, device="cuda")
    return (j <= pos) & ((j > pos - window) | (j < sinks))


def _reference(q, cache, table, lens, nqs, scale, window, sinks):
    """out, lse, and each output's tolerance and each lse's, in 64 bits."""
    T, Hq, D = q.shape
    Hkv, S = cache.k_scales.shape[1:]
    G = Hq // Hkv
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    t = 0
    for b, (n, nq) in enumerate(zip(lens, nqs)):
        if n and nq:
            seen = _seen(n, nq, window, sinks)
            some = seen.any(1)
            any_key = seen.any(0).nonzero().squeeze(1)          # (the others are not there at all)
            seen = seen[:, any_key]
            page, off = table[b].long()[any_key // S], any_key % S
            for h in range(Hkv):
                k = _unpack(cache.k_codes[page, h, off], cache.k_scales[page, h, off])
                v = _unpack(cache.v_codes[page, h, off], cache.v_scales[page, h, off])
                x = q[t:t + nq, h * G:(h + 1) * G].double()
                s = (scale * torch.einsum("tgd,nd->tgn", x, k)).masked_fill(~seen.unsqueeze(1), -math.inf)[some]
                p, z = torch.softmax(s, -1), torch.logsumexp(s, -1)
                qk = (abs(scale) * torch.einsum("tgd,nd->tgn", x.abs(), k.abs())).masked_fill(~seen.unsqueeze(1), 0)[some].amax(-1)
                count = seen[some].sum(1).double().view(-1, 1) + 8
                ds = 2 * U32 * (D + 4) * qk
                o = p @ v
                small = 2.0 ** -25 * (seen[some].double() @ v.abs()).unsqueeze(1) / (s - s.amax(-1, keepdim=True)).exp().sum(-1, keepdim=True)
                sv = cache.v_scales[page, h, off].double()
                codes = _unpack(cache.v_codes[page, h, off], torch.ones_like(cache.v_scales[page, h, off])).abs()
                small = small + 2.0 ** -31 * (p * sv.abs()).amax(-1, keepdim=True) * (seen[some].double() @ codes).unsqueeze(1)
                rows = torch.arange(t, t + nq, device="cuda")[some]
                H = slice(h * G, (h + 1) * G)
                out[rows, H], lse[rows, H] = o, z
                tol[rows, H] = UB * o.abs() + (U16 + (2 * ds + 2 * U32 * count).unsqueeze(-1)) * (p @ v.abs()) + small
                ltol[rows, H] = ds + 2 * U32 * count + 2 * U32 * z.abs()
        t += nq
    return out, lse, tol, ltol


def _hide(cache, table, lens, nqs, window, sinks):
    """Takes away what no query sees: pages out of the tables, NaN for single keys."""
    S = cache.k_scales.shape[2]
    for b, (n, nq) in enumerate(zip(lens, nqs)):
        if not n:
            continue
        hidden = ~_seen(n, nq, window, sinks).any(0) if nq else torch.ones(n, dtype=torch.bool, device="cuda")
        j = hidden.nonzero().squeeze(1)
        page, off = table[b].long()[j // S], j % S
        cache.k_scales[page, :, off] = math.nan
        cache.v_scales[page, :, off] = math.nan
        whole = torch.nn.functional.pad(hidden, (0, -n % S), value=True).view(-1, S).all(1)
        table[b, : whole.shape[0]][whole] = -1


def _run(q, cache, table, lens, nqs, window, sinks, scale=None, max_q=None, ws=None):
    T, Hq, D = q.shape
    Hkv = cache.k_scales.shape[1]
    ws = moe.kv4_workspace(T, Hq, Hkv, D) if ws is None else ws
    cu = _i32(0, *torch.tensor(nqs).cumsum(0).tolist())
    out, lse = moe.moe_kv4_attention_window(q, cache, table, _i32(*lens), window, sinks, cu_q=cu, max_q=max_q or max(max(nqs), 1), scale=scale,
                                            lse=True, ws=ws)
    assert moe.moe_check_device_error(ws) == 0
    return out, lse


def _check(q, cache, table, lens, nqs, window, sinks, scale=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    _hide(cache, table, lens, nqs, window, sinks)
    want, z, tol, ltol = _reference(q, cache, table, lens, nqs, scale, window, sinks)
    empty = z == -math.inf
    for max_q in (max(max(nqs), 1), 1, 4096):
        out, lse = _run(q, cache, table, lens, nqs, window, sinks, scale, max_q)
        off = (out.double() - want).abs()
        assert (off <= tol).all(), (max_q, float((off - tol).nan_to_num(nan=9e9).max()))
        assert (lse[empty] == -math.inf).all() and (out[empty] == 0).all()
        off = (lse.double() - z)[~empty].abs()
        assert (off <= ltol[~empty]).all(), (max_q, float((off - ltol[~empty]).max()))


def _case(g, Hkv, G, D, S, nqs, lens):
    pages = sum(-(-n // S) for n in lens) + 5
    cache = _filled(g, pages, Hkv, S, D)
    return (1.6 * _randn(g, sum(nqs), Hkv * G, D)).bfloat16(), cache, _tables(g, lens, S, pages, M=-(-max(lens) // S) + 2), lens, nqs


WINDOWS = [(1, 0), (1, 1), (5, 3), (16, 0), (127, 4), (128, 128), (129, 130), (300, 0), (333, 257), (1000, 1), (5000, 7)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("Hkv,G,D,S,nqs,lens", [
    (2, 4, 128, 16, [1], [1]),
    (4, 7, 64, 32, [1] * 9, [0, 1, 15, 16, 17, 127, 128, 129, 2000]),     # a length of zero leaves its row empty
    (1, 8, 128, 64, [1, 1, 1, 1], [700, 513, 1025, 3000]),
    (2, 4, 64, 16, [3, 1, 0, 8, 2], [100, 1, 50, 8, 1700]),               # a sequence without queries
    (1, 8, 128, 32, [4, 4], [3, 1]),                                      # more queries than keys: empty rows
    (1, 1, 128, 128, [31, 32, 33], [400, 801, 1600]),                     # rows whose windows begin in different units
    (2, 3, 128, 16, [130, 7], [130, 1000]),
    (1, 7, 64, 16, [200, 1, 77], [200, 513, 1000]),
    (1, 32, 64, 1024, [50], [2049]),
    (2, 1, 128, 32, [300, 280], [1300, 281]),
])
def test_window(Hkv, G, D, S, nqs, lens, window, sinks):
    g = _gen(sum(lens) + G + window)
    _check(*_case(g, Hkv, G, D, S, nqs, lens), window, sinks)


@pytest.mark.parametrize("window,sinks", [(1024, 4), (4000, 600), (20000, 0)])
def test_long_contexts(window, sinks):
    g = _gen(window)
    _check(*_case(g, 1, 8, 128, 64, [1, 6], [70001, 30000]), window, sinks)
    _check(*_case(g, 2, 4, 64, 64, [1500], [9000]), window, sinks)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,window", [(40, 100), (700, 30)])
def test_many_sequences(B, window, D):
    g = _gen(B + D)
    lens = [(i * 97) % 600 + 1 for i in range(B)]
    nqs = [min(1 + i % 5, n) for i, n in enumerate(lens)]
    _check(*_case(g, 1, 4, D, 16, nqs, lens), window, 5)


@pytest.mark.parametrize("sinks", [0, 2, 140])
@pytest.mark.parametrize("G,nq", [(1, 32), (1, 9), (4, 8), (1, 300)])
def test_scores_far_below_zero(G, nq, sinks):
    """Every score near -2700 or -90000: rows whose windows begin in a later unit than their tile's first one have seen
    nothing until then, and their exponents must come from what they see."""
    D, S, n, window = 128, 16, 700, 240
    for size in (3.0, 100.0):
        g = _gen(nq)
        q, cache, table, lens, nqs = _case(g, 1, G, D, S, [nq], [n])
        cache.k_codes.fill_(-1)      # every code 15: the value 7
        cache.k_scales.copy_((1 + torch.rand(cache.k_scales.shape, generator=g, device="cuda") / 64).bfloat16())
        q.fill_(-size)
        _check(q, cache, table, lens, nqs, window, sinks, scale=1.0)


@pytest.mark.parametrize("nq", [1, 5, 40, 300])
@pytest.mark.parametrize("huge", [2.0 ** 60, 2.0 ** -60])
def test_hidden_keys_of_other_sizes(nq, huge):
    """Keys that some rows see and some do not, with V scales far from the others'."""
    g = _gen(nq)
    q, cache, table, lens, nqs = _case(g, 2, 4, 128, 16, [nq], [1200])
    j = torch.arange(100, 1199 - nq, 7, device="cuda")
    cache.v_scales[table[0].long()[j // 16], :, j % 16] *= huge
    _check(q, cache, table, lens, nqs, 150, 3)


def test_a_wide_window_is_the_call_without_one():
    g = _gen(3)
    q, cache, table, lens, nqs = _case(g, 2, 4, 128, 32, [1, 70, 3], [900, 600, 77])
    cu = _i32(0, 1, 71, 74)
    for max_q in (1, 70):
        want = moe.moe_kv4_attention(q, cache, table, _i32(*lens), cu_q=cu, max_q=max_q, lse=True)
        for window, sinks in ((table.shape[1] * 32, 0), (2 ** 31 - 1, 5), (10, 2 ** 31 - 1)):
            got = moe.moe_kv4_attention_window(q, cache, table, _i32(*lens), window, sinks, cu_q=cu, max_q=max_q, lse=True)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        # a window that hides nothing from these lengths, through the window's own kernels
        out, lse = moe.moe_kv4_attention_window(q, cache, table, _i32(*lens), 900, 0, cu_q=cu, max_q=max_q, lse=True)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_rows_that_are_not_finite():
    g = _gen(4)
    for nq in (1, 6, 140):
        q, cache, table, lens, nqs = _case(g, 1, 4, 128, 16, [nq], [500])
        want, z = _run(q, cache, table, lens, nqs, 64, 2)
        at = 500 - nq - 10   # a key that the first queries see
        cache.v_scales[int(table[0, at // 16]), :, at % 16] = math.nan
        for max_q in (1, 4096):
            out, lse = _run(q, cache, table, lens, nqs, 64, 2, max_q=max_q)
            sees = _seen(500, nq, 64, 2)[:, at]
            assert out[sees].isnan().all() and lse[sees].isnan().all()
            assert not out[~sees].isnan().any()
            if (~sees).any():   # (the other kernel's roundings: two of bf16, and the probabilities')
                off = (out[~sees].double() - want[~sees].double()).abs()
                assert (off <= (2 * UB + 4 * U16) * want[~sees].double().abs() + 4 * U16 * 7 * 0.6).all()
        q[0, 1, 7] = math.inf
        out, _ = _run(q, cache, table, lens, nqs, 5, 0)   # (the key above is out of it)
        assert out[0, 1].isnan().all() and not out[0, [0, 2, 3]].isnan().any()


def test_a_page_out_of_range_is_an_error_only_where_it_is_seen():
    g = _gen(5)
    for nq in (1, 5, 70):
        for max_q in (1, 4096):
            q, cache, table, lens, nqs = _case(g, 2, 4, 64, 16, [nq], [1000])
            cu, ws = _i32(0, nq), moe.kv4_workspace(nq, 8, 2, 64)
            low = (1000 - nq - 100 + 1) // 16
            table[0, 1:low] = 1 << 30
            moe.moe_kv4_attention_window(q, cache, table, _i32(1000), 100, 16, cu_q=cu, max_q=max_q, ws=ws)
            assert moe.moe_check_device_error(ws) == 0
            table[0, low] = -5
            moe.moe_kv4_attention_window(q, cache, table, _i32(1000), 100, 16, cu_q=cu, max_q=max_q, ws=ws)
            assert moe.moe_check_device_error(ws) == 5


@pytest.mark.parametrize("max_q", [1, 4096])
def test_rows_behind_the_last_sequence_views_and_graphs(max_q):
    g = _gen(6)
    q, cache, table, lens, nqs = _case(g, 2, 3, 128, 16, [4, 60], [300, 900])
    wide = torch.zeros(70, 10, 128, dtype=torch.bfloat16, device="cuda")
    wide[:64, 2:8] = q
    out = torch.full((70, 6, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((70, 6), 7.0, device="cuda")
    ws = moe.kv4_workspace(70, 6, 2, 128)
    args = (cache, table, _i32(*lens), 100, 4)
    cu = _i32(0, 4, 64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            moe.moe_kv4_attention_window(wide[:, 2:8], *args, cu_q=cu, max_q=max_q, out=out, lse=lse, ws=ws)
    graph.replay()
    assert moe.moe_check_device_error(ws) == 0
    assert (out[64:] == 7).all() and (lse[64:] == 7).all()
    want, z = moe.moe_kv4_attention_window(q, *args, cu_q=cu, max_q=max_q, lse=True)
    assert torch.equal(out[:64], want) and torch.equal(lse[:64], z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_kv4_attention_window(q, *args, cu_q=cu, max_q=max_q, lse=True, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want) and torch.equal(got[1], z)

"""Attention over the 4-bit cache with a sliding window: what lies in keys that no query sees, but that share a run of 16
keys or a page with keys that one does, changes no bit of a result. Every case runs through both kernels. The results
over ordinary hidden keys are compared with the formula in 64 bits (the tolerances of test_gpu_kv4_window.py), those over
any other hidden keys with them, bit by bit."""
import math

import pytest
import torch

import w4a16_mixture_experts_gb300 as moe
from test_gpu_kv4 import _gen
from test_gpu_kv4_window import _case, _reference, _run, _seen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.lib()


FAR = (2.0 ** 120, -2.0 ** 120, 3e38, 2.0 ** -120, 1e-40, 0.0, 2.0 ** 12, 2.0 ** -12, math.nan, math.inf)


def _set(cache, table, keys, k=None, v=None):
    """Scales of the given keys of the (only) sequence."""
    page, off = table[0].long()[keys // cache.k_scales.shape[2]], keys % cache.k_scales.shape[2]
    if k is not None:
        cache.k_scales[page, :, off] = k
    if v is not None:
        cache.v_scales[page, :, off] = v


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,nq,n,window,sinks", [
    (4, 1, 1000, 100, 0),     # keys 896 to 899 lie in the first run that is read
    (4, 1, 1000, 100, 3),     # and 3 to 15 behind the first keys
    (8, 3, 777, 260, 130),
    (16, 2, 500, 33, 1),      # up to 32 rows a tile
    (1, 40, 641, 77, 17),
    (4, 300, 1500, 150, 5),   # several tiles of either kernel
    (7, 65, 3001, 1025, 0),
])
def test_hidden_keys_change_no_bit(G, nq, n, window, sinks, D):
    g = _gen(n + D)
    q, cache, table, lens, nqs = _case(g, 2, G, D, 16, [nq], [n])
    hidden = (~_seen(n, nq, window, sinks).any(0)).nonzero().squeeze(1)
    assert hidden.numel() > 0
    want, z, tol, ltol = _reference(q, cache, table, lens, nqs, D ** -0.5, window, sinks)
    for max_q in (1, nq, 4096):
        _set(cache, table, hidden, 0.4, 0.4)
        first = _run(q, cache, table, lens, nqs, window, sinks, max_q=max_q)
        assert ((first[0].double() - want).abs() <= tol).all() and ((first[1].double() - z).abs() <= ltol).all()
        for far in FAR:
            for k, v in ((0.4, far), (far, 0.4), (far, far)):
                _set(cache, table, hidden, k, v)
                got = _run(q, cache, table, lens, nqs, window, sinks, max_q=max_q)
                assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1]), (max_q, far, k, v)


@pytest.mark.parametrize("D", [64, 128])
def test_keys_that_other_rows_see_change_no_bit_of_a_tile_that_does_not(D):
    # 600 rows of one head, those of the middle tile of 256 at the positions 556 to 811: key 353 is out of its windows, but
    # in a run of 16 that it reads, key 820 behind its last row, but in its last 128 keys; its tiles of 8 too see neither
    g = _gen(D)
    n, nq, window = 900, 600, 200
    q, cache, table, lens, nqs = _case(g, 1, 1, D, 16, [nq], [n])
    ends = torch.tensor([353, 820], device="cuda")
    for max_q in (1, 4096):
        middle = slice(256, 512)
        _set(cache, table, ends, 0.4, 0.4)
        first = _run(q, cache, table, lens, nqs, window, 0, max_q=max_q)
        for far in FAR:
            _set(cache, table, ends, far, far)
            got = _run(q, cache, table, lens, nqs, window, 0, max_q=max_q)
            assert torch.equal(got[0][middle], first[0][middle]) and torch.equal(got[1][middle], first[1][middle]), (max_q, far)


@pytest.mark.parametrize("nq", [1, 300])
def test_a_cache_that_was_filled_from_the_window_on(nq):
    """The rows before the window are those that kv4_cache makes: zeros."""
    g = _gen(nq)
    n, window = 2000, 400
    q, cache, table, lens, nqs = _case(g, 2, 4, 128, 64, [nq], [n])
    hidden = (~_seen(n, nq, window, 0).any(0)).nonzero().squeeze(1)
    want, z, tol, ltol = _reference(q, cache, table, lens, nqs, 128 ** -0.5, window, 0)
    page, off = table[0].long()[hidden // 64], hidden % 64
    tensors = (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales)
    for max_q in (1, 4096):
        first = _run(q, cache, table, lens, nqs, window, 0, max_q=max_q)
        kept = [t[page, :, off] for t in tensors]
        for t in tensors:
            t[page, :, off] = 0
        got = _run(q, cache, table, lens, nqs, window, 0, max_q=max_q)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
        assert ((got[0].double() - want).abs() <= tol).all() and ((got[1].double() - z).abs() <= ltol).all()
        for t, old in zip(tensors, kept):
            t[page, :, off] = old


def test_windows_past_32_bits_hide_nothing_and_negative_ones_are_refused():
    g = _gen(8)
    q, cache, table, lens, nqs = _case(g, 2, 4, 64, 16, [3], [300])
    want = _run(q, cache, table, lens, nqs, 2 ** 31 - 1, 0)
    for window, sinks in ((2 ** 32 + 5, 0), (2 ** 32, 0), (2 ** 40, 0), (5, 2 ** 32 + 1), (5, 2 ** 33)):
        got = _run(q, cache, table, lens, nqs, window, sinks)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (window, sinks)
    for window, sinks in ((5 - 2 ** 32, 0), (0, 0), (5, 1 - 2 ** 32), (5, -1)):
        with pytest.raises(moe.MoeError) as e:
            _run(q, cache, table, lens, nqs, window, sinks)
        assert e.value.status == 1

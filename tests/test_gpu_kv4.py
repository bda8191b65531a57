"""The attention block on the GPU, against its formulas in 64 bits: per-head norms with the rotary turn,
rows of the 4-bit cache, and attention over it.

Tolerances. A rounding to a type is off by at most half a step, u(t) = finfo(t).eps / 2 relative to the
value. With A = sum_j p_j |v_j| (the mass an output is made of) and Q = max_j scale * sum_d |q_d k_jd|:
 - a score is a sum of D exact products, so it is off by at most D * 2 u(fp32) * Q (a tensor core may cut
   off instead of rounding: a whole step an addition), and a probability by that, relative;
 - a probability enters the tensor core in fp16: u(fp16), and 2^-25 absolute against a largest of 1;
 - n additions in fp32: n * 2 u(fp32) of A at most;
 - the output is rounded to bf16 once: u(bf16) of itself.
The log-sum-exp has the first and the third, and its own rounding.
"""
import math

import pytest
import torch

import w4a16_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu

U16, UB, U32 = (torch.finfo(t).eps / 2 for t in (torch.float16, torch.bfloat16, torch.float32))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.lib()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


# ---- norms and the rotary turn -------------------------------------------------------------------------------

def _turned(x, w, pos, freq, eps, interleaved):
    """(result, |a| + |b| of each value's pair) in 64 bits."""
    x = x.double()
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        y = y * w.double()
    mass = y.abs()
    if freq is None:
        return y, mass
    rot = 2 * freq.numel()
    theta = (pos.double()[:, None] * freq.double())[:, None]
    c, s = theta.cos(), theta.sin()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    out, both = y.clone(), a.abs() + b.abs()
    mass = mass.clone()
    if interleaved:
        out[..., 0:rot:2], out[..., 1:rot:2] = a * c - b * s, a * s + b * c
        mass[..., 0:rot:2], mass[..., 1:rot:2] = both, both
    else:
        out[..., :rot // 2], out[..., rot // 2:rot] = a * c - b * s, a * s + b * c
        mass[..., :rot // 2], mass[..., rot // 2:rot] = both, both
    return out, mass


def _near_turned(got, x, w, pos, freq, eps, interleaved):
    want, mass = _turned(x, w, pos, freq, eps, interleaved)
    # half the row's squares are summed one after another at most, sixteen roundings follow
    tol = UB * want.abs() + (x.shape[-1] / 2 + 16) * U32 * mass
    off = (got.double() - want).abs()
    assert (off <= tol).all(), float((off - tol).max())


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,interleaved,far", [
    (1, 32, 4, 128, 128, False, 1 << 20),
    (3, 7, 1, 64, 64, True, 1 << 31),
    (5, 8, 8, 256, 64, False, 4096),
    (777, 12, 4, 128, 32, True, 1 << 17),
    (1300, 5, 5, 64, 16, False, 1 << 20),
    (333, 24, 2, 256, 256, True, 1 << 24),
    (2049, 3, 1, 128, 96, False, 1 << 16),
    (17, 33, 1, 64, 48, False, 1 << 10),
])
def test_norm_rope(T, Hq, Hkv, D, rot, interleaved, far):
    g = _gen(T * 131 + D)
    qkv = (_randn(g, T, (Hq + 2 * Hkv) * D) * 2).bfloat16()
    q, k = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    pos = torch.randint(0, far, (T,), generator=g, device="cuda").to(torch.int32)
    pos[-1] = far - 1
    freq = (1e6 ** (-torch.arange(0, rot, 2, device="cuda").double() / rot)).float()
    qw, kw = (1 + 0.3 * _randn(g, D)).bfloat16(), (1 + 0.3 * _randn(g, D)).bfloat16()
    qo, ko = moe.moe_qk_norm_rope(q, k, pos, freq, qw, kw, interleaved=interleaved)
    _near_turned(qo, q, qw, pos, freq, 1e-6, interleaved)
    _near_turned(ko, k, kw, pos, freq, 1e-6, interleaved)
    # the same bits in place, through strides
    want_q, want_k = qo.clone(), ko.clone()
    rest = qkv[:, (Hq + Hkv) * D:].clone()
    moe.moe_qk_norm_rope(q, k, pos, freq, qw, kw, interleaved=interleaved, q_out=q, k_out=k)
    assert torch.equal(q, want_q) and torch.equal(k, want_k)
    assert torch.equal(qkv[:, (Hq + Hkv) * D:], rest)


def test_norm_rope_without_turn_or_weights():
    g = _gen(4)
    q, k = _randn(g, 9, 4, 128).bfloat16(), _randn(g, 9, 2, 128).bfloat16()
    q[2] = 0
    qo, ko = moe.moe_qk_norm_rope(q, k, None, None, eps=1e-5)
    _near_turned(qo, q, None, None, None, 1e-5, False)
    _near_turned(ko, k, None, None, None, 1e-5, False)
    assert (qo[2] == 0).all()


def test_norm_rope_negative_and_extreme_positions():
    g = _gen(5)
    pos = torch.tensor([0, -1, -(1 << 31), (1 << 31) - 1, 123456789], dtype=torch.int32, device="cuda")
    q, k = _randn(g, 5, 2, 64).bfloat16(), _randn(g, 5, 1, 64).bfloat16()
    freq = (1e4 ** (-torch.arange(0, 64, 2, device="cuda").double() / 64)).float()
    qo, ko = moe.moe_qk_norm_rope(q, k, pos, freq)
    _near_turned(qo, q, None, pos, freq, 1e-6, False)
    _near_turned(ko, k, None, pos, freq, 1e-6, False)


def test_norm_rope_rows_do_not_share_nan():
    g = _gen(6)
    q, k = _randn(g, 40, 6, 128).bfloat16(), _randn(g, 40, 2, 128).bfloat16()
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    freq = torch.full((64,), 0.1, device="cuda")
    clean, _ = moe.moe_qk_norm_rope(q, k, pos, freq)
    q[7, 3, 5] = float("nan")
    q[8, 0, 0] = float("inf")
    dirty, _ = moe.moe_qk_norm_rope(q, k, pos, freq)
    assert dirty[7, 3].isnan().all() and dirty[8, 0].isnan().any()
    clean[7, 3] = dirty[7, 3] = 0
    clean[8, 0] = dirty[8, 0] = 0
    assert torch.equal(clean, dirty)


# ---- rows of the cache ----------------------------------------------------------------------------------------

def _unpack(words, scales):
    n = torch.stack([(words >> (4 * i)) & 15 for i in range(8)], -1).flatten(-2) - 8
    return n.double() * scales.double().unsqueeze(-1)


def _quantised(x):
    """(codes - 8, scales) by the formula, in the fp32 steps it names."""
    x = x.float()
    s = (x.abs().amax(-1) / 7).bfloat16()
    f = s.float().unsqueeze(-1)
    return torch.where(f == 0, torch.zeros_like(x), (x / f).round().clamp(-8, 7)), s


def _rows(words):
    return torch.stack([(words >> (4 * i)) & 15 for i in range(8)], -1).flatten(-2) - 8


@pytest.mark.parametrize("T,Hkv,D,S", [(1, 1, 64, 16), (1, 8, 128, 1024), (37, 3, 128, 32), (500, 4, 64, 64), (4099, 2, 128, 128)])
def test_append_and_read(T, Hkv, D, S):
    g = _gen(T + Hkv)
    kv = (_randn(g, T, 2, Hkv, D) * 10 ** (_randn(g, T, 2, Hkv, 1) * 2)).bfloat16()
    kv[0, 0, 0] = 0                                   # a row of zeros
    if T > 30:
        kv[5, 1, 0] = 1e-40                           # subnormal values
        kv[6, 0, 1, 3] = 3e38                         # the largest scale
        kv[7, 0, 0] = torch.arange(D, device="cuda").bfloat16() * 0.5 - 3.5   # ties
    k, v = kv[:, 0], kv[:, 1]
    n = -(-T // S) + 3
    cache = moe.kv4_cache(n, Hkv, S, D)
    before = [t.clone() for t in cache]
    slots = torch.randperm(n * S, generator=g, device="cuda")[:T].to(torch.int32)
    if T > 4:
        slots[3] = -1
    ws = moe.kv4_workspace()
    moe.moe_kv4_append(k, v, slots, cache, ws=ws)
    assert moe.moe_check_device_error(ws) == 0
    kept = slots >= 0
    page, off = slots[kept].long() // S, slots[kept].long() % S
    for x, codes, scales in ((k, cache.k_codes, cache.k_scales), (v, cache.v_codes, cache.v_scales)):
        q, s = _quantised(x[kept])
        assert torch.equal(_rows(codes[page, :, off]).float(), q)
        assert torch.equal(scales[page, :, off], s)
    # nothing else was written
    for old, new in zip(before, cache):
        untouched = torch.ones(n, S, dtype=torch.bool, device="cuda")
        untouched[page, off] = False
        assert torch.equal(old.transpose(1, 2)[untouched], new.transpose(1, 2)[untouched])
    ko, vo = moe.moe_kv4_read(slots, cache, ws=ws)
    for x, o in ((k, ko), (v, vo)):
        q, s = _quantised(x)
        want = (q * s.float().unsqueeze(-1)).bfloat16()
        want[~kept] = 0
        assert torch.equal(o, want)


def test_append_is_the_quantiser_without_its_search():
    g = _gen(9)
    x = _randn(g, 64, 4, 128).bfloat16()
    cache = moe.kv4_cache(4, 4, 16, 128)
    slots = torch.arange(64, dtype=torch.int32, device="cuda")
    moe.moe_kv4_append(x, x, slots, cache)
    packed, scales = moe.moe_quantize_int4(x.view(256, 128), nclip=1)
    got = cache.k_codes.transpose(1, 2).reshape(256, 16)
    assert torch.equal(got, packed)
    assert torch.equal(cache.v_scales.transpose(1, 2).reshape(256), scales.view(-1))


def test_append_rows_that_are_not_finite():
    g = _gen(10)
    x = _randn(g, 8, 2, 64).bfloat16()
    x[2, 1, 9] = float("nan")
    x[5, 0, 0] = -float("inf")
    cache = moe.kv4_cache(1, 2, 16, 64)
    slots = torch.arange(8, dtype=torch.int32, device="cuda")
    moe.moe_kv4_append(x, x, slots, cache)
    bad = cache.k_scales[0, :, :8].isnan().T
    want = torch.zeros(8, 2, dtype=torch.bool, device="cuda")
    want[2, 1] = want[5, 0] = True
    assert torch.equal(bad, want) and torch.equal(cache.v_scales[0, :, :8].isnan().T, want)
    ko, _ = moe.moe_kv4_read(slots, cache)
    assert torch.equal(ko.isnan().all(-1), want) and torch.equal(ko.isnan().any(-1), want)


def test_slots_outside_the_cache():
    g = _gen(11)
    x = _randn(g, 6, 2, 64).bfloat16()
    cache = moe.kv4_cache(2, 2, 16, 64)
    before = [t.clone() for t in cache]
    ws = moe.kv4_workspace()
    out_of_it = torch.tensor([32, -2, 1 << 30, -(1 << 31), (1 << 31) - 1, -1], dtype=torch.int32, device="cuda")
    moe.moe_kv4_append(x, x, out_of_it, cache, ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(before, cache))
    assert moe.moe_check_device_error(ws) == 5 and moe.moe_check_device_error(ws) == 0
    ko, vo = moe.moe_kv4_read(out_of_it, cache, ws=ws)
    assert (ko == 0).all() and (vo == 0).all() and moe.moe_check_device_error(ws) == 5


# ---- attention ------------------------------------------------------------------------------------------------

def _filled(g, pages, Hkv, S, D):
    cache = moe.kv4_cache(pages, Hkv, S, D)
    for codes, scales in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        w = torch.zeros_like(codes)
        for i in range(8):
            w |= ((_randn(g, *codes.shape) * 2.4).round().clamp(-8, 7).to(torch.int32) + 8) << (4 * i)
        codes.copy_(w)
        scales.copy_((0.25 + 0.35 * torch.rand(scales.shape, generator=g, device="cuda")).bfloat16())
    return cache


def _tables(g, lens, S, pages, M=None):
    used = [-(-max(n, 0) // S) for n in lens]
    M = M or max(max(used), 1)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    assert sum(used) <= pages
    table = torch.full((len(lens), M), -1, dtype=torch.int32, device="cuda")   # unused entries are never followed
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    return table


def _reference(q, cache, table, lens, nqs, scale):
    """out, lse, and each output's tolerance and each lse's, in 64 bits."""
    T, Hq, D = q.shape
    Hkv, S = cache.k_scales.shape[1:]
    G = Hq // Hkv
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    t = 0
    for b, (n, nq) in enumerate(zip(lens, nqs)):
        pages = table[b, :-(-n // S)].long() if n else table[b, :0].long()
        for h in range(Hkv):
            k = _unpack(cache.k_codes[pages, h], cache.k_scales[pages, h]).reshape(-1, D)[:n]
            v = _unpack(cache.v_codes[pages, h], cache.v_scales[pages, h]).reshape(-1, D)[:n]
            for i in range(nq):
                seen = n - nq + i + 1
                if seen <= 0:
                    continue
                x = q[t + i, h * G:(h + 1) * G].double()
                s = scale * (x @ k[:seen].T)
                p = torch.softmax(s, -1)
                z = torch.logsumexp(s, -1)
                mass = p @ v[:seen].abs()
                qk = (abs(scale) * (x.abs() @ k[:seen].abs().T)).amax(-1)
                ds = 2 * U32 * (D + 4) * qk
                o = p @ v[:seen]
                rows = slice(h * G, (h + 1) * G)
                out[t + i, rows], lse[t + i, rows] = o, z
                small = 2.0 ** -25 * v[:seen].abs().sum(0) / (s - s.amax(-1, keepdim=True)).exp().sum(-1, keepdim=True)
                tol[t + i, rows] = UB * o.abs() + (U16 + (2 * ds + 2 * U32 * (seen + 8)).unsqueeze(-1)) * mass + small
                ltol[t + i, rows] = ds + 2 * U32 * (seen + 8) + 2 * U32 * z.abs()
        t += nq
    return out, lse, tol, ltol


def _check(q, cache, table, lens, nqs, scale=None, cu=True, max_q=None, ws=None):
    T, Hq, D = q.shape
    Hkv = cache.k_scales.shape[1]
    scale = D ** -0.5 if scale is None else scale
    cu_q = torch.tensor([0] + list(torch.tensor(nqs).cumsum(0)), dtype=torch.int32, device="cuda") if cu else None
    ws = moe.kv4_workspace(T, Hq, Hkv, D) if ws is None else ws
    out, lse = moe.moe_kv4_attention(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), cu_q=cu_q,
                                     max_q=max(nqs) if max_q is None else max_q, scale=scale, lse=True, ws=ws)
    assert moe.moe_check_device_error(ws) == 0
    want, z, tol, ltol = _reference(q, cache, table, lens, nqs, scale)
    off = (out.double() - want).abs()
    assert (off <= tol).all(), (float((off - tol).max()), float((off / tol.clamp(min=1e-30)).max()))
    empty = z == -math.inf
    assert (lse[empty] == -math.inf).all() and (out[empty] == 0).all()
    off = (lse.double() - z)[~empty].abs()
    assert (off <= ltol[~empty]).all(), float((off - ltol[~empty]).max())
    return out, lse


@pytest.mark.parametrize("Hkv,G,D,S,nqs,lens", [
    (1, 1, 64, 16, [1], [1]),
    (1, 1, 128, 16, [1], [1]),
    (8, 4, 128, 16, [1], [500]),
    (2, 8, 128, 64, [1, 1, 1], [1, 64, 65]),
    (4, 7, 64, 32, [1] * 9, [0, 1, 15, 16, 17, 127, 128, 129, 2000]),     # a length of zero leaves its row empty
    (1, 3, 128, 1024, [1, 1], [1023, 1025]),
    (2, 16, 64, 16, [1] * 4, [4000, 3, 0, 900]),
    (1, 32, 128, 128, [1, 1], [700, 33]),
    (2, 12, 128, 16, [1], [3333]),
    (1, 1, 64, 16, [1] * 300, [(i * 37) % 211 for i in range(300)]),      # more sequences than SMs
])
def test_decode(Hkv, G, D, S, nqs, lens):
    g = _gen(sum(lens) + G)
    pages = sum(-(-n // S) for n in lens) + 5
    cache = _filled(g, pages, Hkv, S, D)
    table = _tables(g, lens, S, pages)
    q = (1.6 * _randn(g, sum(nqs), Hkv * G, D)).bfloat16()
    with_cu, _ = _check(q, cache, table, lens, nqs)
    without, _ = _check(q, cache, table, lens, nqs, cu=False)
    assert torch.equal(with_cu, without)


@pytest.mark.parametrize("Hkv,G,D,S,nqs,lens", [
    (2, 4, 128, 16, [5], [5]),
    (2, 4, 64, 16, [3, 1, 0, 8, 2], [100, 1, 50, 8, 700]),                # a sequence without queries
    (1, 8, 128, 32, [4, 4], [3, 1]),                                      # more queries than keys: empty rows
    (1, 5, 64, 64, [9, 2], [1000, 2]),
    (4, 1, 128, 16, [7] * 20, [(i * 91) % 400 + 7 for i in range(20)]),
    (1, 6, 128, 16, [33], [40]),
    (2, 8, 128, 64, [130], [130]),
    (1, 7, 64, 16, [200, 1, 77], [200, 513, 1000]),
    (2, 3, 128, 128, [257, 40], [700, 40]),
    (1, 16, 64, 32, [65, 0, 300], [64, 0, 299]),                          # a first row that sees nothing
    (1, 32, 128, 16, [50], [2049]),
    (8, 1, 64, 16, [300, 280], [1300, 281]),
])
def test_several_queries(Hkv, G, D, S, nqs, lens):
    g = _gen(sum(lens) + G)
    pages = sum(-(-n // S) for n in lens) + 5
    cache = _filled(g, pages, Hkv, S, D)
    table = _tables(g, lens, S, pages, M=-(-max(lens) // S) + 3)
    q = (1.6 * _randn(g, sum(nqs), Hkv * G, D)).bfloat16()
    ws = moe.kv4_workspace(sum(nqs), Hkv * G, Hkv, D)
    _check(q, cache, table, lens, nqs, ws=ws)
    # whichever kernel max_q chooses
    _check(q, cache, table, lens, nqs, max_q=1, ws=ws)
    _check(q, cache, table, lens, nqs, max_q=4096, ws=ws)


def test_long_context():
    g = _gen(21)
    lens, S, Hkv, G, D = [70001], 64, 1, 8, 128
    cache = _filled(g, 1100, Hkv, S, D)
    table = _tables(g, lens, S, 1100)
    q = (1.6 * _randn(g, 1, Hkv * G, D)).bfloat16()
    _check(q, cache, table, lens, [1])
    q = (1.6 * _randn(g, 6, Hkv * G, D)).bfloat16()
    _check(q, cache, table, lens, [6])


@pytest.mark.parametrize("nq", [1, 5, 300])
def test_far_offsets(nq):
    # rows whose byte offsets pass 32 bits
    g = _gen(22)
    Hkv, G, D, S = 8, 4, 128, 1024
    pages = 9000                                       # 4.7 GB of codes each
    cache = moe.Kv4Cache(*(torch.empty(pages, Hkv, S, D // 8, dtype=torch.int32, device="cuda") if i % 2 == 0 else
                           torch.empty(pages, Hkv, S, dtype=torch.bfloat16, device="cuda") for i in range(4)))
    small = _filled(g, 2, Hkv, S, D)
    for big, few in zip(cache, small):
        big[-2:] = few
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    near = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    q = (1.6 * _randn(g, nq, Hkv * G, D)).bfloat16()
    lens = torch.tensor([1500], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, nq], dtype=torch.int32, device="cuda")
    a = moe.moe_kv4_attention(q, cache, table, lens, cu_q=cu, max_q=nq)
    b = moe.moe_kv4_attention(q, small, near, lens, cu_q=cu, max_q=nq)
    assert torch.equal(a, b)
    x = _randn(g, 3, Hkv, D).bfloat16()
    slots = torch.tensor([pages * S - 1, 8191 * S + 5, 0], dtype=torch.int32, device="cuda")
    moe.moe_kv4_append(x, x, slots, cache)
    k, v = moe.moe_kv4_read(slots, cache)
    qq, s = _quantised(x)
    assert torch.equal(k, (qq * s.float().unsqueeze(-1)).bfloat16()) and torch.equal(k, v)


@pytest.mark.parametrize("nq", [1, 6, 140])
def test_rows_that_are_not_finite_reach_only_who_sees_them(nq):
    g = _gen(23)
    Hkv, G, D, S, n = 2, 4, 128, 16, 300
    cache = _filled(g, 40, Hkv, S, D)
    table = _tables(g, [n], S, 40, M=30)
    table[table < 0] = 0
    q = (1.6 * _randn(g, nq, Hkv * G, D)).bfloat16()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, nq], dtype=torch.int32, device="cuda")
    # behind the last key of its page: nobody sees it
    page, off = int(table[0, (n - 1) // S]), n % S
    clean, lse = moe.moe_kv4_attention(q, cache, table, lens, cu_q=cu, max_q=nq, lse=True)
    for s in (cache.k_scales, cache.v_scales):
        s[page, :, off:] = float("nan")
    again = moe.moe_kv4_attention(q, cache, table, lens, cu_q=cu, max_q=nq)
    assert torch.equal(clean, again)
    # the last key: only the last query sees it, and only its head
    page, off = int(table[0, (n - 1) // S]), (n - 1) % S
    for which, bits in ((cache.k_scales, float("nan")), (cache.v_scales, float("inf"))):
        old = which[page, 1, off].clone()
        which[page, 1, off] = bits
        got, z = moe.moe_kv4_attention(q, cache, table, lens, cu_q=cu, max_q=nq, lse=True)
        which[page, 1, off] = old
        assert got[-1, G:].isnan().all() and z[-1, G:].isnan().all()
        assert torch.equal(got[:-1], clean[:-1]) and torch.equal(got[-1, :G], clean[-1, :G])
        assert torch.equal(z[:-1], lse[:-1])


@pytest.mark.parametrize("nq", [1, 6, 140])
def test_large_and_small_magnitudes(nq):
    g = _gen(24)
    Hkv, G, D, S, n = 1, 8, 128, 16, 700
    for qmul, kmul, vmul in ((1e3, 1e-3, 1e-6), (1e-3, 1e4, 1e5), (3e4, 1e-6, 1.0), (1e-20, 1e20, 1e-20), (1.0, 1.0, 1e30)):
        cache = _filled(g, 50, Hkv, S, D)
        cache.k_scales.mul_(kmul)
        cache.v_scales.mul_(vmul)
        table = _tables(g, [n], S, 50)
        q = (1.6 * qmul * _randn(g, nq, Hkv * G, D)).bfloat16()
        _check(q, cache, table, [n], [nq], scale=0.09 / (qmul * kmul))


@pytest.mark.parametrize("nq", [1, 6, 140])
def test_peaked_rows(nq):
    # scores hundreds apart: the running maximum moves by far in some tiles
    g = _gen(25)
    Hkv, G, D, S, n = 2, 4, 64, 32, 1500
    cache = _filled(g, 60, Hkv, S, D)
    table = _tables(g, [n], S, 60)
    _check((40 * _randn(g, nq, Hkv * G, D)).bfloat16(), cache, table, [n], [nq])
    # zero queries: the mean of what is seen
    _check(torch.zeros(nq, Hkv * G, D, dtype=torch.bfloat16, device="cuda"), cache, table, [n], [nq])


@pytest.mark.parametrize("nq", [1, 6, 140])
def test_zero_rows(nq):
    g = _gen(26)
    Hkv, G, D, S, n = 1, 4, 128, 16, 400
    cache = _filled(g, 30, Hkv, S, D)
    cache.v_scales.zero_()
    cache.k_scales[::2].zero_()
    table = _tables(g, [n], S, 30)
    out, _ = _check((1.6 * _randn(g, nq, Hkv * G, D)).bfloat16(), cache, table, [n], [nq])
    assert (out == 0).all()


@pytest.mark.parametrize("nq", [1, 4, 150])
def test_strides_streams_and_repeats(nq):
    g = _gen(27)
    Hkv, G, D, S, B = 2, 4, 128, 16, 3
    lens = [900, 150, 333]
    cache = _filled(g, 100, Hkv, S, D)
    table = _tables(g, lens, S, 100)
    T, Hq = B * nq, Hkv * G
    # query and gate of a head side by side; out as heads first
    wide = (1.6 * _randn(g, T, Hq, 2, D)).bfloat16()
    q = wide[:, :, 0]
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = torch.arange(0, T + 1, nq, dtype=torch.int32, device="cuda")
    ws = moe.kv4_workspace(T, Hq, Hkv, D)
    plain = moe.moe_kv4_attention(q.contiguous(), cache, table, lens_t, cu_q=cu, max_q=nq, ws=ws)
    out = torch.full((Hq, T, D), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    moe.moe_kv4_attention(q, cache, table, lens_t, cu_q=cu, max_q=nq, out=out, ws=ws)
    assert torch.equal(out, plain)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            again = moe.moe_kv4_attention(q, cache, table, lens_t, cu_q=cu, max_q=nq, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again, plain)
    graph = torch.cuda.CUDAGraph()
    held = torch.empty_like(plain)
    with torch.cuda.graph(graph):
        moe.moe_kv4_attention(q, cache, table, lens_t, cu_q=cu, max_q=nq, out=held, ws=ws)
    # lengths and tables may change between replays
    for _ in range(2):
        held.zero_()
        graph.replay()
        assert torch.equal(held, plain)
    lens_t.copy_(torch.tensor([500, 150, 200], device="cuda"))
    graph.replay()
    want = moe.moe_kv4_attention(q, cache, table, lens_t, cu_q=cu, max_q=nq, ws=ws)
    assert torch.equal(held, want) and not torch.equal(held, plain)
    assert moe.moe_check_device_error(ws) == 0


def test_values_out_of_range_are_reported():
    g = _gen(28)
    Hkv, G, D, S = 2, 2, 64, 16
    cache = _filled(g, 10, Hkv, S, D)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for nq in (1, 40):
        T = 2 * nq
        q = _randn(g, T, Hkv * G, D).bfloat16()
        table = torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5)
        cu = i32(0, nq, T)
        ws = moe.kv4_workspace(T, Hkv * G, Hkv, D)
        good = moe.moe_kv4_attention(q, cache, table, i32(80, 70), cu_q=cu, max_q=nq, ws=ws)
        assert moe.moe_check_device_error(ws) == 0
        # a bad page: its rows read as zero, the other sequence is as it was
        for page in (-1, 10, 1 << 30):
            t2 = table.clone()
            t2[0, 1] = page
            got = moe.moe_kv4_attention(q, cache, t2, i32(80, 70), cu_q=cu, max_q=nq, ws=ws)
            assert moe.moe_check_device_error(ws) == 5
            assert torch.equal(got[nq:], good[nq:]) and got.isfinite().all()
            zeroed = moe.Kv4Cache(*(x.clone() for x in cache))
            zeroed.k_scales[1], zeroed.v_scales[1] = 0, 0
            assert torch.equal(got, moe.moe_kv4_attention(q, zeroed, table, i32(80, 70), cu_q=cu, max_q=nq, ws=ws))
        # lengths beyond the table, or negative
        got = moe.moe_kv4_attention(q, cache, table, i32(80, 1 << 20), cu_q=cu, max_q=nq, ws=ws)
        assert moe.moe_check_device_error(ws) == 5
        assert torch.equal(got, moe.moe_kv4_attention(q, cache, table, i32(80, 80), cu_q=cu, max_q=nq, ws=ws))
        got = moe.moe_kv4_attention(q, cache, table, i32(-5, 70), cu_q=cu, max_q=nq, ws=ws)
        assert moe.moe_check_device_error(ws) == 5 and (got[:nq] == 0).all() and torch.equal(got[nq:], good[nq:])
        # query offsets outside the queries
        moe.moe_kv4_attention(q, cache, table, i32(80, 70), cu_q=i32(-3, nq, T + 9), max_q=nq, ws=ws)
        assert moe.moe_check_device_error(ws) == 5
        # and the workspace is as good as new
        assert torch.equal(good, moe.moe_kv4_attention(q, cache, table, i32(80, 70), cu_q=cu, max_q=nq, ws=ws))
        assert moe.moe_check_device_error(ws) == 0


def test_block_together_with_the_experts():
    """A decode step's attention block, then the MoE block, on one workspace: norms and turn, rows into the
    cache, attention, experts; the cache's rows and the attention's output by their formulas."""
    g = _gen(30)
    B, Hkv, G, D, S, H = 4, 2, 4, 64, 16, 512
    Hq = Hkv * G
    E, k, I = 16, 2, 128
    cache = _filled(g, 64, Hkv, S, D)
    lens = [33, 100, 16, 1]
    table = _tables(g, lens, S, 64, M=8)
    table[table < 0] = 0
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.zeros(max(moe.kv4_workspace(B, Hq, Hkv, D).numel(), moe.moe_workspace_size(B, H, E, k, I)),
                     dtype=torch.uint8, device="cuda")
    qkv = _randn(g, B, (Hq + 2 * Hkv) * D).bfloat16()
    pos = lens_t - 1
    freq = (1e4 ** (-torch.arange(0, D, 2, device="cuda").double() / D)).float()
    slots = (table.gather(1, (pos // S).long().unsqueeze(1)).squeeze(1) * S + pos % S).to(torch.int32)
    rw = _randn(g, E, H).bfloat16() / H ** 0.5
    w1 = torch.randint(-2 ** 31, 2 ** 31 - 1, (E, 2 * I, H // 8), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    w2 = torch.randint(-2 ** 31, 2 ** 31 - 1, (E, H, I // 8), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    s1 = torch.full((E, 2 * I, H // 128), 0.01, dtype=torch.bfloat16, device="cuda")
    s2 = torch.full((E, H, I // 128), 0.01, dtype=torch.bfloat16, device="cuda")
    outs = []
    for _ in range(2):
        x = qkv.clone()
        q, kk, v = x[:, :Hq * D].view(B, Hq, D), x[:, Hq * D:(Hq + Hkv) * D].view(B, Hkv, D), x[:, (Hq + Hkv) * D:].view(B, Hkv, D)
        moe.moe_qk_norm_rope(q, kk, pos, freq, q_out=q, k_out=kk)
        moe.moe_kv4_append(kk, v, slots, cache, ws=ws)
        att = moe.moe_kv4_attention(q, cache, table, lens_t, ws=ws)
        out, ids, w = moe.moe_layer_forward(att.view(B, H), rw, k, w1, s1, w2, s2, ws=ws)
        outs.append((att, out, ids, w))
    assert moe.moe_check_device_error(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    want, _, tol, _ = _reference(q, cache, table, lens, [1] * B, D ** -0.5)
    assert ((att.double() - want).abs() <= tol).all()
    got, _ = moe.moe_kv4_read(slots, cache)
    qq, s = _quantised(kk)
    assert torch.equal(got, (qq * s.float().unsqueeze(-1)).bfloat16())

"""The verification of drafted tokens on the GPU, against its definition in 64 bits, sequence by sequence.

The results are whole numbers and have to be equal. They are decided by comparisons of numbers that the sums of
exponentials scale: a row's sum has an error of a few 2^-24 of itself (each fp32 exponential is off by 2^-21 at most, and its
argument by 2^-24 of up to 90: 2^-17 for terms that are 2^-90 of the largest, less for larger ones). A decision is taken for
clear where its sides differ by more than 2^-18 of the larger weights: the inputs are drawn until all are.
"""
import pytest
import torch

import w4a16_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu

CLEAR = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.lib()


def _definition(logits, drafts, rows, uniform, noise, draft, temperature):
    """(tokens, accepted, whether every decision is clear) in 64 bits, on the CPU."""
    logits, noise = logits.double().cpu(), noise.double().cpu()
    draft = None if draft is None else draft.double().cpu()
    drafts, uniform, temperature = drafts.tolist(), uniform.double().tolist(), temperature.tolist()
    tokens, accepted, clear, at = [], [], True, 0
    for b, n in enumerate(rows):
        if n == 0:
            accepted.append(0)
            continue
        t, a = temperature[b], 0
        while True:
            row, last, x = logits[at + a], a == n - 1, drafts[at + a]
            if t == 0:
                chosen = int((row == row.max()).nonzero()[0])
                if last or x != chosen:
                    break
            else:
                p = torch.softmax(row / t, 0)
                q = torch.zeros_like(p)
                if not last and draft is not None:
                    q = torch.softmax(draft[at + a] / t, 0)
                elif not last and 0 <= x < len(q):
                    q[x] = 1
                if last:
                    keep = False
                else:
                    inside = 0 <= x < len(q)
                    keep = inside and uniform[at + a] * float(q[x]) < float(p[x])
                    if inside:
                        clear &= abs(uniform[at + a] * float(q[x]) - float(p[x])) > CLEAR * float(p[x]) or float(p[x]) == 0
                if not keep:
                    r = (p - q).clip(min=0)
                    if not bool((r > 0).any()):
                        r = p
                    e = noise[b].clip(min=2.0 ** -126)
                    score = torch.where(r > 0, r / e, torch.full_like(r, -1))
                    chosen = int(score.argmax())
                    # how far each may move: by CLEAR of p and q, not of their difference
                    off = CLEAR * (p + q) / e
                    other = torch.where((p > 0) | (r > 0), score.clip(min=0) + off, torch.zeros_like(score))
                    other[chosen] = 0
                    clear &= bool(other.max() < score[chosen] - off[chosen]) or len(p) == 1
                    break
            a += 1
        tokens += drafts[at: at + a] + [chosen] + [-1] * (n - a - 1)
        accepted.append(a)
        at += n
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(accepted, dtype=torch.int32), clear


def _inputs(rows, V, with_q, greedy, seed, spread=2.0, apart=0.6, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, B = sum(rows), len(rows)
    pitch = -(-V // 8) * 8 + pad
    l = torch.randn(T, pitch, generator=g, device="cuda") * spread
    if V > 64:
        l.scatter_add_(1, torch.randint(0, V, (T, 8), generator=g, device="cuda"), 3 + 9 * torch.rand(T, 8, generator=g, device="cuda"))
    d = l + apart * torch.randn(T, pitch, generator=g, device="cuda")
    logits, draft = l.bfloat16()[:, :V], d.bfloat16()[:, :V]
    temperature = 0.5 + torch.rand(B, generator=g, device="cuda")
    temperature[torch.rand(B, generator=g, device="cuda") < greedy] = 0
    of = torch.repeat_interleave(torch.arange(B), torch.tensor(rows)).cuda()
    e = torch.empty(T, V, device="cuda").exponential_(generator=g)
    t = temperature[of].unsqueeze(1) if T else torch.ones(0, 1, device="cuda")
    drafts = (draft.float() / t.clamp(min=1e-3) - e.log()).argmax(1).to(torch.int32)
    noise = torch.empty(B, -(-V // 4) * 4 + pad, device="cuda").exponential_(generator=g)[:, :V]
    cu = torch.tensor([0] + rows).cumsum(0).to(torch.int32).cuda()
    return dict(logits=logits, drafts=drafts, cu=cu, uniform=torch.rand(T, generator=g, device="cuda"), noise=noise,
                draft=draft if with_q else None, temperature=temperature)


def _call(i, **over):
    i = dict(i, **over)
    return moe.moe_verify_drafts(i["logits"], i["drafts"], i["cu"], i["uniform"], i["noise"], draft_logits=i["draft"],
                                 temperature=i["temperature"], tokens=i.get("tokens"), accepted=i.get("accepted"), ws=i.get("ws"))


def _compare(i, rows, ws=None):
    tokens, accepted, clear = _definition(i["logits"], i["drafts"], rows, i["uniform"], i["noise"], i["draft"], i["temperature"])
    if not clear:
        return False
    got = _call(i, ws=ws)
    assert torch.equal(got[1].cpu(), accepted)
    assert torch.equal(got[0].cpu(), tokens)
    return True


CASES = [
    ([1], 1), ([3], 1), ([2, 2], 2), ([1], 7), ([4], 8), ([5, 1, 0, 9], 9), ([2], 100), ([4, 4, 4], 1000), ([6] * 5, 8191), ([3, 7], 8192),
    ([3, 7], 8193), ([2, 0, 0, 5, 1], 50257), ([4], 32000), ([5] * 12, 100003), ([3, 3], 248320), ([1] * 70, 300), ([40, 70, 33], 500),
    ([0, 0], 64), ([1, 0] * 60, 40),
]


@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("rows,V", CASES)
def test_verify(rows, V, with_q):
    ws = moe.verify_workspace(len(rows), sum(rows), V)
    done = 0
    for seed in range(12):   # until three draws are clear
        i = _inputs(rows, V, with_q, (0, 0.4, 1)[seed % 3], 100 * V + seed, spread=(2.0, 0.3, 6.0)[seed % 3], pad=8 * (seed % 2))
        done += _compare(i, rows, ws)
        if done == 3:
            break
    assert done == 3
    assert moe.moe_check_device_error(ws) == 0


def test_distribution():
    # one row's next token over many draws: the target's probabilities, whatever the draft's
    V, n = 12, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    l, d = torch.randn(1, 16, generator=g, device="cuda").bfloat16(), torch.randn(1, 16, generator=g, device="cuda").bfloat16()
    p, q = torch.softmax(l[0, :V].double(), 0), torch.softmax(d[0, :V].double(), 0)
    counts = torch.zeros(V, device="cuda")
    for k in range(16):
        drafts = torch.zeros(2 * n, dtype=torch.int32, device="cuda")
        drafts[::2] = (q.log().float() - torch.empty(n, V, device="cuda").exponential_(generator=g).log()).argmax(1).to(torch.int32)
        t, _ = moe.moe_verify_drafts(l.repeat(2 * n, 1)[:, :V], drafts, torch.arange(0, 2 * n + 1, 2, dtype=torch.int32, device="cuda"),
                                     torch.rand(2 * n, generator=g, device="cuda"), torch.empty(n, V, device="cuda").exponential_(generator=g),
                                     draft_logits=d.repeat(2 * n, 1)[:, :V])
        counts += torch.bincount(t[::2].long(), minlength=V)
    N = counts.sum()
    # five standard deviations of a count
    assert ((counts / N - p).abs() < 5 * (p * (1 - p) / N).sqrt()).all()


def test_all_accepted_and_none():
    rows, V = [4, 4], 3000
    for with_q in (True, False):
        i = _inputs(rows, V, with_q, 0, 5)
        i["uniform"].zero_()   # u = 0: accepted wherever p > 0
        t, a = _call(i)
        assert a.tolist() == [3, 3] and t[:3].tolist() == i["drafts"][:3].tolist() and int(t[3]) >= 0
        if with_q:
            i["draft"] = i["logits"]   # the draft is the target: always accepted
            i["uniform"].fill_(1 - 2.0 ** -24)
            assert _call(i)[1].tolist() == [3, 3]
        i = _inputs(rows, V, with_q, 0, 6)
        i["logits"][torch.arange(8, device="cuda"), i["drafts"].long()] = -torch.inf   # tokens of probability zero
        t, a = _call(i)
        assert a.tolist() == [0, 0] and _compare(i, rows)
        assert int(t[0]) != int(i["drafts"][0]) and t[1:4].tolist() == [-1] * 3


def test_equal_distributions_that_refuse_fall_back_on_the_target():
    # u = 1 (outside its range, but defined): refused with p = q everywhere
    i = _inputs([2], 5000, True, 0, 1)
    i["draft"] = i["logits"]
    i["uniform"].fill_(1.0)
    t, a = _call(i)
    p = torch.softmax(i["logits"][0].double() / i["temperature"][0].double(), 0)
    assert a.tolist() == [0] and int(t[0]) == int((p / i["noise"][0].double()).argmax()) and int(t[1]) == -1


def test_ties_go_to_the_lowest():
    V = 20000
    for t in (0.0, 1.0):
        l = torch.zeros(1, V, dtype=torch.bfloat16, device="cuda")
        e = torch.ones(1, V, device="cuda")
        for at in (0, 7, 8191, 8192, 19999):
            l[0, :at] = -1
            l[0, at:] = 1
            tok, a = moe.moe_verify_drafts(l, torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                                           torch.zeros(1, device="cuda"), e, temperature=torch.tensor([t], device="cuda"))
            assert tok.tolist() == [at] and a.tolist() == [0]


def test_temperatures_at_the_ends_of_the_range():
    rows, V = [3], 2000
    for t in (1e-42, 1e-30, 1e-3, 100.0, 1e30, 3e38):
        for seed in range(20):
            i = _inputs(rows, V, True, 0, seed)
            i["temperature"].fill_(t)
            if _compare(i, rows):
                break
        else:
            raise AssertionError("no clear draw")


def test_far_apart_logits_and_noise():
    rows, V = [2, 2], 700
    i = _inputs(rows, V, True, 0, 2)
    i["logits"][0, 3], i["logits"][1] = 3e38, -3e38
    i["logits"][1, 5] = 3e38
    i["noise"][0, :] = 0        # counts as the smallest normal number
    i["noise"][1, 10:] = float("inf")
    i["noise"][1, :10] = float("nan")
    i["noise"][1, 4] = -1.0
    i["uniform"].fill_(0.999)
    t, a = _call(i)
    assert t[0] == 3 or (t[0] == i["drafts"][0] and t[1] == 5)
    j = dict(i, noise=torch.where(i["noise"] >= 2.0 ** -126, i["noise"], torch.full_like(i["noise"], 2.0 ** -126)))
    assert torch.equal(_call(j)[0], t)


def _error(i):
    B, T, V = i["cu"].shape[0] - 1, *i["logits"].shape
    ws = moe.verify_workspace(B, T, V)
    t, a = _call(i, ws=ws, tokens=torch.full((T,), -7, dtype=torch.int32, device="cuda"))
    return t.tolist(), a.tolist(), moe.moe_check_device_error(ws)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_rows_without_a_distribution(value):
    for greedy in (0, 1):
        i = _inputs([3, 3], 20000, True, greedy, 4)
        i["uniform"].zero_()
        if greedy:
            i["drafts"][:] = i["logits"].float().argmax(1)
        good = _error(i)
        assert good[2] == 0 and good[1] == [2, 2]
        i["logits"][1, 12345] = value
        t, a, err = _error(i)
        assert err == 5 and a == [1, 2] and t == [good[0][0], -1, -1] + good[0][3:]
        i["logits"][0, :] = -torch.inf
        t, a, err = _error(i)
        assert err == 5 and a == [0, 2] and t == [-1, -1, -1] + good[0][3:]
        if not greedy:
            i = _inputs([3, 3], 20000, True, 0, 4)
            i["uniform"].zero_()
            i["draft"][4, 1] = value
            t, a, err = _error(i)
            assert err == 5 and a == [2, 1] and t == good[0][:4] + [-1, -1]
        # behind a refusal nothing is looked at
        i = _inputs([4], 20000, True, greedy, 4)
        i["logits"][0, int(i["drafts"][0])] = -torch.inf
        i["logits"][2, 5] = value
        t, a, err = _error(i)
        assert err == 0 and a == [0] and t[1:] == [-1, -1, -1]


def test_drafts_temperatures_and_offsets_out_of_range():
    for with_q in (True, False):
        for x in (-1, 500, 2 ** 31 - 1, -2 ** 31):
            i = _inputs([3, 2], 500, with_q, 0, 8)
            i["uniform"].zero_()
            i["drafts"][1] = x
            t, a, err = _error(i)
            assert err == 5 and a[0] == 1 and 0 <= t[1] < 500 and t[2] == -1 and a[1] == 1
            want = _definition(i["logits"], i["drafts"], [3, 2], i["uniform"], i["noise"], i["draft"], i["temperature"])
            assert t == want[0].tolist()
            i["drafts"][1], i["drafts"][2] = 3, x   # a last row's draft is not read
            assert _error(i)[2] == 0
    for t in (-1.0, float("nan"), float("inf")):
        i = _inputs([3, 2], 500, True, 0, 8)
        i["temperature"][0] = t
        tok, a, err = _error(i)
        assert err == 5 and a[0] == 0 and tok[:3] == [-1, -1, -1] and tok[3] >= 0
    for cu in ([0, 9, 5], [-3, 2, 5], [4, 2, 5], [0, 3, 2 ** 31 - 1], [5, 4, 3]):
        i = _inputs([3, 2], 500, True, 0, 8)
        i["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        assert _error(i)[2] == 5


def test_rows_of_no_sequence_are_left_alone():
    i = _inputs([3, 2, 4], 500, True, 0, 9)
    i["cu"] = i["cu"][1:3].contiguous()   # the second sequence alone
    i["noise"], i["temperature"] = i["noise"][1:2], i["temperature"][1:2].contiguous()
    t, a, err = _error(i)
    assert err == 0 and t[:3] == [-7] * 3 and t[5:] == [-7] * 4 and min(t[3:5]) >= -1


def test_streams_graphs_and_a_shared_workspace():
    rows, V = [5, 3, 1], 30011
    i = _inputs(rows, V, True, 0.3, 10)
    want = _call(i)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_verify_drafts(i["logits"], i["drafts"], i["cu"], i["uniform"], i["noise"], i["draft"], i["temperature"], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    n = max(moe.moe_verify_workspace_size(3, 9, V), moe.moe_workspace_size(4, 256, 16, 2, 128))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    graph, out = torch.cuda.CUDAGraph(), [torch.zeros_like(x) for x in want]
    with torch.cuda.graph(graph):
        for _ in range(2):
            _call(i, ws=ws, tokens=out[0], accepted=out[1])
    for seed in (11, 12):
        j = _inputs(rows, V, True, 0.3, seed)
        for k in ("logits", "drafts", "uniform", "noise", "draft", "temperature"):
            i[k].copy_(j[k])
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, _call(i)))
    assert not ws[: 512 + 1024 * 128].any()


def test_refuses_other_layouts():
    i = _inputs([3, 2], 504, True, 0, 0)
    for bad in (dict(logits=i["logits"].float()), dict(logits=i["logits"].t()), dict(draft=i["draft"][:4]), dict(draft=i["draft"][:, :500]),
                dict(drafts=i["drafts"].long()), dict(drafts=i["drafts"][:3]), dict(uniform=i["uniform"].double()), dict(noise=i["noise"][:1]),
                dict(noise=i["noise"].bfloat16()), dict(temperature=i["temperature"][:1]), dict(cu=i["cu"][:0]),
                dict(tokens=torch.empty(4, dtype=torch.int32, device="cuda")), dict(accepted=torch.empty(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            _call(i, **bad)
    with pytest.raises(moe.MoeError) as e:   # rows that do not begin on 16 bytes
        _call(i, logits=i["logits"].float().bfloat16().repeat(1, 2)[:, 4:508], draft=None)
    assert e.value.status == 1
    odd = torch.zeros(5, 503, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoeError) as e:
        _call(i, logits=odd, draft=None, noise=i["noise"][:, :503])
    assert e.value.status == 1


def test_logits_past_32_bit_offsets():
    T, V = 9000, 260000   # 2.3e9 values
    l = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    hot = (torch.arange(T, device="cuda") * 7919) % V
    l[torch.arange(T, device="cuda"), hot] = 40.0
    cu = torch.tensor([0, 3, T - 4, T], dtype=torch.int32, device="cuda")
    drafts = hot.to(torch.int32)
    e = torch.ones(3, V, device="cuda")
    t, a = moe.moe_verify_drafts(l, drafts, cu, torch.full((T,), 0.5, device="cuda"), e)
    assert a.tolist() == [2, T - 8, 3] and torch.equal(t, drafts)

"""The operators of a step with drafted tokens, measured: linears with 4-bit weights, attention over a window of a
paged 4-bit cache, and the verification of the drafts.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits) or, where ``own`` is true,
through the library's entry points on the same tensors. Formats: a weight matrix [N, K] is int32 words [N, K / 8] of
eight codes q + 8 with q in [-8, 7], lowest nibble first, and a bf16 scale per 128 values of a row [N, K / 128]. The
cache keeps each row of D values of one (token, KV head) the same way with one scale a row: codes int32
[pages, Hkv, page_size, D / 8], scales bf16 [pages, Hkv, page_size], for K and for V; a sequence's rows are found
through its row of the page table.
"""
import math

import torch

own = False

# the largest listed cases' sizes: drawn ones cost no more
WEIGHTS = 248320 * 2560          # values of a weight matrix
PRODUCTS = 4001 * 5121 * 4096    # of a linear
LOGITS = 160 * 248320            # rows of them times the vocabulary
SCORES = 4096 * 32 * 16384       # (query row, key) pairs, hidden ones among them: the plain form holds them all
KEYS = 1 << 21                   # (token, KV head) rows of cache


# ---- the cases -------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token's query, key and value projection: latency
        dict(name="linear token", op="linear", T=1, N=5120, K=2560),
        # the head's logits of a few drafts of one sequence: bandwidth
        dict(name="linear head", op="linear", T=4, N=248320, K=2560),
        # an odd batch through a long reduction with few rows
        dict(name="linear down", op="linear", T=7, N=2560, K=10240),
        # a decode batch, ragged rows
        dict(name="linear batch", op="linear", T=100, N=10200, K=2560),
        # a prompt chunk, both sides ragged
        dict(name="linear prompt", op="linear", T=4001, N=5121, K=4096),
        # a server's decode batch whose layers see a short window and the first tokens
        dict(name="window decode", op="window", B=96, Hkv=4, G=8, D=128, S=64, nq=1, qvar=0, kv=12001, kvar=90, window=1024, sinks=4),
        # few sequences with a long context: most of it out of the window
        dict(name="window long", op="window", B=2, Hkv=8, G=7, D=128, S=32, nq=1, qvar=0, kv=131072, kvar=1, window=32768, sinks=130),
        # drafts under verification, small heads, no first tokens
        dict(name="window drafts", op="window", B=24, Hkv=8, G=4, D=64, S=16, nq=5, qvar=60, kv=2777, kvar=70, window=333, sinks=0),
        # a prompt chunk behind a long prefix
        dict(name="window prompt", op="window", B=1, Hkv=4, G=8, D=128, S=64, nq=4096, qvar=0, kv=12288, kvar=0, window=4096, sinks=64),
        # one sequence's drafts, a small vocabulary: latency
        dict(name="verify one", op="verify", B=1, n=3, nvar=0, V=32000, q=True, greedy=0),
        # a server's batch with the draft's probabilities, the head's full width: bandwidth
        dict(name="verify batch", op="verify", B=32, n=4, nvar=0, V=248320, q=True, greedy=0),
        # drafts that were looked up (no probabilities), ragged counts, some sequences greedy, an odd vocabulary
        dict(name="verify ragged", op="verify", B=61, n=8, nvar=100, V=50257, q=False, greedy=30),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(hi, lo))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "window", "window", "verify"])
    if op == "linear":
        K = 128 * _log(rng, 1, 128)
        T = _log(rng, 1, 4096) if rng.random() < 0.5 else rng.randint(1, 16)
        most = min(WEIGHTS // K, PRODUCTS // (T * K), 1 << 18)
        return dict(op=op, T=T, N=_log(rng, 16, max(most, 17)), K=K)
    if op == "verify":
        V = _log(rng, 100, 260000)
        n = rng.randint(0, 8)
        return dict(op=op, B=_log(rng, 1, max(1, min(256, LOGITS // (V * (n + 1))))), n=n, nvar=rng.choice([0, 100]), V=V,
                    q=rng.random() < 0.5, greedy=rng.choice([0, 0, 30, 100]))
    D, S = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    window = _log(rng, 1, 40000)
    sinks = rng.choice([0, 1, 4, _log(rng, 1, 1000)])
    form = rng.choice(["decode", "verify", "prompt", "chunk"])
    c = dict(op=op, B=1, Hkv=Hkv, G=G, D=D, S=S, nq=1, qvar=0, kv=0, kvar=rng.choice([0, 60, 95]), window=window, sinks=sinks)
    if form == "decode":
        B = _log(rng, 1, 256)
        c.update(B=B, kv=_log(rng, 16, max(17, min(131072, KEYS // (B * Hkv)))))
        return c
    if form == "verify":
        B = _log(rng, 1, 64)
        c.update(B=B, nq=rng.randint(2, 9), qvar=rng.choice([0, 80]), kv=_log(rng, 16, max(17, min(32768, KEYS // (B * Hkv)))))
        return c
    B, nq, kv = _log(rng, 1, 12), _log(rng, 32, 4096), 0 if form == "prompt" else _log(rng, 100, 60000)
    # halve it until it fits: no more scores than the largest listed case, and a cache of its size
    while B * nq * (kv + nq) * Hkv * G > SCORES or B * (kv + nq) * Hkv > KEYS:
        if kv > nq:
            kv //= 2
        elif B > 1:
            B //= 2
        else:
            nq //= 2
    c.update(B=B, nq=nq, qvar=rng.choice([0, 90]), kv=kv)
    return c


def _lengths(case):
    """(queries, keys) of each sequence: up to qvar and kvar percent below nq and kv, from the case alone."""
    q, n = [], []
    for b in range(case["B"]):
        f = ((b * 40503 + 12345) % 65536) / 65536
        g = ((b * 30011 + 777) % 65536) / 65536
        nq = max(1, int(case["nq"] * (1 - case["qvar"] / 100 * f)))
        q.append(nq)
        n.append(nq + int(case["kv"] * (1 - case["kvar"] / 100 * g)))
    return q, n


def _rows(case):
    """Rows of logits of each sequence: its drafts and one more."""
    return [1 + int(case["n"] * (1 - case["nvar"] / 100 * (((b * 40503 + 12345) % 65536) / 65536)) + 0.5) for b in range(case["B"])]


def work(case):
    if case["op"] == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": N * K // 2 + N * K // 64 + 2 * T * K + 2 * T * N, "flops": 2.0 * T * N * K}
    if case["op"] == "verify":
        B, T, V = case["B"], sum(_rows(case)), case["V"]
        read = 2 * T * V + (2 * (T - B) * V if case["q"] else 0) + 4 * B * V
        return {"bytes": read + 12 * T + 12 * B, "flops": 4.0 * (T + (T - B if case["q"] else 0)) * V + 4.0 * B * V}
    D, w, sinks = case["D"], case["window"], case["sinks"]
    q, n = _lengths(case)
    Hq = case["Hkv"] * case["G"]
    rows = pairs = pages = 0
    for a, c in zip(q, n):
        first = max(0, c - a - w + 1)                      # the first key that the window of any query holds
        rows += c - first + min(sinks, first)
        pages += -(-(c - first) // case["S"]) + -(-min(sinks, first) // case["S"])
        for i in range(c - a, c):
            low = max(0, i - w + 1)
            pairs += i + 1 - low + min(sinks, low)
    return {"bytes": rows * case["Hkv"] * (D + 4) + sum(q) * Hq * (4 * D + 4) + 8 * case["B"] + 4 * pages, "flops": 4.0 * D * Hq * pairs}


# ---- inputs ----------------------------------------------------------------------------------------------------

def _codes(gen, shape):
    """Words of eight codes of a roughly normal row (its largest near 7)."""
    words = torch.zeros(shape, dtype=torch.int32, device="cuda")
    for i in range(8):
        n = (torch.randn(shape, generator=gen, device="cuda") * 2.4).round_().clamp_(-8, 7).to(torch.int32) + 8
        words |= n << (4 * i)
    return words


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda *s: torch.rand(*s, generator=gen, device="cuda")   # noqa: E731
    st = {"case": dict(case)}
    if own:
        import w4a16_mixture_experts_gb300 as moe
        st["moe"] = moe
    if case["op"] == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        x = rand(T, K) * (1 + 9 * (unit(K) < 0.003))       # a few channels stand out
        st.update(x=x.to(torch.bfloat16), w=_codes(gen, (N, K // 8)), scales=((0.5 + unit(N, K // 128)) * 0.4 / math.sqrt(K)).to(torch.bfloat16),
                  y=torch.empty(T, N, dtype=torch.bfloat16, device="cuda"))
        if own:
            st.update(ws=torch.zeros(moe.moe_w4a16_workspace_size(T, N, K), dtype=torch.uint8, device="cuda"))
        return st
    if case["op"] == "verify":
        B, V, rows = case["B"], case["V"], _rows(case)
        T, pitch = sum(rows), -(-V // 8) * 8                # rows of a multiple of 16 bytes
        cu = [0]
        for r in rows:
            cu.append(cu[-1] + r)
        target = rand(T, pitch) * 2
        target.scatter_add_(1, torch.randint(0, V, (T, 24), generator=gen, device="cuda"), 4 + 9 * unit(T, 24))
        near = target + 0.6 * rand(T, pitch)                # the draft model's logits: near the target's
        temperature = 0.6 + 0.6 * unit(B)
        temperature[torch.arange(B, device="cuda") * 37 % 100 < case["greedy"]] = 0
        of = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(rows, device="cuda"))
        logits, draft = target.to(torch.bfloat16)[:, :V], near.to(torch.bfloat16)[:, :V]
        del target, near
        t = temperature[of].clamp(min=1e-3).unsqueeze(1)
        drafts = torch.empty(T, dtype=torch.int32, device="cuda")
        for lo in range(0, T, 64):                          # drafted by the same draw as the sampling's
            e = torch.empty(min(64, T - lo), V, device="cuda").exponential_(generator=gen)
            drafts[lo: lo + 64] = (draft[lo: lo + 64].float() / t[lo: lo + 64] - e.log()).argmax(1).to(torch.int32)
        noise = torch.empty(B, -(-V // 4) * 4, device="cuda").exponential_(generator=gen)[:, :V]
        st.update(logits=logits, draft=draft if case["q"] else None, drafts=drafts, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                  temperature=temperature, uniform=unit(T), noise=noise, tokens=torch.empty(T, dtype=torch.int32, device="cuda"),
                  accepted=torch.empty(B, dtype=torch.int32, device="cuda"), most=max(rows))
        if own:
            st.update(ws=moe.verify_workspace(B, T, V, device="cuda"))
        return st
    D, Hkv, S = case["D"], case["Hkv"], case["S"]
    nq, n = _lengths(case)
    B, Hq = case["B"], Hkv * case["G"]
    T, M = sum(nq), max(-(-c // S) for c in n)
    used = [-(-c // S) for c in n]
    pages = sum(used) + 16
    cache = []
    for _ in range(2):
        cache += [_codes(gen, (pages, Hkv, S, D // 8)), (0.25 + 0.35 * unit(pages, Hkv, S)).to(torch.bfloat16)]
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(B, M, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, : used[b]] = order[at: at + used[b]]
        at += used[b]
    cu = [0]
    for a in nq:
        cu.append(cu[-1] + a)
    st.update(q=(1.6 * rand(T, Hq, D)).to(torch.bfloat16), cache=cache, table=table,
              lens=torch.tensor(n, dtype=torch.int32, device="cuda"), cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"),
              max_q=max(nq), scale=D ** -0.5, out=torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda"),
              lse=torch.empty(T, Hq, dtype=torch.float32, device="cuda"))
    if own:
        st.update(cache=moe.Kv4Cache(*cache), ws=moe.kv4_workspace(T, Hq, Hkv, D, device="cuda"))
    return st


# ---- the plain forms -------------------------------------------------------------------------------------------

def _unpack(words):
    shifts = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    return (((words.unsqueeze(-1) >> shifts) & 15) - 8).flatten(-2).float()


def _linear(x, w, scales):
    W = (_unpack(w).unflatten(-1, (-1, 128)) * scales.float().unsqueeze(-1)).flatten(-2)
    return (x.float() @ W.t()).to(torch.bfloat16)


def _window(q, cache, table, lens, cu_q, max_q, scale, window, sinks):
    kc, ks, vc, vs = cache
    B, M = table.shape
    T, Hq, D = q.shape
    Hkv, S = ks.shape[1:]
    G, L = Hq // Hkv, M * S
    at = table.long()
    k = (_unpack(kc[at]) * ks[at].float().unsqueeze(-1)).transpose(1, 2).reshape(B, Hkv, L, D)
    v = (_unpack(vc[at]) * vs[at].float().unsqueeze(-1)).transpose(1, 2).reshape(B, Hkv, L, D)
    i = torch.arange(max_q, device=q.device)
    nq = (cu_q[1:] - cu_q[:-1]).unsqueeze(1)
    there = i < nq
    rows = (cu_q[:-1].unsqueeze(1) + i).clamp(max=T - 1).long()
    x = q[rows].float().view(B, max_q, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, max_q * G, D)
    s = (x @ k.transpose(-1, -2)) * scale
    last = (lens.unsqueeze(1) - nq + i).unsqueeze(-1)                    # [B, max_q, 1]: the last key a query sees
    j = torch.arange(L, device=q.device)
    seen = (j <= last) & ((j > last - window) | (j < sinks))
    s = s.masked_fill(~seen.repeat_interleave(G, 1).unsqueeze(1), -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = torch.where(l > 0, (p @ v) / l, torch.zeros_like(l))
    lse = (m + torch.log(l)).squeeze(-1)
    o = o.view(B, Hkv, max_q, G, D).transpose(1, 2)[there].reshape(T, Hq, D)
    return o.to(torch.bfloat16), lse.view(B, Hkv, max_q, G).transpose(1, 2)[there].reshape(T, Hq)


def _probabilities(logits, t):
    """Softmax of rows at the rows' temperatures, in 64 bits: the tests and the choice go by their differences."""
    x = logits.double() / t
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _verify(logits, draft, drafts, cu, temperature, uniform, noise, most):
    T, V = logits.shape
    B = cu.shape[0] - 1
    i = torch.arange(most, device=logits.device)
    n = (cu[1:] - cu[:-1]).unsqueeze(1)                                   # rows of each sequence
    of = torch.repeat_interleave(torch.arange(B, device=logits.device), n.squeeze(1), output_size=T)
    greedy = temperature == 0
    t = torch.where(greedy, torch.ones_like(temperature), temperature).double()[of].unsqueeze(1)
    x = drafts.long().unsqueeze(1)
    best = (logits == logits.amax(1, keepdim=True)).to(torch.uint8).argmax(1)   # (the first of the largest)
    p = _probabilities(logits, t)
    q = torch.zeros(T, V, dtype=torch.float64, device=logits.device).scatter_(1, x, 1.0) if draft is None else _probabilities(draft, t)
    keep = torch.where(greedy[of], best == drafts, uniform * q.gather(1, x).squeeze(1) < p.gather(1, x).squeeze(1))
    rows = (cu[:-1].unsqueeze(1) + i).clamp(max=T - 1).long()             # [B, most]
    accepted = ((keep[rows] & (i < n - 1)).long().cumprod(1)).sum(1)
    at = (cu[:-1] + accepted).long()                                      # the row that gives the next token
    last = (accepted == n.squeeze(1) - 1).unsqueeze(1)
    r = torch.where(last, p[at], (p[at] - q[at]).clamp(min=0))
    r = torch.where(r.sum(1, keepdim=True) > 0, r, p[at])
    chosen = torch.where(greedy, best[at], (r / noise).argmax(1))
    place = torch.arange(T, device=logits.device) - cu[of]
    tokens = torch.where(place < accepted[of], drafts.long(), torch.where(place == accepted[of], chosen[of], torch.full_like(place, -1)))
    return tokens.to(torch.int32), accepted.to(torch.int32)


def run(st):
    case = st["case"]
    if case["op"] == "linear":
        if own:
            return st["moe"].moe_w4a16_linear(st["x"], st["w"], st["scales"], y=st["y"], ws=st["ws"])
        return _linear(st["x"], st["w"], st["scales"])
    if case["op"] == "verify":
        if own:
            return st["moe"].moe_verify_drafts(st["logits"], st["drafts"], st["cu"], st["uniform"], st["noise"], draft_logits=st["draft"],
                                               temperature=st["temperature"], tokens=st["tokens"], accepted=st["accepted"], ws=st["ws"])
        return _verify(st["logits"], st["draft"], st["drafts"], st["cu"], st["temperature"], st["uniform"], st["noise"], st["most"])
    if own:
        return st["moe"].moe_kv4_attention_window(st["q"], st["cache"], st["table"], st["lens"], case["window"], case["sinks"], cu_q=st["cu_q"],
                                                  max_q=st["max_q"], scale=st["scale"], out=st["out"], lse=st["lse"], ws=st["ws"])
    return _window(st["q"], st["cache"], st["table"], st["lens"], st["cu_q"], st["max_q"], st["scale"], case["window"], case["sinks"])


# ---- the definitions in 64 bits --------------------------------------------------------------------------------

def _exact_codes(words):
    """Codes in 64 bits: the words as bytes, low nibble first."""
    b = words.contiguous().view(torch.uint8)
    out = torch.empty(*b.shape[:-1], b.shape[-1] * 2, dtype=torch.float64, device=words.device)
    out[..., 0::2] = (b % 16).double() - 8
    out[..., 1::2] = (b // 16).double() - 8
    return out


def _exact_linear(st, case):
    x, K = st["x"].double(), case["K"]
    y = torch.empty(case["T"], case["N"], dtype=torch.float64, device="cuda")
    for lo in range(0, case["N"], 8192):
        w = _exact_codes(st["w"][lo: lo + 8192])
        for g in range(K // 128):
            w[:, g * 128: (g + 1) * 128] *= st["scales"][lo: lo + 8192, g: g + 1].double()
        y[:, lo: lo + 8192] = x @ w.T
    return y


def _exact_window(st, case):
    kc, ks, vc, vs = st["cache"]
    S, D, Hkv, G, w, sinks = case["S"], case["D"], case["Hkv"], case["G"], case["window"], case["sinks"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for nq, n, pages in zip(*_lengths(case), st["table"]):
        pages = pages[: -(-n // S)].long()
        for lo in range(0, nq, 512):
            hi = min(nq, lo + 512)
            first = n - nq + lo                                      # the block's first position
            low = max(0, first - w + 1)
            pick = torch.cat([torch.arange(min(sinks, low)), torch.arange(low, n - nq + hi)]).cuda()   # the keys its queries see
            page, off = pages[pick // S], pick % S
            k = _exact_codes(kc[page, :, off]) * ks[page, :, off].double().unsqueeze(-1)   # [keys, Hkv, D]
            v = _exact_codes(vc[page, :, off]) * vs[page, :, off].double().unsqueeze(-1)
            pos = torch.arange(first, n - nq + hi, device="cuda").unsqueeze(1)
            hidden = (pick > pos) | ((pos - pick >= w) & (pick >= sinks))
            for h in range(Hkv):
                q = st["q"][at + lo: at + hi, h * G: (h + 1) * G].double()
                logits = torch.einsum("tgd,nd->gtn", q, k[:, h]) * st["scale"]
                logits.masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(logits, -1, keepdim=True)
                out[at + lo: at + hi, h * G: (h + 1) * G] = torch.einsum("gtn,nd->tgd", (logits - z).exp(), v[:, h])
                lse[at + lo: at + hi, h * G: (h + 1) * G] = z.squeeze(-1).T
        at += nq
    return out, lse


def _exact_verify(st, case):
    """Sequence by sequence and draft by draft, as the definition reads."""
    tokens, accepted, at = [], [], 0
    temperature, uniform, drafts = st["temperature"].tolist(), st["uniform"].tolist(), st["drafts"].tolist()
    for b, rows in enumerate(_rows(case)):
        t, a, chosen = temperature[b], 0, None
        while True:
            row, x = st["logits"][at + a].double(), drafts[at + a]
            last = a == rows - 1
            if t == 0:
                first = int((row == row.max()).nonzero()[0])
                if last or first != x:
                    chosen = first
                    break
            else:
                p = torch.softmax(row / t, 0)
                if last:
                    r = p
                else:
                    if st["draft"] is not None:
                        q = torch.softmax(st["draft"][at + a].double() / t, 0)
                    else:
                        q = torch.zeros_like(p)
                        q[x] = 1
                    r = (p - q).clip(min=0)
                    if not bool((r > 0).any()):
                        r = p
                if last or not uniform[at + a] * float(q[x]) < float(p[x]):
                    chosen = int((r.log() - st["noise"][b].double().log()).argmax())
                    break
            a += 1
        tokens += drafts[at: at + a] + [chosen] + [-1] * (rows - a - 1)
        accepted.append(a)
        at += rows
    return torch.tensor(tokens, dtype=torch.int32, device="cuda"), torch.tensor(accepted, dtype=torch.int32, device="cuda")


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_linear(st, case)
    return _exact_verify(st, case) if case["op"] == "verify" else _exact_window(st, case)

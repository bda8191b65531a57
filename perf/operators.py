"""The attention block's operators, measured: per-head norms with the rotary turn, rows written to and read from
a paged 4-bit cache, and attention over that cache.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits) or, where ``own`` is
true, through the library's entry points on the same tensors. The cache's format: a row is the D values of one
(token, KV head); its codes are q + 8 with q in [-8, 7], eight to an int32 word, lowest nibble first, and one
bf16 scale. Codes are int32 [pages, Hkv, page_size, D / 8], scales bf16 [pages, Hkv, page_size], for K and for V;
a sequence's rows are found through its row of the page table.
"""
import math

import torch

own = False

LARGEST = 1.2e12     # flops of the largest listed attention case; drawn ones cost no more
KEYS = 1 << 21       # (token, KV head) rows of cache a drawn case may hold


# ---- the cases -------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a small batch, far into a long context: latency
        dict(name="norm_rope decode", op="norm_rope", T=4, Hq=32, Hkv=4, D=128, rot=128, interleaved=False, far=1 << 20),
        # a prompt whose heads turn by a quarter of their values, interleaved pairs, odd length
        dict(name="norm_rope partial", op="norm_rope", T=1777, Hq=24, Hkv=8, D=64, rot=16, interleaved=True, far=1 << 17),
        # a whole prompt chunk: bandwidth
        dict(name="norm_rope prompt", op="norm_rope", T=16384, Hq=32, Hkv=8, D=128, rot=128, interleaved=False, far=1 << 15),
        # the rows of one decode step
        dict(name="append decode", op="append", T=16, Hkv=8, D=128, S=16),
        # the rows of a prompt chunk
        dict(name="append prompt", op="append", T=32768, Hkv=8, D=128, S=64),
        # one sequence, one token, a short context: latency
        dict(name="decode short", op="attention", B=1, Hkv=8, G=4, D=128, S=16, nq=1, qvar=0, kv=500, kvar=0),
        # a server's decode batch, ragged lengths
        dict(name="decode batch", op="attention", B=96, Hkv=4, G=8, D=128, S=64, nq=1, qvar=0, kv=4001, kvar=90),
        # few sequences with a long context: one token's work split over the whole card
        dict(name="decode long", op="attention", B=2, Hkv=8, G=7, D=128, S=32, nq=1, qvar=0, kv=131072, kvar=1),
        # draft tokens verified together, small heads
        dict(name="verify drafts", op="attention", B=24, Hkv=8, G=4, D=64, S=16, nq=5, qvar=60, kv=2777, kvar=70),
        # ragged prompts from their first token on
        dict(name="prompts ragged", op="attention", B=12, Hkv=4, G=6, D=64, S=16, nq=1500, qvar=90, kv=0, kvar=0),
        # a prompt chunk behind a long prefix
        dict(name="prompt chunk", op="attention", B=1, Hkv=4, G=8, D=128, S=64, nq=4096, qvar=0, kv=12288, kvar=0),
        # a small chunk behind a long prefix: few rows, a long axis
        dict(name="chunk long", op="attention", B=1, Hkv=2, G=8, D=128, S=128, nq=192, qvar=0, kv=60000, kvar=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attention", "attention", "attention"])
    D = rng.choice([64, 128])
    if op == "norm_rope":
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
        T = _log(rng, 1, 16384 * 40 * 128 // (Hkv * (G + 1) * D) if Hkv * (G + 1) * D > 40 * 128 else 16384)
        rot = rng.choice([D, D // 2, D // 4])
        return dict(op=op, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, rot=rot, interleaved=rng.random() < 0.5, far=1 << rng.randint(10, 21))
    S = rng.choice([16, 32, 64, 128])
    if op == "append":
        Hkv = rng.choice([1, 2, 3, 4, 8, 16])
        return dict(op=op, T=_log(rng, 1, 32768 * 8 // max(Hkv, 8)), Hkv=Hkv, D=D, S=S)
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    form = rng.choice(["decode", "verify", "prompt", "chunk"])
    if form == "decode":
        B = _log(rng, 1, 256)
        kv = _log(rng, 16, max(17, min(131072, KEYS // (B * Hkv))))
        return dict(op=op, B=B, Hkv=Hkv, G=G, D=D, S=S, nq=1, qvar=0, kv=kv, kvar=rng.choice([0, 50, 95]))
    if form == "verify":
        B = _log(rng, 1, 64)
        kv = _log(rng, 16, max(17, min(32768, KEYS // (B * Hkv))))
        return dict(op=op, B=B, Hkv=Hkv, G=G, D=D, S=S, nq=rng.randint(2, 9), qvar=rng.choice([0, 80]), kv=kv, kvar=rng.choice([0, 90]))
    B = _log(rng, 1, 12)
    nq = _log(rng, 32, 4096)
    kv = 0 if form == "prompt" else _log(rng, 100, 60000)
    c = dict(op=op, B=B, Hkv=Hkv, G=G, D=D, S=S, nq=nq, qvar=rng.choice([0, 90]), kv=kv, kvar=rng.choice([0, 60]))
    # halve it until it fits: no more work than the largest listed case, and scores the plain form can hold
    while 4.0 * D * B * nq * (kv + nq) * Hkv * G > LARGEST or B * (kv + nq) * Hkv > KEYS:
        if kv > nq:
            kv //= 2
        elif B > 1:
            B //= 2
        else:
            nq //= 2
        c.update(B=B, nq=nq, kv=kv)
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


def work(case):
    D = case["D"]
    if case["op"] == "norm_rope":
        v = case["T"] * (case["Hq"] + case["Hkv"]) * D
        return {"bytes": 4 * v + 4 * case["T"] + 4 * D + 2 * case["rot"], "flops": 8 * v}
    if case["op"] == "append":   # rows in, their codes and scales out, and read back as values
        rows = 2 * case["T"] * case["Hkv"]
        return {"bytes": rows * (2 * D + 2 * (D // 2 + 2) + 2 * D) + 8 * case["T"], "flops": 6 * rows * D}
    q, n = _lengths(case)
    Hq = case["Hkv"] * case["G"]
    rows = sum(n) * case["Hkv"]
    pairs = sum(a * (c - a) + a * (a + 1) // 2 for a, c in zip(q, n))
    return {"bytes": rows * (D + 4) + sum(q) * Hq * (4 * D + 4) + 8 * case["B"] + 4 * sum(-(-c // case["S"]) for c in n),
            "flops": 4.0 * D * Hq * pairs}


# ---- inputs ----------------------------------------------------------------------------------------------------

def _codes(gen, pages, Hkv, S, D):
    """Packed codes of a roughly normal row distribution (the largest of a row near 7) and scales near 0.4."""
    words = torch.zeros(pages, Hkv, S, D // 8, dtype=torch.int32, device="cuda")
    for i in range(8):
        n = (torch.randn(words.shape, generator=gen, device="cuda") * 2.4).round_().clamp_(-8, 7).to(torch.int32) + 8
        words |= n << (4 * i)
    scales = (0.25 + 0.35 * torch.rand(pages, Hkv, S, generator=gen, device="cuda")).to(torch.bfloat16)
    return words, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    op, D, Hkv = case["op"], case["D"], case["Hkv"]
    st = {"case": dict(case)}
    if own:
        import w4a16_mixture_experts_gb300 as moe
        st["moe"] = moe
    if op == "norm_rope":
        T, Hq, rot = case["T"], case["Hq"], case["rot"]
        # the query, key and value rows as one projection leaves them
        qkv = (rand(T, (Hq + 2 * Hkv) * D) * 1.5).to(torch.bfloat16)
        start = torch.randint(0, case["far"] - min(T, case["far"] - 1), (1,), generator=gen, device="cuda")
        st.update(q=qkv[:, : Hq * D].view(T, Hq, D), k=qkv[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D),
                  positions=(start + torch.arange(T, device="cuda")).to(torch.int32),
                  inv_freq=(1e6 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)).float(),
                  q_weight=(1 + 0.2 * rand(D)).to(torch.bfloat16), k_weight=(1 + 0.2 * rand(D)).to(torch.bfloat16),
                  q_out=torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda"),
                  k_out=torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda"))
        return st
    S = case["S"]
    if op == "append":
        T = case["T"]
        pages = -(-T // S) + 8
        kv = rand(T, 2 * Hkv * D)
        kv *= 1 + 3 * (torch.rand(T, 2 * Hkv * D, generator=gen, device="cuda") < 0.01)   # outliers set a row's scale
        kv = kv.to(torch.bfloat16)
        cache = [torch.zeros(pages, Hkv, S, D // 8, dtype=torch.int32, device="cuda"), torch.zeros(pages, Hkv, S, dtype=torch.bfloat16, device="cuda")] + \
                [torch.zeros(pages, Hkv, S, D // 8, dtype=torch.int32, device="cuda"), torch.zeros(pages, Hkv, S, dtype=torch.bfloat16, device="cuda")]
        order = torch.randperm(pages, generator=gen, device="cuda")
        t = torch.arange(T, device="cuda")
        st.update(k=kv[:, : Hkv * D].view(T, Hkv, D), v=kv[:, Hkv * D:].view(T, Hkv, D), cache=cache,
                  slots=(order[t // S] * S + t % S).to(torch.int32),
                  k_out=torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda"),
                  v_out=torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda"))
        if own:
            st.update(cache=moe.Kv4Cache(*cache), ws=moe.kv4_workspace(device="cuda"))
        return st
    nq, n = _lengths(case)
    B, Hq = case["B"], Hkv * case["G"]
    T, M = sum(nq), max(-(-c // S) for c in n)
    used = [-(-c // S) for c in n]
    pages = sum(used) + 16
    kc, ks = _codes(gen, pages, Hkv, S, D)
    vc, vs = _codes(gen, pages, Hkv, S, D)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(B, M, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, : used[b]] = order[at: at + used[b]]
        at += used[b]
    cu = [0]
    for a in nq:
        cu.append(cu[-1] + a)
    st.update(q=(1.6 * rand(T, Hq, D)).to(torch.bfloat16), cache=[kc, ks, vc, vs], table=table,
              lens=torch.tensor(n, dtype=torch.int32, device="cuda"), cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"),
              max_q=max(nq), scale=D ** -0.5, out=torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda"),
              lse=torch.empty(T, Hq, dtype=torch.float32, device="cuda"))
    if own:
        st.update(cache=moe.Kv4Cache(kc, ks, vc, vs), ws=moe.kv4_workspace(T, Hq, Hkv, D, device="cuda"))
    return st


# ---- the plain forms -------------------------------------------------------------------------------------------

def _unpack(words, scales):
    shifts = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    q = ((words.unsqueeze(-1) >> shifts) & 15) - 8
    return q.flatten(-2).float() * scales.float().unsqueeze(-1)


def _pack(x):
    """Codes and scales of rows x [..., D] in 32 bits."""
    s = (x.abs().amax(-1) / 7).to(torch.bfloat16)
    f = s.float().unsqueeze(-1)
    q = torch.where(f == 0, torch.zeros_like(x), torch.round(x / f).clamp(-8, 7)).to(torch.int32) + 8
    shifts = torch.arange(0, 32, 4, device=x.device, dtype=torch.int32)
    return (q.unflatten(-1, (-1, 8)) << shifts).sum(-1).to(torch.int32), s


def _norm_rope(x, cos, sin, w, rot, interleaved):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    turn, rest = y[..., :rot], y[..., rot:]
    a, b = (turn[..., 0::2], turn[..., 1::2]) if interleaved else (turn[..., : rot // 2], turn[..., rot // 2:])
    u, v = a * cos - b * sin, a * sin + b * cos
    turn = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((turn, rest), -1).to(torch.bfloat16)


def _attention(q, cache, table, lens, cu_q, max_q, scale):
    kc, ks, vc, vs = cache
    B, M = table.shape
    T, Hq, D = q.shape
    Hkv, S = ks.shape[1:]
    G, L = Hq // Hkv, M * S
    at = table.long()
    k = _unpack(kc[at], ks[at]).transpose(1, 2).reshape(B, Hkv, L, D)
    v = _unpack(vc[at], vs[at]).transpose(1, 2).reshape(B, Hkv, L, D)
    i = torch.arange(max_q, device=q.device)
    nq = (cu_q[1:] - cu_q[:-1]).unsqueeze(1)
    there = i < nq
    rows = (cu_q[:-1].unsqueeze(1) + i).clamp(max=T - 1).long()
    x = q[rows].float().view(B, max_q, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, max_q * G, D)
    s = (x @ k.transpose(-1, -2)) * scale
    last = lens.unsqueeze(1) - nq + i                                    # [B, max_q]: the last key a query sees
    seen = (torch.arange(L, device=q.device) <= last.unsqueeze(-1)).repeat_interleave(G, 1).unsqueeze(1)
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = torch.where(l > 0, (p @ v) / l, torch.zeros_like(l))
    lse = (m + torch.log(l)).squeeze(-1)
    o = o.view(B, Hkv, max_q, G, D).transpose(1, 2)[there].reshape(T, Hq, D)
    lse = lse.view(B, Hkv, max_q, G).transpose(1, 2)[there].reshape(T, Hq)
    return o.to(torch.bfloat16), lse


def run(st):
    case = st["case"]
    op = case["op"]
    if op == "norm_rope":
        if own:
            return st["moe"].moe_qk_norm_rope(st["q"], st["k"], st["positions"], st["inv_freq"], st["q_weight"], st["k_weight"],
                                              eps=1e-6, interleaved=case["interleaved"], q_out=st["q_out"], k_out=st["k_out"])
        theta = st["positions"].double().unsqueeze(-1) * st["inv_freq"].double()   # far positions: 64 bits
        cos, sin = theta.cos().float().unsqueeze(1), theta.sin().float().unsqueeze(1)
        return (_norm_rope(st["q"], cos, sin, st["q_weight"], case["rot"], case["interleaved"]),
                _norm_rope(st["k"], cos, sin, st["k_weight"], case["rot"], case["interleaved"]))
    if op == "append":
        if own:
            st["moe"].moe_kv4_append(st["k"], st["v"], st["slots"], st["cache"], ws=st["ws"])
            return st["moe"].moe_kv4_read(st["slots"], st["cache"], k_out=st["k_out"], v_out=st["v_out"], ws=st["ws"])
        kc, ks, vc, vs = st["cache"]
        page, off = st["slots"].long() // case["S"], st["slots"].long() % case["S"]
        for_k, for_v = _pack(st["k"].float()), _pack(st["v"].float())
        kc[page, :, off], ks[page, :, off] = for_k
        vc[page, :, off], vs[page, :, off] = for_v
        return (_unpack(kc[page, :, off], ks[page, :, off]).to(torch.bfloat16),
                _unpack(vc[page, :, off], vs[page, :, off]).to(torch.bfloat16))
    if own:
        return st["moe"].moe_kv4_attention(st["q"], st["cache"], st["table"], st["lens"], cu_q=st["cu_q"], max_q=st["max_q"],
                                           scale=st["scale"], out=st["out"], lse=st["lse"], ws=st["ws"])
    return _attention(st["q"], st["cache"], st["table"], st["lens"], st["cu_q"], st["max_q"], st["scale"])


# ---- the definitions in 64 bits --------------------------------------------------------------------------------

def _exact_turn(x, w, theta, rot, interleaved):
    """Each pair as a complex number, turned by exp(i theta)."""
    x = x.double()
    y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * w.double()
    i = torch.arange(rot // 2, device=x.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.ones_like(theta), theta).unsqueeze(1)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rows(words, scales):
    """Values of rows in 64 bits: the words as bytes, low nibble first."""
    bytes_ = words.contiguous().view(torch.uint8)
    out = torch.empty(*bytes_.shape[:-1], bytes_.shape[-1] * 2, dtype=torch.float64, device=words.device)
    out[..., 0::2] = (bytes_ % 16).double() - 8
    out[..., 1::2] = (bytes_ // 16).double() - 8
    return out * scales.double().unsqueeze(-1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm_rope":
        theta = st["positions"].double().outer(st["inv_freq"].double())
        return (_exact_turn(st["q"], st["q_weight"], theta, case["rot"], case["interleaved"]),
                _exact_turn(st["k"], st["k_weight"], theta, case["rot"], case["interleaved"]))
    if case["op"] == "append":
        def there_and_back(x):
            x = x.double()
            # a scale's own definition: the 32-bit quotient, then 16 bits of it
            s = (x.abs().max(-1, keepdim=True).values.float() / 7).bfloat16().double()
            q = torch.floor(x / s)
            q = q + torch.where((x / s - q > 0.5) | ((x / s - q == 0.5) & (q % 2 != 0)), 1.0, 0.0)
            return torch.where(s > 0, q.clip(-8, 7) * s, torch.zeros_like(x))
        return there_and_back(st["k"]), there_and_back(st["v"])
    kc, ks, vc, vs = st["cache"]
    S, D, Hkv, G = case["S"], case["D"], case["Hkv"], case["G"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (nq, n) in enumerate(zip(*_lengths(case))):
        pages = st["table"][b, : -(-n // S)].long()
        for h in range(Hkv):
            k = _exact_rows(kc[pages, h], ks[pages, h]).reshape(-1, D)[:n]
            v = _exact_rows(vc[pages, h], vs[pages, h]).reshape(-1, D)[:n]
            for lo in range(0, nq, 512):
                hi = min(nq, lo + 512)
                q = st["q"][at + lo: at + hi, h * G: (h + 1) * G].double()
                logits = torch.einsum("tgd,nd->gtn", q, k) * st["scale"]
                hidden = torch.arange(n, device="cuda") > torch.arange(n - nq + lo, n - nq + hi, device="cuda").unsqueeze(1)
                logits.masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(logits, -1, keepdim=True)
                out[at + lo: at + hi, h * G: (h + 1) * G] = torch.einsum("gtn,nd->tgd", (logits - z).exp(), v)
                lse[at + lo: at + hi, h * G: (h + 1) * G] = z.squeeze(-1).T
        at += nq
    return out, lse

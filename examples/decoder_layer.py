"""One decoder layer on the library's calls: prompts of several sequences in one pass, then one token of each
sequence a step, replayed as a CUDA graph.

    python examples/decoder_layer.py [--steps 64]

    x += attention(norm(x)):  moe_w8a16_linear (q, k, v) -> moe_qk_norm_rope, in place -> moe_kv4_append
                              -> moe_kv4_attention -> moe_w8a16_linear
    x += experts(norm(x)):    moe_layer_forward

The weights are random (this shows the calls and their shapes, not a model). The cache holds pages of `page`
tokens; a sequence's pages are given out by the host, which alone knows the lengths, before the steps run.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import synth  # noqa: E402
import w4a16_mixture_experts_gb300 as moe  # noqa: E402


def rms(x, eps=1e-6):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + eps)).bfloat16()


class Layer:
    """Weights, cache and workspaces of one layer."""

    def __init__(self, H=2560, Hq=32, Hkv=4, D=128, E=64, k=8, I=640, pages=512, page=32, max_tokens=4096, seed=0):
        self.H, self.Hq, self.Hkv, self.D, self.k = H, Hq, Hkv, D, k
        up = lambda d: {n: t.cuda() for n, t in d.items()}   # noqa: E731
        self.qkv, self.o = up(synth.int8_weights((Hq + 2 * Hkv) * D, H, 128, seed)), up(synth.int8_weights(H, Hq * D, 128, seed + 1))
        self.experts, self.router = up(synth.expert_weights(E, H, I, seed)), synth.router(E, H, seed).cuda()
        self.q_norm = self.k_norm = torch.ones(D, dtype=torch.bfloat16, device="cuda")
        self.inv_freq = (1e6 ** (-torch.arange(0, D, 2).double() / D)).float().cuda()
        self.cache, self.page = moe.kv4_cache(pages, Hkv, page, D), page
        # one workspace serves the attention's calls and the experts'; the linears keep their own
        n = max(moe.moe_kv4_workspace_size(max_tokens, Hq, Hkv, D), moe.moe_workspace_size(max_tokens, H, E, k, I))
        m = max(moe.moe_w8a16_workspace_size(max_tokens, w["w_packed"].shape[0], w["w_packed"].shape[1] * 4, 128)
                for w in (self.qkv, self.o))
        self.ws, self.ws_linear = (torch.zeros(b, dtype=torch.uint8, device="cuda") for b in (n, m))

    def linear(self, x, w):
        return moe.moe_w8a16_linear(x, w["w_packed"], w["scales"], 128, ws=self.ws_linear)

    def __call__(self, x, positions, slots, table, lens, cu_q=None, max_q=1):
        """x bf16 [T, H] -> the layer's output; the new tokens' rows go into the cache at `slots`."""
        T, D = x.shape[0], self.D
        q, k, v = self.linear(rms(x), self.qkv).view(T, -1, D).split([self.Hq, self.Hkv, self.Hkv], 1)
        moe.moe_qk_norm_rope(q, k, positions, self.inv_freq, self.q_norm, self.k_norm, q_out=q, k_out=k)
        moe.moe_kv4_append(k, v, slots, self.cache, ws=self.ws)
        a = moe.moe_kv4_attention(q, self.cache, table, lens, cu_q, max_q, ws=self.ws)
        x = x + self.linear(a.view(T, -1), self.o)
        e = self.experts
        y, _, _ = moe.moe_layer_forward(rms(x), self.router, self.k, e["w1_packed"], e["w1_scales"], e["w2_packed"],
                                        e["w2_scales"], ws=self.ws)
        return x + y


def slots_of(table, positions, rows, page):
    """Slots of tokens at `positions` of the sequences `rows`."""
    return (table[rows, positions // page] * page + positions % page).to(torch.int32)


def prefill(layer, x, lens, table):
    """All sequences' tokens x [sum(lens), H] (their first) in one pass."""
    cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)
    rows = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).cuda()
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
    return layer(x, pos, slots_of(table, pos, rows, layer.page), table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 cu.cuda(), max(lens))


class Decode:
    """One step for B sequences as a graph: write x, call step(), read y. The lengths advance on the device."""

    def __init__(self, layer, lens, table):
        self.B = len(lens)
        self.x = torch.zeros(self.B, layer.H, dtype=torch.bfloat16, device="cuda")
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.rows, self.table = torch.arange(self.B, device="cuda"), table   # (the graph reads them: they must live as long)

        def body():
            pos = self.lens.clone()
            self.lens += 1
            return layer(self.x, pos, slots_of(self.table, pos, self.rows, layer.page), self.table, self.lens)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            body()   # (a step outside a graph first; what it wrote is written again by the first step)
            self.lens -= 1
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = body()

    def step(self):
        self.graph.replay()
        return self.y


def run(layer, prompts, steps, seed=0):
    """(outputs of the last step [B, H], outputs of the same tokens from one pass over whole sequences, us a step)"""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, page = len(prompts), layer.page
    need = [-(-(n + steps) // page) for n in prompts]
    if 2 * sum(need) > layer.cache.k_codes.shape[0]:
        raise ValueError("the cache holds %d pages, these sequences (twice) take %d" % (layer.cache.k_codes.shape[0], 2 * sum(need)))
    free = iter(torch.randperm(2 * sum(need)).tolist())
    tables = torch.zeros(2, B, max(need), dtype=torch.int32)
    for t in tables:
        for b, n in enumerate(need):
            t[b, :n] = torch.tensor([next(free) for _ in range(n)])
    tables = tables.cuda()
    whole = [torch.randn(n + steps, layer.H, generator=g, device="cuda").bfloat16() for n in prompts]
    prefill(layer, torch.cat([x[:n] for x, n in zip(whole, prompts)]), prompts, tables[0])
    decode = Decode(layer, prompts, tables[0])
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for i in range(steps):
        decode.x.copy_(torch.stack([x[n + i] for x, n in zip(whole, prompts)]))
        y = decode.step()
    end.record()
    torch.cuda.synchronize()
    lens = [n + steps for n in prompts]
    every = prefill(layer, torch.cat(whole), lens, tables[1])
    last = (torch.tensor(lens).cumsum(0) - 1).cuda()
    for ws in (layer.ws, layer.ws_linear):
        if moe.moe_check_device_error(ws):
            raise RuntimeError("the device reported an error")
    return y.clone(), every[last], start.elapsed_time(end) * 1e3 / steps


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    prompts = [700, 64, 233, 1, 129, 511, 320, 90]
    y, want, us = run(Layer(), prompts, a.steps)
    off = float((y.float() - want.float()).norm() / want.float().norm())
    print("%d sequences, %d steps: %.1f us a step; the last step's outputs are within %.2g of one pass over the whole sequences"
          % (len(prompts), a.steps, us, off))


if __name__ == "__main__":
    main()

"""Decoder layers end to end on one GPU: rotary positions, the 4-bit paged cache
and attention over it, then the MoE layer.

    python examples/decoder_layers.py

runs a prompt through a few random layers and decodes further tokens from a
CUDA graph. The projections around attention are plain matrix products;
everything else goes through the library.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from expert_moe_layer_gb300 import binding as B  # noqa: E402


def _norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Cache:
    """Pages of every layer and the page table of a batch of requests."""

    def __init__(self, cfg, layers, requests, max_tokens):
        per = -(-max_tokens // cfg.page_size)
        pages = per * requests
        block = cfg.page_size * cfg.head_dim * 9 // 8
        self.layers = [torch.zeros(pages, cfg.num_kv_heads, block, dtype=torch.uint8, device="cuda")
                       for _ in range(layers)]
        order = torch.randperm(pages, device="cuda", dtype=torch.int32)
        self.page_table = order.reshape(requests, per).contiguous()
        self.page_size = cfg.page_size
        self.tokens = min(per * cfg.page_size, cfg.rope_positions)   # room of a request

    def room(self, lens, new):
        """Refuses, before anything is enqueued, what has no page or no position."""
        if max(lens) + new > self.tokens:
            raise ValueError(f"a request of {max(lens) + new} tokens; the cache holds {self.tokens}")

    def slots(self, request, position):
        """Slot of each (request, position) pair."""
        page = self.page_table[request, position // self.page_size].long()
        return page * self.page_size + position % self.page_size


class Decoder:
    """Random layers: attention over the cache, then the MoE layer."""

    def __init__(self, layers=2, hidden=1024, heads=16, kv_heads=4, head_dim=64, experts=8,
                 intermediate=512, max_positions=4096, page_size=16, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def w(*shape):
            return (torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5).bfloat16()

        self.attn = B.make_attn_config(heads, kv_heads, head_dim, page_size, rotary_dim=head_dim,
                                       rope_positions=max_positions)
        self.moe = B.make_config(experts, 2, hidden, intermediate)
        self.norm = B.make_norm_config(hidden)
        self.table = torch.empty(max_positions, head_dim, device="cuda")
        B.moe_rope_table(self.attn, max_positions, None, B.make_rope_scaling(), self.table)
        self.layers = [dict(qkv=w((heads + 2 * kv_heads) * head_dim, hidden),
                            o=w(hidden, heads * head_dim), router=w(experts, hidden),
                            w13=w(experts, 2 * intermediate, hidden), w2=w(experts, hidden, intermediate))
                       for _ in range(layers)]
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim

    def workspaces(self, requests, tokens, longest):
        """Device scratch of one call shape, kept by the caller."""
        size = max(B.kv_attention_workspace_size(self.attn, requests, tokens, longest),
                   B.workspace_size(self.moe, tokens))
        return torch.empty(size, dtype=torch.uint8, device="cuda")

    def attend(self, t, longest, q, q_offsets, seq_lens, cache, pages, out, ws):
        B.moe_kv_attention(self.attn, seq_lens.shape[0], t, longest, q, q_offsets, seq_lens,
                           cache.page_table, pages, out, None, ws)

    def forward(self, x, cache, positions, slots, q_offsets, seq_lens, longest, ws):
        """x [T, hidden] of all requests' new tokens -> the same after the layers."""
        t = x.shape[0]
        y, h = None, torch.empty_like(x)    # the block before, and its sum's norm
        for w, pages in zip(self.layers, cache.layers):
            x = self._join(y, x, h)
            qkv = (h @ w["qkv"].T).unflatten(1, (-1, self.head_dim))
            q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
            turned = torch.empty(t, self.heads, self.head_dim, dtype=x.dtype, device="cuda")
            B.moe_kv_append(self.attn, t, q, k, v, positions, slots, self.table, turned, pages)
            out = torch.empty_like(turned)
            self.attend(t, longest, turned, q_offsets, seq_lens, cache, pages, out, ws)
            x = self._join(out.flatten(1) @ w["o"].T, x, h)
            y = torch.empty_like(x)
            B.moe_forward(self.moe, t, h, w["router"], None, w["w13"], w["w2"], None, None, None, y, ws)
        return self._join(y, x, None)

    def _join(self, y, x, h):
        """The residual x with a block's output y added (there is none before the
        first), and into h its norm for the next block."""
        out = x if y is None else torch.empty_like(x)
        B.moe_norm(self.norm, x.shape[0], y, x, None, None, None, None, None, None if y is None else out, h)
        return out


def prompt(model, cache, xs):
    """The prompts xs [n_b, hidden] of all requests in one call."""
    lens = [x.shape[0] for x in xs]
    cache.room(lens, 0)
    request = torch.repeat_interleave(torch.arange(len(xs)), torch.tensor(lens)).cuda()
    position = torch.cat([torch.arange(n) for n in lens]).cuda()
    offsets = torch.tensor([0] + lens).cumsum(0).int().cuda()
    return model.forward(torch.cat(xs), cache, position.int(), cache.slots(request, position),
                         offsets, torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens),
                         model.workspaces(len(xs), sum(lens), max(lens)))


class DecodeGraph:
    """One token per request, captured once; the lengths live on the device."""

    def __init__(self, model, cache, lens):
        cache.room(lens, 1)             # (the warm-up writes a token)
        self.host_lens = list(lens)
        n, hidden = len(lens), model.layers[0]["o"].shape[0]
        self.x = torch.zeros(n, hidden, dtype=torch.bfloat16, device="cuda")
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")   # cached tokens so far
        # the graph holds addresses only: what it reads lives as long as this object
        self.model, self.cache = model, cache
        self.ws = model.workspaces(n, n, 1)
        self.request = torch.arange(n, device="cuda")

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            before = self.lens.clone()
            self._step()                 # loads the kernels; its token is written again later
            self.lens.copy_(before)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph, stream=side):
                self.out = self._step()
        torch.cuda.current_stream().wait_stream(side)

    def _step(self):
        slots = self.cache.slots(self.request, self.lens.long())
        out = self.model.forward(self.x, self.cache, self.lens, slots, None, self.lens + 1, 1, self.ws)
        self.lens.add_(1)
        return out

    def step(self, x):
        self.cache.room(self.host_lens, 1)
        self.host_lens = [n + 1 for n in self.host_lens]
        self.x.copy_(x)
        self.graph.replay()
        return self.out


def main():
    model = Decoder()
    lens = [300, 17, 64]
    cache = Cache(model.attn, len(model.layers), len(lens), 512)
    xs = [torch.randn(n, 1024, device="cuda").bfloat16() for n in lens]
    last = prompt(model, cache, xs)[torch.tensor(lens).cumsum(0) - 1]
    decode = DecodeGraph(model, cache, lens)
    for i in range(8):
        last = decode.step(_norm(last)).clone()
        print(f"step {i}: |x| {last.float().norm(dim=-1).tolist()}")


if __name__ == "__main__":
    main()

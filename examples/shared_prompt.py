"""Several samples of one prompt through decoder layers: the prompt runs once, its
pages are forked, and each step attends to the prompt's keys once for all samples.

    python examples/shared_prompt.py

The steps run from one CUDA graph: reserving the next token's pages (which copies
a page that samples still share), appending, attention over the shared prefix and
the samples' own tokens, and the MoE layers. Samples that end give their pages
back; the pool is compacted at the end.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from decoder_layers import B, Decoder, _norm  # noqa: E402


class PoolCache:
    """Pages of every layer that rows of one page table share."""

    def __init__(self, cfg, layers, rows, max_tokens, pages):
        self.cfg, self.rows, self.pages = cfg, rows, pages
        self.tokens = min(-(-max_tokens // cfg.page_size) * cfg.page_size, cfg.rope_positions)
        block = cfg.page_size * cfg.head_dim * 9 // 8
        self.layers = [torch.zeros(pages, cfg.num_kv_heads, block, dtype=torch.uint8, device="cuda")
                       for _ in range(layers)]
        self.page_table = torch.full((rows, -(-max_tokens // cfg.page_size)), -1, dtype=torch.int32,
                                     device="cuda")
        self.held = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.pool = B.make_kv_pool(cfg, self.page_table, self.held, self.refs, self.layers)
        self.ws = torch.empty(B.kv_pool_workspace_size(cfg, self.pool, rows), dtype=torch.uint8,
                              device="cuda")
        self.used = torch.zeros(1, dtype=torch.int32, device="cuda")

    def room(self, tokens):
        """Refuses requests that outgrow their row of the page table or the rotary table."""
        if tokens > self.tokens:
            raise ValueError(f"a request of {tokens} tokens; the cache holds {self.tokens}")

    def reserve(self, rows, start, end):
        B.moe_kv_reserve(self.cfg, self.pool, start.shape[0], rows, start, end, self.ws)

    def fork(self, parents, children, tokens):
        B.moe_kv_fork(self.cfg, self.pool, parents.shape[0], parents, children, tokens, self.ws)

    def release(self, rows):
        B.moe_kv_release(self.cfg, self.pool, rows.shape[0], rows, None, self.ws)

    def compact(self):
        """Pages in use, which are the first ones afterwards."""
        B.moe_kv_compact(self.cfg, self.pool, self.used, self.ws)
        return self.used.item()

    def slots(self, request, position):
        page = self.page_table[request, position // self.cfg.page_size].long()
        return page * self.cfg.page_size + position % self.cfg.page_size

    def check(self):
        """Raises what the last pool call found wrong (synchronises)."""
        code, flags = B.moe_get_status(self.ws)
        if flags & B.DEV_NO_PAGE:
            raise RuntimeError("no free page")
        if code:
            raise RuntimeError(f"pool call: status {code}, flags {flags:#x}")


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Samples:
    """n rows that go on from one prompt of `tokens` tokens, a token per step."""

    def __init__(self, model, cache, first, n, tokens):
        cache.room(tokens + 1)
        self.model, self.cache, self.n, self.host_len = model, cache, n, tokens
        hidden = model.layers[0]["o"].shape[0]
        self.rows = torch.arange(first, first + n, dtype=torch.int32, device="cuda")
        self.table = cache.page_table[first:first + n]
        self.x = torch.zeros(n, hidden, dtype=torch.bfloat16, device="cuda")
        self.lens = torch.full((n,), tokens, dtype=torch.int32, device="cuda")
        self.groups, self.prefix = _ints([0, n]), _ints([tokens])
        size = max(B.kv_attention_shared_workspace_size(model.attn, n, n, 1, 1, n),
                   B.workspace_size(model.moe, n))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        self.graph = None

    # what Decoder.forward asks of a cache and of its attention
    layers = property(lambda self: self.cache.layers)

    def attend(self, t, longest, q, q_offsets, seq_lens, cache, pages, out, ws):
        B.moe_kv_attention_shared(self.model.attn, self.n, t, longest, 1, self.n, q, q_offsets, seq_lens,
                                  self.table, self.groups, self.prefix, pages, out, None, ws)

    def _step(self):
        self.cache.reserve(self.rows, self.lens, self.lens + 1)
        slots = self.cache.slots(self.rows.long(), self.lens.long())
        plain, self.model.attend = self.model.attend, self.attend
        try:
            out = self.model.forward(self.x, self, self.lens, slots, None, self.lens + 1, 1, self.ws)
        finally:
            self.model.attend = plain
        self.lens.add_(1)
        return out

    def step(self, x):
        """The samples' next tokens x [n, hidden] -> the same after the layers. Raises
        where a sample finds no free page; the step can be taken again then."""
        self.cache.room(self.host_len + 1)
        self.host_len += 1
        if self.graph is None:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                before = self.lens.clone()
                self._step()        # loads the kernels; the token is written again
                self.lens.copy_(before)
                self.graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(self.graph, stream=side):
                    self.out = self._step()
            torch.cuda.current_stream().wait_stream(side)
        self.x.copy_(x)
        self.graph.replay()
        try:
            self.cache.check()      # (a token without a page is stored nowhere)
        except RuntimeError:
            self.host_len -= 1
            self.lens.sub_(1)
            raise
        return self.out


def sample(model, cache, prompt, n):
    """Runs a prompt [tokens, hidden] in row 0 and forks it into rows 0 .. n - 1."""
    t = prompt.shape[0]
    cache.room(t + 1)
    if not 1 <= n <= cache.rows:
        raise ValueError(f"{n} samples; the cache holds 1 to {cache.rows}")
    cache.reserve(_ints([0]), _ints([0]), _ints([t]))
    cache.check()
    at = torch.arange(t, device="cuda")
    ws = model.workspaces(1, t, t)
    row = type("Row", (), dict(layers=cache.layers, page_table=cache.page_table[:1]))
    out = model.forward(prompt, row, at.int(), cache.slots(torch.zeros_like(at), at), _ints([0, t]),
                        _ints([t]), t, ws)
    if n > 1:
        cache.fork(_ints([0] * (n - 1)), _ints(range(1, n)), _ints([t] * (n - 1)))
    cache.check()
    return out, Samples(model, cache, 0, n, t)


def main():
    torch.manual_seed(0)
    model, n, tokens = Decoder(), 16, 777
    cache = PoolCache(model.attn, len(model.layers), n, 1024, pages=256)
    prompt = torch.randn(tokens, 1024, device="cuda").bfloat16()
    out, samples = sample(model, cache, prompt, n)
    last = out[-1:] + 0.1 * torch.randn(n, 1024, device="cuda").bfloat16()
    for i in range(20):
        last = samples.step(_norm(last)).clone()
    held = int((cache.refs > 0).sum())
    print(f"{n} samples of {samples.host_len} tokens: {held} pages of {int(cache.held.sum())} held")
    cache.release(_ints(range(1, n, 2)))
    print(f"half of them ended: {cache.compact()} pages in use")


if __name__ == "__main__":
    main()
